"""CUDA attention over the paged cache, rotary positions with the cache write, and sampling vs float64."""
import math

import numpy as np
import pytest
import torch

from tests import step_reference as R

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sv():
    import draft_verification_spec_gb300 as m
    m.lib()
    return m


def _batch(new, kv, page, hkv, d, dtype, seed, layout="nhd", junk=float("nan"), pad_cols=1):
    """Caches (every slot outside the requests' tokens holds `junk`), a page table with -1 beyond the used
    columns and a wider row stride, kv_lens, cu_q."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-k // page) for k in kv]
    pages = sum(used) + 2
    order = torch.randperm(pages, generator=g).tolist()
    width = max(1, max(used))
    table = torch.full((len(kv), width + pad_cols), -1, dtype=torch.int32)
    kc, vc = (torch.full((pages, page, hkv, d), junk, dtype=dtype) for _ in range(2))
    at = 0
    for b, k in enumerate(kv):
        for j in range(used[b]):
            table[b, j] = order[at]
            m = min(page, k - j * page)
            kc[order[at], :m] = torch.randn(m, hkv, d, generator=g).to(dtype)
            vc[order[at], :m] = torch.randn(m, hkv, d, generator=g).to(dtype)
            at += 1
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32)
    dev = "cuda"
    if layout == "hnd":   # [pages, heads, page_size, dim] in memory
        kc, vc = (t.permute(0, 2, 1, 3).contiguous().to(dev).permute(0, 2, 1, 3) for t in (kc, vc))
    else:
        kc, vc = kc.to(dev), vc.to(dev)
    return kc, vc, table.to(dev)[:, :width], torch.tensor(kv, dtype=torch.int32, device=dev), cu.to(dev)


def _attention(sv, new, kv, page, hq, hkv, d, dtype="bf16", causal=True, window=0, seed=0, layout="nhd", scale=None,
               strided_q=False, max_q=None):
    dt = DTYPES[dtype]
    kc, vc, table, lens, cu = _batch(new, kv, page, hkv, d, dt, seed, layout)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(sum(new), hq + (3 if strided_q else 0), d, generator=g) * 1.5).to(dt).cuda()
    if strided_q:
        q = q[:, 2:2 + hq]
    out, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, max(new) if max_q is None else max_q, causal=causal,
                                  window=window, scale=scale, want_lse=True)
    assert sv.default_workspace().status() == 0
    s = d ** -0.5 if scale is None else scale
    ro, rl, size, spread = R.attention(q, kc, vc, table, lens, cu, causal, window, s)
    bo, bl = R.attention_bounds(dt, size, spread, d)
    out, lse = out.cpu().double(), lse.cpu().double()
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert (out[empty] == 0).all()
    assert ((out - ro).abs() <= bo).all(), float(((out - ro).abs() / bo.clamp(min=1e-30)).max())
    # lse itself is rounded to fp32
    err = (lse - rl).abs()[~empty]
    assert (err <= (bl + rl.abs() * 2.0 ** -23)[~empty]).all(), float(err.max())
    return q, kc, vc, table, lens, cu


@pytest.mark.parametrize("d", [8, 64, 80, 128, 256])
@pytest.mark.parametrize("nq", [1, 5, 40])
def test_attention_head_sizes(sv, d, nq):
    _attention(sv, [nq, nq, nq], [nq, 70, 131], 16, 8, 2, d, seed=d + nq)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 128, 256])
@pytest.mark.parametrize("nq", [1, 17, 33])
def test_attention_page_sizes(sv, page, nq):
    """Pages that end inside a key tile, and a key tile that ends inside a page."""
    _attention(sv, [nq, nq], [200, 127], page, 16, 2, 64, seed=page)
    _attention(sv, [nq, nq], [300, 129], page, 16, 2, 128, seed=page, dtype="f16")


@pytest.mark.parametrize("G", [1, 2, 7, 8, 16, 40])
def test_attention_head_groups(sv, G):
    _attention(sv, [1, 3, 9], [33, 64, 65], 16, 2 * G, 2, 64, seed=G)


@pytest.mark.parametrize("kv", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_lengths(sv, kv, causal):
    _attention(sv, [1], [kv], 16, 4, 4, 64, causal=causal, seed=kv)
    _attention(sv, [kv], [kv], 32, 2, 1, 128, causal=causal, seed=kv)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 7, 64, 100])
def test_attention_window(sv, window, causal):
    _attention(sv, [1, 20, 150], [300, 300, 150], 16, 8, 2, 64, window=window, causal=causal, seed=window)
    _attention(sv, [1, 20, 150], [300, 300, 150], 16, 8, 2, 128, window=window, causal=causal, seed=window)


def test_attention_rows_without_keys(sv):
    """Idle slots (no cached token), requests shorter than their new tokens, requests without new tokens."""
    for d, hq in ((64, 4), (128, 32)):
        _attention(sv, [3, 0, 17, 1, 4, 0], [0, 5, 9, 1, 0, 0], 8, hq, 2, d, seed=d)
        _attention(sv, [4], [0], 16, hq, 2, d)
    _attention(sv, [0, 2], [10, 10], 16, 4, 2, 64)


def test_attention_many_requests_and_mixed(sv):
    rng = np.random.RandomState(3)
    kv = rng.randint(0, 90, 300).tolist()
    _attention(sv, [1] * 300, kv, 16, 2, 1, 64, seed=5)
    _attention(sv, [130, 1, 1, 2, 1], [200, 513, 1, 40, 64], 16, 8, 2, 128, seed=6)
    _attention(sv, [130, 1, 1, 2, 1], [200, 513, 1, 40, 64], 16, 8, 2, 64, seed=6, causal=False)


@pytest.mark.parametrize("nq", [1, 4, 17, 64])
def test_attention_long_split(sv, nq):
    """One request over a long cache: the key axis is split over many CTAs and joined."""
    _attention(sv, [nq], [5000], 16, 4, 1, 128, seed=nq)


def test_attention_layouts_strides_scale(sv):
    for nq in (2, 40):
        _attention(sv, [nq, nq], [77, 260], 16, 8, 4, 128, layout="hnd", seed=1)
        _attention(sv, [nq, nq], [77, 260], 16, 8, 4, 128, strided_q=True, seed=2)
        _attention(sv, [nq, nq], [77, 260], 16, 8, 4, 64, scale=0.01, seed=3)
        _attention(sv, [nq, nq], [77, 260], 16, 8, 4, 64, scale=-0.3, seed=4)


def test_attention_wrong_hint_changes_nothing(sv):
    """max_q only chooses the kernel: too small a bound still gives the rows."""
    _attention(sv, [50, 3], [90, 200], 16, 8, 2, 128, max_q=1)
    _attention(sv, [1, 3], [90, 200], 16, 8, 2, 128, max_q=500)


def test_attention_growing_scores(sv):
    """Scores that rise along the keys (the running maximum moves at every tile), by far more than fp16 holds."""
    for nq in (1, 40):
        dt = torch.bfloat16
        kc, vc, table, lens, cu = _batch([nq], [400], 16, 1, 64, dt, 9)
        ramp = torch.linspace(0.0, 30.0, 400)
        for t in range(400):
            kc[int(table[0, t // 16]), t % 16] *= float(ramp[t])
        q = torch.randn(nq, 2, 64, generator=torch.Generator().manual_seed(1)).to(dt).cuda()
        out, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, want_lse=True)
        ro, rl, size, spread = R.attention(q, kc, vc, table, lens, cu, True, 0, 64 ** -0.5)
        bo, bl = R.attention_bounds(dt, size, spread, 64)
        assert ((out.cpu().double() - ro).abs() <= bo).all()
        assert ((lse.cpu().double() - rl).abs() <= bl + rl.abs() * 2.0 ** -23).all()


def test_attention_repeats_bit_for_bit(sv):
    q, kc, vc, table, lens, cu = _attention(sv, [2, 40], [900, 700], 16, 8, 2, 128)
    a = sv.chunk_attention(q, kc, vc, table, lens, cu, 40)
    for _ in range(3):
        assert torch.equal(a, sv.chunk_attention(q, kc, vc, table, lens, cu, 40))


def test_attention_side_stream_and_graph(sv):
    q, kc, vc, table, lens, cu = _attention(sv, [17, 17], [300, 200], 16, 16, 2, 128)
    want = sv.chunk_attention(q, kc, vc, table, lens, cu, 17)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.chunk_attention(q, kc, vc, table, lens, cu, 17, stream=s)
    s.synchronize()
    assert torch.equal(want, got)
    ws = sv.Workspace()
    out = torch.empty_like(want)
    sv.chunk_attention(q, kc, vc, table, lens, cu, 17, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.chunk_attention(q, kc, vc, table, lens, cu, 17, out=out, workspace=ws)
    lens.copy_(torch.tensor([130, 190], dtype=torch.int32))   # lengths are read when the graph runs
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, sv.chunk_attention(q, kc, vc, table, lens, cu, 17))


def test_attention_page_range_status(sv):
    """A page id outside the cache reads as zeros and is reported."""
    for nq in (1, 40):
        kc, vc, table, lens, cu = _batch([nq], [80], 16, 2, 64, torch.bfloat16, 4)
        q = torch.randn(nq, 4, 64).to(torch.bfloat16).cuda()
        bad = table.clone()
        bad[0, 2] = kc.shape[0] + 5
        got = sv.chunk_attention(q, kc, vc, bad, lens, cu, nq)
        assert sv.default_workspace().status() == 7
        assert sv.default_workspace().status() == 0
        zk, zv = kc.clone(), vc.clone()
        zk[table[0, 2].long()] = 0
        zv[table[0, 2].long()] = 0
        assert torch.equal(got, sv.chunk_attention(q, zk, zv, table, lens, cu, nq))


@pytest.mark.parametrize("nq", [1, 17])
def test_attention_and_rope_far_pages(sv, nq):
    """A cache of more than 2^31 values: page offsets pass 32 bits."""
    dt, page, hkv, d = torch.bfloat16, 16, 8, 128
    pages = 2 ** 31 // (page * hkv * d) + 64
    kc, vc = (torch.empty(pages, page, hkv, d, dtype=dt, device="cuda") for _ in range(2))
    ids = torch.tensor([[pages - 1, 3, pages - 7, pages // 2 + 1]], dtype=torch.int32, device="cuda")
    small_k, small_v = (torch.randn(4, page, hkv, d, device="cuda").to(dt) for _ in range(2))
    kc[ids[0].long()], vc[ids[0].long()] = small_k, small_v
    near = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    lens, cu = torch.tensor([60], dtype=torch.int32, device="cuda"), torch.tensor([0, nq], dtype=torch.int32, device="cuda")
    q = torch.randn(nq, 16, d, device="cuda").to(dt)
    got = sv.chunk_attention(q, kc, vc, ids, lens, cu, nq)
    assert torch.equal(got, sv.chunk_attention(q, small_k, small_v, near, lens, cu, nq))
    plan, k = sv.RopePlan(d), torch.randn(nq, hkv, d, device="cuda").to(dt)
    sv.rope_append(q, k, k, plan, kc, vc, ids, lens, cu)
    sv.rope_append(q, k, k, plan, small_k, small_v, near, lens, cu)
    assert torch.equal(kc[ids[0].long()], small_k) and torch.equal(vc[ids[0].long()], small_v)
    assert sv.default_workspace().status() == 0


def test_attention_refusals(sv):
    kc, vc, table, lens, cu = _batch([2], [20], 16, 2, 64, torch.bfloat16, 4)
    q = torch.randn(2, 4, 64).to(torch.bfloat16).cuda()
    bad = [
        (TypeError, dict(q=q.float())), (TypeError, dict(q=q.half())), (ValueError, dict(q=q[0])),
        (ValueError, dict(k=kc[0])), (ValueError, dict(v=vc[:, :8])), (TypeError, dict(table=table.long())),
        (TypeError, dict(lens=lens.float())), (ValueError, dict(cu=cu[:1])), (ValueError, dict(q=q.cpu())),
        (sv.SpecError, dict(q=q[:, :3])), (ValueError, dict(out=torch.empty(1, 4, 64, device="cuda"))),
        (sv.SpecError, dict(window=-1)), (sv.SpecError, dict(scale=math.nan)), (sv.SpecError, dict(max_q=-1)),
    ]
    for err, change in bad:
        a = dict(q=q, k=kc, v=vc, table=table, lens=lens, cu=cu, max_q=2)
        kw = {n: change.pop(n) for n in ("out", "window", "scale") if n in change}
        a.update(change)
        with pytest.raises(err):
            sv.chunk_attention(a["q"], a["k"], a["v"], a["table"], a["lens"], a["cu"], a["max_q"], **kw)
    k7 = torch.zeros(2, 16, 2, 12, dtype=torch.bfloat16, device="cuda")     # 12 is no multiple of 8
    with pytest.raises(sv.SpecError):
        sv.chunk_attention(torch.zeros(2, 4, 12, dtype=torch.bfloat16, device="cuda"), k7, k7, table, lens, cu, 2)
    with pytest.raises(sv.SpecError):                                        # a base that is not 16-byte aligned
        flat = torch.zeros(2 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:1 + 2 * 4 * 64].view(2, 4, 64)
        sv.chunk_attention(flat, kc, vc, table, lens, cu, 2)


# ------------------------------------------------------------------------------------------- rope

def _rope(sv, new, kv, page, hq, hkv, d, dtype="bf16", rotary=None, layout="half", scaling=None, theta=10000.0, seed=0,
          k_out=False, first_page=None):
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    n = sum(new)
    q, k, v = (torch.randn(n, h, d, generator=g).to(dt).cuda() for h in (hq, hkv, hkv))
    first = [max(0, (L - m) // page) for m, L in zip(new, kv)]     # pages before the new tokens are not touched
    used = [max(0, -(-L // page) - f) for L, f in zip(kv, first)]
    pages = sum(used) + 2
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(kv), max(1, max(u + f for u, f in zip(used, first)))), -1, dtype=torch.int32)
    at = 0
    for b in range(len(kv)):
        for j in range(used[b]):
            table[b, first[b] + j] = order[at]
            at += 1
    kc, vc = (torch.full((pages, page, hkv, d), 7.0, dtype=dt, device="cuda") for _ in range(2))
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    plan = sv.RopePlan(d, rotary_dim=rotary, theta=theta, layout=layout, scaling=scaling)
    ko = torch.empty_like(k) if k_out else None
    qo = sv.rope_append(q, k, v, plan, kc, vc, table.cuda(), lens, cu, k_out=ko)
    assert sv.default_workspace().status() == 0
    eps = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    want_k, want_v = (torch.full((pages, page, hkv, d), 7.0, dtype=torch.float64) for _ in range(2))
    r = plan.rotary_dim

    def check(got, x, pos):
        ref = R.rope(x.cpu().double(), pos, plan.frequencies, plan.factor, r, layout)
        # half a unit of the output's type; cos, sin and three operations in fp32, 2^-22 of |x| + |y| in all;
        # the frequency's 2^-65 of a turn and the phase's 2^-32
        size = torch.zeros_like(ref)
        for j in range(r // 2):
            a, b = (2 * j, 2 * j + 1) if layout == "interleaved" else (j, j + r // 2)
            size[:, a] = size[:, b] = (x[:, a].abs() + x[:, b].abs()).cpu().double() * plan.factor
        assert ((got.cpu().double() - ref).abs() <= eps * ref.abs() + size * 2.0 ** -22 * (1 + eps) + tiny).all()
        assert torch.equal(got.cpu()[:, r:], x.cpu()[:, r:])
        return ref

    for b in range(len(kv)):
        for i, pos in enumerate(R.positions(cu.tolist(), kv, b)):
            t = cu.tolist()[b] + i
            check(qo[t], q[t], pos)
            if ko is not None:
                check(ko[t], k[t], pos)
            if pos >= 0:
                pg, s = int(table[b, pos // page]), pos % page
                check(kc[pg, s], k[t], pos)
                want_k[pg, s] = kc[pg, s].cpu().double()
                want_v[pg, s] = v[t].cpu().double()
    assert torch.equal(kc.cpu().double(), want_k)          # nothing else was written
    assert torch.equal(vc.cpu().double(), want_v)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (128, 64), (80, 80), (80, 20), (128, 2), (256, 256), (24, 10)])
def test_rope_layouts(sv, layout, dtype, d, rotary):
    _rope(sv, [1, 3, 5], [1, 20, 40], 16, 4, 2, d, dtype=dtype, rotary=rotary, layout=layout, seed=d + rotary)


@pytest.mark.parametrize("scaling", [None, {"type": "linear", "factor": 4.0}, {"type": "ntk", "factor": 8.0},
                                     {"type": "yarn", "factor": 16.0, "original": 4096}])
@pytest.mark.parametrize("pos", [100, 131071, 1000003])
def test_rope_far_positions(sv, scaling, pos):
    """fp32 outputs stay exact to fp32 where a position x frequency in fp32 would be off by up to 0.03 radians."""
    _rope(sv, [2, 1], [pos, pos + 7], 64, 2, 1, 64, dtype="f32", scaling=scaling, theta=500000.0)


@pytest.mark.parametrize("page", [1, 5, 16, 128])
def test_rope_pages_groups_idle(sv, page):
    _rope(sv, [4, 0, 17, 1, 3], [0, 5, 9, 1, 700], page, 7, 1, 64, k_out=True)
    _rope(sv, [1] * 70, list(range(1, 71)), page, 2, 2, 64)


def test_rope_in_place_strided_and_uncached(sv):
    dt = torch.bfloat16
    qkv = torch.randn(9, 8 + 2 + 2, 64).to(dt).cuda()               # one projection's output
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    lens, cu = torch.tensor([50], dtype=torch.int32, device="cuda"), torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    plan = sv.RopePlan(64)
    ko = torch.empty(9, 2, 64, dtype=dt, device="cuda")
    want = sv.rope_append(q.contiguous(), k.contiguous(), None, plan, None, None, None, lens, cu, k_out=ko)
    sv.rope_append(q, k, None, plan, None, None, None, lens, cu, q_out=q, k_out=k)
    assert torch.equal(q, want) and torch.equal(k, ko)
    odd = torch.randn(9 * 2 * 64 + 1, device="cuda").to(dt)[1:].view(9, 2, 64)      # 2-byte aligned rows
    a, b = torch.empty_like(k).contiguous(), torch.empty(9, 2, 64, dtype=dt, device="cuda")
    sv.rope_append(odd, odd, None, plan, None, None, None, lens, cu, q_out=a, k_out=b)
    c = sv.rope_append(odd.clone(), odd.clone(), None, plan, None, None, None, lens, cu, k_out=b)
    assert torch.equal(a, c) and torch.equal(a, b)


def test_rope_page_range_status_and_refusals(sv):
    dt = torch.bfloat16
    q, k = torch.randn(2, 4, 64).to(dt).cuda(), torch.randn(2, 2, 64).to(dt).cuda()
    kc, vc = torch.zeros(3, 16, 2, 64, dtype=dt, device="cuda"), torch.zeros(3, 16, 2, 64, dtype=dt, device="cuda")
    table = torch.tensor([[0, 9]], dtype=torch.int32, device="cuda")
    lens, cu = torch.tensor([18], dtype=torch.int32, device="cuda"), torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    plan = sv.RopePlan(64)
    sv.rope_append(q, k, k, plan, kc, vc, table, lens, cu)
    assert sv.default_workspace().status() == 7
    assert not kc.any() and not vc.any()
    lens.fill_(40)                                                  # beyond the table
    sv.rope_append(q, k, k, plan, kc, vc, table, lens, cu)
    assert sv.default_workspace().status() == 7
    for err, f in ((TypeError, lambda: sv.rope_append(q, k.float(), k, plan, kc, vc, table, lens, cu)),
                   (TypeError, lambda: sv.rope_append(q.double(), k, k, plan, kc, vc, table, lens, cu)),
                   (ValueError, lambda: sv.rope_append(q, k, k, sv.RopePlan(128), kc, vc, table, lens, cu)),
                   (ValueError, lambda: sv.rope_append(q, k, k, plan, None, None, None, lens, cu)),
                   (ValueError, lambda: sv.rope_append(q, k[:1], k, plan, kc, vc, table, lens, cu)),
                   (ValueError, lambda: sv.RopePlan(64, rotary_dim=7)), (ValueError, lambda: sv.RopePlan(64, layout="x")),
                   (ValueError, lambda: sv.RopePlan(64, scaling={"type": "y", "factor": 2.0}))):
        with pytest.raises(err):
            f()


# ------------------------------------------------------------------------------------------- sampling

def _check_sample(sv, logits, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    rows, V = logits.shape
    out = sv.sample_tokens(logits, u, T, top_k, top_p, min_p, want_filtered=True)
    z, uu = logits.float().cpu().numpy(), u.cpu().numpy()
    at = lambda v, i: v[i].item() if isinstance(v, torch.Tensor) else v  # noqa: E731
    tok, prob, kept, filt = out.tokens.cpu().numpy(), out.probs.cpu().numpy(), out.kept.cpu().numpy(), out.filtered
    assert filt.dtype == logits.dtype
    bits = torch.int16 if logits.dtype == torch.bfloat16 else torch.int32
    fb, lb = filt.cpu().view(bits).numpy(), logits.cpu().contiguous().view(bits).numpy()
    low = torch.tensor([-math.inf], dtype=logits.dtype).view(bits).item()
    for r in range(rows):
        t, p, n, keep = R.sample(z[r], uu[r], at(T, r), at(top_k, r), at(top_p, r), at(min_p, r))
        assert (tok[r], kept[r]) == (t, n), (r, V)
        assert abs(prob[r] - p) <= 2.0 ** -23 * p
        want = np.full(V, low, dtype=fb.dtype)
        want[keep] = lb[r, keep]
        np.testing.assert_array_equal(fb[r], want)
    only = sv.sample_tokens(logits, u, T, top_k, top_p, min_p)     # the same without the filtered row
    assert only.filtered is None
    assert torch.equal(only.tokens, out.tokens) and torch.equal(only.probs, out.probs) and torch.equal(only.kept, out.kept)
    return out


def _logits(rows, V, dtype, seed, scale=3.0, zipf=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, V, generator=g) * (0.5 if zipf else scale)
    if zipf:
        z -= 1.1 * torch.log1p(torch.rand(rows, V, generator=g) * V)
    return z.to(DTYPES[dtype]).cuda(), torch.rand(rows, generator=g).cuda()


SETTINGS = [dict(), dict(T=0.0), dict(T=0.6), dict(T=1.4), dict(top_k=1), dict(top_k=17), dict(top_p=0.9), dict(top_p=0.3),
            dict(top_p=0.0), dict(min_p=0.05), dict(min_p=1.0), dict(min_p=2.0), dict(top_k=50, top_p=0.8),
            dict(T=0.8, top_k=400, top_p=0.95, min_p=0.01), dict(top_k=10 ** 9, top_p=1.5, min_p=-1.0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 1024, 4097, 50000])
def test_sample_settings(sv, dtype, V):
    for i, s in enumerate(SETTINGS):
        z, u = _logits(3, V, dtype, seed=V + i, zipf=i % 2 == 1)
        _check_sample(sv, z, u, **s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [128000, 131071, 262144])
def test_sample_large_vocabulary(sv, dtype, V):
    z, u = _logits(4, V, dtype, seed=V, zipf=True)
    for s in (dict(T=0.9, top_p=0.95), dict(), dict(T=0.7, top_k=50, min_p=0.02)):
        _check_sample(sv, z, u, **s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_settings_per_row(sv, dtype):
    rows = 40
    z, u = _logits(rows, 3001, dtype, seed=2)
    g = torch.Generator().manual_seed(5)
    pick = lambda v, dt: torch.tensor(v, dtype=dt)[torch.randint(len(v), (rows,), generator=g)].cuda()  # noqa: E731
    _check_sample(sv, z, u, pick([0.0, 0.5, 1.0, 1.5], torch.float32), pick([0, 1, 20, 5000], torch.int32),
                  pick([1.0, 0.9, 0.5], torch.float32), pick([0.0, 0.1], torch.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_ties_zeros_infinities(sv, dtype):
    """Equal logits go by index (-0 equals 0); -inf and NaN are never drawn; +inf takes all."""
    dt, V, inf, nan = DTYPES[dtype], 600, math.inf, math.nan
    z = torch.zeros(9, V)
    z[1, ::2] = -0.0
    z[2] = -inf
    z[3] = -inf
    z[3, 77] = -5.0
    z[4, 100:] = -inf
    z[5, ::3] = nan
    z[6, 10] = z[6, 400] = inf
    z[7] = nan
    z[8] = torch.arange(V) // 100 * 1.0
    u = torch.tensor([0.5, 0.999, 0.5, 0.999, 0.9999999, 0.3, 0.7, 0.1, 0.0]).cuda()
    for s in (dict(), dict(top_k=7), dict(top_p=0.5), dict(T=0.0), dict(min_p=0.5), dict(top_k=300, top_p=0.7)):
        _check_sample(sv, z.to(dt).cuda(), u, **s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_logits_of_any_size(sv, dtype):
    """Masks of -1e9 and of the type's lowest value, logits in the hundreds and thousands, and vanishing ones."""
    dt, V = DTYPES[dtype], 3000
    g = torch.Generator().manual_seed(21)
    z = torch.randn(8, V, generator=g) * 3.0
    low = torch.finfo(dt).min
    z[0, 100:] = -1e9
    z[1, 5:] = low
    z[2, ::2] = -300.0 - torch.arange(V // 2) % 50
    z[3] = z[3] * 400.0
    z[4, ::7] = torch.randn(len(z[4, ::7]), generator=g) * 1e-20
    z[5] = -500.0 + z[5]
    z[6] = low
    z[6, 9] = -1e30
    z[7] = z[7] * 1e-18
    z, u = z.to(dt).cuda(), torch.rand(8, generator=g).cuda()
    for s in SETTINGS + [dict(top_k=2000), dict(top_k=2999, top_p=0.99), dict(T=100.0, top_p=0.9), dict(T=1e4, top_k=1700)]:
        _check_sample(sv, z, u, **s)


def test_sample_crowded_bins(sv):
    """fp32 logits of which thousands share their 16 top bits."""
    z = 3.0 + torch.rand(3, 40000, generator=torch.Generator().manual_seed(2)) * 0.01
    z[2, 10000:] = -7.0
    u = torch.rand(3, generator=torch.Generator().manual_seed(3)).cuda()
    for s in (dict(), dict(top_k=777, top_p=0.9), dict(top_p=0.4), dict(min_p=0.997)):
        _check_sample(sv, z.cuda(), u, **s)


def test_sample_far_rows(sv):
    """Rows that lie more than 2^31 values apart, in the logits and in the filtered output."""
    V, far = 3001, 2 ** 31 + 8
    store = torch.zeros(far + V, dtype=torch.bfloat16, device="cuda")
    z = store.as_strided((2, V), (far, 1))
    z[0], z[1] = torch.randn(2, V, device="cuda").to(torch.bfloat16)
    keep = torch.empty_like(store).as_strided((2, V), (far, 1))
    u = torch.rand(2, device="cuda")
    want = sv.sample_tokens(z.contiguous(), u, 0.8, 40, want_filtered=True)
    out = sv.SampleOutput(torch.empty_like(want.tokens), torch.empty_like(want.probs), torch.empty_like(want.kept), keep)
    sv.sample_tokens(z, u, 0.8, 40, out=out)
    assert torch.equal(out.tokens, want.tokens) and torch.equal(out.kept, want.kept)
    assert torch.equal(out.filtered.contiguous(), want.filtered)


def test_sample_uniform_ends(sv):
    """u = 0 takes the most likely token; the largest u below 1 (and 1, and beyond) a kept one."""
    z, _ = _logits(6, 5000, "f32", seed=8)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan]).cuda()
    out = sv.sample_tokens(z, u, 1.0, 30)
    top = torch.sort(z, dim=1, descending=True).indices
    assert torch.equal(out.tokens[[0, 4, 5]].long(), top[[0, 4, 5], 0])
    assert torch.equal(out.tokens[1:4].long(), top[1:4, 29])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_strided_rows_and_distribution(sv, dtype):
    """Rows of a [B, K + 1, V] tensor without its last position; an odd vocabulary leaves rows unaligned."""
    dt = DTYPES[dtype]
    z = torch.randn(3, 5, 1001).to(dt).cuda()
    u = torch.rand(3).cuda()
    view = z[:, 2]
    assert not view.is_contiguous()
    _check_sample(sv, view, u, T=0.9, top_p=0.9)
    # the drawn tokens follow the weights: a row's frequencies over 20000 even uniforms
    row = torch.randn(1, 12, generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    n = 20000
    uu = ((torch.arange(n) + 0.5) / n).cuda()
    got = torch.bincount(sv.sample_tokens(row.expand(n, 12).contiguous(), uu).tokens.long(), minlength=12).cpu() / n
    np.testing.assert_allclose(got.numpy(), torch.softmax(row[0].double().cpu(), 0).numpy(), atol=1.5 / n)


def test_sample_filtered_feeds_the_verification(sv):
    """The filtered logits of draft and target give the acceptance test of the truncated distributions."""
    B, K, V = 4, 3, 2000
    g = torch.Generator().manual_seed(11)
    zt = torch.randn(B, K + 1, V, generator=g).mul(3.0)
    zd = zt[:, :K] + 0.7 * torch.randn(B, K, V, generator=g)
    zt, zd = zt.to(torch.bfloat16).cuda(), zd.to(torch.bfloat16).cuda()
    u = torch.rand(B * K, generator=g).cuda()
    d = sv.sample_tokens(zd.view(-1, V), u, 0.9, 40, 0.95, want_filtered=True)
    t = sv.sample_tokens(zt.view(-1, V), torch.rand(B * (K + 1)).cuda(), 0.9, 40, 0.95, want_filtered=True)
    x = d.tokens.view(B, K)
    out = sv.verify_chain(t.filtered.view(B, K + 1, V), d.filtered.view(B, K, V), x, torch.rand(B, K + 1).cuda(), 0.9,
                          want_alpha=True)
    p = torch.softmax(t.filtered.view(B, K + 1, V)[:, :K].double() / 0.9, -1)
    q = torch.softmax(d.filtered.view(B, K, V).double() / 0.9, -1)
    assert torch.allclose(out.alpha.double(), torch.minimum(p, q).sum(-1), atol=1e-5)
    assert torch.allclose(q.gather(2, x.long()[..., None])[..., 0], d.probs.view(B, K).double(), rtol=1e-5)
    assert int(out.accepted.min()) >= 0


def test_sample_refusals(sv):
    z, u = _logits(2, 100, "f32", 1)
    for err, f in ((TypeError, lambda: sv.sample_tokens(z.half(), u)), (ValueError, lambda: sv.sample_tokens(z[0], u)),
                   (ValueError, lambda: sv.sample_tokens(z, u[:1])), (ValueError, lambda: sv.sample_tokens(z, u.double())),
                   (ValueError, lambda: sv.sample_tokens(z.t(), u)), (ValueError, lambda: sv.sample_tokens(z[:1].expand(2, 100), u)),
                   (ValueError, lambda: sv.sample_tokens(z, u, temperature=u[:1])),
                   (ValueError, lambda: sv.sample_tokens(z, u, top_k=u)), (ValueError, lambda: sv.sample_tokens(z.cpu(), u)),
                   (sv.SpecError, lambda: sv.sample_tokens(z, u, -1.0)), (sv.SpecError, lambda: sv.sample_tokens(z, u, math.nan)),
                   (sv.SpecError, lambda: sv.sample_tokens(torch.zeros(1, 262145, device="cuda"), u[:1]))):
        with pytest.raises(err):
            f()
    assert sv.sample_tokens(z[:0], u[:0]).tokens.shape == (0,)
