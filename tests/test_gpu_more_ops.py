"""CUDA attention with first tokens kept behind a window and over caches in 4 bits, and the write into those, vs float64."""
import math

import pytest
import torch

from tests import more_reference as M
from tests import step_reference as R
from tests.test_gpu_step_ops import DTYPES, _batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import draft_verification_spec_gb300 as m
    m.lib()
    return m


def _check(got, lse, ref, dtype, keys, d, bits):
    ro, rl, size, spread, reach, top = ref
    bo, bl = M.bounds(dtype, size, spread, reach, top, keys, d, bits)
    out, lse = got.cpu().double(), lse.cpu().double()
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert (out[empty] == 0).all()
    assert ((out - ro).abs() <= bo).all(), float(((out - ro).abs() / bo.clamp(min=1e-30)).max())
    err = (lse - rl).abs()[~empty]
    assert (err <= (bl + rl.abs() * 2.0 ** -23)[~empty]).all(), float(err.max())


# ------------------------------------------------------------------------------ first tokens kept

def _sinks(sv, new, kv, page, hq, hkv, d, window, sinks, dtype="bf16", causal=True, seed=0, layout="nhd"):
    dt = DTYPES[dtype]
    kc, vc, table, lens, cu = _batch(new, kv, page, hkv, d, dt, seed, layout)
    q = (torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(seed + 1)) * 1.5).to(dt).cuda()
    n = max(new)
    got, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, n, causal=causal, window=window, sinks=sinks, want_lse=True)
    assert sv.default_workspace().status() == 0
    ref = M.attention(q, kc.cpu().double(), vc.cpu().double(), table, lens, cu, causal, window, sinks, d ** -0.5)
    _check(got, lse, ref, dt, max(kv), d, 16)
    # pages behind the window that hold no first token may be gone, or hold anything
    gone = table.clone()
    for b, k in enumerate(kv):
        behind = max(0, k - new[b] - window + 1) // page
        gone[b, -(-sinks // page):behind] = -1
    again, lse2 = sv.chunk_attention(q, kc, vc, gone, lens, cu, n, causal=causal, window=window, sinks=sinks, want_lse=True)
    assert sv.default_workspace().status() == 0
    assert torch.equal(got, again) and torch.equal(lse, lse2)
    return q, kc, vc, table, lens, cu, got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sinks", [1, 4, 64, 130, 1000])
@pytest.mark.parametrize("window", [1, 40, 200])
def test_sinks_and_windows(sv, window, sinks, causal):
    _sinks(sv, [1, 9, 1, 3], [700, 640, 30, 0], 16, 8, 2, 64, window, sinks, causal=causal, seed=window)
    _sinks(sv, [150, 1], [640, 300], 16, 4, 2, 128, window, sinks, causal=causal, seed=sinks)


@pytest.mark.parametrize("page", [1, 7, 16, 128, 256])
@pytest.mark.parametrize("nq,hq,d", [(1, 8, 128), (4, 4, 64), (40, 4, 256), (17, 8, 80), (70, 8, 64), (140, 2, 128)])
def test_sinks_pages_and_kernels(sv, nq, hq, d, page):
    _sinks(sv, [nq, nq], [nq + 500, nq + 90], page, hq, 2, d, 100, 6, seed=nq + page, dtype="f16" if page == 7 else "bf16")


def test_sinks_of_no_consequence(sv):
    """Without a window, or with one that hides nothing, first tokens change no bit; more of them than keys neither."""
    for nq in (1, 40):
        kc, vc, table, lens, cu = _batch([nq] * 2, [300, 190], 16, 2, 128, torch.bfloat16, 3)
        q = torch.randn(2 * nq, 8, 128).to(torch.bfloat16).cuda()
        call = lambda **kw: sv.chunk_attention(q, kc, vc, table, lens, cu, nq, **kw)  # noqa: E731
        want = call()
        assert torch.equal(want, call(sinks=5)) and torch.equal(want, call(window=400, sinks=5))
        assert torch.equal(want, call(window=2 ** 31 - 1, sinks=2 ** 40))
        assert torch.allclose(want.float(), call(window=3, sinks=2 ** 31 - 1).float(), atol=2.0 ** -6)
        with pytest.raises(sv.SpecError):
            call(window=3, sinks=-1)
        with pytest.raises(sv.SpecError):
            call(sinks=-2 ** 40)


def test_sinks_length_beyond_the_table_and_bad_pages(sv):
    """Positions count from the length: the window's begin lies behind the table's last key, the first tokens are seen."""
    dt, page, cols, d = torch.bfloat16, 16, 5, 64
    for nq, hq in ((1, 4), (30, 4)):
        kc, vc, table, lens, cu = _batch([nq], [page * cols], page, 2, d, dt, 8)
        q = torch.randn(nq, hq, d).to(dt).cuda()
        far = torch.tensor([page * cols + 500], dtype=torch.int32, device="cuda")
        got, lse = sv.chunk_attention(q, kc, vc, table[:, :cols], far, cu, nq, window=10, sinks=20, want_lse=True)
        assert sv.default_workspace().status() == 7
        short = torch.tensor([20], dtype=torch.int32, device="cuda")
        want, lse2 = sv.chunk_attention(q, kc, vc, table, short, cu, nq, causal=False, want_lse=True)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
        assert (lse - lse2).abs().max() < 1e-4
        bad = table.clone()
        bad[0, 0] = kc.shape[0]
        sv.chunk_attention(q, kc, vc, bad, lens, cu, nq, window=10, sinks=20)
        assert sv.default_workspace().status() == 7 and sv.default_workspace().status() == 0


def test_sinks_repeat_graph_and_stream(sv):
    for nq in (1, 60):
        q, kc, vc, table, lens, cu, want = _sinks(sv, [nq, nq], [3000, 700], 16, 8, 2, 128, 900, 30)
        ws, out = sv.Workspace(), torch.empty_like(want)
        call = lambda **kw: sv.chunk_attention(q, kc, vc, table, lens, cu, nq, window=900, sinks=30, **kw)  # noqa: E731
        call(out=out, workspace=ws)
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out=out, workspace=ws)
        lens.copy_(torch.tensor([2500, 699], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()) and ws.status() == 0
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        side.synchronize()
        assert torch.equal(got, out)


# ------------------------------------------------------------------------------- caches in 4 bits

def _fp4_batch(sv, new, kv, page, hkv, d, seed, layout="hnd", units=(1.0, 1.0)):
    """Caches whose slots outside the requests' tokens hold codes of anything and the scale NaN."""
    g = torch.Generator().manual_seed(seed)
    _, _, table, lens, cu = _batch(new, kv, page, 1, 8, torch.bfloat16, seed)
    pages = sum(-(-k // page) for k in kv) + 2
    seen = torch.zeros(pages, page, dtype=torch.bool)
    for b, k in enumerate(kv):
        for j in range(-(-k // page)):
            seen[table[b, j].item(), : min(page, k - j * page)] = True
    caches, exact = [], []
    for unit in units:
        codes = torch.randint(0, 256, (pages, page, hkv, d // 2), generator=g, dtype=torch.uint8)
        scales = torch.randint(40, 64, (pages, page, hkv, d // 16), generator=g, dtype=torch.uint8)   # 1/16 to 1/2
        scales[~seen] = 127
        exact.append(torch.nan_to_num(M.values(codes, scales, unit)))
        if layout == "hnd":
            codes, scales = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (codes, scales))
        caches.append(sv.FP4Cache.of(codes.cuda(), scales.cuda().view(torch.float8_e4m3fn), unit))
    return caches, exact, table, lens, cu


def _fp4(sv, new, kv, page, hq, hkv, d, dtype="bf16", causal=True, window=0, sinks=0, seed=0, layout="hnd", scale=None,
         units=(1.0, 1.0), max_q=None, grow=1.0):
    dt = DTYPES[dtype]
    (kc, vc), (ke, ve), table, lens, cu = _fp4_batch(sv, new, kv, page, hkv, d, seed, layout, units)
    q = (torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(seed + 1)) * grow / units[0]).to(dt).cuda()
    got, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, max(new) if max_q is None else max_q, causal=causal, window=window,
                                  sinks=sinks, scale=scale, want_lse=True)
    assert sv.default_workspace().status() == 0
    ref = M.attention(q, ke, ve, table, lens, cu, causal, window, sinks, d ** -0.5 if scale is None else scale)
    _check(got, lse, ref, dt, max(kv), d, 4)
    return q, kc, vc, table, lens, cu, got


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("nq", [1, 5, 40])
def test_fp4_head_sizes(sv, d, nq, dtype, layout):
    _fp4(sv, [nq, nq, nq], [nq, 70, 131], 16, 8, 2, d, dtype=dtype, seed=d + nq, layout=layout)


@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 256])
@pytest.mark.parametrize("nq", [1, 17, 33])
def test_fp4_page_sizes(sv, page, nq):
    _fp4(sv, [nq, nq], [200, 127], page, 16, 2, 64, seed=page)
    _fp4(sv, [nq, nq], [300, 129], page, 16, 2, 128, seed=page, dtype="f16")


@pytest.mark.parametrize("G", [1, 2, 7, 8, 16, 40])
def test_fp4_head_groups(sv, G):
    _fp4(sv, [1, 3, 9], [33, 64, 65], 16, 2 * G, 2, 64, seed=G)


@pytest.mark.parametrize("kv", [1, 31, 32, 33, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("causal", [True, False])
def test_fp4_lengths(sv, kv, causal):
    _fp4(sv, [1], [kv], 16, 4, 4, 64, causal=causal, seed=kv)
    _fp4(sv, [kv], [kv], 32, 2, 1, 128, causal=causal, seed=kv)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (64, 40), (100, 200), (300, 1)])
def test_fp4_windows_and_sinks(sv, window, sinks, causal):
    _fp4(sv, [1, 20, 150], [500, 300, 150], 16, 8, 2, 64, window=window, sinks=sinks, causal=causal, seed=window)
    _fp4(sv, [1, 20, 150], [500, 300, 150], 16, 4, 2, 128, window=window, sinks=sinks, causal=causal, seed=window)


def test_fp4_rows_without_keys(sv):
    for d, hq in ((64, 4), (128, 32), (256, 4)):
        _fp4(sv, [3, 0, 17, 1, 4, 0], [0, 5, 9, 1, 0, 0], 8, hq, 2, d, seed=d)
        _fp4(sv, [4], [0], 16, hq, 2, d)


def test_fp4_many_requests_split_and_hints(sv):
    kv = torch.randint(0, 90, (300,), generator=torch.Generator().manual_seed(3)).tolist()
    _fp4(sv, [1] * 300, kv, 16, 2, 1, 64, seed=5)
    _fp4(sv, [130, 1, 1, 2, 1], [200, 513, 1, 40, 64], 16, 8, 2, 128, seed=6)
    for nq in (1, 4, 17):
        _fp4(sv, [nq], [5000], 16, 4, 1, 128, seed=nq)
    _fp4(sv, [50, 3], [90, 200], 16, 8, 2, 128, max_q=1)
    _fp4(sv, [1, 3], [90, 200], 16, 8, 2, 128, max_q=500)


@pytest.mark.parametrize("nq", [2, 40])
def test_fp4_units_and_scales(sv, nq):
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 128, units=(2.0 ** -10, 2.0 ** 7), seed=1)
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 128, units=(2.0 ** 20, 2.0 ** -20), seed=2)
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 64, scale=-0.3, seed=4)
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 64, grow=30.0, seed=5)      # scores whose maximum keeps moving


@pytest.mark.parametrize("nq", [1, 4, 40])
def test_fp4_strides_of_all_kinds(sv, nq):
    """Keys and values, codes and scales laid out apart, heads that are every second one of a wider cache, rows of scales at odd
    places: the same rows as from caches of the usual layout, to rounding."""
    new, kv, page, hkv, d = [nq, nq], [300, 77], 16, 2, 128
    (kc, vc), (ke, ve), table, lens, cu = _fp4_batch(sv, new, kv, page, hkv, d, 21)
    q = torch.randn(2 * nq, 8, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    ref = M.attention(q, ke, ve, table, lens, cu, True, 0, 0, d ** -0.5)
    byte = lambda c: c.scales.view(torch.uint8)  # noqa: E731
    nhd = lambda c: sv.FP4Cache.of(c.codes.contiguous(), byte(c).contiguous().view(torch.float8_e4m3fn))  # noqa: E731

    def wide(c):
        codes = torch.full((*c.shape[:2], 2 * hkv, d // 2), 0x77, dtype=torch.uint8, device="cuda")
        scales = torch.full((*c.shape[:2], 2 * hkv, d // 16), 127, dtype=torch.uint8, device="cuda")
        codes[:, :, ::2], scales[:, :, ::2] = c.codes, byte(c)
        return sv.FP4Cache.of(codes[:, :, ::2], scales.view(torch.float8_e4m3fn)[:, :, ::2])

    def odd(c):
        scales = torch.full((*c.shape[:2], hkv, d // 16 + 3), 127, dtype=torch.uint8, device="cuda")
        scales[..., 1:1 + d // 16] = byte(c)
        return sv.FP4Cache.of(c.codes, scales.view(torch.float8_e4m3fn)[..., 1:1 + d // 16])

    x = torch.randn(2 * nq, 4, d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    mine = [sv.FP4Cache.of(c.codes.clone(), c.scales.clone()) for c in (kc, vc)]
    sv.rope_append(q, x[:, :2], x[:, 2:], sv.RopePlan(d), *mine, table, lens, cu)
    for form in ((nhd, nhd), (nhd, None), (None, nhd), (wide, wide), (wide, None), (odd, odd), (None, odd)):
        k, v = (f(c) if f else sv.FP4Cache.of(c.codes.clone(), c.scales.clone()) for f, c in zip(form, (kc, vc)))
        got, lse = sv.chunk_attention(q, k, v, table, lens, cu, nq, want_lse=True)
        assert sv.default_workspace().status() == 0
        _check(got, lse, ref, torch.bfloat16, max(kv), d, 4)
        if odd not in form:
            sv.rope_append(q, x[:, :2], x[:, 2:], sv.RopePlan(d), k, v, table, lens, cu)
            for a, b in zip(mine, (k, v)):
                assert torch.equal(a.codes, b.codes) and torch.equal(byte(a), byte(b))


def test_fp4_scale_of_zero(sv):
    """Every key that is seen counts the same."""
    for nq in (1, 40):
        _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 64, scale=0.0, seed=4)


@pytest.mark.parametrize("nq", [1, 5, 12, 40])
def test_fp4_scores_too_small_to_tell(sv, nq):
    """The product of scale, unit and the queries' power of two lies below every fp32 number, or the scale is zero and the queries
    are large: every key that is seen counts the same."""
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 128, scale=1e-30, units=(2.0 ** -64, 1.0), seed=6)
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 64, scale=1e-12, grow=1e-35, seed=7)
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 64, scale=0.0, grow=1e25, seed=8)
    _fp4(sv, [nq, nq], [77, 260], 16, 8, 4, 128, dtype="f16", scale=1e-40, units=(2.0 ** -10, 1.0), seed=9)


@pytest.mark.parametrize("d,nq,hq", [(64, 17, 4), (128, 40, 16), (80, 40, 4), (128, 4, 8)])
def test_fp4_wait_that_runs_out_writes_nothing(sv, d, nq, hq):
    """Every bounded wait gives up at once: the status says so, no row is written; the next call is right."""
    ws = sv.Workspace()
    (bk, bv), _, *big = _fp4_batch(sv, [4 * nq] * 6, [3000] * 6, 16, 2, d, 3)
    big_q = torch.randn(24 * nq, hq, d).bfloat16().cuda()
    (kc, vc), _, table, lens, cu = _fp4_batch(sv, [nq], [700], 16, 2, d, 4)
    q = torch.randn(nq, hq, d).bfloat16().cuda()
    want = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, workspace=ws)
    sv.chunk_attention(big_q, bk, bv, *big, 4 * nq, workspace=ws)       # splits items: leaves records
    assert ws.status() == 0
    out = torch.ones_like(want)
    got = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, out=out, workspace=ws, tuning=sv.Tuning(wait_limit_us=-1))
    waits = nq * hq // 2 > 32                                           # the kernel for few rows waits for nothing
    assert ws.status() == (4 if waits else 0)
    assert torch.equal(got, torch.ones_like(got) if waits else want)
    for tuning in (None, sv.Tuning(wait_limit_us=10 ** 6)):
        sv.chunk_attention(q, kc, vc, table, lens, cu, nq, out=out, workspace=ws, tuning=tuning)
        assert ws.status() == 0 and torch.equal(out, want)


def test_fp4_all_numbers(sv):
    """Every e4m3 scale with every code: the values that the kernel multiplies are exact."""
    d, page = 128, 16
    scales = torch.arange(127, dtype=torch.uint8).repeat(2)[: 7 * page].view(7, page, 1, 1).expand(-1, -1, 1, d // 16).contiguous()
    codes = torch.arange(7 * page * d // 2).remainder(256).to(torch.uint8).view(7, page, 1, d // 2).contiguous()
    kc = sv.FP4Cache.of(torch.zeros_like(codes).cuda(), torch.full_like(scales, 56).cuda().view(torch.float8_e4m3fn))
    vc = sv.FP4Cache.of(codes.cuda(), scales.cuda().view(torch.float8_e4m3fn))
    table = torch.arange(7, dtype=torch.int32, device="cuda")[None]
    n = 7 * page
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, n]))
    q = torch.zeros(n, 1, d, dtype=torch.float16, device="cuda")
    exact = M.values(codes, scales).view(n, d)
    out = sv.chunk_attention(q, kc, vc, table, lens, cu, n, window=1)      # every token sees itself alone: its own values
    assert torch.equal(out.view(n, d).cpu().double(), exact)
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    for i in (0, 5, 100):                                                  # the kernel for few rows
        t = table.clone()
        lens1 = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        got = sv.chunk_attention(q[:1], kc, vc, t, lens1, torch.cat([0 * one, one]), 1, window=1)
        assert torch.equal(got.view(d).cpu().double(), exact[i])
    for dt in (torch.bfloat16, torch.float32):
        assert torch.equal(vc.values(dt).cpu().double().view(n, d), exact)


def test_fp4_repeats_graph_stream_status(sv):
    for nq in (1, 40):
        q, kc, vc, table, lens, cu, want = _fp4(sv, [nq, nq], [900, 700], 16, 8, 2, 128)
        ws, out = sv.Workspace(), torch.empty_like(want)
        call = lambda t=table, **kw: sv.chunk_attention(q, kc, vc, t, lens, cu, nq, **kw)  # noqa: E731
        call(out=out, workspace=ws)
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out=out, workspace=ws)
        lens.copy_(torch.tensor([130, 690], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()) and ws.status() == 0
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        side.synchronize()
        assert torch.equal(got, out)
        bad = table.clone()
        bad[0, 2] = kc.shape[0] + 5
        got = call(bad)
        assert sv.default_workspace().status() == 7
        zk, zv = (sv.FP4Cache.of(c.codes.clone(), c.scales.clone(), c.unit) for c in (kc, vc))
        for z in (zk, zv):
            z.codes[table[0, 2].long()] = 0
            z.scales.view(torch.uint8)[table[0, 2].long()] = 0
        assert torch.equal(got, sv.chunk_attention(q, zk, zv, table, lens, cu, nq))


@pytest.mark.parametrize("nq", [1, 17])
def test_fp4_far_pages(sv, nq):
    """A cache of more than 2^31 bytes: page offsets pass 32 bits, of codes and (of a wide pool) of scales."""
    page, hkv, d = 16, 8, 128
    pages = 2 ** 31 // (page * hkv * d // 2) + 64
    far = [sv.FP4Cache(pages, page, hkv, d) for _ in range(2)]
    (kc, vc), _, _, _, _ = _fp4_batch(sv, [1], [60], page, hkv, d, 3)
    ids = torch.tensor([[pages - 1, 3, pages - 7, pages // 2 + 1]], dtype=torch.int32, device="cuda")
    for f, c in zip(far, (kc, vc)):
        c.scales.view(torch.uint8)[c.scales.view(torch.uint8) == 127] = 50
        f.codes[ids[0].long()] = c.codes[:4]
        f.scales.view(torch.uint8)[ids[0].long()] = c.scales.view(torch.uint8)[:4]
    near = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([60], [0, nq]))
    q = torch.randn(nq, 16, d, device="cuda").to(torch.bfloat16)
    assert torch.equal(sv.chunk_attention(q, *far, ids, lens, cu, nq), sv.chunk_attention(q, kc, vc, near, lens, cu, nq))
    plan, k = sv.RopePlan(d), torch.randn(nq, hkv, d, device="cuda").to(torch.bfloat16)
    sv.rope_append(q, k, k, plan, *far, ids, lens, cu)
    sv.rope_append(q, k, k, plan, kc, vc, near, lens, cu)
    for f, c in zip(far, (kc, vc)):
        assert torch.equal(f.codes[ids[0].long()], c.codes[:4])
        assert torch.equal(f.scales.view(torch.uint8)[ids[0].long()], c.scales.view(torch.uint8)[:4])
    assert sv.default_workspace().status() == 0


# ------------------------------------------------------------------------ the write into 4 bits

def _append(sv, new, kv, page, hq, hkv, d, dtype="bf16", rotary=None, layout="half", scaling=None, theta=10000.0, seed=0,
            units=(1.0, 1.0), k_out=False, in_place=False, make=None, memory="hnd", strided=False):
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    n = sum(new)
    if strided:     # one projection's output, heads that start at odd places
        qkv = torch.randn(n, hq + 2 * hkv, d + 2, generator=g).to(dt).cuda()[..., 1:d + 1]
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = (torch.randn(n, h, d, generator=g).to(dt).cuda() for h in (hq, hkv, hkv))
    if make:
        make(k, v)
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
    caches = []
    for unit in units:
        codes = torch.full((pages, page, hkv, d // 2), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((pages, page, hkv, d // 16), 0x31, dtype=torch.uint8, device="cuda")
        if memory == "hnd":
            codes, scales = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (codes, scales))
        caches.append(sv.FP4Cache.of(codes, scales.view(torch.float8_e4m3fn), unit))
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    plan = sv.RopePlan(d, rotary_dim=rotary, theta=theta, layout=layout, scaling=scaling)
    want_q = torch.empty_like(q)
    rotated = torch.empty(n, hkv, d, dtype=dt, device="cuda")
    sv.rope_append(q, k, v, plan, None, None, None, lens, cu, q_out=want_q, k_out=rotated)
    k0, v0 = k.cpu().double(), v.cpu().double()
    ko = k if in_place else torch.empty_like(rotated) if k_out else None
    qo = sv.rope_append(q, k, v, plan, *caches, table.cuda(), lens, cu, k_out=ko, q_out=q if in_place else None)
    assert sv.default_workspace().status() == 0
    assert torch.equal(qo, want_q) and (ko is None or torch.equal(ko, rotated))
    want = [(torch.full((pages, page, hkv, d // 2), 0xA5), torch.full((pages, page, hkv, d // 16), 0x31)) for _ in range(2)]
    starts = cu.tolist()
    for b in range(len(kv)):
        for i, pos in enumerate(R.positions(starts, kv, b)):
            if pos < 0:
                continue
            t, pg, s = starts[b] + i, int(table[b, pos // page]), pos % page
            key = R.rope(k0[t], pos, plan.frequencies, plan.factor, plan.rotary_dim, layout).float().to(dt).double()
            for x, (codes, scales), unit, cache in zip((key, v0[t]), want, units, caches):
                for h in range(hkv):
                    for j in range(d // 16):
                        byte, c = M.quantize(x[h, 16 * j:16 * j + 16].tolist(), unit)
                        scales[pg, s, h, j] = byte
                        if c is None:       # a NaN: only the scale says so
                            codes[pg, s, h, 8 * j:8 * j + 8] = cache.codes[pg, s, h, 8 * j:8 * j + 8].cpu()
                            continue
                        codes[pg, s, h, 8 * j:8 * j + 8] = torch.tensor([c[2 * m] | c[2 * m + 1] << 4 for m in range(8)])
    for (codes, scales), c in zip(want, caches):
        assert torch.equal(c.scales.view(torch.uint8).cpu().long(), scales)     # and nothing else was written
        zero = lambda x: torch.where(torch.tensor([y % 8 == 0 for y in range(16)])[x], 0, x)  # noqa: E731 (-0 is 0)
        for half in (lambda x: x & 15, lambda x: x >> 4):
            assert torch.equal(zero(half(c.codes.cpu().long())), zero(half(codes.long())))
    return caches, plan


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (128, 64), (80, 80), (80, 20), (80, 40), (128, 128), (256, 256), (96, 48), (128, 48), (112, 112),
                                      (48, 48), (16, 16), (16, 2), (80, 72)])
def test_append_layouts(sv, layout, dtype, d, rotary):
    _append(sv, [1, 3, 5], [1, 20, 40], 16, 4, 2, d, dtype=dtype, rotary=rotary, layout=layout, seed=d + rotary)


@pytest.mark.parametrize("page", [1, 5, 16, 128])
@pytest.mark.parametrize("memory", ["hnd", "nhd"])
def test_append_pages_groups_idle(sv, page, memory):
    _append(sv, [4, 0, 17, 1, 3], [0, 5, 9, 1, 700], page, 7, 1, 64, k_out=True, memory=memory)
    _append(sv, [1] * 40, list(range(1, 41)), page, 2, 2, 64, memory=memory)


@pytest.mark.parametrize("pos", [100, 131071, 1000003])
def test_append_far_positions(sv, pos):
    _append(sv, [8, 5], [pos, pos + 7], 64, 2, 4, 128, theta=500000.0, seed=pos)
    _append(sv, [8, 5], [pos, pos + 7], 64, 2, 4, 80, theta=500000.0, seed=pos)
    _append(sv, [3], [pos], 64, 2, 4, 64, scaling={"type": "linear", "factor": 4.0}, dtype="f16", seed=pos)


def test_append_in_place_and_strided(sv):
    for d, rotary in ((64, 64), (128, 64), (80, 80)):
        for layout in ("half", "interleaved"):
            _append(sv, [9], [50], 16, 4, 2, d, rotary=rotary, layout=layout, in_place=True)
            _append(sv, [9], [50], 16, 4, 2, d, rotary=rotary, layout=layout, strided=True)


def test_append_units_and_edges_of_the_format(sv):
    """Ties between codes and between scales, blocks of zeros, of tiny and of huge values, infinities and NaN."""
    def ties(k, v):     # multiples of small fractions: quotients fall on borders between codes
        for x in (k, v):
            x.copy_((torch.randint(-48, 49, x.shape) / 8.0).to(x.dtype))
            x[..., 0] = 6.0

    def extremes(k, v):
        v[0] = 0.0
        v[1] *= 1e-3
        v[2] *= 1e-6
        v[3] *= 1000.0
        v[4] *= 2.0 ** 13
        v[5, :, 3] = math.inf
        v[6, :, 5] = -math.inf
        v[7, :, 7] = k[7, :, 9] = math.nan
        v[8] = -0.0

    for dtype in ("bf16", "f16"):
        for rotary in (2, 64):
            _append(sv, [9], [9], 16, 2, 2, 64, dtype=dtype, make=ties, rotary=rotary, theta=1e30)
            _append(sv, [9], [9], 16, 2, 2, 64, dtype=dtype, make=extremes, rotary=rotary)
        _append(sv, [9], [9], 16, 2, 2, 128, dtype=dtype, units=(2.0 ** -8, 2.0 ** 3))


def test_append_many_blocks_hold_the_exactly_rotated_keys(sv):
    """2^20 keys: some hundred would have another code by fp32's error, were it let through."""
    for dtype, layout in (("bf16", "half"), ("f16", "interleaved")):
        dt, n, hkv, d, page = DTYPES[dtype], 1024, 8, 128, 64
        g = torch.Generator(device="cuda").manual_seed(7)
        k = torch.randn(n, hkv, d, generator=g, device="cuda").to(dt)
        plan = sv.RopePlan(d, theta=500000.0, layout=layout)
        pos0 = 100000
        cols = (pos0 + n) // page + 1
        table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
        first = pos0 // page
        table[0, first:] = torch.arange(cols - first, dtype=torch.int32, device="cuda")
        kc, vc = (sv.FP4Cache(cols - first, page, hkv, d) for _ in range(2))
        lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([pos0 + n], [0, n]))
        sv.rope_append(k, k, k, plan, kc, vc, table, lens, cu)
        pos = torch.arange(pos0, pos0 + n, device="cuda", dtype=torch.float64)
        angle = pos[:, None, None] * torch.tensor(plan.frequencies, dtype=torch.float64, device="cuda")
        x = k.double()
        a, b = (x[..., :64], x[..., 64:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
        a, b = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
        y = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
        y = y.float().to(dt).double().unflatten(-1, (-1, 16))
        scale = (y.abs().amax(-1) / 6).clamp(2.0 ** -9, 448.0).float().to(torch.float8_e4m3fn)
        got_s = kc.scales.view(torch.uint8).flatten(0, 1)[pos0 % page:pos0 % page + n]
        assert torch.equal(got_s, scale.view(torch.uint8))
        codes = torch.tensor(M.CODES, dtype=torch.float64, device="cuda")
        q = y.abs() / scale.double()[..., None]
        borders = (codes[1:] + codes[:-1]) / 2
        at = torch.bucketize(q, borders)                # 0 to 7: a border belongs to the code below it,
        up = (at < 7) & (at % 2 == 1) & (q == borders[at.clamp(max=6)])     # or to the one above where that is even
        want = codes[at + up.long()] * torch.sign(y) * scale.double()[..., None]
        got = kc.values(torch.float32).double().flatten(0, 1)[pos0 % page:pos0 % page + n]
        assert torch.equal(got, want.flatten(-2))


def test_append_then_attention(sv):
    """Two steps of a request: a prompt and a token, written and read in 4 bits, against the values that the cache holds."""
    d, hq, hkv, page = 128, 8, 2, 16
    kc, vc = (sv.FP4Cache(8, page, hkv, d) for _ in range(2))
    table = torch.tensor([[5, 0, 7, 2]], dtype=torch.int32, device="cuda")
    plan = sv.RopePlan(d)
    for n, L in ((37, 37), (1, 38)):
        x = torch.randn(n, hq + 2 * hkv, d, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
        lens, cu = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([L], [0, n]))
        q = sv.rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], plan, kc, vc, table, lens, cu)
        got, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, n, want_lse=True)
        ref = M.attention(q, kc.values(torch.float32).cpu().double(), vc.values(torch.float32).cpu().double(), table, lens, cu,
                          True, 0, 0, d ** -0.5)
        _check(got, lse, ref, torch.bfloat16, L, d, 4)


def test_fp4_refusals(sv):
    (kc, vc), _, table, lens, cu = _fp4_batch(sv, [2], [20], 16, 2, 64, 4)
    q = torch.randn(2, 4, 64).to(torch.bfloat16).cuda()
    call = lambda q=q, k=kc, v=vc, **kw: sv.chunk_attention(q, k, v, table, lens, cu, 2, **kw)  # noqa: E731
    dense = torch.zeros(kc.shape, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k=dense), dict(v=dense), dict(q=q.float())):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(ValueError):
        call(v=sv.FP4Cache(3, 16, 2, 128))
    for bad in (dict(sinks=-1), dict(window=-1), dict(scale=math.inf), dict(scale=1e38 * 3)):
        if "scale" in bad and bad["scale"] < 1e39:
            big = sv.FP4Cache.of(kc.codes, kc.scales, 2.0 ** 64)
            with pytest.raises(sv.SpecError):
                call(k=big, **bad)
            continue
        with pytest.raises(sv.SpecError):
            call(**bad)
    k = torch.randn(2, 2, 64, device="cuda")
    plan = sv.RopePlan(64)
    with pytest.raises(sv.SpecError):       # float32 tokens
        sv.rope_append(torch.randn(2, 4, 64, device="cuda"), k, k, plan, kc, vc, table, lens, cu)
    with pytest.raises(TypeError):
        sv.rope_append(q, k.bfloat16(), k.bfloat16(), plan, kc, dense, table, lens, cu)
    loose = torch.zeros(4, 16, 2, 33, dtype=torch.uint8, device="cuda")[..., :32]     # rows 33 bytes apart
    with pytest.raises(sv.SpecError):
        call(k=sv.FP4Cache.of(loose, torch.zeros(4, 16, 2, 4, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)),
             v=sv.FP4Cache(4, 16, 2, 64))


def test_fp4_page_range_status_of_the_write(sv):
    kc, vc = (sv.FP4Cache(2, 16, 2, 64) for _ in range(2))
    q, k = torch.randn(3, 4, 64).to(torch.bfloat16).cuda(), torch.randn(3, 2, 64).to(torch.bfloat16).cuda()
    lens, cu = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([17], [0, 3]))
    for entry in (-1, 2):
        table = torch.tensor([[1, entry]], dtype=torch.int32, device="cuda")
        for rotary in (64, 20):     # both forms of the kernel
            plan = sv.RopePlan(64, rotary_dim=rotary)
            for c in (kc, vc):
                c.codes.zero_()
            sv.rope_append(q, k, k, plan, kc, vc, table, lens, cu)
            assert sv.default_workspace().status() == 7
            assert kc.codes[1, 14:].any() and not kc.codes[1, :14].any() and not kc.codes[0].any()
