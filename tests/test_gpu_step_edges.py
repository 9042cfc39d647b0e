"""Edges of the step operators on the GPU: waits that run out, buffers and streams that are shared, windows, lengths
and sizes at their limits."""
import pytest
import torch

from tests import step_reference as R
from tests.test_gpu_step_ops import DTYPES, _batch, _check_sample, _rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import draft_verification_spec_gb300 as m
    m.lib()
    return m


def _guarded(shape, dtype, pad=4096):
    """A tensor in the middle of a buffer of ones, and the buffer's two ends."""
    n = 1
    for s in shape:
        n *= s
    flat = torch.ones(n + 2 * pad, dtype=dtype, device="cuda")
    return flat[pad:pad + n].view(shape), (flat[:pad], flat[pad + n:])


@pytest.mark.parametrize("d,nq,hq", [(64, 17, 4), (128, 40, 16), (128, 4, 8)])
def test_attention_wait_that_runs_out_writes_nothing(sv, d, nq, hq):
    """Every bounded wait gives up at once: the status says so, and whatever records an earlier, larger call has left in
    the workspace, the kernel that joins split rows writes no row of this one; the next call is right."""
    dt, hkv = torch.bfloat16, 2
    ws = sv.Workspace()
    big = _batch([4 * nq] * 6, [3000] * 6, 16, hkv, d, dt, 3)
    big_q = torch.randn(24 * nq, hq, d).to(dt).cuda()
    sv.chunk_attention(big_q, *big, 4 * nq, workspace=ws)                # splits items: leaves records
    kc, vc, table, lens, cu = _batch([nq], [700], 16, hkv, d, dt, 4)
    q = torch.randn(nq, hq, d).to(dt).cuda()
    want = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, workspace=ws)
    sv.chunk_attention(big_q, *big, 4 * nq, workspace=ws)
    assert ws.status() == 0
    out, ends = _guarded((nq, hq, d), dt)
    got = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, out=out, workspace=ws, tuning=sv.Tuning(wait_limit_us=-1))
    waits = nq * hq // hkv > 16                                          # the kernel for few rows waits for nothing
    assert ws.status() == (4 if waits else 0)
    assert all((e == 1).all() for e in ends)
    assert torch.equal(got, torch.ones_like(got) if waits else want)
    sv.chunk_attention(q, kc, vc, table, lens, cu, nq, out=out, workspace=ws)
    assert ws.status() == 0 and torch.equal(out, want)
    sv.chunk_attention(q, kc, vc, table, lens, cu, nq, out=out, workspace=ws, tuning=sv.Tuning(wait_limit_us=10 ** 6))
    assert ws.status() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("hq,hkv,dtype", [(155, 50, "f32"), (156, 50, "f32"), (200, 50, "f32"), (500, 50, "bf16")])
def test_rope_of_very_wide_tokens(sv, hq, hkv, dtype):
    """Tokens of 65,280 to 76,800 16-byte pieces: on either side of what the piece kernel's quotients hold."""
    _rope(sv, [2, 1], [2, 20], 16, hq, hkv, 1024, dtype=dtype, seed=hq)


def test_graph_of_a_workspace_that_grew_later(sv):
    """A graph captured with a workspace for single tokens; a prompt over the same workspace needs a larger buffer; the
    graph's replays write neither over memory that others have got since, nor wrong rows."""
    dt, hq, hkv, d = torch.bfloat16, 8, 2, 128
    ws = sv.Workspace()
    kc, vc, table, lens, cu = _batch([1], [2000], 16, hkv, d, dt, 4)
    q = torch.randn(1, hq, d).to(dt).cuda()
    want = sv.chunk_attention(q, kc, vc, table, lens, cu, 1)
    out = torch.empty_like(want)
    sv.chunk_attention(q, kc, vc, table, lens, cu, 1, out=out, workspace=ws)
    size = ws.step_buf.numel()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.chunk_attention(q, kc, vc, table, lens, cu, 1, out=out, workspace=ws)
    big = _batch([200], [300], 16, hkv, d, dt, 5)
    sv.chunk_attention(torch.randn(200, hq, d).to(dt).cuda(), *big, 200, workspace=ws)
    assert ws.step_buf.numel() > size
    others = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    out.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not any(o.any() for o in others)
    assert ws.status() == 0


def test_status_survives_a_larger_call(sv):
    """rope_append reports a page; an attention over the same workspace needs a larger buffer before anybody looks."""
    dt = torch.bfloat16
    ws = sv.Workspace()
    kc, vc, table, lens, cu = _batch([2], [40], 16, 2, 64, dt, 4)
    q, k = torch.randn(2, 4, 64).to(dt).cuda(), torch.randn(2, 2, 64).to(dt).cuda()
    bad = torch.full_like(table, -1)
    sv.rope_append(q, k, k, sv.RopePlan(64), kc, vc, bad, lens, cu, workspace=ws)
    sv.chunk_attention(q, kc, vc, table, lens, cu, 2, workspace=ws)
    assert ws.status() == 7 and ws.status() == 0


def test_attention_first_call_of_a_thread(sv):
    """A thread's first call runs the same kernel as every other: equal bit for bit."""
    import threading
    dt, nq = torch.bfloat16, 20
    c = _batch([nq] * 2, [1500, 750], 16, 2, 128, dt, 2)
    q = torch.randn(2 * nq, 8, 128).to(dt).cuda()
    want = sv.chunk_attention(q, *c, nq)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        t = threading.Thread(target=lambda: got.append(sv.chunk_attention(q, *c, nq)))
        t.start()
        t.join()
    assert all(torch.equal(g, want) for g in got) and len(got) == 3


def test_attention_from_threads_on_one_stream(sv):
    """Threads that share the default workspace of a stream: calls of different sizes, every one right."""
    import threading
    dt, hq, hkv, d = torch.bfloat16, 8, 2, 128
    cases = []
    for i, (nq, kv) in enumerate(((1, 3000), (3, 900), (20, 1500))):
        c = _batch([nq] * 2, [kv, kv // 2], 16, hkv, d, dt, i)
        q = torch.randn(2 * nq, hq, d).to(dt).cuda()
        cases.append((q, c, nq, sv.chunk_attention(q, *c, nq)))
    torch.cuda.synchronize()
    bad = []

    def work(q, c, nq, want):
        for _ in range(200):
            if not torch.equal(sv.chunk_attention(q, *c, nq), want):
                bad.append(nq)

    threads = [threading.Thread(target=work, args=a) for a in cases]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad and sv.default_workspace().status() == 0


@pytest.mark.parametrize("page", [8, 16, 24, 128])
@pytest.mark.parametrize("nq,hq,d", [(1, 8, 128), (4, 4, 64), (40, 8, 256), (17, 8, 128), (150, 8, 64), (300, 4, 128)])
def test_attention_window_ignores_pages_behind_it(sv, nq, hq, d, page):
    """A cache that has given up the pages behind the window: no entry in the table, or another request's page with
    anything in it.  Nothing is reported and the rows are those of the whole cache."""
    dt, hkv, window = torch.bfloat16, 2, 100
    kv = [nq + 310, nq + 700, nq + 20]
    kc, vc, table, lens, cu = _batch([nq] * 3, kv, page, hkv, d, dt, page + nq)
    q = torch.randn(3 * nq, hq, d).to(dt).cuda()
    want, want_lse = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, window=window, want_lse=True)
    if page == 16:
        ro, rl, size, spread = R.attention(q, kc, vc, table, lens, cu, True, window, d ** -0.5)
        bo, bl = R.attention_bounds(dt, size, spread, d)
        assert ((want.cpu().double() - ro).abs() <= bo).all()
    junk = kc.shape[0]     # one page more, of NaN
    kc, vc = (torch.cat([c, torch.full_like(c[:1], float("nan"))]) for c in (kc, vc))
    for stale in (-1, junk):
        t = table.clone()
        for b, n in enumerate(kv):
            t[b, : max(0, n - nq - window + 1) // page] = stale    # pages that end at or before the first visible key
        for causal in (True, False):
            full = want if causal else sv.chunk_attention(q, kc, vc, table, lens, cu, nq, window=window, causal=False)
            got, lse = sv.chunk_attention(q, kc, vc, t, lens, cu, nq, window=window, causal=causal, want_lse=True)
            assert sv.default_workspace().status() == 0
            assert torch.equal(got, full)
            assert not causal or torch.equal(lse, want_lse)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 30])
@pytest.mark.parametrize("hq,d", [(2, 64), (8, 64), (16, 128), (8, 256)])
def test_attention_window_as_wide_as_its_type(sv, hq, d, window):
    """Such a window hides nothing, whatever the position, that of tokens before the request's first one included."""
    dt, hkv, new, kv = torch.bfloat16, 2, [17, 40, 17, 1, 3], [9, 33, 300, 0, 3]
    kc, vc, table, lens, cu = _batch(new, kv, 16, hkv, d, dt, hq)
    q = torch.randn(sum(new), hq, d).to(dt).cuda()
    for causal in (True, False):
        want = sv.chunk_attention(q, kc, vc, table, lens, cu, 40, causal=causal, want_lse=True)
        got = sv.chunk_attention(q, kc, vc, table, lens, cu, 40, causal=causal, window=window, want_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sv.default_workspace().status() == 0


@pytest.mark.parametrize("window", [0, 20, 5])
@pytest.mark.parametrize("nq,hq,d", [(1, 4, 64), (20, 4, 64), (20, 8, 256), (150, 4, 128)])
def test_attention_length_beyond_the_table(sv, nq, hq, d, window):
    """More tokens than the table has pages for: reported, and the rows' positions stay what rope_append makes of them;
    they see the keys that the table holds."""
    dt, page, cols, hkv = torch.bfloat16, 16, 13, 2
    cap, kv = page * cols, [page * cols + 4, page * cols - 3, page * cols + 60]
    kc, vc, table, lens, cu = _batch([nq] * 3, [min(k, cap) for k in kv], page, hkv, d, dt, nq)
    q = torch.randn(3 * nq, hq, d).to(dt).cuda()
    out, lse = sv.chunk_attention(q, kc, vc, table[:, :cols], torch.tensor(kv, dtype=torch.int32, device="cuda"), cu, nq,
                                  window=window, want_lse=True)
    assert sv.default_workspace().status() == 7 and sv.default_workspace().status() == 0
    kd, vd, qd = kc.double().cpu(), vc.double().cpu(), q.double().cpu()
    ids = table.cpu().long()
    for b, n in enumerate(kv):
        K, V = (c[ids[b, :cols]].flatten(0, 1)[:n] for c in (kd, vd))
        for i in range(nq):
            pos = n - nq + i
            see = slice(max(0, pos - window + 1) if window else 0, max(0, min(cap, pos + 1)))
            for h in range(hq):
                row, g = b * nq + i, h // (hq // hkv)
                k, v = K[see, g], V[see, g]
                if len(k) == 0:
                    assert float(lse[row, h]) == float("-inf") and not out[row, h].any()
                    continue
                x = k @ qd[row, h] * d ** -0.5
                w = torch.softmax(x, 0)
                spread = (k.abs() @ qd[row, h].abs() * d ** -0.5).max()
                bo, bl = R.attention_bounds(dt, w @ v.abs(), spread, d)
                assert ((out[row, h].double().cpu() - w @ v).abs() <= bo).all()
                want = float(torch.logsumexp(x, 0))
                assert abs(float(lse[row, h]) - want) <= float(bl) + abs(want) * 2.0 ** -23


def test_calls_on_another_stream_leave_queued_work_alone(sv):
    """The current stream's free memory may still be read by work that is queued there: a call on another stream must not
    get it for its outputs or its workspace, and its own tensors' memory must last until it is done."""
    dt, nq, hq, hkv, d = torch.bfloat16, 20, 8, 2, 128
    c = _batch([nq] * 2, [1500, 750], 16, hkv, d, dt, 2)
    q = torch.randn(2 * nq, hq, d).to(dt).cuda()
    k = torch.randn(2 * nq, hkv, d).to(dt).cuda()
    logits, u = torch.randn(8, 4096, device="cuda"), torch.rand(8, device="cuda")
    plan = sv.RopePlan(d)
    side, rotated = torch.cuda.Stream(), torch.empty_like(k)

    def attention(stream):
        return sv.chunk_attention(q, *c, nq, stream=stream, want_lse=True)

    def rope(stream):
        return (sv.rope_append(q, k, None, plan, None, None, None, *c[3:], k_out=rotated, stream=stream),)

    def sample(stream):
        s = sv.sample_tokens(logits, u, 0.8, 40, want_filtered=True, stream=stream)
        return s.tokens, s.probs, s.kept, s.filtered

    for call in (attention, rope, sample):
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        for _ in range(3):
            # blocks of the outputs' sizes, freed while a kernel that reads them is still to run
            held = [torch.full_like(t, 5) for t in want for _ in range(4)]
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)                      # some 10 ms on the current stream
            read = [h + 1 for h in held]
            del held
            got = call(side)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            torch.cuda.synchronize()
            assert all((r == 6).all() for r in read)
    # an input that the caller drops while the other stream has not come to it
    torch.cuda.synchronize()
    want = sv.sample_tokens(logits, u, 0.8, 40).tokens
    torch.cuda.synchronize()
    mine, mine_u = logits.clone(), u.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = sv.sample_tokens(mine, mine_u, 0.8, 40, stream=side)
    del mine, mine_u
    over = [torch.full_like(logits, -1.0) for _ in range(4)] + [torch.zeros_like(u) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got.tokens, want) and len(over) == 8


def test_workspace_of_another_device_is_refused(sv):
    kc, vc, table, lens, cu = _batch([2], [20], 16, 2, 64, torch.bfloat16, 4)
    q, k = torch.randn(2, 4, 64).to(torch.bfloat16).cuda(), torch.randn(2, 2, 64).to(torch.bfloat16).cuda()
    plan = sv.RopePlan(64)
    for ws in (sv.Workspace("cpu"), sv.Workspace("cuda:1")):
        with pytest.raises(ValueError):
            sv.chunk_attention(q, kc, vc, table, lens, cu, 2, workspace=ws)
        with pytest.raises(ValueError):
            sv.rope_append(q, k, k, plan, kc, vc, table, lens, cu, workspace=ws)
    want = sv.chunk_attention(q, kc, vc, table, lens, cu, 2)
    assert torch.equal(want, sv.chunk_attention(q, kc, vc, table, lens, cu, 2, workspace=sv.Workspace("cuda")))


def test_integers_beyond_32_bits(sv):
    """A window or a number of tokens that no C int holds: as much as the largest one, and no less than nothing."""
    kc, vc, table, lens, cu = _batch([20, 3], [90, 200], 16, 2, 64, torch.bfloat16, 4)
    q = torch.randn(23, 8, 64).to(torch.bfloat16).cuda()
    want = sv.chunk_attention(q, kc, vc, table, lens, cu, 20)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1, 2 ** 64 + 1):
        assert torch.equal(want, sv.chunk_attention(q, kc, vc, table, lens, cu, 20, window=window))
        assert torch.equal(want, sv.chunk_attention(q, kc, vc, table, lens, cu, max_q=window))
    for bad in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(sv.SpecError):
            sv.chunk_attention(q, kc, vc, table, lens, cu, 20, window=bad)
        with pytest.raises(sv.SpecError):
            sv.chunk_attention(q, kc, vc, table, lens, cu, bad)
    z, u = torch.randn(2, 500, device="cuda"), torch.rand(2, device="cuda")
    want = sv.sample_tokens(z, u).tokens
    for top_k in (2 ** 31 - 1, 2 ** 31, 2 ** 40, -2 ** 40):
        out = sv.sample_tokens(z, u, top_k=top_k)
        assert torch.equal(out.tokens, want) and (out.kept == 500).all()


def test_sample_filtered_over_its_own_logits_is_refused(sv):
    z = torch.randn(3, 1000, device="cuda")
    u = torch.rand(3, device="cuda")
    fresh = lambda f: sv.SampleOutput(*(torch.empty(3, dtype=t, device="cuda") for t in (torch.int32, torch.float32, torch.int32)), f)  # noqa: E731
    both = torch.randn(3, 2000, device="cuda")
    for f, logits in ((z, z), (both[:, 500:1500], both[:, :1000])):
        with pytest.raises(ValueError):
            sv.sample_tokens(logits, u, 0.8, 40, out=fresh(f))
    want = sv.sample_tokens(both[:, :1000], u, 0.8, 40, want_filtered=True)
    got = sv.sample_tokens(both[:, :1000], u, 0.8, 40, out=fresh(both[:, 1000:]))    # side by side: apart
    assert torch.equal(got.filtered, want.filtered) and torch.equal(got.tokens, want.tokens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [32768, 65537, 131071])
def test_sample_clusters_ties_zeros_infinities(sv, dtype, V):
    """Rows shared by 2 to 8 CTAs: no logit above -inf, NaN, +inf, zeros of both signs, ties across the CTAs' shares."""
    dt, inf, nan = DTYPES[dtype], float("inf"), float("nan")
    z = torch.zeros(10, V)
    z[1, ::2] = -0.0
    z[2] = -inf
    z[3] = -inf
    z[3, V - 3] = -5.0
    z[4, 100:] = -inf
    z[5, ::3] = nan
    z[6, 10] = z[6, V // 2] = z[6, V - 1] = inf
    z[7] = nan
    z[8] = torch.arange(V) // (V // 6) * 1.0
    z[9, : V - 7] = -inf                     # all that counts is the last CTA's
    u = torch.tensor([0.5, 0.999, 0.5, 0.999, 0.9999999, 0.3, 0.7, 0.1, 0.0, 0.6]).cuda()
    z = z.to(dt).cuda()
    for s in (dict(), dict(top_k=V // 2 + 7), dict(top_p=0.5), dict(T=0.0), dict(min_p=0.5), dict(top_k=V - 9, top_p=0.7)):
        _check_sample(sv, z, u, **s)
    for r in range(10):                      # a row alone takes the largest cluster
        _check_sample(sv, z[r:r + 1], u[r:r + 1], top_p=0.6, top_k=V // 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [32768, 100003])
def test_sample_clusters_logits_of_any_size(sv, dtype, V):
    """The general descent and the bins below -2^8 in clusters: masks of -1e9 and of the type's lowest value, logits in the
    hundreds and thousands, vanishing ones."""
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(V)
    z = torch.randn(8, V, generator=g) * 3.0
    low = torch.finfo(dt).min
    z[0, 100:] = -1e9
    z[1, 5:] = low
    z[2, ::2] = -300.0 - torch.arange((V + 1) // 2) % 50
    z[3] = z[3] * 400.0
    z[4, ::7] = torch.randn(len(z[4, ::7]), generator=g) * 1e-20
    z[5] = -500.0 + z[5]
    z[6] = low
    z[6, V - 9] = -1e30
    z[7] = z[7] * 1e-18
    z, u = z.to(dt).cuda(), torch.rand(8, generator=g).cuda()
    for s in (dict(), dict(T=0.0), dict(T=0.6), dict(top_k=17), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=V - V // 3),
              dict(top_k=V - 1, top_p=0.99), dict(T=100.0, top_p=0.9), dict(T=1e4, top_k=V // 2),
              dict(T=0.8, top_k=400, top_p=0.95, min_p=0.01)):
        _check_sample(sv, z, u, **s)
        _check_sample(sv, z[3:4], u[3:4], **s)


def test_sample_clusters_crowded_bins(sv):
    """fp32 logits of which thousands share their 16 top bits, more and fewer than a CTA gathers, in shares of several CTAs."""
    z = 3.0 + torch.rand(3, 70000, generator=torch.Generator().manual_seed(2)) * 0.01
    z[1, ::9] = 3.5
    z[2, 10000:] = -7.0
    u = torch.rand(3, generator=torch.Generator().manual_seed(3)).cuda()
    for s in (dict(), dict(top_k=777, top_p=0.9), dict(top_p=0.4), dict(min_p=0.997), dict(top_k=9000)):
        _check_sample(sv, z.cuda(), u, **s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 9, 10, 18, 19, 38, 39, 76, 77])
def test_sample_rows_per_cluster(sv, dtype, rows):
    """Every size of cluster on 152 SMs (8, 4, 2 CTAs a row and one), settings of their own, rows out of line with 16 bytes."""
    V = 65537
    g = torch.Generator().manual_seed(rows)
    z = (torch.randn(rows, V, generator=g) * 2.0).to(DTYPES[dtype]).cuda()
    u = torch.rand(rows, generator=g).cuda()
    pick = lambda v, t: torch.tensor(v, dtype=t)[torch.randint(len(v), (rows,), generator=g)].cuda()  # noqa: E731
    _check_sample(sv, z, u, pick([0.0, 0.5, 1.0, 1.5], torch.float32), pick([0, 1, 20, 5000], torch.int32),
                  pick([1.0, 0.9, 0.5], torch.float32), pick([0.0, 0.1], torch.float32))
