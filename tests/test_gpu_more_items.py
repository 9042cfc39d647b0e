"""Attention in which a CTA works through several items, and in which the maximum outgrows the reference at chosen keys, vs
float64 on the device: over caches in 16 and in 4 bits."""
import math

import pytest
import torch

from tests import more_reference as M
from tests.test_gpu_more_ops import _check, _fp4_batch
from tests.test_gpu_step_ops import DTYPES, _batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import draft_verification_spec_gb300 as m
    m.lib()
    return m


def _reference(q, kc, vc, table, kv, new, causal, window, sinks, scale):
    """more_reference.attention by requests, in float64 on the device."""
    q, kc, vc = q.cuda().double(), kc.cuda(), vc.cuda()
    n, hq, d = q.shape
    P, hkv = kc.shape[1], kc.shape[2]
    G = hq // hkv
    out, lse = torch.zeros_like(q), torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    size, spread, reach, top = torch.zeros_like(q), torch.zeros_like(lse), torch.zeros_like(lse), torch.zeros_like(lse)
    at = 0
    for b, (L, m) in enumerate(zip(kv, new)):
        rows = slice(at, at + m)
        at += m
        if m == 0 or L == 0:
            continue
        t = torch.arange(L, device="cuda")
        K = kc[table[b, t // P].long(), t % P].repeat_interleave(G, 1)      # [L, hq, d]
        V = vc[table[b, t // P].long(), t % P].repeat_interleave(G, 1)
        pos = (L - m + torch.arange(m, device="cuda"))[:, None]
        see = (t <= pos) if causal else (t >= 0).expand(m, L)
        if window:
            see = see & ((t > pos - window) | (t < sinks))
        some, see = see.any(1), see[:, None]
        x = torch.einsum("mhd,lhd->mhl", q[rows], K) * scale
        x = torch.where(see, x, -math.inf)
        most = x.amax(-1, keepdim=True)
        w = torch.exp(x - torch.where(torch.isinf(most), 0.0, most))
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
        out[rows], size[rows] = torch.einsum("mhl,lhd->mhd", w, V), torch.einsum("mhl,lhd->mhd", w, V.abs())
        lse[rows] = torch.where(some[:, None], (most + total.log()).squeeze(-1), -math.inf)
        big = lambda y: torch.where(see, y, 0.0).amax(-1)  # noqa: E731
        spread[rows] = big(torch.einsum("mhd,lhd->mhl", q[rows].abs(), K.abs())) * abs(scale)
        reach[rows] = big(K.abs().sum(-1).t()[None] * q[rows].abs().amax(-1)[..., None]) * abs(scale)
        top[rows] = big(V.abs().amax(-1).t()[None].expand(m, -1, -1))
    return [y.cpu() for y in (out, lse, size, spread, reach, top)]


def test_the_reference_on_the_device(sv):
    new, kv = [3, 0, 2, 4], [40, 9, 0, 30]
    (kc, vc), (ke, ve), table, lens, cu = _fp4_batch(sv, new, kv, 8, 2, 16, 1)
    q = torch.randn(9, 4, 16)
    for causal, window, sinks in ((True, 0, 0), (True, 5, 2), (False, 3, 0)):
        a = M.attention(q, ke, ve, table, lens, cu, causal, window, sinks, 0.3)
        for x, y in zip(a, _reference(q, ke, ve, table, kv, new, causal, window, sinks, 0.3)):
            assert torch.allclose(x, y, rtol=1e-12, atol=1e-13)


def _run(sv, bits, dtype, new, kv, page, hq, hkv, d, window, sinks, seed, causal=True, layout="hnd"):
    dt = DTYPES[dtype]
    if bits == 4:
        (kc, vc), (ke, ve), table, lens, cu = _fp4_batch(sv, new, kv, page, hkv, d, seed, layout)
    else:
        kc, vc, table, lens, cu = _batch(new, kv, page, hkv, d, dt, seed, layout)
        ke, ve = kc.double(), vc.double()
    q = (torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(seed + 1)) * 1.5).to(dt).cuda()
    call = lambda: sv.chunk_attention(q, kc, vc, table, lens, cu, max(new), causal=causal, window=window, sinks=sinks,  # noqa: E731
                                      want_lse=True)
    out, lse = call()
    assert sv.default_workspace().status() == 0
    ref = _reference(q, ke, ve, table, kv, new, causal, window, sinks, d ** -0.5)
    _check(out, lse, ref, dt, max(kv), d, bits)
    again = call()
    assert torch.equal(out, again[0]) and torch.equal(lse.nan_to_num(), again[1].nan_to_num())


def _mixed(seed, B, sizes, longest):
    """New tokens and lengths of a batch, idle requests and ones without keys before the new tokens among them."""
    g = torch.Generator().manual_seed(seed)
    new = [sizes[i] for i in torch.randint(0, len(sizes), (B,), generator=g).tolist()]
    kv = [n + int(x) for n, x in zip(new, torch.randint(0, longest, (B,), generator=g).tolist())]
    kv[1], kv[B // 2] = new[1], max(new[B // 2] - 1, 0)
    return new, kv


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (4, "f16"), (16, "bf16"), (16, "f16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
@pytest.mark.parametrize("sizes,hq,hkv,d", [
    ([0, 1, 5, 16, 20, 40], 32, 4, 64),         # 256-row tiles: items of two halves, of shared halves behind them, and the reverse
    ([17], 32, 4, 128),                         # 136 rows: all of 256
    ([17, 3, 33], 32, 4, 80),
    ([5, 1, 16, 0], 32, 4, 128),                # 128 rows at most
    ([10, 3], 16, 4, 64),
    ([1], 32, 8, 128), ([1, 4, 2], 32, 8, 64),  # up to 32 rows
    ([4, 8, 3], 16, 4, 128),
    ([1, 3], 32, 8, 96),
])
def test_a_cta_works_through_several_items(sv, sizes, hq, hkv, d, window, sinks, bits, dtype):
    """Runs of 20 and more units a CTA (a unit is a key tile; an item has four or five of its own), of items of 1 to 11 tiles."""
    new, kv = _mixed(d + len(sizes), 70, sizes, 1300)
    tile = 128 if max(new) * hq // hkv > 16 else 64
    items = hkv * sum(-(-n * (hq // hkv) // 256) for n in new)
    units = items * 3 + hkv * sum(min(k, (window or k) + tile) // tile for n, k in zip(new, kv) if n)
    assert units > 152 * 6 and items > 150
    _run(sv, bits, dtype, new, kv, 16, hq, hkv, d, window, sinks, seed=d + window)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("page", [1, 24, 128])
def test_several_items_other_pages_and_both_ways(sv, page, bits):
    new, kv = _mixed(page, 60, [1, 7, 18, 40], 1000)
    _run(sv, bits, "bf16", new, kv, page, 16, 4, 64, 0, 0, page, causal=False, layout="nhd")
    _run(sv, bits, "bf16", new, kv, page, 16, 4, 128, 90, 7, page, causal=False)


# keys (tile of 128, column) at which the maximum grows, one for every 16 values of a head
GROWN = [(2, 40), (3, 70), (4, 100), (5, 33), (6, 64), (7, 96), (2, 127), (3, 0)]


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (4, "f16"), (16, "bf16"), (16, "f16")])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("nq,G,B", [(10, 4, 48), (40, 4, 24), (1, 4, 48), (4, 4, 48), (6, 5, 40)])
def test_the_reference_is_outgrown_in_the_midst_of_a_tile(sv, nq, G, B, d, bits, dtype):
    """Scores are 0, but for one key of a row, in some column of a later tile, whose weight is 2^9 of the others' (2^8 is what lets
    the reference stand): what was summed up before is rescaled, and is a good part of the row.  A second one outgrows the first for
    every third row."""
    dt, hkv, page, blocks = DTYPES[dtype], 4, 64, d // 16
    L = 1024 + nq
    new, kv = [nq] * B, [L + b % 3 for b in range(B)]
    g = torch.Generator().manual_seed(d + nq)
    width = -(-max(kv) // page)
    pages = B * width
    table = torch.randperm(pages, generator=g).to(torch.int32).view(B, width).cuda()
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    cu = (torch.arange(B + 1, dtype=torch.int32) * nq).cuda()
    scale, a = d ** -0.5, 1.0
    # 16 values of 6 s each against queries of a: 9 powers of two
    unit_score = 16 * 6 * a * scale * math.log2(math.e)
    grown = [GROWN[(i + d // 16) % len(GROWN)] for i in range(blocks)]
    if bits == 4:
        s = torch.tensor(9.0 / unit_score).to(torch.float8_e4m3fn)
        if float(s) < 9.0 / unit_score:
            s = (s.view(torch.uint8) + 1).view(torch.float8_e4m3fn)
        kcodes = torch.zeros(pages, page, hkv, d // 2, dtype=torch.uint8)
        kscales = torch.full((pages, page, hkv, d // 16), 56, dtype=torch.uint8)
        vcodes = torch.randint(0, 256, (pages, page, hkv, d // 2), generator=g, dtype=torch.uint8)
        vscales = torch.randint(44, 60, (pages, page, hkv, d // 16), generator=g, dtype=torch.uint8)
        for i, (tile, col) in enumerate(grown):
            key = tile * 128 + col
            kcodes[table[:, key // page].cpu().long(), key % page, :, 8 * i:8 * i + 8] = 0x77
            kscales[table[:, key // page].cpu().long(), key % page, :, i] = s.view(torch.uint8)
        kc, vc = (sv.FP4Cache.of(c.transpose(1, 2).contiguous().transpose(1, 2).cuda(),
                                 x.transpose(1, 2).contiguous().transpose(1, 2).cuda().view(torch.float8_e4m3fn))
                  for c, x in ((kcodes, kscales), (vcodes, vscales)))
        ke, ve = M.values(kcodes, kscales).cuda(), M.values(vcodes, vscales).cuda()
    else:
        kc, vc = torch.zeros(pages, page, hkv, d), torch.randn(pages, page, hkv, d, generator=g)
        for i, (tile, col) in enumerate(grown):
            key = tile * 128 + col
            kc[table[:, key // page].cpu().long(), key % page, :, 16 * i:16 * i + 16] = 9.2 / unit_score * 6
        kc, vc = kc.to(dt).cuda(), vc.to(dt).cuda()
        ke, ve = kc.double(), vc.double()
    q = torch.zeros(B * nq, hkv * G, d)
    row = torch.arange(B * nq)[:, None] * G + torch.arange(hkv * G) % G
    for i in range(blocks):
        q[..., 16 * i:16 * i + 16] += ((row % blocks) == i).unsqueeze(-1).float() * a
        q[..., 16 * i:16 * i + 16] += ((row % 3 == 0) & ((row + 1) % blocks == i)).unsqueeze(-1).float() * 2 * a
    q = q.to(dt).cuda()
    out, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, want_lse=True)
    assert sv.default_workspace().status() == 0
    ref = _reference(q, ke, ve, table, kv, new, True, 0, 0, scale)
    one = ref[1][(row % 3 != 0)]
    assert (one > math.log(2.0 ** 9 + 500)).all() and (one < math.log(2.0 ** 10.5 + 1500)).all()
    _check(out, lse, ref, dt, max(kv), d, bits)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nq", [10, 40])
def test_probabilities_are_rounded_once(sv, nq, dtype):
    """32 keys of one weight, whose f16 is half a unit above it, and behind them in the tile a key that outgrows the reference by
    so little more than 2^8 that the rescaled ones would be rounded up by half a unit again.  Only the 32 have values."""
    dt, B, G, hkv, d, page = DTYPES[dtype], 100, 4, 4, 64, 64
    L = 3 * 128 + nq
    width = -(-L // page)
    pages = B * width
    up = 1.05 * 2.0 ** -11                                        # beyond a tie of 11 bits
    weight = 7 + math.log2(1 + up)
    outgrows = 8 + math.log2((1 + 2.0 ** -10) / (1 + up))
    assert math.log2(1 + 2.0 ** -11) < weight - 7 and 8 < outgrows < 8.001
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(nq)).to(torch.int32).view(B, width).cuda()
    kcodes, vcodes = (torch.zeros(pages, page, hkv, d // 2, dtype=torch.uint8) for _ in range(2))
    kscales, vscales = (torch.full((pages, page, hkv, d // 16), 56, dtype=torch.uint8) for _ in range(2))
    at = lambda key: (table[:, key // page].cpu().long(), key % page)  # noqa: E731
    for key in range(256, 288):
        kcodes[at(key)] = torch.tensor([0x22] * 8 + [0] * 24, dtype=torch.uint8)          # 1 in the first block
        vcodes[at(key)] = torch.tensor([0x12, 0x32, 0x54, 0x76] * 8, dtype=torch.uint8)
        vscales[at(key)] = torch.tensor([56, 59, 61, 63], dtype=torch.uint8)
    kcodes[at(296)] = torch.tensor([0] * 8 + [0x22] * 8 + [0] * 16, dtype=torch.uint8)
    kc, vc = (sv.FP4Cache.of(c.cuda(), x.cuda().view(torch.float8_e4m3fn)) for c, x in ((kcodes, kscales), (vcodes, vscales)))
    q = torch.zeros(B * nq, hkv * G, d)
    q[..., :4], q[..., 4] = 1.75, weight - 7
    q[..., 16:20], q[..., 20] = 2.0, outgrows - 8
    q = q.to(dt).cuda()
    lens, cu = torch.full((B,), L, dtype=torch.int32, device="cuda"), torch.arange(B + 1, dtype=torch.int32, device="cuda") * nq
    out, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, scale=math.log(2.0), want_lse=True)
    assert sv.default_workspace().status() == 0
    ref = _reference(q, M.values(kcodes, kscales), M.values(vcodes, vscales), table, [L] * B, [nq] * B, True, 0, 0, math.log(2.0))
    _check(out, lse, ref, dt, L, d, 4)


# ------------------------------------------------------------------------------------- other calls

@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 10)])
@pytest.mark.parametrize("new,kv,hq,hkv,d", [
    ([1, 1, 2], [300, 4, 130], 128, 1, 64), ([1, 3], [260, 129], 300, 1, 64), ([1, 2], [257, 300], 130, 1, 128),   # many heads a key head
    ([2] * 900, [2 + i % 37 for i in range(900)], 4, 2, 64),                                                       # many short requests
    ([3], [400003], 4, 1, 64), ([20], [150001], 4, 1, 128), ([300], [70001], 2, 1, 64),                            # one long one
])
def test_shapes_far_from_the_usual(sv, new, kv, hq, hkv, d, window, sinks, bits):
    _run(sv, bits, "bf16", new, kv, 32, hq, hkv, d, window, sinks, seed=len(new) + hq)


@pytest.mark.parametrize("nq", [1, 9, 20, 70])
@pytest.mark.parametrize("d", [64, 80, 128])
def test_fp4_units_at_their_ends(sv, d, nq):
    """Units of 2^-64 and 2^64, with queries that bring the scores back to size, whole items and ones that CTAs share."""
    dt, new, kv = torch.bfloat16, [nq, nq], [nq + 5000, nq + 40]
    for ku, vu in ((2.0 ** -64, 2.0 ** 64), (2.0 ** 64, 2.0 ** -64)):
        (kc, vc), (ke, ve), table, lens, cu = _fp4_batch(sv, new, kv, 16, 2, d, d + nq, units=(ku, vu))
        q = (torch.randn(2 * nq, 8, d, generator=torch.Generator().manual_seed(9)) / ku).to(dt).cuda()
        out, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, want_lse=True)
        assert sv.default_workspace().status() == 0
        ref = _reference(q, ke, ve, table, kv, new, True, 0, 0, d ** -0.5)
        _check(out, lse, ref, dt, max(kv), d, 4)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("nq", [1, 5, 20, 70])
def test_strided_queries_and_rows_of_nobody(sv, nq, bits):
    """Queries that are part of one projection's output, rows behind the last request's: those of out, lse, q_out and the
    cache stay as they were."""
    hq, hkv, d, page, more = 8, 2, 128, 16, 3
    new, kv = [nq, 0, nq], [nq + 77, 9, nq + 200]
    if bits == 4:
        (kc, vc), _, table, lens, cu = _fp4_batch(sv, new, kv, page, hkv, d, 5)
    else:
        kc, vc, table, lens, cu = _batch(new, kv, page, hkv, d, torch.bfloat16, 5, "hnd")
    qkv = torch.randn(2 * nq + more, hq + 2 * hkv, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q = qkv[:, :hq]
    out = torch.full((2 * nq + more, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    sv.chunk_attention(q, kc, vc, table, lens, cu, nq, out=out)
    want = sv.chunk_attention(q[:2 * nq].contiguous(), kc, vc, table, lens, cu, nq)
    assert torch.equal(out[:2 * nq], want) and (out[2 * nq:] == 7.0).all()
    plan, q_out = sv.RopePlan(d), torch.full_like(out, 7.0)
    held = lambda: [t.clone() for c in (kc, vc) for t in ((c.codes, c.scales.view(torch.uint8)) if bits == 4 else (c.nan_to_num(),))]  # noqa: E731
    sv.rope_append(q, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], plan, kc, vc, table, lens, cu, q_out=q_out)
    first = held()
    part = [x[:2 * nq].contiguous() for x in (q, qkv[:, hq:hq + hkv], qkv[:, hq + hkv:])]
    want = sv.rope_append(*part, plan, kc, vc, table, lens, cu)
    assert torch.equal(q_out[:2 * nq], want) and (q_out[2 * nq:] == 7.0).all()
    assert all(torch.equal(a, b) for a, b in zip(first, held()))
    assert sv.default_workspace().status() == 0


def test_two_graphs_over_one_workspace(sv):
    """Replayed by turns, with other lengths in between: a graph finds nothing of the other's in the workspace."""
    d, page = 128, 16
    (kc, vc), (ke, ve), table, lens, cu = _fp4_batch(sv, [40, 40], [3000, 700], page, 2, d, 2)
    (k1, v1), (e1, f1), table1, lens1, cu1 = _fp4_batch(sv, [1] * 5, [900, 30, 500, 2000, 0], page, 2, d, 3)
    q, q1 = torch.randn(80, 8, d).bfloat16().cuda(), torch.randn(5, 8, d).bfloat16().cuda()
    ws = sv.Workspace()
    out, out1 = torch.empty_like(q), torch.empty_like(q1)
    pool = sv.PagePool([], pages=300)
    pages, n, moved, packed, used = table.clone(), lens.clone(), table.clone(), table.clone(), lens[:1].clone()
    def first():
        sv.chunk_attention(q, kc, vc, table, lens, cu, 40, out=out, workspace=ws)
        sv.assign_pages(pool, pages, n, page, kept=n, out=moved, workspace=ws)
    def second():
        sv.compact_pages(pool, moved, out=packed, used=used, workspace=ws)
        sv.chunk_attention(q1, k1, v1, table1, lens1, cu1, 1, out=out1, workspace=ws)
    graphs = []
    for f in (first, second):
        f()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for a, b in ((2500, 680), (41, 60), (3000, 700)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        out.fill_(9.0), out1.fill_(9.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sv.chunk_attention(q, kc, vc, table, lens, cu, 40))
        assert torch.equal(out1, sv.chunk_attention(q1, k1, v1, table1, lens1, cu1, 1))
        want, copies, ok = M.assign(pages.tolist(), n.tolist(), page, 300, n.tolist())
        assert ok and moved.tolist() == want and packed.tolist() == M.compact(want, 300)[0]
    assert ws.status() == 0
