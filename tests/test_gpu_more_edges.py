"""Edges of the operators on pages, caches in 4 bits and first tokens that the other files do not reach, vs float64."""
import math
import random
import threading

import pytest
import torch

from tests import more_reference as M
from tests.test_gpu_more_ops import _append, _check, _fp4_batch
from tests.test_gpu_step_ops import _batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import draft_verification_spec_gb300 as m
    m.lib()
    return m


# ------------------------------------------------------------------------ the write into 4 bits

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rotary", [(64, 32), (64, 8), (16, 8), (256, 2), (80, 40), (128, 64), (96, 48)])
def test_append_nan_behind_the_rotated_part(sv, d, rotary, layout, dtype):
    """A NaN, and a negative zero beside it, in values that are not rotated: blocks of their own and ones that the rotated part
    ends in.  There is no frequency for them."""
    def make(k, v):
        k[:, 0, -1], k[:, 0, -2] = math.nan, -0.0
        k[2:, 1, rotary], k[2:, 1, rotary + 1] = math.nan, -0.0
        k[4, :, rotary:] = math.nan
    _append(sv, [6], [900], 16, 2, 2, d, dtype=dtype, rotary=rotary, layout=layout, make=make, seed=d + rotary)


# ------------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 9)])
@pytest.mark.parametrize("nq,hq,d", [(1, 4, 64), (3, 4, 128), (9, 8, 80), (20, 8, 64), (20, 8, 128), (70, 8, 128), (30, 4, 256)])
def test_nan_keys_are_no_empty_rows(sv, nq, hq, d, window, sinks, bits):
    """A NaN among a row's scores: NaN in out and lse.  -inf stands for rows without keys alone; rows that do not see the NaN are
    those of the definition."""
    new, kv, page, hkv = [nq, nq, nq], [nq + 200, nq + 31, 0], 16, 2
    if bits == 4:
        (kc, vc), (ke, ve), table, lens, cu = _fp4_batch(sv, new, kv, page, hkv, d, 7)
    else:
        kc, vc, table, lens, cu = _batch(new, kv, page, hkv, d, torch.bfloat16, 7, "hnd")
        ke, ve = kc.cpu().double(), vc.cpu().double()
    q = torch.randn(3 * nq, hq, d, generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    ref = M.attention(q, ke, ve, table, lens, cu, True, window, sinks, d ** -0.5)
    at = kv[0] - nq // 2 - 1                # a key of the first request that its later new tokens alone see
    where = (table[0, at // page].item(), at % page)
    if bits == 4:
        kc.scales.view(torch.uint8)[where] = 127
    else:
        kc[where] = math.nan
    out, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, window=window, sinks=sinks, want_lse=True)
    assert sv.default_workspace().status() == 0
    seen = torch.arange(3 * nq) < nq
    seen &= torch.arange(3 * nq) + kv[0] - nq >= at
    assert seen.any() and torch.isnan(lse[seen.cuda()]).all() and torch.isnan(out[seen.cuda()]).all()
    rest = [x[~seen] for x in ref]
    assert torch.isinf(rest[1]).any()
    _check(out[~seen.cuda()], lse[~seen.cuda()], rest, torch.bfloat16, max(kv), d, bits)


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 6), (200, 33), (130, 0)])
@pytest.mark.parametrize("nq,hq", [(1, 4), (4, 8), (10, 4), (17, 8), (70, 8)])
def test_fp4_pages_behind_the_window_may_be_gone(sv, nq, hq, window, sinks, d, layout):
    """No bit changes where pages that no new token sees are unmapped or hold anything."""
    new, kv, page, hkv = [nq, nq], [nq + 500, nq + 90], 16, 2
    (kc, vc), _, table, lens, cu = _fp4_batch(sv, new, kv, page, hkv, d, nq + window, layout)
    q = torch.randn(2 * nq, hq, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    call = lambda t: sv.chunk_attention(q, kc, vc, t, lens, cu, nq, window=window, sinks=sinks, want_lse=True)  # noqa: E731
    want = call(table)
    gone = table.clone()
    for b, k in enumerate(kv):
        behind = max(0, k - new[b] - window + 1) // page
        pages = range(-(-sinks // page), behind)
        for j in pages:
            kc.scales.view(torch.uint8)[table[b, j].item()] = 127
            vc.scales.view(torch.uint8)[table[b, j].item()] = 127
        if pages:
            gone[b, pages.start:pages.stop] = -1
    assert (gone != table).any()
    for t in (gone, table):
        got = call(t)
        assert sv.default_workspace().status() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("nq", [1, 17])
def test_fp4_codes_beyond_2_to_the_32(sv, nq):
    """A cache of more than 2^32 bytes of codes: what a 32-bit offset would find in a page's place is another page's."""
    page, hkv, d = 16, 8, 128
    size = page * hkv * d // 2
    wrap = 2 ** 32 // size
    pages = wrap + 40
    far = [sv.FP4Cache(pages, page, hkv, d) for _ in range(2)]
    assert far[0].codes.stride(0) == size and pages * size > 2 ** 32
    (kc, vc), _, _, _, _ = _fp4_batch(sv, [1], [60], page, hkv, d, 3)
    (kx, vx), _, _, _, _ = _fp4_batch(sv, [1], [60], page, hkv, d, 4)
    ids = torch.tensor([wrap + 3, wrap - 1, 7, wrap + 20], device="cuda")
    low = torch.tensor([3, 5, wrap + 7, 20], device="cuda")      # the same bytes modulo 2^32, and others
    byte = lambda c: c.scales.view(torch.uint8)  # noqa: E731
    for f, c, x in zip(far, (kc, vc), (kx, vx)):
        for y in (c, x):
            byte(y)[byte(y) == 127] = 50
        f.codes[low], byte(f)[low] = x.codes[:4], byte(x)[:4]
        f.codes[ids], byte(f)[ids] = c.codes[:4], byte(c)[:4]
    near, table = torch.arange(4, dtype=torch.int32, device="cuda")[None], ids.int()[None]
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([60], [0, nq]))
    q = torch.randn(nq, 16, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    for kw in (dict(), dict(scale=-0.2), dict(window=20, sinks=3)):
        assert torch.equal(sv.chunk_attention(q, *far, table, lens, cu, nq, **kw),
                           sv.chunk_attention(q, kc, vc, near, lens, cu, nq, **kw))
    plan, k = sv.RopePlan(d), torch.randn(nq, hkv, d, device="cuda").bfloat16()
    sv.rope_append(q, k, k, plan, *far, table, lens, cu)
    sv.rope_append(q, k, k, plan, kc, vc, near, lens, cu)
    for f, c, x in zip(far, (kc, vc), (kx, vx)):
        assert torch.equal(f.codes[ids], c.codes[:4]) and torch.equal(byte(f)[ids], byte(c)[:4])
        assert torch.equal(f.codes[low], x.codes[:4]) and torch.equal(byte(f)[low], byte(x)[:4])
    assert sv.default_workspace().status() == 0


@pytest.mark.parametrize("nq", [1, 17])
def test_fp4_scales_beyond_2_to_the_32(sv, nq):
    """Rows of scales in pages so far apart that their own offsets pass 32 bits."""
    page, hkv, d, apart = 16, 2, 128, 3 * 2 ** 29
    (kc, vc), _, table, lens, cu = _fp4_batch(sv, [nq], [nq + 40], page, hkv, d, 6)
    assert kc.shape[0] * apart > 2 ** 32
    q = torch.randn(nq, 4, d, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    k = torch.randn(nq, hkv, d, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    wide = []
    for c in (kc, vc):
        room = torch.zeros((kc.shape[0] - 1) * apart + page * hkv * d // 16, dtype=torch.uint8, device="cuda")
        s = room.as_strided(c.scales.shape, (apart, hkv * d // 16, d // 16, 1))
        s.copy_(c.scales.view(torch.uint8))
        wide.append(sv.FP4Cache.of(c.codes.clone(), s.view(torch.float8_e4m3fn)))
    for kw in (dict(), dict(window=20, sinks=3)):
        ref, lse = sv.chunk_attention(q, kc, vc, table, lens, cu, nq, want_lse=True, **kw)
        got, lse2 = sv.chunk_attention(q, *wide, table, lens, cu, nq, want_lse=True, **kw)
        assert sv.default_workspace().status() == 0
        # two kernels' roundings of the same numbers: the output's in each, the probabilities' and the fp32 part
        assert (got.double() - ref.double()).abs().max() <= 4 * 2.0 ** -8 * ref.double().abs().max()
        assert (lse - lse2).abs().max() <= 1e-4
    for caches in ((kc, vc), wide):
        sv.rope_append(q, k, k, sv.RopePlan(d), *caches, table, lens, cu)
    for c, w in zip((kc, vc), wide):
        assert torch.equal(c.codes, w.codes) and torch.equal(c.scales.view(torch.uint8), w.scales.view(torch.uint8))
        assert torch.equal(c.values().nan_to_num(), w.values().nan_to_num())


# ------------------------------------------------------------------------------------------ pages

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_pages_from_several_threads(sv):
    """Threads with a pool each, on streams of their own and on the same one, in one workspace and in their streams': plans and
    copies are each thread's own."""
    shared_stream, shared_ws = torch.cuda.Stream(), sv.Workspace()
    failed = []

    def work(n):
        try:
            rng = random.Random(n)
            own = n % 2 == 0
            side = torch.cuda.Stream() if own else shared_stream
            kw = dict(stream=side) if own else dict(stream=side, workspace=shared_ws)
            rows, width, page, pages = 5 + n, 30, 16, 400
            ids = rng.sample(range(pages), rows * width // 2)
            lens = [rng.randint(1, width // 2 * page) for _ in range(rows)]
            table = [[ids.pop() if j < -(-x // page) else -1 for j in range(width)] for x in lens]
            data = torch.randint(0, 255, (pages, 3001 + n), dtype=torch.uint8, device="cuda")
            pool = sv.PagePool([data])
            for step in range(6):
                parents = [rng.randrange(rows) for _ in range(rows)]
                kept = [rng.randint(0, lens[p]) for p in parents]
                after = [min(width // 2 * page, k + rng.randint(0, 40)) for k in kept]
                before, args = data.clone(), [_i32(x) for x in (table, after, kept, parents)]
                torch.cuda.current_stream().synchronize()
                out = sv.assign_pages(pool, args[0], args[1], page, kept=args[2], parents=args[3], **kw)
                packed, used = sv.compact_pages(pool, out, **kw)
                side.synchronize()
                want, copies, ok = M.assign(table, after, page, pages, kept, parents)
                final, u, moves = M.compact(want, pages)
                assert ok and out.tolist() == want and packed.tolist() == final and used.tolist() == [u]
                for some in (copies, moves):
                    x = before.clone()
                    for s, d in some:
                        x[d] = before[s]
                    before = x
                assert torch.equal(before, data)
                table, lens = final, after
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(6)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed
    assert shared_ws.status() == 0


def test_one_pool_on_two_streams(sv):
    """Steps that go to two streams by turns, each behind the other, change no bit."""
    pages, page, width = 64, 8, 20
    data = torch.randint(0, 255, (pages, 4096), dtype=torch.uint8, device="cuda")
    pool, streams = sv.PagePool([data]), [torch.cuda.Stream(), torch.cuda.Stream()]
    table, lens = [[3, 9, -1] + [-1] * (width - 3), [50] + [-1] * (width - 1), [-1] * width], [13, 8, 0]
    now, before = _i32(table), data.clone()
    torch.cuda.synchronize()
    last = None
    for step in range(12):
        side = streams[step % 2]
        kept = [max(0, n - step % 3) for n in lens]
        parents = [0, 1, step % 2] if step % 4 == 0 else [0, 1, 2]
        kept[2] = kept[parents[2]]
        after = [k + 5 for k in kept]
        with torch.cuda.stream(side):
            args = [_i32(x) for x in (after, kept, parents)]
        if last is not None:
            side.wait_stream(last)
        now = sv.assign_pages(pool, now, args[0], page, kept=args[1], parents=args[2], stream=side)
        now, used = sv.compact_pages(pool, now, stream=side)
        last = side
        table, copies, ok = M.assign(table, after, page, pages, kept, parents)
        assert ok
        table, u, moves = M.compact(table, pages)
        for some in (copies, moves):
            x = before.clone()
            for s, d in some:
                x[d] = before[s]
            before = x
        lens = after
    torch.cuda.synchronize()
    assert now.tolist() == table and used.tolist() == [u] and torch.equal(data, before)


def test_accepted_drafts_decide_what_is_kept(sv):
    """A verification's counts go to assign_pages on the device: a request keeps its tokens up to the last accepted draft, and
    has room for the next chain."""
    B, K, V, page, width = 7, 4, 300, 8, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    data = torch.randint(0, 255, (B * width, 100), dtype=torch.uint8, device="cuda")
    pool = sv.PagePool([data])
    table, lens = [[-1] * width for _ in range(B)], [0] * B
    start = [3 + 5 * b for b in range(B)]
    now = sv.assign_pages(pool, _i32(table), _i32(start), page, kept=_i32(lens))
    table, _, _ = M.assign(table, start, page, B * width, lens)
    length, lens = _i32(start), start
    seen = set()
    for _ in range(5):
        draft = torch.randn(B, K, V, generator=g, device="cuda")
        target = torch.randn(B, K + 1, V, generator=g, device="cuda") * 0.3
        target[:, :K] += draft
        tokens = draft.softmax(-1).flatten(0, 1).multinomial(1, generator=g).view(B, K).int()
        # the chain's K + 1 tokens get their slots, then the counts say which of them stay
        room = sv.assign_pages(pool, now, length + K + 1, page, kept=length)
        accepted = sv.verify_chain(target, draft, tokens, torch.rand(B, K + 1, generator=g, device="cuda"), 1.0).accepted
        kept = length + accepted + 1
        now = sv.assign_pages(pool, room, kept, page, kept=kept)
        table, _, ok = M.assign(table, [n + K + 1 for n in lens], page, B * width, lens)
        assert ok and room.tolist() == table
        counts = accepted.tolist()
        seen |= set(counts)
        lens = [n + a + 1 for n, a in zip(lens, counts)]
        table, copies, ok = M.assign(table, lens, page, B * width, lens)
        assert ok and not copies and now.tolist() == table and all(0 <= a <= K for a in counts)
        length = kept
    assert len(seen) > 1 and sv.default_workspace().status() == 0
