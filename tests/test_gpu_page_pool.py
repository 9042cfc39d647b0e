"""The pages of a cache: assign_pages and compact_pages against plain forms (lists), and what they copy."""
import random

import pytest
import torch

from tests import more_reference as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import draft_verification_spec_gb300 as m
    m.lib()
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _caches(sv, pages, page, seed=0):
    """Arrays of several shapes and alignments: 16-bit ones of two layouts, one of odd rows, a 4-bit one, a slice of a wider one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    a = torch.randn(pages, page, 2, 64, generator=g, device="cuda").bfloat16()
    b = torch.randn(pages, 3, page, 40, generator=g, device="cuda").half().transpose(1, 2)
    odd = byte(pages, page, 1, 3)
    four = sv.FP4Cache.of(byte(pages, 2, page, 24).transpose(1, 2), byte(pages, 2, page, 3).view(torch.float8_e4m3fn).transpose(1, 2))
    wide = torch.randn(pages, 2, page, 5, generator=g, device="cuda")[:, 1]
    return [a, b, odd, four, wide]


def _tensors(caches):
    return [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for c in caches
            for t in ((c.codes, c.scales) if hasattr(c, "codes") else (c,))]


def _copied(before, caches, copies):
    for x, y in zip(before, _tensors(caches)):
        want = x.clone()
        for s, d in copies:
            want[d] = x[s]
        assert torch.equal(y, want)


def _table(rng, rows, width, pages, page, lens):
    ids = rng.sample(range(pages), pages)
    table = [[-1] * width for _ in range(rows)]
    for b in range(rows):
        for j in range(-(-lens[b] // page)):
            table[b][j] = ids.pop()
    return table


def _assign(sv, table, lens, page, pages, kept, parents=None, strided=False):
    caches = _caches(sv, pages, page)
    before = [t.clone() for t in _tensors(caches)]
    pool = sv.PagePool(caches)
    t = _i32(table)
    if strided:
        wide = torch.full((t.shape[0], t.shape[1] + 3), -7, dtype=torch.int32, device="cuda")
        wide[:, 1:1 + t.shape[1]] = t
        t = wide[:, 1:1 + t.shape[1]]
    out = sv.assign_pages(pool, t, _i32(lens), page, kept=_i32(kept), parents=None if parents is None else _i32(parents))
    want, copies, ok = M.assign(table, lens, page, pages, kept, parents)
    assert sv.default_workspace().status() == (0 if ok else 7)
    assert out.tolist() == want
    assert torch.equal(t.cpu(), torch.tensor(table, dtype=torch.int32))
    _copied(before, caches, copies)
    return copies


@pytest.mark.parametrize("page", [1, 3, 16])
@pytest.mark.parametrize("rows,width,pages", [(1, 1, 1), (1, 4, 7), (5, 9, 60), (70, 3, 400), (300, 2, 700), (3, 300, 1000), (1500, 2, 3300)])
def test_assign_steps(sv, rows, width, pages, page):
    """Between two steps: some tokens dropped, some more wanted, requests that end and begin."""
    for seed in range(3):
        rng = random.Random(seed)
        most = min(width * page, max(1, pages // rows) * page)
        lens = [rng.randint(0, most) for _ in range(rows)]
        table = _table(rng, rows, width, pages, page, lens)
        kept = [max(0, n - rng.randint(0, 5)) if rng.random() < 0.8 else 0 for n in lens]
        after = [min(width * page, k + rng.randint(0, 7)) if rng.random() < 0.9 else 0 for k in kept]
        _assign(sv, table, after, page, pages, kept, strided=seed == 1)


@pytest.mark.parametrize("page", [1, 4, 16])
def test_assign_forks(sv, page):
    """Requests that go on from others': whole pages shared, the last one copied for all but one; a beam reordered."""
    copies = 0
    for seed in range(12):
        rng = random.Random(seed)
        rows, width, pages = rng.choice([2, 9, 40]), rng.choice([2, 7, 33]), 2000
        lens = [rng.randint(0, width * page) for _ in range(rows)]
        table = _table(rng, rows, width, pages, page, lens)
        parents = [rng.randrange(-1, rows) if rng.random() < 0.9 else rows for _ in range(rows)]
        kept = [rng.randint(0, lens[p]) if 0 <= p < rows else 5 for p in parents]
        after = [min(width * page, max(0, k + rng.randint(-2, 2 * page))) for k in kept]
        copies += len(_assign(sv, table, after, page, pages, kept, parents))
    assert copies > 0 or page == 1


def test_assign_a_page_that_one_reads_and_another_writes(sv):
    """Row 1 has the page whole, row 0 and 2 want to write behind its third token: both get a copy."""
    assert _assign(sv, [[4, 2], [4, 2], [4, -1]], [5, 8, 4], 4, 12, [3, 4, 3], [0, 0, 0]) == [(4, 0), (4, 3)]
    # the same page twice in a row, and the same parent twice
    _assign(sv, [[3, 3, 5], [3, 5, 5]], [9, 10], 4, 12, [9, 6], [0, 0])


def test_assign_of_what_is_not_there(sv):
    """Too few free pages, rows longer than the table, inherited entries outside the pool: -1, nothing copied, reported."""
    _assign(sv, [[0, 1], [2, -1]], [8, 8], 4, 4, [8, 3])                       # fits exactly
    _assign(sv, [[0, 1], [2, -1]], [8, 8], 4, 3, [8, 3])                       # one too few
    _assign(sv, [[0, -1], [-1, -1]], [3, 3], 4, 1, [2, 2], [0, 0])             # none left for the copy
    _assign(sv, [[0, 1], [2, -1]], [9, 100], 4, 9, [8, 4])                     # beyond the columns
    _assign(sv, [[0, 99], [-5, 3]], [8, 8], 4, 9, [8, 7])                      # nobody's pages
    _assign(sv, [[0, 1], [2, 3]], [-3, 2 ** 31 - 1], 4, 9, [-1, 2 ** 31 - 1])
    _assign(sv, [[0, 1], [2, 3]], [0, 0], 4, 9, [8, 8])                        # all freed


def test_assign_of_nothing(sv):
    pool = sv.PagePool(_caches(sv, 3, 4))
    for shape in ((0, 4), (3, 0)):
        t = torch.zeros(shape, dtype=torch.int32, device="cuda")
        n = torch.zeros(shape[0], dtype=torch.int32, device="cuda")
        assert sv.assign_pages(pool, t, n, 4, kept=n).shape == shape
        out, used = sv.compact_pages(pool, t)
        assert out.shape == shape and used.tolist() == [0]
    bare = sv.PagePool([], pages=5)      # a table without caches
    out = sv.assign_pages(bare, _i32([[4, -1]]), _i32([9]), 8, kept=_i32([3]))
    assert out.tolist() == [[4, 0]]
    assert sv.compact_pages(bare, out)[0].tolist() == [[1, 0]]


def _compact(sv, table, pages, page=4):
    caches = _caches(sv, pages, page)
    before = [t.clone() for t in _tensors(caches)]
    out, used = sv.compact_pages(sv.PagePool(caches), _i32(table))
    want, u, copies = M.compact(table, pages)
    bad = any(p != -1 and not 0 <= p < pages for row in table for p in row)
    assert sv.default_workspace().status() == (7 if bad else 0)
    assert out.tolist() == want and used.tolist() == [u]
    _copied(before, caches, copies)


@pytest.mark.parametrize("rows,width,pages", [(1, 1, 1), (2, 3, 6), (4, 9, 50), (60, 5, 1100), (3, 400, 5000)])
def test_compact(sv, rows, width, pages):
    for load in (0.0, 0.1, 0.5, 0.9, 1.0):
        rng = random.Random(pages * load)
        ids = rng.sample(range(pages), min(int(pages * load), rows * width))
        flat = ids + [-1] * (rows * width - len(ids))
        rng.shuffle(flat)
        table = [flat[b * width:(b + 1) * width] for b in range(rows)]
        _compact(sv, table, pages)
    shared = [[rng.randrange(pages) for _ in range(width)] for _ in range(rows)]     # pages in several rows
    _compact(sv, shared, pages)


def test_compact_ignores_and_reports_other_pages(sv):
    _compact(sv, [[7, 99, -2], [-1, 9, 7]], 12)


def test_pages_of_a_large_pool(sv):
    """More pages than a CTA's threads several times over, and copies of pages that are several chunks long."""
    pages, rows, width = 300007, 9, 4000
    rng = random.Random(5)
    ids = rng.sample(range(pages), rows * width)
    table = [ids[b * width:(b + 1) * width] for b in range(rows)]
    bare = sv.PagePool([], pages=pages)
    out, used = sv.compact_pages(bare, _i32(table))
    want, u, _ = M.compact(table, pages)
    assert out.tolist() == want and used.tolist() == [u]
    kept = [rng.randrange(width * 16) for _ in range(rows)]
    lens = [min(width * 16, k + rng.randrange(2000)) for k in kept]
    parents = [rng.randrange(rows) for _ in range(rows)]
    out = sv.assign_pages(bare, _i32(table), _i32(lens), 16, kept=_i32(kept), parents=_i32(parents))
    want, _, ok = M.assign(table, lens, 16, pages, kept, parents)
    assert ok and out.tolist() == want and sv.default_workspace().status() == 0
    big = torch.randn(6, 50001, device="cuda")      # 200,004 bytes a page: 13 chunks, 4-byte aligned
    before = big.clone()
    out, _ = sv.compact_pages(sv.PagePool([big]), _i32([[5, 3, 0]]))
    assert out.tolist() == [[2, 1, 0]]
    assert torch.equal(big[1], before[3]) and torch.equal(big[2], before[5]) and torch.equal(big[3:], before[3:])


def test_pages_beyond_32_bit_offsets(sv):
    big = torch.zeros(5, 2 ** 30 + 16, dtype=torch.uint8, device="cuda")
    big[4, -64:] = torch.arange(64, dtype=torch.uint8, device="cuda")
    big[4, :64] = 7
    out, used = sv.compact_pages(sv.PagePool([big]), _i32([[4, 0]]))
    assert out.tolist() == [[1, 0]] and used.tolist() == [2]
    assert torch.equal(big[1], big[4])


def test_pages_repeat_graph_and_stream(sv):
    rng = random.Random(1)
    table = _table(rng, 6, 20, 200, 16, [320] * 6)
    caches = _caches(sv, 200, 16)
    pool, t = sv.PagePool(caches), _i32(table)
    lens, kept, parents = _i32([100, 40, 300, 0, 17, 16]), _i32([90, 40, 290, 0, 16, 15]), _i32([0, 0, 2, 3, 2, 0])
    call = lambda **kw: sv.assign_pages(pool, t, lens, 16, kept=kept, parents=parents, **kw)  # noqa: E731
    want = call()
    assert torch.equal(want, call())
    ws, out, packed, used = sv.Workspace(), torch.empty_like(want), torch.empty_like(want), torch.empty_like(lens[:1])
    call(out=out, workspace=ws)
    sv.compact_pages(pool, out, out=packed, used=used, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=out, workspace=ws)
        sv.compact_pages(pool, out, out=packed, used=used, workspace=ws)
    lens.copy_(_i32([10, 41, 310, 5, 0, 16]))
    before = [x.clone() for x in _tensors(caches)]
    g.replay()
    torch.cuda.synchronize()
    new, copies, _ = M.assign(table, lens.tolist(), 16, 200, kept.tolist(), parents.tolist())
    final, u, moves = M.compact(new, 200)
    assert out.tolist() == new and packed.tolist() == final and used.tolist() == [u] and ws.status() == 0
    for x, y in zip(before, _tensors(caches)):
        z = x.clone()
        for s, d in copies:
            z[d] = x[s]
        zz = z.clone()
        for s, d in moves:
            zz[d] = z[s]
        assert torch.equal(y, zz)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert got.tolist() == new


def test_pages_and_attention_share_a_workspace(sv):
    """Calls that leave records in one workspace, one behind the other."""
    d, page = 64, 16
    kc, vc = (torch.randn(40, page, 2, d, device="cuda").bfloat16() for _ in range(2))
    table = _i32([list(range(20)), list(range(20, 40))])
    lens, cu = _i32([300, 320]), _i32([0, 1, 2])
    q = torch.randn(2, 4, d, device="cuda").bfloat16()
    ws = sv.Workspace()
    want = sv.chunk_attention(q, kc, vc, table, lens, cu, 1, workspace=ws)
    pool = sv.PagePool([kc, vc])
    for _ in range(5):
        packed, _ = sv.compact_pages(pool, table, workspace=ws)
        assert torch.equal(packed, table)
        assert torch.equal(want, sv.chunk_attention(q, kc, vc, packed, lens, cu, 1, workspace=ws))
    assert ws.status() == 0


def test_page_refusals(sv):
    caches = _caches(sv, 6, 4)
    for bad in ([caches[0], torch.zeros(7, 2, device="cuda")], [caches[0], torch.zeros(6, 2)],
                [torch.zeros(6, 4, 4, device="cuda")[:, :, :2]], [torch.zeros(1, 4, device="cuda").expand(6, 4)], []):
        with pytest.raises(ValueError):
            sv.PagePool(bad)
    pool, t, n = sv.PagePool(caches), _i32([[0, 1], [2, 3]]), _i32([4, 4])
    for err, kw in ((TypeError, dict(t=t.long())), (ValueError, dict(t=t[0])), (ValueError, dict(t=t.t().contiguous().t())),
                    (ValueError, dict(t=t.cpu())), (ValueError, dict(n=n[:1])), (ValueError, dict(kept=n.long())),
                    (ValueError, dict(parents=n.cpu())), (ValueError, dict(out=t)), (ValueError, dict(out=t[:1])),
                    (sv.SpecError, dict(page=0)), (sv.SpecError, dict(page=-2 ** 40))):
        a = dict(t=t, n=n, kept=n, page=4)
        a.update(kw)
        with pytest.raises(err):
            sv.assign_pages(pool, a["t"], a["n"], a["page"], kept=a["kept"], parents=a.get("parents"), out=a.get("out"))
    with pytest.raises(ValueError):
        sv.compact_pages(pool, t, out=t)
    with pytest.raises(ValueError):
        sv.compact_pages(pool, t, used=n)
