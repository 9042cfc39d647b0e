"""The operators on pages, caches in 4 bits and first tokens together, as a serving loop uses them."""
import os
import random
import sys
import zlib

import pytest
import torch

from tests import more_reference as M
from tests.test_gpu_more_ops import _check

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE = 8, 2, 64, 16


@pytest.fixture(scope="module")
def sv():
    import draft_verification_spec_gb300 as m
    m.lib()
    return m


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _token(history, pos):
    """q, k, v of a token: the same for all requests that share the history."""
    g = torch.Generator().manual_seed(zlib.crc32(repr((history, pos)).encode()))
    return torch.randn(HQ + 2 * HKV, D, generator=g)


def _append(sv, caches, plan, histories, kv, new, table):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    x = torch.stack([_token(histories[b], kv[b] - new[b] + i) for b in range(len(kv)) for i in range(new[b])]).bfloat16().cuda()
    lens, cu = _i32(kv), _i32(cu)
    q = sv.rope_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], plan, *caches, table, lens, cu)
    return q, lens, cu


def _caches(sv, bits, pages):
    if bits == 4:
        return [sv.FP4Cache(pages, PAGE, HKV, D) for _ in range(2)]
    return [torch.full((pages, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 5)])
def test_shared_pages_change_no_bit(sv, bits, window, sinks):
    """Prompts, forks, steps with rejected drafts, requests that end, compactions: over a pool of shared pages and
    over caches in which every request has pages of its own, the rows are equal bit for bit."""
    rng = random.Random(bits + window)
    B, width = 6, 20
    plan = sv.RopePlan(D)
    shared, alone = _caches(sv, bits, 70), _caches(sv, bits, B * width)
    fixed = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    pool = sv.PagePool(shared)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")

    def both(histories, kv, new):
        outs = []
        for caches, t in ((shared, table), (alone, fixed)):
            q, lens, cu = _append(sv, caches, plan, histories, kv, new, t)
            outs.append(sv.chunk_attention(q, *caches, t, lens, cu, max(new), window=window, sinks=sinks, want_lse=True))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        return outs[0]

    # two prompts, in rows 0 and 1
    kv, hist = [70, 45, 0, 0, 0, 0], [("p", 0), ("p", 1)] + [("none", b) for b in range(2, B)]
    table = sv.assign_pages(pool, table, _i32(kv), PAGE, kept=_i32([0] * B))
    both(hist, kv, kv)
    # forked into six: three of each; the pages that the prompts end in are copied for four of them
    parents = [0, 0, 0, 1, 1, 1]
    kept = [kv[p] for p in parents]
    kv = [k + 3 for k in kept]
    before = int((table >= 0).sum())
    table = sv.assign_pages(pool, table, _i32(kv), PAGE, kept=_i32(kept), parents=_i32(parents))
    assert len(set(table[table >= 0].tolist())) < before + 4 * 2 + 2
    # the other world reads the prompts again
    q, _, _ = _append(sv, alone, plan, [hist[p] for p in parents], kept, kept, fixed)
    hist = [(hist[p], b) for b, p in enumerate(parents)]
    both(hist, kv, [3] * B)
    for step in range(8):
        kept = [k - rng.randint(0, 2) for k in kv]               # rejected drafts
        if step == 4:
            kept[2] = 0                                           # a request ends, another one begins in its place
            hist[2] = ("p", 9)
        new = [rng.randint(1, 3) if k else 20 for k in kept]
        hist = [(h, step) for h in hist]
        kv = [k + n for k, n in zip(kept, new)]
        table = sv.assign_pages(pool, table, _i32(kv), PAGE, kept=_i32(kept))
        if step % 3 == 2:
            table, used = sv.compact_pages(pool, table)
            assert int(table.max()) < int(used)
        got, lse = both(hist, kv, new)
    assert sv.default_workspace().status() == 0
    # and they are the rows of the definition, over what the cache holds
    held = [c.values(torch.float32).cpu().double() if bits == 4 else c.cpu().double() for c in shared]
    q, lens, cu = _append(sv, shared, plan, hist, kv, new, table)
    ref = M.attention(q, *held, table, lens, cu, True, window, sinks, D ** -0.5)
    _check(got, lse, ref, torch.bfloat16, max(kv), D, bits)


@pytest.mark.parametrize("bits", [4, 16])
def test_the_example_runs(bits):
    import parallel_samples as ex
    out, (shared, held, used) = ex.decode(prompts=2, samples=3, steps=10, bits=bits)
    assert len(out) == 6 and all(1 <= len(t) <= 10 and all(0 <= x < 500 for x in t) for t in out)
    assert shared == 3 + 4 and used == held
