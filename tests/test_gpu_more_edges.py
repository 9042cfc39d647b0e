"""Edges of the operators on pages, caches in 4 bits and first tokens that the other files do not reach, vs float64."""
import math

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
