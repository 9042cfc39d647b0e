"""Edges of the operators on pages, caches in 4 bits and first tokens that the other files do not reach, vs float64."""
import math

import pytest
import torch

from tests.test_gpu_more_ops import _append

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
