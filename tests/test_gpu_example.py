"""The speculative decoding example: the operators together, as a program uses them."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_speculative_sampling_runs():
    import speculative_step as ex
    tokens, accepted = ex.decode(steps=4, K=3, B=3)
    assert len(accepted) == 12 and 0 <= min(accepted) and max(accepted) <= 3
    assert [len(t) for t in tokens] == [sum(a + 1 for a in accepted[b::3]) for b in range(3)]
    assert all(0 <= x < 2000 for t in tokens for x in t)


def test_greedy_speculation_gives_the_target_s_own_tokens():
    import speculative_step as ex
    got, accepted = ex.decode(steps=5, K=3, B=3, T=0.0, top_p=1.0, noise=0.02)
    want, _ = ex.decode(steps=max(len(t) for t in got), K=3, B=3, speculative=False)
    assert sum(accepted) > 0
    for g, w in zip(got, want):
        assert g == w[: len(g)]
