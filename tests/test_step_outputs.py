"""Whether an output of the step operators shares memory with an input, against a count of the addresses."""
import pytest
import torch

from draft_verification_spec_gb300 import step


def _addresses(t):
    rows, V = t.shape
    return {t.data_ptr() + (r * t.stride(0) + c) * t.element_size() for r in range(rows) for c in range(V)}


@pytest.mark.parametrize("rows", [0, 1, 2, 3])
@pytest.mark.parametrize("V", [1, 3, 4])
def test_overlap_is_what_the_addresses_say(rows, V):
    store = torch.zeros(64)
    for sa in range(V, 2 * V + 3):
        for at in range(0, 40):
            a, b = (torch.as_strided(store, (rows, V), (sa, 1), o) for o in (20, at))
            assert step._overlap(a, b) == bool(_addresses(a) & _addresses(b)), (sa, at)


def test_overlap_of_rows_with_other_strides_is_refused_where_their_ranges_meet():
    store = torch.zeros(200)
    a = torch.as_strided(store, (3, 4), (10, 1), 0)
    assert step._overlap(a, torch.as_strided(store, (3, 4), (11, 1), 20))
    assert not step._overlap(a, torch.as_strided(store, (3, 4), (11, 1), 24))
    assert not step._overlap(torch.as_strided(store, (3, 4), (11, 1), 24), a)
