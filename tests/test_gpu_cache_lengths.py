"""Lengths outside the page table in calls of the cache operators: flagged, and taken as the nearest valid
one."""
import pytest
import torch

from long_context_prefill_rr_b200 import cache, native

pytestmark = pytest.mark.gpu


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new", [0, -3])
@pytest.mark.parametrize("length,after", [(-7, 0), (33, 32), (2 ** 31 - 1, 32), (-2 ** 31, 0)])
@pytest.mark.parametrize("advance", [False, True])
def test_append_flags_lengths_of_sequences_without_new_tokens(cuda_device, new, length, after, advance):
    c = cache.PagedCache.allocate(3, 32, 2, 1, 64, page_size=16)
    x = torch.ones(3, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 3, 4, dtype=torch.int32, device="cuda")
    c.lengths.copy_(ints([5, length, 32]))
    c.append(cache.RopeTable(64), pos, None, x, x, new_len=ints([2, new, 0]), advance=advance)
    assert c.lengths.tolist() == ([7, after, 32] if advance else [5, length, 32])
    with pytest.raises(native.RraError):
        c.check()
    c.lengths.copy_(ints([0, 32, 31]))               # nothing wrong with these
    c.append(cache.RopeTable(64), pos, None, x, x, new_len=ints([0, new, 1]), advance=advance)
    c.check()
