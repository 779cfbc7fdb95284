"""Eviction where the page table is much wider than its sequences: the launch is sized by the table, so most
blocks of an entry's cluster have nothing to do."""
import pytest
import torch

from test_gpu_cache import HF, Paged, evicted, ordinals, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "zero", "odd", "tiny"])
@pytest.mark.parametrize("lens,budget,ps,width", [([65, 64, 0, 66, 1], 64, 16, 64 * 65),
                                                  ([2049, 2050, 2048, 7], 2048, 64, 131072),
                                                  ([300, 5000, 129], 128, 7, 64 * 5000)])
def test_evict_with_a_wide_table(cuda_device, kind, lens, budget, ps, width):
    p = Paged(lens, 2, 2, 64, ps, HF, seed=91, track=True, max_pages=width // ps)
    order, seen = ordinals(p, 92)
    evicted(p, weights(p, kind, 93), order, seen, budget, sinks=3, recent=11)
    out, again = p.cache.decode(p.query()), p.cache.decode(p.query())
    assert torch.equal(out, again) and p.lens.tolist() == [min(n, budget) for n in lens]
