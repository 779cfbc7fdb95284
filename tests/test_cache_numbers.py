"""Numbers that do not fit the C ABI's integers are refused by the binding, not cut to their low bits."""
import pytest
import torch

from long_context_prefill_rr_b200 import cache, native

FAR = 2 ** 32


@pytest.mark.parametrize("args,kw", [
    ((64 + FAR,), {}),
    ((64 - FAR,), {}),
    ((64, 32 + FAR), {}),
    ((64,), dict(sections=[32 + FAR])),
    ((64,), dict(sections=[FAR, 32])),
    ((64,), dict(axis_of_pair=[FAR] * 32)),
    ((64,), dict(axis_of_pair=[0] * 31 + [1 - FAR])),
    ((64,), dict(axes=1 + FAR)),
    ((64,), dict(axes=2 ** 31, axis_of_pair=[0] * 32)),
])
def test_table_numbers(args, kw):
    with pytest.raises(ValueError, match="32 bits"):
        cache.RopeTable(*args, **kw)


def test_table_without_pairs():
    with pytest.raises((ValueError, native.RraError)):
        cache.RopeTable(64, 0, axis_of_pair=[])


def test_cache_numbers(monkeypatch):
    monkeypatch.setattr(cache, "_cuda", lambda t, name: t.device)      # refused before any device call
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for heads in (8 + FAR, 8 - FAR, 2 ** 31):
        with pytest.raises(ValueError, match="32 bits"):
            cache.PagedCache(k, k, table, lens, heads_q=heads)
