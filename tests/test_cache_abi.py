"""The cache operators' C ABI and binding on the CPU: what include/rra_cache.h declares is exported,
the structs agree, and wrong arguments are refused before anything touches a GPU."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from long_context_prefill_rr_b200 import cache, native

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rra_cache.h")
INVALID, UNSUPPORTED, NO_DEVICE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(native.LIB_PATH):
        from long_context_prefill_rr_b200 import build
        build.build()
    return native.load()


def _declared():
    txt = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(rra_[a-z_]+)\s*\(", txt)))


def test_header_and_library_agree(lib):
    assert _declared() == ["rra_cache_append", "rra_cache_decode", "rra_cache_evict",
                           "rra_cache_workspace_bytes", "rra_rope_init", "rra_rope_rotate"]
    for name in _declared():
        assert hasattr(lib, name) and name in native._SIGS


def test_struct_layouts():
    assert ctypes.sizeof(cache._Rope) == 16 + 64 * 8 + 64
    assert ctypes.sizeof(cache._View) == 32 and ctypes.sizeof(cache._Positions) == 32
    assert ctypes.sizeof(cache._Tokens) == 24 + 32 + 6 * 32
    assert cache._Cache.page_stride.offset == 40 and cache._Cache.k.offset == 72
    assert ctypes.sizeof(cache._Cache) == 144
    # the packed forms that the binding passes are these structs
    t = cache._Tokens.from_buffer_copy(cache._pack_tokens(1, 2, 3, 4, 1, *range(10, 38)))
    assert (t.batch, t.heads_q, t.heads_kv, t.tokens, t.dtype) == (1, 2, 3, 4, 1)
    assert (t.positions.data, t.positions.token) == (10, 13)
    assert (t.q.data, t.k.batch, t.v.head, t.q_out.token) == (14, 19, 24, 29)
    assert (t.k_out.data, t.v_out.token) == (30, 37)
    v = cache._View.from_buffer_copy(cache._pack_view(5, 6, 7, 8))
    assert (v.data, v.batch, v.head, v.token) == (5, 6, 7, 8)


# ------------------------------------------------------------------------------------ rope tables
def test_table_holds_turns_and_axes(lib):
    t = cache.RopeTable(128, theta=500000.0, sections=[16, 24, 24])
    assert list(t.raw.axis) == [0] * 16 + [1] * 24 + [2] * 24
    for i in range(64):
        turns = 500000.0 ** (-2.0 * i / 128) / (2 * math.pi)
        # the fixed point is off by half of 2^-64, the fp64 quotient by two roundings
        assert abs(t.raw.turn[i] / 2.0 ** 64 - turns) <= 2.0 ** -65 + 2.0 ** -52 * turns
    t = cache.RopeTable(64, 32, inv_freq=[-1.0] + [0.25] * 15, axis_of_pair=[0, 1, 2, 3] * 4,
                        pairing="adjacent")
    assert t.axes == 4 and list(t.raw.axis)[:16] == [0, 1, 2, 3] * 4
    assert abs(t.raw.turn[0] / 2.0 ** 64 - (1 - 1 / (2 * math.pi))) < 1e-15   # a turn backwards


@pytest.mark.parametrize("kw,expect", [
    (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=128, rotary_dim=40), INVALID),
    (dict(head_dim=64, rotary_dim=128), INVALID),
    (dict(head_dim=64, rotary_dim=0), INVALID),
    (dict(head_dim=64, theta=0.0), INVALID),
    (dict(head_dim=64, theta=float("nan")), INVALID),
    (dict(head_dim=64, theta=float("inf")), INVALID),
    (dict(head_dim=64, inv_freq=[float("inf")] * 32), INVALID),
    (dict(head_dim=64, sections=[16, 15]), INVALID),
    (dict(head_dim=64, sections=[33, -1]), INVALID),
    (dict(head_dim=64, sections=[8, 8, 8, 4, 4]), INVALID),
    (dict(head_dim=64, axes=2), INVALID),                       # two axes, no assignment
    (dict(head_dim=64, axes=2, axis_of_pair=[0, 1, 2, 0] * 8), INVALID),
])
def test_table_refusals(lib, kw, expect):
    with pytest.raises(native.RraError) as e:
        cache.RopeTable(kw.pop("head_dim"), kw.pop("rotary_dim", None), **kw)
    assert e.value.status == expect


def test_table_refusals_of_the_binding(lib):
    for kw in (dict(pairing="thirds"), dict(inv_freq=[1.0]), dict(axis_of_pair=[0]),
               dict(sections=[32], axis_of_pair=[0] * 32), dict(sections=[16, 16], axes=3)):
        with pytest.raises(ValueError):
            cache.RopeTable(64, **kw)


# -------------------------------------------------------------------------------- call arguments
def _tokens(**kw):
    t = cache._Tokens()
    t.batch, t.heads_q, t.heads_kv, t.tokens, t.dtype = 2, 4, 2, 3, 0
    t.positions = cache._Positions(16, 6, 3, 1)
    for name, heads in (("q", 4), ("k", 2), ("v", 2)):
        for end in ("", "_out"):
            setattr(t, name + end, cache._View(16, heads * 3 * 64, 3 * 64, 64))
    for name, value in kw.items():
        setattr(t, name, value)
    return t


def _table():
    return cache.RopeTable(64)


def _rotate(table, t):
    return native.load().rra_rope_rotate(table._ref, ctypes.byref(t), 0, None)


V = cache._View


@pytest.mark.parametrize("kw,expect", [
    (dict(), NO_DEVICE),
    (dict(batch=0), 0),
    (dict(tokens=0), 0),
    (dict(batch=-1), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(dtype=2), UNSUPPORTED),
    (dict(tokens=(1 << 30) + 1), UNSUPPORTED),
    (dict(heads_q=70000), UNSUPPORTED),
    (dict(positions=cache._Positions(None, 0, 0, 0)), INVALID),
    (dict(positions=cache._Positions(18, 0, 0, 0)), INVALID),
    (dict(positions=cache._Positions(16, 0, 0, 0)), NO_DEVICE),    # broadcast positions
    (dict(q=V(24, 768, 192, 64)), INVALID),                        # 8-byte aligned
    (dict(q=V(16, 768, 192, 60)), INVALID),                        # rows not 16-byte aligned
    (dict(q=V(16, -768, 192, 64)), INVALID),
    (dict(q=V(16, 0, 0, 64)), NO_DEVICE),                          # broadcast input
    (dict(q_out=V(16, 0, 192, 64)), INVALID),                      # overlapping outputs
    (dict(q_out=V(16, 768, 128, 64)), INVALID),
    (dict(q_out=V(16, 768, 192, 56)), INVALID),
    (dict(q_out=V(16, 64 * 4 * 3, 64, 64 * 4)), NO_DEVICE),        # token-major output
    (dict(q_out=V(None, 0, 0, 0)), INVALID),                       # q without q_out
    (dict(q=V(None, 0, 0, 0)), INVALID),                           # q_out without q
    (dict(k_out=V(None, 0, 0, 0)), INVALID),
    (dict(v_out=V(None, 0, 0, 0)), INVALID),
    (dict(v=V(None, 0, 0, 0), v_out=V(None, 0, 0, 0)), NO_DEVICE),
    (dict(q=V(None, 0, 0, 0), q_out=V(None, 0, 0, 0)), NO_DEVICE),
])
def test_rotate_checks_before_any_launch(lib, kw, expect):
    if torch.cuda.is_available() and expect == NO_DEVICE:
        pytest.skip("made-up pointers stay off a GPU")
    assert _rotate(_table(), _tokens(**kw)) == expect


def test_a_table_that_was_never_filled_is_refused(lib):
    empty = cache._Rope()
    assert lib.rra_rope_rotate(ctypes.byref(empty), ctypes.byref(_tokens()), 0, None) == INVALID
    assert lib.rra_rope_rotate(None, ctypes.byref(_tokens()), 0, None) == INVALID
    assert lib.rra_rope_rotate(_table()._ref, None, 0, None) == INVALID
    bad = _table()
    bad.raw.axis[5] = 1                                            # axis 1 of one axis
    assert _rotate(bad, _tokens()) == INVALID


def _cache(**kw):
    c = cache._Cache(2, 4, 2, 64, 0, 16, 10, 4, -1.0, 0, 2 * 16 * 64, 16 * 64, 64, 4, 16, 16, 16,
                     16, 16, 16, 16, 16, 1 << 40)
    for name, value in kw.items():
        setattr(c, name, value)
    return c


BAD_CACHES = [
    (dict(batch=-1), INVALID), (dict(heads_q=5), INVALID), (dict(heads_kv=0), INVALID),
    (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(reserved=1), INVALID), (dict(dtype=7), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED),
    (dict(max_pages=1 << 27), UNSUPPORTED),                        # 2^31 entries
    (dict(batch=1 << 20, max_pages=1 << 20, table_stride=1 << 20), UNSUPPORTED),
    (dict(entry_stride=60), INVALID), (dict(head_stride=0), INVALID),
    (dict(entry_stride=56), INVALID), (dict(page_stride=1024), INVALID),
    (dict(table_stride=3), INVALID), (dict(k=None), INVALID), (dict(k=24), INVALID),
    (dict(v=None), INVALID), (dict(page_table=None), INVALID), (dict(page_table=18), INVALID),
    (dict(len=None), INVALID), (dict(workspace=None), INVALID), (dict(weight=None), INVALID),
    (dict(order=None), INVALID), (dict(seen=None), INVALID),
]


@pytest.mark.parametrize("kw,expect", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, kw, expect):
    c, q = _cache(**kw), V(16, 256, 64, 0)
    ref = ctypes.byref(c)
    assert lib.rra_cache_decode(ref, ctypes.byref(q), ctypes.byref(q), None, 0, None) == expect
    assert lib.rra_cache_evict(ref, 8, 0, 0, 1, None) == expect
    assert lib.rra_cache_append(ref, _table()._ref, ctypes.byref(_tokens()), None, 1,
                                None) == expect


def test_workspace_query_refuses_bad_sizes(lib):
    assert lib.rra_cache_workspace_bytes(None) == 0
    for kw, _ in BAD_CACHES[:11]:
        assert lib.rra_cache_workspace_bytes(ctypes.byref(_cache(**kw))) == 0


def test_decode_arguments(lib):
    ok = V(16, 256, 64, 0)

    def call(c, q=ok, out=ok, lse=None, add=0):
        return lib.rra_cache_decode(ctypes.byref(c), q and ctypes.byref(q),
                                    out and ctypes.byref(out), lse, add, None)

    assert call(_cache(), q=None) == INVALID and call(_cache(), out=None) == INVALID
    assert call(_cache(), q=V(None, 256, 64, 0)) == INVALID
    assert call(_cache(), q=V(8, 256, 64, 0)) == INVALID
    assert call(_cache(), q=V(16, 256, 60, 0)) == INVALID
    assert call(_cache(), out=V(16, 0, 64, 0)) == INVALID
    assert call(_cache(), out=V(16, 256, 32, 0)) == INVALID
    assert call(_cache(), lse=18) == INVALID
    assert call(_cache(weight=None, order=None, seen=None), add=1) == INVALID
    assert call(_cache(batch=0), q=None) == 0
    if not torch.cuda.is_available():
        assert call(_cache()) == NO_DEVICE
        assert call(_cache(weight=None, order=None, seen=None)) == NO_DEVICE


def test_evict_arguments(lib):
    def call(c, budget=8, sinks=0, recent=0):
        return lib.rra_cache_evict(ctypes.byref(c), budget, sinks, recent, 1, None)

    for args in (dict(budget=0), dict(budget=-1), dict(sinks=-1), dict(recent=-1), dict(sinks=9),
                 dict(sinks=4, recent=5), dict(sinks=8, recent=2 ** 31 - 1)):
        assert call(_cache(), **args) == INVALID, args
    assert call(_cache(weight=None, order=None, seen=None)) == INVALID
    assert call(_cache(batch=0)) == 0
    if not torch.cuda.is_available():
        assert call(_cache(), sinks=4, recent=4) == NO_DEVICE


def test_append_arguments(lib):
    def call(c=None, t=None, table=None, new_len=None):
        return lib.rra_cache_append(ctypes.byref(c or _cache()), (table or _table())._ref,
                                    ctypes.byref(t or _tokens()), new_len, 1, None)

    assert call(t=_tokens(batch=3)) == INVALID
    assert call(t=_tokens(heads_kv=4, k=V(16, 768, 192, 64), k_out=V(16, 768, 192, 64),
                          v=V(16, 768, 192, 64), v_out=V(16, 768, 192, 64))) == INVALID
    assert call(t=_tokens(dtype=1)) == INVALID
    assert call(table=cache.RopeTable(128)) == INVALID
    none = V(None, 0, 0, 0)
    assert call(t=_tokens(k=none, k_out=none)) == INVALID
    assert call(t=_tokens(v=none, v_out=none)) == INVALID
    assert call(new_len=18) == INVALID
    assert call(t=_tokens(tokens=0)) == 0
    if not torch.cuda.is_available():
        assert call(t=_tokens(q=none, q_out=none, k_out=none, v_out=none)) == NO_DEVICE


# ------------------------------------------------------------------------------------ the binding
def test_binding_wants_cuda_tensors(lib):
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 1, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        cache.rope(_table(), pos, x)
    with pytest.raises(ValueError, match="nothing to rotate"):
        cache.rope(_table(), pos)
    with pytest.raises(ValueError, match="4 dimensions"):
        cache.rope(_table(), pos, x[0])
    with pytest.raises(ValueError, match="CUDA"):
        cache.PagedCache(x, x, pos[0], torch.zeros(1, dtype=torch.int32), heads_q=2)


def test_oracle_rotation_is_a_rotation():
    """Closed forms that pin the oracle: unit determinant, composition of positions, the inverse."""
    from oracle import cache_oracle as orc
    rng = np.random.default_rng(0)
    x = rng.standard_normal((1, 2, 3, 64))
    f, ax = orc.rope_frequencies(64), [0] * 32
    pos = np.array([[[5, 7, 1000]]])
    for pairing in ("halves", "adjacent"):
        y = orc.rotate(x, pos, f, ax, pairing)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(orc.rotate(y, pos, f, ax, pairing, inverse=True), x)
        assert np.allclose(orc.rotate(y, pos, f, ax, pairing), orc.rotate(x, 2 * pos, f, ax, pairing))
        # scores depend on the distance alone
        k = orc.rotate(x, pos + 13, f, ax, pairing)
        far = orc.rotate(x, pos + 113, f, ax, pairing)
        near = orc.rotate(x, pos + 100, f, ax, pairing)
        assert np.allclose((y * k).sum(-1), (near * far).sum(-1))


def test_oracle_eviction_by_hand():
    from oracle import cache_oracle as orc
    w = np.array([0.0, 5.0, np.nan, 1.0, 5.0, -3.0, 0.0, 2.0]).reshape(2, 1, 4)
    o = np.arange(8).reshape(2, 1, 4)
    table, x = np.array([[1, 0]]), np.arange(8.0).reshape(2, 1, 4)
    # entries 0-3 are page 1 (weights 5 -3 0 2, ordinals 4-7), 4-7 page 0 (0 5 nan 1, ordinals 0-3)
    new = orc.evict([x], w, o, table, np.array([8]), np.array([8]), 4, 1, 1)
    # kept: ordinal 0 (entry 4), ordinal 7 (entry 3), weights 5 (entry 0) and 5 (entry 5)
    assert new.tolist() == [4]
    assert o[1, 0].tolist() == [4, 0, 1, 7] and x[1, 0].tolist() == [4.0, 0.0, 1.0, 7.0]
    assert o[0, 0].tolist() == [0, 1, 2, 3]
