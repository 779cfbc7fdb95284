"""Binding of the cache operators (the C ABI declared in ``include/rra_cache.h``): what stands
before and behind the prefill of ``native``.

* ``RopeTable`` and ``rope`` - rotary positions with one or several axes, and their gradient;
* ``PagedCache`` - a paged key-value cache: ``append`` (rotate new tokens and write them),
  ``decode`` (attention of one new token per sequence), ``evict`` (keep the entries with the
  largest accumulated attention weight).

Like ``native`` this is argument marshalling only, on torch CUDA tensors; every operator runs in the
library's kernels. Calls run on the tensors' device, on its current stream unless ``stream`` is
given, do not synchronise and are not recorded by autograd. With ``stream`` the caller orders the
streams: the call does not wait for the current stream's work on its inputs, nor the current stream for
the outputs. Inputs and outputs may be dropped as soon as the call has returned.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import native

_c = ctypes
MAX_PAIRS, MAX_AXES = 64, 4
PAIRINGS = {"halves": 0, "adjacent": 1}


class _Rope(_c.Structure):
    """Mirror of ``rra_rope``."""
    _fields_ = [("head_dim", _c.c_int), ("rotary_dim", _c.c_int), ("axes", _c.c_int),
                ("pairing", _c.c_int), ("turn", _c.c_uint64 * MAX_PAIRS),
                ("axis", _c.c_uint8 * MAX_PAIRS)]


class _View(_c.Structure):
    """Mirror of ``rra_view``."""
    _fields_ = [("data", _c.c_void_p), ("batch", _c.c_int64), ("head", _c.c_int64),
                ("token", _c.c_int64)]


class _Positions(_c.Structure):
    """Mirror of ``rra_positions``."""
    _fields_ = [("data", _c.c_void_p), ("axis", _c.c_int64), ("batch", _c.c_int64),
                ("token", _c.c_int64)]


class _Tokens(_c.Structure):
    """Mirror of ``rra_tokens``."""
    _fields_ = [("batch", _c.c_int), ("heads_q", _c.c_int), ("heads_kv", _c.c_int),
                ("tokens", _c.c_int), ("dtype", _c.c_int), ("positions", _Positions),
                ("q", _View), ("k", _View), ("v", _View),
                ("q_out", _View), ("k_out", _View), ("v_out", _View)]


class _Cache(_c.Structure):
    """Mirror of ``rra_cache``."""
    _fields_ = [("batch", _c.c_int), ("heads_q", _c.c_int), ("heads_kv", _c.c_int),
                ("head_dim", _c.c_int), ("dtype", _c.c_int), ("page_size", _c.c_int),
                ("num_pages", _c.c_int), ("max_pages", _c.c_int), ("softmax_scale", _c.c_float),
                ("reserved", _c.c_int), ("page_stride", _c.c_int64), ("head_stride", _c.c_int64),
                ("entry_stride", _c.c_int64), ("table_stride", _c.c_int64), ("k", _c.c_void_p),
                ("v", _c.c_void_p), ("page_table", _c.c_void_p), ("len", _c.c_void_p),
                ("weight", _c.c_void_p), ("order", _c.c_void_p), ("seen", _c.c_void_p),
                ("workspace", _c.c_void_p), ("workspace_bytes", _c.c_size_t)]


def _dtype_code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return code


def _need(t, name, device, dtype, shape):
    if t.dtype is dtype and t.shape == shape and t.device == device:
        return
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name):
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _cuda(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


# A call's views and tokens are packed in one step (field by field costs more than the launch); the
# classes above give the layout.
_pack_view = struct.Struct("@P3q").pack
_pack_tokens = struct.Struct("@5i4x" + "P3q" * 7).pack
_NO_VIEW = (0, 0, 0, 0)
_CODES = {torch.bfloat16: 0, torch.float16: 1}


def _call(device, function, *args):
    """Runs a library call with the tensors' device current (the library runs on the current one)."""
    if torch.cuda.current_device() == device.index:
        return function(*args)
    with torch.cuda.device(device):
        return function(*args)


def _current_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# the same without building a Stream object, where torch has it
_raw_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device):
    if stream is None:
        return _raw_current(device.index) if _raw_current else _current_stream(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return stream.cuda_stream


def _new(shape, dtype, device, stream):
    """An output, allocated for the stream that writes it: a block of the current stream's may still be in
    use there by what was freed, and nothing makes ``stream`` wait for that."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        x = torch.empty(shape, dtype=dtype, device=device)
    x.record_stream(torch.cuda.current_stream(device))    # where the caller reads it
    return x


def _used(stream, *tensors):
    """Keeps the blocks of a call's tensors until ``stream`` is done with them, also where the caller drops
    the tensors before."""
    if stream is not None:
        for x in tensors:
            if x is not None:
                x.record_stream(stream)


def _int32(name, *values):
    """ctypes takes the low 32 bits of anything longer."""
    for x in values:
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{name} must fit 32 bits, got {x}")


class RopeTable:
    """A rotation of the first ``rotary_dim`` of ``head_dim`` dimensions.

    Pair i turns by ``positions[axis of i] * inv_freq[i]``. ``inv_freq`` (rotary_dim / 2 values, in
    radians per position) defaults to ``theta ** (-2 i / rotary_dim)``. The axes of the pairs come
    from ``sections`` (the first sections[0] pairs follow axis 0, and so on) or, for any other
    assignment such as alternating axes, from ``axis_of_pair``. ``pairing`` is "halves"
    (i, i + rotary_dim / 2) or "adjacent" (2 i, 2 i + 1).
    """

    def __init__(self, head_dim, rotary_dim=None, *, theta=10000.0, inv_freq=None, sections=None,
                 axis_of_pair=None, axes=None, pairing="halves"):
        if pairing not in PAIRINGS:
            raise ValueError(f"pairing must be one of {sorted(PAIRINGS)}, got {pairing!r}")
        if sections is not None and axis_of_pair is not None:
            raise ValueError("give sections or axis_of_pair, not both")
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        _int32("head_dim", head_dim)
        _int32("rotary_dim", rotary_dim)
        pairs = rotary_dim // 2
        freq = sec = ax = None
        if inv_freq is not None:
            values = [float(x) for x in inv_freq]
            if len(values) != pairs:
                raise ValueError(f"inv_freq must have {pairs} values, got {len(values)}")
            freq = (_c.c_double * pairs)(*values)
        if sections is not None:
            axes = len(sections) if axes is None else axes
            if len(sections) != axes:
                raise ValueError(f"sections must have {axes} values, got {len(sections)}")
            values = [int(x) for x in sections]
            _int32("sections", *values)
            sec = (_c.c_int32 * axes)(*values)
        if axis_of_pair is not None:
            values = [int(x) for x in axis_of_pair]
            if len(values) != pairs:
                raise ValueError(f"axis_of_pair must have {pairs} values, got {len(values)}")
            _int32("axis_of_pair", *values)
            axes = max(values, default=-1) + 1 if axes is None else axes
            ax = (_c.c_int32 * pairs)(*values)
        self.head_dim, self.rotary_dim, self.pairing = head_dim, rotary_dim, pairing
        self.axes = 1 if axes is None else axes
        _int32("axes", self.axes)
        self.raw = _Rope()
        native._check(native.load().rra_rope_init(
            _c.byref(self.raw), head_dim, rotary_dim, self.axes, PAIRINGS[pairing], float(theta),
            freq, sec, ax), "rra_rope_init")
        self._ref = _c.byref(self.raw)


def _rows_of(x, name, b, n, d, dtype, device):
    """Address and strides of one tensor [b, heads, n, d], and its heads."""
    if x.dim() == 4:
        xb, heads, xn, xd = x.shape
        s0, s1, s2, s3 = x.stride()
        if xb == b and xn == n and xd == d and s3 == 1 and x.dtype is dtype and x.device == device:
            return (x.data_ptr(), s0, s1, s2), heads
        if xb == b and xn == n and xd == d and x.dtype is dtype and x.device == device:
            raise ValueError(f"{name}: the last dimension must be contiguous")
    raise ValueError(f"{name} must be {dtype} [{b}, heads, {n}, {d}] on {device}, got {x.dtype} "
                     f"{tuple(x.shape)} on {x.device}")


def _out_of(o, x, name, b, heads, n, d, dtype, device, stream):
    """An output and its view: none (None), the caller's, or a new one (True)."""
    if o is None:
        return None, _NO_VIEW
    if o is True:
        o = _new(x.shape, dtype, device, stream)
    view, h = _rows_of(o, name, b, n, d, dtype, device)
    if h != heads:
        raise ValueError(f"{name} has {h} heads, its input has {heads}")
    return o, view


def _fill_tokens(table, positions, q, k, v, q_out, k_out, v_out, stream):
    """Checks the tensors of a call and packs them; returns (tokens, device, heads_q, outputs)."""
    first = k if k is not None else (q if q is not None else v)
    if first is None:
        raise ValueError("nothing to rotate: give q, k or both")
    if first.dim() != 4:
        raise ValueError("q, k and v must have 4 dimensions: [batch, heads, tokens, head_dim]")
    device, dtype = first.device, first.dtype
    if device.type != "cuda":
        raise ValueError("q, k and v must be CUDA tensors")
    code = _dtype_code(first, "q, k and v")
    b, _, n, d = first.shape
    if d != table.head_dim:
        raise ValueError(f"head_dim is {d}, the table's is {table.head_dim}")
    if positions.dtype is not torch.int32 or positions.device != device or \
            positions.shape != (table.axes, b, n):
        raise ValueError(f"positions must be torch.int32 {(table.axes, b, n)} on {device}, got "
                         f"{positions.dtype} {tuple(positions.shape)} on {positions.device}")
    p0, p1, p2 = positions.stride()
    heads_q = heads_kv = 0
    q_view = k_view = v_view = q_to = k_to = v_to = _NO_VIEW
    if q is not None:
        q_view, heads_q = _rows_of(q, "q", b, n, d, dtype, device)
        q_out, q_to = _out_of(q_out, q, "q_out", b, heads_q, n, d, dtype, device, stream)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    if k is not None:
        k_view, heads_kv = _rows_of(k, "k", b, n, d, dtype, device)
        k_out, k_to = _out_of(k_out, k, "k_out", b, heads_kv, n, d, dtype, device, stream)
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    if v is not None:
        v_view, heads_v = _rows_of(v, "v", b, n, d, dtype, device)
        if k is not None and heads_v != heads_kv:
            raise ValueError(f"k has {heads_kv} heads, v has {heads_v}")
        heads_kv = heads_v
        v_out, v_to = _out_of(v_out, v, "v_out", b, heads_v, n, d, dtype, device, stream)
    elif v_out is not None:
        raise ValueError("v_out is given without v")
    t = _pack_tokens(b, heads_q, heads_kv, n, code, positions.data_ptr(), p0, p1, p2, *q_view,
                     *k_view, *v_view, *q_to, *k_to, *v_to)
    _used(stream, positions, q, k, v, q_out, k_out, v_out)
    return t, device, heads_q, (q_out, k_out, v_out)


def rope(table, positions, q=None, k=None, v=None, *, q_out=None, k_out=None, v_out=None,
         inverse=False, stream=None):
    """Rotates q and k [batch, heads, tokens, head_dim] (any strides, the last dimension
    contiguous) by int32 positions [axes, batch, tokens]; v, if given, is copied. Outputs default to
    new contiguous tensors, the layout of ``native.prefill``; ``q_out=q`` works in place.
    ``inverse=True`` turns back: it takes the gradients of the outputs to those of the inputs. (The call is
    not recorded by autograd: in training call it from the forward and, with ``inverse=True``, from the
    backward of a ``torch.autograd.Function``.) Returns the outputs of the tensors that were given, in the order q, k, v."""
    q_out = True if q is not None and q_out is None else q_out
    k_out = True if k is not None and k_out is None else k_out
    v_out = True if v is not None and v_out is None else v_out
    t, device, _, outs = _fill_tokens(table, positions, q, k, v, q_out, k_out, v_out, stream)
    native._check(_call(device, native.load().rra_rope_rotate, table._ref, t, 1 if inverse else 0,
                        _raw_stream(stream, device)), "rra_rope_rotate")
    outs = [o for o in outs if o is not None]
    return outs[0] if len(outs) == 1 else tuple(outs)


class PagedCache:
    """A paged key-value cache over the caller's tensors.

    k, v         [num_pages, heads_kv, page_size, head_dim], bf16 or fp16; any strides with the last
                 dimension contiguous (a token-major cache is passed as its transposed view)
    page_table   int32 [batch, max_pages]: the pages of each sequence
    lengths      int32 [batch]: the entries of each sequence
    weight       fp32 [num_pages, heads_kv, page_size]: attention weight accumulated by ``decode``
    order        int32, like weight: the ordinal of each entry's token
    seen         int32 [batch]: the tokens each sequence has seen

    weight, order and seen come together; a cache that has them can be evicted from. The tensors'
    contents may change between calls, the tensors themselves stay (the object holds their
    addresses); lengths and seen are tensors of their own. The object owns its workspace: its calls
    must not overlap on the GPU, and it has to live until they are done on the GPU.
    """

    def __init__(self, k, v, page_table, lengths, *, heads_q, softmax_scale=-1.0, weight=None,
                 order=None, seen=None):
        device = _cuda(k, "k")
        if k.dim() != 4 or page_table.dim() != 2:
            raise ValueError("k must be [num_pages, heads_kv, page_size, head_dim] and page_table "
                             "[batch, max_pages]")
        _int32("heads_q", heads_q)
        pages, hkv, ps, d = k.shape
        b, max_pages = page_table.shape
        _need(v, "v", device, k.dtype, k.shape)
        if v.stride() != k.stride():
            raise ValueError(f"k and v must have the same strides, got {k.stride()} and "
                             f"{v.stride()}")
        _rows(k, "k")
        _need(page_table, "page_table", device, torch.int32, (b, max_pages))
        _rows(page_table, "page_table")
        _need(lengths, "lengths", device, torch.int32, (b,))
        track = [x is not None for x in (weight, order, seen)]
        if any(track) and not all(track):
            raise ValueError("weight, order and seen come together")
        self.tracked = all(track)
        if self.tracked:
            _need(weight, "weight", device, torch.float32, (pages, hkv, ps))
            _need(order, "order", device, torch.int32, (pages, hkv, ps))
            _need(seen, "seen", device, torch.int32, (b,))
        for name, x in (("lengths", lengths), ("weight", weight), ("order", order),
                        ("seen", seen)):
            if x is not None and not x.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self._tensors = (k, v, page_table, lengths, weight, order, seen)
        self.dtype = k.dtype
        self.device, self.batch, self.heads_q = device, b, heads_q
        s = k.stride()
        ptr = (lambda x: None if x is None else x.data_ptr())
        self.raw = _Cache(b, heads_q, hkv, d, _dtype_code(k, "k"), ps, pages, max_pages,
                          softmax_scale, 0, s[0], s[1], s[2], page_table.stride(0), ptr(k), ptr(v),
                          ptr(page_table), ptr(lengths), ptr(weight), ptr(order), ptr(seen),
                          None, 0)
        self._ref = _c.byref(self.raw)
        self._lib = native.load()
        n = int(_call(device, self._lib.rra_cache_workspace_bytes, self._ref))
        if n == 0:
            raise native.RraError(1, "rra_cache_workspace_bytes")
        self.ws = torch.zeros(n, dtype=torch.uint8, device=device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(device).synchronize()   # ready for calls on any stream
        self.raw.workspace, self.raw.workspace_bytes = self.ws.data_ptr(), n
        self._q_shape = (b, heads_q, d)

    # the tensors that were given; read only, because the library holds their addresses
    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    page_table = property(lambda self: self._tensors[2])
    lengths = property(lambda self: self._tensors[3])
    weight = property(lambda self: self._tensors[4])
    order = property(lambda self: self._tensors[5])
    seen = property(lambda self: self._tensors[6])

    @classmethod
    def allocate(cls, batch, max_len, heads_q, heads_kv, head_dim, *, page_size=64, dtype=None,
                 softmax_scale=-1.0, track=False, device="cuda"):
        """An empty cache with pages of its own for ``max_len`` entries per sequence."""
        dtype = torch.bfloat16 if dtype is None else dtype
        per = max(1, -(-max_len // page_size))
        kv = torch.zeros(2, max(1, batch * per), heads_kv, page_size, head_dim, dtype=dtype,
                         device=device)
        table = torch.arange(batch * per, dtype=torch.int32, device=device).view(batch, per)
        more = {}
        if track:
            more = {"weight": torch.zeros(kv.shape[1:4], device=device),
                    "order": torch.zeros(kv.shape[1:4], dtype=torch.int32, device=device),
                    "seen": torch.zeros(batch, dtype=torch.int32, device=device)}
        return cls(kv[0], kv[1], table, torch.zeros(batch, dtype=torch.int32, device=device),
                   heads_q=heads_q, softmax_scale=softmax_scale, **more)

    def append(self, table, positions, q, k, v, *, new_len=None, q_out=None, k_out=None,
               v_out=None, advance=True, stream=None):
        """Rotates q and k [batch, heads, tokens, head_dim] and writes k and v behind the entries
        of their sequences. q may be None. q_out defaults to a new contiguous tensor; k_out and v_out
        (the rotated keys and the values in the layout of the prefill) are written if given, or
        made with ``True``. new_len: int32 [batch], the tokens of each sequence that are real; the
        rest is padding, neither read nor written. ``advance=False`` leaves lengths and seen as they
        are (for all but the last of the layers that share them). Returns q_out, or
        (q_out, k_out, v_out) if k_out or v_out is given."""
        q_out = True if q is not None and q_out is None else q_out
        if k is None or v is None:
            raise ValueError("k and v are required")
        t, device, heads_q, outs = _fill_tokens(table, positions, q, k, v, q_out, k_out, v_out, stream)
        if device != self.device:
            raise ValueError(f"the cache is on {self.device}, the tokens are on {device}")
        if q is not None and heads_q != self.heads_q:
            raise ValueError(f"q has {heads_q} heads, the cache was made for {self.heads_q}")
        if new_len is not None:
            _need(new_len, "new_len", device, torch.int32, (self.batch,))
            if not new_len.is_contiguous():
                raise ValueError("new_len must be contiguous")
            _used(stream, new_len)
        native._check(_call(device, self._lib.rra_cache_append, self._ref, table._ref, t,
                            None if new_len is None else new_len.data_ptr(), 1 if advance else 0,
                            _raw_stream(stream, device)), "rra_cache_append")
        return outs[0] if k_out is None and v_out is None else outs

    def decode(self, q, *, out=None, lse=None, add_weight=False, stream=None):
        """Attention of one new token per sequence, q [batch, heads_q, head_dim] or
        [batch, heads_q, 1, head_dim], over the sequence's entries; returns ``out``, like q. ``lse``:
        fp32 [batch, heads_q], receives the logarithm of the softmax's denominator.
        ``add_weight=True`` adds the softmax weights to ``weight``."""
        shape = self._q_shape if q.dim() != 4 else self._q_shape[:2] + (1, self._q_shape[2])
        device, dtype = self.device, self.dtype
        sq = q.stride()
        if q.shape != shape or q.dtype is not dtype or q.device != device or sq[-1] != 1:
            _need(q, "q", device, dtype, shape)
            _rows(q, "q")
        if out is None:
            out = _new(shape, dtype, device, stream)
        so = out.stride()
        if out.shape != shape or out.dtype is not dtype or out.device != device or so[-1] != 1:
            _need(out, "out", device, dtype, shape)
            _rows(out, "out")
        at = None
        if lse is not None:
            _need(lse, "lse", device, torch.float32, shape[:2])
            if not lse.is_contiguous():
                raise ValueError("lse must be contiguous")
            at = lse.data_ptr()
        if add_weight and not self.tracked:
            raise ValueError("add_weight needs a cache with weight, order and seen")
        _used(stream, q, out, lse)
        native._check(_call(device, self._lib.rra_cache_decode, self._ref,
                            _pack_view(q.data_ptr(), sq[0], sq[1], 0),
                            _pack_view(out.data_ptr(), so[0], so[1], 0), at,
                            1 if add_weight else 0, _raw_stream(stream, device)),
                      "rra_cache_decode")
        return out

    def evict(self, budget, *, sinks=0, recent=0, advance=True, stream=None):
        """Cuts every sequence down to ``budget`` entries per KV head: the first ``sinks`` and last
        ``recent`` tokens stay, then the entries of the largest accumulated weight, the lower entry where
        weights are equal. Weights are what ``decode(add_weight=True)`` has added, or the caller has written
        to ``weight``: right after a prompt they are all 0. Sequences that share pages stay as they are."""
        if not self.tracked:
            raise ValueError("evict needs a cache with weight, order and seen")
        if not all(0 <= x < 2 ** 31 for x in (budget, sinks, recent)):
            raise ValueError("budget, sinks and recent must fit 31 bits and not be negative")
        native._check(_call(self.device, self._lib.rra_cache_evict, self._ref, budget, sinks, recent,
                            1 if advance else 0, _raw_stream(stream, self.device)),
                      "rra_cache_evict")

    def check(self, stream=None):
        """Synchronises ``stream`` (the current one by default) and raises if a call on it met a bad page,
        length or shared page since the last check (the error word is cleared)."""
        word = _c.c_uint32(0)
        st = _call(self.device, self._lib.rra_check_device_status, self.ws.data_ptr(),
                   _raw_stream(stream, self.device), _c.byref(word))
        native._check(int(st), f"device status word {word.value:#x}")
