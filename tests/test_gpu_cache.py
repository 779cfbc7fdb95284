"""The cache operators on the GPU against their fp64 forms (oracle/cache_oracle.py).

Tolerances, from the arithmetic of the kernels (eps / 2 is half a step of the element type, relative):

* a rotated value x cos - y sin: half a step of the result for the final rounding, and for the
  fp32 angle, sine, cosine, products and sum less than 2^-20 of |(x, y)|. With u = 2^-24: the angle within its
  quadrant is at most pi / 4; its conversion, the factor and the product are off by u of it each, and its last
  bit is 2^-32 of a turn: 2.4 u. The series of the sine is off by 0.9 u, that of the cosine by 1.0 u for
  roundings and 0.4 u for what is cut off (test_gpu_rope_angles.py adds it up); products and sum 2 u. In all
  6.1 u < 2^-21. fp16 results below 2^-14 have steps of 2^-24. The fp64 angle is itself off by
  2^-53 |angle|.
* a logit: products of 16-bit values are exact in fp32; d of them are added in fp32, each addition
  off by at most 2^-23 (the tensor cores truncate) of the sum of the magnitudes, R = scale * sum |q_i k_i|.
  Scaling to log2 and back costs 3 roundings. delta = (d + 4) 2^-23 R bounds its absolute error.
* a weight's relative error: delta + 2^-21 (subtraction, exp2 and the reciprocal of the sum), and
  2^-17 for the two 16-bit parts that multiply V (bf16: (2^-9)^2, doubled; fp16: (2^-12)^2, doubled, or
  2^-40 of the largest weight). An output is a mean of V rows
  with those weights: 2 (delta + 2^-17 + 2^-20) max |v|, and half a step.
* lse: delta + 2^-21 (1 + |lse|) for the sum, the logarithm and the change of base.
* an accumulated weight: for each of the g heads (delta + 2^-21) of itself for the logit and as much
  again for the denominator, 2^-23 (|logit| + |lse|) for the subtraction in log2, and the fp32 additions.
"""
import math

import numpy as np
import pytest
import torch

from long_context_prefill_rr_b200 import cache, native
from oracle import cache_oracle as orc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------- rope
def check_rotated(got, x, positions, freq, axes_of, pairing, inverse, dtype):
    x64, pos = f64(x), positions.cpu().numpy()
    ref = orc.rotate(x64, pos, freq, axes_of, pairing, inverse)
    pairs = len(freq)
    size = np.zeros_like(x64)
    for i in range(pairs):
        a, b = (i, i + pairs) if pairing == "halves" else (2 * i, 2 * i + 1)
        size[..., a] = size[..., b] = np.hypot(x64[..., a], x64[..., b])
    turned = 2.0 ** -20 + np.abs(pos).max(initial=0) * max(freq) * 2.0 ** -52
    tol = half_step(dtype) * (np.abs(ref) + size * turned) + size * turned
    if dtype == HF:
        tol = np.maximum(tol, 2.0 ** -25 + size * turned)
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), float((err - tol).max())
    rest = 2 * pairs
    assert torch.equal(got[..., rest:], x[..., rest:])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("d,rot,sections", [(128, 128, [16, 24, 24]), (128, 64, [32]),
                                            (64, 64, [1, 30, 1]), (64, 16, [2, 2, 2, 2]),
                                            (64, 48, [24, 0]), (128, 112, [56])])
@pytest.mark.parametrize("b,hq,hkv,n", [(1, 4, 2, 1), (2, 7, 1, 5), (3, 3, 3, 129)])
def test_rope(cuda_device, dtype, pairing, d, rot, sections, b, hq, hkv, n):
    theta = 10000.0
    table = cache.RopeTable(d, rot, theta=theta, sections=sections, pairing=pairing)
    freq, axes_of = orc.rope_frequencies(rot, theta), sum(([a] * s for a, s in
                                                           enumerate(sections)), [])
    q = randn((b, n, hq, d), dtype, 1).transpose(1, 2)          # the projection's layout
    k = randn((b, hkv, n, d), dtype, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 200000, (len(sections), b, n), generator=g, device="cuda",
                        dtype=torch.int32)
    for inverse in (False, True):
        qo, ko = cache.rope(table, pos, q, k, inverse=inverse)
        assert qo.is_contiguous() and qo.shape == q.shape
        check_rotated(qo, q, pos, freq, axes_of, pairing, inverse, dtype)
        check_rotated(ko, k, pos, freq, axes_of, pairing, inverse, dtype)


@pytest.mark.parametrize("positions", [[2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 1],
                                       [-1, -2 ** 31, -77777], [1 << 20, 999999, 1048575]])
def test_rope_far_and_negative_positions(cuda_device, positions):
    table = cache.RopeTable(128, theta=500000.0)
    x, pos = randn((1, 2, 3, 128), HF, 5), ints([[positions]])
    check_rotated(cache.rope(table, pos, x), x, pos, orc.rope_frequencies(128, 500000.0), [0] * 64,
                  "halves", False, HF)


def test_rope_frequencies_and_axes_of_the_caller(cuda_device):
    freq = [(-1.0) ** i * (0.3 + i) for i in range(32)]
    axes_of = [0, 1, 2] * 10 + [2, 0]
    table = cache.RopeTable(64, inv_freq=freq, axis_of_pair=axes_of)
    x, pos = randn((2, 3, 9, 64), BF, 6), ints(np.arange(54).reshape(3, 2, 9).tolist())
    check_rotated(cache.rope(table, pos, x), x, pos, freq, axes_of, "halves", False, BF)


def test_rope_in_place_broadcast_and_strided(cuda_device):
    table, freq = cache.RopeTable(64), orc.rope_frequencies(64)
    pos = ints([[0, 3, 9, 10]]).view(1, 1, 4).expand(1, 2, 4)         # one row for both sequences
    x = randn((2, 4, 6, 64), BF, 7).transpose(1, 2)
    keep = x.clone()
    assert cache.rope(table, pos, x, q_out=x) is x
    check_rotated(x, keep, pos, freq, [0] * 32, "halves", False, BF)
    shared = randn((2, 1, 4, 64), BF, 8).expand(2, 5, 4, 64)           # one head for five
    out = torch.full((2, 5, 8, 64), 7.0, dtype=BF, device="cuda")
    cache.rope(table, pos, shared, q_out=out[:, :, ::2])
    check_rotated(out[:, :, ::2], shared, pos, freq, [0] * 32, "halves", False, BF)
    assert (out[:, :, 1::2] == 7).all()
    v = randn((2, 4, 3, 64), BF, 9).transpose(1, 2)
    k_out, v_out = cache.rope(table, pos, k=v, v=v)
    assert torch.equal(v_out, v) and v_out.is_contiguous()
    with pytest.raises(native.RraError):
        cache.rope(table, pos, keep, q_out=keep[:1].expand(2, 6, 4, 64))
    assert cache.rope(table, pos[:, :, :0], keep[:, :, :0]).shape == (2, 6, 0, 64)


@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
def test_rope_gradient(cuda_device, pairing):
    """The inverse rotation is the gradient: against autograd of the formula, against differences of
    the operator, and summed over the heads of a broadcast input."""
    b, h, n, d, rot = 2, 3, 5, 64, 32
    freq, axes_of = orc.rope_frequencies(rot), [0] * 8 + [1] * 8
    table = cache.RopeTable(d, rot, sections=[8, 8], pairing=pairing)
    g = torch.Generator(device="cuda").manual_seed(11)
    pos = torch.randint(0, 5000, (2, b, n), generator=g, device="cuda", dtype=torch.int32)
    x, dy = randn((b, h, n, d), HF, 12), randn((b, h, n, d), HF, 13)
    dx = cache.rope(table, pos, dy, inverse=True)
    leaf = x.double().cpu().requires_grad_()
    pieces = [leaf[..., j] for j in range(d)]
    y = list(pieces)
    for i, f in enumerate(freq):
        a, c = (i, i + rot // 2) if pairing == "halves" else (2 * i, 2 * i + 1)
        angle = pos[axes_of[i]].double().cpu()[:, None] * f
        y[a] = pieces[a] * angle.cos() - pieces[c] * angle.sin()
        y[c] = pieces[c] * angle.cos() + pieces[a] * angle.sin()
    (torch.stack(y, -1) * dy.double().cpu()).sum().backward()
    size = float(dy.abs().max()) * math.sqrt(2)
    tol = size * (half_step(HF) * (1 + 2.0 ** -18) + 2.0 ** -19)
    assert float((dx.double().cpu() - leaf.grad).abs().max()) <= tol
    # differences: the operator is linear, so a unit step along e changes the outputs by its image
    for j in (0, 1, 17, 31, 40):
        unit = torch.zeros_like(x)
        unit[..., j] = 1.0
        image = cache.rope(table, pos, unit)
        got = (image.double() * dy.double()).sum(-1)
        # an image has at most two values other than 0, each off by half a step
        assert float((got - dx[..., j].double()).abs().max()) <= 2 * tol
    total = cache.rope(table, pos, dy, inverse=True).double().sum(1, keepdim=True)
    ref = leaf.grad.sum(1, keepdim=True)
    assert float((total.cpu() - ref).abs().max()) <= h * tol


# ----------------------------------------------------------------------------------------- decode
class Paged:
    """A cache with pages in random order, sequences of the given lengths, and its numpy mirror."""

    def __init__(self, lens, hq, hkv, d, ps, dtype=BF, layout="HND", seed=0, track=False, spare=2,
                 max_pages=None, scale=-1.0, spread=1.0):
        rng = np.random.default_rng(seed)
        need = [max(1, -(-max(n, 1) // ps)) for n in lens]
        width = max_pages or max(need)
        total = sum(need) + spare
        perm = rng.permutation(total)
        table = np.full((len(lens), width), -1, dtype=np.int64)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        shape = (total, hkv, ps, d) if layout == "HND" else (total, ps, hkv, d)
        self.k, self.v = (randn(shape, dtype, seed + i, spread) for i in (1, 2))
        if layout == "NHD":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.table, self.lens = ints(table.tolist()), ints(list(lens))
        self.hq, self.d, self.dtype, self.scale = hq, d, dtype, scale
        more = {}
        if track:
            g = torch.Generator(device="cuda").manual_seed(seed + 3)
            more = {"weight": torch.rand((total, hkv, ps), generator=g, device="cuda"),
                    "order": torch.zeros((total, hkv, ps), dtype=torch.int32, device="cuda"),
                    "seen": self.lens.clone()}
        self.cache = cache.PagedCache(self.k, self.v, self.table, self.lens, heads_q=hq,
                                      softmax_scale=scale, **more)

    def query(self, seed=50, spread=1.0):
        q = randn((len(self.lens), self.hq, self.d), torch.float32, seed)
        q *= torch.linspace(0.2, 2.0, self.hq, device="cuda")[:, None] * spread
        return q.to(self.dtype)

    def check(self, q, out, lse, weight=None, before=None):
        scale = self.scale if self.scale > 0 else 1 / math.sqrt(self.d)
        ref, rlse, share, reach = orc.decode(f64(q), f64(self.k), f64(self.v),
                                             self.table.cpu().numpy(), self.lens.cpu().numpy(),
                                             scale)
        delta = (self.d + 4) * 2.0 ** -23 * reach
        vmax = float(np.nanmax(np.abs(f64(self.v))))
        tol = half_step(self.dtype) * np.abs(ref) * (1 + 2.0 ** -8) + \
            (2 * vmax * (delta + 2.0 ** -17 + 2.0 ** -20))[..., None]
        if self.dtype == HF:
            tol += 2.0 ** -25
        err = np.abs(f64(out) - ref)
        assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(~(err <= tol))[:4])
        empty = np.isinf(rlse)
        assert np.array_equal(f64(lse)[empty], rlse[empty])
        assert not f64(out)[empty].any()
        ok = ~empty
        err = np.abs(f64(lse)[ok] - rlse[ok])
        assert (err <= delta[ok] + 2.0 ** -21 * (1 + np.abs(rlse[ok]))).all(), float(err.max())
        if weight is not None:
            g = self.hq // self.k.shape[1]
            worst = float((2 * delta + 2.0 ** -20).max(initial=0)) + \
                2.0 ** -22 * float(np.where(empty, 0, np.abs(rlse) + 2 * reach).max(initial=0))
            got, was = f64(weight) - f64(before), f64(before)
            tol = share * worst + (share + np.abs(was)) * 2.0 ** -23 * (g + 1)
            assert (np.abs(got - share) <= tol).all(), float((np.abs(got - share) - tol).max())
            assert np.array_equal(f64(weight)[share == 0], was[share == 0])


def run_decode(p, q=None, add_weight=False):
    q = p.query() if q is None else q
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    before = p.cache.weight.clone() if add_weight else None
    out = p.cache.decode(q, lse=lse, add_weight=add_weight)
    torch.cuda.synchronize()
    p.check(q, out, lse, p.cache.weight if add_weight else None, before)
    return out, lse


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 500]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (8, 8, 64), (14, 2, 128), (8, 1, 64),
                                      (9, 1, 128), (32, 2, 64), (40, 2, 128)])
@pytest.mark.parametrize("ps", [1, 7, 16, 20, 64])
def test_decode(cuda_device, dtype, layout, hq, hkv, d, ps):
    p = Paged(LENS, hq, hkv, d, ps, dtype, layout, seed=ps)
    run_decode(p)
    p.cache.check()


@pytest.mark.parametrize("hq,hkv,d,ps", [(28, 4, 128, 64), (8, 8, 64, 20), (18, 2, 64, 7)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_decode_weights(cuda_device, dtype, hq, hkv, d, ps):
    p = Paged(LENS, hq, hkv, d, ps, dtype, seed=3, track=True)
    plain = p.cache.decode(p.query())
    out, _ = run_decode(p, add_weight=True)
    assert torch.equal(out, plain)          # the same output with and without the weights
    run_decode(p, add_weight=True)          # and a second step on top
    p.cache.check()


@pytest.mark.parametrize("lens,hq,hkv", [([70001], 8, 1), ([40000], 4, 4), ([33000, 0, 5, 9999], 7, 1),
                                         ([129] * 700, 2, 1), ([0] * 300 + [3000], 4, 2),
                                         ([0, 0], 4, 2), (list(range(300)), 3, 3)])
def test_decode_split(cuda_device, lens, hq, hkv):
    """Long sequences cut over the grid, and more sequences than threads of a block."""
    p = Paged(lens, hq, hkv, 128, 32, seed=9, track=True)
    out, lse = run_decode(p, add_weight=True)
    again = torch.empty_like(lse)
    for _ in range(3):                      # equal calls, equal bits
        assert torch.equal(p.cache.decode(p.query(), lse=again), out) and torch.equal(again, lse)
    p.cache.check()


def test_decode_scale_and_sharp_logits(cuda_device):
    """Logits of hundreds: one entry takes all the weight; the running maximum jumps."""
    p = Paged([300, 77], 4, 2, 128, 16, HF, seed=4, scale=3.0, spread=1.5)
    run_decode(p)
    p = Paged([2000, 77], 4, 2, 64, 16, BF, seed=5, scale=1e-6)
    run_decode(p)


def test_decode_views(cuda_device):
    """Strided queries and outputs, 4-dimensional ones, broadcast queries, out over q."""
    p = Paged([100, 37, 64], 6, 2, 64, 16, seed=6)
    q = p.query()
    ref = p.cache.decode(q)
    wide = torch.zeros(3, 9, 6, 64, dtype=BF, device="cuda")
    wide[:, 4] = q
    out = torch.full((6, 3, 128), 5.0, dtype=BF, device="cuda")
    got = p.cache.decode(wide[:, 4], out=out.transpose(0, 1)[..., :64])
    assert torch.equal(got, ref) and (out[..., 64:] == 5).all()
    four = p.cache.decode(q[:, :, None])
    assert four.shape == (3, 6, 1, 64) and torch.equal(four[:, :, 0], ref)
    one = p.cache.decode(q[:1].expand(3, 6, 64))
    assert torch.equal(one[0], ref[0])
    q2 = q.clone()
    assert p.cache.decode(q2, out=q2) is q2 and torch.equal(q2, ref)
    for bad in (q[:2], q.half(), q.float(), q.cpu(), q[..., ::2]):
        with pytest.raises(ValueError):
            p.cache.decode(bad)
    with pytest.raises(ValueError):
        p.cache.decode(q, add_weight=True)
    with pytest.raises(native.RraError):
        p.cache.decode(q, out=torch.empty(1, 6, 64, dtype=BF, device="cuda").expand(3, 6, 64))


def test_decode_what_is_behind_the_entries_does_not_count(cuda_device):
    """NaN and infinities in the rest of the last page, in spare pages and in unused table places."""
    p = Paged([5, 16, 33, 0], 4, 2, 128, 16, seed=7, max_pages=9)
    q = p.query()
    ref, _ = run_decode(p, q)
    live = torch.zeros(p.k.shape[:3], dtype=torch.bool, device="cuda")
    for b, n in enumerate(p.lens.tolist()):
        for e in range(n):
            live[p.table[b, e // 16].long(), :, e % 16] = True
    for i, x in enumerate((math.nan, math.inf, -math.inf)):
        p.k[~live], p.v[~live] = x, x if i != 1 else math.nan
        assert torch.equal(p.cache.decode(q), ref)
    p.cache.check()


def test_decode_infinite_and_nan_logits(cuda_device):
    p = Paged([40, 40, 40, 40], 2, 1, 64, 16, seed=8)
    q = p.query().abs() + 0.5
    at = [(p.table[b, 1].long(), 0, 3) for b in range(4)]      # entry 19 of every sequence
    p.k[at[0]] = -math.inf                                      # a logit of -inf: absent
    p.k[at[1]] = math.nan                                       # the row is NaN
    p.k[p.table[2].long()[:3]] = -math.inf                      # nothing is left
    lse = torch.zeros(4, 2, device="cuda")
    out = p.cache.decode(q, lse=lse)
    clean = Paged([39], 2, 1, 64, 1, seed=8)
    rows = [e for e in range(40) if e != 19]
    for name in ("k", "v"):
        src, dst = getattr(p, name), getattr(clean, name)
        for i, e in enumerate(rows):
            dst[clean.table[0, i].long(), 0, 0] = src[p.table[0, e // 16].long(), 0, e % 16]
    ref = clean.cache.decode(q[:1])
    # two results near the same value may round to neighbours, a step (2^-7) apart
    assert (out[0].float() - ref[0].float()).abs().max() <= \
        2.0 ** -7 * (ref.float().abs().max() + clean.v.float().abs().max() * 2.0 ** -8)
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert not out[2].any() and (lse[2] == -math.inf).all()
    assert out[3].isfinite().all()


def test_decode_bad_tables_and_lengths_are_flagged(cuda_device):
    """The kernels check pages and lengths themselves: a bad page's entries are absent."""
    p = Paged([60, 60, 60], 4, 2, 64, 16, seed=9, track=True)
    p.table[0, 1], p.table[1, 3], p.table[2, 0] = -5, p.k.shape[0], 2 ** 30
    run_decode(p, add_weight=True)
    with pytest.raises(native.RraError) as e:
        p.cache.check()
    assert e.value.status == 1
    p.cache.check()                          # cleared
    p = Paged([30, 30], 4, 2, 64, 16, seed=10)
    p.lens.copy_(ints([-3, 1000]))
    run_decode(p)
    with pytest.raises(native.RraError):
        p.cache.check()
    p = Paged([30], 4, 2, 64, 16, seed=11)
    p.table.fill_(-1)                        # no page at all
    run_decode(p)


def test_decode_rows_may_share_pages(cuda_device):
    p = Paged([200], 4, 2, 64, 16, seed=12, track=True)
    table, lens = p.table.expand(5, -1).contiguous(), ints([200, 1, 0, 64, 150])
    weight = torch.zeros_like(p.cache.weight)
    many = cache.PagedCache(p.k, p.v, table, lens, heads_q=4, weight=weight,
                            order=p.cache.order, seen=lens.clone())
    p.table, p.lens, p.cache = table, lens, many
    run_decode(p, add_weight=True)


def test_decode_far_offsets(cuda_device):
    """Keys and values more than 2^32 bytes (and 2^31 elements) into the cache."""
    pages, hkv, ps, d = 40000, 8, 64, 128                      # 5.2 GB each
    k = torch.empty(pages, hkv, ps, d, dtype=BF, device="cuda")
    v = torch.empty(pages, hkv, ps, d, dtype=BF, device="cuda")
    use = [39999, 0, 39990, 20000]
    small = Paged([230], 16, hkv, d, ps, seed=13, track=True, spare=0)
    assert small.k.shape[0] == 4
    for i, pg in enumerate(use):
        src = small.table[0, i].long()
        k[pg], v[pg] = small.k[src], small.v[src]
    big = cache.PagedCache(k, v, ints([use]), ints([230]), heads_q=16)
    assert torch.equal(big.decode(small.query()), small.cache.decode(small.query()))
    big.check()
    table = cache.RopeTable(128)
    big.lengths.fill_(231)
    new = randn((1, hkv, 1, d), BF, 14)
    big.append(table, ints([[[0]]]), None, new, new)
    assert torch.equal(v[20000, :, 231 - 192], new[0, :, 0]) and big.lengths.item() == 232
    assert torch.equal(k[20000, :, 231 - 192], new[0, :, 0])   # position 0 turns nothing


# ----------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("layout,ps", [("HND", 16), ("NHD", 7), ("HND", 1)])
@pytest.mark.parametrize("lens,n,new", [([0, 3, 40], 1, None), ([5, 0, 31], 33, [33, 0, 10]),
                                        ([0, 0, 0], 200, [200, 1, 199])])
def test_append(cuda_device, dtype, layout, ps, lens, n, new):
    hq, hkv, d = 6, 2, 128
    p = Paged([m + n for m in lens], hq, hkv, d, ps, dtype, layout, seed=20, track=True)
    c = p.cache
    c.lengths.copy_(ints(lens))
    c.seen.copy_(ints([1000, 7, 40]))
    table = cache.RopeTable(d, theta=10000.0, sections=[16, 24, 24])
    freq, axes_of = orc.rope_frequencies(d), [0] * 16 + [1] * 24 + [2] * 24
    qkv = randn((3, n, hq + 2 * hkv, d), dtype, 21).transpose(1, 2)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    g = torch.Generator(device="cuda").manual_seed(22)
    pos = torch.randint(0, 9000, (3, 3, n), generator=g, device="cuda", dtype=torch.int32)
    was = {name: getattr(c, name).clone() for name in ("k", "v", "weight", "order")}
    q_out = torch.full((3, hq, n, d), 9.0, dtype=dtype, device="cuda")
    k_out = torch.full((3, hkv, n, d), 9.0, dtype=dtype, device="cuda")
    real = [n] * 3 if new is None else new
    got = c.append(table, pos, q, k, v, new_len=None if new is None else ints(new), q_out=q_out,
                   k_out=k_out, v_out=True, advance=False)
    assert got[0] is q_out and got[1] is k_out
    assert c.lengths.tolist() == lens and c.seen.tolist() == [1000, 7, 40]
    for b, m in enumerate(real):
        sl = slice(b, b + 1)
        check_rotated(q_out[sl, :, :m], q[sl, :, :m], pos[:, sl, :m], freq, axes_of, "halves",
                      False, dtype)
        check_rotated(k_out[sl, :, :m], k[sl, :, :m], pos[:, sl, :m], freq, axes_of, "halves",
                      False, dtype)
        assert (q_out[b, :, m:] == 9).all() and (k_out[b, :, m:] == 9).all()
        assert torch.equal(got[2][b, :, :m], v[b, :, :m])
        for t in range(m):
            pg, off = orc.entry(p.table, b, lens[b] + t, ps)
            was["k"][pg, :, off], was["v"][pg, :, off] = k_out[b, :, t], v[b, :, t]
            was["weight"][pg, :, off] = 0
            was["order"][pg, :, off] = [1000, 7, 40][b] + t
    for name, x in was.items():              # everything else is as it was
        assert torch.equal(getattr(c, name), x), name
    c.append(table, pos, None, k, v, new_len=None if new is None else ints(new))
    assert c.lengths.tolist() == [m + r for m, r in zip(lens, real)]
    assert c.seen.tolist() == [s + r for s, r in zip([1000, 7, 40], real)]
    assert torch.equal(c.k, was["k"])        # the same entries again
    c.check()


def test_append_past_the_table_and_bad_pages(cuda_device):
    p = Paged([32, 32, 32], 2, 1, 64, 16, seed=23, track=True)
    c, table = p.cache, cache.RopeTable(64)
    c.lengths.copy_(ints([30, 31, 5]))
    p.table[2, 0] = 10 ** 6
    x = randn((3, 1, 4, 64), BF, 24)
    pos = torch.zeros(1, 3, 4, dtype=torch.int32, device="cuda")
    was = c.v.clone()
    c.append(table, pos, None, x, x)
    for b, e, t in ((0, 30, 0), (0, 31, 1), (1, 31, 0)):
        was[p.table[b, e // 16].long(), :, e % 16] = x[b, :, t]
    assert torch.equal(c.v, was) and c.lengths.tolist() == [32, 32, 9]
    with pytest.raises(native.RraError):
        c.check()
    c.lengths.copy_(ints([-7, 2 ** 31 - 1, 0]))      # flagged; counts as the nearest valid length
    c.append(table, pos, None, x, x, new_len=ints([1, 1, -5]))
    assert c.lengths.tolist() == [1, 32, 0]
    with pytest.raises(native.RraError):
        c.check()


def test_strides_of_single_places_do_not_count(cuda_device):
    """One head, one page or one entry per page: the stride that goes with it may be anything."""
    p = Paged([5, 9], 2, 1, 64, 1, seed=27)
    table, x = cache.RopeTable(64), randn((2, 1, 1, 64), BF, 28)
    pos = torch.zeros(1, 2, 1, dtype=torch.int32, device="cuda")
    p.cache.lengths.copy_(ints([4, 8]))
    p.cache.raw.head_stride = p.cache.raw.entry_stride = -7
    out = torch.zeros_like(x)
    view = (x.data_ptr(), 64, -3, -5)
    tokens = cache._pack_tokens(2, 0, 1, 1, 0, pos.data_ptr(), 0, 1, 0, *(0,) * 4, *view, *view,
                                *(0,) * 4, out.data_ptr(), 64, -3, -5, *(0,) * 4)
    stream = torch.cuda.current_stream().cuda_stream
    assert native.load().rra_cache_append(p.cache._ref, table._ref, tokens, None, 1, stream) == 0
    assert p.lens.tolist() == [5, 9] and torch.equal(out, x)      # position 0 turns nothing
    for b, e in ((0, 4), (1, 8)):
        assert torch.equal(p.v[p.table[b, e].long(), 0, 0], x[b, 0, 0])
    run_decode(p)


def test_append_refusals(cuda_device):
    p = Paged([32], 2, 1, 64, 16, seed=25)
    x, pos = randn((1, 1, 4, 64), BF, 26), torch.zeros(1, 1, 4, dtype=torch.int32, device="cuda")
    table = cache.RopeTable(64)
    for kw in (dict(q=x), dict(k=x.half()), dict(v=x[:, :, :2]), dict(new_len=ints([1, 2])),
               dict(positions=pos.long()), dict(positions=pos[:, :, :3]), dict(v=None)):
        args = dict(positions=pos, q=None, k=x, v=x) | kw
        with pytest.raises(ValueError):
            p.cache.append(table, **args)
    with pytest.raises(ValueError):
        p.cache.append(cache.RopeTable(128), pos, None, x, x)
    with pytest.raises(native.RraError):
        p.cache.append(table, pos[:, :, 1:], None, x[:, :, 1:].expand(1, 3, 3, 64),
                       x[:, :, 1:].expand(1, 3, 3, 64))


# ---------------------------------------------------------------------------------------- evict
def evicted(p, weight, order, seen, budget, sinks=0, recent=0, lens_ref=None, flagged=False):
    c = p.cache
    c.weight.copy_(weight)
    c.order.copy_(order)
    c.seen.copy_(seen)
    mirror = {n: getattr(c, n).cpu().numpy().copy() if n in ("weight", "order") else
              getattr(c, n).float().cpu().numpy().copy() for n in ("k", "v", "weight", "order")}
    lens = c.lengths.cpu().numpy().copy()
    new = orc.evict([mirror["k"], mirror["v"]], mirror["weight"], mirror["order"],
                    p.table.cpu().numpy(), lens, c.seen.cpu().numpy(), budget, sinks, recent)
    c.evict(budget, sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    assert c.lengths.tolist() == new.tolist()
    for n, x in mirror.items():
        got = getattr(c, n)
        got = got.float() if n in ("k", "v") else got
        assert np.array_equal(got.cpu().numpy(), x, equal_nan=True), n
    if flagged:
        with pytest.raises(native.RraError):
            c.check()
    c.check()


def ordinals(p, seed=0):
    """Distinct ordinals in random order per sequence and head, and the tokens seen."""
    rng = np.random.default_rng(seed)
    order = np.zeros(p.k.shape[:3], dtype=np.int64)
    table, lens, ps = p.table.cpu().numpy(), p.lens.cpu().numpy(), p.k.shape[2]
    seen = [max(0, int(n)) * 5 // 4 for n in lens]
    for b, n in enumerate(lens):
        for h in range(p.k.shape[1]):
            o = rng.permutation(seen[b])[:n]
            e = np.arange(n)
            order[table[b, e // ps], h, e % ps] = o
    return torch.tensor(order, dtype=torch.int32, device="cuda"), ints(seen)


def weights(p, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.exp(3 * torch.randn(p.k.shape[:3], generator=g, device="cuda"))
    r = torch.rand(p.k.shape[:3], generator=g, device="cuda")
    if kind == "ties":
        w = torch.floor(r * 4)
    elif kind == "equal":
        w.fill_(0.5)
    elif kind == "zero":
        w.zero_()
    elif kind == "tiny":                    # the smallest weights: multiples of 2^-149, zeros among them
        w = torch.floor(r * 40 - 8).clamp(min=0).to(torch.int32).view(torch.float32)
    elif kind == "odd":
        for i, x in enumerate((math.nan, -1.0, math.inf, -0.0, 1e-42, -math.inf)):
            w[(r > i * 0.1) & (r < i * 0.1 + 0.1)] = x
    return w


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "zero", "odd", "tiny"])
@pytest.mark.parametrize("lens,budget,sinks,recent,ps,hkv,d", [
    ([1, 0, 2, 3], 1, 0, 1, 1, 2, 64), ([64, 65, 66, 200], 64, 4, 20, 16, 3, 128),
    ([500, 31, 32, 33], 32, 0, 0, 7, 2, 64), ([1500, 1499], 1499, 100, 1399, 20, 1, 128),
    (list(range(300)), 40, 3, 9, 8, 3, 64),
    ([900], 450, 450, 0, 64, 2, 64), ([9000, 100, 4500], 2000, 16, 500, 64, 2, 64)])
def test_evict(cuda_device, kind, lens, budget, sinks, recent, ps, hkv, d):
    p = Paged(lens, hkv, hkv, d, ps, seed=30, track=True)
    order, seen = ordinals(p)
    evicted(p, weights(p, kind), order, seen, budget, sinks, recent)


@pytest.mark.parametrize("layout,dtype,lens,budget,kind", [
    ("NHD", HF, [40000], 39999, "plain"), ("HND", BF, [33333, 20000], 5000, "ties"),
    ("HND", BF, [20000], 10000, "equal")])
def test_evict_long(cuda_device, layout, dtype, lens, budget, kind):
    p = Paged(lens, 2, 2, 64, 64, dtype, layout, seed=31, track=True)
    order, seen = ordinals(p)
    evicted(p, weights(p, kind), order, seen, budget, 4, 700)


def test_evict_weights_off_a_vector(cuda_device):
    """Weights and ordinals that start 4 and 8 bytes past a multiple of 16 are read one by one."""
    p = Paged([700, 333], 2, 2, 64, 16, seed=39, track=True)
    order, seen = ordinals(p)
    n = p.cache.weight.numel()
    w = torch.zeros(n + 4, device="cuda")[1:n + 1].view(p.cache.weight.shape)
    o = torch.zeros(n + 4, dtype=torch.int32, device="cuda")[2:n + 2].view(p.cache.weight.shape)
    p.cache = cache.PagedCache(p.k, p.v, p.table, p.lens, heads_q=2, weight=w, order=o, seen=seen)
    evicted(p, weights(p, "ties"), order, seen, 300, 5, 50)
    p.lens.fill_(300)
    run_decode(p, add_weight=True)


def test_evict_shares_longer_than_shared_memory(cuda_device):
    """Keys that do not fit the cluster's shared memory are read again for every digit."""
    n = 8 * 32768 + 12345
    p = Paged([n], 1, 1, 64, 128, seed=32, track=True)
    order, seen = ordinals(p)
    evicted(p, weights(p, "plain"), order, seen, n // 3, 16, 1000)
    p.lens.fill_(n)
    evicted(p, weights(p, "ties"), order, seen, n // 2, 0, 0)


def test_evict_repeated_ordinals_and_far_recent(cuda_device):
    """More protected entries than the budget: the lower entries stay."""
    p = Paged([100], 2, 2, 64, 16, seed=33, track=True)
    order = torch.zeros_like(p.cache.order)
    evicted(p, weights(p, "plain"), order, ints([100]), 40, 1, 0)
    p.lens.fill_(100)
    evicted(p, weights(p, "plain"), order, ints([-2 ** 31]), 40, 0, 39)


def test_evict_leaves_shared_and_bad_pages_alone(cuda_device):
    p = Paged([100, 100, 100, 30, 100], 2, 2, 64, 16, seed=34, track=True)
    order, seen = ordinals(p)
    p.table[1, 5] = p.table[0, 2]            # rows 0 and 1 share a page
    p.table[4, 3] = p.table[3, 0]            # row 4 has one of row 3, which is under its budget
    evicted(p, weights(p, "plain"), order, seen, 50, 2, 10, flagged=True)
    p = Paged([100, 100], 2, 2, 64, 16, seed=35, track=True)
    order, seen = ordinals(p)
    p.table[0, 6], p.table[1, 1] = -1, p.table[1, 4].clone()   # a bad page; one page twice
    evicted(p, weights(p, "plain"), order, seen, 50, 2, 10, flagged=True)
    # sequences within the budget may share, and are not the others' concern
    p = Paged([100, 40, 40], 2, 2, 64, 16, seed=38, track=True)
    order, seen = ordinals(p)
    p.table[1, 0] = p.table[2, 0]
    evicted(p, weights(p, "plain"), order, seen, 50, 2, 10)
    # a page behind a sequence's entries may be anybody's
    p = Paged([100, 100], 2, 2, 64, 16, seed=36, track=True, max_pages=9)
    order, seen = ordinals(p)
    p.table[0, 8] = p.table[1, 0]
    evicted(p, weights(p, "plain"), order, seen, 50, 2, 10)


def test_evict_without_advance_and_lengths_outside(cuda_device):
    p = Paged([100, 90], 2, 2, 64, 16, seed=37, track=True)
    order, seen = ordinals(p)
    p.cache.order.copy_(order)
    p.cache.seen.copy_(seen)
    p.cache.evict(60, sinks=3, recent=9, advance=False)
    assert p.lens.tolist() == [100, 90]
    p.cache.check()
    p.lens.copy_(ints([-4, 10 ** 9]))
    evicted(p, weights(p, "plain"), order, seen, 60, flagged=True)
    with pytest.raises(native.RraError):
        p.cache.evict(10, sinks=6, recent=5)
    for bad in (-1, 2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            p.cache.evict(bad)
    with pytest.raises(ValueError):
        Paged([10], 2, 2, 64, 16).cache.evict(5)


# ------------------------------------------------------------------------------------- together
def test_prefill_decode_evict_chain(cuda_device):
    """A prompt through rope, the prefill and the cache; then steps, an eviction, and more steps. With
    every block kept (tau = 1) the prefill's last row is what decode gives for the same query."""
    b, hq, hkv, n, d, ps = 2, 8, 2, 256, 128, 20
    c = cache.PagedCache.allocate(b, 320, hq, hkv, d, page_size=ps, track=True)
    table = cache.RopeTable(d, sections=[16, 24, 24])
    x = randn((b, n, hq + 2 * hkv, d), BF, 40).transpose(1, 2)
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    pos = torch.stack([i // 64, (i // 8) % 8, i % 8])[:, None].expand(3, b, n)
    q, k, v = c.append(table, pos, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], k_out=True,
                       v_out=True)
    assert c.lengths.tolist() == [n, n] == c.seen.tolist()
    prm = native.params(b, hq, hkv, n, d, 8, 1.0)
    run = native.RRAttentionPrefill(prm)
    out = run(q, k, v)
    run.check()
    last = c.decode(q[:, :, -1], add_weight=True)
    # the prefill's own bound against the oracle is 2e-2 absolute
    assert float((last.float() - out[:, :, -1].float()).abs().max()) <= 2e-2
    scale, g = 1 / math.sqrt(d), hq // hkv
    for step in range(24):
        t = randn((b, 1, hq + 2 * hkv, d), BF, 41 + step).transpose(1, 2)
        at = torch.full((3, b, 1), n + step, dtype=torch.int32, device="cuda")
        q1 = c.append(table, at, t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:])
        before, lse = c.weight.clone(), torch.empty(b, hq, device="cuda")
        out = c.decode(q1, lse=lse, add_weight=True)
        p = Paged.__new__(Paged)
        p.k, p.v, p.table, p.lens, p.cache = c.k, c.v, c.page_table, c.lengths, c
        p.hq, p.d, p.dtype, p.scale = hq, d, BF, scale
        p.check(q1[:, :, 0], out[:, :, 0], lse, c.weight, before)
        if step in (7, 8, 15):
            mirror = [f64(c.k), f64(c.v), f64(c.weight), f64(c.order)]
            orc.evict(mirror[:2], mirror[2], mirror[3], c.page_table.cpu().numpy(),
                      c.lengths.cpu().numpy(), c.seen.cpu().numpy(), 128, 4, 16)
            c.evict(128, sinks=4, recent=16)
            for ref, got in zip(mirror, (c.k, c.v, c.weight, c.order)):
                assert np.array_equal(f64(got), ref)
            assert c.lengths.tolist() == [128, 128]
            # the protected tokens are there
            for bb in range(b):
                pg, e = c.page_table[bb].long(), torch.arange(128, device="cuda")
                o = c.order[pg[e // ps], :, e % ps]
                for h in range(hkv):
                    have = set(o[:, h].tolist())
                    seen = int(c.seen[bb])
                    assert have >= set(range(4)) | set(range(seen - 16, seen))
                    assert len(have) == 128
    assert c.seen.tolist() == [n + 24] * b
    c.check()


def test_captured_steps_follow_lengths(cuda_device):
    """A captured decoding step (append, decode with weights, evict) replayed while lengths grow gives what
    eager calls give; two graphs on one workspace replay one after the other."""
    b, hq, hkv, d, ps = 3, 8, 2, 64, 16
    table = cache.RopeTable(d)
    tokens = [randn((b, hq + 2 * hkv, 1, d), BF, 60 + i) for i in range(40)]

    def fresh():
        c = cache.PagedCache.allocate(b, 48, hq, hkv, d, page_size=ps, track=True)
        c.lengths.copy_(ints([0, 11, 30]))
        c.seen.copy_(ints([0, 11, 30]))
        c.k.copy_(randn(c.k.shape, BF, 1))
        c.v.copy_(randn(c.v.shape, BF, 2))
        return c

    def step(c, x, out):
        q = c.append(table, c.seen.view(1, b, 1), x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])
        c.decode(q, out=out, add_weight=True)

    eager, outs = fresh(), []
    for i, x in enumerate(tokens):
        out = torch.empty(b, hq, 1, d, dtype=BF, device="cuda")
        step(eager, x, out)
        eager.evict(32, sinks=2, recent=8)
        outs.append(out)
    c, x, out = fresh(), torch.empty_like(tokens[0]), torch.empty_like(outs[0])
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        step(c, x, out)
    with torch.cuda.graph(graphs[1]):
        c.evict(32, sinks=2, recent=8)
    for i, t in enumerate(tokens):
        x.copy_(t)
        for g in graphs:
            g.replay()
        assert torch.equal(out, outs[i]), i
    for name in ("k", "v", "weight", "order", "lengths", "seen"):
        assert torch.equal(getattr(c, name), getattr(eager, name)), name
    c.check()
    eager.check()


def test_allocate_and_what_it_holds(cuda_device):
    c = cache.PagedCache.allocate(3, 100, 4, 2, 64, page_size=16, dtype=HF, track=True)
    assert c.k.shape == (21, 2, 16, 64) and c.k.dtype == HF and c.page_table.shape == (3, 7)
    assert not c.lengths.any() and c.weight.shape == c.order.shape == (21, 2, 16)
    with pytest.raises(AttributeError):
        c.lengths = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = c.decode(torch.ones(3, 4, 64, dtype=HF, device="cuda"))
    assert not out.any()
    none = cache.PagedCache.allocate(0, 100, 4, 2, 64)
    assert none.decode(torch.ones(0, 4, 64, dtype=BF, device="cuda")).shape == (0, 4, 64)
    for kw in (dict(weight=c.weight), dict(order=c.order, seen=c.seen)):
        with pytest.raises(ValueError):
            cache.PagedCache(c.k, c.v, c.page_table, c.lengths, heads_q=4, **kw)
    with pytest.raises(ValueError):
        cache.PagedCache(c.k, c.v.transpose(1, 2).contiguous().transpose(1, 2), c.page_table,
                         c.lengths, heads_q=4)
    with pytest.raises(ValueError):
        cache.PagedCache(c.k, c.v, c.page_table.long(), c.lengths, heads_q=4)
    with pytest.raises(native.RraError):
        cache.PagedCache(c.k, c.v, c.page_table, c.lengths, heads_q=5)


def test_other_streams(cuda_device):
    """Calls on a stream of the caller's wait for nothing but that stream; two caches at once on two."""
    a, b = (Paged([3000, 20], 8, 2, 128, 16, seed=s, track=True) for s in (70, 71))
    ref = [p.cache.decode(p.query()) for p in (a, b)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, p in enumerate((a, b)):
            with torch.cuda.stream(s[i]):
                outs[i].append(p.cache.decode(p.query()))
    mine = a.query()
    torch.cuda.synchronize()
    got = a.cache.decode(mine, stream=s[0])
    s[0].synchronize()
    assert torch.equal(got, ref[0])
    assert all(torch.equal(o, ref[i]) for i in (0, 1) for o in outs[i])
