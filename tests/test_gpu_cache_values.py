"""Decode attention where the values or the weights are out of the ordinary: weights far below the
largest one, values at the end of the type's range,
infinities and NaN among the values. Against the definition in 64 bits; the tolerances of each test are derived beside it.
"""
import math

import numpy as np
import pytest
import torch

from long_context_prefill_rr_b200 import cache

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("nats", [17.5, 14.5, 11.0])
@pytest.mark.parametrize("group,d", [(1, 64), (12, 128)])
def test_decode_long_tail_behind_a_sink(cuda_device, dtype, nats, group, d):
    """Entry 0 takes nearly all the weight and has the value 0; the output is what the other entries
    add up to, each of them e^-nats. 96 sequences share the pages, so that the blocks' runs are longer
    than an item and a warp adds thousands of small weights to its large one.

    Logits: 0 and nats, whose products are exact; scaled to log2 nats * log2(e) is off by 2^-24 of
    itself for the factor and again for the product, 2^-18.6 absolute at most, and the exponential by
    2^-22: 2^-18 of a small weight. The weights' two parts keep 2^-17 of it (bf16), or (fp16)
    2^-22 of it and 2^-40 of the largest, which is 2^-14.7 of the smallest here, e^-17.5. Of sums over
    n entries each warp takes n / 4, 16 at a time (n / 64 products, each truncated to 2^-23, and n / 32
    additions of a thread's weights, each rounded to 2^-24), so 2^-13 + 2^-14 for n = 32768."""
    n, batch, hkv, ps = 32768, 96, 2, 64
    pages = n // ps
    k = torch.zeros(pages, hkv, ps, d, dtype=dtype, device="cuda")
    v = torch.ones(pages, hkv, ps, d, dtype=dtype, device="cuda")
    v[..., ::2] = -0.5
    k[0, :, 0, 3], v[0, :, 0] = 1.0, 0.0
    table = ints([list(range(pages))]).expand(batch, pages).contiguous()
    c = cache.PagedCache(k, v, table, ints([n] * batch), heads_q=hkv * group, softmax_scale=1.0)
    q = torch.zeros(batch, hkv * group, d, dtype=dtype, device="cuda")
    q[..., 3] = nats
    lse = torch.empty(batch, hkv * group, device="cuda")
    out = c.decode(q, lse=lse)
    tail = (n - 1) * math.exp(-nats)
    ref = tail / (1.0 + tail) * torch.tensor([-0.5, 1.0], dtype=torch.float64).repeat(d // 2)
    tol = half_step(dtype) + 2.0 ** -18 + 2.0 ** -14.7 + 2.0 ** -13 + 2.0 ** -14
    err = ((out.double().cpu() - ref) / ref).abs()
    assert float(err.max()) <= tol, float(err.max())
    # 2^-18 of the tail's share, the sums as above, the logarithm and the change of base
    assert float((lse.double().cpu() - nats - math.log1p(tail)).abs().max()) <= \
        2.0 ** -18 + 2.0 ** -14 + 2.0 ** -21 * (1 + nats)
    c.check()


# ------------------------------------------------------------------------------------- large values
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group,d", [(1, 128), (12, 64)])
@pytest.mark.parametrize("n", [3, 500, 20000])
def test_decode_values_at_the_end_of_the_range(cuda_device, dtype, group, d, n):
    """The type's largest values, of one sign and of both: their sums pass fp32's range in bf16, their means
    do not. All keys are 0, so all weights are equal; each truncated addition is off by 2^-23 of the sum of
    the magnitudes, and a warp makes at most n / 16 + 1 of them, the joins, of 148 * 3 pieces at most but
    fewer here, and the quotients by the sums of the weights (2^-22 each, three of them) 300 more. What is past the largest value by less than half a step rounds
    to it, and the mean of one value cannot be more."""
    hkv, ps, top = 2, 20, torch.finfo(dtype).max
    pages = -(-n // ps)
    k = torch.zeros(pages, hkv, ps, d, dtype=dtype, device="cuda")
    v = torch.full((pages, hkv, ps, d), top, dtype=dtype, device="cuda")
    v[..., 1::4] = -top
    g = torch.Generator(device="cuda").manual_seed(n)
    v[..., 2::4] *= torch.randint(0, 2, v[..., 2::4].shape, generator=g, device="cuda").to(dtype) * 2 - 1
    c = cache.PagedCache(k, v, ints([list(range(pages))]), ints([n]), heads_q=hkv * group)
    out = c.decode(torch.ones(1, hkv * group, d, dtype=dtype, device="cuda"))
    ref = v.transpose(0, 1).reshape(hkv, pages * ps, d)[:, :n].double().mean(1)
    ref = ref.repeat_interleave(group, 0)[None]
    tol = half_step(dtype) * ref.abs() + top * ((n / 16 + 301) * 2.0 ** -23 + 2.0 ** -22)
    assert out.isfinite().all()
    assert ((out.double() - ref).abs() <= tol).all()
    c.check()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group,d", [(1, 128), (12, 64)])
@pytest.mark.parametrize("n", [3, 500, 20000])
@pytest.mark.parametrize("size", ["smallest", "subnormal"])
def test_decode_values_at_the_small_end_of_the_range(cuda_device, dtype, group, d, n, size):
    """The type's smallest values, of one sign and of both. Products, sums and means have steps of 2^-149 in
    fp32, which is 2^-23 of bf16's smallest normal value: n / 16 + 301 additions as above, for each head's
    n products as much again in all. A subnormal output rounds to a step of the smallest subnormal."""
    hkv, ps, low = 2, 20, torch.finfo(dtype).tiny * (1.0 if size == "smallest" else 0.25)
    step = torch.finfo(dtype).tiny * torch.finfo(dtype).eps       # the smallest subnormal
    pages = -(-n // ps)
    k = torch.zeros(pages, hkv, ps, d, dtype=dtype, device="cuda")
    v = torch.full((pages, hkv, ps, d), low, dtype=dtype, device="cuda")
    v[..., 1::4] = -low
    g = torch.Generator(device="cuda").manual_seed(n)
    v[..., 2::4] *= torch.randint(0, 2, v[..., 2::4].shape, generator=g, device="cuda").to(dtype) * 2 - 1
    assert float(v.double().abs().min()) == low
    c = cache.PagedCache(k, v, ints([list(range(pages))]), ints([n]), heads_q=hkv * group)
    out = c.decode(torch.ones(1, hkv * group, d, dtype=dtype, device="cuda"))
    ref = v.transpose(0, 1).reshape(hkv, pages * ps, d)[:, :n].double().mean(1)
    ref = ref.repeat_interleave(group, 0)[None]
    tol = step / 2 + low * 2 * ((n / 16 + 301) * 2.0 ** -23 + 2.0 ** -22) * \
        (4 if size == "subnormal" else 1)                         # the steps of 2^-149 are larger beside these
    assert ((out.double() - ref).abs() <= tol).all(), float(((out.double() - ref).abs() / low).max())
    assert out[..., 0].any()
    c.check()


# --------------------------------------------------------------------- values that are not finite
def cached(n, hkv, d, ps, dtype, seed):
    """A cache of one sequence whose pages are in order: the contiguous keys and values behind its pages'
    views are k, v [hkv, n, d]."""
    pages = -(-n // ps)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(hkv, pages * ps, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    def paged(x):
        return x.view(hkv, pages, ps, d).transpose(0, 1)
    return k, v, lambda hq, **kw: cache.PagedCache(paged(k), paged(v), ints([list(range(pages))]), ints([n]),
                                                   heads_q=hq, **kw)


def by_definition(q, k, v, n, scale):
    """out, lse [hq, ...] in 64 bits; entries with a logit of -inf are left out."""
    hq, hkv = q.shape[0], k.shape[0]
    q, k, v = (x.double().cpu().numpy() for x in (q, k[:, :n], v[:, :n]))
    out, lse = np.zeros(q.shape), np.full(hq, -math.inf)
    reach = np.zeros(hq)
    with np.errstate(invalid="ignore", over="ignore"):
        for h in range(hq):
            s = k[h // (hq // hkv)] @ q[h] * scale
            live = s > -math.inf
            if live.any():
                top = s[live].max()
                p = np.exp(s[live] - top)
                # no weight is 0, so that an infinite value is infinite behind any of them
                p = np.maximum(p / p.sum(), 1e-300)
                out[h] = (p[:, None] * v[h // (hq // hkv)][live]).sum(0)
                lse[h] = top + math.log(np.exp(s[live] - top).sum())
                reach[h] = (np.abs(k[h // (hq // hkv)][live]) @ np.abs(q[h])).max() * scale
    return out, lse, reach


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group,d", [(4, 64), (5, 128), (11, 64), (16, 128)])
@pytest.mark.parametrize("n,ps", [(1, 16), (90, 7), (3001, 16), (40000, 64)])
def test_decode_values_that_are_not_finite(cuda_device, dtype, group, d, n, ps):
    """Infinities and NaN among the values, in entries that have a weight (some of them e^-200 of the
    largest) and in entries whose logit is -inf, which do not count. The other outputs as always: a logit is
    off by delta = (d + 4) 2^-23 scale sum |q k|, a weight by that and 2^-21, its two parts by 2^-17; the
    output by twice their sum of max |v|, and half a step."""
    hkv = 2
    k, v, make = cached(n, hkv, d, ps, dtype, n + d)
    scale = 1 / math.sqrt(d)
    q = torch.randn(hkv * group, d, generator=torch.Generator().manual_seed(n)).cuda().to(dtype)
    q[:, 0], k[:, :, 0] = 1.0, 0.0
    rng = np.random.default_rng(n + d)
    vmax = float(v.abs().max())
    for i in range(12 if n > 1 else 1):
        e, h = int(rng.integers(n)), int(rng.integers(hkv))
        v[h, e, int(rng.integers(d))] = (math.inf, -math.inf, math.nan)[i % 3]
        if i % 4 == 1:
            k[h, e, 0] = -200.0 * math.sqrt(d)                      # a weight of e^-200
    if n > 1:
        v[0, n // 2, 5], v[0, n // 3, 5] = math.inf, -math.inf      # NaN together
        v[1, n // 2, 6], v[1, n // 3, 6] = -math.inf, -math.inf
        gone = rng.choice(n, size=n // 8, replace=False)            # no weight at all
        gone = gone[(gone != n // 2) & (gone != n // 3)]
        k[:, gone, 0] = -math.inf
        v[:, gone[::2], 7:9] = math.nan
        v[:, gone[1::2], 8:10] = math.inf
    # and behind the last entry
    k[:, n:], v[:, n:] = math.nan, math.nan
    c = make(hkv * group)
    lse = torch.zeros(1, hkv * group, device="cuda")
    out = c.decode(q[None], lse=lse)[0].double().cpu().numpy()
    ref, rlse, reach = by_definition(q, k, v, n, scale)
    assert np.isnan(ref).any() == (n > 1) and np.isinf(ref).any() and (n == 1 or (~np.isfinite(ref)).sum() < ref.size / 2)
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    assert np.array_equal(out[np.isinf(ref)], ref[np.isinf(ref)])
    ok = np.isfinite(ref)
    delta = (d + 4) * 2.0 ** -23 * reach
    tol = half_step(dtype) * np.abs(ref) + (2 * vmax * (delta + 2.0 ** -17 + 2.0 ** -20))[:, None] + \
        (2.0 ** -25 if dtype == HF else 0)
    assert (np.abs(out[ok] - ref[ok]) <= tol[ok]).all()
    assert (np.abs(lse[0].double().cpu().numpy() - rlse) <=
            delta + 2.0 ** -21 * (1 + np.abs(rlse))).all()
    c.check()


def test_decode_nothing_left_but_values_that_are_not_finite(cuda_device):
    k, v, make = cached(50, 2, 64, 16, BF, 1)
    k[:], v[:] = -math.inf, math.nan
    q = torch.ones(1, 4, 64, dtype=BF, device="cuda")
    lse = torch.zeros(1, 4, device="cuda")
    assert not make(4).decode(q, lse=lse).any() and (lse == -math.inf).all()
    k[:, 20] = 0.0
    v[:, 20] = 3.0
    assert (make(4).decode(q, lse=lse) == 3).all() and not lse.any()
    v[0, 20] = math.inf
    out = make(4).decode(q, lse=lse)[0]
    assert (out[:2] == math.inf).all() and (out[2:] == 3).all() and not lse.any()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_decode_logits_that_are_not_finite(cuda_device, bad):
    """A logit of +inf or NaN: NaN for its head alone, also where its values are infinite."""
    k, v, make = cached(300, 1, 64, 16, HF, 2)
    k[0, :, :2], k[0, 100, 0] = 0.0, bad
    v[0, 100, 3], v[0, 200, 4] = math.inf, math.inf
    q = torch.randn(1, 3, 64, generator=torch.Generator().manual_seed(3)).to(HF).cuda()
    q[0, :, 0] = torch.tensor([1.0, 2.0, -1.0], dtype=HF)
    shape = (19, 1, 16)
    weight = torch.zeros(shape, device="cuda")
    c = make(3, weight=weight, order=torch.zeros(shape, dtype=torch.int32, device="cuda"),
             seen=ints([300]))
    lse = torch.zeros(1, 3, device="cuda")
    out = c.decode(q, lse=lse, add_weight=True)
    assert out[0, :2].isnan().all() and lse[0, :2].isnan().all()
    if bad == math.inf:                    # the third head's logit is -inf: absent, with its value
        assert out[0, 2, 4] == math.inf and out[0, 2, 3].isfinite() and lse[0, 2].isfinite()
        assert out[0, 2].isfinite().sum() == 63
    else:
        assert out[0, 2].isnan().all()
    assert weight.view(-1)[:300].isnan().all()
