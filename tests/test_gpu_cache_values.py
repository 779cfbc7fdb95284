"""Decode attention where the values or the weights are out of the ordinary: weights far below the
largest one, values at the end of the type's range. Against the definition in 64 bits; the tolerances of each test are derived beside it.
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
    do not. All keys are 0, so all weights are equal (1 / n, exact but for the reciprocal of n, 2^-23);
    each truncated addition is off by 2^-23 of the sum of the magnitudes, and a warp makes at most
    n / 16 + 1 of them, the joins 300 more. What is past the largest value by less than half a step rounds
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
