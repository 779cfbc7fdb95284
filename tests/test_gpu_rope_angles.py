"""Rotations where the sine and cosine of the kernel are least exact, at the ends of its quadrants.

The kernel takes the angle as a quadrant and a rest x, |x| <= pi / 4, and both series in fp32. u = 2^-24 is
half a step, relative. Errors, in u:

* x: conversion of the rest to fp32, the factor 2 pi / 2^32 and the product, 1 each, of pi / 4: 2.36. The last
  bit of the angle, 2^-32 of a turn, and the frequency's, 2^-65 of a turn at positions up to 2^31: 0.03.
* sine x + x^3 p, p = -1/6 + x^2 / 120 ...: p is off by 0.34 (its constant 0.17, its rounding 0.16, the rest
  0.02), x^3 by 2 of itself, so x^3 p by 0.48 * 0.34 + 0.078 * 2 = 0.32; the last sum rounds by 0.5; cut
  off is x^11 / 11! = 0.03. Together 0.86.
* cosine 1 + x^2 p, p = -1/2 + x^2 / 24 ...: p is off by 0.33, x^2 by 1 of itself, so the product by
  0.62 * 0.33 + 0.29 = 0.50; the last sum rounds by 0.5; cut off is x^10 / 10! = 0.41. Together 1.41.
* a result a cos - b sin: sqrt(0.86^2 + 1.41^2) = 1.66 of |(a, b)| for these, the angle's 2.39, the products
  and the sum 2. In all 6.05 u of |(a, b)|, less than 2^-21, and half a step of the element type.

Near pi / 4 and its odd multiples the two products nearly cancel for a = +-b, so the half step is small and
the sine and cosine show.
"""
import math

import numpy as np
import pytest
import torch

from long_context_prefill_rr_b200 import cache
from oracle import cache_oracle as orc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotation_at_the_ends_of_the_quadrants(cuda_device, dtype, inverse):
    d, pairs, n = 128, 64, 16
    # pair i: an odd eighth of a turn, and 2^-(i / 2) of a radian before or behind it
    freq = [2 * math.pi * (2 * (i // 2 % 4) + 1) / 8 + (-1.0) ** i * 2.0 ** (-2 - i // 2) for i in range(pairs)]
    table = cache.RopeTable(d, inv_freq=freq)
    pos = torch.ones(1, 1, n, dtype=torch.int32, device="cuda")
    pos[0, 0, n // 2:] = -1
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.rand(1, 4, n, d, generator=g, device="cuda") + 0.5
    x[:, 1] = 1.0
    x[:, :, :, pairs:] = x[:, :, :, :pairs]
    x[:, 2:, :, :pairs] *= -1.0
    x = x.to(dtype)
    got = cache.rope(table, pos, x, inverse=inverse).double().cpu().numpy()
    x64 = x.double().cpu().numpy()
    ref = orc.rotate(x64, pos.cpu().numpy(), freq, [0] * pairs, "halves", inverse)
    size = np.tile(np.hypot(x64[..., :pairs], x64[..., pairs:]), 2)
    off = size * (2.0 ** -21 + 8 * math.pi * 2.0 ** -52)
    half = torch.finfo(dtype).eps / 2 * (np.abs(ref) + off)
    if dtype == torch.float16:
        half = np.maximum(half, 2.0 ** -25)       # results below 2^-14 have steps of 2^-24
    err = np.abs(got - ref)
    assert (np.abs(ref) < 2.0 ** -20).any()       # the cancelling ones are among them
    assert (err <= half + off).all(), float((err / (half + off)).max())
