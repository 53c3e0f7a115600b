"""Clipping by factors below the smallest normal float: norms past the largest float, or small bounds and large
elements.

Bounds. max_norm as a float is taken as it is; the norm is right to 2^-20, the factor is rounded (2^-24) and so
is the product with it (2^-24): 2^-19 of the value in all. A second product, by a power of two, rounds only below the
smallest normal float, to half its step of 2^-149; bf16 adds its own half unit of 2^-8, or half a step of 2^-133 there."""
import math

import pytest
import torch

import combine_ep_route_gb300 as ep
from tests.test_gpu_clip import BF16, F32, built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
CASES = [(3e38, 100, 1.0), (3e38, 1 << 20, 1.0), (3e38, (1 << 24) + 3, 1.0), (3e38, 1 << 24, 1e3), (3e38, 1 << 30, 1e-10), (1e20, 64, 1e-25),
         (1e10, 101, 1e-33), (1e5, 1001, 1e-37), (1.0, 77, 1e-37), (1.0, 77, 1e-39), (1e30, 5000, 1e-44), (1e30, 5000, 0.0), (2.0, 9, 1e-3)]


@pytest.mark.parametrize("dtype", (F32, BF16))
@pytest.mark.parametrize("inplace", (True, False))
@pytest.mark.parametrize("size,n,max_norm", CASES)
def test_small_factors(size, n, max_norm, inplace, dtype):
    g = torch.Generator(device="cuda").manual_seed(n % 1000)
    t = (size * (2 * torch.rand(n, generator=g, device="cuda") - 1)).to(dtype)
    norm = math.sqrt(sum(float(c.double().square().sum()) for c in t.split(1 << 26)))
    factor = float(torch.tensor(max_norm)) / norm
    out = None if inplace else torch.empty_like(t)
    before = t.clone()
    ep.clip_grad_norm([t], max_norm, out=None if inplace else [out])
    got = t if inplace else out
    for b, o in zip(before.split(1 << 26), got.split(1 << 26)):
        exact = b.double() * factor
        off = exact.abs() * 2.0 ** -19 + 2.0 ** -149
        if dtype is BF16:
            off = off + exact.abs() * 2.0 ** -8 + 2.0 ** -134
        assert ((o.double() - exact).abs() <= off).all()
