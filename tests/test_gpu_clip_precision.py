"""The gradient norm of long tensors whose elements are so small or large that their squares leave fp32's range:
as precise as for any others, by the bound of test_gpu_clip.py (2^-20 of the norm: what a piece's squares add
up to is kept with what rounding takes from it, whatever their scale)."""
import math

import pytest
import torch

import combine_ep_route_gb300 as ep
from tests.test_gpu_clip import BF16, F32, INF, TOL, built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", (F32, BF16))
@pytest.mark.parametrize("value", (1e-16, 3e-20, 1e-30, 1e17, 7e25, 1e30))
@pytest.mark.parametrize("n", (9011, 1 << 28, (1 << 30) + 5))
def test_many_equal_elements(n, value, dtype):
    t = torch.full((n,), value, dtype=dtype, device="cuda")
    want = math.sqrt(n) * float(t[0])
    got = float(ep.clip_grad_norm([t], INF))
    assert abs(got - want) <= TOL * want


def test_all_scales_at_once():
    """Each tensor has a sum of its own scale to keep; the largest outweighs the others, and then is taken away."""
    parts = [torch.full((1 << 27,), v, device="cuda") for v in (1e-18, 0.3, 3e19)]
    for i in (3, 2, 1):
        want = math.sqrt(sum((1 << 27) * float(p[0]) ** 2 for p in parts[:i]))
        assert abs(float(ep.clip_grad_norm(parts[:i], INF)) - want) <= TOL * want
