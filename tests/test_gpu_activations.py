"""The activations far from zero, where a value is small and has to keep its digits: values
(through a product whose pre-activation is exact) and slopes against 64 bits, with bounds
relative to the result."""
import math

import pytest
import torch

import combine_ep_route_gb300 as ep

pytestmark = pytest.mark.gpu
BF16, F32, D = torch.bfloat16, torch.float32, torch.float64
C, A = math.sqrt(2 / math.pi), 0.044715


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def values(f32_of_z):
    """bf16 numbers from -8 to -2 and from 2 to 8, every one of them."""
    pos = torch.arange(0x4000, 0x4101, dtype=torch.int32).to(torch.int16).view(BF16)
    return torch.cat((-pos, pos)).to(f32_of_z).cuda()


def forward(z, act, dtype):
    """act(z) by a product with one non-zero term per output: z * 1, exact in fp32."""
    x, w = torch.zeros(z.numel(), 8, dtype=BF16, device="cuda"), torch.zeros(8, 8, dtype=BF16, device="cuda")
    x[:, 0], w[:, 0] = z, 1
    return ep.linear(x, w, act=act, out_dtype=dtype)[:, 3]


def slope(z, act):
    rows = z.view(-1, 1).expand(-1, 8).contiguous()
    return ep.act_grad(torch.ones_like(rows), rows, act)[:, 5]


def fits(got, want, fp32_error):
    """Between the roundings, to the result's type, of what the fp32 evaluation may come to."""
    ends = want * (1 - fp32_error), want * (1 + fp32_error)
    lo, hi = torch.minimum(*ends).to(got.dtype), torch.maximum(*ends).to(got.dtype)
    bad = ~((lo <= got) & (got <= hi))
    worst = ((got.to(D) - want) / want).abs().max()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst relative error {float(worst):.2e}"


def sigmoid_error(a):
    """Relative error of 1 / (1 + 2^x) for x = a log2(e): six roundings of the exponent, which
    scale with it, and a unit or two of each of exponential, sum and reciprocal."""
    return (6 * a.abs() + 16) * 2.0 ** -24


@pytest.mark.parametrize("dtype", (BF16, F32))
def test_gelu_tanh_tail(dtype):
    z = values(BF16)
    z64 = z.to(D)
    u2 = 2 * C * (z64 + A * z64 ** 3)
    fits(forward(z, "gelu_tanh", dtype), z64 * torch.sigmoid(u2), sigmoid_error(u2))


def test_gelu_tanh_slope_tail():
    z = values(BF16)
    z64 = z.to(D)
    s, u2 = torch.sigmoid(2 * C * (z64 + A * z64 ** 3)), 2 * C * (z64 + A * z64 ** 3)
    rest = z64 * 2 * C * (1 + 3 * A * z64 ** 2)
    # s + s (1 - s) rest: the terms' errors over their sum
    want = s + s * (1 - s) * rest
    err = (s * sigmoid_error(u2) + (s * (1 - s) * rest).abs() * 2 * sigmoid_error(u2)
           + (z64 > 0) * rest * s * 2.0 ** -23) / want.abs()
    fits(slope(z, "gelu_tanh"), want, err)


def test_gelu_tanh_of_huge_values():
    z = torch.tensor([1e3, 3e18, 1e20, 3e38], device="cuda").to(BF16)
    for sign, want in ((1, 1.0), (-1, 0.0)):
        assert (slope(sign * z, "gelu_tanh") == want).all()
        assert torch.equal(forward(sign * z, "gelu_tanh", BF16), (sign * z * want).to(BF16))
    nan = torch.tensor([float("nan")], device="cuda", dtype=BF16)
    assert torch.isnan(slope(nan, "gelu_tanh")).all() and torch.isnan(forward(nan, "gelu_tanh", F32)).all()


def normal_parts(z):
    """64-bit (Phi, phi) and the relative error of a tail: fit 3.8e-7, and an exponential whose
    argument z^2 / 2 is rounded three times."""
    phi = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return 0.5 * torch.erfc(-z * math.sqrt(0.5)), phi, (16 + 3 * z * z) * 2.0 ** -24


@pytest.mark.parametrize("dtype", (BF16, F32))
def test_gelu_tail(dtype):
    z = values(BF16)
    cdf, _, err = normal_parts(z.to(D))
    # above zero the tail's error is small beside one
    err = torch.where(z < 0, err, err * (1 - cdf) + 4 * 2.0 ** -24)
    fits(forward(z, "gelu", dtype), z.to(D) * cdf, err)


def test_gelu_slope_tail():
    z = values(BF16)
    z64 = z.to(D)
    cdf, phi, err = normal_parts(z64)
    want = cdf + z64 * phi
    tail = torch.where(z < 0, cdf * err, (1 - cdf) * err + 2 * 2.0 ** -24)
    fits(slope(z, "gelu"), want, (tail + (z64 * phi).abs() * err + want.abs() * 2.0 ** -23) / want.abs())


def test_gelu_of_huge_values():
    z = torch.tensor([1e3, 3e18, 1e20, 3e38], device="cuda").to(BF16)
    for sign, want in ((1, 1.0), (-1, 0.0)):
        assert (slope(sign * z, "gelu") == want).all()
        assert torch.equal(forward(sign * z, "gelu", BF16), (sign * z * want).to(BF16))
