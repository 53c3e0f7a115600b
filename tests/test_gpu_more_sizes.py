"""The 4-bit products, the balance loss and the gradient norm where offsets pass 32 bits, and on many rows."""
import math

import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 100e9:
        pytest.skip("needs the memory")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


def weight(g, groups, n, k, group):
    codes = torch.randint(0, 256, (groups, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    return codes, torch.full((groups, k // group, n), k ** -0.5 / 4, dtype=BF16, device="cuda")


def check(y, x, codes, scales, kind="int4"):
    want, off, _, _ = R.forward(x, ep.dequantize_weight4(codes, scales, kind), None, "none", None, BF16)
    assert ((y.double() - want).abs() <= off).all()


def test_rows_far_into_x():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(3, 90000, 32768, dtype=BF16, device="cuda")       # 8.8e9 elements
    x[2, :17] = rand(g, 17, 32768)
    codes, scales = weight(g, 3, 24, 32768, 128)
    y = ep.experts_product_w4(x, codes, scales, torch.tensor([0, 0, 17], dtype=I32, device="cuda"))
    check(y[2, :17], x[2, :17], codes[2], scales[2])
    x[1, -130:] = rand(g, 130, 32768)
    y = ep.linear_w4(x[1], codes[1], scales[1])                       # 90000 rows of a dense product
    check(y[-130:], x[1, -130:], codes[1], scales[1])
    assert (y[:-130] == 0).all()
    ep.check_products()


def test_experts_far_into_the_codes():
    g = torch.Generator(device="cuda").manual_seed(2)
    codes, scales = weight(g, 40, 16384, 16384, 128)                  # 5.4 GB
    x = rand(g, 40, 20, 16384)
    cnt = torch.zeros(40, dtype=I32, device="cuda")
    cnt[39] = 20
    y = ep.experts_product_w4(x, codes, scales, cnt)
    check(y[39], x[39], codes[39], scales[39])
    ep.check_products()


def test_one_row_of_a_wide_product():
    g = torch.Generator(device="cuda").manual_seed(3)
    n = (1 << 18) + 1032
    codes, scales = weight(g, 1, n, 32768, 64)                        # 4.3 GB
    x = rand(g, 1, 32768)
    y = ep.linear_w4(x, codes[0], scales[0])
    check(y[:, -2000:], x, codes[0, -2000:], scales[0, :, -2000:])
    check(y[:, :500], x, codes[0, :500], scales[0, :, :500])
    ep.check_products()


def test_many_tokens():
    T, E = (1 << 23) + 3, 512                                         # 4.3e9 logits
    z = torch.zeros(1, T, E, dtype=BF16, device="cuda")
    ids = (torch.arange(T, device="cuda") % E).to(I32).view(1, T, 1)
    z[0, -1, 5] = 20.0
    losses, counts = ep.balance_loss(z, ids)
    want = torch.bincount(ids.flatten().long(), minlength=E)
    assert torch.equal(counts.long(), want)
    # probabilities are even but for the last token's, which is one of 8 million
    assert abs(float(losses[0]) - 1) < 1e-5
    last = (20 + math.log1p((E - 1) * math.exp(-20))) ** 2
    mean = ((T - 1) * math.log(E) ** 2 + last) / T
    assert abs(float(losses[1]) - mean) <= 2.0 ** -17 * (mean + 1)
    d = ep.balance_loss_backward(torch.tensor([0.0, float(T)], device="cuda"), z, counts, 1)
    soft = torch.softmax(z[0, -1].double(), 0)
    exact = 2 * (20 + math.log1p((E - 1) * math.exp(-20))) * soft
    assert ((d[0, -1].double() - exact).abs() <= exact * (2.0 ** -8 + 2.0 ** -15) + 1e-12).all()
    even = 2 * math.log(E) / E
    assert ((d[0, T // 2].double() - even).abs() <= even * (2.0 ** -8 + 2.0 ** -15)).all()


@pytest.mark.parametrize("dtype", (BF16, F32))
def test_a_tensor_of_more_than_two_thousand_million(dtype):
    n = (1 << 31) + 77
    t = torch.ones(n, dtype=dtype, device="cuda")
    t[-1] = 1024.0
    small = torch.full((5,), 2.0, device="cuda")
    want = math.sqrt(n - 1 + 1024.0 ** 2 + 20)
    norm = ep.clip_grad_norm([t, small], want / 4)
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    # the factor: max_norm as fp32 (2^-24) over a norm right to 2^-20, rounded (2^-24); the product rounded (2^-24, or
    # in bf16 to a power of two that is near): 2^-19 in all
    got = torch.cat((t[:1], t[n // 2:n // 2 + 1], t[-1000:], small)).double()
    exact = torch.tensor([0.25, 0.25] + [0.25] * 999 + [256.0] + [0.5] * 5, dtype=torch.float64, device="cuda")
    assert ((got - exact).abs() <= exact * 2.0 ** -19).all()
