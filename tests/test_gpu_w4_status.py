"""A bounded wait of a product with 4-bit weights that runs out is reported as the other products' are, and
calls after it are right. The limit is a microsecond, which the waits exceed: of the tiles' epilogue for a long
reduction, of the few rows' kernel for a chunk behind 130 MB of others. Every wait ends by itself."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def short_limit():
    ep.product_status()
    ep.set_product_wait_limit(1000)
    yield
    ep.set_product_wait_limit(2_000_000_000)


def operands(rows, n, groups=1, k=32768):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(groups, rows, k, generator=g, device="cuda").to(BF16)
    codes = torch.randint(0, 256, (groups, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    return x, codes, torch.full((groups, k // 128, n), 2.0 ** -10, device="cuda", dtype=BF16)


def calls(**kw):
    """Tiles of single CTAs that share the reduction, of pairs, and the kernel for few rows."""
    x, c, s = operands(64, 256)
    yield lambda: ep.linear_w4(x[0], c[0], s[0], **kw), (x, c, s)
    x2, c2, s2 = operands(130, 512, 40, 4096 * 4)
    cnt = torch.full((40,), 130, dtype=I32, device="cuda")
    yield lambda: ep.experts_product_w4(x2, c2, s2, cnt, **kw), (x2, c2, s2)
    x3, c3, s3 = operands(1, 8192)
    yield lambda: ep.linear_w4(x3[0], c3[0], s3[0], **kw), (x3, c3, s3)


def test_without_a_tensor_the_device_keeps_it(short_limit):
    for call, _ in calls():
        call()
        with pytest.raises(ep.EpError) as e:
            ep.check_products()
        assert e.value.code == L.EP_ERR_TIMEOUT
        ep.check_products()                     # taken


def test_a_tensor_of_its_own(short_limit):
    status = torch.zeros(1, dtype=I32, device="cuda")
    for call, _ in calls(status=status):
        status.zero_()
        call()
        assert status.item() == L.EP_ERR_TIMEOUT
    assert ep.product_status() == 0


def test_calls_after_it_are_right():
    for call, (x, c, s) in calls():
        ep.set_product_wait_limit(1000)
        call()
        ep.set_product_wait_limit(2_000_000_000)
        assert ep.product_status() == L.EP_ERR_TIMEOUT
        got = call()
        e = x.shape[0] - 1
        want = x[e].double() @ ep.dequantize_weight4(c[e], s[e]).double().T
        assert float((got.view(*x.shape[:2], -1)[e].double() - want).norm() / want.norm()) < 2.0 ** -8
        ep.check_products()
