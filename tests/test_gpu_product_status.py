"""A product's bounded wait that runs out is reported: in the call's status tensor, or without
one in the device's word that check_products reads. The limit is set to a microsecond, which the
epilogue's wait for a long reduction exceeds; every wait still ends by itself."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


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


def calls(x, w, **kw):
    """A dense product whose CTAs share the reduction, a paired one and a weight gradient."""
    cnt = torch.tensor([x.shape[0]], dtype=torch.int32, device="cuda")
    yield lambda: ep.linear(x[:64], w[:128], **kw)
    yield lambda: ep.linear(x, w, **kw)
    yield lambda: ep.experts_product(x[None], w[None], cnt, **kw)
    yield lambda: ep.linear_wgrad(w, w[:, :256].contiguous(), **kw)


def operands():
    g = torch.Generator(device="cuda").manual_seed(1)
    return [torch.randn(n, 16384, generator=g, device="cuda").to(BF16) for n in (2048, 4096)]


def test_without_a_tensor_the_device_keeps_it(short_limit):
    x, w = operands()
    for call in calls(x, w):
        call()
        with pytest.raises(ep.EpError) as e:
            ep.check_products()
        assert e.value.code == L.EP_ERR_TIMEOUT
        ep.check_products()                     # taken


def test_a_tensor_of_its_own(short_limit):
    x, w = operands()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in calls(x, w, status=status):
        status.zero_()
        call()
        assert status.item() == L.EP_ERR_TIMEOUT
    assert ep.product_status() == 0


def test_a_captured_call_reports_too(short_limit):
    x, w = operands()
    out = torch.empty(x.shape[0], w.shape[0], dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.linear(x, w, out=out)
    assert ep.product_status() == 0
    graph.replay()
    assert ep.product_status() == L.EP_ERR_TIMEOUT


def test_calls_after_it_are_right():
    x, w = operands()
    ep.set_product_wait_limit(1000)
    ep.linear(x, w)
    ep.set_product_wait_limit(2_000_000_000)
    assert ep.product_status() == L.EP_ERR_TIMEOUT
    got = ep.linear(x, w).double()
    want = x.double() @ w.double().T
    assert float((got - want).norm() / want.norm()) < 2.0 ** -8
    side = torch.cuda.Stream()
    ep.check_products(stream=side)
    ep.check_products(torch.device("cuda", 0))


def test_limits_outside_are_refused():
    for ns in (0, 999, 60_000_000_001, -1):
        with pytest.raises(ep.EpError):
            ep.set_product_wait_limit(ns)
