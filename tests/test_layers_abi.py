"""The products and the router on the host: every refusal of the C entry points comes
before any GPU work, calls with nothing to do succeed without a GPU, the binding
refuses what it cannot pass on, and the 64-bit definitions the GPU tests compare with
have the gradients that differences give."""
import ctypes as C

import pytest
import torch

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L
from tests import _layers64 as R

P = 0x7F0000000000      # an aligned address; never dereferenced by these tests
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from combine_ep_route_gb300 import build
    build.build()
    return L.lib()


def prod(groups=4, rows=16, k=64, n=32, act=0, out=L.EP_BF16, counts=P, status=None):
    return C.byref(L.EpProductC(groups, rows, k, n, act, out, counts, status))


BAD_PRODUCTS = [dict(groups=0), dict(groups=1025), dict(rows=-1), dict(k=0), dict(k=12), dict(n=4), dict(n=20),
                dict(k=(1 << 24) + 8), dict(groups=1024, rows=1 << 21), dict(act=-1), dict(act=6), dict(out=3),
                dict(counts=P + 2), dict(status=P + 1)]


@pytest.mark.parametrize("bad", BAD_PRODUCTS)
def test_bad_products_are_refused(lib, bad):
    a = prod(**bad)
    assert lib.ep_product(a, P, P, None, None, P, None, None) == L.EP_ERR_INVALID_ARG
    if "act" not in bad:
        assert lib.ep_product_dgrad(a, P, P, None, P, None) == L.EP_ERR_INVALID_ARG
    assert lib.ep_product_wgrad(a, P, P, 0, P, None, None) == L.EP_ERR_INVALID_ARG
    if "k" not in bad and "status" not in bad:
        bad = dict(act=2) | bad
        assert lib.ep_act_grad(prod(**bad), P, P, P, None) == L.EP_ERR_INVALID_ARG


def test_missing_and_misaligned_buffers_are_refused(lib):
    inv = L.EP_ERR_INVALID_ARG
    for at in (0, 1, 4):                       # x, w, out
        for v in (None, P + 8):
            args = [P, P, None, None, P, None]
            args[at] = v
            assert lib.ep_product(prod(), *args, None) == inv
    for at in (2, 3, 5):                       # bias, residual, preact may be absent, not misaligned
        args = [P, P, None, None, P, None]
        args[at] = P + 8
        assert lib.ep_product(prod(), *args, None) == inv
    assert lib.ep_product(None, P, P, None, None, P, None, None) == inv
    for at in (0, 1, 3):
        for v in (None, P + 8):
            args = [P, P, None, P]
            args[at] = v
            assert lib.ep_product_dgrad(prod(), *args, None) == inv
    assert lib.ep_product_dgrad(prod(act=2), P, P, None, P, None) == inv     # an activation needs its input
    assert lib.ep_product_dgrad(prod(act=0), P, P, P, P, None) == inv
    for args in ((None, P, 0, P, None), (P, None, 0, P, None), (P, P, 0, None, None), (P, P, 2, P, None),
                 (P + 8, P, 0, P, None), (P, P + 8, 0, P, None), (P, P, 0, P + 8, None), (P, P, 0, P, P + 8)):
        assert lib.ep_product_wgrad(prod(), *args, None) == inv
    assert lib.ep_product_wgrad(prod(act=1), P, P, 0, P, None, None) == inv
    for args in ((None, P, P), (P, None, P), (P, P, None), (P + 8, P, P), (P, P + 8, P), (P, P, P + 8)):
        assert lib.ep_act_grad(prod(act=3), *args, None) == inv
    assert lib.ep_act_grad(prod(act=0), P, P, P, None) == inv
    assert lib.ep_act_grad(prod(act=3, out=L.EP_F32), P, P, P, None) == inv


def test_nothing_to_do_is_not_an_error(lib):
    a = prod(rows=0)
    assert lib.ep_product(a, None, P, None, None, None, None, None) == L.EP_OK
    assert lib.ep_product_dgrad(a, None, P, None, None, None) == L.EP_OK
    assert lib.ep_product_wgrad(a, None, None, 1, P, None, None) == L.EP_OK
    assert lib.ep_act_grad(prod(rows=0, act=2), None, None, None, None) == L.EP_OK
    t = C.byref(L.EpTopkC(0, 8, 2, 0, 1, L.EP_F32, 1.0))
    assert lib.ep_topk_route(t, None, None, None, None, None) == L.EP_OK
    assert lib.ep_topk_route_backward(t, None, None, None, None, None) == L.EP_OK


@pytest.mark.parametrize("bad", [(-1, 8, 2, 0, 1, 2), (4, 0, 1, 0, 1, 2), (4, 1025, 2, 0, 1, 2), (4, 8, 0, 0, 1, 2),
                                 (4, 8, 9, 0, 1, 2), (4, 64, 17, 0, 1, 2), (4, 8, 2, 2, 1, 2), (4, 8, 2, 0, 2, 2),
                                 (4, 8, 2, 0, 1, 3)])
def test_bad_routers_are_refused(lib, bad):
    t = C.byref(L.EpTopkC(*bad, 1.0))
    assert lib.ep_topk_route(t, P, None, P, P, None) == L.EP_ERR_INVALID_ARG
    assert lib.ep_topk_route_backward(t, P, P, P, P, None) == L.EP_ERR_INVALID_ARG


def test_router_buffers_are_checked(lib):
    t = C.byref(L.EpTopkC(4, 8, 2, 0, 1, L.EP_F32, 1.0))
    for args in ((None, None, P, P), (P, None, None, P), (P, None, P, None), (P + 2, None, P, P), (P, P + 2, P, P),
                 (P, None, P + 2, P), (P, None, P, P + 2)):
        assert lib.ep_topk_route(t, *args, None) == L.EP_ERR_INVALID_ARG
    for at in range(4):
        for v in (None, P + 2):
            args = [P, P, P, P]
            args[at] = v
            assert lib.ep_topk_route_backward(t, *args, None) == L.EP_ERR_INVALID_ARG


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 16, dtype=BF16), torch.zeros(8, 16, dtype=BF16)
    cnt = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: ep.linear(x, w), lambda: ep.linear_dgrad(x[:, :8].contiguous(), w),
                 lambda: ep.linear_wgrad(x, x), lambda: ep.act_grad(x, x, "silu"),
                 lambda: ep.experts_product(x[None], w[None], cnt),
                 lambda: ep.experts_product_dgrad(x[None, :, :8].contiguous(), w[None], cnt),
                 lambda: ep.experts_product_wgrad(x[None], x[None], cnt),
                 lambda: ep.route_topk(torch.zeros(4, 8), 2),
                 lambda: ep.route_topk_backward(torch.zeros(4, 2), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("act", ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"))
def test_definition_slopes_match_differences(act):
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.013
    h = 1e-5
    value = lambda v: R.act64(v, act)[0]  # noqa: E731
    slope = (value(z + h) - value(z - h)) / (2 * h)
    assert (slope - R.act64(z, act)[1]).abs().max() < 1e-8


def test_definition_gradients_match_differences():
    g = torch.Generator().manual_seed(1)
    dy, w = torch.randn(5, 8, generator=g, dtype=R.D), torch.randn(8, 6, generator=g, dtype=R.D)
    z = torch.randn(5, 12, generator=g, dtype=R.D)
    d, _ = R.dgrad(dy, w, "swiglu", z, torch.float32)
    v = torch.randn(5, 12, generator=g, dtype=R.D)
    loss = lambda z: float((dy * ((R.act64(z[:, :6], "silu")[0] * z[:, 6:]) @ w.T)).sum())  # noqa: E731
    h = 1e-6
    assert abs((loss(z + h * v) - loss(z - h * v)) / (2 * h) - float((d * v).sum())) < 1e-6
