"""Arguments of the products and the router on the host: what the entry points take and
refuse beyond the form of single fields, without a GPU."""
import ctypes as C

import pytest
import torch

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L
from combine_ep_route_gb300 import product


@pytest.fixture(scope="module")
def lib():
    from combine_ep_route_gb300 import build
    build.build()
    return L.lib()


def test_bias_on_score_is_a_flag_of_either_score(lib):
    for score, want in ((L.EP_SCORE_SOFTMAX, L.EP_OK), (L.EP_SCORE_SIGMOID, L.EP_OK), (2, L.EP_ERR_INVALID_ARG),
                        (32, L.EP_ERR_INVALID_ARG)):
        t = C.byref(L.EpTopkC(0, 8, 2, score | L.EP_BIAS_ON_SCORE, 1, L.EP_F32, 1.0))
        assert lib.ep_topk_route(t, None, None, None, None, None) == want
        assert lib.ep_topk_route_backward(t, None, None, None, None, None) == want


def test_wait_limits_outside_are_refused(lib):
    for ns in (-1, 0, 999, 60_000_000_001):
        assert lib.ep_product_wait_limit(ns) == L.EP_ERR_INVALID_ARG
    assert lib.ep_product_wait_limit(2_000_000_000) == L.EP_OK


@pytest.mark.parametrize("rows,columns", [((1 << 32) + 5, 8), (1 << 31, 8), (5, (1 << 32) + 8)])
def test_sizes_that_do_not_fit_are_refused(rows, columns):
    t = torch.empty(rows, columns, device="meta")
    for refused in (lambda: product._split(t, "x", False), lambda: product._split(t[None], "x", True),
                    lambda: product._weight(t, 1, False), lambda: product._split(t.view(1, rows, columns), "x", False)):
        with pytest.raises(ValueError):
            refused()
    most = torch.empty((1 << 31) - 1, 8, device="meta")
    assert product._split(most, "x", False) == (1, (1 << 31) - 1, 8)


def test_experts_without_counts_are_refused():
    x, w = torch.zeros(2, 4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    for call in (lambda: ep.experts_product(x, w, None), lambda: ep.experts_product_dgrad(x, w, None),
                 lambda: ep.experts_product_wgrad(x, x, None)):
        with pytest.raises(ValueError, match="counts"):
            call()
