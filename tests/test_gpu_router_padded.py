"""A router whose number of experts is not a multiple of 8: its weight padded with rows whose
bias is minus infinity, which masks the experts that do not exist."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R
from tests.test_gpu_router import FORMS, WEIGHT_TOL, built  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32, D = torch.bfloat16, torch.float32, torch.float64


@pytest.mark.parametrize("score,renormalize", FORMS)
@pytest.mark.parametrize("T,E,k,h", [(37, 60, 8, 264), (5, 4, 2, 72), (130, 100, 4, 136), (3, 1, 1, 64)])
def test_padded_router(T, E, k, h, score, renormalize):
    g = torch.Generator(device="cuda").manual_seed(E)
    x, w = (torch.randn(n, h, generator=g, device="cuda").to(BF16) for n in (T, E))
    padded = -(-E // 8) * 8
    wide = torch.zeros(padded, h, dtype=BF16, device="cuda")
    wide[:E] = w
    bias = torch.zeros(padded, dtype=BF16, device="cuda")
    bias[E:] = float("-inf")
    logits = ep.linear(x, wide, bias=bias, out_dtype=F32)
    assert torch.isinf(logits[:, E:]).all()
    ids, weights = ep.route_topk(logits, k, score=score, renormalize=renormalize)
    want_ids, want = R.route(logits[:, :E], k, score, renormalize, None, 1.0)
    assert torch.equal(ids.cpu(), want_ids)
    assert ((weights.cpu().double() - want).abs() <= WEIGHT_TOL * want + 1e-37).all()
    dw = torch.randn(T, k, generator=g, device="cuda")
    dlogits = ep.route_topk_backward(dw, logits, ids, score=score, renormalize=renormalize)
    assert (dlogits[:, E:] == 0).all()
    d = dlogits.to(BF16)
    dx, edx = R.dgrad(d[:, :E], w, "none", None, F32)
    assert ((ep.linear_dgrad(d, wide, out_dtype=F32).double() - dx).abs() <= edx).all()
    dwide = ep.linear_wgrad(d, x, out_dtype=F32)
    want, e, _, _ = R.wgrad(d[:, :E], x, F32)
    assert ((dwide[:E].double() - want).abs() <= e).all() and (dwide[E:] == 0).all()
