"""The top-k router and its gradient against 64-bit definitions: exact choices (ties,
masks, NaN), weights to a few units of fp32, gradients by autograd and by differences."""
import math

import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
FORMS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]
# an exponential of a rounded difference (|z| up to 16: 2^-20), a sum of up to 1024 terms by a
# tree of 32 and a chain of 32 (2^-18.9), a division
WEIGHT_TOL = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def logits_of(T, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (2 * torch.randn(T, E, generator=g)).to(dtype).cuda()


def check(z, k, score, renormalize, bias=None, scale=1.0):
    ids, w = ep.route_topk(z, k, score=score, renormalize=renormalize, bias=bias, scale=scale)
    want_ids, want_w = R.route(z, k, score, renormalize, bias, scale)
    assert torch.equal(ids.cpu(), want_ids)
    assert ((w.cpu().double() - want_w).abs() <= WEIGHT_TOL * want_w.abs() + 1e-37).all()
    return ids, w


@pytest.mark.parametrize("score,renormalize", FORMS)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (7, 33, 8), (3, 60, 16), (4, 64, 8), (9, 257, 8),
                                   (6, 1024, 16), (2, 16, 16)])
@pytest.mark.parametrize("dtype", (BF16, F32))
def test_choices_and_weights(T, E, k, dtype, score, renormalize):
    z = logits_of(T, E, dtype, T * 1000 + E)
    check(z, k, score, renormalize)
    bias = torch.linspace(-1, 1, E).cuda()
    check(z, k, score, renormalize, bias=bias, scale=2.5)


def test_ties_go_to_the_lowest_expert():
    z = torch.zeros(3, 96, device="cuda")
    z[1, ::2] = -0.0            # equal to 0
    z[2, 40:] = 1.0
    ids, w = check(z, 8, "softmax", True)
    assert ids.tolist() == [list(range(8)), list(range(8)), list(range(40, 48))]


@pytest.mark.parametrize("score,renormalize", FORMS)
def test_masks(score, renormalize):
    z = logits_of(8, 40, F32, 3)
    z[0] = -INF                                  # nothing left
    z[1] = NAN
    z[2, 3:] = -INF                              # fewer than top_k left
    z[3, ::2] = NAN
    z[4, 7] = INF
    z[5] = torch.finfo(F32).min                  # the lowest finite value is a value
    z[6, :] = -300.0                             # scores that underflow
    z[7, 11] = 500.0
    ids, w = check(z, 6, score, renormalize)
    assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[2, 3:] == -1).all()
    bias = torch.zeros(40, device="cuda")
    bias[:36] = -INF                             # a mask through the bias
    bias[38] = NAN
    ids, _ = check(z, 6, score, renormalize, bias=bias)
    assert set(ids[7].tolist()) == {36, 37, 39, -1}


def test_leading_dimensions_and_no_tokens():
    z = logits_of(12, 16, F32, 4)
    ids, w = ep.route_topk(z.view(3, 4, 16), 2)
    flat = ep.route_topk(z, 2)
    assert torch.equal(ids.view(12, 2), flat[0]) and torch.equal(w.view(12, 2), flat[1])
    ids, w = ep.route_topk(z[:0], 2)
    assert ids.shape == w.shape == (0, 2)
    assert ep.route_topk_backward(w, z[:0], ids).shape == (0, 16)


@pytest.mark.parametrize("score,renormalize", FORMS)
@pytest.mark.parametrize("T,E,k", [(5, 8, 2), (7, 33, 8), (4, 64, 8), (9, 257, 8), (3, 1024, 16), (2, 1, 1)])
@pytest.mark.parametrize("dtype", (BF16, F32))
def test_gradient(T, E, k, dtype, score, renormalize):
    z = logits_of(T, E, dtype, T + E)
    ids, _ = ep.route_topk(z, k, score=score, renormalize=renormalize)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    got = ep.route_topk_backward(dw, z, ids, score=score, renormalize=renormalize, scale=1.5)
    z64 = z.double().requires_grad_()
    w = R.route_weights(z64, ids, score, renormalize, 1.5)
    want, = torch.autograd.grad(w, z64, dw.double())
    z64 = z64.detach()
    # dq - sum(q dq) cancels: rounding is relative to the terms, each at most 1.5 max |dw| q
    size = 1.5 * dw.abs().amax(1, keepdim=True).double() * (torch.softmax(z64, 1) if score == "softmax" and not renormalize
                                                           else torch.ones_like(z64))
    bound = (2.0 ** -8 if dtype == BF16 else 0) * want.abs() + 2.0 ** -17 * size + 1e-37
    assert ((got.double() - want).abs() <= bound).all()
    # and against differences of the 64-bit weights
    d = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).cuda().double()
    h = 1e-6
    slope = ((R.route_weights(z64 + h * d, ids, score, renormalize, 1.5)
              - R.route_weights(z64 - h * d, ids, score, renormalize, 1.5)) * dw.double()).sum() / (2 * h)
    assert abs(float((got.double() * d).sum() - slope)) <= float((bound * d.abs()).sum()) + 1e-6


def test_gradient_ignores_what_was_not_chosen():
    z = logits_of(4, 40, F32, 9)
    z[0] = -INF
    z[1, 3:] = -INF
    z[2, 5] = NAN
    ids, _ = ep.route_topk(z, 6)
    dw = torch.ones(4, 6, device="cuda")
    dw[0] = NAN                                  # the weights of ids -1 have no gradient
    for score, renormalize in FORMS:
        got = ep.route_topk_backward(dw, z, ids, score=score, renormalize=renormalize)
        assert (got[0] == 0).all() and (got[1, 3:] == 0).all() and torch.isfinite(got).all()
    bad = ids.clone()
    bad[3, 0], bad[3, 1] = 40, 1 << 30           # out of range: no part, nothing out of bounds
    assert torch.isfinite(ep.route_topk_backward(dw, z, bad)[3]).all()


def test_feeds_dispatch():
    """Masked rows come out as rows dispatch drops."""
    z = logits_of(2 * 8, 8, F32, 10).view(2, 8, 8)
    z[1, 5:] = -INF
    ids, w = ep.route_topk(z, 2)
    ctx = ep.EpContext(ep.EpConfig(2, 8, 2, 8, 64), torch.device("cuda", 0))
    a1 = torch.randn(2, 8, 64, device="cuda").to(BF16)
    d = ctx.dispatch(a1, ids, w)
    assert int(d.expert_num_tokens.sum()) == 2 * (16 - 3)
    y = ctx.combine(d.b_a1)
    ctx.check()
    assert (y[1, 5:] == 0).all()
    assert ((y[0].double() - a1[0].double()).abs() <= 2.0 ** -7 * a1[0].double().abs()).all()


def test_refusals():
    z = torch.zeros(4, 16, device="cuda")
    for kw in (dict(top_k=0), dict(top_k=17), dict(top_k=2, score="tanh"), dict(top_k=2, bias=torch.zeros(15, device="cuda"))):
        with pytest.raises(ValueError):
            ep.route_topk(z, **kw)
    with pytest.raises(ValueError):
        ep.route_topk(z.half(), 2)
    with pytest.raises(ValueError):
        ep.route_topk(z.t(), 2)
    with pytest.raises(ValueError):
        ep.route_topk(torch.zeros(4, 1025, device="cuda"), 2)
    with pytest.raises(ValueError):
        ep.route_topk_backward(torch.zeros(4, 2, device="cuda"), z, torch.zeros(4, 3, dtype=torch.int32, device="cuda"))
    assert math.isfinite(float(ep.route_topk(z, 2)[1].sum()))
