"""The router's choice by score + bias (a correction bias trained on the scores): against the
64-bit scores, where it differs from the choice by logit + bias, ties and masks."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R
from tests.test_gpu_router import FORMS, INF, NAN, WEIGHT_TOL, built, logits_of  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def scores64(z, score):
    return torch.softmax(z.double(), -1) if score == "softmax" else torch.sigmoid(z.double())


@pytest.mark.parametrize("score,renormalize", FORMS)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (7, 33, 8), (4, 64, 8), (300, 256, 8), (6, 1024, 16)])
@pytest.mark.parametrize("dtype", (BF16, F32))
def test_choices_by_score_plus_bias(T, E, k, dtype, score, renormalize):
    z = logits_of(T, E, dtype, T * 1000 + E)
    bias = (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E))).cuda()
    ids, w = ep.route_topk(z, k, score=score, renormalize=renormalize, bias=bias, bias_on="scores", scale=2.5)
    s = scores64(z, score)
    key = s + bias.double()
    got, best = key.gather(1, ids.long()), key.sort(1, descending=True).values[:, :k]
    # a score's error as the weights', and the rounding of the sum
    tol = 2 * (WEIGHT_TOL * s.amax(1, keepdim=True) + 2.0 ** -23 * key.abs().amax(1, keepdim=True))
    assert ((got - best).abs() <= tol).all()
    assert all(len(set(row)) == k for row in ids.tolist())
    want = R.route_weights(z.double(), ids, score, renormalize, 2.5)
    assert ((w.double() - want).abs() <= WEIGHT_TOL * want + 1e-37).all()


def test_differs_from_the_choice_by_logits():
    z = torch.tensor([[0.0, 4.0, 5.0, -1.0]], device="cuda")
    bias = torch.tensor([0.9, 0.0, 0.0, 0.0], device="cuda")
    assert ep.route_topk(z, 2, score="sigmoid", bias=bias)[0].tolist() == [[2, 1]]
    assert ep.route_topk(z, 2, score="sigmoid", bias=bias, bias_on="scores")[0].tolist() == [[0, 2]]
    many = logits_of(64, 256, F32, 1)
    bias = (0.2 * torch.randn(256, generator=torch.Generator().manual_seed(2))).cuda()
    a, b = (ep.route_topk(many, 8, score="sigmoid", bias=bias, bias_on=on)[0].sort(1).values for on in ("logits", "scores"))
    assert (a != b).any(1).float().mean() > 0.9
    # without a bias the two are one choice
    assert torch.equal(ep.route_topk(many, 8, score="sigmoid", bias_on="scores")[0], ep.route_topk(many, 8, score="sigmoid")[0])


@pytest.mark.parametrize("score,renormalize", FORMS)
@pytest.mark.parametrize("E", (40, 96, 256))
def test_ties_and_masks(E, score, renormalize):
    z = torch.zeros(6, E, device="cuda")
    z[1] = -INF                                   # nothing left
    z[2, ::2] = NAN
    z[3, 7] = INF
    z[4, 3:] = -INF                               # fewer than top_k left
    bias = torch.full((E,), 0.5, device="cuda")
    kw = dict(score=score, renormalize=renormalize, bias_on="scores")
    ids, w = ep.route_topk(z, 6, bias=bias, **kw)
    assert ids[0].tolist() == list(range(6)) and ids[1].tolist() == [-1] * 6
    assert ids[2].tolist() == [1, 3, 5, 7, 9, 11] and int(ids[3, 0]) == 7
    assert ids[4].tolist() == [0, 1, 2, -1, -1, -1]
    assert torch.isfinite(w).all() and (w[ids < 0] == 0).all()
    bias[:36] = -INF                              # a mask through the bias
    bias[38] = NAN
    assert ep.route_topk(z, 6, bias=bias, **kw)[0][0, :3].tolist() == [36, 37, 39]


def test_a_name_that_is_not_known_is_refused():
    with pytest.raises(ValueError):
        ep.route_topk(torch.zeros(4, 16, device="cuda"), 2, bias=torch.zeros(16, device="cuda"), bias_on="score")
