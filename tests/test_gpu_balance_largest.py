"""The gradient of the z loss for logits next to the largest float: a logsumexp times the loss's unit (twice its
gradient over the tokens) may be past the largest float although no expert's share is, or meets probabilities of
zero. Nothing is NaN then; a share past the largest float is infinite, and every other one right to the bounds of
test_gpu_balance.py (relative to the share, so they hold at any size)."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests.test_gpu_balance import BF16, F32, I32, bounds, built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("E", (16, 100, 256))
@pytest.mark.parametrize("tokens", (1, 3))
@pytest.mark.parametrize("v", (1e38, -1e38, 3.3e38, -3.3e38))
@pytest.mark.parametrize("d1", (0.25, 1.0, 3.0, -2.0))
def test_shares_of_the_z_loss(d1, v, tokens, E, dtype, score):
    z = torch.randn(1, tokens, E, generator=torch.Generator().manual_seed(E))
    z[0, 0] = v                    # even: a share is 1 / E of it
    if tokens > 1:
        z[0, 1, 5] = v             # one that has everything, or nothing
        z[0, 2, ::2] = v
    z = z.to(dtype)
    ids = torch.zeros(1, tokens, 1, dtype=I32)
    _, counts = ep.balance_loss(z.cuda(), ids.cuda(), score=score)
    d = torch.tensor([0.5, d1], device="cuda")
    grad = ep.balance_loss_backward(d, z.cuda(), counts, 1, score=score).cpu().double()
    _, _, _, want, off = bounds(z, ids, score, False, None, d.cpu().double().tolist())
    most = torch.finfo(dtype).max
    if dtype is BF16:
        off = off + want.abs() * 2.0 ** -8
    fits = want.abs() <= most * (1 - 2.0 ** -8)
    assert ((grad - want).abs() <= off)[fits].all()
    past = want.abs() > most * (1 + 2.0 ** -8)
    assert (grad[past] == want[past].sign() * float("inf")).all() and (fits | past).all()


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_an_infinite_logit_of_a_lone_token(score):
    z = torch.zeros(1, 1, 16, device="cuda")
    z[0, 0, 3] = float("inf")       # counts as the largest float
    _, counts = ep.balance_loss(z, torch.zeros(1, 1, 1, dtype=I32, device="cuda"), score=score)
    grad = ep.balance_loss_backward(torch.tensor([0.0, 1.0], device="cuda"), z, counts, 1, score=score)
    assert grad[0, 0, 3] == float("inf") and (grad[0, 0, :3] == 0).all() and (grad[0, 0, 4:] == 0).all()
