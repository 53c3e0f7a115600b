"""The balance and z losses and their gradient for tokens with large logits, on both sides of 2^16, from which
the exponentials are formed another way, up to the largest floats: rows masked by a large number as a whole or
in part, among ordinary ones.

The error bounds are those of test_gpu_balance.py: they are relative to the probabilities and the logsumexp, and
logits beside a large one are either next to it (|z - m| up to 20) or have no probability. Where the exact z loss
is past the largest float, the loss is infinite; no size here has a z loss between that and its tokens' sum."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests.test_gpu_balance import BF16, F32, I32, bounds, built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
FLOAT_MAX = 3.4028234663852886e38
SIZES = (60000.0, 65536.0, 66000.0, 1e6, 3e9, 1e10, 1e18, 1e20, 1e30, 9e37, 1.1e38, 3e38)


def inputs(v, E, K, dtype):
    g = torch.Generator().manual_seed(E)
    z = 2 * torch.randn(2, 11, E, generator=g)
    z[0, 0] = v                                       # wholly
    z[0, 1] = v + 1e-6 * v * torch.rand(E, generator=g)   # nearly the same
    z[0, 2, 1:] = v                                   # all but one
    z[0, 3, ::2] = v                                  # half of it
    z[0, 4, E // 2] = v                               # one
    z[1, 5] = -v
    z[1, 5, 3] = v
    z = z.to(dtype)
    ids = torch.rand(2, 11, E, generator=g).topk(K, dim=-1).indices.to(I32)
    return z, ids


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("E,K", [(16, 2), (100, 4), (256, 8), (1000, 16)])
@pytest.mark.parametrize("v", SIZES + tuple(-v for v in SIZES))
def test_large_logits(v, E, K, dtype, score):
    z, ids = inputs(v, E, K, dtype)
    for lengths in (None, torch.tensor([11, 3], dtype=I32)):
        per_sequence = lengths is not None
        kw = dict(score=score, per_sequence=per_sequence, num_tokens=None if lengths is None else lengths.cuda())
        losses, counts = ep.balance_loss(z.cuda(), ids.cuda(), **kw)
        d = torch.tensor([0.7, 0.3], device="cuda")
        grad = ep.balance_loss_backward(d, z.cuda(), counts, K, **kw)
        want, off, want_counts, want_grad, gbound = bounds(z, ids, score, per_sequence, lengths, d.cpu().double().tolist())
        assert torch.equal(counts.cpu().long().view(want_counts.shape), want_counts)
        got = losses.cpu().double()
        assert (got[0] - want[0]).abs() <= off[0]
        if want[1] > FLOAT_MAX:
            assert got[1] == float("inf")
        else:
            assert (got[1] - want[1]).abs() <= off[1]
        if dtype is BF16:
            gbound = gbound + want_grad.abs() * 2.0 ** -8
        assert ((grad.cpu().double() - want_grad).abs() <= gbound).all()
