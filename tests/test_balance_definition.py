"""The balance loss on the host: its 64-bit definition against differences and by hand, and the
refusals of the entry points, which come before any GPU work."""
import ctypes as C

import pytest
import torch

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L
from tests import _balance64 as B

P = 0x7F0000000000      # an aligned address; never dereferenced by these tests


@pytest.fixture(scope="module")
def lib():
    from combine_ep_route_gb300 import build
    build.build()
    return L.lib()


def args(seqs=2, tokens=8, E=16, top_k=4, score=0, per_sequence=0, dtype=L.EP_F32, num_tokens=None):
    return C.byref(L.EpBalanceC(seqs, tokens, E, top_k, score, per_sequence, dtype, num_tokens))


def test_even_use_costs_one():
    z = torch.zeros(1, 8, 4, dtype=B.D)
    ids = torch.arange(8)[:, None].remainder(4)[None]
    balance, zloss, counts = B.losses(z, ids, "softmax", False, None)
    assert abs(float(balance) - 1) < 1e-12 and counts.tolist() == [[2, 2, 2, 2]]
    assert abs(float(zloss) - float(torch.log(torch.tensor(4., dtype=B.D))) ** 2) < 1e-12
    ids = torch.zeros_like(ids)          # one expert does everything, and is sure to be chosen
    z[..., 0] = 50.0
    assert abs(float(B.losses(z, ids, "softmax", False, None)[0]) - 4) < 1e-9


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("per_sequence", (False, True))
def test_gradient_matches_differences(score, per_sequence):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(3, 5, 7, generator=g, dtype=B.D)
    z[0, 1, 2] = -float("inf")
    ids = z.topk(2, dim=-1).indices
    lengths = [5, 0, 3]

    def total(z):
        balance, zloss, _ = B.losses(z, ids, score, per_sequence, lengths)
        return 0.7 * balance + 0.3 * zloss

    zr = z.clone().requires_grad_()
    d, = torch.autograd.grad(total(zr), zr)
    v = torch.randn(z.shape, generator=g, dtype=B.D)
    h = 1e-6
    diff = (total(z + h * v) - total(z - h * v)) / (2 * h)
    assert abs(float(diff) - float((d * torch.where(torch.isfinite(z), v, torch.zeros_like(v))).sum())) < 1e-8
    assert (d[1] == 0).all() and (d[2, 3:] == 0).all()


@pytest.mark.parametrize("bad", [dict(seqs=-1), dict(tokens=-1), dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=17),
                                 dict(E=8, top_k=9), dict(score=2), dict(score=16), dict(per_sequence=2), dict(dtype=3),
                                 dict(seqs=1 << 16, tokens=1 << 15), dict(num_tokens=P + 2)])
def test_bad_arguments_are_refused(lib, bad):
    a, size, inv = args(**bad), C.c_size_t(), L.EP_ERR_INVALID_ARG
    assert lib.ep_balance_workspace_bytes(a, C.byref(size)) == inv
    assert lib.ep_balance_loss(a, P, P, P, P, P, 1 << 30, None) == inv
    assert lib.ep_balance_loss_backward(a, P, P, P, 0, P, None) == inv


def test_bad_buffers_are_refused(lib):
    a, size, inv = args(), C.c_size_t(), L.EP_ERR_INVALID_ARG
    assert lib.ep_balance_workspace_bytes(a, None) == inv
    assert lib.ep_balance_workspace_bytes(a, C.byref(size)) == L.EP_OK and size.value > 0
    for at in range(4):
        for v in (None, P + 2):
            given = [P] * 4
            given[at] = v
            assert lib.ep_balance_loss(a, *given, P, size.value, None) == inv
            given = [P] * 4
            given[at] = v
            assert lib.ep_balance_loss_backward(a, *given[:3], 0, given[3], None) == inv
    assert lib.ep_balance_loss_backward(a, P, P, P, 2, P, None) == inv
    for work, bytes_ in ((P, size.value - 1), (P + 8, size.value), (None, size.value)):
        assert lib.ep_balance_loss(a, P, P, P, P, work, bytes_, None) == L.EP_ERR_WORKSPACE
    for few in (args(tokens=0), args(seqs=0)):
        assert lib.ep_balance_workspace_bytes(few, C.byref(size)) == L.EP_OK and size.value == 0
        assert lib.ep_balance_loss_backward(few, None, None, None, 0, None, None) == L.EP_OK


def test_host_tensors_and_bad_calls_are_refused():
    z, ids = torch.zeros(2, 4, 8), torch.zeros(2, 4, 2, dtype=torch.int32)
    for call in (lambda: ep.balance_loss(z, ids), lambda: ep.balance_loss(z, ids, score="tanh"),
                 lambda: ep.balance_loss(z[0, 0], ids), lambda: ep.balance_loss(z.double(), ids),
                 lambda: ep.balance_loss_backward(torch.zeros(2), z, torch.zeros(8, dtype=torch.int32), 2)):
        with pytest.raises(ValueError):
            call()
