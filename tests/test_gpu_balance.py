"""The balance loss, the counts and the logits' gradient against the 64-bit definition.

Error bounds. An exponential is off by at most (2 + 1.5 |z - m|) 2^-23 of itself (|z - m| up to
about 20 here: 2^-18), a sum of up to 1024 of them by a tree, a division and the sums over
tokens add less: 2^-17 of a probability in all. The logsumexp is off by 2^-17 + 2^-23 |m|."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _balance64 as B

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
TOL = 2.0 ** -17
SIZES = [(1, 1, 1, 1), (1, 5, 8, 2), (3, 7, 33, 8), (2, 64, 64, 8), (5, 50, 256, 8), (2, 9, 257, 8), (1, 3, 1024, 16),
         (3, 40, 512, 16), (2, 33, 120, 4), (4, 700, 60, 16)]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def inputs(S, T, E, K, dtype, seed, ragged):
    g = torch.Generator().manual_seed(seed)
    z = (2 * torch.randn(S, T, E, generator=g)).to(dtype)
    ids = z.float().topk(K, dim=-1).indices.to(I32)
    lengths = None
    if ragged:
        lengths = torch.randint(0, T + 1, (S,), generator=g).to(I32)
        lengths[0] = T + 3        # more than there are: all
        if S > 2:
            lengths[1], lengths[2] = 0, -1
    return z, ids, lengths


def bounds(z, ids, score, per_sequence, lengths, d):
    """(losses, their bounds, counts, gradient, its bound) for the losses' gradient d."""
    zr = z.double().requires_grad_()
    balance, zloss, counts = B.losses(zr, ids, score, per_sequence, lengths)
    grad, = torch.autograd.grad(d[0] * balance + d[1] * zloss, zr)
    S, T, E = z.shape
    pools = B.pools_of(z, per_sequence, lengths)
    n_all, some = sum(len(r) for r in pools), max(1, sum(1 for r in pools if len(r)))
    p, lse = B.scores(z.double(), score)
    soft, _ = B.scores(z.double(), "softmax")
    p, soft, lse = p.reshape(-1, E), soft.reshape(-1, E), lse.reshape(-1, 1)
    bound = torch.zeros(S * T, E, dtype=B.D)
    for i, rows in enumerate(pools):
        if len(rows):
            g = abs(d[0]) * E * counts[i].double() / (ids.shape[-1] * len(rows) ** 2 * some)
            bound[rows] = p[rows] * (g + (p[rows] * g).sum(1, keepdim=True)) \
                + soft[rows] * (abs(d[1]) * 2 / n_all * (lse[rows].abs() + 1))
    used = lse[torch.cat(pools)] if n_all else lse[:0]
    losses = torch.stack((balance.detach(), zloss.detach()))
    off = torch.stack((balance.detach() * TOL, ((used.square() + 1).mean() if n_all else losses[1] * 0) * TOL))
    return losses, off + 1e-30, counts, grad, 4 * TOL * bound.view(S, T, E) + 1e-30


def check(z, ids, lengths, score, per_sequence, d=(0.7, 0.3), where=lambda t: t.cuda()):
    zc, idc, lc = where(z), where(ids), None if lengths is None else lengths.cuda()
    kw = dict(score=score, per_sequence=per_sequence, num_tokens=lc)
    losses, counts = ep.balance_loss(zc, idc, **kw)
    dl = torch.tensor(d, device="cuda")
    grad = ep.balance_loss_backward(dl, zc, counts, ids.shape[-1], **kw)
    want, off, want_counts, want_grad, gbound = bounds(z, ids, score, per_sequence, lengths, dl.cpu().double().tolist())
    assert torch.equal(counts.cpu().long().view(want_counts.shape), want_counts)
    assert ((losses.cpu().double() - want).abs() <= off).all()
    if z.dtype is BF16:
        gbound = gbound + want_grad.abs() * 2.0 ** -8
    assert ((grad.cpu().double() - want_grad).abs() <= gbound).all()
    return zc, idc, losses, counts, grad, kw, dl


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("per_sequence", (False, True))
@pytest.mark.parametrize("ragged", (False, True))
@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("size", SIZES)
def test_losses_counts_and_gradient(size, dtype, ragged, per_sequence, score):
    S, T, E, K = size
    z, ids, lengths = inputs(S, T, E, K, dtype, S * 100 + E, ragged)
    check(z, ids, lengths, score, per_sequence)


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_masks(score):
    z, ids, _ = inputs(2, 9, 40, 6, F32, 5, False)
    z[0, 0] = -float("inf")                 # nothing left
    z[0, 1] = float("nan")
    z[0, 2, 3:] = -float("inf")
    z[0, 3, ::2] = float("nan")
    z[0, 4] = -300.0                        # sigmoids that underflow
    z[0, 5] = -300.0
    z[0, 5, 7] = -290.0
    z[0, 6, 11] = 60.0
    ids[0, 0], ids[0, 1], ids[0, 2, 3:] = -1, -1, -1
    ids[1, 0, 0], ids[1, 0, 1] = 40, 1 << 30     # out of range: not counted
    ids[1, 1] = 7                                # an expert chosen more than once counts each time
    check(z, ids, None, score, False)
    check(z, ids, torch.tensor([9, 2], dtype=I32), score, True)


def test_an_infinite_logit_counts_as_the_largest_finite():
    z = torch.zeros(1, 2, 16, device="cuda")
    z[0, 0, 3] = float("inf")
    ids = torch.tensor([[[3], [5]]], dtype=I32, device="cuda")
    losses, counts = ep.balance_loss(z, ids)
    # p of the first token is 1 at expert 3, of the second 1/16 everywhere
    assert abs(float(losses[0]) - 16 / 2 * (1.0625 + 0.0625) / 2) < 1e-5 and counts[3] == 1 and counts[5] == 1
    d = ep.balance_loss_backward(torch.tensor([1.0, 0.0], device="cuda"), z, counts, 1)
    assert torch.isfinite(d).all() and (d[0, 0] == 0).all()


@pytest.mark.parametrize("dtype", (BF16, F32))
def test_added_to_another_gradient(dtype):
    z, ids, lengths = inputs(3, 50, 64, 8, dtype, 9, True)
    zc, idc, losses, counts, grad, kw, dl = check(z, ids, lengths, "softmax", False)
    before = torch.randn(z.shape, device="cuda").to(dtype)
    out = before.clone()
    got = ep.balance_loss_backward(dl, zc, counts, 8, out=out, accumulate=True, **kw)
    assert got is out
    used = torch.zeros(3, 50, dtype=torch.bool)
    for s, n in enumerate(lengths.tolist()):
        used[s, :max(0, min(n, 50))] = True
    used = used.cuda()
    assert torch.equal(out[~used], before[~used])       # rows that hold no token stay
    assert (grad[~used] == 0).all()
    exact = before.double() + bounds(z, ids, "softmax", False, lengths, dl.cpu().double().tolist())[3].cuda()
    # the sum's rounding, and the gradient's own error
    off = exact.abs() * (2.0 ** -8 if dtype is BF16 else 2.0 ** -23) + 2.0 ** -15 * (exact - before.double()).abs().max()
    assert ((out.double() - exact).abs() <= off)[used].all()


def test_odd_addresses_and_leading_dimensions():
    z, ids, lengths = inputs(4, 21, 64, 8, F32, 11, True)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.reshape(-1).cuda()
        return flat[1:].view(t.shape)

    check(z, ids, lengths, "sigmoid", True, where=shifted)
    a, c = ep.balance_loss(z.view(2, 2, 21, 64).cuda(), ids.view(2, 2, 21, 8).cuda(), per_sequence=True,
                           num_tokens=lengths.view(2, 2).cuda())
    b, d = ep.balance_loss(z.cuda(), ids.cuda(), per_sequence=True, num_tokens=lengths.cuda())
    assert c.shape == (2, 2, 64) and torch.equal(c.view(4, 64), d) and torch.equal(a, b)
    a, c = ep.balance_loss(z[0].cuda(), ids[0].cuda())
    assert c.shape == (64,)
    check(z[:1], ids[:1], None, "softmax", False)


def test_no_tokens():
    z, ids = torch.empty(3, 0, 8, device="cuda"), torch.empty(3, 0, 2, dtype=I32, device="cuda")
    losses, counts = ep.balance_loss(z, ids, per_sequence=True)
    assert losses.tolist() == [0, 0] and counts.tolist() == [[0] * 8] * 3
    assert ep.balance_loss_backward(losses, z, counts, 2, per_sequence=True).shape == z.shape
    z, ids, _ = inputs(2, 6, 8, 2, F32, 1, False)
    none = torch.zeros(2, dtype=I32)
    *_, losses, counts, grad, _, _ = check(z, ids, none, "softmax", False)
    assert losses.tolist() == [0, 0] and (grad == 0).all() and (counts == 0).all()


def test_long_batches_and_many_sequences():
    z, ids, lengths = inputs(1, 20000, 64, 4, BF16, 2, False)
    check(z, ids, lengths, "softmax", False)
    z, ids, lengths = inputs(900, 3, 16, 2, F32, 2, True)
    check(z, ids, lengths, "sigmoid", True)
    check(z, ids, lengths, "softmax", False)


def test_same_bits_each_time_on_any_stream_and_in_a_graph():
    z, ids, lengths = inputs(6, 300, 256, 8, F32, 4, True)
    zc, idc, losses, counts, grad, kw, dl = check(z, ids, lengths, "sigmoid", True)

    def both(stream=None):
        a, c = ep.balance_loss(zc, idc, stream=stream, **kw)
        return a, c, ep.balance_loss_backward(dl, zc, c, 8, stream=stream, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(got, (losses, counts, grad)):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    other = inputs(6, 300, 256, 8, F32, 5, True)
    zc.copy_(other[0])
    idc.copy_(other[1])
    for _ in range(2):
        graph.replay()
    want = both()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_what_requires_a_gradient_is_refused():
    z, ids, _ = inputs(1, 4, 8, 2, F32, 1, False)
    zc, idc = z.cuda().requires_grad_(), ids.cuda()
    with pytest.raises(ValueError, match="gradient"):
        ep.balance_loss(zc, idc)
    with torch.no_grad():
        losses, counts = ep.balance_loss(zc, idc)
    d = ep.balance_loss_backward(losses, zc, counts, 2)     # the logits of a gradient call may
    assert d.shape == z.shape
    with pytest.raises(ValueError, match="gradient"):
        ep.balance_loss_backward(losses.clone().requires_grad_(), zc, counts, 2)


def test_bad_tensors_are_refused():
    z, ids, _ = inputs(2, 4, 8, 2, F32, 1, False)
    z, ids = z.cuda(), ids.cuda()
    losses, counts = ep.balance_loss(z, ids)
    for call in (lambda: ep.balance_loss(z, ids.long()), lambda: ep.balance_loss(z, ids[:1]),
                 lambda: ep.balance_loss(z.transpose(0, 1), ids),
                 lambda: ep.balance_loss(z, ids, num_tokens=torch.zeros(3, dtype=I32, device="cuda")),
                 lambda: ep.balance_loss(z, ids, num_tokens=torch.zeros(2, dtype=I32)),
                 lambda: ep.balance_loss_backward(losses, z, counts, 2, per_sequence=True),
                 lambda: ep.balance_loss_backward(losses, z, counts.long(), 2),
                 lambda: ep.balance_loss_backward(losses[:1], z, counts, 2),
                 lambda: ep.balance_loss_backward(losses, z, counts, 9),
                 lambda: ep.balance_loss_backward(losses, z, counts, 2, accumulate=True),
                 lambda: ep.balance_loss_backward(losses, z, counts, 2, out=z.to(BF16))):
        with pytest.raises(ValueError):
            call()
