"""The balance loss of many short sequences: right, and in time that grows with their number, not its square."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests.test_gpu_balance import BF16, F32, I32, built, check, inputs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("size", [(1217, 2, 24, 3), (2500, 1, 60, 4), (2433, 9, 8, 1), (1300, 3, 257, 8), (1400, 2, 128, 4), (1250, 2, 256, 8),
                                  (1250, 2, 512, 8), (1300, 2, 1024, 16), (1219, 1, 1001, 16)])
@pytest.mark.parametrize("ragged", (False, True))
@pytest.mark.parametrize("per_sequence", (False, True))
@pytest.mark.parametrize("dtype", (F32, BF16))
def test_more_sequences_than_work_at_a_time(dtype, per_sequence, ragged, size, score):
    z, ids, lengths = inputs(*size, dtype, 3, ragged)
    zc, _, _, counts, grad, kw, dl = check(z, ids, lengths, score, per_sequence)
    # added to what is there: the gradient and one more rounding, rows without a token left alone
    out = torch.ones_like(zc)
    ep.balance_loss_backward(dl, zc, counts, size[3], out=out, accumulate=True, **kw)
    used = torch.ones(size[:2], dtype=torch.bool, device="cuda") if lengths is None else \
        torch.arange(size[1], device="cuda") < lengths.cuda()[:, None]
    assert (out[~used] == 1).all()
    want = 1 + grad[used].double()
    # (in bf16 the gradient compared with is rounded too)
    off = want.abs() * (2.0 ** -8 if dtype is BF16 else 2.0 ** -24) + (grad[used].double().abs() * 2.0 ** -8 if dtype is BF16 else 0)
    assert ((out[used].double() - want).abs() <= off).all()


@pytest.mark.parametrize("lengths", (False, True))
def test_more_tokens_than_work_at_a_time(lengths):
    """Chunks of 4096 tokens, the most there are, and more of them than a gradient with lengths has CTAs."""
    T, E = 4096 * 1216 + 4097, 8
    z = torch.randn(1, T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF16)
    ids = torch.zeros(1, T, 1, dtype=I32, device="cuda")
    kw = dict(num_tokens=torch.tensor([T], dtype=I32, device="cuda")) if lengths else {}
    _, counts = ep.balance_loss(z, ids, **kw)
    d = torch.tensor([0.0, float(T)], device="cuda")
    grad = ep.balance_loss_backward(d, z, counts, 1, **kw)
    for at in (0, T // 2, 4096 * 1216 - 2048, 4096 * 1216 + 2048, T - 2048):
        own = z[0, at:at + 2048].double()
        want = 2 * torch.logsumexp(own, -1, keepdim=True) * torch.softmax(own, -1)
        assert ((grad[0, at:at + 2048].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -15) + 2.0 ** -17).all()


def test_the_same_sequence_gives_the_same_bits_wherever_it_lies():
    """A gradient by a CTA that takes several sequences is the one that it has alone."""
    S, T, E = 5000, 3, 64
    z = torch.randn(S, T, E, device="cuda")
    z[-1] = z[0]
    ids = z.topk(4, dim=-1).indices.to(I32)
    lengths = torch.randint(0, T + 1, (S,), device="cuda").to(I32)
    lengths[0] = lengths[-1] = 2
    kw = dict(per_sequence=True, num_tokens=lengths)
    losses, counts = ep.balance_loss(z, ids, **kw)
    grad = ep.balance_loss_backward(torch.ones(2, device="cuda"), z, counts, 4, **kw)
    assert torch.equal(counts[0], counts[-1]) and torch.equal(grad[0], grad[-1]) and (grad[-1, 2:] == 0).all()


@pytest.mark.parametrize("ragged", (False, True))
def test_time_grows_with_the_number_of_sequences(ragged):
    """Four times the sequences: four times the work, and sixteen before the lengths were added up once a CTA.
    (8192 sequences take hundreds of microseconds, so that neither the launch nor the clock decides.)"""
    def least(S):
        z = torch.randn(S, 1, 256, device="cuda")
        ids = z.topk(2, dim=-1).indices.to(I32)
        kw = dict(per_sequence=True, num_tokens=torch.ones(S, dtype=I32, device="cuda") if ragged else None)
        took = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            ep.balance_loss(z, ids, **kw)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        return min(took)

    assert least(32768) < 8 * least(8192)


def test_as_many_sequences_as_there_may_be():
    """2^31 - 1 of one token: the CTAs' numbers and the last one's walk over them stay in range (as a signed number
    that walk passed 2^31). Half a minute: every pool has a CTA of its own. Sums of ones with what rounding takes
    from them, one division: 2^-22."""
    if torch.cuda.get_device_properties(0).total_memory < 100e9:
        pytest.skip("needs the memory")
    S = (1 << 31) - 1
    z = torch.ones(S, 1, 1, dtype=BF16, device="cuda")
    ids = torch.zeros(S, 1, 1, dtype=I32, device="cuda")
    losses, counts = ep.balance_loss(z, ids, per_sequence=True)
    assert ((losses - 1).abs() <= 2.0 ** -22).all()     # one expert, chosen by all; its logit's square is 1
    assert bool((counts[::1 << 20] == 1).all()) and bool((counts[-4096:] == 1).all())
    del losses, counts, z, ids
    torch.cuda.empty_cache()
