"""The layers' calls record nothing for autograd: an operand that requires a gradient is refused
where one would be expected, and taken under no_grad and in gradient calls."""
import pytest
import torch

import combine_ep_route_gb300 as ep

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def make(*shape, dtype=BF16):
    return torch.ones(*shape, dtype=dtype, device="cuda")


def test_what_would_lose_a_gradient_is_refused():
    cnt = torch.tensor([4], dtype=torch.int32, device="cuda")
    kinds = {
        "x": (4, 8), "w": (16, 8), "bias": (16,), "residual": (4, 16),
    }
    for name in kinds:
        kw = {k: make(*s).requires_grad_(k == name) for k, s in kinds.items()}
        with pytest.raises(ValueError, match=name):
            ep.linear(**kw)
        with pytest.raises(ValueError, match=name):
            ep.experts_product(counts=cnt, **{k: v[None] for k, v in kw.items()})
        with torch.no_grad():
            assert (ep.linear(**kw) == 10).all()
        assert (ep.linear(**{k: v.detach() for k, v in kw.items()}) == 10).all()
    z = make(4, 8, dtype=torch.float32).requires_grad_()
    with pytest.raises(ValueError, match="logits"):
        ep.route_topk(z, 2)
    with torch.no_grad():
        ep.route_topk(z, 2)


def test_gradient_calls_refuse_a_recorded_gradient_only():
    x, w = make(4, 8).requires_grad_(), make(16, 8).requires_grad_()
    dy, preact = make(4, 16), make(4, 8).requires_grad_()
    ep.linear_dgrad(dy, w)
    ep.linear_dgrad(dy, w, act="relu", preact=preact)
    ep.linear_wgrad(dy, x)
    ep.act_grad(make(4, 8), preact, "relu")
    tracked = make(4, 16).requires_grad_()
    for call in (lambda: ep.linear_dgrad(tracked, w), lambda: ep.linear_wgrad(tracked, x),
                 lambda: ep.act_grad(tracked, make(4, 16), "silu"),
                 lambda: ep.route_topk_backward(make(4, 2, dtype=torch.float32).requires_grad_(), make(4, 16),
                                                torch.zeros(4, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()


def test_a_function_of_its_own():
    """How a user records them: forward and backward of a torch.autograd.Function."""
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x, w)
            return ep.linear(x, w)

        @staticmethod
        def backward(ctx, dy):
            x, w = ctx.saved_tensors
            return ep.linear_dgrad(dy.contiguous(), w), ep.linear_wgrad(dy.contiguous(), x)

    x, w = make(4, 8).requires_grad_(), make(16, 8).requires_grad_()
    Linear.apply(x, w).sum().backward()
    assert (x.grad == 16).all() and (w.grad == 4).all()
