"""The example layer's training step with the router's losses and clipping, and its served form with
4-bit weights, as they are used together: against 64-bit autograd with the same choice of experts."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _balance64 as B
from tests.test_gpu_moe_layer import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def make(W, E, K, T, h, seed):
    from examples.moe_layer import MoeLayer
    layer = MoeLayer(ep.EpConfig(W, E, K, T, h), inner=96, shared=160, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x, dout = (torch.randn(W, T, h, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    return layer, x, dout


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("size", [(2, 8, 2, 16, 128), (4, 16, 4, 24, 256)])
def test_a_training_step(size):
    layer, x, dout = make(*size, seed=3)
    layer.forward(x)
    d = [3.0, 0.5]          # large, so that the losses' part of the router's gradient counts
    grads = layer.backward(dout, torch.tensor(d, device="cuda"))
    _, want = reference(layer, x, layer.ids, dout)
    # the losses' own part, from the bf16 weight and input
    c = layer.cfg
    router, xd = layer.router.double().requires_grad_(), x.double().requires_grad_()
    logits = (xd.reshape(-1, c.hidden) @ router.T).reshape(c.W, c.max_tokens, c.E)
    balance, zloss, counts = B.losses(logits.cpu(), layer.ids.cpu(), "softmax", False, None)
    assert torch.equal(layer.load.cpu().long(), counts[0])
    # logits of h products: 2^-20 of them at most; a loss of theirs twice that and its own 2^-17
    assert abs(float(layer.losses[0]) - float(balance.detach())) <= 2.0 ** -16 * float(balance.detach())
    assert abs(float(layer.losses[1]) - float(zloss.detach())) <= 2.0 ** -16 * (float(zloss.detach()) + 1)
    more = torch.autograd.grad(d[0] * balance + d[1] * zloss, (router, xd))
    want["router"] = want["router"] + more[0]
    want["x"] = want["x"] + more[1].reshape(want["x"].shape)
    for name, g64 in want.items():      # at most six bf16 roundings on the way
        assert off(grads[name].reshape(g64.shape), g64) <= 6 * 2.0 ** -9, name
    names = [n for n in grads if n != "x"]
    total = sum(float(grads[n].double().square().sum()) for n in names) ** 0.5
    before = {n: grads[n].clone() for n in names}
    norm = layer.clip(grads, 0.5 * total)
    assert abs(float(norm) - total) <= 2.0 ** -20 * total
    for n in names:
        exact = before[n].double() * 0.5
        assert ((grads[n].double() - exact).abs() <= exact.abs() * (2.0 ** -8 + 2.0 ** -18)).all(), n
    layer.check()


@pytest.mark.parametrize("kind", ("int4", "fp4"))
@pytest.mark.parametrize("size", [(2, 8, 2, 16, 128), (4, 16, 4, 24, 256), (2, 8, 1, 1, 128)])
def test_serving_with_4_bit_weights(size, kind):
    layer, x, dout = make(*size, seed=5)
    layer.quantize(32, kind)
    out = layer.forward_w4(x)
    layer.check()
    # the same layer with the bf16 weights that the codes stand for
    for name, (codes, scales) in layer.q.items():
        w = ep.dequantize_weight4(codes, scales, kind)
        assert off(w, getattr(layer, name).double()) < 0.2      # a weight of its own, not of another layer
        setattr(layer, name, w)
    full = layer.forward(x)
    want, _ = reference(layer, x, layer.ids, dout)
    assert off(out, want) <= 6 * 2.0 ** -9 and off(full, want) <= 6 * 2.0 ** -9


def test_a_captured_step_replays():
    layer, x, _ = make(2, 8, 2, 16, 128, seed=7)
    layer.quantize()
    layer.forward_w4(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward_w4(x)
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, layer.forward_w4(x))
    layer.check()
