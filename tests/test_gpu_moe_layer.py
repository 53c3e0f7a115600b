"""The example layer: router, dispatch, experts, combine and shared expert together,
forward and backward, against 64-bit autograd with the same choice of experts."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def reference(layer, x, ids, dout):
    c = layer.cfg
    p = {k: getattr(layer, k).double().requires_grad_() for k in ("router", "w13", "w2", "s1", "b1", "s2")}
    x = x.double().requires_grad_()
    flat = x.reshape(-1, c.hidden)
    w = R.route_weights(flat @ p["router"].T, ids.reshape(-1, c.top_k), "softmax", True, 1.0)
    w13, w2 = p["w13"].reshape(c.E, -1, c.hidden), p["w2"].reshape(c.E, c.hidden, -1)
    inner = w2.shape[-1]
    routed = 0
    for k in range(c.top_k):
        e = ids.reshape(-1, c.top_k)[:, k].long()
        z = torch.einsum("th,tih->ti", flat, w13[e])
        hid = torch.nn.functional.silu(z[:, :inner]) * z[:, inner:]
        routed = routed + w[:, k:k + 1] * torch.einsum("ti,thi->th", hid, w2[e])
    sh = torch.nn.functional.gelu(flat @ p["s1"].T + p["b1"]) @ p["s2"].T
    out = (routed + sh).reshape(x.shape)
    grads = torch.autograd.grad(out, [x, *p.values()], dout.double())
    return out.detach(), dict(zip(["x", *p], grads))


@pytest.mark.parametrize("W,E,K,T,h", [(2, 8, 2, 16, 128), (4, 16, 4, 24, 256)])
def test_layer_forward_and_backward(W, E, K, T, h):
    from examples.moe_layer import MoeLayer
    layer = MoeLayer(ep.EpConfig(W, E, K, T, h), inner=72, shared=136, seed=W)
    g = torch.Generator(device="cuda").manual_seed(7)
    x, dout = (torch.randn(W, T, h, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out = layer.forward(x)
    grads = layer.backward(dout)
    layer.check()
    want, want_grads = reference(layer, x, layer.ids, dout)

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    # at most six bf16 roundings (2^-9 each) on the way to any of these
    assert off(out, want) <= 6 * 2.0 ** -9
    for name, g64 in want_grads.items():
        assert off(grads[name].reshape(g64.shape), g64) <= 6 * 2.0 ** -9, name
