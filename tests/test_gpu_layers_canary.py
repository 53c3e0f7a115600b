"""Writes outside the buffers of the products and the router: every output sits between
guard regions that must stay untouched, at shapes whose last tiles overhang every edge."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests.test_gpu_canary import Guarded, dev  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rand(dev, *shape):  # noqa: F811
    return torch.randn(*shape, device=dev).to(BF16)


@pytest.mark.parametrize("E,rows,k,n", [(1, 1, 8, 8), (3, 33, 72, 40), (40, 70, 136, 264), (2, 300, 2056, 136),
                                        (1, 45, 4104, 24)])
def test_products_write_inside_their_buffers(dev, E, rows, k, n):  # noqa: F811
    g = Guarded(dev)
    counts = (torch.arange(E, device=dev, dtype=torch.int32) * 17 + rows) % (rows + 1)
    for grouped in (True, False):
        lead = (E, rows) if grouped else (E * rows,)
        groups = (E,) if grouped else ()
        cnt = (counts,) if grouped else ()
        fwd, dgrad, wgrad = ((ep.experts_product, ep.experts_product_dgrad, ep.experts_product_wgrad) if grouped
                             else (ep.linear, ep.linear_dgrad, ep.linear_wgrad))
        status = g.tensor((1,), torch.int32)
        status.zero_()
        for act in ("none", "gelu", "swiglu"):
            two = 2 if act == "swiglu" else 1
            for dtype in (BF16, F32):
                fwd(rand(dev, *lead, k), rand(dev, *groups, two * n, k), *cnt, act=act, out=g.tensor((*lead, n), dtype),
                    preact=g.tensor((*lead, two * n), BF16), residual=rand(dev, *lead, n),
                    bias=rand(dev, *groups, two * n), status=status)
                dgrad(rand(dev, *lead, n), rand(dev, *groups, n, k), *cnt, act=act,
                      preact=None if act == "none" else rand(dev, *lead, two * k),
                      out=g.tensor((*lead, two * k), dtype), status=status)
            if act != "none":
                ep.act_grad(rand(dev, *lead, n), rand(dev, *lead, two * n), act, counts=counts if grouped else None,
                            out=g.tensor((*lead, two * n), BF16))
        for dtype in (BF16, F32):
            out, db = g.tensor((*groups, n, k), dtype), g.tensor((*groups, n), dtype)
            wgrad(rand(dev, *lead, n), rand(dev, *lead, k), *cnt, out=out, bias_grad=db, status=status)
            wgrad(rand(dev, *lead, n), rand(dev, *lead, k), *cnt, out=out, bias_grad=db, accumulate=True, status=status)
        g.check()
        assert int(status.item()) == 0


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 33, 8), (130, 257, 16), (3, 1024, 16)])
def test_router_writes_inside_its_buffers(dev, T, E, k):  # noqa: F811
    g = Guarded(dev)
    z = torch.randn(T, E, device=dev)
    ids, w = ep.route_topk(z, k, out=(g.tensor((T, k), torch.int32), g.tensor((T, k), F32)))
    ep.route_topk_backward(torch.ones(T, k, device=dev), z, ids, score="softmax", renormalize=False,
                           out=g.tensor((T, E), F32))
    zb = z.to(BF16)
    ep.route_topk_backward(torch.ones(T, k, device=dev), zb, ids, score="sigmoid", out=g.tensor((T, E), BF16))
    g.check()
