"""The products and the router on seeded random shapes, counts and options against the
64-bit definitions of tests/_layers64.py (40 cases by default, any number through
EP_RANDOM_LAYER_CASES)."""
import os
import random

import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R
from tests.test_gpu_products import close, gen, normal
from tests.test_gpu_products import built  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")
CASES = int(os.environ.get("EP_RANDOM_LAYER_CASES", "40"))


def spread(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(CASES))
def test_random_product(seed):
    rng = random.Random(seed)
    g = gen(seed)
    E = rng.choice((None, 1, 2, 5, 16, 61, 400))
    lim = 700 if E is None or E < 16 else 300 if E < 100 else 40
    rows = spread(rng, 1, lim if E else 3000)
    k, n = 8 * spread(rng, 1, 300 if E is None or E < 16 else 40), 8 * spread(rng, 1, 300 if E is None or E < 16 else 40)
    act, dtype = rng.choice(ACTS), rng.choice((BF16, F32))
    two = 2 if act == "swiglu" else 1
    lead = (rows,) if E is None else (E, rows)
    groups = () if E is None else (E,)
    counts = [rows] if E is None else [rng.choice((0, 1, rows, rng.randint(0, rows), rng.randint(0, rows))) for _ in range(E)]
    cnt = () if E is None else (torch.tensor(counts, dtype=torch.int32, device="cuda"),)
    fwd, dgrad, wgrad = ((ep.linear, ep.linear_dgrad, ep.linear_wgrad) if E is None else
                         (ep.experts_product, ep.experts_product_dgrad, ep.experts_product_wgrad))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def spoiled(*shape):
        """Rows past the counts hold NaN or infinities."""
        t = normal(g, *shape)
        if E is not None:
            for e, c in enumerate(counts):
                t[e, c:] = rng.choice((float("nan"), float("inf"), -float("inf")))
        return t

    def each(t):
        return t[None] if E is None else t

    x, w = spoiled(*lead, k), normal(g, *groups, two * n, k, std=k ** -0.5)
    b = normal(g, *groups, two * n) if rng.random() < 0.5 else None
    r = spoiled(*lead, n) if rng.random() < 0.5 else None
    z = torch.full((*lead, two * n), 7.0, dtype=BF16, device="cuda") if rng.random() < 0.5 else None
    out = torch.full((*lead, n), 7.0, dtype=dtype, device="cuda")
    fwd(x, w, *cnt, bias=b, act=act, residual=r, out=out, preact=z, status=status)
    dy, w2, zin = spoiled(*lead, n), normal(g, *groups, n, k, std=n ** -0.5), spoiled(*lead, two * k)
    dx = torch.full((*lead, two * k), 7.0, dtype=dtype, device="cuda")
    dgrad(dy, w2, *cnt, act=act, preact=None if act == "none" else zin, out=dx, status=status)
    add = rng.random() < 0.5
    dw = normal(g, *groups, n, k, dtype=dtype)
    db = normal(g, *groups, n, dtype=dtype)
    before = (dw.clone(), db.clone()) if add else None
    wgrad(dy, x, *cnt, out=dw, bias_grad=db, accumulate=add, status=status)
    assert status.item() == 0
    for e, c in enumerate(counts):
        y, ey, zz, ez = R.forward(each(x)[e, :c], each(w)[e], None if b is None else each(b)[e], act,
                                  None if r is None else each(r)[e, :c], dtype)
        close(each(out)[e, :c], y, ey, f"out {e}")
        assert (each(out)[e, c:] == 7.0).all()
        if z is not None:
            close(each(z)[e, :c], zz, ez, f"z {e}")
            assert (each(z)[e, c:] == 7.0).all()
        d, ed = R.dgrad(each(dy)[e, :c], each(w2)[e], act, each(zin)[e, :c], dtype)
        close(each(dx)[e, :c], d, ed, f"dx {e}")
        assert (each(dx)[e, c:] == 7.0).all()
        w64, ew, b64, eb = R.wgrad(each(dy)[e, :c], each(x)[e, :c], dtype,
                                   None if before is None else (each(before[0])[e], each(before[1])[e]))
        close(each(dw)[e], w64, ew, f"dw {e}")
        close(each(db)[e], b64, eb, f"db {e}")


@pytest.mark.parametrize("seed", range(CASES))
def test_random_router(seed):
    from tests.test_gpu_router import FORMS, check
    rng = random.Random(1000 + seed)
    E = spread(rng, 1, 1024)
    T, k = spread(rng, 1, 60), rng.randint(1, min(16, E))
    dtype = rng.choice((BF16, F32))
    z = (2 * torch.randn(T, E, generator=torch.Generator().manual_seed(seed))).to(dtype)
    if rng.random() < 0.5:           # ties, and experts masked out
        z = z.round()
        z[torch.rand(T, E, generator=torch.Generator().manual_seed(seed + 1)) < rng.random()] = -float("inf")
    bias = torch.randn(E, generator=torch.Generator().manual_seed(seed + 2)).cuda() if rng.random() < 0.5 else None
    check(z.cuda(), k, *rng.choice(FORMS), bias=bias, scale=rng.choice((1.0, 2.5)))
