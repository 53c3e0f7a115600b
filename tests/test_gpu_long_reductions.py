"""Long reductions: the error of a sum does not grow with its length. Operands are not
negative, so that a one-sided rounding of every step would add up, and the bounds are
relative to the result.

The tensor cores truncate: a step of 16 terms is taken to be off by up to a unit (2^-23) of the
running sum (measured 0.45 in chains of 64 steps, 1.2 in chains of 1024). That sum grows evenly here (to a
tenth), so a chain of s steps is off by at most 1.1 s / 2 units, and a few for its first steps and the
joins of chains; P passes are added up with rounding by at most half a unit each of a sum that grows
as evenly, P / 4 in all. The bound of bf16 results leaves room for chains longer than the kernel's."""
import pytest
import torch

import combine_ep_route_gb300 as ep

pytestmark = pytest.mark.gpu
BF16, F32, D = torch.bfloat16, torch.float32, torch.float64
CHAIN = {F32: 1024, BF16: 65536}     # terms of a chain, at most


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def positive(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda").to(BF16)


def sum_error(k, dtype):
    steps, passes = min(k, CHAIN[dtype]) / 16, k / CHAIN[dtype] + 1
    return (1.1 * steps / 2 + 16 + passes / 4) * 2.0 ** -23


def fits(got, want, k, extra=0.0):
    """Between the roundings, to the result's type, of what the sums may come to."""
    e = sum_error(k, got.dtype) + extra + 2.0 ** -23
    lo, hi = (want * (1 - e)).to(got.dtype), (want * (1 + e)).to(got.dtype)
    bad = ~((lo <= got) & (got <= hi))
    worst = float(((got.to(D) - want) / want).abs().max())
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst relative error {worst:.2e} (sums: {e:.2e})"


def matmul64(a, b):
    """a @ b in 64 bits, the reduction in parts that fit."""
    return sum(a[:, i:i + 65536].to(D) @ b[i:i + 65536].to(D) for i in range(0, a.shape[1], 65536))


@pytest.mark.parametrize("rows,k,n", [(1024, 264, 264), (1025, 264, 264), (40000, 264, 520), (50001, 136, 72), (66000, 24, 16),
                                      (12345, 2056, 2048)])
def test_weight_gradient_f32(rows, k, n):
    g = gen(rows)
    dy, x = positive(g, rows, n), positive(g, rows, k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = ep.linear_wgrad(dy, x, out_dtype=F32, status=status)
    fits(dw, matmul64(dy.T, x), rows)
    assert torch.equal(dw, ep.linear_wgrad(dy, x, out_dtype=F32)) and status.item() == 0
    before = positive(g, n, k).float()
    out = before.clone()
    ep.linear_wgrad(dy, x, out=out, accumulate=True)
    fits(out, matmul64(dy.T, x) + before.to(D), rows)


@pytest.mark.parametrize("dtype", (F32, BF16))
@pytest.mark.parametrize("k,n", [(136, 264), (392, 40)])
def test_experts_weight_gradient(k, n, dtype):
    """Groups of one, two and many passes by turns on the same CTAs."""
    counts = [5000, 0, 1, 1024, 1030, 2048, 7, 3000, 4999, 64] * 8
    g = gen(k)
    dy, x = positive(g, len(counts), 5000, n), positive(g, len(counts), 5000, k)
    for e, c in enumerate(counts):
        dy[e, c:], x[e, c:] = float("nan"), float("inf")
    dw = ep.experts_product_wgrad(dy, x, torch.tensor(counts, dtype=torch.int32, device="cuda"), out_dtype=dtype)
    for e, c in enumerate(counts):
        if c:
            fits(dw[e], matmul64(dy[e, :c].T, x[e, :c]), c)
        else:
            assert (dw[e] == 0).all()


@pytest.mark.parametrize("rows,k,n", [(1, 20000, 40), (7, 70000, 264), (40, 16392, 136), (300, 16392, 520), (2100, 7168, 2056)])
def test_forward_and_input_gradient_f32(rows, k, n):
    g = gen(rows + k)
    x, w, r, b = positive(g, rows, k), positive(g, n, k), positive(g, rows, n), positive(g, n)
    y = ep.linear(x, w, bias=b, residual=r, out_dtype=F32)
    fits(y, matmul64(x, w.T) + b.to(D) + r.to(D), k, 2.0 ** -22)
    w2 = positive(g, k, n)
    fits(ep.linear_dgrad(x, w2, out_dtype=F32), matmul64(x, w2), k)
    # through relu: its slope is 1 on positive inputs
    z = positive(g, rows, n) + 1
    fits(ep.linear_dgrad(x, w2, act="relu", preact=z, out_dtype=F32), matmul64(x, w2), k)


def test_experts_forward_f32():
    counts = [0, 1, 15, 33, 64, 100, 255, 257, 300] * 9
    g = gen(3)
    x, w = positive(g, len(counts), 300, 5000), positive(g, len(counts), 264, 5000)
    y = ep.experts_product(x, w, torch.tensor(counts, dtype=torch.int32, device="cuda"), out_dtype=F32)
    for e, c in enumerate(counts):
        if c:
            fits(y[e, :c], matmul64(x[e, :c], w[e].T), 5000)


def test_bf16_results():
    g = gen(4)
    rows = (1 << 20) + 77
    dy, x = positive(g, rows, 264), positive(g, rows, 136)
    fits(ep.linear_wgrad(dy, x), matmul64(dy.T, x), rows)
    x, w = positive(g, 40, 300000), positive(g, 136, 300000)
    fits(ep.linear(x, w), matmul64(x, w.T), 300000)
    gated = positive(g, 2 * 72, 300000)
    y = ep.linear(x, gated, act="swiglu", out_dtype=F32)   # of gates this large silu is the identity
    z = matmul64(x, gated.T)
    fits(y, z[:, :72] * z[:, 72:], 300000, sum_error(300000, F32) + 2.0 ** -22)


def test_a_group_of_800_million_rows():
    """One tile, one CTA, over two seconds of reduction: no wait of the kernel covers all of it."""
    rows = 800_000_001
    ones = torch.ones(1, rows, 8, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cnt = torch.tensor([rows], dtype=torch.int32, device="cuda")
    for dtype in (BF16, F32):
        dw = ep.experts_product_wgrad(ones, ones, cnt, out_dtype=dtype, status=status)
        assert status.item() == 0
        assert torch.equal(dw, torch.full((1, 8, 8), rows, dtype=D, device="cuda").to(dtype))


def test_the_most_rows():
    """2^31 - 1 rows, the last block of which ends past what 32 bits with a sign hold."""
    rows = (1 << 31) - 1
    ones = torch.ones(rows, 8, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = ep.linear_wgrad(ones, ones, out_dtype=F32, status=status)
    assert status.item() == 0 and (dw == 2.0 ** 31).all()
