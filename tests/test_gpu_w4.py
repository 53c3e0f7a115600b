"""Products with 4-bit weights against 64 bits: the definition of a product (tests/_layers64.py, with its
error bounds: fp32 sums in steps of 16, one rounding) on the weight that the codes and scales stand for."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)


def weight(g, groups, rows, k, group):
    """Random codes and scales, packed, with a leading dimension of groups."""
    codes = torch.randint(0, 16, (groups, rows, k), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.5 + torch.rand(groups, rows, k // group, generator=g, device="cuda")) * k ** -0.5 / 4
    scales[..., 0] *= -1
    return ep.pack_weight4(codes, scales)


def check_linear(rows, k, n, act="none", kind="int4", group=32, bias=False, residual=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + k + n + seed)
    wn = 2 * n if act == "swiglu" else n
    x, (codes, scales) = rand(g, rows, k), weight(g, 1, wn, k, group)
    b = rand(g, wn) if bias else None
    r = rand(g, rows, n) if residual else None
    y = ep.linear_w4(x, codes[0], scales[0], kind=kind, bias=b, act=act, residual=r)
    want, off, _, _ = R.forward(x, ep.dequantize_weight4(codes[0], scales[0], kind), b, act, r, BF16)
    assert y.shape == (rows, n) and ((y.double() - want).abs() <= off).all()
    ep.check_products()


@pytest.mark.parametrize("kind", ("int4", "fp4"))
@pytest.mark.parametrize("group", (32, 64, 128))
@pytest.mark.parametrize("rows,k,n", [(1, 128, 8), (1, 256, 24), (3, 384, 136), (8, 1024, 64), (9, 128, 128), (16, 640, 72),
                                      (17, 512, 40), (33, 896, 264), (65, 128, 16), (130, 1152, 200), (300, 256, 392)])
def test_linear(rows, k, n, group, kind):
    check_linear(rows, k, n, "none", kind, group)
    check_linear(rows, k, n, "swiglu", kind, group, bias=True, residual=True)


@pytest.mark.parametrize("act", ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"))
@pytest.mark.parametrize("rows", (2, 40, 200))
def test_epilogues(rows, act):
    for bias in (False, True):
        for residual in (False, True):
            check_linear(rows, 96, 56, act, "fp4", 32, bias, residual)


@pytest.mark.parametrize("k", (32, 64, 96, 160, 2080, 2176, 32768))
@pytest.mark.parametrize("rows", (1, 20, 150))
def test_reductions_of_any_length(rows, k):
    check_linear(rows, k, 48, kind="int4")
    check_linear(rows, k, 8, "swiglu", kind="fp4")


@pytest.mark.parametrize("rows,k,n", [(1, 7168, 7168), (7, 2048, 4096), (64, 4096, 1024), (513, 2048, 2048)])
def test_larger_sizes(rows, k, n):
    check_linear(rows, k, n, "silu", "int4", 128, True, True)


def experts(counts, rows, k, n, act, kind, group, seed=0, bias=True, residual=True):
    E = len(counts)
    g = torch.Generator(device="cuda").manual_seed(E * 1000 + rows + seed)
    wn = 2 * n if act == "swiglu" else n
    x, (codes, scales) = rand(g, E, rows, k), weight(g, E, wn, k, group)
    b = rand(g, E, wn) if bias else None
    r = rand(g, E, rows, n) if residual else None
    cnt = torch.tensor(counts, dtype=I32, device="cuda")
    for e, c in enumerate(counts):      # what no token wrote may hold anything
        x[e, max(0, c):] = NAN
        if r is not None:
            r[e, max(0, c):] = NAN
    out = torch.full((E, rows, n), 7.0, dtype=BF16, device="cuda")
    y = ep.experts_product_w4(x, codes, scales, cnt, kind=kind, bias=b, act=act, residual=r, out=out)
    assert y is out
    w = ep.dequantize_weight4(codes, scales, kind)
    for e, c in enumerate(counts):
        c = max(0, min(c, rows))
        want, off, _, _ = R.forward(x[e, :c], w[e], None if b is None else b[e], act, None if r is None else r[e, :c], BF16)
        assert ((y[e, :c].double() - want).abs() <= off).all(), e
        assert (y[e, c:] == 7.0).all(), e
    ep.check_products()
    return x, codes, scales, cnt, b, r, y


@pytest.mark.parametrize("kind,group", (("int4", 32), ("fp4", 64), ("int4", 128)))
@pytest.mark.parametrize("act", ("none", "swiglu"))
@pytest.mark.parametrize("counts,rows", [([3], 4), ([0, 1, 8, 5], 8), ([0, 0], 16), ([16, 1, 9, 0, 15], 16),
                                         ([0, 17, 64, 1, 33, 90], 70), ([-3, 300, 128, 129, 0, 255, 256, 7], 300),
                                         ([1] * 60, 33)])
def test_experts(counts, rows, act, kind, group):
    experts(counts, rows, 256, 72, act, kind, group)


@pytest.mark.parametrize("act,n", (("none", 136), ("none", 400), ("swiglu", 72), ("swiglu", 200)))
@pytest.mark.parametrize("rows,most", ((17, 8), (40, 40), (130, 130), (300, 300)))
def test_many_experts(act, n, rows, most):
    """Enough tiles for pairs of CTAs, with an odd number of tiles of the weight among them, and counts on both
    sides of what one CTA of a pair holds."""
    g = torch.Generator().manual_seed(rows + n)
    counts = torch.randint(0, most + 1, (90,), generator=g).tolist()
    counts[:8] = [0, 1, min(16, most), min(17, most), min(32, most), min(33, most), most, most]
    experts(counts, rows, 352, n, act, "fp4" if n > 150 else "int4", 32)


def test_experts_with_leading_dimensions():
    x, codes, scales, cnt, b, r, y = experts([3, 0, 9, 40, 1, 2], 40, 128, 64, "swiglu", "fp4", 32)
    lead = lambda t: t.view(2, 3, *t.shape[1:])  # noqa: E731
    z = ep.experts_product_w4(lead(x), lead(codes), lead(scales), lead(cnt), kind="fp4", bias=lead(b), act="swiglu",
                              residual=lead(r))
    for e, c in enumerate(cnt.tolist()):
        assert torch.equal(z.view(y.shape)[e, :c], y[e, :c])


@pytest.mark.parametrize("rows,counts", ((7, (7, 0, 3)), (40, (40, 1, 17)), (140, (140, 0, 129))))
@pytest.mark.parametrize("act", ("none", "swiglu"))
def test_what_lies_around_stays(rows, counts, act):
    """Results are written to the rows in use alone, whatever lies before and behind the output."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = 72
    x, (codes, scales) = rand(g, 3, rows, 160), weight(g, 3, 2 * n if act == "swiglu" else n, 160, 32)
    flat = torch.full((3 * rows * n + 4096,), 5.0, dtype=BF16, device="cuda")
    out = flat[2048:2048 + 3 * rows * n].view(3, rows, n)
    ep.experts_product_w4(x, codes, scales, torch.tensor(counts, dtype=I32, device="cuda"), act=act, out=out)
    assert (flat[:2048] == 5.0).all() and (flat[-2048:] == 5.0).all()
    for e, c in enumerate(counts):
        assert (out[e, c:] == 5.0).all() and not (out[e, :c] == 5.0).all(dim=-1).any()


def test_residual_in_place_and_nothing_to_do():
    g = torch.Generator(device="cuda").manual_seed(1)
    for rows in (5, 100):
        x, (codes, scales), r = rand(g, rows, 128), weight(g, 1, 64, 128, 32), rand(g, rows, 64)
        want = ep.linear_w4(x, codes[0], scales[0], residual=r)
        assert torch.equal(ep.linear_w4(x, codes[0], scales[0], residual=r, out=r), want)
    assert ep.linear_w4(x[:0], codes[0], scales[0]).shape == (0, 64)


@pytest.mark.parametrize("rows", (1, 12, 70, 260))
def test_rows_do_not_touch_one_another_and_give_the_same_bits(rows):
    """A row's result depends on that row alone, and two calls agree to the bit."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, (codes, scales) = rand(g, rows, 512), weight(g, 1, 128, 512, 64)
    y = ep.linear_w4(x, codes[0], scales[0])
    assert torch.equal(y, ep.linear_w4(x, codes[0], scales[0]))
    x2 = x.clone()
    x2[rows // 2] = NAN
    z = ep.linear_w4(x2, codes[0], scales[0])
    keep = torch.arange(rows, device="cuda") != rows // 2
    assert torch.equal(y[keep], z[keep]) and z[rows // 2].isnan().all()


@pytest.mark.parametrize("rows,n,groups", ((64, 256, 1), (130, 512, 40), (128, 512, 8), (1, 4096, 1)))
def test_long_reductions_agree_each_time(rows, n, groups):
    """Copies of a long reduction arrive in no fixed order (rows of codes 16 KB apart, other traffic between
    the calls): the result is the same to the bit each time, and right."""
    g = torch.Generator(device="cuda").manual_seed(8)
    k = 32768 if groups == 1 else 8192
    x, (codes, scales) = rand(g, groups, rows, k), weight(g, groups, n, k, 64)
    cnt = torch.full((groups,), rows, dtype=I32, device="cuda")
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def call():
        if groups == 1:
            return ep.linear_w4(x[0], codes[0], scales[0])[None]
        return ep.experts_product_w4(x, codes, scales, cnt)

    first = call()
    want, off, _, _ = R.forward(x[-1], ep.dequantize_weight4(codes[-1], scales[-1]), None, "none", None, BF16)
    assert ((first[-1].double() - want).abs() <= off).all()
    for i in range(30):
        if i % 2:
            other.fill_(i)
        assert torch.equal(call(), first), i
    ep.check_products()


def test_scales_of_any_size():
    """Scales so small or large that a weight leaves bf16's normal numbers, or is infinite."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for kind in ("int4", "fp4"):
        x, (codes, scales) = rand(g, 3, 64), weight(g, 1, 32, 64, 32)
        codes[0, :, :16] = 0x21               # no code of zero beside the infinite ones
        scales[0, 0] = torch.tensor([2.0 ** -130, 2.0 ** 100, -2.0 ** -126, 1e-38] * 8, device="cuda").to(BF16)
        y = ep.linear_w4(x, codes[0], scales[0], kind=kind)
        want, off, _, _ = R.forward(x, ep.dequantize_weight4(codes[0], scales[0], kind), None, "none", None, BF16)
        assert ((y.double() - want).abs() <= off).all()
        scales[0, 0, 5] = float("inf")
        y = ep.linear_w4(x.abs(), codes[0], scales[0], kind=kind)
        assert torch.isinf(y[:, 5]).all() and torch.isfinite(y[:, 6]).all()
        scales[0, 1, 9] = NAN
        assert ep.linear_w4(x, codes[0], scales[0], kind=kind)[:, 9].isnan().all()


@pytest.mark.parametrize("rows", (1, 30, 200))
def test_streams_and_graphs(rows):
    g = torch.Generator(device="cuda").manual_seed(4)
    x, (codes, scales) = rand(g, rows, 1024), weight(g, 1, 512, 1024, 128)
    want = ep.linear_w4(x, codes[0], scales[0], act="swiglu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ep.linear_w4(x, codes[0], scales[0], act="swiglu", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ep.linear_w4(x, codes[0], scales[0], act="swiglu")
    x.copy_(rand(g, rows, 1024))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ep.linear_w4(x, codes[0], scales[0], act="swiglu"))
    ep.check_products()


def test_same_as_the_bf16_product():
    """The bf16 product of the weight that the codes stand for differs by the order of its sums alone."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x, (codes, scales) = rand(g, 100, 2048), weight(g, 1, 256, 2048, 32)
    w = ep.dequantize_weight4(codes[0], scales[0], "fp4")
    y, z = ep.linear_w4(x, codes[0], scales[0], kind="fp4"), ep.linear(x, w)
    assert ((y.double() - z.double()).norm() <= 2.0 ** -9 * z.double().norm())


def test_refusals():
    g = torch.Generator(device="cuda").manual_seed(6)
    x, (codes, scales) = rand(g, 4, 128), weight(g, 2, 16, 128, 32)
    c, s = codes[0], scales[0]
    cnt = torch.ones(2, dtype=I32, device="cuda")
    for call in (lambda: ep.linear_w4(x.float(), c, s), lambda: ep.linear_w4(x, c.to(torch.int8), s),
                 lambda: ep.linear_w4(x, c, s.float()), lambda: ep.linear_w4(x, c, s.t()),
                 lambda: ep.linear_w4(x, c, s.t().contiguous()), lambda: ep.linear_w4(x, c[:, :32].contiguous(), s),
                 lambda: ep.linear_w4(x, c.cpu(), s), lambda: ep.linear_w4(x, c[:12].contiguous(), s),
                 lambda: ep.linear_w4(x, c[:8].contiguous(), s[:, :8].contiguous(), act="swiglu"),
                 lambda: ep.linear_w4(x, codes, scales), lambda: ep.linear_w4(x, c, s, bias=x[0]),
                 lambda: ep.linear_w4(x, c, s, residual=x), lambda: ep.linear_w4(x, c, s, out=x),
                 lambda: ep.linear_w4(x, c, s, out=torch.empty(4, 16, device="cuda")),
                 lambda: ep.experts_product_w4(x[None], codes, scales, cnt),
                 lambda: ep.experts_product_w4(x.view(2, 2, 128), codes, scales, cnt[:1]),
                 lambda: ep.experts_product_w4(x.view(2, 2, 128), codes, scales, cnt.long()),
                 lambda: ep.experts_product_w4(x.view(2, 2, 128), codes, scales, None),
                 lambda: ep.linear_w4(x.clone().requires_grad_(), c, s),
                 lambda: ep.linear_w4(x, c, s, bias=rand(g, 16).requires_grad_())):
        with pytest.raises(ValueError):
            call()
    w = x.clone().requires_grad_()
    with torch.no_grad():
        ep.linear_w4(w, c, s)
