"""The experts' and linear products and their gradients against 64-bit definitions,
at the sizes, counts and contents where a tiled kernel can go wrong. Bounds are those
of tests/_layers64.py."""
import pytest
import torch

import combine_ep_route_gb300 as ep
from tests import _layers64 as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def close(got, want, bound, what=""):
    got = got.to(torch.float64)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(((got - want).abs() / bound).max())} bounds"


def check_forward(E, rows, k, n, act, counts, *, bias=False, residual=False, keep=False, dtype=BF16, seed=0):
    g = gen(seed)
    wn = 2 * n if act == "swiglu" else n
    x = normal(g, E, rows, k)
    w = normal(g, E, wn, k, std=k ** -0.5)
    b = normal(g, E, wn) if bias else None
    r = normal(g, E, rows, n) if residual else None
    for e, c in enumerate(counts):
        x[e, max(c, 0):] = float("nan")           # rows not in use hold anything
        if residual:
            r[e, max(c, 0):] = float("nan")
    out = torch.full((E, rows, n), 7.0, dtype=dtype, device="cuda")
    z = torch.full((E, rows, wn), 7.0, dtype=BF16, device="cuda") if keep else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    got = ep.experts_product(x, w, cnt, bias=b, act=act, residual=r, out=out, preact=z, status=status)
    assert got is out and status.item() == 0
    for e, c in enumerate(counts):
        c = min(max(c, 0), rows)
        y, ey, zz, ez = R.forward(x[e, :c], w[e], None if b is None else b[e], act, None if r is None else r[e, :c], dtype)
        close(out[e, :c], y, ey, f"expert {e}")
        assert (out[e, c:] == 7.0).all(), "a row past the count was written"
        if keep:
            close(z[e, :c], zz, ez, f"pre-activation of expert {e}")
            assert (z[e, c:] == 7.0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("k,n", [(64, 128), (8, 8), (72, 24), (200, 136), (520, 264)])
def test_experts_forward(act, k, n):
    check_forward(6, 40, k, n, act, [0, 1, 15, 16, 17, 40], bias=True, keep=True)


@pytest.mark.parametrize("act", ("none", "swiglu"))
def test_experts_forward_wide_tiles(act):
    check_forward(7, 600, 136, 144, act, [255, 256, 257, 300, 513, 600, 0])


# enough tiles for pairs of CTAs to share each (two lane tiles, more than the GPU's pairs in all)
PAIRED = [0, 1, 15, 16, 17, 31, 32, 33, 64, 100, 255, 256, 257, 300] * 3


@pytest.mark.parametrize("act", ("none", "gelu", "swiglu"))
@pytest.mark.parametrize("k,n", [(136, 264), (72, 392)])
def test_experts_forward_paired(act, k, n):
    check_forward(len(PAIRED), 300, k, n, act, PAIRED, bias=True, residual=True, keep=True)


@pytest.mark.parametrize("act", ("none", "swiglu"))
def test_experts_wide_tiles_long_reduction(act):
    """257..512 rows of a group as one tile over both accumulators, among narrow ones."""
    counts = [512, 257, 256, 300, 513, 0, 400, 511, 1, 600, 320, 288] * 4
    check_forward(len(counts), 600, 2120, 264, act, counts, bias=True, residual=True, keep=True)
    g = gen(31)
    E, rows, n, k, two = len(counts), 600, 2120, 136, 2 if act == "swiglu" else 1
    dy, w, z = normal(g, E, rows, n), normal(g, E, n, k, std=n ** -0.5), normal(g, E, rows, two * k)
    out = torch.full((E, rows, two * k), 7.0, dtype=BF16, device="cuda")
    ep.experts_product_dgrad(dy, w, torch.tensor(counts, dtype=torch.int32, device="cuda"), act=act,
                             preact=None if act == "none" else z, out=out)
    for e, c in enumerate(counts):
        d, ed = R.dgrad(dy[e, :c], w[e], act, z[e, :c], BF16)
        close(out[e, :c], d, ed, f"expert {e}")
        assert (out[e, c:] == 7.0).all()


@pytest.mark.parametrize("rows", [1, 7, 16, 33, 64])
@pytest.mark.parametrize("k,n", [(2048, 7168), (712, 4104), (4096, 2056), (7168, 2432)])
def test_linear_few_rows(rows, k, n):
    """Few rows on many features: lane tiles narrower than the accumulator."""
    g = gen(rows + n)
    for act, dtype in (("none", F32), ("gelu", BF16), ("swiglu", BF16)):
        wn = 2 * n if act == "swiglu" else n
        x, w, b, r = normal(g, rows, k), normal(g, wn, k, std=k ** -0.5), normal(g, wn), normal(g, rows, n)
        z = torch.empty(rows, wn, dtype=BF16, device="cuda")
        got = ep.linear(x, w, bias=b, act=act, residual=r, out_dtype=dtype, preact=z)
        y, ey, zz, ez = R.forward(x, w, b, act, r, dtype)
        close(got, y, ey, act)
        close(z, zz, ez, act)


@pytest.mark.parametrize("rows", [1, 7, 64, 130, 300])
@pytest.mark.parametrize("k,n", [(4104, 136), (7168, 16), (1000, 3080)])
def test_linear_long_reduction_few_tiles(rows, k, n):
    """Few tiles: the CTAs of a cluster share a tile's reduction."""
    g = gen(rows + k)
    for act, dtype in (("none", F32), ("swiglu", BF16)):
        wn = 2 * n if act == "swiglu" else n
        x, w, b, r = normal(g, rows, k), normal(g, wn, k, std=k ** -0.5), normal(g, wn), normal(g, rows, n)
        z = torch.empty(rows, wn, dtype=BF16, device="cuda")
        got = ep.linear(x, w, bias=b, act=act, residual=r, out_dtype=dtype, preact=z)
        y, ey, zz, ez = R.forward(x, w, b, act, r, dtype)
        close(got, y, ey, act)
        close(z, zz, ez, act)
        dy, w2, zin = normal(g, rows, k), normal(g, k, n, std=k ** -0.5), normal(g, rows, 2 * n)
        d, ed = R.dgrad(dy, w2, "swiglu", zin, dtype)
        close(ep.linear_dgrad(dy, w2, act="swiglu", preact=zin, out_dtype=dtype), d, ed)


@pytest.mark.parametrize("rows,k,n", [(4097, 72, 40), (2000, 264, 136), (3001, 1032, 2056), (700, 5000, 4104)])
def test_linear_gradients_large(rows, k, n):
    """Weight gradients split over the rows, and paired tiles."""
    g = gen(rows)
    dy, x, w, z = normal(g, rows, n), normal(g, rows, k), normal(g, n, k, std=n ** -0.5), normal(g, rows, k)
    before = normal(g, n, k, dtype=F32), normal(g, n, dtype=F32)
    dw, db = before[0].clone(), before[1].clone()
    ep.linear_wgrad(dy, x, out=dw, bias_grad=db, accumulate=True)
    w64, ew, b64, eb = R.wgrad(dy, x, F32, before)
    close(dw, w64, ew)
    close(db, b64, eb)
    d, ed = R.dgrad(dy, w, "gelu", z, BF16)
    close(ep.linear_dgrad(dy, w, act="gelu", preact=z), d, ed)


def test_experts_forward_residual_and_f32():
    check_forward(3, 70, 96, 72, "silu", [70, 0, 33], bias=True, residual=True)
    check_forward(3, 70, 96, 72, "swiglu", [70, 0, 33], bias=True, residual=True)
    check_forward(3, 70, 96, 72, "none", [70, 0, 33], residual=True, dtype=F32)


def test_counts_outside_the_rows_are_clamped():
    check_forward(3, 20, 64, 64, "none", [-5, 25, 3])


def test_no_expert_has_rows():
    check_forward(5, 20, 64, 64, "swiglu", [0] * 5, bias=True, keep=True)


def test_many_experts():
    g = torch.Generator().manual_seed(3)
    check_forward(1024, 5, 64, 40, "none", torch.randint(0, 6, (1024,), generator=g).tolist())


def test_long_reduction():
    check_forward(2, 48, 7168, 136, "none", [48, 7])


def test_infinite_and_nan_inputs_stay_in_their_rows():
    g = gen(5)
    x, w = normal(g, 1, 32, 64), normal(g, 1, 48, 64)
    x[0, 3, 5] = float("inf")
    x[0, 9, 9] = float("nan")
    got = ep.experts_product(x, w, torch.tensor([32], dtype=torch.int32, device="cuda"))
    clean = torch.ones(32, dtype=torch.bool, device="cuda")
    clean[3] = clean[9] = False
    y, ey, _, _ = R.forward(x[0, clean], w[0], None, "none", None, BF16)
    close(got[0, clean], y, ey)
    assert torch.isnan(got[0, 9]).all() and torch.isinf(got[0, 3]).all()


def test_leading_dimensions_are_groups():
    g = gen(6)
    x, w = normal(g, 2, 3, 9, 64), normal(g, 2, 3, 32, 64)
    cnt = torch.tensor([[9, 0, 4], [1, 2, 3]], dtype=torch.int32, device="cuda")
    got = ep.experts_product(x, w, cnt)
    flat = ep.experts_product(x.view(6, 9, 64), w.view(6, 32, 64), cnt.view(-1))
    for e, c in enumerate(cnt.view(-1).tolist()):
        assert torch.equal(got.view(6, 9, 32)[e, :c], flat[e, :c])


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 64, 129, 300, 777])
@pytest.mark.parametrize("k,n", [(64, 64), (136, 392), (1032, 8)])
def test_linear_forward(rows, k, n):
    g = gen(rows)
    for act, dtype in (("none", F32), ("gelu", BF16), ("swiglu", BF16)):
        wn = 2 * n if act == "swiglu" else n
        x, w, b, r = normal(g, rows, k), normal(g, wn, k, std=k ** -0.5), normal(g, wn), normal(g, rows, n)
        z = torch.empty(rows, wn, dtype=BF16, device="cuda")
        got = ep.linear(x, w, bias=b, act=act, residual=r, out_dtype=dtype, preact=z)
        y, ey, zz, ez = R.forward(x, w, b, act, r, dtype)
        assert got.dtype == dtype
        close(got, y, ey, act)
        close(z, zz, ez, act)


def test_linear_output_may_be_the_residual():
    g = gen(8)
    x, w, r = normal(g, 45, 128), normal(g, 72, 128, std=0.1), normal(g, 45, 72)
    y, ey, _, _ = R.forward(x, w, None, "relu", r, BF16)
    assert ep.linear(x, w, act="relu", residual=r, out=r) is r
    close(r, y, ey)


def test_linear_without_rows():
    w = torch.zeros(16, 8, dtype=BF16, device="cuda")
    assert ep.linear(torch.zeros(0, 8, dtype=BF16, device="cuda"), w).shape == (0, 16)
    assert ep.linear_dgrad(torch.zeros(0, 16, dtype=BF16, device="cuda"), w).shape == (0, 8)
    dw, db = ep.linear_wgrad(torch.zeros(0, 16, dtype=BF16, device="cuda"), torch.zeros(0, 8, dtype=BF16, device="cuda"),
                             bias_grad=True)
    assert (dw == 0).all() and (db == 0).all()
    assert ep.linear(torch.ones(2, 3, 8, dtype=BF16, device="cuda"), w).shape == (2, 3, 16)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("k,n", [(64, 128), (8, 8), (24, 72), (136, 200), (264, 520)])
def test_experts_dgrad(act, k, n):
    g = gen(11)
    counts, rows = [0, 1, 15, 16, 17, 300, 257], 300
    E, two = len(counts), 2 if act == "swiglu" else 1
    dy, w = normal(g, E, rows, n), normal(g, E, n, k, std=n ** -0.5)
    z = normal(g, E, rows, two * k, std=2.0)
    for e, c in enumerate(counts):
        dy[e, c:] = float("nan")
        z[e, c:] = float("nan")
    out = torch.full((E, rows, two * k), 7.0, dtype=BF16, device="cuda")
    ep.experts_product_dgrad(dy, w, torch.tensor(counts, dtype=torch.int32, device="cuda"), act=act,
                             preact=None if act == "none" else z, out=out)
    for e, c in enumerate(counts):
        d, ed = R.dgrad(dy[e, :c], w[e], act, z[e, :c], BF16)
        close(out[e, :c], d, ed, f"expert {e}")
        assert (out[e, c:] == 7.0).all()


@pytest.mark.parametrize("act", ("none", "silu", "swiglu"))
def test_experts_gradients_paired(act):
    g = gen(21)
    E, rows, n, k, two = len(PAIRED), 300, 136, 264, 2 if act == "swiglu" else 1
    dy, w, x = normal(g, E, rows, n), normal(g, E, n, k, std=n ** -0.5), normal(g, E, rows, k)
    z = normal(g, E, rows, two * k)
    for e, c in enumerate(PAIRED):
        dy[e, c:] = float("nan")
        z[e, c:] = float("nan")
        x[e, c:] = float("-inf")
    cnt = torch.tensor(PAIRED, dtype=torch.int32, device="cuda")
    out = torch.full((E, rows, two * k), 7.0, dtype=BF16, device="cuda")
    ep.experts_product_dgrad(dy, w, cnt, act=act, preact=None if act == "none" else z, out=out)
    dw, db = ep.experts_product_wgrad(dy, x, cnt, out_dtype=F32, bias_grad=True)
    for e, c in enumerate(PAIRED):
        d, ed = R.dgrad(dy[e, :c], w[e], act, z[e, :c], BF16)
        close(out[e, :c], d, ed, f"expert {e}")
        assert (out[e, c:] == 7.0).all()
        w64, ew, b64, eb = R.wgrad(dy[e, :c], x[e, :c], F32)
        close(dw[e], w64, ew, f"expert {e}")
        close(db[e], b64, eb, f"bias of expert {e}")


@pytest.mark.parametrize("act", ("none", "gelu", "swiglu"))
def test_linear_dgrad_f32(act):
    g = gen(12)
    dy, w = normal(g, 77, 328), normal(g, 328, 88, std=0.05)
    z = None if act == "none" else normal(g, 77, 176 if act == "swiglu" else 88)
    d, ed = R.dgrad(dy, w, act, z, F32)
    close(ep.linear_dgrad(dy, w, act=act, preact=z, out_dtype=F32), d, ed)


@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("k,n", [(64, 128), (8, 8), (24, 72), (136, 200), (264, 520)])
def test_experts_wgrad(dtype, k, n):
    g = gen(13)
    counts, rows = [0, 1, 15, 16, 17, 63, 64, 65, 100, 300], 300
    E = len(counts)
    dy, x = normal(g, E, rows, n), normal(g, E, rows, k)
    for e, c in enumerate(counts):   # infinities too: 0 * inf must not get into a sum
        dy[e, c:] = float("nan")
        x[e, c:] = float("inf")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = torch.full((E, n, k), 7.0, dtype=dtype, device="cuda")
    dw, db = ep.experts_product_wgrad(dy, x, cnt, out=out, bias_grad=True)
    assert dw is out and db.dtype == dtype
    before = normal(g, E, n, k, dtype=dtype), normal(g, E, n, dtype=dtype)
    aw, ab = before[0].clone(), before[1].clone()
    ep.experts_product_wgrad(dy, x, cnt, out=aw, bias_grad=ab, accumulate=True)
    for e, c in enumerate(counts):
        w64, ew, b64, eb = R.wgrad(dy[e, :c], x[e, :c], dtype)
        close(dw[e], w64, ew, f"expert {e}")
        close(db[e], b64, eb, f"bias of expert {e}")
        w64, ew, b64, eb = R.wgrad(dy[e, :c], x[e, :c], dtype, (before[0][e], before[1][e]))
        close(aw[e], w64, ew, f"expert {e}, added")
        close(ab[e], b64, eb, f"bias of expert {e}, added")


@pytest.mark.parametrize("rows", [1, 64, 130, 1000, 5001])
def test_linear_wgrad(rows):
    g = gen(14)
    dy, x = normal(g, rows, 264), normal(g, rows, 136)
    dw, db = ep.linear_wgrad(dy, x, bias_grad=True)
    w64, ew, b64, eb = R.wgrad(dy, x, BF16)
    close(dw, w64, ew)
    close(db, b64, eb)


@pytest.mark.parametrize("act", ACTS[1:])
def test_act_grad(act):
    g = gen(15)
    n, two, counts = 72, 2 if act == "swiglu" else 1, [0, 5, 33]
    dy, z = normal(g, 3, 33, n), normal(g, 3, 33, two * n, std=2.0)
    out = torch.full((3, 33, two * n), 7.0, dtype=BF16, device="cuda")
    ep.act_grad(dy, z, act, counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), out=out)
    whole = ep.act_grad(dy, z, act)
    eye = torch.eye(n, dtype=BF16, device="cuda")
    for e, c in enumerate(counts):
        d, ed = R.dgrad(dy[e], eye, act, z[e], BF16)
        close(whole[e], d, ed)
        close(out[e, :c], d[:c], ed[:c])
        assert (out[e, c:] == 7.0).all()


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """A product, its activation and a second product: directional derivatives of
    sum(c * y) by central differences of the 64-bit forward against the kernels' gradients."""
    g = gen(16)
    m, k, n, o = 37, 72, 40, 56
    wn = 2 * n if act == "swiglu" else n
    x, w1, w2, c = normal(g, m, k), normal(g, wn, k, std=k ** -0.5), normal(g, o, n, std=n ** -0.5), normal(g, m, o)
    b1 = normal(g, wn)
    z = torch.empty(m, wn, dtype=BF16, device="cuda")
    h = ep.linear(x, w1, bias=b1, act=act, preact=z)
    dz = ep.linear_dgrad(c, w2, act=act, preact=None if act == "none" else z)
    dx = ep.linear_dgrad(dz, w1)
    dw1, db1 = ep.linear_wgrad(dz, x, bias_grad=True, out_dtype=F32)
    dw2 = ep.linear_wgrad(c, h, out_dtype=F32)

    def loss(x, w1, b1, w2):
        zz = x @ w1.T + b1
        hh = R.act64(zz[:, :n], "silu")[0] * zz[:, n:] if act == "swiglu" else R.act64(zz, act)[0]
        return float((c.double() * (hh @ w2.T)).sum())

    at = [t.double() for t in (x, w1, b1, w2)]
    for i, grad in enumerate((dx, dw1, db1, dw2)):
        d = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * d, at[i] - step * d
        slope = (loss(*up) - loss(*down)) / (2 * step)
        got = float((grad.double() * d).sum())
        # three bf16 roundings (h or dz, z, the gradient) of independent sign over the sum's terms
        size = float((grad.double() * d).norm())
        assert abs(got - slope) <= 3 * 2.0 ** -8 * 4 * size + 1e-6, (i, got, slope)


def test_runs_on_a_side_stream_and_in_a_graph():
    g = gen(17)
    x, w = normal(g, 4, 90, 136), normal(g, 4, 72, 136, std=0.1)
    cnt = torch.tensor([90, 3, 0, 50], dtype=torch.int32, device="cuda")
    want = ep.experts_product(x, w, cnt, out=torch.zeros(4, 90, 72, dtype=BF16, device="cuda"))
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    ep.experts_product(x, w, cnt, out=out, stream=side)
    fresh = [ep.experts_product(x, w, cnt, stream=side), ep.linear(x, w[0], stream=side),
             *ep.linear_wgrad(x, x, bias_grad=True, stream=side), ep.act_grad(x, x, "relu", stream=side),
             *ep.route_topk(x[0], 2, stream=side)]
    torch.cuda.current_stream().wait_stream(side)
    for t in fresh:
        t.record_stream(torch.cuda.current_stream())
    assert torch.equal(out, want)
    for e, c in enumerate(cnt.tolist()):
        assert torch.equal(fresh[0][e, :c], want[e, :c])
    assert torch.equal(fresh[1], ep.linear(x, w[0]))
    for a, b in zip(fresh[2:], (*ep.linear_wgrad(x, x, bias_grad=True), ep.act_grad(x, x, "relu"), *ep.route_topk(x[0], 2))):
        assert torch.equal(a, b)
    graph, out2 = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        ep.experts_product(x, w, cnt, out=out2)
    cnt.copy_(torch.tensor([1, 90, 17, 0], dtype=torch.int32))
    graph.replay()
    want2 = ep.experts_product(x, w, cnt, out=torch.zeros_like(want))
    assert torch.equal(out2, want2)


def test_results_do_not_change_from_run_to_run():
    g = gen(18)
    dy, x = normal(g, 3000, 264), normal(g, 3000, 392)
    first = ep.linear_wgrad(dy, x, bias_grad=True, out_dtype=F32)
    for _ in range(3):
        again = ep.linear_wgrad(dy, x, bias_grad=True, out_dtype=F32)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refusals():
    x, w = torch.zeros(4, 16, dtype=BF16, device="cuda"), torch.zeros(8, 16, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        ep.linear(x.float(), w)
    with pytest.raises(ValueError):
        ep.linear(x.t(), w)
    with pytest.raises(ValueError):
        ep.linear(x, torch.zeros(8, 24, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        ep.linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        ep.linear(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        ep.linear(x, w, bias=torch.zeros(9, dtype=BF16, device="cuda"))
    with pytest.raises(ep.EpError):      # k not a multiple of 8
        ep.linear(x[:, :12].contiguous(), w[:, :12].contiguous())
    with pytest.raises(ep.EpError):      # 16-byte alignment
        ep.linear(torch.zeros(4 * 16 + 1, dtype=BF16, device="cuda")[1:].view(4, 16), w)
    with pytest.raises(ValueError):
        ep.linear_dgrad(torch.zeros(4, 8, dtype=BF16, device="cuda"), w, act="gelu")
    with pytest.raises(ValueError):
        ep.linear_wgrad(torch.zeros(4, 8, dtype=BF16, device="cuda"), x, accumulate=True)
    with pytest.raises(ValueError):
        ep.experts_product(x[None], w[None], torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ep.experts_product(x[None], w[None], torch.zeros(1, dtype=torch.int64, device="cuda"))


def test_offsets_past_32_bits():
    """An output of over 2^32 elements, its first and last rows."""
    g = gen(40)
    rows, k, n = 140001, 64, 32768
    x, w = normal(g, rows, k), normal(g, n, k, std=0.125)
    y = ep.linear(x, w, act="relu")
    assert y.numel() > 1 << 32
    for at in (slice(0, 40), slice(rows - 40, rows)):
        want, e, _, _ = R.forward(x[at], w, None, "relu", None, BF16)
        close(y[at], want, e)


def test_two_host_threads_on_their_own_streams():
    """Launches of two threads interleave on the GPU; none disturbs the other's results."""
    import threading
    g = gen(41)
    jobs = []
    for E, rows, k, n, act in ((24, 200, 264, 520, "swiglu"), (3, 40, 4104, 136, "none")):
        x, w = normal(g, E, rows, k), normal(g, E, 2 * n if act == "swiglu" else n, k, std=k ** -0.5)
        cnt = torch.randint(0, rows + 1, (E,), generator=g, device="cuda", dtype=torch.int32)
        dy = normal(g, E, rows, n)
        jobs.append((x, w, cnt, dy, act))

    def run(job, stream=None):
        x, w, cnt, dy, act = job
        out = torch.zeros(*dy.shape, dtype=BF16, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        ep.experts_product(x, w, cnt, act=act, out=out, stream=stream)
        dw = ep.experts_product_wgrad(dy, x, cnt, out_dtype=F32, stream=stream)
        y = ep.linear(x[0], w[0], act=act, stream=stream)
        return out, dw, y

    want = [run(j) for j in jobs]
    torch.cuda.synchronize()
    bad = []

    def worker(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(25):
                got = run(jobs[i], s)
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not any(t.is_alive() for t in threads) and not bad
