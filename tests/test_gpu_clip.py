"""The global gradient norm and clipping against 64 bits.

Error bounds. A vector's squares are a chain of 8 roundings, a thread's vectors of a piece at
most 9 more; pieces are summed with their roundings kept, threads and CTAs in 64 bits: 17 2^-24
of the sum, half of that in its root, and the root's own rounding: 2^-20. A clipped value adds
the factor's rounding and its own."""
import math

import pytest
import torch

import combine_ep_route_gb300 as ep

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
TOL = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def tensors(sizes, seed=1, std=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * std).to(BF16 if i % 2 else F32) for i, s in enumerate(sizes)]


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check(ts, max_norm, out=None):
    """In place unless out is given; returns the norm."""
    before = [t.clone() for t in ts]
    want = norm64(before)
    got = ep.clip_grad_norm(ts, max_norm, out=out)
    assert got.shape == () and got.dtype == F32
    assert abs(float(got) - want) <= TOL * want + 1e-45
    factor = max_norm / want if want > max_norm else 1.0
    for b, t, o in zip(before, ts, ts if out is None else out):
        if out is not None:
            assert torch.equal(b, t)
        if factor == 1.0:
            assert torch.equal(o, b)
        else:
            exact = b.double() * factor
            # (below the smallest normal number half its step, 2^-134 at most)
            off = exact.abs() * (2 * TOL + (2.0 ** -8 if b.dtype is BF16 else 2.0 ** -24)) + 2.0 ** -133
            assert ((o.double() - exact).abs() <= off).all()
    return got


SIZES = [[1], [7, 8, 9], [16384, 16385, 16383, 1, 0, 5], [100003, 3, 1 << 20, 77], [0, 0, 4], list(range(1, 40)),
         [40000] * 130, [31] * 513, [5] * 1300]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("share", (0.25, 4.0))
@pytest.mark.parametrize("inplace", (True, False))
def test_norm_and_clipping(sizes, share, inplace):
    ts = tensors(sizes)
    out = None if inplace else [torch.full_like(t, NAN) for t in ts]
    check(ts, norm64(ts) * share, out)


def test_no_bound_gives_the_norm_alone():
    ts = tensors([1000, 12345, 3])
    check(ts, INF)
    check(ts, INF, [torch.empty_like(t) for t in ts])
    check([torch.zeros(50, device="cuda")], 1.0)
    check([torch.zeros(50, device="cuda")], 0.0)
    check([torch.empty(0, device="cuda")], 1.0)
    ts = tensors([1000, 12345, 3])
    check(ts, 0.0)
    assert all((t == 0).all() for t in ts)


@pytest.mark.parametrize("scale", (1e-30, 1e-22, 1e-12, 1e14, 1e18, 1e30))
def test_squares_neither_overflow_nor_underflow(scale):
    ts = [t * scale for t in tensors([5000, 4001, 9], std=1.0)]
    check(ts, 0.5 * norm64(ts))
    mixed = tensors([3000, 20], std=1.0) + [t * scale for t in tensors([70, 4001], std=1.0)]
    check(mixed, 2 * norm64(mixed))
    check(mixed, 0.5 * norm64(mixed))


def test_a_norm_past_the_largest_float():
    ts = [torch.full((100,), 3e38, device="cuda")]
    got = ep.clip_grad_norm(ts, 1.0)
    assert float(got) == INF and ((ts[0] - 0.1).abs() < 1e-6).all()     # 3e39 as a float; the gradients are finite


@pytest.mark.parametrize("bad", (INF, -INF, NAN))
@pytest.mark.parametrize("at", (0, 7, 4096, 5006))
@pytest.mark.parametrize("dtype", (BF16, F32))
@pytest.mark.parametrize("rest", (0.0, 1.0))
def test_a_norm_that_is_not_finite_changes_nothing(bad, at, dtype, rest):
    ts = [torch.full((5007,), rest, device="cuda", dtype=dtype), torch.ones(4, device="cuda")]
    ts[0][at] = bad
    before = [t.clone() for t in ts]
    out = [torch.zeros_like(t) for t in ts]
    got = ep.clip_grad_norm(ts, 1.0, out=out)
    assert (torch.isnan(got) if bad != bad else got == INF)
    assert torch.equal(ep.clip_grad_norm(ts, 1.0).isnan(), got.isnan())
    for b, t, o in zip(before, ts, out):
        assert torch.equal(b.nan_to_num(5.0, 6.0, 7.0), t.nan_to_num(5.0, 6.0, 7.0))
        assert torch.equal(b.nan_to_num(5.0, 6.0, 7.0), o.nan_to_num(5.0, 6.0, 7.0))


@pytest.mark.parametrize("dtype", (BF16, F32))
def test_odd_addresses_and_what_lies_around(dtype):
    size = torch.empty(0, dtype=dtype).element_size()
    flat, to = torch.randn(70000, device="cuda").to(dtype), torch.full((70000,), 3.0, device="cuda", dtype=dtype)
    spans = [(1, 5), (6, 33), (40, 1), (43, 20001), (20050, 16 // size), (20071, 40000)]
    ts, outs = [flat[a:a + n] for a, n in spans], [to[a:a + n] for a, n in spans]
    shifted = [to[a + 3:a + 3 + n] for a, n in spans[3:4]]
    rest = torch.ones(70000, dtype=torch.bool, device="cuda")
    for a, n in spans:
        rest[a:a + n] = False
    check(ts, 0.1 * norm64(ts), outs)
    assert (to[rest] == 3.0).all()
    check(ts[3:4], 0.1 * norm64(ts[3:4]), shifted)
    kept = flat[rest].clone()
    check(ts, 0.1 * norm64(ts))
    assert torch.equal(flat[rest], kept)


def test_same_bits_each_time_on_any_stream_and_in_a_graph():
    ts = tensors([200001, 3, 70000, 9, 500000])
    outs = [torch.empty_like(t) for t in ts]
    first = ep.clip_grad_norm(ts, 0.01, out=outs)
    kept = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = ep.clip_grad_norm(ts, 0.01, out=outs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, again) and all(torch.equal(a, b) for a, b in zip(kept, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = ep.clip_grad_norm(ts, 0.01, out=outs)
    fresh = tensors([200001, 3, 70000, 9, 500000], seed=2)
    for t, f in zip(ts, fresh):
        t.copy_(f)
    graph.replay()
    torch.cuda.synchronize()
    want = [torch.empty_like(t) for t in ts]
    assert torch.equal(norm, ep.clip_grad_norm(ts, 0.01, out=want))
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_refusals():
    a, b = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda", dtype=BF16)
    for call in (lambda: ep.clip_grad_norm([a.double()], 1.0), lambda: ep.clip_grad_norm([a.view(2, 4).t()], 1.0),
                 lambda: ep.clip_grad_norm([a, torch.zeros(3)], 1.0), lambda: ep.clip_grad_norm([a], 1.0, out=[b]),
                 lambda: ep.clip_grad_norm([a], 1.0, out=[a[:4]]), lambda: ep.clip_grad_norm([a, b], 1.0, out=[a]),
                 lambda: ep.clip_grad_norm([a, a], 1.0), lambda: ep.clip_grad_norm([a, a[2:]], 1.0),
                 lambda: ep.clip_grad_norm([torch.zeros(4, device="cuda", requires_grad=True)], 1.0)):
        with pytest.raises((ValueError, ep.EpError)):
            call()
    w = torch.zeros(4, device="cuda", requires_grad=True)
    with torch.no_grad():
        ep.clip_grad_norm([w], 1.0)
