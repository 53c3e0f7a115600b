"""The bounded wait of the 4-bit products' kernel for few rows: one that runs out is reported, its CTAs leave
together, and calls after it are right. A limit of 1 us is kept by polling, and is exceeded by far:
  one row of 65536 x 7168, held whole (which goes to that kernel whatever its size): three CTAs an SM bring 58 KB
    each at a time, 26 MB, 3.9 us at the copy's rate;
  one row of 7168 x 32768 with counts, in chunks: 448 CTAs with three chunks of 21 KB each on their way, 29 MB,
    4.2 us until all have the last of them.
L2 is overwritten before the calls, so that the codes come from memory. Every wait ends by itself."""
import pytest
import torch
from torch.profiler import ProfilerActivity, profile

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L
from tests import _layers64 as R
from tests.test_gpu_w4 import built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
# kind, group, activation, columns of x, rows of the weight, with counts
FORMS = [("int4", 128, "none", 7168, 65536, False), ("fp4", 32, "swiglu", 7168, 65536, False),
         ("int4", 64, "none", 32768, 7168, True), ("fp4", 128, "swiglu", 32768, 7168, True)]


@pytest.fixture
def short_limit():
    ep.product_status()
    ep.set_product_wait_limit(1000)
    yield
    ep.set_product_wait_limit(2_000_000_000)


class Call:
    def __init__(self, kind, group, act, k, wide, counted):
        g = torch.Generator(device="cuda").manual_seed(group)
        self.x = torch.randn(1, 1, k, generator=g, device="cuda").to(BF16)
        self.codes = torch.randint(0, 256, (1, wide, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = torch.full((1, k // group, wide), 2.0 ** -9, device="cuda", dtype=BF16)
        self.kw, self.counted = dict(kind=kind, act=act), counted
        self.counts = torch.ones(1, dtype=I32, device="cuda")
        torch.zeros(512 << 20, dtype=torch.uint8, device="cuda")

    def __call__(self, **kw):
        if self.counted:
            return ep.experts_product_w4(self.x, self.codes, self.scales, self.counts, **self.kw, **kw)[0]
        return ep.linear_w4(self.x[0], self.codes[0], self.scales[0], **self.kw, **kw)


@pytest.mark.parametrize("form", FORMS)
def test_the_call_goes_to_the_kernel_for_few_rows(form):
    call = Call(*form)

    def names():
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            call.x + 1
            call()
            torch.cuda.synchronize()
        return [e.key for e in p.key_averages()]

    names()                         # (the profiler's first use may record nothing)
    seen = names()
    if not any("elementwise" in n for n in seen):
        pytest.skip("the profiler sees no launches here")
    assert any("w4_rows_kernel" in n for n in seen) and not any("w4_tiles_kernel" in n for n in seen)


@pytest.mark.parametrize("form", FORMS)
def test_a_wait_that_runs_out_is_reported(short_limit, form):
    call = Call(*form)
    call()
    with pytest.raises(ep.EpError) as e:
        ep.check_products()
    assert e.value.code == L.EP_ERR_TIMEOUT
    ep.check_products()                     # taken
    status = torch.zeros(1, dtype=I32, device="cuda")
    call = Call(*form)
    call(status=status)
    assert status.item() == L.EP_ERR_TIMEOUT and ep.product_status() == 0


@pytest.mark.parametrize("form", FORMS)
def test_calls_after_it_are_right(form):
    call = Call(*form)
    ep.set_product_wait_limit(1000)
    call()
    ep.set_product_wait_limit(2_000_000_000)
    assert ep.product_status() == L.EP_ERR_TIMEOUT
    y = call()
    ep.check_products()
    w = ep.dequantize_weight4(call.codes[0], call.scales[0], form[0])
    want, off, _, _ = R.forward(call.x[0], w, None, form[2], None, BF16)
    assert ((y.double() - want).abs() <= off).all()
