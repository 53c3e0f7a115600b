"""4-bit weights on the host: the packed layout, the codes' values, quantisation, and the refusals
of the products, which come before any GPU work."""
import ctypes as C

import pytest
import torch

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L

P = 0x7F0000000000      # an aligned address; never dereferenced by these tests
BF16 = torch.bfloat16
FP4 = [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]


@pytest.fixture(scope="module")
def lib():
    from combine_ep_route_gb300 import build
    build.build()
    return L.lib()


def test_fields_of_a_word():
    codes = torch.arange(32).remainder(16)[None].repeat(3, 1)
    packed, scales = ep.pack_weight4(codes, torch.ones(3, 1))
    assert packed.shape == (3, 16) and scales.shape == (1, 3) and packed.dtype == torch.uint8
    word = int.from_bytes(bytes(packed[0, :4].tolist()), "little")
    assert [(word >> (4 * i)) & 15 for i in range(8)] == [0, 2, 4, 6, 1, 3, 5, 7]
    word = int.from_bytes(bytes(packed[0, 4:8].tolist()), "little")
    assert [(word >> (4 * i)) & 15 for i in range(8)] == [8, 10, 12, 14, 9, 11, 13, 15]


@pytest.mark.parametrize("kind", ("int4", "fp4"))
@pytest.mark.parametrize("group", (32, 64, 128))
def test_values_of_codes(kind, group):
    g = torch.Generator().manual_seed(group)
    codes = torch.randint(0, 16, (2, 5, 256), generator=g)
    scales = torch.randn(2, 5, 256 // group, generator=g).to(BF16)
    w = ep.dequantize_weight4(*ep.pack_weight4(codes, scales), kind)
    table = torch.tensor([i if i < 8 else i - 16 for i in range(16)] if kind == "int4" else FP4)
    want = (table.double()[codes] * scales.double().repeat_interleave(group, -1)).to(BF16)
    assert w.dtype == BF16 and torch.equal(w, want)
    signed = torch.where(codes > 7, codes - 16, codes).to(torch.int8)     # codes as signed numbers are the same codes
    assert all(torch.equal(a, b) for a, b in zip(ep.pack_weight4(signed, scales), ep.pack_weight4(codes, scales)))


@pytest.mark.parametrize("kind,step", (("int4", 0.5), ("fp4", 1.0)))
@pytest.mark.parametrize("shape", ((8, 64), (2, 3, 8, 128)))
def test_quantisation_takes_the_nearest_code(kind, step, shape):
    w = torch.randn(*shape, generator=torch.Generator().manual_seed(1)) * 3
    w[..., 0, :32] = 0
    codes, scales = ep.quantize_weight4(w, 32, kind)
    assert codes.shape == shape[:-1] + (shape[-1] // 2,) and scales.shape == shape[:-2] + (shape[-1] // 32, shape[-2])
    back = ep.dequantize_weight4(codes, scales, kind).double()
    s = scales.double().transpose(-1, -2).repeat_interleave(32, -1)
    # half the widest step between codes, the scale's rounding of the largest, the weight's own rounding
    assert ((back - w.double()).abs() <= s * step + back.abs() * (2.0 ** -8 + 2.0 ** -8)).all()
    assert (back[..., 0, :32] == 0).all()


def test_bad_weights_are_refused():
    codes, scales = torch.zeros(8, 64, dtype=torch.int8), torch.ones(8, 2)
    for call in (lambda: ep.pack_weight4(codes.float(), scales), lambda: ep.pack_weight4(codes[:, :48], scales),
                 lambda: ep.pack_weight4(codes, scales[:4]), lambda: ep.pack_weight4(codes, torch.ones(8, 3)),
                 lambda: ep.pack_weight4(codes, torch.ones(8, 64)), lambda: ep.pack_weight4(codes[0], scales[0]),
                 lambda: ep.quantize_weight4(codes, 32), lambda: ep.quantize_weight4(codes.float(), 16),
                 lambda: ep.quantize_weight4(codes.float(), 128), lambda: ep.quantize_weight4(codes.float(), 32, "int3"),
                 lambda: ep.dequantize_weight4(*ep.pack_weight4(codes, scales), "nf4")):
        with pytest.raises(ValueError):
            call()


def args(groups=4, rows=16, k=64, n=32, act=0, kind=0, group=32, counts=P, status=None):
    return C.byref(L.EpW4C(groups, rows, k, n, act, kind, group, counts, status))


@pytest.mark.parametrize("bad", [dict(groups=0), dict(groups=1025), dict(rows=-1), dict(k=0), dict(k=48), dict(k=96, group=64),
                                 dict(k=L.EP_W4_MAX_K + 32), dict(n=4), dict(n=20), dict(n=(1 << 24) + 8), dict(act=-1),
                                 dict(act=6), dict(kind=2), dict(kind=-1), dict(group=16), dict(group=48), dict(group=256, k=256),
                                 dict(groups=1024, rows=1 << 21), dict(groups=1, rows=(1 << 31) - 1, k=32768),
                                 dict(counts=P + 2), dict(status=P + 1)])
def test_bad_products_are_refused(lib, bad):
    assert lib.ep_product_w4(args(**bad), P, P, P, None, None, P, None) == L.EP_ERR_INVALID_ARG


def test_missing_and_misaligned_buffers_are_refused(lib):
    for at in range(6):
        for v in ([P + 8] if at in (3, 4) else [None, P + 8]):
            given = [P, P, P, None, None, P]
            given[at] = v
            assert lib.ep_product_w4(args(), *given, None) == L.EP_ERR_INVALID_ARG
    assert lib.ep_product_w4(None, P, P, P, None, None, P, None) == L.EP_ERR_INVALID_ARG
    assert lib.ep_product_w4(args(rows=0), None, None, None, None, None, None, None) == L.EP_OK


def test_host_tensors_and_bad_calls_are_refused():
    x = torch.zeros(4, 64, dtype=BF16)
    codes, scales = ep.pack_weight4(torch.zeros(8, 64, dtype=torch.int8), torch.ones(8, 2))
    cnt = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: ep.linear_w4(x, codes, scales), lambda: ep.linear_w4(x, codes, scales, kind="int3"),
                 lambda: ep.linear_w4(x, codes, scales, act="tanh"),
                 lambda: ep.experts_product_w4(x[None], codes[None], scales[None], cnt),
                 lambda: ep.experts_product_w4(x[None], codes[None], scales[None], None)):
        with pytest.raises(ValueError):
            call()
