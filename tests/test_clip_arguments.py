"""The gradient norm's refusals on the host: they come before any GPU work."""
import ctypes as C

import pytest
import torch

import combine_ep_route_gb300 as ep
from combine_ep_route_gb300 import _lib as L

P = 0x7F0000000000      # an aligned address; never dereferenced by these tests
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    from combine_ep_route_gb300 import build
    build.build()
    return L.lib()


def grads(spans, out=None, dtypes=None, keep=[]):
    """A list of tensors given as (address, elements); float32 unless said."""
    n = len(spans)
    arrays = [(C.c_void_p * n)(*[s[0] for s in spans]), (C.c_int64 * n)(*[s[1] for s in spans]),
              (C.c_int32 * n)(*(dtypes or [L.EP_F32] * n))]
    if out is not None:
        arrays.append((C.c_void_p * n)(*out))
    keep.append(arrays)
    at = [C.addressof(x) for x in arrays]
    return C.byref(L.EpGradsC(n, at[0], at[3] if out is not None else None, at[1], at[2]))


def call(lib, a, max_norm=1.0, norm=P + (1 << 40), work=P + (1 << 41), size=1 << 20):
    return lib.ep_clip_grad_norm(a, max_norm, norm, work, size, None)


def test_bad_lists_are_refused(lib):
    inv, size = L.EP_ERR_INVALID_ARG, C.c_size_t()
    for bad in (grads([(P, -1)]), grads([(P, 1 << 44)]), grads([(P, 4)], dtypes=[3]), None,
                C.byref(L.EpGradsC(-1, None, None, None, None)), C.byref(L.EpGradsC(2, None, None, None, None))):
        assert lib.ep_clip_workspace_bytes(bad, C.byref(size)) == inv
        assert call(lib, bad) == inv
    assert lib.ep_clip_workspace_bytes(grads([(P, 4)]), None) == inv
    for bad in (grads([(None, 4)]), grads([(P + 2, 4)]), grads([(P + 1, 4)], dtypes=[L.EP_BF16]),
                grads([(P, 4)], out=[None]), grads([(P, 4)], out=[P + 18])):
        assert lib.ep_clip_workspace_bytes(bad, C.byref(size)) == L.EP_OK and size.value >= 8
        assert call(lib, bad) == inv
    good = grads([(P, 4)])
    for max_norm in (-1.0, float("nan"), -INF):
        assert call(lib, good, max_norm=max_norm) == inv
    assert call(lib, good, norm=None) == inv and call(lib, good, norm=P + 2) == inv
    for work, size in ((None, 1 << 20), (P + 8, 1 << 20), (P, 7)):
        assert call(lib, good, work=work, size=size) == L.EP_ERR_WORKSPACE


@pytest.mark.parametrize("spans,out", [
    ([(P, 8), (P, 8)], None), ([(P, 8), (P + 28, 8)], None), ([(P + 28, 8), (P, 8)], None),
    ([(P, 100), (P + 16, 1), (P + 4096, 8)], None), ([(P, 8)], [P + 16]), ([(P + 16, 8)], [P]),
    ([(P, 8), (P + 4096, 8)], [P + 8192, P + 8192]), ([(P, 8), (P + 4096, 8)], [P + 4096, P]),
    ([(P, 8), (P, 8)], [P, P + 8192])])
def test_overlapping_tensors_are_refused(lib, spans, out):
    assert call(lib, grads(spans, out)) == L.EP_ERR_INVALID_ARG


def test_host_tensors_and_bad_calls_are_refused():
    t = torch.zeros(4)
    for bad in (lambda: ep.clip_grad_norm([t], 1.0), lambda: ep.clip_grad_norm([], 1.0),
                lambda: ep.clip_grad_norm([t], -1.0), lambda: ep.clip_grad_norm([t], float("nan")),
                lambda: ep.clip_grad_norm([t], 1.0, out=[])):
        with pytest.raises(ValueError):
            bad()
