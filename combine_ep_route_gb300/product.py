"""The layers' matrix products: the experts' (ragged rows per expert, in the
batched-experts layout dispatch writes) and dense ones, with their gradients.

Each call passes tensor pointers and the current stream to ``ep_product``,
``ep_product_dgrad``, ``ep_product_wgrad`` or ``ep_act_grad`` (include/ep.h).
Operands are contiguous bf16; ``k`` and ``n`` are multiples of 8. Nothing is recorded for autograd: an
operand that requires a gradient is refused unless under ``torch.no_grad()``.

The kernels' waits are bounded. One that runs out (the outputs of its call are then invalid) is
reported in the call's ``status`` tensor, or without one in a word of the device that
:func:`check_products` reads.
"""
from __future__ import annotations

import ctypes as C
from math import prod
from typing import Optional, Tuple, Union

import torch

from . import _lib as L
from .ep import _cuda_device, _stream_ptr

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ACTS = {"none": L.EP_ACT_NONE, "relu": L.EP_ACT_RELU, "silu": L.EP_ACT_SILU, "gelu": L.EP_ACT_GELU,
        "gelu_tanh": L.EP_ACT_GELU_TANH, "swiglu": L.EP_ACT_SWIGLU}
INT32_MAX = (1 << 31) - 1
# (the C entry takes every row then, also what dispatch never wrote)
_NO_COUNTS = "counts: want the rows in use per expert, got None"
_OUT = {BF16: L.EP_BF16, F32: L.EP_F32}

# The current stream's handle without a Stream object: building one costs as much as
# the rest of a small call. (device index) -> cudaStream_t
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_of(stream: Optional[torch.cuda.Stream], dev: torch.device) -> int:
    """ep._stream_ptr, by the short way for the current stream."""
    if stream is None and _raw_stream is not None and dev.index == torch.cuda.current_device():
        return _raw_stream(dev.index)
    return _stream_ptr(stream, dev)


def empty(shape: Tuple[int, ...], dtype: torch.dtype, dev: torch.device,
          stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A new result, of the memory of the stream it is written on: another stream's may still be
    in use by what that stream has pending."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _act(act: str) -> int:
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act: want one of {sorted(ACTS)}, got {act!r}")
    return code


def untracked(**tensors: Optional[torch.Tensor]) -> None:
    """Refuses what autograd would record: the result has no ``grad_fn``, so the gradient would be lost
    without a word. (The gradient calls look at the incoming gradient only.)"""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if t is not None and t.requires_grad:
                raise ValueError(f"{name}: requires a gradient, which this call does not record; call it under "
                                 "torch.no_grad() or on a detached tensor (gradients have calls of their own)")


def _want(t: torch.Tensor, name: str, shape: Tuple[int, ...], dev, dtype=BF16) -> None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name}: want contiguous {dtype} {tuple(shape)} on {dev}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")


def _operands(a: torch.Tensor, b: torch.Tensor, names: Tuple[str, str]) -> None:
    dev = a.device
    if (a.dtype is BF16 and b.dtype is BF16 and a.is_cuda and b.device == dev and a.is_contiguous()
            and b.is_contiguous()):
        return
    for t, name in ((a, names[0]), (b, names[1])):
        if t.dtype != BF16 or not t.is_contiguous() or not t.is_cuda or t.device != dev:
            raise ValueError(f"{name}: want contiguous {BF16} on one CUDA device, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")


def _out(out: Optional[torch.Tensor], shape: Tuple[int, ...], dtype: Optional[torch.dtype], dev,
         stream: Optional[torch.cuda.Stream], name: str = "out") -> torch.Tensor:
    if out is None:
        if dtype is not None and dtype not in _OUT:
            raise ValueError(f"{name}: want bfloat16 or float32, got {dtype}")
        return empty(shape, dtype or BF16, dev, stream)
    if dtype is not None and out.dtype != dtype:
        raise ValueError(f"{name}: want {dtype}, got {out.dtype}")
    if out.dtype not in _OUT:
        raise ValueError(f"{name}: want bfloat16 or float32, got {out.dtype}")
    _want(out, name, shape, dev, out.dtype)
    return out


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _args(groups: int, rows: int, k: int, n: int, act: int, out: torch.Tensor,
          counts: Optional[torch.Tensor], status: Optional[torch.Tensor], dev) -> L.EpProductC:
    if counts is not None:
        if (counts.dtype != I32 or counts.numel() != groups or not counts.is_contiguous()
                or counts.device != dev):
            raise ValueError(f"counts: want contiguous int32 of {groups} groups on {dev}, got "
                             f"{counts.dtype} {tuple(counts.shape)} on {counts.device}")
    if status is not None:
        _want(status, "status", (1,), dev, I32)
    return L.EpProductC(groups, rows, k, n, act, _OUT[out.dtype], _ptr(counts), _ptr(status))


def _split(t: torch.Tensor, name: str, grouped: bool) -> Tuple[int, int, int]:
    """(groups, rows, columns) of a row operand; leading dimensions of the experts' form are groups."""
    shape = t.shape
    if len(shape) < (3 if grouped else 2):
        raise ValueError(f"{name}: want {'[groups, rows, columns]' if grouped else '[rows, columns]'}, "
                         f"got {tuple(shape)}")
    if grouped:
        groups, rows = shape[0] if len(shape) == 3 else prod(shape[:-2]), shape[-2]
    else:
        groups, rows = 1, shape[0] if len(shape) == 2 else prod(shape[:-1])
    columns = shape[-1]
    if rows > INT32_MAX or columns > INT32_MAX:   # ctypes would cut them down to 32 bits
        raise ValueError(f"{name}: want at most {INT32_MAX} rows and columns, got {rows} x {columns}")
    return groups, rows, columns


def _weight(w: torch.Tensor, groups: int, grouped: bool) -> Tuple[int, int]:
    """(rows, columns) of one weight."""
    shape = w.shape
    if (len(shape) < 2 or (not grouped and len(shape) != 2)
            or (shape[0] if len(shape) == 3 else prod(shape[:-2])) != groups):
        raise ValueError(f"w: want {groups} weight(s) [rows, columns], got {tuple(shape)}")
    rows, columns = shape[-2], shape[-1]
    if rows > INT32_MAX or columns > INT32_MAX:
        raise ValueError(f"w: want at most {INT32_MAX} rows and columns, got {rows} x {columns}")
    return rows, columns


def _forward(x, w, counts, grouped, bias, act, residual, out, out_dtype, preact, status, stream):
    if grouped and counts is None:
        raise ValueError(_NO_COUNTS)
    _operands(x, w, ("x", "w"))
    if (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad)
            or (residual is not None and residual.requires_grad)):
        untracked(x=x, w=w, bias=bias, residual=residual)
    dev, code = x.device, _act(act)
    groups, rows, k = _split(x, "x", grouped)
    wn, wk = _weight(w, groups, grouped)
    if wk != k or (code == L.EP_ACT_SWIGLU and wn % 2):
        raise ValueError(f"w: {tuple(w.shape)} does not fit x {tuple(x.shape)} with act {act!r}")
    n = wn // 2 if code == L.EP_ACT_SWIGLU else wn
    lead = x.shape[:-1]
    out = _out(out, lead + (n,), out_dtype, dev, stream)
    if bias is not None:
        _want(bias, "bias", w.shape[:-1], dev)
    if residual is not None:
        _want(residual, "residual", lead + (n,), dev)
    if preact is not None:
        _want(preact, "preact", lead + (wn,), dev)
    a = _args(groups, rows, k, n, code, out, counts, status, dev)
    L.check(L.lib().ep_product(C.byref(a), x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual),
                               out.data_ptr(), _ptr(preact), stream_of(stream, dev)), "ep_product")
    return out


def _dgrad(dy, w, counts, grouped, act, preact, out, out_dtype, status, stream):
    if grouped and counts is None:
        raise ValueError(_NO_COUNTS)
    _operands(dy, w, ("dy", "w"))
    if dy.requires_grad:
        untracked(dy=dy)
    dev, code = dy.device, _act(act)
    groups, rows, n = _split(dy, "dy", grouped)
    wn, k = _weight(w, groups, grouped)
    if wn != n:
        raise ValueError(f"w: {tuple(w.shape)} does not fit dy {tuple(dy.shape)}")
    shape = dy.shape[:-1] + (2 * k if code == L.EP_ACT_SWIGLU else k,)
    if (preact is None) != (code == L.EP_ACT_NONE):
        raise ValueError("preact: wanted with an activation, and only then")
    if preact is not None:
        _want(preact, "preact", shape, dev)
    out = _out(out, shape, out_dtype, dev, stream)
    a = _args(groups, rows, k, n, code, out, counts, status, dev)
    L.check(L.lib().ep_product_dgrad(C.byref(a), dy.data_ptr(), w.data_ptr(), _ptr(preact), out.data_ptr(),
                                     stream_of(stream, dev)), "ep_product_dgrad")
    return out


def _wgrad(dy, x, counts, grouped, out, out_dtype, accumulate, bias_grad, status, stream):
    if grouped and counts is None:
        raise ValueError(_NO_COUNTS)
    _operands(dy, x, ("dy", "x"))
    if dy.requires_grad:
        untracked(dy=dy)
    dev = dy.device
    groups, rows, n = _split(dy, "dy", grouped)
    gx, rx, k = _split(x, "x", grouped)
    if (gx, rx) != (groups, rows):
        raise ValueError(f"x: {tuple(x.shape)} does not fit dy {tuple(dy.shape)}")
    lead = dy.shape[:-2] if grouped else ()
    if accumulate and out is None:
        raise ValueError("out: wanted with accumulate")
    out = _out(out, lead + (n, k), out_dtype, dev, stream)
    db = None
    if isinstance(bias_grad, torch.Tensor):
        db = _out(bias_grad, lead + (n,), out.dtype, dev, stream, "bias_grad")
    elif bias_grad:
        if accumulate:
            raise ValueError("bias_grad: want a tensor to add to with accumulate")
        db = empty(lead + (n,), out.dtype, dev, stream)
    a = _args(groups, rows, k, n, L.EP_ACT_NONE, out, counts, status, dev)
    L.check(L.lib().ep_product_wgrad(C.byref(a), dy.data_ptr(), x.data_ptr(), 1 if accumulate else 0,
                                     out.data_ptr(), _ptr(db), stream_of(stream, dev)), "ep_product_wgrad")
    return out if db is None else (out, db)


Grad = Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]


# ------------------------------------------------------------------ the experts

def experts_product(x: torch.Tensor, w: torch.Tensor, counts: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                    act: str = "none", residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    out_dtype: Optional[torch.dtype] = None, preact: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``act(x[e] @ w[e]^T + bias[e]) + residual[e]`` on each expert's first ``counts[e]`` rows.

    ``x`` ``[..., E, rows, k]`` (dispatch's ``b_a1`` as it is), ``w`` ``[..., E, n, k]`` (``swiglu``:
    ``[..., E, 2n, k]``, gate rows first), ``counts`` int32 on the device (``expert_num_tokens``).
    Rows past the counts are not written. ``preact`` receives the pre-activation for the backward pass.
    """
    return _forward(x, w, counts, True, bias, act, residual, out, out_dtype, preact, status, stream)


def experts_product_dgrad(dy: torch.Tensor, w: torch.Tensor, counts: torch.Tensor, *, act: str = "none",
                          preact: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          out_dtype: Optional[torch.dtype] = None, status: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``(dy[e] @ w[e]) * act'(preact[e])`` on the rows in use: the gradient of the product's input,
    taken on through the activation that made it (``act`` "none": the input's own)."""
    return _dgrad(dy, w, counts, True, act, preact, out, out_dtype, status, stream)


def experts_product_wgrad(dy: torch.Tensor, x: torch.Tensor, counts: torch.Tensor, *,
                          out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                          accumulate: bool = False, bias_grad: Union[bool, torch.Tensor] = False,
                          status: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> Grad:
    """``dy[e]^T @ x[e]`` over the rows in use (zeros for an idle expert), added to ``out`` with
    ``accumulate``; with ``bias_grad`` also the sums of ``dy``'s rows."""
    return _wgrad(dy, x, counts, True, out, out_dtype, accumulate, bias_grad, status, stream)


# ----------------------------------------------------------------------- linear

def linear(x: torch.Tensor, w: torch.Tensor, *, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           out_dtype: Optional[torch.dtype] = None, preact: Optional[torch.Tensor] = None,
           status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``act(x @ w^T + bias) + residual`` for ``x`` ``[..., k]`` and ``w`` ``[n, k]`` (``swiglu``: ``[2n, k]``).

    ``n`` and ``k`` are multiples of 8. A router for another number of experts keeps its weight padded with
    zero rows and a ``bias`` of minus infinity there: such logits are never chosen and have no gradient.
    """
    return _forward(x, w, None, False, bias, act, residual, out, out_dtype, preact, status, stream)


def linear_dgrad(dy: torch.Tensor, w: torch.Tensor, *, act: str = "none", preact: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                 status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``(dy @ w) * act'(preact)``; see :func:`experts_product_dgrad`."""
    return _dgrad(dy, w, None, False, act, preact, out, out_dtype, status, stream)


def linear_wgrad(dy: torch.Tensor, x: torch.Tensor, *, out: Optional[torch.Tensor] = None,
                 out_dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                 bias_grad: Union[bool, torch.Tensor] = False, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Grad:
    """``dy^T @ x`` and, with ``bias_grad``, the sum of ``dy``'s rows; see :func:`experts_product_wgrad`."""
    return _wgrad(dy, x, None, False, out, out_dtype, accumulate, bias_grad, status, stream)


def act_grad(dy: torch.Tensor, preact: torch.Tensor, act: str, *, counts: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``dy * act'(preact)``, for an activation that no product follows. With ``counts``, ``dy`` is
    ``[..., E, rows, n]`` and only the rows in use are written."""
    _operands(dy, preact, ("dy", "preact"))
    if dy.requires_grad:
        untracked(dy=dy)
    dev, code = dy.device, _act(act)
    if code == L.EP_ACT_NONE:
        raise ValueError("act: want an activation")
    groups, rows, n = _split(dy, "dy", counts is not None)
    shape = dy.shape[:-1] + (2 * n if code == L.EP_ACT_SWIGLU else n,)
    _want(preact, "preact", shape, dev)
    out = _out(out, shape, BF16, dev, stream)
    a = _args(groups, rows, n, n, code, out, counts, None, dev)
    L.check(L.lib().ep_act_grad(C.byref(a), dy.data_ptr(), preact.data_ptr(), out.data_ptr(),
                                stream_of(stream, dev)), "ep_act_grad")
    return out


# ----------------------------------------------------------------------- status

def product_status(device: Optional[torch.device] = None, stream: Optional[torch.cuda.Stream] = None) -> int:
    """Wait for ``stream`` (the current one) and return the status code (0 = ok) of the products on
    ``device`` that were given no ``status`` tensor; clears it."""
    dev = _cuda_device(device)
    with torch.cuda.device(dev):
        return int(L.lib().ep_product_status(_stream_ptr(stream, dev)))


def check_products(device: Optional[torch.device] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Raise what :func:`product_status` returns."""
    L.check(product_status(device, stream), "device status of the products")


def set_product_wait_limit(ns: int) -> None:
    """The bound of every device-side wait of later products, 1000..60e9 ns (default 2e9)."""
    L.check(L.lib().ep_product_wait_limit(int(ns)), "ep_product_wait_limit")
