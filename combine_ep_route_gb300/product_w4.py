"""Products with 4-bit weights and group scales: the experts' and dense ones of ``product.py`` for serving
(``ep_product_w4`` in include/ep.h), and the packing of weights for them.

A weight ``[..., n, k]`` is two tensors: ``codes`` uint8 ``[..., n, k / 2]``, and ``scales`` bf16
``[..., k / group, n]`` with a scale for each ``group`` (32, 64 or 128) consecutive elements of a row. Its
elements are ``bf16(value * scale)`` with a code's value of ``kind`` "int4" (two's complement, -8..7) or "fp4"
(sign, two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6). :func:`pack_weight4` lays out
codes and scales of a checkpoint, :func:`quantize_weight4` makes them from a weight; both run once, on any device.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Tuple

import torch

from . import _lib as L
from .product import BF16, I32, _NO_COUNTS, _act, _out, _ptr, _split, _want, _weight, stream_of, untracked

U8 = torch.uint8
KINDS = {"int4": L.EP_W4_INT4, "fp4": L.EP_W4_FP4}
GROUPS = (32, 64, 128)
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# the element that each 4-bit field of a word holds, lowest field first
_FIELDS = (0, 2, 4, 6, 1, 3, 5, 7)


def _kind(kind: str) -> int:
    code = KINDS.get(kind)
    if code is None:
        raise ValueError(f"kind: want one of {sorted(KINDS)}, got {kind!r}")
    return code


def _group(k: int, scales: torch.Tensor, axis: int) -> int:
    """Elements that share a scale, from the scales' extent along k."""
    parts = scales.shape[axis]
    if parts < 1 or k // parts not in GROUPS or k % parts:
        raise ValueError(f"scales: want one for each {', '.join(map(str, GROUPS))} of {k} elements, got {tuple(scales.shape)}")
    return k // parts


# ------------------------------------------------------- weights, once per model

def pack_weight4(codes: torch.Tensor, scales: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """The layout that the products read: ``codes`` of any integer type ``[..., n, k]`` (a code in the low four
    bits: 0..15, or -8..7 of an int8 tensor) and ``scales`` ``[..., n, k / group]`` as a checkpoint has them, rounded to
    bf16 (an fp16 scale loses up to three bits, 2^-8 of itself and of its weights). Codes have no zero point."""
    if codes.dim() < 2 or codes.is_floating_point() or codes.shape[-1] % 32 or codes.shape[-1] == 0:
        raise ValueError(f"codes: want integers [..., n, k] with k a multiple of 32, got {codes.dtype} {tuple(codes.shape)}")
    if scales.shape[:-1] != codes.shape[:-1]:
        raise ValueError(f"scales: want [..., n, k / group] for codes {tuple(codes.shape)}, got {tuple(scales.shape)}")
    _group(codes.shape[-1], scales, -1)
    words = (codes & 15).to(U8).reshape(*codes.shape[:-1], -1, 8)[..., list(_FIELDS)]
    packed = words[..., 0::2] | (words[..., 1::2] << 4)
    return packed.reshape(*codes.shape[:-1], codes.shape[-1] // 2).contiguous(), \
        scales.to(BF16).transpose(-1, -2).contiguous()


def _codes_of(packed: torch.Tensor) -> torch.Tensor:
    """Codes 0..15 ``[..., n, k]`` of a packed weight."""
    fields = torch.stack((packed & 15, packed >> 4), dim=-1).reshape(*packed.shape[:-1], -1, 8)
    order = [_FIELDS.index(e) for e in range(8)]
    return fields[..., order].reshape(*packed.shape[:-1], 2 * packed.shape[-1])


def dequantize_weight4(codes: torch.Tensor, scales: torch.Tensor, kind: str = "int4") -> torch.Tensor:
    """The bf16 weight ``[..., n, k]`` that a packed one stands for, exactly as the products use it."""
    code, k = _kind(kind), 2 * codes.shape[-1]
    group = _group(k, scales, -2)
    c = _codes_of(codes).int()
    if code == L.EP_W4_INT4:
        q = ((c ^ 8) - 8).float()
    else:
        q = torch.tensor(FP4_VALUES + tuple(-v for v in FP4_VALUES), device=c.device)[c]
    s = scales.float().transpose(-1, -2)
    return (q.unflatten(-1, (-1, group)) * s.unsqueeze(-1)).flatten(-2).to(BF16)


def quantize_weight4(w: torch.Tensor, group: int = 32, kind: str = "int4") -> Tuple[torch.Tensor, torch.Tensor]:
    """``(codes, scales)`` of a floating weight ``[..., n, k]``, packed: each group's largest magnitude becomes the
    largest code (7, or 6 in fp4), every element the nearest code's value times the scale."""
    code = _kind(kind)
    if group not in GROUPS or w.dim() < 2 or not w.is_floating_point() or w.shape[-1] % group or w.shape[-1] == 0:
        raise ValueError(f"w: want floating [..., n, k] with k a multiple of the group ({GROUPS}), got {w.dtype} "
                         f"{tuple(w.shape)} and {group}")
    if w.dim() > 2:   # one weight at a time: the steps in between take several times its size
        flat = w.flatten(0, -3)
        if not len(flat):
            raise ValueError("w: want one weight at least")
        codes, scales = zip(*(quantize_weight4(x, group, kind) for x in flat))
        return torch.stack(codes).unflatten(0, w.shape[:-2]), torch.stack(scales).unflatten(0, w.shape[:-2])
    v = w.detach().float().unflatten(-1, (-1, group))
    scales = (v.abs().amax(-1) / (7.0 if code == L.EP_W4_INT4 else 6.0)).to(BF16)
    s = scales.float().unsqueeze(-1)
    ratio = torch.where(s > 0, v / s, torch.zeros_like(v)).flatten(-2)
    if code == L.EP_W4_INT4:
        codes = ratio.round().clamp(-8, 7).to(torch.int8)
    else:
        values = torch.tensor(FP4_VALUES, device=w.device)
        codes = torch.bucketize(ratio.abs(), (values[1:] + values[:-1]) / 2).to(torch.int8)
        codes = codes + 8 * (ratio < 0).to(torch.int8)
    return pack_weight4(codes, scales)


# ----------------------------------------------------------------- the products

def _forward(x, codes, scales, counts, grouped, kind, bias, act, residual, out, status, stream):
    if grouped and counts is None:
        raise ValueError(_NO_COUNTS)
    kind, code, dev = _kind(kind), _act(act), x.device
    if x.dtype is not BF16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError(f"x: want contiguous {BF16} on a CUDA device, got {x.dtype} {tuple(x.shape)} on {x.device} "
                         f"(contiguous={x.is_contiguous()})")
    if (x.requires_grad or scales.requires_grad or (bias is not None and bias.requires_grad)
            or (residual is not None and residual.requires_grad)):
        untracked(x=x, scales=scales, bias=bias, residual=residual)
    groups, rows, k = _split(x, "x", grouped)
    wn, half = _weight(codes, groups, grouped)
    n = wn // 2 if code == L.EP_ACT_SWIGLU else wn
    if (2 * half != k or k % 32 or not 32 <= k <= L.EP_W4_MAX_K or n < 8 or n % 8 or n > 1 << 24
            or (code == L.EP_ACT_SWIGLU and wn % 2)):
        raise ValueError(f"codes: want [rows, k / 2] with rows in multiples of 8 (of 16 with act 'swiglu') and k a multiple "
                         f"of 32 up to {L.EP_W4_MAX_K}, got {tuple(codes.shape)} for x {tuple(x.shape)}")
    if scales.dim() < 2:
        raise ValueError(f"scales: want [..., k / group, rows], got {tuple(scales.shape)}")
    group, lead = _group(k, scales, -2), x.shape[:-1]
    if codes.dtype is not U8 or codes.device != dev or not codes.is_contiguous():
        _want(codes, "codes", codes.shape, dev, U8)
    _want(scales, "scales", codes.shape[:-2] + (k // group, wn), dev)
    out = _out(out, lead + (n,), BF16, dev, stream)
    if bias is not None:
        _want(bias, "bias", codes.shape[:-1], dev)
    if residual is not None:
        _want(residual, "residual", lead + (n,), dev)
    if counts is not None and (counts.dtype != I32 or counts.numel() != groups or not counts.is_contiguous()
                               or counts.device != dev):
        raise ValueError(f"counts: want contiguous int32 of {groups} groups on {dev}, got {counts.dtype} "
                         f"{tuple(counts.shape)} on {counts.device}")
    if status is not None:
        _want(status, "status", (1,), dev, I32)
    a = L.EpW4C(groups, rows, k, n, code, kind, group, _ptr(counts), _ptr(status))
    L.check(L.lib().ep_product_w4(C.byref(a), x.data_ptr(), codes.data_ptr(), scales.data_ptr(), _ptr(bias), _ptr(residual),
                                  out.data_ptr(), stream_of(stream, dev)), "ep_product_w4")
    return out


def experts_product_w4(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, counts: torch.Tensor, *,
                       kind: str = "int4", bias: Optional[torch.Tensor] = None, act: str = "none",
                       residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """:func:`experts_product` with 4-bit weights: ``act(x[e] @ w[e]^T + bias[e]) + residual[e]`` in bf16 on each
    expert's first ``counts[e]`` rows, with ``w = dequantize_weight4(codes, scales, kind)``.

    ``x`` ``[..., E, rows, k]``, ``codes`` ``[..., E, n, k / 2]`` (``swiglu``: 2n rows, gate rows first), ``scales``
    ``[..., E, k / group, n]``, ``counts`` int32 on the device. Rows past the counts are not written.
    """
    return _forward(x, codes, scales, counts, True, kind, bias, act, residual, out, status, stream)


def linear_w4(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, *, kind: str = "int4",
              bias: Optional[torch.Tensor] = None, act: str = "none", residual: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """:func:`linear` with a 4-bit weight, in bf16: ``x`` ``[..., k]``, ``codes`` ``[n, k / 2]`` (``swiglu``: 2n rows),
    ``scales`` ``[k / group, n]``."""
    return _forward(x, codes, scales, None, False, kind, bias, act, residual, out, status, stream)
