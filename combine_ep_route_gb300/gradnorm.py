"""The global norm of many gradients and their clipping by it (``ep_clip_grad_norm`` in include/ep.h)."""
from __future__ import annotations

import ctypes as C
from array import array
from typing import Optional, Sequence

import torch

from . import _lib as L
from .product import _OUT, _want, INT32_MAX, empty, stream_of, untracked


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, *, out: Optional[Sequence[torch.Tensor]] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The norm of all ``grads`` together (float32, no dimensions), which are scaled in place by ``max_norm / norm``
    where it is finite and above ``max_norm``, and otherwise left as they are; a norm that is not finite is the
    caller's to handle. (Finite elements have a finite norm in the 64 bits that decide: one past the largest float is
    returned as infinity, and clipped.)

    ``grads`` are contiguous bf16 and float32 tensors of any shape on one CUDA device, of which no two overlap;
    ``max_norm`` of infinity gives the norm alone. With ``out`` (tensors of the same shapes and types) the
    gradients, scaled or not, are written there and ``grads`` stay as they are. Nothing waits for the GPU.
    """
    grads = list(grads)
    outs = grads if out is None else list(out)
    max_norm = float(max_norm)
    if not grads:
        raise ValueError("grads: want one tensor at least")
    if not max_norm >= 0:
        raise ValueError(f"max_norm: want a number from 0, got {max_norm}")
    if len(outs) != len(grads):
        raise ValueError(f"out: want {len(grads)} tensors, got {len(outs)}")
    n, dev, at = len(grads), grads[0].device, grads[0].get_device()
    if n > INT32_MAX:
        raise ValueError("grads: too many")
    # (whole lists at a time, and a look at each tensor where something is wrong: there may be hundreds)
    types = [t.dtype for t in grads]
    kinds = [_OUT.get(d) for d in types]
    if None in kinds or at < 0 or [t.get_device() for t in grads] != [at] * n or not all([t.is_contiguous() for t in grads]):
        for t in grads:
            if t.dtype not in _OUT or not t.is_cuda or t.get_device() != at or not t.is_contiguous():
                raise ValueError(f"grads: want contiguous bfloat16 or float32 on one CUDA device, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")
    if any([t.requires_grad for t in grads]):
        untracked(**{f"grads[{i}]": t for i, t in enumerate(grads)})
    # (arrays of 64 and 32 bits: a ctypes array of as many pointers takes several times as long to fill)
    ptrs, to = array("Q", [t.data_ptr() for t in grads]), None
    if out is not None:
        if ([o.dtype for o in outs] != types or [o.shape for o in outs] != [t.shape for t in grads]
                or [o.get_device() for o in outs] != [at] * n or not all([o.is_contiguous() for o in outs])):
            for o, t in zip(outs, grads):
                _want(o, "out", t.shape, dev, t.dtype)
        if any([o.requires_grad for o in outs]):
            untracked(**{f"out[{i}]": o for i, o in enumerate(outs)})
        to = array("Q", [t.data_ptr() for t in outs])
    numel, kinds = array("q", [t.numel() for t in grads]), array("i", kinds)
    a = L.EpGradsC(n, ptrs.buffer_info()[0], None if to is None else to.buffer_info()[0], numel.buffer_info()[0],
                   kinds.buffer_info()[0])
    size, lib = C.c_size_t(), L.lib()
    L.check(lib.ep_clip_workspace_bytes(C.byref(a), C.byref(size)), "ep_clip_workspace_bytes")
    norm, work = empty((), torch.float32, dev, stream), empty((size.value,), torch.uint8, dev, stream)
    L.check(lib.ep_clip_grad_norm(C.byref(a), max_norm, norm.data_ptr(), work.data_ptr(), size.value,
                                  stream_of(stream, dev)), "ep_clip_grad_norm (tensors must not overlap)")
    return norm
