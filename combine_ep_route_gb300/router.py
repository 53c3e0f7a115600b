"""The top-k router: logits to the expert ids and weights that dispatch takes, and
the logits' gradient (``ep_topk_route``, ``ep_topk_route_backward`` in include/ep.h)."""
from __future__ import annotations

import ctypes as C
from typing import Optional, Tuple

import torch

from . import _lib as L
from .product import INT32_MAX, _want, empty, stream_of, untracked

_SCORES = {"softmax": L.EP_SCORE_SOFTMAX, "sigmoid": L.EP_SCORE_SIGMOID}
_BIASED = {"logits": 0, "scores": L.EP_BIAS_ON_SCORE}
_I32, _F32 = torch.int32, torch.float32
_TYPES = {torch.bfloat16: L.EP_BF16, torch.float32: L.EP_F32}


def _args(logits: torch.Tensor, top_k: int, score: str, renormalize: bool, scale: float) -> L.EpTopkC:
    code, kind, E = _SCORES.get(score), _TYPES.get(logits.dtype), logits.shape[-1] if logits.dim() else 0
    if (code is not None and kind is not None and logits.is_cuda and logits.is_contiguous()
            and 1 <= top_k <= E <= L.EP_MAX_E and top_k <= L.EP_MAX_TOPK
            and (tokens := logits.numel() // E) <= INT32_MAX):
        return L.EpTopkC(tokens, E, top_k, code, 1 if renormalize else 0, kind, scale)
    if code is None:
        raise ValueError(f"score: want one of {sorted(_SCORES)}, got {score!r}")
    if kind is None or not logits.dim() or not logits.is_contiguous() or not logits.is_cuda:
        raise ValueError(f"logits: want contiguous bfloat16 or float32 [..., E] on a CUDA device, got {logits.dtype} "
                         f"{tuple(logits.shape)} on {logits.device} (contiguous={logits.is_contiguous()})")
    raise ValueError(f"want 1..{L.EP_MAX_E} experts, top_k in 1..min(E, {L.EP_MAX_TOPK}) and at most {INT32_MAX} tokens, "
                     f"got {tuple(logits.shape)}, top_k={top_k}")


def _chosen(logits: torch.Tensor, a: L.EpTopkC) -> Tuple[int, ...]:
    """The shape of ids and weights."""
    return (a.tokens, a.top_k) if logits.dim() == 2 else logits.shape[:-1] + (a.top_k,)


def route_topk(logits: torch.Tensor, top_k: int, *, score: str = "softmax", renormalize: bool = True,
               bias: Optional[torch.Tensor] = None, bias_on: str = "logits", scale: float = 1.0,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``(topk_ids int32, topk_weights float32)``, both ``[..., top_k]``, for ``logits`` ``[..., E]``.

    Experts are chosen by ``logits + bias``, or with ``bias_on="scores"`` by ``score + bias``, largest
    first, ties to the lowest id; weights are ``scale`` times the score of the unbiased logit, divided by
    the chosen scores' sum with ``renormalize``. The two choices differ: a correction bias that balances
    the experts of a sigmoid (or softmax) gate is trained on the scores and needs ``bias_on="scores"``.
    A logit of minus infinity (or NaN) masks its expert; a row with fewer than ``top_k`` experts left ends
    in ids of -1, which dispatch drops.
    """
    a = _args(logits, top_k, score, renormalize, scale)
    if logits.requires_grad or (bias is not None and bias.requires_grad):
        untracked(logits=logits, bias=bias)
    dev, shape = logits.device, _chosen(logits, a)
    if bias_on not in _BIASED:
        raise ValueError(f"bias_on: want one of {sorted(_BIASED)}, got {bias_on!r}")
    if bias is not None:
        _want(bias, "bias", (a.E,), dev, _F32)
        a.score |= _BIASED[bias_on]
    if out is None:
        ids, weights = empty(shape, _I32, dev, stream), empty(shape, _F32, dev, stream)
    else:
        ids, weights = out
        _want(ids, "topk_ids", shape, dev, _I32)
        _want(weights, "topk_weights", shape, dev, _F32)
    L.check(L.lib().ep_topk_route(C.byref(a), logits.data_ptr(), None if bias is None else bias.data_ptr(),
                                  ids.data_ptr(), weights.data_ptr(), stream_of(stream, dev)), "ep_topk_route")
    return ids, weights


def route_topk_backward(dweights: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, *,
                        score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                        out: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The logits' gradient (of the logits' type) for the gradient of ``route_topk``'s weights."""
    if topk_ids.dim() < 1:
        raise ValueError("topk_ids: want [..., top_k]")
    a = _args(logits, topk_ids.shape[-1], score, renormalize, scale)
    if dweights.requires_grad:
        untracked(dweights=dweights)
    dev, shape = logits.device, _chosen(logits, a)
    _want(topk_ids, "topk_ids", shape, dev, _I32)
    _want(dweights, "dweights", shape, dev, _F32)
    if out is None:
        out = empty(logits.shape, logits.dtype, dev, stream)
    else:
        _want(out, "out", logits.shape, dev, logits.dtype)
    L.check(L.lib().ep_topk_route_backward(C.byref(a), dweights.data_ptr(), logits.data_ptr(), topk_ids.data_ptr(),
                                           out.data_ptr(), stream_of(stream, dev)), "ep_topk_route_backward")
    return out
