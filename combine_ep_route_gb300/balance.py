"""The router's balance loss: per-expert counts, the loss that keeps the experts evenly used, the z loss
that keeps the logits small, and the logits' gradient of both (``ep_balance_loss`` and
``ep_balance_loss_backward`` in include/ep.h)."""
from __future__ import annotations

import ctypes as C
from math import prod
from typing import Optional, Tuple

import torch

from . import _lib as L
from .product import INT32_MAX, _want, empty, stream_of, untracked
from .router import _SCORES, _TYPES

_I32, _F32 = torch.int32, torch.float32


def _args(logits: torch.Tensor, top_k: int, score: str, per_sequence: bool,
          num_tokens: Optional[torch.Tensor]) -> Tuple[L.EpBalanceC, Tuple[int, ...]]:
    """The call's arguments and the shape of counts."""
    code, kind, shape = _SCORES.get(score), _TYPES.get(logits.dtype), logits.shape
    if code is None:
        raise ValueError(f"score: want one of {sorted(_SCORES)}, got {score!r}")
    if kind is None or len(shape) < 2 or not logits.is_contiguous() or not logits.is_cuda:
        raise ValueError(f"logits: want contiguous bfloat16 or float32 [..., T, E] on a CUDA device, got "
                         f"{logits.dtype} {tuple(logits.shape)} on {logits.device} "
                         f"(contiguous={logits.is_contiguous()})")
    lead, tokens, E = shape[:-2], shape[-2], shape[-1]
    seqs = lead[0] if len(lead) == 1 else prod(lead)
    if not 1 <= E <= L.EP_MAX_E or not 1 <= top_k <= min(E, L.EP_MAX_TOPK) or max(seqs, tokens, seqs * tokens) > INT32_MAX:
        raise ValueError(f"want 1..{L.EP_MAX_E} experts, top_k in 1..min(E, {L.EP_MAX_TOPK}) and at most {INT32_MAX} "
                         f"tokens, got {tuple(logits.shape)}, top_k={top_k}")
    ptr = None
    if num_tokens is not None:
        _want(num_tokens, "num_tokens", lead or (1,), logits.device, _I32)
        ptr = num_tokens.data_ptr()
    a = L.EpBalanceC(seqs, tokens, E, top_k, code, 1 if per_sequence else 0, kind, ptr)
    return a, (lead + (E,) if per_sequence else (E,))


def balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, *, score: str = "softmax", per_sequence: bool = False,
                 num_tokens: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``(losses float32 [2], counts int32 [E])`` of the router's ``logits`` ``[..., T, E]`` and the choices
    ``topk_ids`` ``[..., T, K]`` (as ``route_topk`` gives them; ids of -1 are not counted).

    With ``c_e`` the tokens' choices of expert e, N the tokens and ``p_e`` a token's probability of it (softmax, or
    its sigmoid over the sum of all): ``losses[0] = sum_e E c_e / (K N) * mean(p_e)``, 1 where both are even, and
    ``losses[1]`` is the mean square of the logits' logsumexp (the z loss). ``num_tokens`` int32 ``[...]`` (dispatch's)
    says how many of each sequence's T tokens there are. With ``per_sequence`` every sequence has counts (``[..., E]``)
    and a loss of its own, and ``losses[0]`` is their mean over the sequences that have tokens. Infinite and NaN
    logits count as in ``route_topk``. A total is formed as ``total + 1e-2 * losses[0] + 1e-3 * losses[1]``, with
    ``torch.tensor([1e-2, 1e-3])`` (times the total's gradient) as ``dlosses`` of the gradient.
    """
    if topk_ids.dim() < 1:
        raise ValueError("topk_ids: want [..., T, top_k]")
    K = topk_ids.shape[-1]
    a, shape = _args(logits, K, score, per_sequence, num_tokens)
    if logits.requires_grad:
        untracked(logits=logits)
    dev = logits.device
    _want(topk_ids, "topk_ids", logits.shape[:-1] + (K,), dev, _I32)
    size, lib, args = C.c_size_t(), L.lib(), C.byref(a)
    L.check(lib.ep_balance_workspace_bytes(args, C.byref(size)), "ep_balance_workspace_bytes")
    losses, counts = empty((2,), _F32, dev, stream), empty(shape, _I32, dev, stream)
    work = empty((size.value,), torch.uint8, dev, stream)
    L.check(lib.ep_balance_loss(args, logits.data_ptr(), topk_ids.data_ptr(), losses.data_ptr(), counts.data_ptr(),
                                work.data_ptr(), size.value, stream_of(stream, dev)), "ep_balance_loss")
    return losses, counts


def balance_loss_backward(dlosses: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor, top_k: int, *,
                          score: str = "softmax", per_sequence: bool = False, num_tokens: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, accumulate: bool = False,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The logits' gradient (of the logits' type) for the losses' gradient ``dlosses`` float32 ``[2]``, with the
    ``counts`` that :func:`balance_loss` gave (they have no gradient). With ``accumulate`` it is added to ``out``
    (``route_topk_backward``'s, say), whose rows past ``num_tokens`` stay as they are; they are zero otherwise."""
    a, shape = _args(logits, top_k, score, per_sequence, num_tokens)
    if dlosses.requires_grad:
        untracked(dlosses=dlosses)
    dev = logits.device
    _want(dlosses, "dlosses", (2,), dev, _F32)
    _want(counts, "counts", shape, dev, _I32)
    if out is None:
        if accumulate:
            raise ValueError("out: wanted with accumulate")
        out = empty(logits.shape, logits.dtype, dev, stream)
    else:
        _want(out, "out", logits.shape, dev, logits.dtype)
    L.check(L.lib().ep_balance_loss_backward(C.byref(a), dlosses.data_ptr(), logits.data_ptr(), counts.data_ptr(),
                                             1 if accumulate else 0, out.data_ptr(), stream_of(stream, dev)),
            "ep_balance_loss_backward")
    return out
