"""The layers' operators in 64 bits, written from their definitions, with the error
each fp32 computation may make. Used by the GPU tests of the products and the router
(and checked against differences on the CPU).

Error bound of a product: bf16 operands multiply exactly in fp32; a sum over k
elements in steps of 16 makes at most one truncation (2^-23 of the running sum of
magnitudes S) per step and a few inside a step: |dz| <= (k / 16 + 16) 2^-23 S. A
function of z adds its slope times that; a bf16 output adds half a unit (2^-9),
doubled for the fast exponential and division in front of it; an fp32 output
2^-20 for them.
"""
import math

import torch

D = torch.float64


def act64(z, act):
    """(value, slope) of an elementwise activation."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).to(z.dtype)
    if act in ("silu", "swiglu"):
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def sum_error(k):
    return (k / 16 + 16) * 2.0 ** -23


def out_error(y, dtype):
    return y.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20) + 1e-30


def forward(x, w, bias, act, residual, dtype):
    """One group: (y, its error bound, z, its error bound); z is kept in bf16."""
    x, w = x.to(D), w.to(D)
    z = x @ w.T
    dz = (x.abs() @ w.abs().T) * sum_error(x.shape[1])
    if bias is not None:
        z = z + bias.to(D)
        dz = dz + z.abs() * 2.0 ** -23
    if act == "swiglu":
        n = w.shape[0] // 2
        g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
        v = act64(g, "silu")[0]
        y = v * u
        dy = 1.1 * dg * u.abs() + v.abs() * du + y.abs() * 2.0 ** -18
    else:
        y = act64(z, act)[0]
        dy = 1.13 * dz + (0 if act in ("none", "relu") else z.abs() * 2.0 ** -20)
    if residual is not None:
        y = y + residual.to(D)
        dy = dy + y.abs() * 2.0 ** -23
    return y, dy + out_error(y, dtype), z, dz + out_error(z, torch.bfloat16)


def dgrad(dy, w, act, preact, dtype):
    """One group: (gradient, its error bound)."""
    dy, w = dy.to(D), w.to(D)
    dh = dy @ w
    e = (dy.abs() @ w.abs()) * sum_error(dy.shape[1])
    if act == "none":
        return dh, e + out_error(dh, dtype)
    z = preact.to(D)
    if act == "swiglu":
        k = w.shape[1]
        value, slope = act64(z[:, :k], "silu")
        u = z[:, k:]
        d = torch.cat((dh * u * slope, dh * value), 1)
        e = torch.cat((e * u.abs() * 1.1, e * value.abs()), 1)
        # rounding inside the slope, relative to its largest term
        e = e + torch.cat(((dh * u).abs() * (1 + z[:, :k].abs()), (dh * value).abs()), 1) * 2.0 ** -20
    else:
        slope = act64(z, act)[1]
        d = dh * slope
        e = e * 1.13 + dh.abs() * (0 if act == "relu" else 1 + z.abs()) * 2.0 ** -20
    return d, e + out_error(d, dtype)


def wgrad(dy, x, dtype, before=None):
    """One group: (dw, error, db, error) over the rows given."""
    dy, x = dy.to(D), x.to(D)
    dw, db = dy.T @ x, dy.sum(0)
    ew = (dy.abs().T @ x.abs()) * sum_error(dy.shape[0])
    eb = dy.abs().sum(0) * (dy.shape[0] / 32 + 48) * 2.0 ** -24
    if before is not None:
        dw, db = dw + before[0].to(D), db + before[1].to(D)
        ew, eb = ew + dw.abs() * 2.0 ** -23, eb + db.abs() * 2.0 ** -23
    return dw, ew + out_error(dw, dtype), db, eb + out_error(db, dtype)


def route(logits, k, score, renormalize, bias, scale):
    """(ids, weights) of a [tokens, E] tensor, row by row."""
    T, E = logits.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    weights = torch.zeros(T, k, dtype=D)
    z32 = logits.float().cpu()
    key32 = z32 if bias is None else z32 + bias.float().cpu()
    big = torch.finfo(torch.float32).max
    for t in range(T):
        left = [e for e in range(E) if z32[t, e] >= -big and key32[t, e] >= -big]
        left.sort(key=lambda e: (-key32[t, e].item(), e))
        pick = left[:k]
        z = z32[t].to(D).clamp(max=big)
        z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
        if not pick:
            continue
        if score == "softmax":
            # renormalised, the sum over all experts cancels (and may be too large to carry)
            logs = z if renormalize else torch.log_softmax(z, 0)
        else:
            logs = torch.nn.functional.logsigmoid(z)
        s = logs[pick]
        w = torch.softmax(s, 0) if renormalize else s.exp()
        ids[t, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
        weights[t, :len(pick)] = scale * w
    return ids, weights


def route_weights(z, ids, score, renormalize, scale):
    """The weights as a differentiable function of 64-bit logits, for chosen ids (all >= 0)."""
    logs = torch.log_softmax(z, 1) if score == "softmax" else torch.nn.functional.logsigmoid(z)
    s = logs.gather(1, ids.long())
    return scale * (torch.softmax(s, 1) if renormalize else s.exp())
