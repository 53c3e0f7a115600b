"""The layer operators around the expert-parallel dispatch and combine, as cases to measure.

Three operators: the experts' products over the batched-experts layout
[E, rows, hidden] with a row count per expert, the linear product with bias,
activation and residual in its epilogue, and the top-k router. ``run`` computes
them through the package (``own`` true) or in plain 32-bit torch operations.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # --- experts
        # a tiny batch on a tiny layer (2 ranks x 16 tokens, 8 experts, top 2): launch latency
        dict(name="experts tiny", op="experts", form="forward", E=8, rows=32, k=128, n=128, act="swiglu",
             pairs=56, ids="uniform", bias=False, keep=False),
        # the gated up-product of a decode batch (8 ranks x 128 tokens, 64 experts, top 8, 5 % padding):
        # the experts' weights stream past about 120 rows each
        dict(name="experts decode", op="experts", form="forward", E=64, rows=1024, k=2048, n=1024, act="swiglu",
             pairs=7784, ids="uniform", bias=False, keep=False),
        # the gated up-product of a prefill batch (8 ranks x 1024 tokens, 256 experts, top 8, hidden 7168),
        # with rows kept for twice the mean
        dict(name="experts prefill", op="experts", form="forward", E=256, rows=512, k=7168, n=2048, act="swiglu",
             pairs=65536, ids="uniform", bias=False, keep=False),
        # the down-product, with bias, under Zipf(1.2) popularity: one expert full, most nearly empty
        dict(name="experts zipf down", op="experts", form="forward", E=64, rows=4096, k=2048, n=4096, act="none",
             pairs=32768, ids="zipf", bias=True, keep=False),
        # training: the down-product's input gradient through the gated activation
        dict(name="experts grad input", op="experts", form="dgrad", E=64, rows=512, k=2048, n=7168, act="swiglu",
             pairs=16384, ids="uniform"),
        # training: the up-product's weight gradient of one rank's 32 experts, in 32 bits
        dict(name="experts grad weight", op="experts", form="wgrad", E=32, rows=512, k=7168, n=4096,
             pairs=8192, ids="uniform", out="f32"),
        # --- linear
        # a dense feed-forward up-product over a prefill batch in training: the pre-activation is kept
        dict(name="linear prefill", op="linear", form="forward", rows=8192, k=7168, n=4096, act="gelu_tanh",
             bias=True, residual=False, keep=True, out="bf16"),
        # a projection with bias and residual on seven decoding sequences: weights stream past few rows
        dict(name="linear decode", op="linear", form="forward", rows=7, k=7168, n=7168, act="none",
             bias=True, residual=True, keep=False, out="bf16"),
        # the router's logits in 32 bits: a long reduction with few outputs
        dict(name="linear logits", op="linear", form="forward", rows=1024, k=7168, n=256, act="none",
             bias=False, residual=False, keep=False, out="f32"),
        # training: the second product of a feed-forward pair, its three gradients
        # (the input's through the activation), on an odd number of rows
        dict(name="linear backward", op="linear", form="backward", rows=5001, k=4096, n=2048, act="gelu"),
        # --- router
        # one rank's decode batch
        dict(name="router decode", op="router", form="forward", rows=128, E=64, top_k=8, score="softmax",
             renormalize=True, bias=False, scale=1.0, type="f32"),
        # a prefill batch in training: ids, weights and the logits' gradient
        dict(name="router train", op="router", form="train", rows=8192, E=256, top_k=8, score="sigmoid",
             renormalize=True, bias=True, scale=2.5, type="bf16"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    acts = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")
    op = rng.choice(("experts", "experts", "linear", "linear", "router"))
    if op == "router":
        E = _spread(rng, 4, 512)
        return dict(op=op, form=rng.choice(("forward", "train")), rows=_spread(rng, 1, 16384), E=E,
                    top_k=rng.randint(1, min(16, E)), score=rng.choice(("softmax", "sigmoid")),
                    renormalize=rng.random() < 0.5, bias=rng.random() < 0.5,
                    scale=rng.choice((1.0, 2.5)), type=rng.choice(("bf16", "f32")))
    if op == "linear":
        rows, k, n = _spread(rng, 1, 8192), 8 * _spread(rng, 8, 896), 8 * _spread(rng, 8, 896)
        if rng.random() < 0.35:
            return dict(op=op, form="backward", rows=rows, k=min(k, 4096), n=min(n, 4096), act=rng.choice(acts[:5]))
        return dict(op=op, form="forward", rows=rows, k=k, n=n, act=rng.choice(acts),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5, keep=rng.random() < 0.3, out="bf16")
    E = rng.choice((4, 8, 13, 32, 60, 64, 128))
    form = rng.choice(("forward", "forward", "dgrad", "wgrad"))
    pairs = _spread(rng, 1, 300 * E)
    rows = min(4096, max(4, 2 * (-(-pairs // E)) + rng.randint(0, 9)))
    c = dict(op=op, form=form, E=E, rows=rows, k=8 * _spread(rng, 8, 512), n=8 * _spread(rng, 8, 256),
             pairs=pairs, ids=rng.choice(("uniform", "zipf")))
    if form == "forward":
        c.update(act=rng.choice(("none", "silu", "swiglu", "swiglu")), bias=rng.random() < 0.3, keep=rng.random() < 0.3)
    elif form == "dgrad":
        c.update(act=rng.choice(("none", "gelu", "swiglu")))
    else:
        c.update(out=rng.choice(("bf16", "f32")))
    return c


# ------------------------------------------------------------------ the inputs

def _popularity(case):
    """Each expert's share of the pairs: even, or P(e) ~ (e + 1)^-1.2."""
    s = 1.2 if case["ids"] == "zipf" else 0.0
    p = torch.arange(1, case["E"] + 1, dtype=torch.float64) ** -s
    return p / p.sum()


def _shapes(case):
    """(rows of the weight per output column, whether the activation is gated)."""
    gated = case.get("act") == "swiglu"
    return (2 if gated else 1), gated


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + 17)

    def normal(*shape, std=1.0, dtype=BF16):
        t = torch.randn(*shape, generator=g, device=dev, dtype=dtype)
        return t if std == 1.0 else t.mul_(std)

    st = {"case": case}
    rows = case["rows"]
    if case["op"] == "router":
        E, K = case["E"], case["top_k"]
        st["logits"] = normal(rows, E, dtype=DTYPES[case["type"]])
        st["bias"] = normal(E, std=0.2, dtype=F32) if case["bias"] else None
        st["dweights"] = normal(rows, K, dtype=F32) if case["form"] == "train" else None
        return st
    k, n = case["k"], case["n"]
    two, _ = _shapes(case)
    lead = () if case["op"] == "linear" else (case["E"],)
    if case["op"] == "experts":
        p = _popularity(case).to(dev)
        hit = torch.multinomial(p, case["pairs"], replacement=True, generator=g)
        st["counts"] = torch.bincount(hit, minlength=case["E"]).clamp(max=rows).to(torch.int32)
    if case["form"] == "forward":
        st["x"] = normal(*lead, rows, k)
        st["w"] = normal(*lead, two * n, k, std=k ** -0.5)
        st["bias"] = normal(*lead, two * n) if case["bias"] else None
        st["residual"] = normal(*lead, rows, n) if case.get("residual") else None
        st["out"] = torch.zeros(*lead, rows, n, dtype=DTYPES[case.get("out", "bf16")], device=dev)
        st["preact"] = torch.zeros(*lead, rows, two * n, dtype=BF16, device=dev) if case["keep"] else None
    elif case["form"] in ("dgrad", "backward"):
        # w [.., n, k] is the product whose input gradient is taken; z is what its input's activation saw
        st["dy"] = normal(*lead, rows, n)
        st["w"] = normal(*lead, n, k, std=n ** -0.5)
        st["z"] = normal(*lead, rows, two * k) if case["act"] != "none" else None
        st["dz"] = torch.zeros(*lead, rows, two * k, dtype=BF16, device=dev)
        if case["form"] == "backward":
            st["x"] = normal(rows, k)
    else:
        st["dy"] = normal(*lead, rows, n)
        st["x"] = normal(*lead, rows, k)
        st["out"] = torch.zeros(*lead, n, k, dtype=DTYPES[case["out"]], device=dev)
    return st


# -------------------------------------------------------------- the plain forms

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    gate, up = z.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _act_grad(dh, z, act):
    if act == "none":
        return dh
    if act == "relu":
        return dh * (z > 0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return dh * s * (1 + z * (1 - s))
    if act == "gelu":
        return dh * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return dh * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
    gate, up = z.chunk(2, dim=-1)
    s = 1 / (1 + torch.exp(-gate))
    return torch.cat((dh * up * s * (1 + gate * (1 - s)), dh * gate * s), dim=-1)


def _plain_product(st, case):
    lead = case["op"] == "experts"
    if lead:
        mask = (torch.arange(case["rows"], device=st["counts"].device) < st["counts"][:, None])[..., None]
    if case["form"] == "forward":
        z = torch.matmul(st["x"].float(), st["w"].float().transpose(-1, -2))
        if st["bias"] is not None:
            z = z + st["bias"].float().unsqueeze(-2)
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        y = y.to(st["out"].dtype)
        out = {"y": torch.where(mask, y, st["out"]) if lead else y}
        if st["preact"] is not None:
            z = z.to(BF16)
            out["z"] = torch.where(mask, z, st["preact"]) if lead else z
        return out
    if case["form"] == "wgrad":
        dy = torch.where(mask, st["dy"].float(), 0.0)
        x = torch.where(mask, st["x"].float(), 0.0)
        return {"dw": torch.matmul(dy.transpose(-1, -2), x).to(st["out"].dtype)}
    dy = st["dy"].float()
    dz = _act_grad(torch.matmul(dy, st["w"].float()), None if st["z"] is None else st["z"].float(), case["act"]).to(BF16)
    if case["form"] == "dgrad":
        return {"dz": torch.where(mask, dz, st["dz"])}
    return {"dz": dz, "dw": torch.matmul(dy.transpose(-1, -2), st["x"].float()).to(BF16), "db": dy.sum(0).to(BF16)}


def _plain_router(st, case):
    z = st["logits"].float()
    key = z if st["bias"] is None else z + st["bias"]
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :case["top_k"]]
    chosen = z.gather(1, ids)
    soft, norm = case["score"] == "softmax", case["renormalize"]
    if soft:
        e = torch.exp(z - z.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    pk = p.gather(1, ids)
    if soft and norm:
        e = torch.exp(chosen - chosen.amax(1, keepdim=True))
        q = e / e.sum(1, keepdim=True)
    else:
        q = pk / pk.sum(1, keepdim=True) if norm else pk
    out = {"ids": ids.to(torch.int32), "weights": case["scale"] * q}
    if case["form"] == "train":
        dq = case["scale"] * st["dweights"]
        mean = (dq * q).sum(1, keepdim=True)
        if soft and norm:
            d = torch.zeros_like(z).scatter(1, ids, q * (dq - mean))
        elif soft:
            d = torch.zeros_like(z).scatter(1, ids, q * dq) - p * mean
        elif norm:
            d = torch.zeros_like(z).scatter(1, ids, q * (1 - pk) * (dq - mean))
        else:
            d = torch.zeros_like(z).scatter(1, ids, q * (1 - pk) * dq)
        out["dlogits"] = d.to(st["logits"].dtype)
    return out


# --------------------------------------------------------------------- one pass

def _own_router(st, case):
    import combine_ep_route_gb300 as ep

    kw = dict(score=case["score"], renormalize=case["renormalize"], scale=case["scale"])
    ids, weights = ep.route_topk(st["logits"], case["top_k"], bias=st["bias"], **kw)
    out = {"ids": ids, "weights": weights}
    if case["form"] == "train":
        out["dlogits"] = ep.route_topk_backward(st["dweights"], st["logits"], ids, **kw)
    return out


def _own_product(st, case):
    import combine_ep_route_gb300 as ep

    if case["op"] == "experts":
        if case["form"] == "forward":
            y = ep.experts_product(st["x"], st["w"], st["counts"], bias=st["bias"], act=case["act"], out=st["out"], preact=st["preact"])
            return {"y": y} if st["preact"] is None else {"y": y, "z": st["preact"]}
        if case["form"] == "dgrad":
            return {"dz": ep.experts_product_dgrad(st["dy"], st["w"], st["counts"], act=case["act"], preact=st["z"], out=st["dz"])}
        return {"dw": ep.experts_product_wgrad(st["dy"], st["x"], st["counts"], out=st["out"])}
    if case["form"] == "forward":
        y = ep.linear(st["x"], st["w"], bias=st["bias"], act=case["act"], residual=st["residual"], out=st["out"], preact=st["preact"])
        return {"y": y} if st["preact"] is None else {"y": y, "z": st["preact"]}
    dz = ep.linear_dgrad(st["dy"], st["w"], act=case["act"], preact=st["z"], out=st["dz"])
    dw, db = ep.linear_wgrad(st["dy"], st["x"], bias_grad=True)
    return {"dz": dz, "dw": dw, "db": db}


def run(state):
    case = state["case"]
    if case["op"] == "router":
        return _own_router(state, case) if own else _plain_router(state, case)
    return _own_product(state, case) if own else _plain_product(state, case)


# ------------------------------------------------------------ what a pass needs

def work(case):
    rows = case["rows"]
    if case["op"] == "router":
        E, K, size = case["E"], case["top_k"], 2 if case["type"] == "bf16" else 4
        b = rows * E * size + rows * K * 8 + (4 * E if case["bias"] else 0)
        f = rows * E * 4
        if case["form"] == "train":
            b += rows * K * 4 + rows * E * size
            f += rows * E * 6
        return {"bytes": b, "flops": f}
    k, n = case["k"], case["n"]
    two, _ = _shapes(case)
    if case["op"] == "experts":
        p = _popularity(case)
        used = float((case["pairs"] * p).clamp(max=rows).sum())
        active = float((1 - (1 - p) ** case["pairs"]).sum())
        groups = case["E"]
    else:
        used, active, groups = rows, 1, 1
    if case["form"] == "forward":
        b = 2 * used * k + 2 * active * two * n * k + (4 if case.get("out") == "f32" else 2) * used * n
        b += (2 * active * two * n if case["bias"] else 0) + (2 * used * n if case.get("residual") else 0)
        b += 2 * used * two * n if case["keep"] else 0
        return {"bytes": b, "flops": 2 * used * two * n * k}
    if case["form"] == "wgrad":
        return {"bytes": 2 * used * (n + k) + (4 if case["out"] == "f32" else 2) * groups * n * k, "flops": 2 * used * n * k}
    b = 2 * used * n + 2 * active * n * k + 2 * used * two * k * (1 if case["act"] == "none" else 2)
    f = 2 * used * n * k
    if case["form"] == "backward":
        b, f = b + 2 * rows * k + 2 * n * k + 2 * n, 2 * f + rows * n
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------ 64-bit definitions

def _phi(z, act):
    """(value, derivative) of an elementwise activation in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.relu(z), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    du = math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    s = torch.sigmoid(2 * u)   # (1 + tanh u) / 2
    return z * s, s + z * 2 * s * (1 - s) * du


def _exact_group(case, x, w, bias, residual):
    z = torch.einsum("rk,nk->rn", x.double(), w.double())
    if bias is not None:
        z += bias.double()
    if case["act"] == "swiglu":
        n = case["n"]
        y = _phi(z[:, :n], "silu")[0] * z[:, n:]
    else:
        y = _phi(z, case["act"])[0]
    return (y if residual is None else y + residual.double()), z


def _exact_dgrad(case, dy, w, z):
    dh = torch.einsum("rn,nk->rk", dy.double(), w.double())
    if case["act"] == "none":
        return dh
    z = z.double()
    if case["act"] == "swiglu":
        k = case["k"]
        value, slope = _phi(z[:, :k], "silu")
        return torch.cat((dh * z[:, k:] * slope, dh * value), 1)
    return dh * _phi(z, case["act"])[1]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "router":
        return _exact_router(case, st)
    D = torch.float64
    if case["op"] == "linear":
        if case["form"] == "forward":
            y, z = _exact_group(case, st["x"], st["w"], st["bias"], st["residual"])
            return {"y": y, "z": z} if case["keep"] else {"y": y}
        dy = st["dy"].double()
        return {"dz": _exact_dgrad(case, st["dy"], st["w"], st["z"]),
                "dw": torch.einsum("rn,rk->nk", dy, st["x"].double()), "db": dy.sum(0)}
    counts = st["counts"].tolist()
    if case["form"] == "forward":
        out = {"y": torch.zeros(st["out"].shape, dtype=D, device="cuda")}
        if case["keep"]:
            out["z"] = torch.zeros(st["preact"].shape, dtype=D, device="cuda")
        for e, c in enumerate(counts):
            if c:
                y, z = _exact_group(case, st["x"][e, :c], st["w"][e], None if st["bias"] is None else st["bias"][e], None)
                out["y"][e, :c] = y
                if case["keep"]:
                    out["z"][e, :c] = z
        return out
    if case["form"] == "dgrad":
        dz = torch.zeros(st["dz"].shape, dtype=D, device="cuda")
        for e, c in enumerate(counts):
            if c:
                dz[e, :c] = _exact_dgrad(case, st["dy"][e, :c], st["w"][e], None if st["z"] is None else st["z"][e, :c])
        return {"dz": dz}
    dw = torch.zeros(st["out"].shape, dtype=D, device="cuda")
    for e, c in enumerate(counts):
        dw[e] = torch.einsum("rn,rk->nk", st["dy"][e, :c].double(), st["x"][e, :c].double())
    return {"dw": dw}


def _exact_router(case, st):
    logits = st["logits"].double()
    key = st["logits"].float() if st["bias"] is None else st["logits"].float() + st["bias"]
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["top_k"]]
    z = logits.detach().requires_grad_(case["form"] == "train")
    if case["score"] == "softmax":
        w = torch.log_softmax(z, 1).gather(1, ids).exp()
    else:
        w = torch.sigmoid(z).gather(1, ids)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    w = case["scale"] * w
    out = {"ids": None, "weights": w.detach()}
    if case["form"] == "train":
        out["dlogits"], = torch.autograd.grad(w, z, st["dweights"].double())
    return out
