"""Further operators of a Mixture-of-Experts layer, as cases to measure.

Three groups of operators: products with 4-bit weights and group scales (one weight, or one per
expert over the batched-experts layout), the router's balance loss and per-expert counts with the
logits' gradient, and the global gradient norm over many tensors with clipping. ``run`` computes
them through the package (``own`` true) or in plain 32-bit torch operations.
"""
import math

import torch

own = False

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DTYPES = {"bf16": BF16, "f32": F32}
# the element that each of the eight 4-bit fields of a 32-bit word holds, lowest field first
FIELDS = (0, 2, 4, 6, 1, 3, 5, 7)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # --- products with 4-bit weights
        # one decoding sequence through a projection with bias and residual: the weight streams past one row
        dict(name="linear_w4 token", op="w4", E=0, rows=1, k=7168, n=7168, act="none", kind="int4", group=128,
             bias=True, residual=True),
        # a shared expert's gated up-product on 33 decoding sequences
        dict(name="linear_w4 shared", op="w4", E=0, rows=33, k=7168, n=2048, act="swiglu", kind="fp4", group=32,
             bias=False, residual=False),
        # a tiny batch on a tiny layer (2 ranks x 16 tokens, 8 experts, top 2): launch latency
        dict(name="experts_w4 tiny", op="w4", E=8, rows=32, k=128, n=128, act="swiglu", kind="int4", group=32,
             bias=False, residual=False, pairs=56, ids="uniform"),
        # the down-product of a small decode batch (8 ranks x 4 tokens, 64 experts, top 8): four rows an expert
        dict(name="experts_w4 few", op="w4", E=64, rows=32, k=2048, n=7168, act="none", kind="int4", group=64,
             bias=True, residual=False, pairs=256, ids="uniform"),
        # the gated up-product of a decode batch (8 ranks x 128 tokens, 64 experts, top 8, 5 % padding)
        dict(name="experts_w4 decode", op="w4", E=64, rows=1024, k=2048, n=1024, act="swiglu", kind="fp4", group=32,
             bias=False, residual=False, pairs=7784, ids="uniform"),
        # the gated up-product of a prefill under Zipf(1.2) popularity: one expert full, most with few rows
        dict(name="experts_w4 prefill", op="w4", E=64, rows=1024, k=4096, n=2048, act="swiglu", kind="int4", group=128,
             bias=False, residual=False, pairs=16384, ids="zipf"),
        # --- the router's balance loss
        # the losses alone of a small batch, as an evaluation logs them
        dict(name="balance small", op="balance", form="forward", seqs=2, tokens=64, E=64, top_k=8, score="softmax",
             per_sequence=False, ragged=True, type="f32"),
        # a sigmoid gate's loss of each sequence of a prefill batch in training, ragged
        dict(name="balance sequences", op="balance", form="train", seqs=8, tokens=1024, E=256, top_k=8, score="sigmoid",
             per_sequence=True, ragged=True, type="bf16"),
        # a long batch in training (64 sequences of 1000 tokens, one loss over all)
        dict(name="balance batch", op="balance", form="train", seqs=64, tokens=1000, E=256, top_k=8, score="softmax",
             per_sequence=False, ragged=False, type="f32"),
        # --- the gradient norm and clipping
        # the small parameters of a layer: routers, norms and biases
        dict(name="clip small", op="clip", tensors=12, most=1 << 17, mean=40000, bf16=0.5, clipped=True),
        # one rank's gradients of several layers: experts' weights among many small tensors
        dict(name="clip layer", op="clip", tensors=50, most=1 << 26, mean=4_000_000, bf16=0.7, clipped=True),
        # a large model's: more than a hundred tensors, gigabytes in all
        dict(name="clip model", op="clip", tensors=160, most=1 << 28, mean=9_000_000, bf16=0.8, clipped=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("w4", "w4", "w4", "balance", "balance", "clip"))
    if op == "clip":
        return dict(op=op, tensors=_spread(rng, 1, 160), most=1 << rng.randint(10, 26), mean=_spread(rng, 20, 4_000_000),
                    bf16=rng.choice((0.0, 0.5, 1.0)), clipped=rng.random() < 0.8)
    if op == "balance":
        E = _spread(rng, 4, 512)
        seqs = _spread(rng, 1, 64)
        return dict(op=op, form=rng.choice(("forward", "train", "train")), seqs=seqs, tokens=_spread(rng, 1, 32768 // seqs),
                    E=E, top_k=rng.randint(1, min(16, E)), score=rng.choice(("softmax", "sigmoid")),
                    per_sequence=rng.random() < 0.5, ragged=rng.random() < 0.6, type=rng.choice(("bf16", "f32")))
    group = rng.choice((32, 64, 128))
    c = dict(op=op, E=0, kind=rng.choice(("int4", "fp4")), group=group, act=rng.choice(("none", "silu", "gelu", "swiglu", "swiglu")),
             bias=rng.random() < 0.3, residual=rng.random() < 0.3)
    if rng.random() < 0.5:
        return c | dict(rows=_spread(rng, 1, 600), k=group * _spread(rng, 1, 7168 // group), n=8 * _spread(rng, 2, 896))
    E = rng.choice((4, 8, 13, 32, 60, 64))
    pairs = _spread(rng, 1, 128 * E)
    rows = min(1024, max(4, 2 * (-(-pairs // E)) + rng.randint(0, 9)))
    return c | dict(E=E, rows=rows, k=group * _spread(rng, 1, 4096 // group), n=8 * _spread(rng, 2, 256), pairs=pairs,
                    ids=rng.choice(("uniform", "zipf")))


# ------------------------------------------------------------------ the inputs

def _popularity(case):
    """Each expert's share of the pairs: even, or P(e) ~ (e + 1)^-1.2."""
    s = 1.2 if case["ids"] == "zipf" else 0.0
    p = torch.arange(1, case["E"] + 1, dtype=torch.float64) ** -s
    return p / p.sum()


def _sizes(case):
    """The tensors' element counts: spread evenly in their logarithm up to `most`, odd ones among
    them, scaled to the wanted mean. The same for every seed, as a model's are."""
    n, most = case["tensors"], case["most"]
    raw = [most ** ((i * 0.6180339887 + 0.31) % 1.0) for i in range(n)]
    scale = case["mean"] * n / sum(raw)
    return [max(1, min(most, int(r * scale))) for r in raw]


def _is_bf16(case, i):
    return int((i + 1) * case["bf16"]) > int(i * case["bf16"])


def _views(flat, sizes):
    """The parts of a flat buffer, each at the next multiple of 8 elements."""
    out, at = [], 0
    for s in sizes:
        out.append(flat[at:at + s])
        at += -(-s // 8) * 8
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 1000003 + 29)

    def normal(*shape, std=1.0, dtype=BF16):
        t = torch.randn(*shape, generator=g, device=dev, dtype=dtype)
        return t if std == 1.0 else t.mul_(std)

    st = {"case": case}
    if case["op"] == "clip":
        # gradients live in one flat buffer of each type, so the tensors are parts of it
        sizes = _sizes(case)
        for name in ("bf16", "f32"):
            own_sizes = [s for i, s in enumerate(sizes) if _is_bf16(case, i) == (name == "bf16")]
            total = sum(-(-s // 8) * 8 for s in own_sizes)
            flat = torch.zeros(total, dtype=DTYPES[name], device=dev)
            st["flat_" + name], st["out_" + name] = flat, torch.zeros_like(flat)
            st["grads_" + name], st["outs_" + name] = _views(flat, own_sizes), _views(st["out_" + name], own_sizes)
            for i, t in enumerate(st["grads_" + name]):   # each tensor at a scale of its own, one in nine idle
                if i % 9 != 8:
                    t.copy_(normal(t.numel(), std=10.0 ** -(2 + i % 4), dtype=F32))
        st["grads"], st["outs"] = st["grads_bf16"] + st["grads_f32"], st["outs_bf16"] + st["outs_f32"]
        # the norm's expectation from the scales, so that the bound lies below it or far above
        expect = math.sqrt(sum(t.numel() * 10.0 ** -(2 * (2 + i % 4)) for n in ("bf16", "f32")
                               for i, t in enumerate(st["grads_" + n]) if i % 9 != 8) + 1e-12)
        st["max_norm"] = expect * (0.3 if case["clipped"] else 3.0)
        return st
    if case["op"] == "balance":
        S, T, E, K = case["seqs"], case["tokens"], case["E"], case["top_k"]
        st["logits"] = normal(S, T, E, dtype=F32).add_(normal(E, std=0.5, dtype=F32)).to(DTYPES[case["type"]])
        if E >= 16:   # the last expert is masked, as padding of a router's weight is
            st["logits"][..., E - 1] = -math.inf
        top = min(K, E - 1 if E >= 16 else E)
        st["ids"] = torch.full((S, T, K), -1, dtype=I32, device=dev)
        st["ids"][..., :top] = st["logits"].float().topk(top, dim=-1).indices.to(I32)
        st["num_tokens"] = None
        if case["ragged"]:
            st["num_tokens"] = torch.randint(T // 2, T + 1, (S,), generator=g, device=dev).to(I32)
        st["dlosses"] = torch.tensor([0.01, 0.001], dtype=F32, device=dev) if case["form"] == "train" else None
        return st
    rows, k, n, E = case["rows"], case["k"], case["n"], case["E"]
    two = 2 if case["act"] == "swiglu" else 1
    lead = (E,) if E else ()
    if E:
        hit = torch.multinomial(_popularity(case).to(dev), case["pairs"], replacement=True, generator=g)
        st["counts"] = torch.bincount(hit, minlength=E).clamp(max=rows).to(I32)
    st["x"] = normal(*lead, rows, k)
    st["codes"] = torch.randint(0, 256, (*lead, two * n, k // 2), generator=g, device=dev, dtype=torch.uint8)
    # of a size that keeps the product's rows near one: a code's mean square is about 21 (int4) or 9 (fp4)
    rms = 4.6 if case["kind"] == "int4" else 3.0
    spread = torch.rand(*lead, k // case["group"], two * n, generator=g, device=dev)
    st["scales"] = ((0.5 + spread) * (k ** -0.5 / rms)).to(BF16)
    st["bias"] = normal(*lead, two * n) if case["bias"] else None
    st["residual"] = normal(*lead, rows, n) if case["residual"] else None
    st["out"] = torch.zeros(*lead, rows, n, dtype=BF16, device=dev)
    return st


# -------------------------------------------------------------- the plain forms

def _plain_weight(st, case):
    """The weight in bf16 (a code's value times its group's scale, rounded once) as 32-bit numbers."""
    b = st["codes"]
    fields = torch.stack((b & 15, b >> 4), dim=-1).reshape(*b.shape[:-1], -1, 8)
    codes = fields[..., [FIELDS.index(e) for e in range(8)]].reshape(*b.shape[:-1], case["k"]).int()
    if case["kind"] == "int4":
        q = ((codes ^ 8) - 8).float()
    else:
        q = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=b.device)[codes]
    s = st["scales"].float().transpose(-1, -2).unsqueeze(-1)
    return (q.reshape(*s.shape[:-1], case["group"]) * s).reshape(q.shape).to(BF16).float()


def _plain_w4(st, case):
    z = torch.matmul(st["x"].float(), _plain_weight(st, case).transpose(-1, -2))
    if st["bias"] is not None:
        z = z + st["bias"].float().unsqueeze(-2)
    if case["act"] == "silu":
        y = z / (1 + torch.exp(-z))
    elif case["act"] == "gelu":
        y = 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    elif case["act"] == "swiglu":
        gate, up = z.chunk(2, dim=-1)
        y = gate / (1 + torch.exp(-gate)) * up
    else:
        y = z
    if st["residual"] is not None:
        y = y + st["residual"].float()
    y = y.to(BF16)
    if case["E"]:
        used = torch.arange(case["rows"], device=y.device) < st["counts"][:, None]
        y = torch.where(used[..., None], y, st["out"])
    return {"y": y}


def _plain_balance(st, case):
    S, T, E, K = case["seqs"], case["tokens"], case["E"], case["top_k"]
    z = st["logits"].float()
    dev = z.device
    length = torch.full((S,), T, device=dev) if st["num_tokens"] is None else st["num_tokens"]
    used = (torch.arange(T, device=dev) < length[:, None])[..., None]
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    soft, lse = e / total, top + torch.log(total)
    if case["score"] == "softmax":
        p = soft
    else:
        s = 1 / (1 + torch.exp(-z))
        p = s / s.sum(-1, keepdim=True)
    p = torch.where(used, p, 0.0)
    chosen = torch.where(used, st["ids"], -1).long()
    counts = torch.zeros(S, E + 1, dtype=I32, device=dev).scatter_add_(
        1, (chosen + 1).reshape(S, -1), torch.ones(S, T * K, dtype=I32, device=dev))[:, 1:]
    psum, n = p.sum(1), length.float()
    if not case["per_sequence"]:
        counts, psum, n = counts.sum(0, keepdim=True, dtype=I32), psum.sum(0, keepdim=True), n.sum(0, keepdim=True)
    n = n[:, None]
    some, many = n > 0, n.clamp(min=1)
    pools = some.sum().clamp(min=1)
    f = counts.float() * E / (K * many)
    all_tokens = length.sum().clamp(min=1)
    balance = torch.where(some, f * psum / many, 0.0).sum() / pools
    zloss = torch.where(used, lse * lse, 0.0).sum() / all_tokens
    out = {"losses": torch.stack((balance, zloss)), "counts": counts if case["per_sequence"] else counts[0]}
    if case["form"] == "train":
        g = torch.where(some, f / (many * pools), 0.0)[:, None]
        d = p * (g - (g * p).sum(-1, keepdim=True))
        if case["score"] == "sigmoid":
            d = d * (1 - s)
        d = st["dlosses"][0] * d + st["dlosses"][1] * 2 / all_tokens * lse * soft
        out["dlogits"] = torch.where(used, d, 0.0).to(st["logits"].dtype)
    return out


def _plain_clip(st, case):
    squares = torch.stack([t.float().square().sum() for t in st["grads"]])
    norm = squares.sum().sqrt()
    factor = torch.where(norm > st["max_norm"], st["max_norm"] / norm, 1.0)
    for out, t in zip(st["outs"], st["grads"]):
        out.copy_(t.float() * factor)
    return {"norm": norm, "bf16": st["out_bf16"], "f32": st["out_f32"]}


# --------------------------------------------------------------------- one pass

def _own(st, case):
    import combine_ep_route_gb300 as ep

    if case["op"] == "clip":
        norm = ep.clip_grad_norm(st["grads"], st["max_norm"], out=st["outs"])
        return {"norm": norm, "bf16": st["out_bf16"], "f32": st["out_f32"]}
    if case["op"] == "balance":
        kw = dict(score=case["score"], per_sequence=case["per_sequence"], num_tokens=st["num_tokens"])
        losses, counts = ep.balance_loss(st["logits"], st["ids"], **kw)
        out = {"losses": losses, "counts": counts}
        if case["form"] == "train":
            out["dlogits"] = ep.balance_loss_backward(st["dlosses"], st["logits"], counts, case["top_k"], **kw)
        return out
    kw = dict(kind=case["kind"], bias=st["bias"], act=case["act"], residual=st["residual"], out=st["out"])
    if case["E"]:
        return {"y": ep.experts_product_w4(st["x"], st["codes"], st["scales"], st["counts"], **kw)}
    return {"y": ep.linear_w4(st["x"], st["codes"], st["scales"], **kw)}


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"w4": _plain_w4, "balance": _plain_balance, "clip": _plain_clip}[case["op"]](state, case)


# ------------------------------------------------------------ what a pass needs

def work(case):
    if case["op"] == "clip":
        sizes = _sizes(case)
        # every gradient read once and written once
        return {"bytes": sum(2 * s * (2 if _is_bf16(case, i) else 4) for i, s in enumerate(sizes)), "flops": 3 * sum(sizes)}
    if case["op"] == "balance":
        E, size = case["E"], 2 if case["type"] == "bf16" else 4
        tokens = case["seqs"] * case["tokens"] * (0.75 if case["ragged"] else 1.0)
        b = tokens * (E * size + 4 * case["top_k"]) + 4 * E * (case["seqs"] if case["per_sequence"] else 1)
        f = tokens * E * 4
        if case["form"] == "train":
            b += case["seqs"] * case["tokens"] * E * size
            f += tokens * E * 6
        return {"bytes": b, "flops": f}
    rows, k, n, E = case["rows"], case["k"], case["n"], case["E"]
    wide = 2 * n if case["act"] == "swiglu" else n
    used, active = rows, 1
    if E:
        p = _popularity(case)
        used = float((case["pairs"] * p).clamp(max=rows).sum())
        active = float((1 - (1 - p) ** case["pairs"]).sum())
    b = active * wide * (k / 2 + 2 * k / case["group"]) + 2 * used * (k + n)
    b += (2 * active * wide if case["bias"] else 0) + (2 * used * n if case["residual"] else 0)
    return {"bytes": b, "flops": 2 * used * wide * k}


# ------------------------------------------------------------ 64-bit definitions

def _exact_weight(case, codes, scales):
    """One weight [rows, k]: element 8 i + e of a row lies in field FIELDS.index(e) of its i-th word."""
    nib = torch.empty(codes.shape[0], case["k"] // 8, 8, dtype=torch.long, device=codes.device)
    word = codes.view(codes.shape[0], case["k"] // 8, 4).long()
    for field, e in enumerate(FIELDS):
        nib[..., e] = (word[..., field // 2] >> (4 * (field % 2))) % 16
    nib = nib.view(codes.shape[0], case["k"])
    if case["kind"] == "int4":
        q = nib.double() - 16.0 * (nib > 7)
    else:
        mag, half = (nib % 8) // 2, (nib % 2).double()
        q = torch.where(mag == 0, half / 2, torch.exp2(mag.double() - 1) * (1 + half / 2)) * (1 - 2.0 * (nib > 7))
    return (q * scales.double().t().repeat_interleave(case["group"], dim=1)).to(BF16).double()


def _exact_w4(case, x, codes, scales, bias, residual):
    z = torch.einsum("rk,nk->rn", x.double(), _exact_weight(case, codes, scales))
    if bias is not None:
        z += bias.double()
    if case["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif case["act"] == "gelu":
        z = z * 0.5 * torch.erfc(-z / math.sqrt(2))
    elif case["act"] == "swiglu":
        n = case["n"]
        z = z[:, :n] * torch.sigmoid(z[:, :n]) * z[:, n:]
    return z if residual is None else z + residual.double()


def _exact_balance(case, st):
    S, T, E, K = case["seqs"], case["tokens"], case["E"], case["top_k"]
    train = case["form"] == "train"
    length = [T] * S if st["num_tokens"] is None else st["num_tokens"].tolist()
    z = st["logits"].double().requires_grad_(train)
    soft = torch.log_softmax(z, -1)
    p = soft.exp()
    if case["score"] == "sigmoid":
        p = torch.sigmoid(z) / torch.sigmoid(z).sum(-1, keepdim=True)
    groups = [[s] for s in range(S)] if case["per_sequence"] else [list(range(S))]
    groups = [g for g in groups if sum(length[s] for s in g) > 0]
    balance = z.new_zeros(())
    for g in groups:
        n = sum(length[s] for s in g)
        c = torch.bincount(torch.cat([st["ids"][s, :length[s]].reshape(-1) for s in g]).long() + 1, minlength=E + 1)[1:]
        mean = torch.stack([p[s, :length[s]].sum(0) for s in g]).sum(0) / n
        balance = balance + (c.double() * E / (K * n) * mean).sum() / len(groups)
    lse = torch.logsumexp(z, -1)
    zloss = torch.stack([lse[s, :length[s]].square().sum() for s in range(S)]).sum() / max(1, sum(length))
    out = {"losses": torch.stack((balance, zloss)).detach(), "counts": None}
    if train:
        d = st["dlosses"].double()
        out["dlogits"], = torch.autograd.grad(d[0] * balance + d[1] * zloss, z)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        norm = torch.stack([torch.linalg.vector_norm(t.double()) for t in st["grads"]])
        norm = torch.linalg.vector_norm(norm)
        factor = min(1.0, st["max_norm"] / max(float(norm), 1e-300))
        return {"norm": norm, "bf16": st["flat_bf16"].double() * factor, "f32": st["flat_f32"].double() * factor}
    if case["op"] == "balance":
        return _exact_balance(case, st)
    if not case["E"]:
        return {"y": _exact_w4(case, st["x"], st["codes"], st["scales"], st["bias"], st["residual"])}
    y = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for e, c in enumerate(st["counts"].tolist()):
        if c:
            y[e, :c] = _exact_w4(case, st["x"][e, :c], st["codes"][e], st["scales"][e],
                                 None if st["bias"] is None else st["bias"][e],
                                 None if st["residual"] is None else st["residual"][e, :c])
    return {"y": y}
