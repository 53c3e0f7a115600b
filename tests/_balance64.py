"""The balance and z losses of a router in 64 bits, from their definition, differentiable in
the logits; the counts are held fixed."""
import torch

D = torch.float64


def scores(z, score):
    """(probabilities, logsumexp) of 64-bit logits [..., E]; infinite and NaN ones take no part,
    and a token without any other has neither."""
    left = torch.isfinite(z)
    some = left.any(-1, keepdim=True)
    z = torch.where(left, z, torch.full_like(z, -1e30))
    top = z.detach().amax(-1, keepdim=True)
    e = torch.where(left, torch.exp(z - top), torch.zeros_like(z))
    total = torch.where(some, e.sum(-1, keepdim=True), torch.ones_like(top))
    lse = torch.where(some, top + torch.log(total), torch.zeros_like(top))[..., 0]
    if score == "softmax":
        return e / total, lse
    logs = torch.nn.functional.logsigmoid(z)   # by logarithms: the sigmoids may all underflow
    s = torch.where(left, torch.exp(logs - logs.detach().amax(-1, keepdim=True)), torch.zeros_like(z))
    return s / torch.where(some, s.sum(-1, keepdim=True), torch.ones_like(top)), lse


def pools_of(z, per_sequence, lengths):
    """Index tensors of each pool's tokens in use, for logits [S, T, E]."""
    S, T = z.shape[:2]
    lengths = [T] * S if lengths is None else [max(0, min(int(n), T)) for n in lengths]
    rows = [torch.arange(n) + s * T for s, n in enumerate(lengths)]
    return rows if per_sequence else [torch.cat(rows) if rows else torch.empty(0, dtype=torch.long)]


def losses(z, ids, score, per_sequence, lengths):
    """(balance, z loss, counts [pools, E]) of 64-bit logits [S, T, E] and ids [S, T, K]."""
    S, T, E = z.shape
    K = ids.shape[-1]
    p, lse = scores(z, score)
    p, lse, ids = p.reshape(-1, E), lse.reshape(-1), ids.reshape(-1, K).long()
    pools = pools_of(z, per_sequence, lengths)
    counts = torch.zeros(len(pools), E, dtype=torch.long)
    balance = z.new_zeros(())
    for i, rows in enumerate(pools):
        own = ids[rows].reshape(-1)
        own = own[(own >= 0) & (own < E)]
        counts[i] = torch.bincount(own, minlength=E)
        if len(rows):
            balance = balance + (counts[i].to(D) * E / (K * len(rows)) * p[rows].mean(0)).sum()
    some = sum(1 for rows in pools if len(rows))
    rows = torch.cat(pools) if pools else torch.empty(0, dtype=torch.long)
    zloss = lse[rows].square().mean() if len(rows) else z.sum() * 0
    return balance / max(1, some), zloss, counts
