"""A Mixture-of-Experts layer on the framework's operators, forward and backward.

    out[t] = sum_k w_k expert_{id_k}(x[t]) + shared(x[t])

with a top-k router, gated experts w2 (silu(w_gate x) * (w_up x)) reached through
dispatch and combine, and a dense shared expert whose second product adds the routed
sum as its residual. Tokens are held as [W, T, h], one block per simulated rank.

The backward pass goes the same way back: the output's gradient is dispatched to the
rows the experts wrote, and the gradients of the rows the experts read are combined
with unit weights.

    python examples/moe_layer.py            # times a forward and a backward pass
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_ep_route_gb300 as ep  # noqa: E402

BF16 = torch.bfloat16


class MoeLayer:
    def __init__(self, cfg: ep.EpConfig, inner: int, shared: int, seed: int = 0, device="cuda:0"):
        self.cfg, self.device = cfg, torch.device(device)
        g = torch.Generator(device=self.device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=self.device) * shape[-1] ** -0.5).to(BF16)

        h = cfg.hidden
        self.router = weight(cfg.E, h)
        self.w13, self.w2 = weight(cfg.W, cfg.e_local, 2 * inner, h), weight(cfg.W, cfg.e_local, h, inner)
        self.s1, self.b1, self.s2 = weight(shared, h), weight(1, shared)[0], weight(h, shared)
        self.ctx, self.back = ep.EpContext(cfg, self.device), ep.EpContext(cfg, self.device)
        # the device-side status of the products: 0, or the code of a wait that ran out
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        c, st = self.cfg, self.status
        self.x = x
        self.logits = ep.linear(x, self.router, out_dtype=torch.float32, status=st)
        self.ids, weights = ep.route_topk(self.logits, c.top_k)
        d = self.ctx.dispatch(x, self.ids, weights)
        self.rows, self.counts = d.b_a1, d.expert_num_tokens
        self.z = torch.empty(*d.b_a1.shape[:-1], self.w13.shape[-2], dtype=BF16, device=self.device)
        self.hidden = ep.experts_product(self.rows, self.w13, self.counts, act="swiglu", preact=self.z, status=st)
        self.y = ep.experts_product(self.hidden, self.w2, self.counts, status=st)
        # combine ends the dispatch: what the backward pass needs of its map is copied first
        meta = self.ctx.metadata()
        self.pair_row, self.pair_w = meta["pair_row"].long().clone(), meta["pair_w"].clone()
        routed = self.ctx.combine(self.y)
        self.zs = torch.empty(*x.shape[:-1], self.s1.shape[0], dtype=BF16, device=self.device)
        self.shared = ep.linear(x, self.s1, bias=self.b1, act="gelu", preact=self.zs, status=st)
        return ep.linear(self.shared, self.s2, residual=routed, status=st)

    def backward(self, dout: torch.Tensor) -> dict:
        c, st, grads = self.cfg, self.status, {}
        # the shared expert
        grads["s2"] = ep.linear_wgrad(dout, self.shared, status=st)
        dzs = ep.linear_dgrad(dout, self.s2, act="gelu", preact=self.zs, status=st)
        grads["s1"], grads["b1"] = ep.linear_wgrad(dzs, self.x, bias_grad=True, status=st)
        dx = ep.linear_dgrad(dzs, self.s1, out_dtype=torch.float32, status=st)
        # the routed experts: dout's rows where the experts' outputs lie, times their weights
        ones = torch.ones_like(self.pair_w)
        dy = self.back.dispatch(dout, self.ids, ones).b_a1
        kept = self.pair_row >= 0
        row_w = torch.zeros(dy[..., 0].numel(), device=self.device)
        row_w[self.pair_row[kept]] = self.pair_w[kept]
        dy *= row_w.view(dy.shape[:-1])[..., None]
        grads["w2"] = ep.experts_product_wgrad(dy, self.hidden, self.counts, status=st)
        dz = ep.experts_product_dgrad(dy, self.w2, self.counts, act="swiglu", preact=self.z, status=st)
        grads["w13"] = ep.experts_product_wgrad(dz, self.rows, self.counts, status=st)
        drows = ep.experts_product_dgrad(dz, self.w13, self.counts, status=st)
        dx += self.back.combine(drows, out_dtype=torch.float32)
        # the router: each weight's gradient is its expert's output along dout
        picked = self.y.view(-1, c.hidden)[self.pair_row.clamp(min=0)]
        dw = (picked.float() * dout[..., None, :].float()).sum(-1) * kept
        dlogits = ep.route_topk_backward(dw, self.logits, self.ids).to(BF16)
        grads["router"] = ep.linear_wgrad(dlogits, self.x, status=st)
        dx += ep.linear_dgrad(dlogits, self.router, out_dtype=torch.float32, status=st)
        grads["x"] = dx
        return grads

    def check(self) -> None:
        """Raises what the kernels reported (synchronises)."""
        self.ctx.check()
        self.back.check()
        if int(self.status.item()):
            raise ep.EpError(int(self.status.item()), "products")


def main() -> None:
    cfg = ep.EpConfig(W=8, E=64, top_k=8, max_tokens=128, hidden=2048)
    layer = MoeLayer(cfg, inner=1024, shared=4096)
    x, dout = (torch.randn(cfg.W, cfg.max_tokens, cfg.hidden, device=layer.device).to(BF16) for _ in range(2))

    def timed(name, f):
        for _ in range(3):
            f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(20):
            f()
        b.record()
        torch.cuda.synchronize()
        print(f"{name}: {a.elapsed_time(b) / 20 * 1e3:.0f} us for {cfg.W * cfg.max_tokens} tokens")

    timed("forward", lambda: layer.forward(x))
    timed("backward", lambda: layer.backward(dout))
    layer.check()


if __name__ == "__main__":
    main()
