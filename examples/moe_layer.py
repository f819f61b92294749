"""One training step of a mixture-of-experts layer, and one decode step, over this
package's operators: the router's projection, the router with its balance loss,
dispatch into the packed per-expert layout, the gated experts, the weighted
combine, and their gradients. Between them, the backward pass takes torch's
elementwise operations for the gradient of combine's weights and for the rows
that it scales by them.

    python examples/moe_layer.py            # prints the loss falling over a few steps

Shapes follow the package's tensors: [R, T, ...] for R simulated expert-parallel
ranks of T tokens, experts of rank r numbered r * E_r .. (r + 1) * E_r - 1. The
routing groups are the ranks' experts, so that a token travels to at most
`topk_groups` ranks.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_route_layout_gb300 import (  # noqa: E402
    EpDispatchCombineConfig, EpDispatchCombineOp, EpLinearConfig, EpLinearOp, EpRouterConfig, EpRouterOp)


class MoeLayer:
    """y_t = sum over the token's experts e of w_te down_e(swiglu(up_e x_t))."""

    def __init__(self, ranks, tokens, hidden, inner, experts_per_rank, topk, topk_groups, device="cuda", seed=0):
        self.R, self.T, self.H, self.I = ranks, tokens, hidden, inner
        self.E_r, self.E, self.k = experts_per_rank, ranks * experts_per_rank, topk
        self.n = ranks * tokens
        bf16 = torch.bfloat16
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return torch.randn(shape, generator=gen, device=device).mul_(shape[-1] ** -0.5).to(bf16)

        self.w_gate = weight(1, self.E, hidden)
        self.w_up = weight(self.E, 2 * inner, hidden)
        self.w_down = weight(self.E, hidden, inner)
        self.gate = EpLinearOp(EpLinearConfig(1, hidden, self.E, self.n, out_dtype=torch.float32,
                                              weight_grad_dtype=torch.float32), device, backward=True)
        self.router = EpRouterOp(EpRouterConfig(
            ranks, tokens, self.E, topk, score_func="sigmoid", num_groups=ranks, topk_groups=topk_groups,
            route_scale=1.0, balance_coef=0.01), device)

        def exchange(weighted):
            return EpDispatchCombineOp(EpDispatchCombineConfig(
                bf16, ranks, hidden, 0, 4, 4, tokens, experts_per_rank, topk, standard_moe=True,
                combine_out_dtype=torch.float32, weighted_combine=weighted), device)

        self.exchange = exchange(True)     # tokens to the experts, and their weighted sum back
        self.back = exchange(False)        # gradients to the experts, and their plain sum back
        pool = ranks * tokens * topk + 127 * self.E
        self.up = EpLinearOp(EpLinearConfig(self.E, hidden, inner, pool, activation="swiglu",
                                            groups_per_base=experts_per_rank), device, backward=True)
        self.down = EpLinearOp(EpLinearConfig(self.E, inner, hidden, pool, groups_per_base=experts_per_rank),
                               device, backward=True)
        # rows of no expert are never written: one buffer each, zeroed once
        self.z = torch.zeros((pool, 2 * inner), dtype=bf16, device=device)
        self.h, self.dh = (torch.zeros((pool, inner), dtype=bf16, device=device) for _ in range(2))
        self.y, self.dx = (torch.zeros((pool, hidden), dtype=bf16, device=device) for _ in range(2))

    def forward(self, x, num_tokens=None, balance=False):
        """y [R, T, H] f32 (and the balance loss) of x [R, T, H] bf16."""
        logits = self.gate.forward(x.view(self.n, self.H), self.w_gate).view(self.R, self.T, self.E)
        routed = self.router.forward(logits, num_tokens=num_tokens, balance=balance)
        weights, indices = routed[:2]
        packed = self.exchange.dispatch_standard_moe(x, weights, None, indices, num_tokens=num_tokens)
        at = {"row_begin": packed["expert_offset"], "row_count": packed["packed_recv_count"],
              "row_base": packed["rank_base"]}
        rows = packed["packed_recv_x"]
        self.up.forward(rows, self.w_up, out=self.h, preact=self.z, **at)
        self.down.forward(self.h, self.w_down, out=self.y, **at)
        out = self.exchange.combine_standard_moe(self.y, weights, indices, call_reset=True)
        self.saved = (x, num_tokens, logits, weights, indices, rows, packed["packed_recv_src_info"], at)
        self.counts = routed[2] if balance else None
        return (out, routed[3]) if balance else out

    def backward(self, dy, d_loss=None):
        """Gradients of (w_gate, w_up, w_down) and of x, from dy [R, T, H] f32 and, with
        balance, the f32 scalar gradient of the loss. Call once after each forward."""
        x, num_tokens, logits, weights, indices, rows, source, at = self.saved
        # each token's dy to its experts' rows, in the rows of the forward's layout
        there = self.back.dispatch_standard_moe(dy.to(torch.bfloat16), weights, None, indices, num_tokens=num_tokens)
        dy_rows = there["packed_recv_x"]
        token, slot = self._slots_of_rows(indices, source, at)
        held = token >= 0
        w_rows = torch.where(held, weights.view(self.n, self.k)[token.clamp(min=0), slot], 0.0)
        dot = torch.where(held, (dy_rows.float() * self.y.float()).sum(-1), 0.0)
        d_weights = torch.zeros((self.n, self.k), device=dy.device)
        d_weights.index_put_((token.clamp(min=0), slot), dot, accumulate=True)
        d_rows = torch.where(held[:, None], dy_rows * w_rows[:, None], 0.0).to(torch.bfloat16)
        _, d_down, _ = self.down.backward(d_rows, self.h, self.w_down, dx=self.dh, **at)
        _, d_up, _ = self.up.backward(self.dh, rows, self.w_up, self.z, dx=self.dx, **at)
        d_x = self.back.combine_standard_moe(self.dx, None, indices, call_reset=True)
        d_logits = self.router.backward(logits, indices, d_weights=d_weights.view_as(weights),
                                        counts=self.counts, d_loss=d_loss, num_tokens=num_tokens)
        d_in, d_gate, _ = self.gate.backward(d_logits.view(self.n, self.E), x.view(self.n, self.H), self.w_gate)
        return d_gate, d_up, d_down, d_x + d_in.view_as(d_x)

    def _slots_of_rows(self, indices, source, at):
        """Token (r * T + t, -1 on rows of nobody) and top-k slot of each pool row."""
        pool = source.numel()
        begin = (at["row_base"].view(-1, 1) + at["row_begin"].view(self.R, self.E_r)).view(-1).long()
        count = at["row_count"].view(-1).long()
        row = torch.arange(pool, device=source.device)
        expert = (torch.searchsorted(begin, row, right=True) - 1).clamp(min=0)
        held = row < begin[expert] + count[expert]
        rank, t = source.long() // (self.R * self.T), source.long() % (self.R * self.T)
        token = torch.where(held, rank * self.T + t, -1)
        of = indices.view(self.n, self.k)[token.clamp(min=0)]
        slot = (of == expert[:, None]).int().argmax(-1)
        return token, slot

    def sync(self):
        for op in (self.gate, self.router, self.exchange, self.back, self.up, self.down):
            op.sync()


def train(steps=8, ranks=4, tokens=64, hidden=256, inner=128, experts_per_rank=4, topk=4, topk_groups=2, lr=0.05):
    """Fit the layer to a fixed random map; returns the losses."""
    layer = MoeLayer(ranks, tokens, hidden, inner, experts_per_rank, topk, topk_groups)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((ranks, tokens, hidden), generator=gen, device="cuda").bfloat16()
    want = torch.randn((ranks, tokens, hidden), generator=gen, device="cuda")
    master = [w.float() for w in (layer.w_gate, layer.w_up, layer.w_down)]
    one = torch.ones((), device="cuda")
    losses = []
    for _ in range(steps):
        y, balance = layer.forward(x, balance=True)
        losses.append(float(0.5 * (y - want).square().mean(-1).sum() / layer.n + balance))
        grads = layer.backward((y - want) / (hidden * layer.n), one)
        for w, m, g in zip((layer.w_gate, layer.w_up, layer.w_down), master, grads):
            m.sub_(g.float().div_(g.float().norm() + 1e-12), alpha=lr * float(m.norm()))
            w.copy_(m)
    layer.sync()
    return losses


if __name__ == "__main__":
    for i, loss in enumerate(train()):
        print(f"step {i}: loss {loss:.4f}")
    decode = MoeLayer(4, 1, 256, 128, 4, 4, 2)
    print("one token a rank:", tuple(decode.forward(torch.randn((4, 1, 256), device="cuda").bfloat16()).shape))
    decode.sync()
