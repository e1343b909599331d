"""Trainable mixture-of-experts blocks from the library's calls.

MoEBlock, experts of two dense products in capacity slots:

    h      = layernorm(x)
    logits = h Wr^T                               (fp32, the router's projection)
    idx, g = topk_gate(logits);  loss = balance_loss(logits, idx)
    routed = combine(experts(dispatch(h)), g)     (capacity layout [e, c, m])
    y      = act(h W1^T + b1) W2^T + b2 + x + routed   (the shared expert; x joins in the epilogue)

A capacity layout puts expert j's rows at [j c, (j + 1) c), known on the host,
so each expert's two products are calls of ``linear`` on its slice.

GatedMoEBlock, gated experts without capacity, each step of theirs one call
over all of them:

    X = dispatch(h);  H = act(X Wg^T) * (X Wu^T);  Y = H Wd^T   (each expert's own W, over its rows)
    y = (act(h Sg^T) * (h Su^T)) Sd^T + x + combine(Y, g)       (the shared expert, gated too)

``python -m combine_moe_topk_gb300.block [gated]`` trains one for some steps
on a synthetic target (needs a GPU).
"""
from __future__ import annotations

import math
import sys

import torch

from . import autograd as A
from . import binding as B


class MoEBlock(torch.nn.Module):
    """x bf16 [s, m] -> (y bf16 [s, m], auxiliary loss, counts i32 [num_seqs, e])."""

    def __init__(self, m: int, e: int, k: int, d_expert: int, d_shared: int, capacity_factor: float = 1.25,
                 act: str = "gelu", balance: float = 1e-2, z_loss: float = 1e-3, seed: int = 0, device="cuda"):
        super().__init__()
        self.e, self.k, self.capacity_factor, self.act = e, k, capacity_factor, act
        self.weights = (balance, z_loss)
        g = torch.Generator().manual_seed(seed)

        def mat(*shape):
            w = torch.randn(*shape, generator=g) / math.sqrt(shape[-1])
            return torch.nn.Parameter(w.to(device=device, dtype=torch.bfloat16))

        def vec(n, value):
            return torch.nn.Parameter(torch.full((n,), value, device=device))

        self.norm_w, self.norm_b = vec(m, 1.0), vec(m, 0.0)
        self.router = mat(e, m)
        self.up, self.down = mat(e, d_expert, m), mat(e, m, d_expert)
        self.up_b = torch.nn.Parameter(torch.zeros(e, d_expert, device=device))
        self.shared_up, self.shared_down = mat(d_shared, m), mat(m, d_shared)
        self.shared_up_b, self.shared_down_b = vec(d_shared, 0.0), vec(m, 0.0)

    def forward(self, x: torch.Tensor, valid: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None,
                topk_idx: torch.Tensor | None = None):
        """valid, seq_offsets: see ``balance_loss`` (padding is left out of the losses; it is routed, and takes up
        capacity, like any other token); topk_idx: routes to take instead of the gate's own choice
        (replay), their gates still the softmax over the chosen logits."""
        h = A.layernorm(x, self.norm_w, self.norm_b)
        logits = A.linear(h, self.router, out_dtype=torch.float32)
        if topk_idx is None:
            idx, gate = A.topk_gate(logits, self.k)
        else:
            idx = topk_idx
            gate = torch.softmax(logits.gather(1, idx.long()), 1)
        loss, counts, _ = A.balance_loss(logits, idx, valid, seq_offsets)
        c = max(1, B.moe_capacity(self.capacity_factor, x.shape[0], self.k, self.e))
        handle = B.moe_dispatch_layout(idx, self.e, c)
        X = A.dispatch(h, handle)
        rows = []
        for j in range(self.e):
            u = A.linear(X[j * c:(j + 1) * c], self.up[j], self.up_b[j], self.act)
            rows.append(A.linear(u, self.down[j]))
        routed = A.combine(torch.cat(rows), gate, handle)
        u = A.linear(h, self.shared_up, self.shared_up_b, self.act)
        y = A.linear(u, self.shared_down, self.shared_down_b, residual=x) + routed
        return y, self.weights[0] * loss[0] + self.weights[1] * loss[1], counts


class GatedMoEBlock(torch.nn.Module):
    """x bf16 [s, m] -> (y bf16 [s, m], auxiliary loss, counts i32 [num_seqs, e]); no route is dropped.
    gather: the experts' first product takes the token rows itself (less memory, one more dispatch backward)."""

    def __init__(self, m: int, e: int, k: int, d_expert: int, d_shared: int, act: str = "silu", balance: float = 1e-2,
                 z_loss: float = 1e-3, gather: bool = False, seed: int = 0, device="cuda"):
        super().__init__()
        self.e, self.k, self.act, self.gather = e, k, act, gather
        self.weights = (balance, z_loss)
        g = torch.Generator().manual_seed(seed)

        def mat(*shape):
            w = torch.randn(*shape, generator=g) / math.sqrt(shape[-1])
            return torch.nn.Parameter(w.to(device=device, dtype=torch.bfloat16))

        self.norm_w = torch.nn.Parameter(torch.ones(m, device=device))
        self.norm_b = torch.nn.Parameter(torch.zeros(m, device=device))
        self.router = mat(e, m)
        self.up, self.down = mat(e, 2 * d_expert, m), mat(e, m, d_expert)  # up: an expert's gate rows, then the factor's
        self.shared_up, self.shared_down = mat(2 * d_shared, m), mat(m, d_shared)

    def forward(self, x: torch.Tensor, valid: torch.Tensor | None = None, seq_offsets: torch.Tensor | None = None):
        h = A.layernorm(x, self.norm_w, self.norm_b)
        logits = A.linear(h, self.router, out_dtype=torch.float32)
        idx, gate = A.topk_gate(logits, self.k)
        loss, counts, _ = A.balance_loss(logits, idx, valid, seq_offsets)
        handle = B.moe_dispatch_layout(idx, self.e, 0)
        if self.gather:
            H = A.dispatch_grouped_gated(h, self.up, handle, self.act)
        else:
            H = A.grouped_gated(A.dispatch(h, handle), self.up, handle, self.act)
        routed = A.combine(A.grouped_gemm(H, self.down, handle), gate, handle)
        y = A.linear(A.gated_linear(h, self.shared_up, act=self.act), self.shared_down, residual=x) + routed
        return y, self.weights[0] * loss[0] + self.weights[1] * loss[1], counts


def main(steps: int = 20, gated: bool = False):
    torch.manual_seed(0)
    s, m = 1024, 512
    block = GatedMoEBlock(m, e=8, k=2, d_expert=704, d_shared=704) if gated else MoEBlock(m, e=8, k=2, d_expert=1024, d_shared=1024)
    x = torch.randn(s, m, device="cuda").bfloat16()
    target = torch.randn(s, m, device="cuda")
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    for step in range(steps):
        y, aux, counts = block(x)
        loss = (y.float() - target).square().mean() + aux
        opt.zero_grad()
        loss.backward()
        norm = A.clip_grad_norm(block.parameters(), 1.0) if gated else None
        opt.step()
        if A.status():
            raise RuntimeError("a kernel of this step reported a time-out, a NaN or a bad route")
        print(f"step {step}: loss {loss.item():.4f} (auxiliary {aux.item():.4f}), routes per expert {counts[0].tolist()}" +
              (f", gradient norm {norm.item():.4f}" if gated else ""))


if __name__ == "__main__":
    main(gated="gated" in sys.argv[1:])
