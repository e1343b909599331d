"""A trainable mixture-of-experts block from the library's calls:

    h      = layernorm(x)
    logits = h Wr^T                               (fp32, the router's projection)
    idx, g = topk_gate(logits);  loss = balance_loss(logits, idx)
    routed = combine(experts(dispatch(h)), g)     (capacity layout [e, c, m])
    y      = act(h W1^T + b1) W2^T + b2 + x + routed   (the shared expert; x joins in the epilogue)

A capacity layout puts expert j's rows at [j c, (j + 1) c), known on the host,
so each expert's two products are calls of ``linear`` on its slice.

``python -m combine_moe_topk_gb300.block`` trains it for some steps on a
synthetic target (needs a GPU).
"""
from __future__ import annotations

import math

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


def main(steps: int = 20):
    torch.manual_seed(0)
    s, m = 1024, 512
    block = MoEBlock(m, e=8, k=2, d_expert=1024, d_shared=1024)
    x = torch.randn(s, m, device="cuda").bfloat16()
    target = torch.randn(s, m, device="cuda")
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    for step in range(steps):
        y, aux, counts = block(x)
        loss = (y.float() - target).square().mean() + aux
        opt.zero_grad()
        loss.backward()
        opt.step()
        if A.status():
            raise RuntimeError("a kernel of this step reported a time-out, a NaN or a bad route")
        print(f"step {step}: loss {loss.item():.4f} (auxiliary {aux.item():.4f}), routes per expert {counts[0].tolist()}")


if __name__ == "__main__":
    main()
