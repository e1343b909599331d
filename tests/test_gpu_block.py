"""The MoE block that strings the calls together, against plain torch in 64
bits on the same weights and routes: outputs, losses and every gradient.

Activations and their gradients are rounded to bf16 between the calls, at most
eight times on the longest path (h, logits' gradient, X, u, z, Y, routed, y and
their duals), each by up to 2^-9 of a value in the mean: 8 * 2^-9 = 1.6 % of
a result's 2-norm bounds them all (independent roundings add to far less)."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B
from combine_moe_topk_gb300.block import MoEBlock

pytestmark = pytest.mark.gpu
TOL = 8 * 2.0 ** -9


def reference(block, x, idx, row, valid, offsets):
    """The block in float64 with autograd; returns (y, aux, parameters)."""
    P = {n: p.detach().double().requires_grad_() for n, p in block.named_parameters()}
    x = x.detach().double().requires_grad_()
    mean = x.mean(1, keepdim=True)
    h = (x - mean) / ((x - mean).square().mean(1, keepdim=True) + 1e-5).sqrt() * P["norm_w"] + P["norm_b"]
    logits = h @ P["router"].t()
    p = torch.softmax(logits, 1)
    gate = torch.softmax(logits.gather(1, idx.long()), 1)
    lse = torch.logsumexp(logits, 1)
    live = valid.bool()
    terms = []
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        at = live[lo:hi]
        n = int(at.sum())
        if n:
            f = torch.bincount(idx[lo:hi][at].reshape(-1).long(), minlength=block.e).double() / (block.k * n)
            terms.append(block.e * (f * p[lo:hi][at].mean(0)).sum())
    aux = block.weights[0] * sum(terms) / len(terms) + block.weights[1] * lse[live].square().mean()
    act = torch.nn.functional.gelu
    routed = torch.zeros_like(x)
    for j in range(block.e):
        out = act(h @ P["up"][j].t() + P["up_b"][j]) @ P["down"][j].t()
        for q in range(block.k):
            here = ((idx[:, q] == j) & (row[:, q] >= 0)).double()[:, None]
            routed = routed + here * gate[:, q:q + 1] * out
    y = act(h @ P["shared_up"].t() + P["shared_up_b"]) @ P["shared_down"].t() + P["shared_down_b"] + x + routed
    return y, aux, P, x


def test_block_outputs_and_gradients():
    s, m, e, k = 300, 256, 4, 2
    block = MoEBlock(m, e, k, d_expert=192, d_shared=320, capacity_factor=1.0, seed=1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(s, m, generator=g).bfloat16().cuda().requires_grad_()
    dy = torch.randn(s, m, generator=g).cuda()
    valid = (torch.rand(s, generator=g) < 0.9).to(torch.uint8).cuda()
    offsets = [0, 120, 120, 300]
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    y, aux, counts = block(x, valid, off)
    (y.float() * dy).sum().add(100.0 * aux).backward()
    with torch.no_grad():
        logits = B.moe_linear(B.moe_layernorm(x.detach(), block.norm_w, block.norm_b, stats=False), block.router,
                              out_dtype=torch.float32)
        idx, _ = B.moe_topk_gate(logits, k)
    row = B.moe_dispatch_layout(idx, e, B.moe_capacity(1.0, s, k, e)).row()
    assert (row < 0).any(), "some routes should be dropped here"
    ry, raux, P, rx = reference(block, x, idx, row, valid, offsets)
    (ry * dy.double()).sum().add(100.0 * raux).backward()

    def off_by(a, b):
        return float(((a.detach().double() - b.detach()).norm() / b.detach().norm()).item())

    assert off_by(y, ry) <= TOL
    assert abs(aux.item() - raux.item()) <= 0.01 * raux.item()
    assert counts.sum().item() == int(valid.sum()) * k and not counts[1].any()
    errs = {"x": off_by(x.grad, rx.grad)}
    for n, p in block.named_parameters():
        errs[n] = off_by(p.grad, P[n].grad)
    assert all(v <= TOL for v in errs.values()), errs


def test_block_learns():
    torch.manual_seed(0)
    block = MoEBlock(128, e=4, k=2, d_expert=256, d_shared=256, seed=3)
    x = torch.randn(512, 128, device="cuda").bfloat16()
    target = torch.randn(512, 128, device="cuda")
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    losses = []
    for _ in range(15):
        y, aux, _ = block(x)
        loss = (y.float() - target).square().mean() + aux
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    assert losses[-1] < 0.8 * losses[0], losses


def test_autograd_wrappers_return_what_was_asked_for():
    x = torch.randn(40, 64, device="cuda").bfloat16()
    W = torch.randn(24, 64, device="cuda").bfloat16().requires_grad_()
    r = torch.randn(40, 24, device="cuda").requires_grad_()
    A.linear(x, W, None, "silu", r).sum().backward()
    assert W.grad is not None and x.grad is None and torch.equal(r.grad, torch.ones_like(r))
    w = torch.ones(64, device="cuda").bfloat16().requires_grad_()
    A.layernorm(x, w).sum().backward()
    assert w.grad.dtype == torch.bfloat16
    # a concatenation's gradient: views that start off 16 bytes
    a, c = (torch.randn(3, 7, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    torch.cat([A.layernorm(a), A.layernorm(c)]).float().square().sum().backward()
    assert torch.isfinite(c.grad).all()
    W3 = torch.randn(5, 64, device="cuda").bfloat16().requires_grad_()
    torch.cat([A.linear(x[:3], W3, act="silu"), A.linear(x[3:8], W3, act="silu")]).float().sum().backward()
    assert torch.isfinite(W3.grad).all()
    # a broadcast upstream gradient (stride 0) reaches the kernels as rows of their own
    xx = x.clone().requires_grad_()
    A.layernorm(xx, w).mean(0).sum().backward()
    assert np.isfinite(xx.grad.float().cpu().numpy()).all()
