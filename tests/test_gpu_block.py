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


@pytest.mark.parametrize("s,e,k", [(300, 8, 2), (2048, 64, 6), (40, 128, 8)])
def test_whole_chain_in_a_graph_equals_calls_one_by_one(s, e, k):
    """Every call of a block's forward and backward back to back in a captured graph, replayed on new inputs,
    against the same calls with the device idle between them: no kernel reads before its forerunner has written."""
    m = 256
    g = torch.Generator().manual_seed(5)
    mk = lambda *shape: torch.randn(*shape, generator=g).bfloat16().cuda()  # noqa: E731
    x, dy, Wr, W1, W2 = mk(s, m), mk(s, m), mk(e, m) * 0.1, mk(384, m) * 0.06, mk(m, 384) * 0.05
    nw, nb = torch.ones(m, device="cuda"), torch.zeros(m, device="cuda")
    dloss = torch.tensor([0.1, 0.01], device="cuda")
    cap = B.moe_capacity(1.25, s, k, e)
    h_graph, h_eager = (B.moe_layout_create(s, e, k, capacity=cap) for _ in range(2))

    def chain(handle, wait):
        out = []

        def do(r):
            out.extend(t for t in (r if isinstance(r, tuple) else (r,)) if torch.is_tensor(t))
            if wait:
                torch.cuda.synchronize()
            return r

        hn, mean, rstd = do(B.moe_layernorm(x, nw, nb))
        logits = do(B.moe_linear(hn, Wr, out_dtype=torch.float32))
        idx, gate = do(B.moe_topk_gate_layout(handle, logits))
        bl = do(B.moe_balance_loss(logits, idx))
        X = do(B.moe_dispatch(handle, hn))
        routed = do(B.moe_combine(handle, X, gate))
        u, z = do(B.moe_linear(hn, W1, act="silu", save_z=True))
        do(B.moe_linear(u, W2, residual=routed))
        dY, dgate = do(B.moe_combine_bwd(handle, dy, gate, X))
        dl = do(B.moe_topk_gate_bwd(logits, idx, gate, dgate, e))
        dl = do(B.moe_balance_loss_bwd(logits, bl.lse, bl.coef, bl.norm, dloss, add=dl))
        dh0 = do(B.moe_dispatch_bwd(handle, dY))
        du, _, _ = do(B.moe_linear_bwd(dy, u, W2))
        do(B.moe_linear_bwd(du, hn, W1, z, "silu"))
        do(B.moe_linear_bwd(dl, hn, Wr))
        do(B.moe_layernorm_bwd(dh0, x, nw, mean, rstd, dres=dy))
        return out

    chain(h_graph, True)  # one-time set-up before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(h_graph, False)
    for seed in range(4):
        x.copy_(torch.randn(s, m, generator=torch.Generator().manual_seed(50 + seed)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in got]
        want = chain(h_eager, True)
        assert len(have) == len(want)
        for i, (a, c) in enumerate(zip(have, want)):
            assert torch.equal(a, c), i
