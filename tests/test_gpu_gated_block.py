"""The block of gated experts that strings the calls together, against plain torch
in 64 bits on the same weights and routes: outputs, losses and every gradient,
with the dispatched buffer and without; and a step with clipping.

Activations and their gradients are rounded to bf16 between the calls, at most
nine times on the longest path (h, logits' gradient, X, Z, H, Y, routed, y and
their duals), each by up to 2^-9 of a value in the mean: 9 * 2^-9 = 1.8 % of a
result's 2-norm bounds them all (independent roundings add to far less)."""
import pytest
import torch

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B
from combine_moe_topk_gb300 import block as block_module
from combine_moe_topk_gb300.block import GatedMoEBlock

pytestmark = pytest.mark.gpu
TOL = 9 * 2.0 ** -9


def reference(block, x, idx):
    P = {n: p.detach().double().requires_grad_() for n, p in block.named_parameters()}
    x = x.detach().double().requires_grad_()
    mean = x.mean(1, keepdim=True)
    h = (x - mean) / ((x - mean).square().mean(1, keepdim=True) + 1e-5).sqrt() * P["norm_w"] + P["norm_b"]
    logits = h @ P["router"].t()
    gate = torch.softmax(logits.gather(1, idx.long()), 1)
    f = torch.bincount(idx.reshape(-1).long(), minlength=block.e).double() / idx.numel()
    lse = torch.logsumexp(logits, 1)
    aux = block.weights[0] * block.e * (f * torch.softmax(logits, 1).mean(0)).sum() + block.weights[1] * lse.square().mean()

    def gated(x, W):
        g, u = (x @ W.t()).chunk(2, 1)
        return torch.nn.functional.silu(g) * u

    y = gated(h, P["shared_up"]) @ P["shared_down"].t() + x
    for j in range(block.e):
        out = gated(h, P["up"][j]) @ P["down"][j].t()
        y = y + ((idx == j).double() * gate).sum(1, keepdim=True) * out
    return y, aux, P, x


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("s,m,e,k,d", [(300, 256, 4, 2, 192), (37, 128, 16, 4, 72), (2500, 128, 8, 2, 136)])
def test_outputs_and_gradients(s, m, e, k, d, gather):
    block = GatedMoEBlock(m, e, k, d_expert=d, d_shared=d + 8, gather=gather, seed=1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(s, m, generator=g).bfloat16().cuda().requires_grad_()
    dy = torch.randn(s, m, generator=g).cuda()
    y, aux, counts = block(x)
    (y.float() * dy).sum().add(100.0 * aux).backward()
    with torch.no_grad():
        logits = B.moe_linear(B.moe_layernorm(x.detach(), block.norm_w, block.norm_b, stats=False), block.router,
                              out_dtype=torch.float32)
        idx, _ = B.moe_topk_gate(logits, k)
    ry, raux, P, rx = reference(block, x, idx)
    (ry * dy.double()).sum().add(100.0 * raux).backward()

    def off_by(a, b):
        return float(((a.detach().double() - b.detach()).norm() / b.detach().norm()).item())

    assert off_by(y, ry) <= TOL and abs(aux.item() - raux.item()) <= 0.01 * raux.item()
    assert counts.sum().item() == s * k
    errs = {"x": off_by(x.grad, rx.grad)}
    for n, p in block.named_parameters():
        errs[n] = off_by(p.grad, P[n].grad)
    assert all(v <= TOL for v in errs.values()), errs
    # clipped to a tenth of their norm
    before = [p.grad.double() for p in block.parameters()]
    norm = float(torch.stack([b.square().sum() for b in before]).sum().sqrt())
    got = float(A.clip_grad_norm(block.parameters(), norm / 10))
    assert abs(got - norm) <= 1e-6 * norm
    for p, b in zip(block.parameters(), before):
        assert ((p.grad.double() - b / 10).abs() <= 2.0 ** -8 * b.abs() / 10 + 1e-30).all()
    assert A.status() == 0


def test_inference_keeps_nothing_and_takes_one_token():
    block = GatedMoEBlock(128, 8, 2, 64, 64, seed=3)
    for s in (0, 1, 5):
        x = torch.randn(s, 128, device="cuda").bfloat16()
        with torch.no_grad():
            y, _, _ = block(x)
        assert y.shape == x.shape and not y.requires_grad and torch.isfinite(y).all()


def test_wrappers_take_every_layout():
    from test_gpu_autograd import every_view

    x = torch.randn(30, 64, device="cuda").bfloat16()
    W, b = torch.randn(48, 64, device="cuda").bfloat16() / 8, torch.randn(48, device="cuda")
    for at in range(3):
        every_view(A.gated_linear, [x, W, b], at)
    h = B.moe_dispatch_layout(torch.arange(60, device="cuda").view(30, 2).remainder(5).int(), 5, 0)
    W3 = torch.randn(5, 48, 64, device="cuda").bfloat16() / 8
    X = B.moe_dispatch(h, x)
    Wd = torch.randn(5, 16, 64, device="cuda").bfloat16() / 8
    for at in range(2):
        every_view(lambda X, W: A.grouped_gated(X, W, h), [X, W3], at)
        every_view(lambda x, W: A.dispatch_grouped_gated(x, W, h, "gelu"), [x, W3], at)
        every_view(lambda X, W: A.grouped_gemm(X, W, h), [X, Wd], at)


def test_the_command_runs(capsys):
    block_module.main(steps=2, gated=True)
    out = capsys.readouterr().out
    assert out.count("gradient norm") == 2
