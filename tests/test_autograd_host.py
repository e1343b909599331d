"""The autograd wrappers without a GPU: the library's calls are replaced by
plain torch forms, so that what the wrappers hand over, keep and return can be
seen."""
import pytest
import torch

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B


@pytest.fixture
def calls(monkeypatch):
    """The library's entry points in plain torch; their arguments are recorded by name."""
    log = []

    def fake(name, fn):
        def call(*args, **kw):
            log.append((name, args, kw))
            return fn(*args, **kw)

        monkeypatch.setattr(B, name, call)

    def layernorm(x, w=None, b=None, eps=1e-5):
        mean = x.float().mean(1)
        rstd = ((x.float() - mean[:, None]).square().mean(1) + eps).rsqrt()
        y = (x.float() - mean[:, None]) * rstd[:, None]
        y = y if w is None else y * w.float()
        return (y if b is None else y + b.float()).to(x.dtype), mean, rstd

    def layernorm_bwd(dy, x, w, mean, rstd, dres=None, need_dweight=True, need_dbias=True):
        xh = (x.float() - mean[:, None]) * rstd[:, None]
        g = dy.float() if w is None else dy.float() * w.float()
        dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return dx.to(x.dtype), (dy.float() * xh).sum(0) if need_dweight else None, dy.float().sum(0) if need_dbias else None

    def linear(x, W, bias=None, act="none", residual=None, out_dtype=None, save_z=False, **kw):
        z = x.float() @ W.float().t()
        z = z if bias is None else z + bias.float()
        y = z if act == "none" else torch.relu(z)
        y = (y if residual is None else y + residual.float()).to(out_dtype or torch.bfloat16)
        return (y, z.bfloat16()) if save_z else y

    def linear_bwd(dy, x, W, z=None, act="none", need_dx=True, need_dw=True, need_db=True, **kw):
        dz = dy.float() if act == "none" else dy.float() * (z > 0)
        return ((dz @ W.float()).to(x.dtype) if need_dx else None, (dz.t() @ x.float()).to(W.dtype) if need_dw else None,
                dz.sum(0) if need_db else None)

    def balance_loss(logits, idx, valid=None, offsets=None, **kw):
        p, e = torch.softmax(logits, 1), logits.shape[1]
        f = torch.bincount(idx.reshape(-1).long(), minlength=e).float() / idx.numel()
        lse = torch.logsumexp(logits, 1)
        loss = torch.stack([e * (f * p.mean(0)).sum(), lse.square().mean()])
        return B.BalanceLoss(loss, torch.zeros(1, e, dtype=torch.int32), p.mean(0)[None], lse, (e * f / len(p))[None],
                             torch.tensor([1.0, 1.0 / len(p)]))

    def balance_loss_bwd(logits, lse, coef, norm, dloss, valid=None, offsets=None, add=None):
        p = torch.softmax(logits, 1)
        return p * (dloss[0] * (coef - (coef * p).sum(1, keepdim=True)) + dloss[1] * norm[1] * 2 * lse[:, None])

    for name, fn in (("moe_layernorm", layernorm), ("moe_layernorm_bwd", layernorm_bwd), ("moe_linear", linear),
                     ("moe_linear_bwd", linear_bwd), ("moe_balance_loss", balance_loss),
                     ("moe_balance_loss_bwd", balance_loss_bwd),
                     ("moe_topk_gate", lambda l, k, renorm=1, **kw: (l.topk(k, 1).indices.int(), torch.softmax(l.topk(k, 1).values, 1))),
                     ("moe_topk_gate_bwd", lambda l, idx, gate, dgate, e, renorm=1: torch.zeros(len(idx), e)),
                     ("moe_dispatch", lambda h, x: x * 1.0), ("moe_dispatch_bwd", lambda h, dX: dX * 1.0),
                     ("moe_combine", lambda h, y, gate: y * gate[:, :1]),
                     ("moe_combine_bwd", lambda h, dout, gate, y: (dout * gate[:, :1], torch.zeros_like(gate)))):
        fake(name, fn)
    return log


def leaf(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).requires_grad_()


def idx_of(logits):
    return logits.detach().topk(2, 1).indices.int()


GRADS = {
    "layernorm": lambda x: A.layernorm(x, leaf(x.shape[1], seed=1)),
    "linear": lambda x: A.linear(x, leaf(6, x.shape[1], seed=1), act="relu", out_dtype=torch.float32),
    "balance_loss": lambda x: A.balance_loss(x, idx_of(x))[0],
    "topk_gate": lambda x: A.topk_gate(x, 2)[1],
    "dispatch": lambda x: A.dispatch(x, None),
    "combine": lambda x: A.combine(x, torch.ones(x.shape[0], 2), None),
}


@pytest.mark.parametrize("name", sorted(GRADS))
def test_a_second_derivative_is_refused(calls, name):
    # the library's gradients carry no graph: taken for constants, a second derivative would lack their part
    # without a word wherever x reaches the result another way as well
    x = leaf(4, 8)
    y = GRADS[name](x).float().square().sum() + x.square().sum()
    g, = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.square().sum(), x)
    # the first one is there without create_graph
    y = GRADS[name](x).float().square().sum()
    g, = torch.autograd.grad(y, x)
    assert torch.isfinite(g).all()


@pytest.mark.parametrize("name", ["layernorm", "linear", "topk_gate"])
def test_a_second_derivative_through_a_copied_input_is_refused(calls, name):
    # a view that the library would not take: what is saved is a copy, which has to lead back to x
    base = leaf(8, 4)
    x = base.t()
    if name == "linear":
        base = leaf(4 * 8 + 2, dtype=torch.bfloat16)
        x = base[2:].view(4, 8)
    w = torch.linspace(1, 2, 4 * 8)[:, None]
    y = GRADS[name](x).float()
    y = (y * w[:y.numel()].view(y.shape)).sum()  # the gradient reaching the call does not depend on x
    g, = torch.autograd.grad(y, base, create_graph=True)
    if name == "linear":  # relu: x's own gradient needs W only; the saved x is a source all the same
        assert g.requires_grad
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().square().sum(), base)


def test_the_residual_of_a_product_can_be_differentiated_twice(calls):
    x, W, r = leaf(4, 8, dtype=torch.bfloat16), leaf(6, 8, dtype=torch.bfloat16, seed=1), leaf(4, 6, seed=2)
    y = A.linear(x, W, residual=r, out_dtype=torch.float32)
    g, = torch.autograd.grad(y.pow(3).sum(), r, create_graph=True)
    h, = torch.autograd.grad(g.sum(), r)
    assert torch.allclose(h, 6 * y.detach(), rtol=1e-6)


def test_every_call_that_can_report_gets_a_status_word(calls, monkeypatch):
    monkeypatch.setattr(A, "_status", lambda t: "the word")
    x, W = leaf(4, 8, dtype=torch.bfloat16), leaf(6, 8, dtype=torch.bfloat16, seed=1)
    A.linear(x, W, act="relu").float().sum().backward()
    logits = leaf(4, 6)
    A.balance_loss(logits, idx_of(logits))[0].sum().backward()
    A.topk_gate(logits, 2)[1].sum().backward()
    for name, _, kw in calls:
        if name in ("moe_linear", "moe_linear_bwd", "moe_balance_loss", "moe_topk_gate"):
            assert kw.get("device_status") == "the word", name


def test_inference_keeps_nothing_for_a_backward_pass(calls):
    x, W = leaf(4, 8, dtype=torch.bfloat16).detach(), leaf(6, 8, dtype=torch.bfloat16, seed=1)

    def saved():
        calls.clear()
        A.linear(x, W, act="relu")
        return [kw["save_z"] for name, _, kw in calls if name == "moe_linear"]

    assert saved() == [True]
    for off in (torch.no_grad(), torch.inference_mode()):
        with off:
            assert saved() == [False]
    W.requires_grad_(False)
    assert saved() == [False]
