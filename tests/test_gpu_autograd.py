"""The autograd wrappers on the GPU: what they report, and the inputs that they take."""
import pytest
import torch

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu


def test_what_kernels_report_can_be_read():
    A.status()
    logits = torch.randn(40, 8, device="cuda")
    idx = logits.topk(2, 1).indices.int()
    A.balance_loss(logits, idx)
    assert A.status() == 0
    logits[3, 1] = float("nan")
    A.balance_loss(logits, idx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bad = idx.clone()
        bad[0, 0] = 99
        A.balance_loss(torch.zeros(40, 8, device="cuda"), bad)
    assert A.status(torch.device("cuda", 0)) == B.MOE_DEV_NONFINITE | B.MOE_DEV_BAD_ROUTE
    assert A.status(0) == 0 and A.status("cuda") == 0
    A.topk_gate(logits, 2)
    assert A.status() == B.MOE_DEV_NONFINITE
    x, W = (torch.randn(n, 64, device="cuda").bfloat16().requires_grad_() for n in (40, 24))
    A.linear(x, W, act="silu").float().sum().backward()
    assert A.status() == 0


def views(t):
    """t's values in every layout that a caller may have: as they are, as a transposed matrix, as a slice of wider rows,
    off 16 bytes, and (rows alike) as a broadcast."""
    yield t
    if t.dim() == 2:
        yield t.t().contiguous().t()
        wide = torch.zeros(t.shape[0], t.shape[1] + 3, dtype=t.dtype, device=t.device)
        wide[:, 3:] = t
        yield wide[:, 3:]
        yield wide[:, :0].new_zeros(t.shape).copy_(t)
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    yield flat[1:].view(t.shape)


def every_view(call, args, at):
    """call(*args) with argument `at` in each layout: the same results and gradients, to the bit."""
    want = None
    for v in views(args[at].detach()):
        v = v.detach()
        leaves = [a.detach().requires_grad_() if torch.is_tensor(a) and a.is_floating_point() else a for a in args]
        v = v.requires_grad_() if v.is_floating_point() else v
        leaves[at] = v
        out = call(*leaves)
        out.float().square().sum().backward()
        got = [out.detach()] + [a.grad for a in leaves if torch.is_tensor(a) and a.is_floating_point()]
        if want is None:
            want = got
        assert len(got) == len(want)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_layernorm_takes_every_layout():
    x, w, b = torch.randn(20, 36, device="cuda").bfloat16(), torch.randn(36, device="cuda"), torch.randn(36, device="cuda")
    for at in range(3):
        every_view(A.layernorm, [x, w, b], at)
    row = torch.randn(1, 64, device="cuda", requires_grad=True)
    A.layernorm(row.expand(5, 64), None).pow(3).sum().backward()
    assert row.grad.shape == (1, 64) and torch.isfinite(row.grad).all()


def test_linear_takes_every_layout():
    x, W = (torch.randn(n, 40, device="cuda").bfloat16() for n in (30, 24))
    b, r = torch.randn(24, device="cuda"), torch.randn(30, 24, device="cuda").bfloat16()
    for at in range(4):
        every_view(lambda x, W, b, r: A.linear(x, W, b, "silu", r), [x, W, b, r], at)
    # one expert's part of packed weights and biases of an odd size
    W3, b3 = torch.randn(3, 5, 40, device="cuda").bfloat16().requires_grad_(), torch.randn(3, 5, device="cuda").requires_grad_()
    torch.cat([A.linear(x, W3[j], b3[j], "gelu") for j in range(3)], 1).float().sum().backward()
    assert torch.isfinite(W3.grad).all() and torch.isfinite(b3.grad).all()


def test_balance_loss_and_gate_take_every_layout():
    logits = torch.randn(50, 10, device="cuda")
    idx = logits.topk(3, 1).indices.int()
    valid = (torch.rand(50, device="cuda") < 0.8).to(torch.uint8)
    off = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    for at in range(4):
        every_view(lambda *a: A.balance_loss(*a)[0], [logits, idx, valid, off], at)
    every_view(lambda l: A.topk_gate(l, 3)[1], [logits], 0)
