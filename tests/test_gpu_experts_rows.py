"""The experts' products through autograd on layouts with rows that no route owns: they
are zero in results and in gradients, whatever the allocator's memory held."""
import pytest
import torch

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B
from oracle import experts as E

pytestmark = pytest.mark.gpu


def handle(kind, idx, e):
    s, k = idx.shape
    if kind == "capacity":
        return B.moe_dispatch_layout(idx, e, max(1, s * k * 3 // (2 * e)))
    if kind == "created":
        h = B.moe_layout_create(s, e, k, capacity=max(1, s * k * 2 // e))
        return B.moe_layout_rebuild(h, idx)
    if kind == "padded":
        return B.moe_dispatch_layout_ex(idx, e, pad_multiple=64)
    if kind == "absent":
        return B.moe_dispatch_layout_ex(torch.where(idx % 3 == 1, -1, idx), e, absent_routes=True)
    if kind == "bound":
        return B.moe_dispatch_layout_ex(torch.where(idx % 3 == 1, -1, idx), e, absent_routes=True, rows_bound=s * k - 1)
    return B.moe_dispatch_layout(idx, e, 0)


def poison():
    """Memory that the allocator hands out next holds NaN."""
    blocks = [torch.full((n,), float("nan"), device="cuda") for n in [1 << i for i in range(8, 20)] * 4]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kind", ["dropless", "capacity", "created", "padded", "absent", "bound"])
def test_rows_of_no_route_are_zero_through_autograd(kind, gather):
    """A scale of the hidden rows, whose gradient sums over all rows, and the gradient of the rows themselves."""
    s, e, k, K, N, m = 90, 6, 2, 64, 72, 64
    g = torch.Generator().manual_seed(11)
    idx = torch.stack([torch.randperm(e, generator=g)[:k] for _ in range(s)]).int().cuda()
    h = handle(kind, idx, e)
    owned = torch.zeros(h.rows, dtype=torch.bool)
    for r in E.segments(h.offsets().cpu().numpy(), h.counts().cpu().numpy()):
        owned[r] = True
    assert owned.all() == (kind == "dropless")
    owned = owned.cuda()
    x = torch.randn(s, K, generator=g).bfloat16().cuda()
    W = (torch.randn(e, 2 * N, K, generator=g) / 8).bfloat16().cuda().requires_grad_()
    Wd = (torch.randn(e, m, N, generator=g) / 8).bfloat16().cuda().requires_grad_()
    gate = torch.rand(s, k, generator=g).cuda()
    rows = B.moe_dispatch(h, x)
    rows[~owned] = 0
    for _ in range(2):
        X = (x if gather else rows).clone().requires_grad_()
        scale = torch.ones(N, device="cuda", requires_grad=True)
        poison()
        H = (A.dispatch_grouped_gated if gather else A.grouped_gated)(X, W, h, "silu")
        assert not H[~owned].any()
        hidden = (H.float() * scale).bfloat16()
        Y = A.grouped_gemm(hidden, Wd, h)
        assert not Y[~owned].any()
        out = A.combine(Y, gate, h)
        poison()
        hidden.retain_grad()
        out.float().square().sum().backward()
        assert not hidden.grad[~owned].any()
        want = (hidden.grad.double() * H.detach().double())[owned].sum(0)
        assert float((scale.grad - want).norm() / want.norm()) <= 2.0 ** -8
        assert torch.isfinite(X.grad).all() and X.grad.any()
        if not gather:
            assert not X.grad[~owned].any()
        assert torch.isfinite(W.grad).all() and torch.isfinite(Wd.grad).all()


@pytest.mark.parametrize("kind", ["dropless", "capacity"])
def test_frozen_experts_give_the_same_gradient(kind):
    s, e, k, K, N = 90, 6, 2, 64, 72
    g = torch.Generator().manual_seed(5)
    idx = torch.stack([torch.randperm(e, generator=g)[:k] for _ in range(s)]).int().cuda()
    h = handle(kind, idx, e)
    x, W = torch.randn(s, K, generator=g).bfloat16().cuda(), torch.randn(e, 2 * N, K, generator=g).bfloat16().cuda()
    d = torch.randn(h.rows, N, generator=g).bfloat16().cuda()
    grads, dispatches = [], []
    for frozen in (True, False):
        X, w = x.clone().requires_grad_(), W.clone().requires_grad_(not frozen)
        before = B.moe_launch_count("dispatch")
        A.dispatch_grouped_gated(X, w, h, "silu").backward(d)
        grads.append(X.grad)
        dispatches.append(B.moe_launch_count("dispatch") - before)
    assert torch.equal(*grads) and dispatches == [0, 1]
