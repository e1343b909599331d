"""The expert-grouped GEMM where it takes longer than a device wait may."""
import pytest
import torch

from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu


def test_a_grouped_product_longer_than_the_limit_of_a_wait():
    """2 * 131072^3 operations take more than two seconds.  Rows repeat every 256, so 256 x 256 values of the definition
    tell all of them."""
    n, r = 131072, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    few = [(torch.randn(r, n, generator=g, device="cuda") / n ** 0.25).bfloat16() for _ in range(2)]
    X, W = (t.repeat(n // r, 1) for t in few)
    h = B.moe_dispatch_layout(torch.zeros(n, 1, dtype=torch.int32, device="cuda"), 1)
    Y = B.moe_grouped_gemm(h, X, W[None])
    assert h.status() == 0
    want = few[0].double() @ few[1].double().t()
    mags = few[0].double().abs() @ few[1].double().abs().t()
    # the chain of the tensor cores' additions, 16 terms each, and the rounding to bf16
    tol = (n / 16 + 48) * 2.0 ** -23 * mags + want.abs() * 2.0 ** -8 + 1e-38
    assert ((Y[:r, :r].double() - want).abs() <= tol).all()
    first = Y[:r]
    assert (first.view(r, n // r, r) == first[:, None, :r]).all()
    for at in range(0, n, 16 * r):
        assert (Y[at:at + 16 * r].view(-1, r, n) == first).all(), at
