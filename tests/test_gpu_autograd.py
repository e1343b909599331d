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
