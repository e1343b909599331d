"""How the binding allocates what it returns."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu


class Sizes(TorchDispatchMode):
    """Bytes of the CUDA tensors that the dispatcher makes."""

    def __init__(self):
        super().__init__()
        self.bytes = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in str(func) and torch.is_tensor(out):
            self.bytes += out.numel() * out.element_size()
        return out


def test_a_dispatch_mode_sees_the_outputs():
    x = torch.randn(64, 128, device="cuda").bfloat16()
    w = torch.ones(128, device="cuda").bfloat16()
    W = torch.randn(32, 128, device="cuda").bfloat16()
    logits = torch.randn(64, 8, device="cuda")
    idx = logits.topk(2, 1).indices.int()
    for call in (lambda: B.moe_layernorm(x, w), lambda: B.moe_linear(x, W), lambda: B.moe_balance_loss(logits, idx)):
        want = call()
        with Sizes() as seen:
            got = call()
        want, got = ((r,) if torch.is_tensor(r) else tuple(r) for r in (want, got))
        assert seen.bytes >= sum(t.numel() * t.element_size() for t in got)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
