"""Clipping to one norm over expert-parallel ranks, on the GPU with a group of one rank:
the kernels and the status word (several ranks run without a GPU, over gloo)."""
import socket

import pytest
import torch
import torch.distributed as dist

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B
from combine_moe_topk_gb300 import ep as EP

pytestmark = pytest.mark.gpu


@pytest.fixture
def group():
    with socket.socket() as sk:
        sk.bind(("127.0.0.1", 0))
        port = sk.getsockname()[1]
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1,
                            device_id=torch.device("cuda", 0))
    yield dist.group.WORLD
    dist.destroy_process_group()


def test_one_rank(group):
    A.status()
    for bad in (None, float("nan"), float("inf")):
        own, common = [torch.randn(5000, device="cuda"), torch.randn(70, device="cuda").bfloat16()], [torch.randn(33, device="cuda")]
        if bad is not None:
            own[1][3] = bad
        before = [t.clone() for t in own + common]
        norm = EP.clip_grad_norm(own, common, 0.5)
        want = torch.stack([t.double().square().sum() for t in before]).sum().sqrt()
        if bad is None:
            assert abs(norm.double() - want) <= 40 * 2.0 ** -24 * want and A.status() == 0
            for a, b in zip(own + common, before):
                step = 2.0 ** -8 if a.dtype == torch.bfloat16 else 2.0 ** -24
                c = 0.5 / (float(norm) + 1e-6)
                assert ((a.double() - b.double() * c).abs() <= (step + 2.0 ** -23) * b.double().abs() * c).all()
        else:
            assert not torch.isfinite(norm).any() and A.status() == B.MOE_DEV_NONFINITE and A.status() == 0
            for a, b in zip(own + common, before):
                assert torch.equal(a[~torch.isnan(b)], b[~torch.isnan(b)])
    # no gradients on this rank, or none that all ranks hold
    for own, common in (([], [torch.ones(9, device="cuda")]), ([torch.ones(9, device="cuda")], [])):
        assert float(EP.clip_grad_norm(own, common, 1e9)) == 3.0
