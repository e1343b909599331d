"""The gradient norm of lists that give a block many chunks, with values whose squares
only add up past fp32's range, and the coefficient's agreement with the norm that
is returned.

Equal values, so that the norm has a closed form: v sqrt(n).  Tolerances: the norm as
in the tests of short lists, (16 + 2) 2^-24; a clipped value is off by the norm's and the
coefficient's slip (20 + 2) 2^-24 and its type's rounding."""
import pytest
import torch

from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


# 64 (bf16) or 32 squares a thread and chunk, 4 to 240 chunks a block: each square is in range, their sum is not
@pytest.mark.parametrize("dtype,n,v", [(torch.bfloat16, 40_000_000, 2.0 ** 59.5), (torch.float32, 40_000_003, 1.1e18),
                                       (torch.bfloat16, 1_200_000_000, 2.0 ** 57), (torch.bfloat16, 1_200_000_000, 1.4e14),
                                       (torch.float32, 300_000_001, 2.0 ** 49), (torch.float32, 300_000_001, 2.0 ** 47.9)])
def test_sums_past_the_range_of_fp32(dtype, n, v):
    g = torch.full((n,), v, dtype=dtype, device="cuda")
    v = float(g[0])
    want = v * n ** 0.5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    alone = float(B.moe_grad_norm([g], device_status=status))
    norm = float(B.moe_clip_grad_norm([g[: n // 3], g[n // 3:]], want / 1024, device_status=status))
    assert abs(alone - want) <= 18 * U * want and abs(norm - want) <= 18 * U * want and int(status) == 0
    lo, hi = (float(x) for x in g.aminmax())
    assert abs(lo - v / 1024) <= (HALF[dtype] + 22 * U) * v / 1024 and lo == hi


def test_huge_values_beside_ordinary_ones():
    """One block of many is past the range: the others' sums are kept as they are."""
    g = torch.full((50_000_000,), 1.0, device="cuda")
    g[12_345_678] = 3e38
    g[40_000_000:40_000_100] = 1e30
    norm = float(B.moe_grad_norm([g]))
    want = float(g.double().square().sum().sqrt())
    assert abs(norm - want) <= 18 * U * want


@pytest.mark.parametrize("n", [40, 5000, 60_000, 3_000_000])
def test_both_ways_to_clip_give_the_same_bits(n):
    """The coefficient is that of the norm which is returned, computed in one call or given to another."""
    for seed in range(12):
        g = torch.randn(n, generator=torch.Generator().manual_seed(seed)).cuda()
        one, two = g.clone(), g.clone()
        norm = B.moe_clip_grad_norm([one], 0.37)
        B.moe_grad_clip([two], norm, 0.37)
        assert torch.equal(one, two), seed
