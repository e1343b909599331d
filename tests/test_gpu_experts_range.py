"""The experts' backward products over contractions past 2^17 terms.

The tensor cores' accumulator drops the bits below its last place, up to 2^-23 of the sum at every
step of 16 terms: n terms of one sign come out up to n / 16 units of 2^-23 short.  It is emptied into an fp32 sum every 2^17 terms, so a sum of any
length of one sign is at most 2^-10 short, to which the result's rounding adds 2^-8 and the fp32
sums (33 of them at most here) 2^-18."""
import pytest
import torch

from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -18


def positive(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(*shape, generator=g, device="cuda", dtype=torch.bfloat16) + 0.5)


def layout(counts):
    idx = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).int().view(-1, 1).cuda()
    return B.moe_dispatch_layout(idx, len(counts), 0)


def off_by(got, want):
    return float(((got.double() - want) / want).abs().max())


# whole blocks and a cut end, one piece and many, with a short segment behind
@pytest.mark.parametrize("rows", [(1 << 17) - 3, 1 << 17, (1 << 17) + 3, (1 << 18) - 3, 1 << 18, (1 << 18) + 128,
                                  (1 << 19) + 5, (1 << 22) + 77])
def test_an_expert_of_many_rows(rows):
    K, N = 72, 264
    if rows > 1 << 20:
        K, N = 64, 64
    h = layout([0, rows, 40])
    X, dY = positive(1, rows + 40, K), positive(2, rows + 40, N)
    W = positive(3, 3, N, K)
    dX, dW = B.moe_grouped_gemm_bwd(h, dY, X, W)
    assert not dW[0].any()
    for x, seg in ((1, slice(0, rows)), (2, slice(rows, rows + 40))):
        want = sum(d.double().t() @ r.double() for d, r in zip(dY[seg].split(1 << 18), X[seg].split(1 << 18)))
        assert off_by(dW[x], want) <= TOL, x
    at = torch.tensor([0, 1, 255, 256, rows - 1, rows, rows + 39])
    for r in at.tolist():
        assert off_by(dX[r], dY[r].double() @ W[1 if r < rows else 2].double()) <= TOL
    again = B.moe_grouped_gemm_bwd(h, dY, X, W)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)
    assert h.status() == 0


@pytest.mark.parametrize("N", [1 << 17, (1 << 17) + 16, 1 << 18, (1 << 18) + 16, (1 << 19) + 80, 1 << 22])
def test_a_wide_result(N):
    K, rows = 72, [20, 0, 3]
    e = 1 if N > 1 << 20 else 3
    h = layout(rows[:e])
    n = sum(rows[:e])
    X, dY, W = positive(4, n, K), positive(5, n, N), positive(6, e, N, K)
    dX, _ = B.moe_grouped_gemm_bwd(h, dY, X, W, need_dw=False)
    for r in range(n):
        assert off_by(dX[r], dY[r].double() @ W[0 if r < rows[0] else 2].double()) <= TOL, r
    # gated, half as wide: the contraction goes over both halves.  g = u = 1 and no activation: dz = [dh | dh]
    Z = torch.ones(n, N, dtype=torch.bfloat16, device="cuda")
    dX, _ = B.moe_grouped_gated_bwd(h, dY[:, :N // 2].contiguous(), X, W, Z, "none", need_dw=False)
    for r in range(n):
        d = dY[r, :N // 2].double()
        assert off_by(dX[r], torch.cat([d, d]) @ W[0 if r < rows[0] else 2].double()) <= TOL, r
    assert h.status() == 0
