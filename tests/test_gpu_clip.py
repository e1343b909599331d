"""The global gradient norm and clipping against 64 bits.

Tolerances.  The norm: up to 32 squares are added in fp32 (each step off by at
most 2^-24 of the sum: 32 steps), the rest in 64 bits, and one rounding to fp32;
the root halves the sum's relative error: (16 + 2) 2^-24.  The coefficient is
rounded once, the product once more in the tensor's type."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B
from oracle import experts as E

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def check(grads, max_norm, out=None):
    before = [f64(g) for g in grads]
    norm, c = E.clip(before, max_norm)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    alone = B.moe_grad_norm(grads, device_status=status)
    got = B.moe_clip_grad_norm(grads, max_norm, out=out, device_status=status)
    assert torch.equal(alone, got) and got.shape == (1,) and int(status) == 0
    # fp32's step below 2^-126 is 2^-149: a norm there is rounded by up to 2^-150 (5.06e-43 is 361.2 steps)
    assert abs(float(got) - norm) <= 18 * U * norm + 2.0 ** -150
    for t, b, g in zip(grads if out is None else out, before, grads):
        assert (np.abs(f64(t) - b * c) <= (HALF[t.dtype] + 20 * U) * np.abs(b * c) + 2.0 ** -134).all()
        if out is not None:
            assert (f64(g) == b).all()


def pieces(sizes, dtype, seed=0, skip=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    flat = (scale * torch.randn(sum(sizes) + skip, generator=g)).to(dtype).cuda()
    return list(flat[skip:].split(list(sizes)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 31, 255, 4095, 4096, 4097, 8191, 8192, 8193, 8200, 16384, 100003])
@pytest.mark.parametrize("skip", [0, 1, 3])
def test_one_tensor(dtype, n, skip):
    check(pieces([n], dtype, seed=n, skip=skip), 0.5)
    check(pieces([n], dtype, seed=n, skip=skip), 1e9)


@pytest.mark.parametrize("count", [2, 63, 64, 65, 300, 1023, 1024, 1025, 2100])
def test_many_tensors(count):
    r = np.random.default_rng(count)
    sizes = [int(v) for v in np.exp(r.uniform(0, 9, count))]
    sizes[0] = 0
    sizes[count // 2] = 0
    half = count // 2
    grads = pieces(sizes[:half], torch.bfloat16, skip=1) + pieces(sizes[half:], torch.float32, seed=1)
    check(grads, 1.0)
    check(grads, 0.25, out=[torch.empty_like(g) for g in grads])
    # other alignments than the gradients'
    flat = {d: torch.empty(sum(sizes) + 1, dtype=d, device="cuda")[1:] for d in HALF}
    check(grads, 0.25, out=[flat[g.dtype][sum(sizes[:i]):][:g.numel()] for i, g in enumerate(grads)])


def test_axes_in_any_order():
    g = torch.Generator().manual_seed(2)
    a = torch.randn(30, 50, generator=g).cuda().t()
    b = torch.randn(3, 5, 7, 2, generator=g).cuda().permute(2, 0, 3, 1)
    check([a, b, torch.randn((), generator=g).cuda()], 0.1)
    check([a, b], 0.1, out=[torch.empty_like(a), torch.empty_like(b)])
    with pytest.raises(B.MoEError, match="strides"):  # the same sizes in another order
        B.moe_clip_grad_norm([a, b], 0.1, out=[torch.empty_like(a), torch.empty(b.shape, device="cuda")])


# squares that leave fp32's range, up and down, alone and beside ordinary ones
@pytest.mark.parametrize("scale", [1e30, 3e36, 1e-30, 1e-38, 1e-44, 1e19, 1e-22])
def test_range(scale):
    grads = pieces([5000, 100], torch.float32, seed=3)
    for g in grads:
        g.clamp_(-1, 1)
        g *= scale
    check([g.clone() for g in grads], 1e-3 * scale if scale > 1e-30 else 1.0)
    check([g.clone() for g in grads] + pieces([9000], torch.bfloat16, seed=4), 1.0)


def test_a_norm_past_the_range_of_fp32_is_infinite():
    g = torch.full((100,), 3e38, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert float(B.moe_clip_grad_norm([g], 1.0, device_status=status)) == float("inf") and int(status) == B.MOE_DEV_NONFINITE
    assert (g == 3e38).all()


def test_coefficient_one_writes_nothing_in_place():
    g = pieces([1000], torch.bfloat16)[0]
    b = g.clone()
    B.moe_clip_grad_norm([g], float("inf"))
    assert torch.equal(g, b)
    B.moe_clip_grad_norm([g], 0.0)
    assert not g.any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norms_that_are_not_finite_leave_the_gradients(bad):
    grads = pieces([3000, 40], torch.float32)
    grads[1][17] = bad
    before = [g.clone() for g in grads]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.zeros_like(g) for g in grads]
    norm = B.moe_clip_grad_norm(grads, 1.0, out=out, device_status=status)
    assert not torch.isfinite(norm).any() and int(status) == B.MOE_DEV_NONFINITE
    assert torch.isnan(norm).item() == (bad != bad)
    B.moe_clip_grad_norm(grads, 1.0)
    B.moe_grad_clip(grads, norm, 1.0)
    for g, o, b in zip(grads, out, before):
        for t in (g, o):
            assert torch.equal(t.view(torch.int32), b.view(torch.int32))


def test_a_given_norm():
    grads = pieces([3000, 40], torch.float32)
    want = [g * (2.0 / (100.0 + 1e-6)) for g in grads]
    B.moe_grad_clip(grads, torch.tensor([100.0], device="cuda"), 2.0)
    for g, w in zip(grads, want):
        assert torch.allclose(g, w, rtol=3 * 2.0 ** -23, atol=0)


def test_no_tensors():
    assert float(B.moe_grad_norm([])) == 0.0
    assert float(B.moe_clip_grad_norm([], 1.0)) == 0.0
    e = torch.empty(0, device="cuda")
    assert float(B.moe_clip_grad_norm([e], 1.0)) == 0.0


def test_a_list_kept_and_captured():
    grads = pieces([70000, 3, 501], torch.bfloat16)
    kept, out = B.GradList(grads), B.GradList([torch.empty_like(g) for g in grads])
    assert len(kept) == 3
    B.moe_clip_grad_norm(kept, 1.0, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = B.moe_clip_grad_norm(kept, 1.0, out=out)
    for seed in range(3):
        for g, n in zip(grads, pieces([70000, 3, 501], torch.bfloat16, seed=seed)):
            g.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in out.tensors]
        assert torch.equal(norm, B.moe_clip_grad_norm(kept, 1.0, out=out))
        for a, c in zip(have, out.tensors):
            assert torch.equal(a, c)


def test_tensors_that_share_memory_are_refused():
    t = torch.randn(100, device="cuda")
    for bad in ([t, t], [t[:60], t[59:]], [t[50:], t[:51]]):
        with pytest.raises(B.MoEError, match="overlap"):
            B.GradList(bad)
    B.GradList([t[:0], t[:50], t[50:50], t[50:]])  # pieces side by side, and empty ones
    a, b = t[:50], t[50:]
    with pytest.raises(B.MoEError, match="overlaps"):
        B.moe_clip_grad_norm([a, b], 1.0, out=[b, a])
    with pytest.raises(B.MoEError, match="overlaps"):
        B.moe_clip_grad_norm([t[:40], t[60:]], 1.0, out=[torch.empty_like(t[:40]), t[10:50]])
    before = t.clone()
    norm = B.moe_clip_grad_norm([a, b], 1.0, out=[a, b])  # their own places
    assert torch.allclose(t, before / float(norm), rtol=1e-5)
    with pytest.raises(B.MoEError):
        B.moe_clip_grad_norm([a], 1.0, out=[a, b])
    with pytest.raises(B.MoEError):
        B.moe_clip_grad_norm([a], 1.0, out=[torch.empty(50, device="cuda", dtype=torch.bfloat16)])


def test_more_than_2_31_elements():
    n = 2 ** 31 + 4099
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-1] = 8.0
    norm = float(B.moe_clip_grad_norm([g[3:]], 1.0))  # off 16 bytes
    want = (0.25 * (n - 4) + 64.0) ** 0.5
    assert abs(norm - want) <= 18 * U * want
    assert float(g[2]) == 0.5 and abs(float(g[-1]) - 8.0 / want) <= 2.0 ** -8 * 8.0 / want
    assert (g[3:-1] == torch.tensor(0.5 / (want + 1e-6)).bfloat16().item()).all()
