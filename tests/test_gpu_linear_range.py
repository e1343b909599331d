"""The dense products at the far ends of their range."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def test_a_product_longer_than_the_limit_of_a_wait():
    """2 * 131072^3 operations take more than two seconds, the limit of one device wait.  Rows repeat every 256, so
    256 x 256 values of the definition tell all of them."""
    n, r = 131072, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    few = [(torch.randn(r, n, generator=g, device="cuda") / n ** 0.25).bfloat16() for _ in range(2)]
    x, W = (t.repeat(n // r, 1) for t in few)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = B.moe_linear(x, W, device_status=st)
    assert st.item() == 0
    want = few[0].double() @ few[1].double().t()
    mags = few[0].double().abs() @ few[1].double().abs().t()
    got = y[:r, :r].double()
    # the chain of the tensor cores' additions, 16 terms each, and the rounding to bf16
    tol = (n / 16 + 48) * 2.0 ** -23 * mags + want.abs() * 2.0 ** -8 + 1e-38
    assert ((got - want).abs() <= tol).all()
    first = y[:r]
    assert (first.view(r, n // r, r) == first[:, None, :r]).all()
    for at in range(0, n, 16 * r):
        block = y[at:at + 16 * r].view(-1, r, n)
        assert (block == first).all(), at


@pytest.mark.parametrize("s,K,N", [(1, 16384, 24), (1, 65536, 24), (8, 65536, 130), (16, 16384, 24), (16, 65536, 24),
                                   (17, 65536, 24), (200, 65536, 24)])
def test_long_fp32_sums(s, K, N):
    """All terms positive, so that what an accumulator drops adds up instead of cancelling.  Up to 16 rows, 256 terms
    go through the tensor cores' accumulator (16 steps, each off by at most 2 u of the sum), K / 2048 such sums and
    those of 8 warps are added in fp32: 32 + K/2048 + 10 u.  From 17 rows on, 512 terms, and K/512 sums."""
    g = torch.Generator().manual_seed(K + s)
    x, W = (torch.rand(n, K, generator=g).bfloat16().cuda() for n in (s, N))
    y = B.moe_linear(x, W, out_dtype=torch.float32)
    want = x.double() @ W.double().t()
    tol = (32 + K / 2048 + 10 if s <= 16 else 64 + K / 512 + 10) * U
    err = ((y.double() - want) / want).abs().max().item()
    assert err <= tol, (err / U, tol / U)


def normal(z):
    """(Phi(z), phi(z)) in 64 bits, the tail by the complementary error function."""
    from scipy.special import erfc

    return 0.5 * erfc(-z / np.sqrt(2.0)), np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)


@pytest.mark.parametrize("s", [1, 40])
def test_gelu_keeps_its_relative_precision_in_the_tail(s):
    """z comes in through the bias, exactly.  Phi's polynomial is good to 8 u, the exponential's argument and itself
    to (4 + 2 z^2) u, three products and a division to 8 u more: (20 + 2 z^2) u of the result, near 0 of which the
    values stay far from fp32's smallest."""
    pytest.importorskip("scipy")
    z = torch.linspace(-12, 8, 8000)
    x, W = torch.zeros(s, 8, device="cuda").bfloat16(), torch.zeros(8000, 8, device="cuda").bfloat16()
    y = f64(B.moe_linear(x, W, z.cuda(), "gelu", out_dtype=torch.float32))
    zz = f64(z)
    cdf, _ = normal(zz)
    want = zz * cdf
    bad = np.abs(y - want) > (20 + 2 * zz * zz) * U * np.abs(want) + 1e-44
    assert not bad.any(), (np.abs(y / want - 1) / U).max()
    # the slope, by the bias' gradient of one row: Phi + z phi, each to the same precision
    zb = z.bfloat16()
    _, _, db = B.moe_linear_bwd(torch.ones(1, 8000, device="cuda"), x[:1], W, zb.cuda()[None], "gelu", need_dx=False,
                                need_dw=False)
    zz = f64(zb)
    cdf, pdf = normal(zz)
    tol = (24 + 2 * zz * zz) * U * (cdf + np.abs(zz) * pdf)
    assert (np.abs(f64(db) - (cdf + zz * pdf)) <= tol + 1e-44).all()


@pytest.mark.parametrize("back", [False, True])
def test_long_sums_into_bf16(back):
    """Half a million terms, all positive: the sum may be off by (64 + K/512 + 10) u before it is rounded to bf16, at
    most half a unit in its last place (2^-8 of the power of two below it)."""
    n, K = 2304, 2 ** 19
    g = torch.Generator(device="cuda").manual_seed(1)
    a, c = (torch.rand(*((K, n) if back else (n, K)), generator=g, device="cuda").bfloat16() for _ in range(2))
    if back:
        W = torch.zeros(n, n, device="cuda").bfloat16()
        _, got, _ = B.moe_linear_bwd(a, c, W, need_dx=False, need_db=False)
        a, c = a[:, :64].t(), c[:, :64].t()
    else:
        got = B.moe_linear(a, c)
    want = a[:64].double() @ c[:64].double().t()
    tol = 2.0 ** (want.log2().floor() - 8) + (64 + K / 512 + 10) * U * want
    assert ((got[:64, :64].double() - want).abs() <= tol).all()


def test_a_backward_without_an_activation_takes_no_room_for_dz():
    s, N, K = 4096, 2048, 64
    dy, x, W = torch.randn(s, N, device="cuda").bfloat16(), torch.randn(s, K, device="cuda").bfloat16(), \
        torch.randn(N, K, device="cuda").bfloat16()
    B.moe_linear_bwd(dy, x, W)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = B.moe_linear_bwd(dy, x, W)
    outputs = sum((t.numel() * t.element_size() + 511) // 512 * 512 for t in out)
    assert torch.cuda.max_memory_allocated() - before < outputs + s * N * 2


@pytest.mark.parametrize("s,K,N", [(1, 64, 8), (7, 136, 33), (130, 264, 129), (300, 1032, 70), (700, 256, 2051), (4100, 72, 130)])
@pytest.mark.parametrize("act,dy_dtype", [("none", torch.float32), ("silu", torch.bfloat16), ("gelu", torch.float32)])
def test_fp32_gradients_take_dz_to_more_than_bf16(s, K, N, act, dy_dtype):
    """An fp32 result takes dz in two bf16 terms: off by 2^-16 of each term at most, the activation's slope by 24 u of
    |dy| times the slope's terms (below 1.2 each), and the sums' own chain."""
    from oracle import block as O

    g = torch.Generator().manual_seed(s + N)
    x, W = torch.randn(s, K, generator=g).bfloat16().cuda(), (torch.randn(N, K, generator=g) / K ** 0.5).bfloat16().cuda()
    dy, z = torch.randn(s, N, generator=g).to(dy_dtype).cuda(), torch.randn(s, N, generator=g).bfloat16().cuda()
    z = z if act != "none" else None
    dx, dW, db = B.moe_linear_bwd(dy, x, W, z, act, dx_dtype=torch.float32, dw_dtype=torch.float32)
    ox, ow, _, dz = O.linear_bwd(f64(dy), f64(x), f64(W), None if z is None else f64(z), act)
    slip = 0 if act == "none" else np.abs(f64(dy)) * 32 * U
    for got, want, k, by, order in ((dx, ox, N, np.abs(f64(W)), lambda m: m), (dW, ow, s, np.abs(f64(x)), lambda m: m.T)):
        tol = ((k / 16 + 48) * 2.0 ** -23 + 2.0 ** -16) * (order(np.abs(dz)) @ by)
        tol = tol + (0 if act == "none" else order(slip) @ by) + U * np.abs(want) + 1e-38
        assert (np.abs(f64(got) - want) <= tol).all()
        if want.size > 1000:
            assert np.linalg.norm(f64(got) - want) <= 2.0 ** -15 * np.linalg.norm(want)
    # one fp32 result beside a bf16 one, and the bf16 one as without it
    a = B.moe_linear_bwd(dy, x, W, z, act, dx_dtype=torch.float32)
    c = B.moe_linear_bwd(dy, x, W, z, act, dw_dtype=torch.float32)
    e = B.moe_linear_bwd(dy, x, W, z, act)
    assert torch.equal(a[0], dx) and torch.equal(c[1], dW) and torch.equal(a[1], e[1]) and torch.equal(c[0], e[0])
    assert torch.equal(db, e[2])


def test_fp32_gradients_of_infinite_rows():
    # an infinity stays what it is in the first term, and the second holds nothing for it
    x, W, dy = torch.randn(200, 64).bfloat16().cuda(), torch.randn(40, 64).bfloat16().cuda(), torch.randn(200, 40).cuda()
    dy[150, 3] = float("inf")
    dy[20, 5] = float("nan")
    W[3], x[150] = 1.0, 1.0
    dx, dW, _ = B.moe_linear_bwd(dy, x, W, dx_dtype=torch.float32, dw_dtype=torch.float32)
    assert (dx[150] == float("inf")).all() and dx[20].isnan().all() and (dW[3] == float("inf")).all() and dW[5].isnan().all()
    rows = [i for i in range(200) if i not in (20, 150)]
    cols = [i for i in range(40) if i not in (3, 5)]
    assert torch.isfinite(dx[rows]).all() and torch.isfinite(dW[cols]).all()
