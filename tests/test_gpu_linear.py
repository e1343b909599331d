"""The dense products with their epilogue, forward and backward, against the
plain 64-bit form.

Tolerances.  Products of bf16 are exact in fp32; the tensor cores add 16 of
them at a time to an fp32 accumulator, each step off by at most one unit in
the last place (2^-23) of a partial sum that the sum of the magnitudes bounds,
and a split contraction adds up to 40 partial sums more: (K/16 + 48) 2^-23 of
sum |x||W|.  An activation's slope is below 1.13; its own arithmetic costs
some units (16 u of |z| + 1).  A bf16 output adds half a unit (2^-8 of the value).  In
the backward pass dz is rounded to bf16 where an activation (or an fp32 dy)
makes it: each term by at most 2^-8, and together, the roundings being
independent, by well under that of the result's 2-norm."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B
from oracle import block as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def chain(K):
    return (K / 16 + 48) * 2.0 ** -23


def half(v, dtype):
    return np.abs(v) * (2.0 ** -8 if dtype == torch.bfloat16 else U) + 1e-38


def make(s, K, N, seed=0, bias=torch.bfloat16, res=None, dy=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(s, K, generator=g).bfloat16().cuda()
    W = (torch.randn(N, K, generator=g) / K ** 0.5).bfloat16().cuda()
    b = (0.5 * torch.randn(N, generator=g)).to(bias).cuda() if bias else None
    r = torch.randn(s, N, generator=g).to(res).cuda() if res else None
    d = torch.randn(s, N, generator=g).to(dy).cuda()
    z = torch.randn(s, N, generator=g).bfloat16().cuda()
    return x, W, b, r, d, z


def mags(x, W):
    return np.abs(f64(x)) @ np.abs(f64(W)).T


def check_fwd(x, W, b, r, act, y, z=None):
    oy, oz = O.linear(f64(x), f64(W), f64(b), act, f64(r))
    ez = chain(x.shape[1]) * mags(x, W) + 2 * U * (np.abs(oz) + (0 if b is None else np.abs(f64(b))))
    if z is not None:
        assert z.dtype == torch.bfloat16
        assert (np.abs(f64(z) - oz) <= ez + half(oz, z.dtype)).all()
    ey = 1.13 * ez + 16 * U * (np.abs(oz) + 1) + half(oy, y.dtype) + 2 * U * np.abs(oy)
    if r is not None:
        ey = ey + 2 * U * np.abs(f64(r))
    err = np.abs(f64(y) - oy)
    assert (err <= ey).all(), (err / ey).max()


def check_bwd(dy, x, W, z, act, got, rounded):
    dx, dW, db = got
    ox, ow, ob, dz = O.linear_bwd(f64(dy), f64(x), f64(W), f64(z), act)
    ez = np.abs(dz) * 8 * U + np.abs(f64(dy)) * 16 * U if act != "none" else np.zeros_like(dz)
    rnd = 2.0 ** -8 if rounded else 0.0
    s, N = dz.shape
    for t, o, terms, slip, k in ((dx, ox, np.abs(dz) @ np.abs(f64(W)), ez @ np.abs(f64(W)), N),
                                 (dW, ow, np.abs(dz).T @ np.abs(f64(x)), ez.T @ np.abs(f64(x)), s)):
        if t is None:
            continue
        err = np.abs(f64(t) - o)
        assert (err <= (chain(k) + rnd) * terms + 1.01 * slip + half(o, t.dtype)).all(), (err / (terms + 1e-30)).max()
        if o.size > 1000:
            assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(o)
    if db is not None:
        # at most s/8 rows a warp (fewer with more blocks), 8 warps, 40 + 16 partial rows
        assert (np.abs(f64(db) - ob) <= (s / 8 + 80) * U * np.abs(dz).sum(0) + ez.sum(0) * 1.01 + 1e-38).all()


# every tile shape, tails of each axis, splits of the contracted axis, one to few rows
SHAPES = [(1, 8, 1), (1, 64, 8), (1, 4096, 512), (2, 512, 1000), (3, 72, 17), (7, 4096, 130), (16, 2048, 264), (17, 1024, 96),
          (33, 264, 257), (64, 4096, 384), (100, 136, 33), (128, 128, 128), (129, 256, 129), (200, 4096, 8), (255, 640, 511),
          (300, 72, 1030), (520, 512, 520), (1000, 8, 64), (1030, 1032, 250), (2100, 200, 2050)]


@pytest.mark.parametrize("s,K,N", SHAPES)
def test_shapes_forward(s, K, N):
    x, W, b, r, _, _ = make(s, K, N, seed=s + K + N, res=torch.bfloat16)
    check_fwd(x, W, None, None, "none", B.moe_linear(x, W))
    check_fwd(x, W, None, None, "none", B.moe_linear(x, W, out_dtype=torch.float32))
    y, z = B.moe_linear(x, W, b, "gelu", r, save_z=True)
    check_fwd(x, W, b, r, "gelu", y, z)


@pytest.mark.parametrize("s,K,N", SHAPES)
def test_shapes_backward(s, K, N):
    x, W, _, _, dy, z = make(s, K, N, seed=s + K + N + 1)
    # without an activation dz is dy: no rounding, fp32 gradients show the products' own error
    got = B.moe_linear_bwd(dy, x, W, dx_dtype=torch.float32, dw_dtype=torch.float32)
    check_bwd(dy, x, W, None, "none", got, rounded=False)
    check_bwd(dy, x, W, z, "silu", B.moe_linear_bwd(dy, x, W, z, "silu"), rounded=True)


# more tiles than workers: accumulators, ring and staging go round; both output types, N of 16-byte rows and not
@pytest.mark.parametrize("s,K,N", [(4100, 640, 5000), (3000, 1032, 2501), (9000, 72, 1032), (300, 264, 9001)])
def test_many_tiles(s, K, N):
    x, W, b, r, dy, z = make(s, K, N, seed=K, res=torch.bfloat16)
    y, zz = B.moe_linear(x, W, b, "silu", r, save_z=True)
    check_fwd(x, W, b, r, "silu", y, zz)
    check_fwd(x, W, b, r, "gelu", B.moe_linear(x, W, b, "gelu", r))
    check_fwd(x, W, None, None, "none", B.moe_linear(x, W, out_dtype=torch.float32))
    check_bwd(dy, x, W, None, "none", B.moe_linear_bwd(dy, x, W, dx_dtype=torch.float32, dw_dtype=torch.float32), rounded=False)
    check_bwd(dy, x, W, z, "gelu_tanh", B.moe_linear_bwd(dy, x, W, z, "gelu_tanh"), rounded=True)


def test_calls_in_a_captured_graph():
    # one decode step and one training step, captured once and replayed on new inputs
    x, W, b, r, dy, z = make(40, 256, 256, seed=12, res=torch.bfloat16)
    w = torch.ones(256, device="cuda")

    def step():
        h, mean, rstd = B.moe_layernorm(x, w, w)
        y, zz = B.moe_linear(h, W, b, "gelu", r, save_z=True)
        few = B.moe_linear(h[:3], W, b, "silu")
        logits = B.moe_linear(y, W[:16], out_dtype=torch.float32)
        idx = torch.zeros(40, 2, dtype=torch.int32, device="cuda")
        bl = B.moe_balance_loss(logits, idx)
        dl = B.moe_balance_loss_bwd(logits, bl.lse, bl.coef, bl.norm, bl.norm)
        dh, dW, db = B.moe_linear_bwd(dy, h, W, zz, "gelu")
        return (h, y, few, bl.loss, dl, dW, db) + B.moe_layernorm_bwd(dh, x, w, mean, rstd)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (13, 14):
        x.copy_(make(40, 256, 256, seed=seed)[0])
        graph.replay()
        got = [t.clone() for t in out]
        for a, c in zip(got, step()):
            assert torch.equal(a, c)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("s,K,N", [(5, 256, 40), (70, 512, 333), (700, 1024, 768)])
def test_activations_and_types(act, s, K, N):
    for bias, res, out in ((None, None, torch.bfloat16), (torch.float32, None, torch.float32),
                           (torch.bfloat16, torch.float32, torch.bfloat16), (torch.float32, torch.bfloat16, torch.float32)):
        x, W, b, r, dy, z = make(s, K, N, seed=len(act) + s, bias=bias, res=res)
        y, zz = B.moe_linear(x, W, b, act, r, out_dtype=out, save_z=True)
        check_fwd(x, W, b, r, act, y, zz)
        assert torch.equal(B.moe_linear(x, W, b, act, r, out_dtype=out), y)
    for dt in (torch.bfloat16, torch.float32):
        x, W, _, _, dy, z = make(s, K, N, seed=9 + s, dy=dt)
        check_bwd(dy, x, W, z, act, B.moe_linear_bwd(dy, x, W, z, act), rounded=act != "none" or dt == torch.float32)


def test_identity_weights_copy_bit_for_bit():
    x = torch.randn(777, 512).bfloat16().cuda()
    eye = torch.eye(512).bfloat16().cuda()
    assert torch.equal(B.moe_linear(x, eye), x)
    dx, dW, _ = B.moe_linear_bwd(x, x, eye)
    assert torch.equal(dx, x)
    e7 = torch.eye(512)[:, torch.randperm(512, generator=torch.Generator().manual_seed(1))].bfloat16().cuda()
    assert torch.equal(B.moe_linear(x, e7), x @ e7.t())
    assert torch.equal(B.moe_linear_bwd(x, x, e7)[0], x @ e7)


def test_strided_rows():
    s, K, N = 150, 256, 200
    g = torch.Generator().manual_seed(3)
    X, Wb = torch.randn(s, K + 64, generator=g).bfloat16().cuda(), torch.randn(N, K + 8, generator=g).bfloat16().cuda()
    R, Z = torch.randn(s, N + 3, generator=g).cuda(), torch.randn(s, N + 5, generator=g).bfloat16().cuda()
    x, W, r, z = X[:, 64:], Wb[:, :K], R[:, :N], Z[:, :N]
    check_fwd(x, W, None, r, "silu", B.moe_linear(x, W, act="silu", residual=r))
    dy = Z[:, :N]
    check_bwd(dy, x, W, z, "relu", B.moe_linear_bwd(dy, x, W, z, "relu"), rounded=True)
    dy = torch.randn(s, N + 8, generator=g).bfloat16().cuda()[:, :N]
    check_bwd(dy, x, W, None, "none", B.moe_linear_bwd(dy, x, W, dx_dtype=torch.float32), rounded=False)
    with pytest.raises(B.MoEError):  # rows that do not start on 16 bytes
        B.moe_linear(torch.empty(s, K + 4, dtype=torch.bfloat16, device="cuda")[:, :K], W)


def test_rows_stay_apart():
    # a row of NaN or infinities reaches its own outputs only; the tail of a tile is zeros, not what lies behind
    x, W, b, _, dy, _ = make(130, 264, 70, seed=4)
    y0 = B.moe_linear(x, W, b)
    x[129] = float("nan")
    x[64] = float("inf")
    y = B.moe_linear(x, W, b)
    keep = [i for i in range(130) if i not in (64, 129)]
    assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[129]).all()
    big = torch.full((200, 264), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:131] = torch.randn(131, 264).bfloat16().cuda()
    part, Wn = big[:131], torch.full((90, 264), float("nan"), dtype=torch.bfloat16, device="cuda")
    Wn[:70] = W
    assert torch.isfinite(B.moe_linear(part, Wn[:70])).all()
    assert all(torch.isfinite(t).all() for t in B.moe_linear_bwd(dy.repeat(2, 1)[:131], part, Wn[:70]))


def test_activation_extremes():
    # exp and tanh saturate without NaN; relu and silu at 0
    K = 8
    x = torch.zeros(6, K)
    x[:, 0] = torch.tensor([0.0, 100.0, -100.0, 1e30, -1e30, -20.0])
    W = torch.zeros(4, K)
    W[:, 0] = 1
    x, W = x.bfloat16().cuda(), W.bfloat16().cuda()
    dy = torch.ones(6, 4, device="cuda")
    for act in ACTS:
        y, z = B.moe_linear(x, W, act=act, save_z=True, out_dtype=torch.float32)
        assert torch.isfinite(y).all()
        if act != "none":
            assert y[0].abs().max() == 0 and torch.equal(y[1], z[1].float()) and y[2].abs().max() < 1e-6
        _, _, db = B.moe_linear_bwd(dy, x, W, z, act)
        assert torch.isfinite(db).all()


def test_same_bits_and_another_stream():
    x, W, b, r, dy, z = make(300, 2048, 640, seed=5, res=torch.bfloat16)
    first = (B.moe_linear(x, W, b, "gelu", r),) + B.moe_linear_bwd(dy, x, W, z, "gelu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = (B.moe_linear(x, W, b, "gelu", r),) + B.moe_linear_bwd(dy, x, W, z, "gelu")
    side.synchronize()
    for a, c in zip(first, again):
        assert torch.equal(a, c)


def test_empty_and_optional():
    x, W, b, _, dy, z = make(40, 64, 24, seed=6)
    e = x[:0]
    assert B.moe_linear(e, W, b).shape == (0, 24)
    dx, dW, db = B.moe_linear_bwd(dy[:0], e, W)
    assert dx.shape == (0, 64) and not dW.any() and not db.any()
    full = B.moe_linear_bwd(dy, x, W, z, "silu")
    for k in range(3):
        need = [i == k for i in range(3)]
        got = B.moe_linear_bwd(dy, x, W, z, "silu", *need)
        assert torch.equal(got[k], full[k]) and all(got[i] is None for i in range(3) if i != k)


def test_gradient_against_differences_of_the_64_bit_form():
    x, W, b, _, dy, _ = make(12, 64, 20, seed=7, bias=torch.float32, dy=torch.float32)
    r, h = np.random.default_rng(0), 1e-6
    for act in ("gelu", "gelu_tanh", "silu"):
        _, z = B.moe_linear(x, W, b, act, save_z=True)
        dx, dW, db = (f64(t) for t in B.moe_linear_bwd(dy, x, W, z, act, dx_dtype=torch.float32, dw_dtype=torch.float32))
        X, Wd, bd, D = f64(x), f64(W), f64(b), f64(dy)
        for grad, at, f in ((dx, X, lambda a: O.linear(a, Wd, bd, act)[0]), (dW, Wd, lambda a: O.linear(X, a, bd, act)[0]),
                            (db, bd, lambda a: O.linear(X, Wd, a, act)[0])):
            v = r.normal(size=at.shape)
            num = ((f(at + h * v) - f(at - h * v)) * D).sum() / (2 * h)
            # z and dz are bf16: 2^-8 of each term, and the slope's change with z's rounding (|act''| < 1, |z| <= 4)
            assert abs(num - (grad * v).sum()) <= 2.0 ** -8 * 6 * np.linalg.norm(grad * v) + 1e-3


def test_refusals():
    x, W, b, _, dy, z = make(10, 64, 24, seed=8)
    for bad in (lambda: B.moe_linear(x.half(), W.half()), lambda: B.moe_linear(x.float(), W.float()),
                lambda: B.moe_linear(x[:, :56], W), lambda: B.moe_linear(x, W, b[:3]), lambda: B.moe_linear(x, W, act="tanh"),
                lambda: B.moe_linear(x, W, residual=dy[:3]), lambda: B.moe_linear(x, W, out_dtype=torch.float16),
                lambda: B.moe_linear(x[:, :4].contiguous(), W[:, :4].contiguous()), lambda: B.moe_linear(x, W.cpu()),
                lambda: B.moe_linear(x.cpu(), W.cpu()), lambda: B.moe_linear_bwd(dy[:5], x, W),
                lambda: B.moe_linear_bwd(dy, x, W, None, "gelu"), lambda: B.moe_linear_bwd(dy, x, W, z.float(), "gelu"),
                lambda: B.moe_linear_bwd(dy.half(), x, W), lambda: B.moe_linear(x.view(-1)[4:516].view(8, 64), W)):
        with pytest.raises(B.MoEError):
            bad()
    with pytest.raises(ValueError):
        B.moe_linear(torch.empty(64, 10, dtype=torch.bfloat16, device="cuda").t(), W)
