"""The gated products of a shared expert, forward and backward, against the plain
64-bit form.

Tolerances.  z as in the dense products: (K/16 + 48) 2^-23 of sum |x||W|, plus
half a step of bf16 where it is stored.  h = act(g) u: g's error times the
activation's slope (below 1.13) and 16 u (|g| + 1) of its own arithmetic, times
|u|; u's error times |act(g)|; half a step of bf16.  Backward: act and slope to
16 u (1 + |g|) (their values are below 1.13 and |g|), two more products; dz
rounded to bf16 takes 2^-8 of each term of a gradient's sum, 2^-16 for an fp32 result."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B
from oracle import experts as E
from oracle.block import act as act64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def chain(K):
    return (K / 16 + 48) * 2.0 ** -23


def half(v, dtype):
    return np.abs(v) * (2.0 ** -8 if dtype == torch.bfloat16 else U) + 1e-38


def make(s, K, N, seed=0, bias=torch.float32, dh=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(s, K, generator=g).bfloat16().cuda()
    W = (torch.randn(2 * N, K, generator=g) / K ** 0.5).bfloat16().cuda()
    b = (0.5 * torch.randn(2 * N, generator=g)).to(bias).cuda() if bias else None
    d = torch.randn(s, N, generator=g).to(dh).cuda()
    z = torch.randn(s, 2 * N, generator=g).bfloat16().cuda()
    return x, W, b, d, z


def check_fwd(x, W, b, act, h, z=None):
    oh, oz = E.gated(f64(x), f64(W), f64(b), act)
    N = oh.shape[1]
    ez = chain(x.shape[1]) * (np.abs(f64(x)) @ np.abs(f64(W)).T) + 2 * U * (np.abs(oz) + (0 if b is None else np.abs(f64(b))))
    if z is not None:
        assert (np.abs(f64(z) - oz) <= ez + half(oz, z.dtype)).all()
    g, u = oz[:, :N], oz[:, N:]
    ea = 1.13 * ez[:, :N] + 16 * U * (np.abs(g) + 1)
    eh = ea * (np.abs(u) + ez[:, N:]) + np.abs(act64(g, act)) * ez[:, N:] + half(oh, h.dtype) + 2 * U * np.abs(oh)
    err = np.abs(f64(h) - oh)
    assert (err <= eh * 1.01).all(), (err / eh).max()


def check_bwd(dh, x, W, z, act, got):
    dx, dW, db = got
    ox, ow, ob, dz = E.gated_bwd(f64(dh), f64(x), f64(W), f64(z), act)
    s, N = f64(dh).shape
    g, u = f64(z)[:, :N], f64(z)[:, N:]
    slip = 16 * U * (np.abs(g) + 1) * np.abs(f64(dh))
    ez = np.concatenate([slip * (np.abs(u) + 1), slip], 1) + 4 * U * np.abs(dz)
    for t, o, terms, sl, k in ((dx, ox, np.abs(dz) @ np.abs(f64(W)), ez @ np.abs(f64(W)), 2 * N),
                               (dW, ow, np.abs(dz).T @ np.abs(f64(x)), ez.T @ np.abs(f64(x)), s)):
        if t is None:
            continue
        rnd = 2.0 ** -8 if t.dtype == torch.bfloat16 else 2.0 ** -16
        err = np.abs(f64(t) - o)
        assert (err <= (2 * chain(k) + rnd) * terms + 1.01 * sl + half(o, t.dtype)).all(), (err / (terms + 1e-30)).max()
        if o.size > 1000 and t.dtype == torch.bfloat16:
            assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(o)
    if db is not None:
        assert (np.abs(f64(db) - ob) <= (s / 8 + 80) * U * np.abs(dz).sum(0) + ez.sum(0) * 1.01 + 1e-38).all()


# every tile shape, tails of each axis, splits of the contracted axis, one to few rows
SHAPES = [(1, 8, 8), (1, 64, 8), (1, 4096, 512), (2, 512, 1000), (3, 72, 24), (7, 4096, 136), (16, 2048, 264), (17, 1024, 96),
          (33, 264, 256), (64, 4096, 384), (100, 136, 40), (128, 128, 64), (129, 256, 136), (200, 4096, 8), (255, 640, 504),
          (300, 72, 1032), (520, 512, 520), (1000, 8, 64), (1030, 1032, 248), (2100, 200, 1064)]


@pytest.mark.parametrize("s,K,N", SHAPES)
def test_shapes_forward(s, K, N):
    x, W, b, _, _ = make(s, K, N, seed=s + K + N)
    check_fwd(x, W, None, "silu", B.moe_gated_linear(x, W))
    h, z = B.moe_gated_linear(x, W, b, "gelu", save_z=True)
    check_fwd(x, W, b, "gelu", h, z)


@pytest.mark.parametrize("s,K,N", SHAPES)
def test_shapes_backward(s, K, N):
    x, W, _, dh, z = make(s, K, N, seed=s + K + N + 1)
    check_bwd(dh, x, W, z, "silu", B.moe_gated_linear_bwd(dh, x, W, z))
    check_bwd(dh, x, W, z, "gelu", B.moe_gated_linear_bwd(dh, x, W, z, "gelu", dx_dtype=torch.float32, dw_dtype=torch.float32))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("s", [5, 40, 700])
def test_activations_and_types(act, s):
    for bias in (None, torch.float32, torch.bfloat16):
        x, W, b, dh, z = make(s, 192, 136, seed=s, bias=bias, dh=torch.float32)
        h, zz = B.moe_gated_linear(x, W, b, act, save_z=True)
        check_fwd(x, W, b, act, h, zz)
        assert torch.equal(h, B.moe_gated_linear(x, W, b, act))
    check_bwd(dh, x, W, z, act, B.moe_gated_linear_bwd(dh, x, W, z, act))
    dx, dW, db = B.moe_gated_linear_bwd(dh, x, W, z, act)
    only = [B.moe_gated_linear_bwd(dh, x, W, z, act, *(i == j for i in range(3)))[j] for j in range(3)]
    for a, c in zip((dx, dW, db), only):  # each alone, and again: the same bits
        assert torch.equal(a, c)


# the last: dx of two products, 19 blocks of 256 rows and 40 more
@pytest.mark.parametrize("s,K,N", [(4100, 640, 2504), (9000, 72, 520), (300, 264, 4504), (4904, 1024, 2048)])
def test_many_tiles(s, K, N):
    x, W, b, dh, z = make(s, K, N, seed=K)
    h, zz = B.moe_gated_linear(x, W, b, "silu", save_z=True)
    check_fwd(x, W, b, "silu", h, zz)
    check_fwd(x, W, None, "relu", B.moe_gated_linear(x, W, act="relu"))
    check_bwd(dh, x, W, z, "gelu_tanh", B.moe_gated_linear_bwd(dh, x, W, z, "gelu_tanh"))


@pytest.mark.parametrize("s", [1, 40])
def test_the_longest_contraction(s):
    x, W, b, _, _ = make(s, 1 << 18, 16, seed=s)
    check_fwd(x, W, b, "silu", B.moe_gated_linear(x, W, b))


@pytest.mark.parametrize("s", [3, 50, 400])
def test_strided_rows(s):
    x, W, b, dh, z = make(s, 128, 64, seed=s)
    xs = torch.zeros(s, 160, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(128, 144, dtype=torch.bfloat16, device="cuda")
    ds = torch.zeros(s, 72, dtype=torch.bfloat16, device="cuda")
    zs = torch.zeros(s, 136, dtype=torch.bfloat16, device="cuda")
    xs[:, 8:136], ws[:, 16:], ds[:, :64], zs[:, 8:] = x, W, dh, z
    xs, ws, ds, zs = xs[:, 8:136], ws[:, 16:], ds[:, :64], zs[:, 8:]
    assert torch.equal(B.moe_gated_linear(xs, ws, b), B.moe_gated_linear(x, W, b))
    for a, c in zip(B.moe_gated_linear_bwd(ds, xs, ws, zs), B.moe_gated_linear_bwd(dh, x, W, z)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("s", [1, 40, 300])
def test_infinite_and_nan_values_stay_in_their_rows_and_columns(s):
    x, W, b, dh, z = make(s, 64, 72, seed=s, bias=None)
    W[3, 5] = float("nan")       # gate column 3
    W[72 + 9, 0] = float("inf")  # factor column 9
    h, zz = B.moe_gated_linear(x, W, save_z=True)
    ok = torch.ones(72, dtype=torch.bool)
    ok[3] = ok[9] = False
    assert torch.isnan(h[:, 3]).all() and not torch.isfinite(h[:, 9]).any()
    Wc = W.clone()
    Wc[3], Wc[72 + 9] = 0, 0
    hc, zc = B.moe_gated_linear(x, Wc, save_z=True)
    assert torch.equal(h[:, ok], hc[:, ok]) and torch.equal(zz[:, :72][:, ok], zc[:, :72][:, ok])


def test_no_rows():
    x, W, b, dh, z = make(4, 64, 16)
    assert B.moe_gated_linear(x[:0], W).shape == (0, 16)
    dx, dW, db = B.moe_gated_linear_bwd(dh[:0], x[:0], W, z[:0])
    assert dx.shape == (0, 64) and not dW.any() and not db.any()


def test_calls_in_a_captured_graph():
    x, W, b, dh, z = make(200, 256, 128, seed=7)

    def step():
        h, zz = B.moe_gated_linear(x, W, b, save_z=True)
        return (h, *B.moe_gated_linear_bwd(h, x, W, zz), B.moe_gated_linear(x[:1], W, b))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        x.copy_(torch.randn(200, 256, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip([t.clone() for t in out], step()):
            assert torch.equal(a, c)


def test_results_of_more_than_2_31_elements():
    s, K, N = 66000, 64, 16384  # z: 2.16e9 elements
    x, W, b, _, _ = make(s, K, N, seed=11)
    h, z = B.moe_gated_linear(x, W, b, "silu", save_z=True)
    check_fwd(x[-40:].contiguous(), W, b, "silu", h[-40:], z[-40:])
    check_fwd(x[:40].contiguous(), W, b, "silu", h[:40], z[:40])
    # its backward pass: rows are apart from one another in dx, and db sums them all
    dh = torch.zeros_like(h)
    dh[-30:] = torch.randn(30, N, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dx, dW, db = B.moe_gated_linear_bwd(dh, x, W, z)
    assert not dx[:-30].any()
    t = slice(s - 30, s)
    check_bwd(dh[t], x[t].contiguous(), W, z[t], "silu", (dx[t], dW, db))


@pytest.mark.parametrize("s", [1, 12, 40])
def test_weights_that_the_kernel_before_has_just_written(s):
    """The weights' first rows are fetched while the kernel before may still write them: what counts is what it wrote."""
    K, N = 2048, 1024
    x = make(s, K, N, seed=s)[0]
    raw = torch.empty(2 * N, K, dtype=torch.bfloat16, device="cuda")

    def step(wait):
        W = B.moe_layernorm(raw, None, None, stats=False)  # lets the next kernel start before it ends
        if wait:
            torch.cuda.synchronize()
        return B.moe_gated_linear(x, W)

    raw.normal_()
    step(True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = step(False)
    for seed in range(8):
        raw.copy_(torch.randn(2 * N, K, generator=torch.Generator().manual_seed(seed)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, step(True))
