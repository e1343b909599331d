"""The experts' gated product and the backward passes over row segments, against
the plain 64-bit form, on every kind of layout.

Tolerances as in the dense gated products; a gradient that sums over an expert's
rows has count terms."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B
from combine_moe_topk_gb300 import workloads as W_
from oracle import experts as E
from oracle.block import act as act64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NAN = float("nan")


def f64(t):
    return t.detach().cpu().double().numpy()


def chain(K):
    return (K / 16 + 48) * 2.0 ** -23


def half(v):
    return np.abs(v) * 2.0 ** -8 + 1e-38


def layout(s, e, k, kind="dropless", seed=0, counts=None):
    if counts is None:
        idx = W_.random_routes(s, e, k, seed=seed).cuda()
    else:  # one route a token, so many to each expert
        idx = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).int().view(-1, 1).cuda()
    if kind == "capacity":
        return B.moe_dispatch_layout(idx, e, max(1, s * k // e))
    if kind == "kmajor":
        return B.moe_dispatch_layout_ex(idx, e, max(1, s * k // (2 * e)), priority="kmajor")
    if kind == "padded":
        return B.moe_dispatch_layout_ex(idx, e, pad_multiple=24)
    if kind == "absent":  # as an expert-parallel rank's arrivals: most routes are to other ranks' experts
        idx[torch.rand(idx.shape, generator=torch.Generator().manual_seed(seed)).cuda() < 0.7] = -1
        return B.moe_dispatch_layout_ex(idx, e, absent_routes=True)
    if kind == "bound":
        return B.moe_dispatch_layout_ex(idx, e, rows_bound=max(1, s * k * 3 // 4))
    return B.moe_dispatch_layout(idx, e, 0)


def segs_of(h):
    return E.segments(h.offsets().cpu().numpy(), h.counts().cpu().numpy())


def owned_of(segs, rows):
    o = np.zeros(rows, bool)
    for r in segs:
        o[r] = True
    return o


def rand(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g)).bfloat16().cuda()


def spoil(t, owned):
    """Rows of no route hold NaN: nothing of theirs may reach a result."""
    t[torch.from_numpy(~owned).cuda()] = NAN
    return t


def check_fwd(X, W, segs, act, H, Z, owned, before):
    oH, oZ = E.grouped_gated(np.nan_to_num(f64(X)), f64(W), segs, act)
    N = oH.shape[1]
    for x, r in enumerate(segs):
        if r.stop <= r.start:
            continue
        ez = chain(X.shape[1]) * (np.abs(f64(X[r])) @ np.abs(f64(W[x])).T)
        g, u = oZ[r][:, :N], oZ[r][:, N:]
        if Z is not None:
            assert (np.abs(f64(Z[r]) - oZ[r]) <= ez + half(oZ[r])).all(), x
        ea = 1.13 * ez[:, :N] + 16 * U * (np.abs(g) + 1)
        eh = ea * (np.abs(u) + ez[:, N:]) + np.abs(act64(g, act)) * ez[:, N:] + half(oH[r]) + 2 * U * np.abs(oH[r])
        assert (np.abs(f64(H[r]) - oH[r]) <= eh * 1.01).all(), x
    rest = torch.from_numpy(~owned)
    assert (H.cpu()[rest] == before).all()
    if Z is not None:
        assert (Z.cpu()[rest] == before).all()


def check_bwd(D, X, W, segs, dX, dW, ez, rnd, owned, before):
    """D: the 64-bit gradient of the product's result, ez its slip before rounding."""
    for x, r in enumerate(segs):
        w, xr, d = f64(W[x]), f64(X[r]), D[r]
        ok = np.abs(d) @ np.abs(w)
        if dX is not None and r.stop > r.start:
            o = d @ w
            assert (np.abs(f64(dX[r]) - o) <= (chain(d.shape[1]) + rnd) * ok + 1.01 * (ez[r] @ np.abs(w)) + half(o)).all(), x
        if dW is not None:
            o = d.T @ xr
            terms = np.abs(d).T @ np.abs(xr)
            assert (np.abs(f64(dW[x]) - o) <= (chain(d.shape[0]) + rnd) * terms + 1.01 * (ez[r].T @ np.abs(xr)) + half(o)).all(), x
    if dX is not None:
        assert (dX.cpu()[torch.from_numpy(~owned)] == before).all()


def run_all(h, s, K, N, act, seed=0, check_gather=True):
    g = torch.Generator().manual_seed(seed)
    segs = segs_of(h)
    owned = owned_of(segs, h.rows)
    x = rand(g, s, K)
    X = spoil(B.moe_dispatch(h, x), owned)
    W = rand(g, h.e, 2 * N, K, scale=K ** -0.5)
    H, Z = (torch.full((h.rows, n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (N, 2 * N))
    B.moe_grouped_gated(h, X, W, act, H=H, Z=Z, save_z=True)
    check_fwd(X, W, segs, act, H, Z, owned, 7.0)
    H1 = torch.full_like(H, 7.0)
    B.moe_grouped_gated(h, X, W, act, H=H1)
    assert torch.equal(H, H1)
    if check_gather:
        H2, Z2 = torch.full_like(H, 7.0), torch.full_like(Z, 7.0)
        B.moe_dispatch_grouped_gated(h, x, W, act, H=H2, Z=Z2, save_z=True)
        assert torch.equal(H, H2) and torch.equal(Z, Z2)
    # backward, on another z and gradient
    dH, Zb = spoil(rand(g, h.rows, N), owned), spoil(rand(g, h.rows, 2 * N), owned)
    dX = torch.full((h.rows, K), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dW = B.moe_grouped_gated_bwd(h, dH, X, W, Zb, act, dX=dX)
    z, d = np.nan_to_num(f64(Zb)), np.nan_to_num(f64(dH))
    D = E.gated_dz(d, z, act)
    slip = 16 * U * (np.abs(z[:, :N]) + 1) * np.abs(d)
    ez = np.concatenate([slip * (np.abs(z[:, N:]) + 1), slip], 1) + 4 * U * np.abs(D)
    check_bwd(D, X, W, segs, dX, dW, ez, 2.0 ** -8, owned, 7.0)
    # the plain product's backward: no rounding of its own
    dY = spoil(rand(g, h.rows, 2 * N), owned)
    dX2 = torch.full_like(dX, 7.0)
    _, dW2 = B.moe_grouped_gemm_bwd(h, dY, X, W, dX=dX2)
    D = np.nan_to_num(f64(dY))
    check_bwd(D, X, W, segs, dX2, dW2, np.zeros_like(D), 0.0, owned, 7.0)
    # each gradient alone: the same bits
    dX3 = torch.full_like(dX, 7.0)
    assert B.moe_grouped_gemm_bwd(h, dY, X, W, need_dw=False, dX=dX3)[1] is None
    none, dW3 = B.moe_grouped_gemm_bwd(h, dY, X, W, need_dx=False)
    assert none is None and torch.equal(dX3, dX2) and torch.equal(dW3, dW2)
    assert h.status() & ~B.MOE_DEV_ROWS_EXCEEDED == 0  # a layout with a bound says that it was reached


@pytest.mark.parametrize("kind", ["dropless", "capacity", "kmajor", "padded", "absent", "bound"])
@pytest.mark.parametrize("s,e,k,K,N", [(1, 4, 2, 64, 8), (9, 8, 2, 72, 24), (100, 8, 3, 128, 136), (700, 16, 4, 264, 128),
                                       (1500, 4, 2, 512, 264), (900, 60, 6, 136, 72)])
def test_layouts(kind, s, e, k, K, N):
    run_all(layout(s, e, k, kind, seed=s), s, K, N, "silu", seed=s)


# segments that end at, before and behind 16, 64, 128 and 256 rows; empty ones first, last and between
@pytest.mark.parametrize("counts", [[0, 1, 0], [15, 16, 17, 0], [0, 63, 64, 65], [127, 128, 129], [255, 256, 257, 1],
                                    [1] * 40, [0, 0, 1000, 3], [513, 0, 511, 0, 2, 0]])
def test_segment_lengths(counts):
    run_all(layout(sum(counts), len(counts), 1, counts=counts), sum(counts), 200, 104, "gelu_tanh", seed=len(counts))


# few rows an expert: blocks of 16 of one expert, several chunks of the contracted axis, more columns than SMs and fewer
@pytest.mark.parametrize("counts,K,N", [([40, 0, 0, 9, 17] + [0] * 40, 200, 72), ([2] * 30, 2600, 136), ([1], 4104, 8),
                                        ([0, 16], 2048, 512), ([3, 0, 1, 33] + [0] * 20, 64, 2504)])
def test_few_rows(counts, K, N):
    run_all(layout(sum(counts), len(counts), 1, counts=counts), sum(counts), K, N, "silu", seed=K)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_activations(act):
    run_all(layout(333, 6, 2, seed=3), 333, 96, 56, act, seed=5)


# more units than pairs of SMs, with and without cut last blocks
@pytest.mark.parametrize("s,e,k,K,N", [(5000, 8, 2, 1032, 520), (3000, 100, 4, 520, 264)])
def test_many_units(s, e, k, K, N):
    run_all(layout(s, e, k, seed=1), s, K, N, "silu", seed=2)


def test_no_rows():
    h = layout(0, 4, 2)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(4, 32, 64, dtype=torch.bfloat16, device="cuda")
    assert B.moe_grouped_gated(h, x, W).shape == (0, 16)
    assert B.moe_dispatch_grouped_gated(h, x, W).shape == (0, 16)
    z = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    dX, dW = B.moe_grouped_gemm_bwd(h, z, x, W)
    assert dX.shape == (0, 64) and not dW.any()
    dX, dW = B.moe_grouped_gated_bwd(h, z[:, :16].contiguous(), x, W, z)
    assert dX.shape == (0, 64) and not dW.any()


def test_two_streams_at_once():
    """The same handle and weights on two streams: each call has a workspace of its own."""
    s, e, k, K, N = 2000, 8, 2, 512, 256
    g = torch.Generator().manual_seed(9)
    h = layout(s, e, k, seed=9)
    W = rand(g, e, 2 * N, K, scale=K ** -0.5)
    sets = [(rand(g, s * k, N), rand(g, s * k, K), rand(g, s * k, 2 * N)) for _ in range(2)]
    want = [B.moe_grouped_gated_bwd(h, dH, X, W, Z) for dH, X, Z in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(B.moe_grouped_gated_bwd(h, sets[i][0], sets[i][1], W, sets[i][2]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_a_training_chain_in_a_captured_graph():
    s, e, k, m, n = 600, 8, 2, 128, 64
    g = torch.Generator().manual_seed(1)
    x, Wi, Wo = rand(g, s, m), rand(g, e, 2 * n, m, scale=0.1), rand(g, e, m, n, scale=0.1)
    logits = torch.randn(s, e, generator=g).cuda()
    h = B.moe_layout_create(s, e, k)

    def step(wait=False):
        outs = []

        def do(*r):
            outs.extend(t for t in r if t is not None)
            if wait:
                torch.cuda.synchronize()
            return r

        idx, gate = do(*B.moe_topk_gate_layout(h, logits))
        X, = do(B.moe_dispatch(h, x))
        H, Z = do(*B.moe_grouped_gated(h, X, Wi, save_z=True))
        Y, = do(B.moe_grouped_gemm(h, H, Wo))
        out, = do(B.moe_combine(h, Y, gate))
        dY, dg = do(*B.moe_combine_bwd(h, out, gate, Y))
        dH, dWo = do(*B.moe_grouped_gemm_bwd(h, dY, H, Wo))
        dX, dWi = do(*B.moe_grouped_gated_bwd(h, dH, X, Wi, Z))
        do(B.moe_dispatch_bwd(h, dX))
        do(B.moe_clip_grad_norm([dWo, dWi], 1e-3))
        return outs

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(s, m, generator=g))
        logits.copy_(torch.randn(s, e, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in out]
        for i, (a, c) in enumerate(zip(have, step(True))):
            assert torch.equal(a, c), i
