"""Layer norm, forward and backward, against the plain 64-bit form.

Tolerances come from counting fp32 roundings (u = 2^-24).  A reduction over m
elements adds at most n_add = 64 + m/512 terms in a row (registers of a
thread, then trees), so a mean is off by n_add u times the mean of the
magnitudes, and rstd by about n_add/2 u of itself.  With bf16 outputs half a
unit in the last place (2^-8 of the value) comes on top."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B
from oracle import block as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().cpu().double().numpy()


def half_ulp(v, dtype):
    return np.abs(v) * 2.0 ** -8 + 1e-40 if dtype == "bf16" else np.abs(v) * U + 1e-40


def make(s, m, dtype, wdtype, seed, scale=1.0, offset=0.25):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(s, m, generator=g) * scale + offset).to(DT[dtype])
    w = (1 + 0.2 * torch.randn(m, generator=g)).to(DT[wdtype]) if wdtype else None
    b = (0.1 * torch.randn(m, generator=g)).to(DT[wdtype]) if wdtype else None
    dy = torch.randn(s, m, generator=g).to(DT[dtype])
    res = torch.randn(s, m, generator=g).to(DT[dtype])
    return [t.cuda() if t is not None else None for t in (x, w, b, dy, res)]


def check_fwd(x, w, b, out, dtype, eps=1e-5):
    y, mean, rstd = (f64(t) for t in out)
    X, W = f64(x), None if w is None else f64(w)
    oy, om, orr = O.layernorm(X, W, None if b is None else f64(b), eps)
    n = (64 + X.shape[1] / 512) * U
    mag = np.abs(X).mean(-1)
    assert (np.abs(mean - om) <= n * mag + 1e-40).all()
    # rstd: relative error of the variance / 2, and of the mean's error inside it
    dm = n * mag * orr
    assert (np.abs(rstd - orr) <= orr * (n + 4 * U + dm * dm + 2 * dm * U)).all()
    wa = np.ones(X.shape[1]) if W is None else np.abs(W)
    xh = np.abs(X - om[:, None]) * orr[:, None]
    tol = wa * (dm[:, None] * (1 + xh * dm[:, None]) + xh * (n + 8 * U)) + 4 * U * np.abs(oy) + half_ulp(oy, dtype)
    if b is not None:
        tol = tol + 2 * U * np.abs(f64(b))
    bad = np.abs(y - oy) > tol
    assert not bad.any(), (np.abs(y - oy) / tol).max()


def check_bwd(dy, x, w, mean, rstd, res, out, dtype):
    dx, dw, db = out
    D, X, W = f64(dy), f64(x), None if w is None else f64(w)
    s, m = X.shape
    ox, ow, ob = O.layernorm_bwd(D, X, W, f64(mean), f64(rstd), None if res is None else f64(res))
    r = f64(rstd)[:, None]
    xh = np.abs(X - f64(mean)[:, None]) * r
    g = np.abs(D) if W is None else np.abs(D * W)
    n = (64 + m / 512) * U
    c1, c2 = g.mean(-1, keepdims=True), (g * xh).mean(-1, keepdims=True)
    tol = r * (n * (c1 + xh * c2) + 8 * U * (g + c1 + xh * c2)) + half_ulp(ox, dtype)
    if res is not None:
        tol = tol + 2 * U * np.abs(f64(res))
    assert (np.abs(f64(dx) - ox) <= tol).all()
    # a column's sum: at most s/150 rows in a register, then up to 8 groups and 40 + 16 partial rows
    k = (96 + s / 150) * U
    if dw is not None:
        assert (np.abs(f64(dw) - ow) <= k * (np.abs(D) * xh).sum(0) + 1e-40).all()
    if db is not None:
        assert (np.abs(f64(db) - ob) <= k * np.abs(D).sum(0) + 1e-40).all()


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 64), (33, 130), (70, 512), (9, 1000), (17, 1024), (4, 2815), (301, 2816), (31, 4097),
          (700, 384), (8, 8192), (6, 8200), (5, 16384), (3, 16385), (2, 32768), (2, 40000), (3, 40001), (2000, 40), (1, 33)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16"),
                                          ("bf16", None)])
@pytest.mark.parametrize("s,m", SHAPES)
def test_layernorm_and_gradient(s, m, dtype, wdtype):
    x, w, b, dy, res = make(s, m, dtype, wdtype, seed=s * 7 + m)
    out = B.moe_layernorm(x, w, b)
    check_fwd(x, w, b, out, dtype)
    _, mean, rstd = out
    check_bwd(dy, x, w, mean, rstd, None, B.moe_layernorm_bwd(dy, x, w, mean, rstd), dtype)
    check_bwd(dy, x, w, mean, rstd, res, B.moe_layernorm_bwd(dy, x, w, mean, rstd, dres=res), dtype)


# enough rows that every group walks over several and the ring goes round, in every width's form
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("s,m", [(30000, 40), (21000, 64), (6000, 256), (5003, 70), (5001, 515), (3001, 1000), (2600, 1537),
                                 (1300, 4096), (1300, 4098), (700, 8192), (640, 8193), (500, 9000), (330, 16384), (321, 16400),
                                 (310, 16385)])
def test_many_rows(s, m, dtype):
    x, w, b, dy, res = make(s, m, dtype, "f32", seed=s + m)
    out = B.moe_layernorm(x, w, b)
    check_fwd(x, w, b, out, dtype)
    _, mean, rstd = out
    check_bwd(dy, x, w, mean, rstd, res, B.moe_layernorm_bwd(dy, x, w, mean, rstd, dres=res), dtype)
    check_bwd(dy, x, w, mean, rstd, None, B.moe_layernorm_bwd(dy, x, w, mean, rstd), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,ld", [(256, 264), (256, 259), (250, 256), (9000, 9016), (33, 50)])
def test_strided_rows(dtype, m, ld):
    s = 37
    g = torch.Generator().manual_seed(m)
    big = [torch.randn(s, ld, generator=g).to(DT[dtype]).cuda() for _ in range(3)]
    x, dy, res = (t[:, :m] for t in big)
    w = torch.randn(m, generator=g).cuda()
    out = B.moe_layernorm(x, w, w)
    check_fwd(x, w, w, out, dtype)
    _, mean, rstd = out
    check_bwd(dy, x, w, mean, rstd, res, B.moe_layernorm_bwd(dy, x, w, mean, rstd, dres=res), dtype)


def test_large_offset_and_outliers():
    # a common offset of 300 standard deviations: E[x^2] - mu^2 would lose the variance
    x, w, b, dy, _ = make(20, 2048, "f32", "f32", seed=5, scale=0.01, offset=3.0)
    x[:, 7] = 50.0
    out = B.moe_layernorm(x, w, b)
    check_fwd(x, w, b, out, "f32")
    check_bwd(dy, x, w, out[1], out[2], None, B.moe_layernorm_bwd(dy, x, w, out[1], out[2]), "f32")


def test_constant_rows_and_nonfinite_rows_stay_apart():
    x = torch.randn(6, 512).cuda()
    x[1] = 2.5
    x[3, 9] = float("nan")
    x[4, 0] = float("inf")
    y, mean, rstd = B.moe_layernorm(x)
    assert (y[1] == 0).all() and rstd[1].item() == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).any()
    keep = [0, 1, 2, 5]
    check_fwd(x[keep], None, None, (y[keep], mean[keep], rstd[keep]), "f32")


def test_optional_outputs_and_empty_batches():
    x, w, b, dy, _ = make(40, 256, "bf16", "bf16", seed=1)
    y, mean, rstd = B.moe_layernorm(x, w, b)
    assert torch.equal(B.moe_layernorm(x, w, b, stats=False), y)
    dx, dw, db = B.moe_layernorm_bwd(dy, x, w, mean, rstd)
    a = B.moe_layernorm_bwd(dy, x, w, mean, rstd, need_dweight=False, need_dbias=False)
    assert a[1] is None and a[2] is None and torch.equal(a[0], dx)
    a = B.moe_layernorm_bwd(dy, x, w, mean, rstd, need_dweight=False)
    assert a[1] is None and torch.equal(a[2], db)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    n = torch.empty(0, device="cuda")
    assert B.moe_layernorm(e, w, b)[0].shape == (0, 256)
    dx, dw, db = B.moe_layernorm_bwd(e, e, w, n, n)
    assert dx.shape == (0, 256) and not dw.any() and not db.any()


def test_same_bits_on_every_run_and_on_another_stream():
    x, w, b, dy, res = make(3000, 1024, "bf16", "f32", seed=2)
    _, mean, rstd = B.moe_layernorm(x, w, b)
    first = B.moe_layernorm_bwd(dy, x, w, mean, rstd, dres=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = B.moe_layernorm_bwd(dy, x, w, mean, rstd, dres=res)
    side.synchronize()
    for a, c in zip(first, again):
        assert torch.equal(a, c)


def test_gradient_against_differences_of_the_64_bit_form():
    x, w, b, dy, _ = make(6, 200, "f32", "f32", seed=3)
    _, mean, rstd = B.moe_layernorm(x, w, b)
    dx, dw, db = (f64(t) for t in B.moe_layernorm_bwd(dy, x, w, mean, rstd))
    X, W, b64, D = f64(x), f64(w), f64(b), f64(dy)
    r, h = np.random.default_rng(0), 1e-6
    for _ in range(3):
        v, u = r.normal(size=X.shape), r.normal(size=200)
        num = ((O.layernorm(X + h * v, W, b64)[0] - O.layernorm(X - h * v, W, b64)[0]) * D).sum() / (2 * h)
        # fp32 gradients: 1e-5 of the sum of the terms' magnitudes is far above their error
        assert abs(num - (dx * v).sum()) <= 1e-5 * np.abs(dx * v).sum()
        num = ((O.layernorm(X, W + h * u, b64)[0] - O.layernorm(X, W - h * u, b64)[0]) * D).sum() / (2 * h)
        assert abs(num - (dw * u).sum()) <= 1e-5 * np.abs(dw * u).sum()
        num = ((O.layernorm(X, W, b64 + h * u)[0] - O.layernorm(X, W, b64 - h * u)[0]) * D).sum() / (2 * h)
        assert abs(num - (db * u).sum()) <= 1e-5 * np.abs(db * u).sum()


def test_refusals():
    x = torch.randn(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    y, mean, rstd = B.moe_layernorm(x, w)
    for bad in (lambda: B.moe_layernorm(x.half()), lambda: B.moe_layernorm(x, w[:8]), lambda: B.moe_layernorm(x, w, w.bfloat16()),
                lambda: B.moe_layernorm(x, w, eps=0.0), lambda: B.moe_layernorm(x, w, eps=float("inf")),
                lambda: B.moe_layernorm(x, w, y=torch.empty(4, 8, device="cuda")), lambda: B.moe_layernorm(x.cpu(), w.cpu()),
                lambda: B.moe_layernorm(x, w.cpu()), lambda: B.moe_layernorm_bwd(y.bfloat16(), x, w, mean, rstd),
                lambda: B.moe_layernorm_bwd(y, x, w, mean[:2], rstd), lambda: B.moe_layernorm_bwd(y, x, w, mean, rstd, dres=y[:2]),
                lambda: B.moe_layernorm(x.view(-1)[1:17].view(1, 16))):
        with pytest.raises(B.MoEError):
            bad()
    for bad in (lambda: B.moe_layernorm(x.t()), lambda: B.moe_layernorm(x[0]),
                lambda: B.moe_layernorm(x[:1].expand(4, 16))):
        with pytest.raises(ValueError):
            bad()
