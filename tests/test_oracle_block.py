"""The plain 64-bit forms of the layer norm, the balance loss and the dense
products: closed forms on small cases, and every gradient against central
differences of its forward form."""
import numpy as np
import pytest

from oracle import block as O


def diff(f, x, v, h=1e-6):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_layernorm_closed_forms():
    y, mean, rstd = O.layernorm(np.array([[1.0, 3.0], [5.0, 5.0]]), eps=1e-30)
    np.testing.assert_allclose(y, [[-1.0, 1.0], [0.0, 0.0]], atol=1e-12)
    np.testing.assert_allclose(mean, [2.0, 5.0])
    assert rstd[0] == pytest.approx(1.0)
    # shifting a row, or scaling it when eps is negligible, leaves y as it was
    x = np.random.default_rng(0).normal(size=(3, 50))
    a = O.layernorm(x, eps=1e-30)[0]
    np.testing.assert_allclose(O.layernorm(3 * x + 7, eps=1e-30)[0], a, atol=1e-10)


@pytest.mark.parametrize("affine", [False, True])
def test_layernorm_gradients_against_differences(affine):
    r = np.random.default_rng(1)
    x, dy = r.normal(size=(4, 9)) * 2 + 1, r.normal(size=(4, 9))
    w, b = (r.normal(size=9), r.normal(size=9)) if affine else (None, None)
    _, mean, rstd = O.layernorm(x, w, b)
    dx, dw, db = O.layernorm_bwd(dy, x, w, mean, rstd)
    v = r.normal(size=x.shape)
    assert diff(lambda a: (O.layernorm(a, w, b)[0] * dy).sum(), x, v) == pytest.approx((dx * v).sum(), rel=1e-6)
    if affine:
        u = r.normal(size=9)
        assert diff(lambda a: (O.layernorm(x, a, b)[0] * dy).sum(), w, u) == pytest.approx((dw * u).sum(), rel=1e-6)
        assert diff(lambda a: (O.layernorm(x, w, a)[0] * dy).sum(), b, u) == pytest.approx((db * u).sum(), rel=1e-6)


def test_balance_loss_of_uniform_routing_is_one():
    # uniform probabilities and uniform counts: e * sum_j (1/e)(1/e) = 1; lse = log e
    s, e = 8, 4
    r = O.balance_loss(np.zeros((s, e)), np.arange(s)[:, None] % e)
    assert r["loss"][0] == pytest.approx(1.0)
    assert r["loss"][1] == pytest.approx(np.log(e) ** 2)
    np.testing.assert_array_equal(r["counts"], [[2] * 4])


def test_balance_loss_masks():
    r = np.random.default_rng(2)
    logits, idx = r.normal(size=(10, 5)), r.integers(0, 5, size=(10, 2))
    valid = np.ones(10, np.uint8)
    valid[[2, 7]] = 0
    a = O.balance_loss(logits, idx, valid)
    keep = valid != 0
    b = O.balance_loss(logits[keep], idx[keep])
    np.testing.assert_allclose(a["loss"], b["loss"])
    np.testing.assert_array_equal(a["counts"], b["counts"])
    none = O.balance_loss(logits, idx, np.zeros(10, np.uint8), np.array([0, 4, 4, 10]))
    assert not none["loss"].any() and not none["counts"].any()


@pytest.mark.parametrize("seqs", [None, [0, 3, 3, 9], [1, 4, 8]])
def test_balance_gradient_against_differences(seqs):
    r = np.random.default_rng(3)
    logits, idx = r.normal(size=(9, 6)), r.integers(0, 6, size=(9, 2))
    valid = (r.random(9) < 0.8).astype(np.uint8)
    off = None if seqs is None else np.array(seqs)
    f = O.balance_loss(logits, idx, valid, off)
    d = O.balance_loss_bwd(logits, f["lse"], f["coef"], f["norm"], [0.7, 0.3], valid, off)
    v = r.normal(size=logits.shape)
    got = diff(lambda a: float((O.balance_loss(a, idx, valid, off)["loss"] * [0.7, 0.3]).sum()), logits, v)
    assert got == pytest.approx((d * v).sum(), rel=1e-6)


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_gradients_against_differences(kind):
    r = np.random.default_rng(4)
    x, W, b, dy = r.normal(size=(5, 7)), r.normal(size=(3, 7)), r.normal(size=3), r.normal(size=(5, 3))
    z = O.linear(x, W, b)[1]
    dx, dW, db, _ = O.linear_bwd(dy, x, W, z, kind)
    for g, at, f in ((dx, x, lambda a: O.linear(a, W, b, kind)[0]), (dW, W, lambda a: O.linear(x, a, b, kind)[0]),
                     (db, b, lambda a: O.linear(x, W, a, kind)[0])):
        v = r.normal(size=at.shape)
        assert diff(lambda a: (f(a) * dy).sum(), at, v) == pytest.approx((g * v).sum(), rel=1e-6)
