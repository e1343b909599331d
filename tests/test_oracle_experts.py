"""Pins of the 64-bit forms of the gated products and the experts' gradients:
hand-worked values, and differences of the forward pass (no GPU needed)."""
import numpy as np
import pytest

from oracle import experts as E
from oracle.block import act

KINDS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def test_gated_by_hand():
    x = np.array([[1.0, 2.0]])
    W = np.array([[1.0, 1.0], [-1.0, 0.0], [2.0, 0.0], [0.0, 3.0]])  # gate rows, factor rows
    h, z = E.gated(x, W, np.array([0.0, 0.5, 0.0, 1.0]), "relu")
    np.testing.assert_array_equal(z, [[3.0, -0.5, 2.0, 7.0]])
    np.testing.assert_array_equal(h, [[6.0, 0.0]])


@pytest.mark.parametrize("kind", KINDS)
def test_gated_gradients_by_differences(kind):
    r = np.random.default_rng(1)
    x, W, b, dh = r.normal(size=(3, 5)), r.normal(size=(8, 5)), r.normal(size=8), r.normal(size=(3, 4))
    f = lambda x, W, b: float((E.gated(x, W, b, kind)[0] * dh).sum())  # noqa: E731
    dx, dW, db, _ = E.gated_bwd(dh, x, W, E.gated(x, W, b, kind)[1], kind)
    eps = 1e-6
    for i, (a, d) in enumerate(((x, dx), (W, dW), (b, db))):
        for at in np.ndindex(a.shape):
            args = [x, W, b]
            up, down = a.copy(), a.copy()
            up[at] += eps
            down[at] -= eps
            args[i] = up
            hi = f(*args)
            args[i] = down
            assert abs((hi - f(*args)) / (2 * eps) - d[at]) < 1e-6


def test_grouped_is_gated_for_each_expert_and_leaves_other_rows():
    r = np.random.default_rng(2)
    X, W = r.normal(size=(9, 4)), r.normal(size=(3, 6, 4))
    segs = E.segments([0, 4, 6], [3, 0, 2])
    H, Z = E.grouped_gated(X, W, segs, "silu")
    assert np.isnan(H[3:6]).all() and np.isnan(Z[8]).all()
    z = X[7] @ W[2].T
    np.testing.assert_allclose(H[7], act(z[:3], "silu") * z[3:])


def test_grouped_gradients_by_differences():
    r = np.random.default_rng(3)
    X, W, dY = r.normal(size=(7, 4)), r.normal(size=(3, 5, 4)), r.normal(size=(7, 5))
    segs = E.segments([0, 2, 2], [2, 0, 5])
    dX, dW = E.grouped_bwd(dY, X, W, segs)
    f = lambda X, W: sum(float((X[r] @ W[x].T * dY[r]).sum()) for x, r in enumerate(segs))  # noqa: E731
    eps = 1e-6
    for a, d, i in ((X, dX, 0), (W, dW, 1)):
        for at in np.ndindex(a.shape):
            up, down = a.copy(), a.copy()
            up[at] += eps
            down[at] -= eps
            args = (up, W) if i == 0 else (X, up), (down, W) if i == 0 else (X, down)
            assert abs((f(*args[0]) - f(*args[1])) / (2 * eps) - d[at]) < 1e-7
    assert not dW[1].any()


def test_clip():
    norm, c = E.clip([np.array([3.0]), np.array([4.0])], 1.0)
    assert norm == 5.0 and abs(c - 0.2) < 1e-6
    assert E.clip([np.array([0.3])], 1.0)[1] == 1.0
    assert E.clip([], 1.0) == (0.0, 1.0)
