"""The balance loss where its numbers get large: rows of huge finite logits,
against the plain 64-bit form.

Tolerances: as for the ordinary sizes (u = 2^-24), 320 u of a mean
probability and 512 u of the balance loss.  The largest term of a row's
softmax is exactly 1 whatever its size, and logits this large differ either by
nothing or by far more than exp can show, so no part of the bound grows with
them.  lse is one fp32: half a unit of its last place, and 8 u of the
logarithm."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B
from oracle import block as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = (-1e3, -1e9, -1e10, -1e11, -1e12, -1e30, -1e38, -1.7e38, -3.3895313892515355e38, 1e3, 1e10, 1e30, 3e38)


def f64(t):
    return t.detach().cpu().double().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(logits, idx, dloss=(0.7, 0.3)):
    s, e = logits.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = B.moe_balance_loss(dev(logits), dev(idx), device_status=st)
    assert st.item() == 0
    L = logits.astype(np.float64)
    ref = O.balance_loss(L, idx)
    np.testing.assert_array_equal(got.counts.cpu().numpy(), ref["counts"])
    assert (np.abs(f64(got.mean_prob) - ref["mean_prob"]) <= 320 * U * ref["mean_prob"]).all()
    assert abs(f64(got.loss)[0] - ref["loss"][0]) <= 512 * U * ref["loss"][0]
    assert (np.abs(f64(got.lse) - ref["lse"]) <= U * np.abs(ref["lse"]) + 8 * U * 6).all()
    # the z loss is the infinity that fp32 makes of it, or itself
    with np.errstate(over="ignore"):
        z = np.float32(ref["loss"][1])
    if np.isinf(z):
        assert f64(got.loss)[1] == np.inf
    else:
        assert abs(f64(got.loss)[1] - ref["loss"][1]) <= 320 * U * ref["loss"][1] + 64 * U
    # the gradient, from what the forward pass kept; p by the definition
    d = f64(B.moe_balance_loss_bwd(dev(logits), got.lse, got.coef, got.norm, torch.tensor(dloss).cuda()))
    p, _ = O._softmax(L)
    c, dl = f64(got.coef)[0], np.float32(dloss).astype(np.float64)
    lse = f64(got.lse)[:, None]
    want = dl[0] * p * (c - (p * c).sum(1, keepdims=True)) + dl[1] / s * 2 * lse * p
    tol = 128 * U * p * (2 * c.max() * dl[0] + 2 * dl[1] / s * np.abs(lse)) + 2 * U * np.abs(want) + 1e-30
    assert (np.abs(d - want) <= tol).all()
    return got


@pytest.mark.parametrize("e", [1, 8, 20, 37, 128, 256])
@pytest.mark.parametrize("size", SIZES)
def test_rows_of_one_huge_value(size, e):
    # a router whose mask is a finite number, and leaves rows nothing else: p = 1/e there
    logits = np.random.default_rng(e).normal(size=(70, e)).astype(np.float32)
    logits[::3] = np.float32(size)
    idx = np.tile(np.arange(min(e, 2), dtype=np.int32), (70, 1))
    check(logits, idx)


@pytest.mark.parametrize("size", SIZES)
def test_rows_with_a_part_masked_and_a_huge_maximum(size):
    e = 24
    logits = np.random.default_rng(1).normal(size=(50, e)).astype(np.float32)
    logits[::2, 5:] = np.float32(size)         # a part of the experts masked, or far ahead of the others
    logits[1::4] = np.float32(size)
    logits[1::4, 3] = -np.inf                  # a real mask beside them
    check(logits, np.tile(np.array([0, 3], np.int32), (50, 1)))


def test_random_rows_of_every_size():
    r = np.random.default_rng(2)
    logits = (r.normal(size=(300, 32)) * 10.0 ** r.uniform(-3, 37, size=(300, 1))).astype(np.float32)
    check(logits, np.argsort(-logits, axis=1)[:, :2].astype(np.int32))


@pytest.mark.parametrize("s", [2 ** 31 - 1, 2 ** 31 - 4097])
def test_as_many_tokens_as_are_accepted(s):
    # one expert, so that s * e may come to 2^31 - 1: token numbers and the ends of blocks at the edge of an int.
    # p = 1, lse = the logit: everything can be said without a reference of this size (four arrays of 8.6 GB)
    logits = torch.full((s, 1), 0.5, device="cuda")
    logits[-3000:] = torch.arange(3000, device="cuda").float()[:, None] / 1024
    idx = torch.zeros(s, 1, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, s - 2000, s - 5], dtype=torch.int32).cuda()  # the last five tokens belong to nobody
    for offsets, live in ((None, s), (off, s - 5)):
        r = B.moe_balance_loss(logits, idx, None, offsets)
        assert torch.equal(r.lse[:live], logits[:live, 0]) and not r.lse[live:].any()
        assert r.counts[:, 0].tolist() == ([s] if offsets is None else [s - 2000, 1995])
        assert abs(r.loss[0].item() - 1) <= 512 * U and ((r.mean_prob - 1).abs() <= 320 * U).all()
        z = 0.25 * (s - 3000) + float(np.square(np.arange(3000 - (s - live)) / 1024).sum())
        assert abs(r.loss[1].item() - z / live) <= 320 * U * z / live
        d = B.moe_balance_loss_bwd(logits, r.lse, r.coef, r.norm, torch.tensor([0.7, 0.3 * live]).cuda(), None, offsets)
        # dz = 0.3 * 2 lse; c - dot is 0 but for the roundings of p = 1 (2 u) times coef (about 1/T)
        want = 0.6 * logits[:, 0]
        assert ((d[:live, 0] - want[:live]).abs() <= 16 * U * (1 + want[:live])).all() and not d[live:].any()
        del d, want, r
