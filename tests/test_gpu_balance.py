"""The balance loss, its counts and its gradient, against the plain 64-bit form.

Tolerances from counting fp32 roundings (u = 2^-24).  A probability's error
is a few u plus u times the distance of its logit from the row's maximum (the
argument of exp; under 64 here): 128 u of itself.  A sequence's mean adds at
most 64 rows in a lane, 16 steps of trees and 96 pieces: below 192 u more, so
320 u of the mean in all, and the losses, sums of positive terms, 512 u."""
import numpy as np
import pytest
import torch

from combine_moe_topk_gb300 import binding as B
from oracle import block as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def make(s, e, k, seqs=1, masked=0.0, zipf=0.0, seed=0):
    r = np.random.default_rng(seed)
    logits = (r.normal(size=(s, e)) * 2 - zipf * np.log(np.arange(1, e + 1))).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    valid = (r.random(s) >= masked).astype(np.uint8) if masked else None
    off = None
    if seqs > 1:
        off = np.concatenate([[0], np.sort(r.integers(0, s + 1, seqs - 1)), [s]]).astype(np.int32)
    return logits, idx, valid, off


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_both(logits, idx, valid=None, off=None, dloss=(0.7, 0.3), add=None):
    got = B.moe_balance_loss(dev(logits), dev(idx), dev(valid), dev(off))
    ref = O.balance_loss(logits.astype(np.float64), idx, valid, off)
    np.testing.assert_array_equal(got.counts.cpu().numpy(), ref["counts"])
    assert (np.abs(f64(got.mean_prob) - ref["mean_prob"]) <= 320 * U * ref["mean_prob"]).all()
    inf = np.isneginf(ref["lse"])
    lse = f64(got.lse)
    assert (np.isneginf(lse) == inf).all()
    scale = np.abs(logits.astype(np.float64), where=np.isfinite(logits), out=np.zeros(logits.shape)).max(1)
    assert (np.abs(lse - ref["lse"])[~inf] <= (8 * U + 2 * U * (scale + np.abs(ref["lse"])))[~inf]).all()
    loss = f64(got.loss)
    assert abs(loss[0] - ref["loss"][0]) <= 512 * U * ref["loss"][0]
    zmag = (np.square(ref["lse"][~inf]) + 2 * np.abs(ref["lse"][~inf]) * (1 + scale[~inf])).sum() * ref["norm"][1]
    assert abs(loss[1] - ref["loss"][1]) <= 320 * U * zmag
    np.testing.assert_allclose(f64(got.norm), ref["norm"], rtol=4 * U)
    assert (np.abs(f64(got.coef) - ref["coef"]) <= 8 * U * ref["coef"]).all()
    # the gradient, from what the forward pass kept
    d = B.moe_balance_loss_bwd(dev(logits), got.lse, got.coef, got.norm, torch.tensor(dloss).cuda(), dev(valid), dev(off),
                               add=dev(add))
    # the kernel reads dloss, lse, coef, norm as fp32: so does the reference
    od = O.balance_loss_bwd(logits.astype(np.float64), lse, f64(got.coef), f64(got.norm),
                            np.float32(dloss).astype(np.float64), valid, off, add)
    cmax = f64(got.coef).max() * abs(dloss[0]) * ref["norm"][0]
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(inf[:, None], 0.0, np.exp(np.minimum(0.0, logits.astype(np.float64) - np.where(inf, 0.0, lse)[:, None])))
    # a row's dot product: 8 + 5 additions; with the argument of exp: 128 u of the terms
    zl = np.where(inf, 0.0, np.abs(lse))[:, None]
    tol = 128 * U * p * (2 * cmax + 2 * abs(dloss[1]) * ref["norm"][1] * zl) + 2 * U * np.abs(od) + 1e-30
    if add is not None:
        tol = tol + 2 * U * np.abs(add)
    live = np.ones(len(logits), bool) if valid is None else valid != 0
    tol = np.where(live[:, None], tol, 0.0 if add is None else 0.0)
    assert (np.abs(f64(d) - od) <= tol).all()
    return got, d


@pytest.mark.parametrize("e", [1, 2, 3, 4, 5, 8, 12, 16, 31, 32, 60, 64, 100, 127, 128, 129, 160, 250, 255, 256])
@pytest.mark.parametrize("s", [1, 7, 300])
def test_every_lane_shape(s, e):
    run_both(*make(s, e, min(e, 3), seed=s + e))


@pytest.mark.parametrize("s,e,k,seqs,masked", [(1000, 8, 2, 1, 0.2), (2500, 64, 6, 9, 0.1), (4096, 128, 8, 4, 0.0),
                                               (3001, 60, 4, 40, 0.3), (700, 256, 8, 200, 0.5), (64, 16, 2, 64, 0.9)])
def test_packed_sequences_and_padding(s, e, k, seqs, masked):
    logits, idx, valid, off = make(s, e, k, seqs, masked, zipf=1.2, seed=s)
    add = np.random.default_rng(1).normal(size=(s, e)).astype(np.float32) * 0.01
    run_both(logits, idx, valid, off, add=add)


def test_every_token_its_own_sequence_and_tokens_outside():
    logits, idx, _, _ = make(130, 12, 2, seed=3)
    run_both(logits, idx, None, np.arange(131, dtype=np.int32))
    run_both(logits, idx, None, np.array([10, 10, 55, 55, 120], np.int32))  # rows before 10 and from 120 on take no part
    run_both(logits, idx, None, np.array([0, 0], np.int32))


def test_nothing_valid_and_empty_batch():
    logits, idx, _, off = make(50, 8, 2, seqs=3, seed=4)
    got, d = run_both(logits, idx, np.zeros(50, np.uint8), off)
    assert not got.loss.any() and not d.any() and not got.lse.any()
    for offsets in (None, torch.zeros(4, dtype=torch.int32, device="cuda")):
        r = B.moe_balance_loss(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                               seq_offsets=offsets)
        assert not r.loss.any() and not r.counts.any() and not r.mean_prob.any() and not r.coef.any()
        assert (r.norm == 1).all()


def test_masked_tokens_may_hold_anything():
    logits, idx, _, _ = make(200, 24, 2, seed=5)
    valid = (np.arange(200) % 3 != 0).astype(np.uint8)
    got, d = run_both(logits, idx, valid)
    dirty, didx = logits.copy(), idx.copy()
    dirty[valid == 0] = np.nan
    dirty[0] = np.inf
    didx[valid == 0] = 10 ** 6
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = B.moe_balance_loss(dev(dirty), dev(didx), dev(valid), device_status=st)
    assert st.item() == 0
    for a, b in zip(r, got):
        assert torch.equal(a, b)
    d2 = B.moe_balance_loss_bwd(dev(dirty), r.lse, r.coef, r.norm, torch.tensor([0.7, 0.3]).cuda(), dev(valid))
    assert torch.equal(d, d2) and not d2[dev(valid) == 0].any()


def test_masked_experts_and_rows_of_nothing():
    logits, idx, _, _ = make(64, 20, 2, seed=6)
    logits[:, 13:] = -np.inf          # experts masked out of the router
    logits[5] = -np.inf               # a row whose mask leaves nothing
    logits[6] = np.finfo(np.float32).min   # the same with the type's lowest value
    idx = np.minimum(idx, 12)
    got, d = run_both(logits, idx)
    assert not d[5].any() and not d[6].any() and torch.isfinite(d).all()
    assert not got.mean_prob[0, 13:].any()


def test_bad_ids_and_nonfinite_logits_are_flagged():
    logits, idx, _, _ = make(100, 8, 2, seed=7)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx2 = idx.copy()
    idx2[3, 1] = -1  # absent: not counted, no flag
    r = B.moe_balance_loss(dev(logits), dev(idx2), device_status=st)
    assert st.item() == 0 and r.counts.sum().item() == 199
    idx2[4, 0], idx2[5, 0] = 8, -2
    r = B.moe_balance_loss(dev(logits), dev(idx2), device_status=st)
    assert st.item() == B.MOE_DEV_BAD_ROUTE and r.counts.sum().item() == 197
    for v in (np.nan, np.inf):
        st.zero_()
        bad = logits.copy()
        bad[50, 2] = v
        r = B.moe_balance_loss(dev(bad), dev(idx), device_status=st)
        assert st.item() == B.MOE_DEV_NONFINITE and torch.isnan(r.loss[0])


def test_counts_with_one_hot_expert_and_same_bits():
    # every token to expert 0: the hottest counter
    s = 20000
    logits, _, _, _ = make(s, 128, 1, seed=8)
    idx = np.zeros((s, 1), np.int32)
    got, _ = run_both(logits, idx)
    assert got.counts[0, 0].item() == s
    again = B.moe_balance_loss(dev(logits), dev(idx))
    for a, b in zip(got, again):
        assert torch.equal(a, b)


def test_gradient_in_place_and_against_differences():
    logits, idx, valid, off = make(60, 10, 2, seqs=3, masked=0.1, seed=9)
    got, d = run_both(logits, idx, valid, off)
    buf = torch.full((60, 10), 0.5, device="cuda")
    out = B.moe_balance_loss_bwd(dev(logits), got.lse, got.coef, got.norm, torch.tensor([0.7, 0.3]).cuda(), dev(valid),
                                 dev(off), add=buf, dlogits=buf)
    assert out is buf and torch.allclose(buf - 0.5, d, atol=1e-7)
    L, h, r = logits.astype(np.float64), 1e-6, np.random.default_rng(2)
    for _ in range(3):
        v = r.normal(size=L.shape)
        num = ((O.balance_loss(L + h * v, idx, valid, off)["loss"] - O.balance_loss(L - h * v, idx, valid, off)["loss"])
               * [0.7, 0.3]).sum() / (2 * h)
        assert abs(num - (f64(d) * v).sum()) <= 1e-5 * np.abs(f64(d) * v).sum()


def test_refusals():
    logits, idx, _, _ = (dev(a) for a in make(10, 8, 2))
    r = B.moe_balance_loss(logits, idx)
    dl = torch.ones(2, device="cuda")
    for bad in (lambda: B.moe_balance_loss(logits.bfloat16(), idx), lambda: B.moe_balance_loss(logits, idx.long()),
                lambda: B.moe_balance_loss(logits, idx[:5]), lambda: B.moe_balance_loss(logits, idx, valid=torch.ones(9, dtype=torch.uint8).cuda()),
                lambda: B.moe_balance_loss(logits, idx, seq_offsets=torch.zeros(3).cuda()),
                lambda: B.moe_balance_loss(torch.zeros(4, 300).cuda(), idx[:4]), lambda: B.moe_balance_loss(logits.cpu(), idx),
                lambda: B.moe_balance_loss_bwd(logits, r.lse[:5], r.coef, r.norm, dl),
                lambda: B.moe_balance_loss_bwd(logits, r.lse, r.coef, r.norm, dl[:1]),
                lambda: B.moe_balance_loss_bwd(logits, r.lse, r.coef, r.norm, dl, add=logits[:3])):
        with pytest.raises(B.MoEError):
            bad()
    L = B.lib()
    p = logits.data_ptr()
    assert L.moe_balance_loss(p, p, None, None, 10, 8, 2, 1, p, p, p, p, p, p, p, 16, None, None) == 1  # workspace too small
    assert "workspace" in L.moe_last_error().decode()
    assert L.moe_balance_loss(p, p, None, None, 10, 8, 2, 2, p, p, p, p, p, p, p, 1 << 30, None, None) == 1  # two sequences, no offsets
