"""The router on the GPU against the fp64 oracle: choice, weights, balance loss and counts, gradient."""

import numpy as np
import pytest
import torch

from around_util import U, f64, pair, rounded, within
from oracle import beside as o

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_e2m1_amd as m
    return m


def logits(rng, T, E, name, off=0.0, spread=2.0):
    z = spread * rng.standard_normal((T, E))
    z[rng.random((T, E)) < off] = -np.inf
    return pair(z, name)


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def score_error(z, E):
    """Bound of the relative error of a fp32 score or a share: the argument's rounding (its size times U), an
    exponential and a division of one step (2 U) each, a sum of E positive terms in any order of at most 16 values a lane and
    5 steps over lanes, with room of as much again."""
    span = np.where(np.isfinite(z), z, 0)
    span = span.max(1, keepdims=True) - span.min(1, keepdims=True)
    return 2 * (span + 16 + 5 + 8) * U


SIZES = [(1, 1, 1), (1, 48, 8), (3, 5, 5), (17, 64, 6), (33, 65, 8), (20, 128, 1), (9, 129, 16), (40, 257, 3), (12, 384, 8),
         (7, 385, 8), (5, 512, 64), (130, 60, 60), (300, 48, 8)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("name", ["fp32", "bf16", "fp16"])
def test_gate(mx, T, E, k, name):
    rng = np.random.default_rng(T * 1000 + E)
    for score in ("softmax", "sigmoid"):
        for bias, renorm, off in ((False, True, 0.0), (False, False, 0.3), (True, True, 0.3), (True, False, 0.0)):
            z, zr = logits(rng, T, E, name, off)
            b, br = pair(0.3 * rng.standard_normal(E), "fp32")
            ids, w = mx.moe_gate(z, k, score=score, bias=b if bias else None, renorm=renorm, scale=2.5)
            ri, rw = o.moe_gate(zr, k, score, br if bias else None, renorm, 2.5)
            what = (score, bias, renorm, off)
            assert np.array_equal(ids.cpu().numpy(), ri), what
            within(w, rw, (2 * score_error(zr, E) + 4 * U) * np.abs(rw) + 2.0 ** -126, what)


def test_gate_ties_and_values_at_the_border(mx):
    E = 300
    z = np.zeros((6, E))
    z[0, ::2] = -0.0                                   # -0 and 0 are equal
    z[1] = np.repeat([1.0, 3.0, 2.0], 100)
    z[2, 7] = np.finfo(np.float32).max
    z[3] = -3.0e38                                     # every one the same, lowest values
    z[3, 250] = -2.9e38
    z[4] = -np.inf
    z[5] = -np.inf
    z[5, [299, 13]] = [-3.0e38, 1.0]
    t, zr = pair(z, "fp32")
    for score in ("softmax", "sigmoid"):
        ids, w = (v.cpu().numpy() for v in mx.moe_gate(t, 4, score=score))
        assert ids[0].tolist() == [0, 1, 2, 3] and ids[1].tolist() == [100, 101, 102, 103]
        assert ids[2].tolist() == [7, 0, 1, 2] and ids[3].tolist() == [250, 0, 1, 2]
        assert ids[4].tolist() == [-1] * 4 and ids[5].tolist() == [13, 299, -1, -1]
        assert (w[4] == 0).all() and w[5].tolist() == [1, 0, 0, 0]
        assert np.isfinite(w).all()
        if score == "sigmoid":
            assert (w[3] == 0).all()                   # scores of 0, a sum of 0
    # one expert's bias is just the difference of two scores apart from another's: 64 bits decide
    z = np.zeros((1, 8))
    z[0, 2], z[0, 5] = 1.0, 0.5
    gap = 1 / (1 + np.exp(-1.0)) - 1 / (1 + np.exp(-0.5))
    for b, first in ((np.nextafter(np.float32(gap), np.float32(1)), 5), (np.nextafter(np.float32(gap), np.float32(0)), 2)):
        if np.float64(b) == gap:
            continue
        bias = np.zeros(8)
        bias[5] = b
        ids, _ = mx.moe_gate(pair(z, "fp32")[0], 1, score="sigmoid", bias=pair(bias, "fp32")[0])
        assert int(ids[0, 0]) == (5 if np.float64(b) > gap else 2)


def test_gate_nan(mx):
    z = np.random.default_rng(0).standard_normal((3, 50))
    z[0, 3] = np.nan
    z[1] = np.nan
    for score in ("softmax", "sigmoid"):
        for bias in (None, pair(np.zeros(50), "fp32")[0]):
            ids, w = (v.cpu().numpy() for v in mx.moe_gate(pair(z, "fp32")[0], 4, score=score, bias=bias, renorm=False))
            assert (ids >= 0).all() and (ids < 50).all() and all(len(set(r)) == 4 for r in ids.tolist())
            assert 3 not in ids[0] or (score == "softmax" and bias is not None)
            assert np.isnan(w[0]).all() == (score == "softmax") and np.isnan(w[1]).all()
            assert np.isfinite(w[2]).all()


BALANCE = [(1, 4, 1, [0, 1]), (64, 48, 8, None), (300, 60, 6, [0, 0, 7, 7, 150, 290]), (700, 257, 3, None),
           (500, 384, 8, [3, 250, 500]), (2100, 512, 2, None), (40, 130, 4, list(range(41))), (5000, 20, 3, None),
           (0, 16, 2, None), (0, 16, 2, [0, 0, 0])]


@pytest.mark.parametrize("T,E,k,off", BALANCE)
@pytest.mark.parametrize("name,score", [("fp32", "softmax"), ("bf16", "sigmoid"), ("fp16", "softmax")])
def test_balance(mx, T, E, k, off, name, score):
    rng = np.random.default_rng(T + E)
    z, zr = logits(rng, T, E, name, 0.2)
    ids = rng.integers(-2, E + 2, size=(T, k)).astype(np.int32)      # some name none
    loss, counts = mx.moe_balance(z, dev(ids, torch.int32), None if off is None else dev(np.array(off), torch.int32), score,
                                  coef=0.5)
    rl, rc = o.moe_balance(zr, ids, off, score, 0.5)
    assert np.array_equal(counts.cpu().numpy(), rc)
    # sums of positive shares over tokens (at most T deep) and of positive products over experts
    tol = ((score_error(zr, E).max() if T else 0) + (T + 16 + 16 + 8) * U) * rl
    within(loss, rl, tol + 2.0 ** -126)


GRADS = [(1, 4, 1, [0, 1]), (64, 48, 8, None), (150, 60, 6, [0, 0, 7, 7, 130]), (60, 257, 3, None), (50, 384, 8, [3, 25, 50]),
         (20, 512, 64, None), (40, 130, 4, list(range(41))), (33, 100, 20, [0, 33])]


@pytest.mark.parametrize("T,E,k,off", GRADS)
@pytest.mark.parametrize("name", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gate_grad(mx, T, E, k, off, name, score, renorm):
    rng = np.random.default_rng(T + E + k)
    z, zr = logits(rng, T, E, name, 0.1)
    zr[0], z[0] = 0.5, 0.5
    ids, _ = o.moe_gate(zr, k, score)
    if k > 2:
        ids[T // 2, 1] = ids[T // 2, 0]                # the same expert twice
        ids[T // 3, 2] = E + 3
    S = 1 if off is None else len(off) - 1
    _, counts = o.moe_balance(zr, ids, off, score)
    dw, dwr = pair(rng.standard_normal((T, k)), "fp32")
    dl, dlr = pair(rng.standard_normal(S) + 2, "fp32")
    di, dc = dev(ids, torch.int32), dev(counts, torch.int32)
    do = None if off is None else dev(np.array(off), torch.int32)
    for what in ("weights", "loss", "both"):
        a, r = {}, {}
        if what != "loss":
            a["d_w"], r["d_w"] = dw, dwr
        if what != "weights":
            a.update(counts=dc, d_loss=dl)
            r.update(counts=counts, d_loss=dlr)
        got = mx.moe_gate_grad(z, di, seq_off=do, score=score, renorm=renorm, scale=2.5, coef=4.0, **a)
        ref, size = o.moe_gate_grad(zr, ids, seq_off=off, score=score, renorm=renorm, scale=2.5, coef=4.0, **r)
        # every part off by the errors of two scores and a few products, and k adds
        tol = (3 * score_error(zr, E) + (k + 30) * U) * size
        within(got, ref, tol + rounded(ref, name) + 2.0 ** -120, what)
        assert (f64(got)[zr == -np.inf] == 0).all()


def test_grad_at_the_ends_of_the_range(mx):
    """Lowest values as masks, saturated sigmoids, rows with nothing on: finite gradients, none for what is off."""
    z = np.zeros((5, 70))
    z[0, ::3] = -3.0e38
    z[1] = -np.inf
    z[2, 5], z[2, 6] = 200.0, -200.0
    z[3] = -np.inf
    z[3, 9] = 1.0
    z[4] = -3.0e38
    t, zr = pair(z, "fp32")
    ids, w = mx.moe_gate(t, 3)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, w = mx.moe_gate(t, 3, score=score, renorm=renorm)
            loss, counts = mx.moe_balance(t, ids, score=score)
            g = mx.moe_gate_grad(t, ids, torch.ones_like(w), counts, torch.ones_like(loss), score=score, renorm=renorm)
            assert torch.isfinite(g).all() and torch.isfinite(loss).all() and (g[1] == 0).all() and (g[3, :9] == 0).all()


def test_outputs_that_are_given(mx):
    rng = np.random.default_rng(5)
    z, _ = logits(rng, 70, 48, "bf16")
    ids, w = mx.moe_gate(z, 4)
    oi, ow = torch.empty_like(ids), torch.empty_like(w)
    gi, gw = mx.moe_gate(z, 4, topk_ids=oi, topk_w=ow)
    assert gi is oi and gw is ow and torch.equal(oi, ids) and torch.equal(ow, w)
    loss, counts = mx.moe_balance(z, ids)
    ol, oc = torch.empty_like(loss), torch.full_like(counts, 99)
    mx.moe_balance(z, ids, loss=ol, counts=oc)
    assert torch.equal(ol, loss) and torch.equal(oc, counts)
    d = mx.moe_gate_grad(z, ids, w)
    od = torch.empty_like(d)
    assert mx.moe_gate_grad(z, ids, w, d_logits=od) is od and torch.equal(od, d)


def test_empty(mx):
    z = torch.empty((0, 48), device="cuda")
    ids, w = mx.moe_gate(z, 8)
    assert ids.shape == (0, 8) and w.shape == (0, 8)
    assert mx.moe_gate_grad(z, ids, w).shape == (0, 48)


def test_many_tokens_run_to_run(mx):
    """A large batch: the same bits twice, and the oracle's on a sample of tokens."""
    rng = np.random.default_rng(7)
    T, E, k = 20011, 384, 8
    z, zr = logits(rng, T, E, "fp32")
    b, br = pair(0.05 * rng.standard_normal(E), "fp32")
    off = dev(np.array([0, 9000, T]), torch.int32)
    a = mx.moe_gate(z, k, "sigmoid", b)
    s = mx.moe_balance(z, a[0], off, "sigmoid")
    d = mx.moe_gate_grad(z, a[0], a[1], s[1], s[0], off, "sigmoid")
    for _ in range(2):
        a2 = mx.moe_gate(z, k, "sigmoid", b)
        s2 = mx.moe_balance(z, a2[0], off, "sigmoid")
        d2 = mx.moe_gate_grad(z, a2[0], a2[1], s2[1], s2[0], off, "sigmoid")
        assert all(torch.equal(p, q) for p, q in zip((*a, *s, d), (*a2, *s2, d2)))
    pick = rng.choice(T, 500, replace=False)
    ri, _ = o.moe_gate(zr[pick], k, "sigmoid", br)
    assert np.array_equal(a[0].cpu().numpy()[pick], ri)
    ids = a[0].cpu().numpy()
    ref = np.stack([np.bincount(ids[p].reshape(-1), minlength=E) for p in (slice(0, 9000), slice(9000, T))])
    assert np.array_equal(s[1].cpu().numpy(), ref)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 8, 16, 17, 32, 33, 64])
def test_scores_close_to_each_other(mx, score, k):
    """Logits a few steps of fp32 apart, with a bias and without: the order of the whole row is decided by 64 bits."""
    rng = np.random.default_rng(k)
    T, E = 21, 384
    z = np.stack([1 + rng.permutation(E) * 2.0 ** -20 for _ in range(T)])
    z[3] = 0.25                                        # all the same: the lower index first
    z[4, 5:] = -np.inf                                 # fewer than k are on
    t, zr = pair(z, "fp32")
    for bias in (None, np.full(E, 0.5), np.full(E, -3.0)):
        b, br = (None, None) if bias is None else pair(bias, "fp32")
        ids, _ = mx.moe_gate(t, k, score, b)
        ri, _ = o.moe_gate(zr, k, score, br)
        # scores 2^-20 s (1 - s) apart (softmax: 2^-20 / 384) are 2^-31 or more, sums of 3 in 64 bits off by 2^-50
        assert np.array_equal(ids.cpu().numpy(), ri), bias is None


def test_infinities_and_the_largest_values_of_a_bias(mx):
    """A bias that swamps the scores: the order is the bias's, equal ones' the lower index."""
    T, E, k = 5, 100, 7
    t, zr = pair(np.random.default_rng(3).standard_normal((T, E)), "fp32")
    bias = np.zeros(E)
    bias[::3], bias[10], bias[90], bias[20:30] = 1e30, 3e38, -3e38, -np.inf
    b, br = pair(bias, "fp32")
    for score in ("softmax", "sigmoid"):
        ids, w = mx.moe_gate(t, k, score, b)
        order = sorted(range(E), key=lambda e: (-br[e], e))[:k]
        assert ids.cpu().tolist() == [order] * T and torch.isfinite(w).all()


LONG = [(9000, 40, 3, [0, 5, 5, 4000, 4001, 8999]), (9000, 100, 8, None), (4100, 257, 2, [0] + list(range(30, 4100, 100)) + [4100]),
        (6000, 33, 4, [10, 10, 90, 5990]), (4096, 60, 6, [0] + [64 * i for i in range(1, 64)] + [4096])]


@pytest.mark.parametrize("T,E,k,off", LONG)
def test_balance_of_long_and_ragged_sequences(mx, T, E, k, off):
    """Sequences that end inside a chunk of tokens, several in one, tokens of none."""
    rng = np.random.default_rng(T + E)
    z, zr = logits(rng, T, E, "fp32", 0.1)
    ids = rng.integers(-1, E + 1, size=(T, k)).astype(np.int32)
    for score in ("softmax", "sigmoid"):
        loss, counts = mx.moe_balance(z, dev(ids, torch.int32), None if off is None else dev(np.array(off), torch.int32),
                                      score, coef=2.0)
        rl, rc = o.moe_balance(zr, ids, off, score, 2.0)
        assert np.array_equal(counts.cpu().numpy(), rc)
        within(loss, rl, (score_error(zr, E).max() + (T + 40) * U) * rl + 2.0 ** -126, score)


def test_grad_of_many_sequences(mx):
    """More sequences than lanes look at once, empty ones among them."""
    T, E, k = 3000, 24, 2
    rng = np.random.default_rng(0)
    off = np.concatenate([[0, 0, 0], np.sort(rng.integers(0, T - 5, size=1500)), [T - 5]])
    z, zr = logits(rng, T, E, "fp32")
    ids, _ = mx.moe_gate(z, k)
    do = dev(off, torch.int32)
    loss, counts = mx.moe_balance(z, ids, do)
    dl, dlr = pair(1 + rng.random(len(off) - 1), "fp32")
    got = mx.moe_gate_grad(z, ids, None, counts, dl, do)
    pick = np.r_[0:40, 1500:1540, T - 30:T]
    seq = np.searchsorted(off, pick, side="right") - 1
    rc = counts.cpu().numpy()
    for i, tok in enumerate(pick):
        q = int(seq[i])
        if tok >= off[-1]:
            assert not got[tok].any()
            continue
        n = off[q + 1] - off[q]
        # the token alone, with its sequence's counts; the mean over n tokens goes into the coefficient
        ref, size = o.moe_gate_grad(zr[tok:tok + 1], ids[tok:tok + 1].cpu().numpy(), None, rc[q:q + 1], dlr[q:q + 1],
                                    [0, 1], coef=1.0 / n ** 2)
        within(got[tok:tok + 1], ref, (3 * score_error(zr[tok:tok + 1], E) + 40 * U) * size + rounded(ref, "fp32") + 2.0 ** -120)


@pytest.mark.parametrize("k", [4, 40])
def test_nan_reaches_renormalised_weights(mx, k):
    """A softmax with a NaN logit has no score, chosen or not; a sigmoid's other scores do not know of it."""
    z = np.random.default_rng(0).standard_normal((4, 50))
    z[0, 3] = np.nan
    z[2, 7:] = -np.inf
    z[2, 2] = np.nan
    t = pair(z, "fp32")[0]
    for bias in (None, pair(np.zeros(50), "fp32")[0]):
        ids, w = (v.cpu().numpy() for v in mx.moe_gate(t, k, bias=bias))
        on = ids >= 0
        assert np.isnan(w[0]).all() and np.isnan(w[2][on[2]]).all() and (w[2][~on[2]] == 0).all()
        assert on[2].sum() == min(k, 7) and np.isfinite(w[[1, 3]]).all()
        ids, w = (v.cpu().numpy() for v in mx.moe_gate(t, k, "sigmoid", bias=bias))
        assert 3 not in ids[0] and np.isfinite(w[[0, 1, 3]]).all()
        assert np.isfinite(w[2]).all() == (k == 4)
