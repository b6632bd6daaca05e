"""The float64 oracle of the operators on logits rows, pinned to what is not
the oracle: definitions by brute force, closed forms, scipy's routines and
differences of the loss."""

import numpy as np
import pytest
from scipy import special

from oracle import rowsref


def test_adjust_by_hand():
    L = np.array([[[2.0, -1.0, 0.5, 3.0]] * 3])
    out, _ = rowsref.adjust(L, draft=np.array([[3, 3]]), history=np.array([[0, 1, 1, 9]]), history_len=[3], prompt_len=[1],
                            repetition=[2.0], frequency=[0.5], presence=[0.25])
    # token 0: prompt (repetition only); token 1: generated twice; token 3: drafted before rows 1 and 2
    want = [[1.0, -2.0 - 1.25, 0.5, 3.0], [1.0, -3.25, 0.5, 1.5 - 0.75], [1.0, -3.25, 0.5, 1.5 - 1.25]]
    np.testing.assert_allclose(out[0], want, rtol=0, atol=1e-15)


def test_adjust_mask_bias_and_ragged():
    L = np.zeros((1, 2, 40))
    mask = np.zeros((2, 2), np.int32)
    mask[0, 0], mask[1, 1] = 5, 128                       # tokens 0 and 2; token 39
    out, _ = rowsref.adjust(L, bias_tokens=np.array([[2, 39, 2, -1]]), bias_values=np.array([[1.0, 2.0, 3.0, 9.0]]), mask=mask)
    assert np.isneginf(out[0, 0]).sum() == 38 and out[0, 0, 0] == 0.0 and out[0, 0, 2] == 3.0
    assert np.isneginf(out[0, 1]).sum() == 39 and out[0, 1, 39] == 2.0
    out, _ = rowsref.adjust(L, mask=mask, mask_index=np.array([[-1, 7]]), gamma_b=[0], out=np.full(L.shape, 8.0))
    assert np.all(out[0, 0] == 0.0) and np.all(out[0, 1] == 8.0)
    out, _ = rowsref.adjust(L, mask=mask, mask_index=np.array([[-1, 7]]))
    assert np.all(np.isneginf(out[0, 1]))


@pytest.mark.parametrize("k", [1, 3, 20, 25])
def test_top_against_scipy(k):
    rng = np.random.default_rng(k)
    L = np.round(rng.normal(size=(6, 20)) * 2) / 2          # ties
    L[1, 5:] = -np.inf
    idx, lp, tail = rowsref.top(L, k, 0.7)
    for r in range(6):
        ref = special.log_softmax(L[r] / 0.7)
        order = sorted(range(20), key=lambda v: (-L[r, v], v))[:k]
        order = [v for v in order if L[r, v] > -np.inf]
        assert idx[r, :len(order)].tolist() == order and np.all(idx[r, len(order):] == -1)
        np.testing.assert_allclose(lp[r, :len(order)], ref[order], atol=1e-12)
        rest = [v for v in range(20) if v not in order]
        np.testing.assert_allclose(np.exp(tail[r]), np.exp(ref[rest]).sum(), atol=1e-14)


def _record(rng, R, V, k):
    idx = np.stack([rng.permutation(V)[:k] for _ in range(R)])
    return idx, rng.normal(size=(R, k)) * 2, rng.normal(size=R)


@pytest.mark.parametrize("tail", [True, False])
def test_distill_loss_is_scipys_relative_entropy(tail):
    rng = np.random.default_rng(5)
    S, (idx, lp, t) = rng.normal(size=(4, 12)) * 2, _record(rng, 4, 12, 5)
    loss, _, _ = rowsref.distill(S, idx, lp, t if tail else None, 1.5)
    for r in range(4):
        q = special.softmax(S[r] / 1.5)
        p = special.softmax(np.append(lp[r], t[r]) if tail else lp[r])
        qq = q[idx[r]]
        if tail:
            qq = np.append(qq, np.delete(q, idx[r]).sum())
        np.testing.assert_allclose(loss[r], special.rel_entr(p, qq).sum(), rtol=1e-12)


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("case", ["plain", "ignored", "twice", "weights"])
def test_distill_gradient_is_the_difference_quotient(tail, case):
    rng = np.random.default_rng(9)
    R, V, k, T = 3, 9, 4, 0.8
    S, (idx, lp, t) = rng.normal(size=(R, V)), _record(rng, R, V, k)
    w = None
    if case == "ignored":
        idx[0, 1], idx[1] = -1, V
    if case == "twice":
        idx[0, 2] = idx[0, 0]
    if case == "weights":
        w = np.array([2.0, 0.0, -0.5])
    t = t if tail else None
    _, grad, _ = rowsref.distill(S, idx, lp, t, T, w)
    h = 1e-6
    for v in range(V):
        up, down = S.copy(), S.copy()
        up[:, v] += h
        down[:, v] -= h
        diff = (rowsref.distill(up, idx, lp, t, T, w)[0] - rowsref.distill(down, idx, lp, t, T, w)[0]) / (2 * h)
        # central differences: h^2 f''' / 6 + eps f / h, both below 1e-9 here
        np.testing.assert_allclose(grad[:, v], diff, atol=1e-8)


def test_distill_planted_mistakes_are_caught():
    """A gradient that forgets the tail's share, and a loss over unnormalised
    probabilities, differ by far more than any tolerance used on the GPU."""
    rng = np.random.default_rng(3)
    S, (idx, lp, t) = rng.normal(size=(2, 50)), _record(rng, 2, 50, 6)
    loss, grad, _ = rowsref.distill(S, idx, lp, t, 1.0)
    p = special.softmax(np.append(lp[0], t[0]))
    wrong = special.softmax(S[0])
    wrong[idx[0]] -= p[:6]
    assert np.abs(wrong - grad[0]).max() > 1e-3
    raw = np.sum(np.exp(lp[0]) * (lp[0] - special.log_softmax(S[0])[idx[0]]))
    assert abs(raw - loss[0]) > 1e-2


def test_distill_empty_and_bad_rows():
    S = np.zeros((5, 4))
    S[1, 2], S[2] = np.nan, -np.inf
    idx = np.array([[-1, 7], [0, 1], [0, 1], [0, 1], [0, 1]])
    lp = np.zeros((5, 2))
    lp[3, 0] = np.nan
    loss, grad, _ = rowsref.distill(S, idx, lp, None, 1.0)
    assert loss[0] == 0 and not grad[0].any()
    for r in (1, 2, 3):
        assert np.isnan(loss[r]) and np.isnan(grad[r]).all()
    assert abs(loss[4] - np.log(2)) < 1e-12
