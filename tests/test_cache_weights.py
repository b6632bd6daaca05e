"""What the attention of a round (attend_kv4) makes of a weight's rounding.

A weight times its value's scale is an operand of float16, of one part for
bfloat16 results and of two for float16 ones, and a result's own rounding hides
what that costs.  Here it cannot: tokens come in pairs with one key and
mirrored values, so that the definition's result is 0 and what is left are the
errors of weights and sums, far above the rounding of so small a result.

* Keys have codes 0 and 15 alone and offset 0, a row of queries one number of
  eight bits in all of its channels: the products are whole multiples of one
  power of two below 2^24 of it, so that the scores of a pair are equal to the
  last bit, and so are its weights.
* Values are c (2 n - 15), c a power of two, with codes n and 15 - n in a pair.
  A pair's terms w s (n - 7.5) cancel whatever w was rounded to, if the middle
  of the row is taken with the same rounding (bfloat16 results) or the rounding
  is below 2^-20 of w (float16).
* Tolerance: a sum over T tokens is T / 16 steps of the tensor cores, of 17
  addends at most, each cut off below 2^-24 of the largest: 2^-20 of what is
  summed a step, which is at most 30 c a weight (w s n); for the middles (w s
  7.5) half of that.  T / 16 additions of float32 in a lane and 16 to join sums,
  half of 2^-23 each.
"""

import numpy as np
import pytest
import torch

from test_gpu_cache_edges import _LongTables

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _pairs(T, D, levels, seed):
    """Of T tokens: channels of a key that are not 0 [T], keys and values [T, D]; tokens 2 u and 2 u + 1 are a pair."""
    g = np.random.default_rng(seed)
    level = np.repeat(np.asarray(levels(g, T // 2)), 2)
    k = np.where(np.arange(D) < level[:, None], 15.0, 0.0) / 8 / 16 * (128 // D)
    n = g.integers(0, 16, (T // 2, D))
    n[:, 0], n[:, 1] = 0, 15
    v = (2 * np.stack([n, 15 - n], 1).reshape(T, D) - 15) * np.repeat(2.0 ** -g.integers(0, 3, T // 2), 2)[:, None]
    return level, k, v


def _sizes(rows):
    """A row's number in all of its channels."""
    return 1.0 + np.arange(rows) % 64 / 64.0


def _close(rows):
    return 1.0 + (np.arange(rows) % 5 - 2) / 128.0


def _bound(T, dtype):
    return (1.5 * T / 16 * 2.0 ** -20 + (T / 32 + 8) * 2.0 ** -23 + (2.0 ** -20 if dtype == "f16" else 0.0)) * 30.0


_SEEDS = (29, 33, 37)


def _few(D):
    """Four pairs of a score near the largest, the others 30 levels below (a level is 0.12 to 0.23 of a score)."""
    def levels(g, n):
        level = 97 - g.integers(0, 60, n)
        level[g.choice(n, 4, replace=False)] = 127 - np.array([0, 2, 5, 7])
        return level * D // 128
    return levels


def _rising(D):
    """A step far below, then one with a pair that is more than 2^8 above the
    first step's largest and two that are less (in tokens of other warps)."""
    def levels(g, n):
        level = 20 - g.integers(0, 8, n)
        level[[3, 64 + 8, 64 + 22, 64 + 46]] = 30, 80, 76, 75
        return level * D // 128
    return levels


def _rounded(w, s):
    """w as a float16 operand gives it, times a power of two and s."""
    return (w * s * 32).astype(np.float16).astype(np.float64) / 32 / s


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [32, 128])
def test_one_part_would_show(T, D):
    """A restatement with one float16 part, and masses and offsets of the
    unrounded weights, is beyond the tolerances in most rows."""
    _, k, v = _pairs(T, D, _few(D), 3)
    off = []
    for x in _sizes(64):
        z = (k @ np.full(D, x)) * 1.4426950408889634
        w = np.exp2(z - z.max())
        s = (v.max(-1) - v.min(-1)) / 15
        codes = np.round((v - v.min(-1, keepdims=True)) / s[:, None])
        shift = np.where(np.arange(T) % 16 < 8, 0, 15)
        out = ((_rounded(w, s) * s) @ (codes - shift[:, None]) + (w * (v.min(-1) + shift * s)).sum()) / w.sum()
        off.append(np.abs(out).max())
    assert (np.array(off) > _bound(T, "f16")).mean() > 0.4, np.array(off) / _bound(T, "f16")


@pytest.mark.parametrize("seed", _SEEDS)
@pytest.mark.parametrize("D", [64, 128])
def test_a_middle_of_another_rounding_would_show(D, seed):
    """Middles taken with the weights' rounding relative to the references that a step found."""
    _, k, v = _pairs(256, D, _rising(D), seed)
    off = []
    for x in _close(64):
        z = (k @ np.full(D, x)) * 1.4426950408889634
        assert 7.0 < z[2 * (64 + 22)] - z[:128].max() < 8.0 < z[2 * (64 + 8)] - z[:128].max()
        w, before = np.exp2(z - z.max()), np.exp2(z - z[:128].max())
        s = (v.max(-1) - v.min(-1)) / 15
        stale = _rounded(before, s) * np.exp2(z[:128].max() - z.max())
        off.append(np.abs((15 * s * (_rounded(w, s) - stale))[::2].sum()) / w.sum())
    assert max(off) > 1.25 * _bound(256, "bf16"), np.array(off) / _bound(256, "bf16")


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_46_gb300 as pkg

    pkg.load_library()
    return pkg


def _held(sv, k, v, B, heads, page, dtype):
    """A cache that holds T tokens and one of zeros behind them, the same for every sequence and head; its table."""
    T, D = k.shape
    pages = T // page + 1
    cache = sv.alloc_kv4_cache(pages, heads, D, page, DEV)
    x, y = (torch.as_tensor(np.concatenate([a, np.zeros((1, D))])).to(DTYPES[dtype]).to(DEV)[None, :, None].expand(1, T + 1, heads, D)
            for a in (k, v))
    slots = torch.arange(T + 1, dtype=torch.int32, device=DEV)[None]
    sv.append_kv4(x, y, slots, cache)
    back = sv.read_kv4(cache, slots[:, :T], page, DTYPES[dtype])
    assert np.array_equal(back[0][0, :, 0].double().cpu().numpy(), k) and np.array_equal(back[1][0, :, 0].double().cpu().numpy(), v)
    return cache, torch.arange(pages, dtype=torch.int32, device=DEV)[None].repeat(B, 1)


def _queries(sizes, B, gamma, heads, group, D, dtype):
    rows = (gamma + 1) * group
    q = torch.as_tensor(sizes(rows)).to(DTYPES[dtype]).to(DEV).view(1, gamma + 1, 1, group, 1)
    return q.expand(B, gamma + 1, heads, group, D).reshape(B, gamma + 1, heads * group, D)


# (gamma + 1) * group rows: every tile of the forms; row 1 sees the token of zeros too
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("gamma, group", [(0, 5), (0, 13), (1, 11), (0, 31), (1, 23), (0, 62), (1, 40), (1, 64)])
def test_mirrored_values(sv, dtype, D, far, gamma, group):
    for T in (32, 128):
        _, k, v = _pairs(T, D, _few(D), 3)
        cache, table = _held(sv, k, v, 2, 2, 32, dtype)
        q = _queries(_sizes, 2, gamma, 2, group, D, dtype)
        lengths = torch.full((2,), T - 1, dtype=torch.int32, device=DEV)
        out = (_LongTables(sv) if far else sv).attend_kv4(q, cache, table, lengths, 32, scale=1.0)
        off = out.double().abs().cpu().numpy()
        assert (off <= _bound(T, dtype)).all(), off.max() / _bound(T, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gamma, group", [(0, 5), (0, 13), (1, 11), (0, 31), (1, 23), (0, 62), (1, 40)])
def test_mirrored_values_behind_a_rise(sv, dtype, D, gamma, group):
    """Terms of some tokens of a step, not of all, outgrow their rows' references
    (by more than 2^8): the step's weights are formed again, relative to others.
    With so many segments that a CTA has several steps of one."""
    T, B, heads = 256, 24, 16
    lengths = torch.full((B,), T - 1, dtype=torch.int32, device=DEV)
    q = _queries(_close, B, gamma, heads, group, D, dtype)
    for seed in _SEEDS:
        _, k, v = _pairs(T, D, _rising(D), seed)
        cache, table = _held(sv, k, v, B, heads, 32, dtype)
        out = _LongTables(sv).attend_kv4(q, cache, table, lengths, 32, scale=1.0)
        off = out.double().abs().cpu().numpy()
        assert (off <= _bound(T, dtype)).all(), off.max() / _bound(T, dtype)
