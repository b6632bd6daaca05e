"""Pins of the float64 restatement of the cache operators: worked examples by
hand and properties that do not come from the restatement itself."""

import numpy as np
import pytest

from oracle import cacheref


def _state(tables, N, free, pool):
    table = np.full((len(tables), N), -1)
    for b, t in enumerate(tables):
        table[b, :len(t)] = t
    return table, np.array([len(t) for t in tables]), np.array(free + [-1] * (pool - len(free))), len(free)


def test_plan_by_hand():
    # two sequences, pages of 16: 20 tokens and a round of 3 in pages 4, 7; 30 tokens in pages 2, 9
    table, blocks, free, count = _state([[4, 7], [2, 9]], 4, [5, 6, 8], 8)
    slots, positions, status, lengths, table, blocks, free, count = cacheref.plan(
        [20, 30], 2, 16, table, blocks, free, count, kept=[1, 2])
    # 21 + 3 = 24 tokens: still two pages; 32 + 3 = 35: a third one, the last of the free list
    assert lengths.tolist() == [21, 32] and table[:, :3].tolist() == [[4, 7, -1], [2, 9, 8]] and count == 2
    assert slots.tolist() == [[7 * 16 + 5, 7 * 16 + 6, 7 * 16 + 7], [8 * 16, 8 * 16 + 1, 8 * 16 + 2]]
    assert positions.tolist() == [[21, 22, 23], [32, 33, 34]] and status.tolist() == [0, 0]
    # the second sequence ends and its pages come back, the last one first; the first waits
    slots, positions, status, lengths, table, blocks, free, count = cacheref.plan(
        lengths, 2, 16, table, blocks, free, count, kept=[0, -32], gamma_b=[0, -1])
    assert blocks.tolist() == [2, 0] and free[:count].tolist() == [5, 6, 8, 9, 2]
    assert slots.tolist() == [[7 * 16 + 5, -1, -1], [-1, -1, -1]] and positions.tolist() == [[21, 0, 0], [0, 0, 0]]


def test_plan_without_enough_pages():
    table, blocks, free, count = _state([[], [], []], 4, [1, 2, 3], 3)
    slots, _, status, lengths, table, blocks, free, count = cacheref.plan([0, 0, 0], 31, 16, table, blocks, free, count)
    assert status.tolist() == [0, cacheref.NO_PAGES, cacheref.NO_PAGES] and blocks.tolist() == [2, 0, 0] and count == 1
    assert (slots[1:] == -1).all() and table[0, :2].tolist() == [3, 2]
    _, _, status, _, _, blocks, _, _ = cacheref.plan([64], 0, 16, np.full((1, 4), 7), [4], [1], 1)
    assert status.tolist() == [cacheref.TOO_LONG] and blocks.tolist() == [4]


@pytest.mark.parametrize("seed", range(4))
def test_plan_back_and_forth_leaves_the_state(seed):
    g = np.random.default_rng(seed)
    B, page, N = 7, 16, 12
    lengths, a, b = g.integers(0, 60, B), g.integers(-1, 40, B), g.integers(-1, 9, B)
    need = -(-(lengths + b + 1) // page)
    ids = g.permutation(B * N)
    table = np.full((B, N), -1)
    used = 0
    for i in range(B):
        table[i, :need[i]] = ids[used:used + need[i]]
        used += need[i]
    free = np.concatenate([ids[used:], np.full(used, -1)])
    first = cacheref.plan(lengths, 39, page, table, need, free, B * N - used, gamma_b=a)
    assert not first[2].any()
    second = cacheref.plan(first[3], 39, page, *first[4:], gamma_b=b)
    assert (second[4] == table).all() and (second[5] == need).all() and second[7] == B * N - used
    assert (second[6][:second[7]] == free[:second[7]]).all()


def test_hold_by_hand():
    x = np.zeros(64)
    x[:16] = np.arange(16) * 0.5 - 3.0            # exact: scale 0.5, offset -3, codes 0 .. 15, zeros are code 6
    codes, scale, offset = cacheref.hold(x, "bf16")
    assert scale == 0.5 and offset == -3.0 and codes[:16].tolist() == list(range(16)) and (codes[16:] == 6).all()
    assert (cacheref.held(x, "f16") == x).all()
    assert (cacheref.held(np.full(64, 1.5), "bf16") == 1.5).all()
    for bad in (np.nan, np.inf, -np.inf):
        x[5] = bad
        codes, scale, offset = cacheref.hold(x, "bf16")
        assert np.isnan(scale) and np.isnan(offset) and not codes.any()
    assert np.isnan(cacheref.hold(np.array([3e38, -3e38] * 32), "bf16")[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_held_values_are_within_half_a_step(dtype):
    g = np.random.default_rng(3)
    x = cacheref.to_model(g.normal(size=(200, 128)) * np.exp2(g.integers(-6, 7, (200, 1))), dtype)
    codes, scale, _ = cacheref.hold(x, dtype)
    assert codes.min() >= 0 and codes.max() <= 15
    # half a step, and what the scale's own rounding leaves at the far end
    half = 2.0 ** (-8 if dtype == "bf16" else -11)
    assert (np.abs(cacheref.held(x, dtype) - x) <= scale[:, None] * (0.5 + 15 * half) * (1 + 1e-6)).all()


def test_attend_by_hand():
    # one head, two tokens before the round and two rows: row 0 sees three tokens, row 1 four
    k = np.zeros((4, 1, 64))
    v = np.arange(4.0)[:, None, None] * np.ones((4, 1, 64))
    q = np.ones((1, 2, 1, 64))
    out, lse, _, _ = cacheref.attend(q, [k], [v], [2], 0.125)
    assert np.allclose(out[0, 0], 1.0) and np.allclose(out[0, 1], 1.5)
    assert np.allclose(lse[0, :, 0], [np.log(3), np.log(4)])
    k[3, 0, 0] = 80.0                             # 0.125 * 80 = 10 for the last token
    out, lse, _, _ = cacheref.attend(q, [k], [v], [2], 0.125)
    assert np.allclose(out[0, 1], (3 * np.exp(10) + 3) / (np.exp(10) + 3)) and np.allclose(out[0, 0], 1.0)
    out, lse, _, _ = cacheref.attend(q, [k], [v], [2], 0.125, hidden=[np.ones(4, bool)])
    assert not out.any() and (lse == -np.inf).all()
