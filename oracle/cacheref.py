"""Float64 restatement of the operators on a round's key/value cache
(include/specverify_cache.h) for tests: plain numpy loops, sharing no code with
the CUDA path.

* ``plan``: the bookkeeping between two rounds, one sequence and one page at a
  time.
* ``hold`` / ``encode`` / ``decode``: the 4-bit format of a row, and a cache's
  bytes.
* ``attend``: attention of a round's rows over held keys and values ("11.1
  核心原理: Draft + Verify 与 Rejection Sampling", section 11.1.1: one forward
  pass of the target gives the gamma+1 distributions).
"""

from __future__ import annotations

import numpy as np

NO_PAGES, TOO_LONG = 1, 2


def plan(lengths, gamma, page, table, blocks, free, free_count, kept=None, gamma_b=None):
    """One round's bookkeeping on copies of the state; returns (slots,
    positions, status, lengths, table, blocks, free, free_count)."""
    B, N = table.shape
    pool = len(free)
    lengths, table, blocks, free = (np.array(x, np.int64) for x in (lengths, table, blocks, free))
    count = int(np.clip(free_count, 0, pool))
    slots, positions = np.full((B, gamma + 1), -1), np.zeros((B, gamma + 1), np.int64)
    status, rows, need = np.zeros(B, np.int64), np.zeros(B, np.int64), np.zeros(B, np.int64)
    blocks = np.clip(blocks, 0, N)
    for b in range(B):
        lengths[b] = min(max(0, lengths[b] + (0 if kept is None else int(kept[b]))), 2 ** 31 - 1)
        rows[b] = gamma + 1 if gamma_b is None else int(np.clip(gamma_b[b], -1, gamma)) + 1
        need[b] = -(-(lengths[b] + rows[b]) // page)
        if need[b] > N:
            status[b] |= TOO_LONG
    for b in reversed(range(B)):
        while not status[b] and blocks[b] > need[b]:
            blocks[b] -= 1
            if count < pool:
                free[count] = table[b, blocks[b]]
                count += 1
            table[b, blocks[b]] = -1
    out = False
    for b in range(B):
        want = need[b] - blocks[b]
        if status[b] or want <= 0:
            continue
        if out or want > count:
            out = True
            status[b] |= NO_PAGES
            continue
        for _ in range(want):
            count -= 1
            table[b, blocks[b]] = free[count]
            blocks[b] += 1
    for b in range(B):
        for i in range(rows[b]):
            p = lengths[b] + i
            positions[b, i] = min(p, 2 ** 31 - 1)
            if not status[b]:
                slots[b, i] = table[b, p // page] * page + p % page
    return slots, positions, status, lengths, table, blocks, free, count


def _round_to(x, bits, lowest):
    """x rounded to `bits` significant bits, ties to even; `lowest` is the exponent of the smallest step."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.where(x == 0, 0.0, np.floor(np.log2(np.abs(np.where(x == 0, 1.0, x)))))
    step = np.exp2(np.maximum(e - (bits - 1), lowest))
    return np.round(x / step) * step


def to_model(x, dtype):
    y = _round_to(x, 8, -133) if dtype == "bf16" else _round_to(x, 11, -24)
    return np.where(np.abs(y) > (3.3895313892515355e38 if dtype == "bf16" else 65504.0), np.copysign(np.inf, y), y)


def hold(x, dtype):
    """(codes [.., D] int, scale [..], offset [..]) of rows of the model's type, given as float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        least, most = x.min(-1), x.max(-1)
        f32 = lambda y: y.astype(np.float32).astype(np.float64)  # noqa: E731
        scale = to_model(f32(f32(most - least) / 15.0), dtype)
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(scale)
        inverse = np.where(scale < 2.0 ** -126, 0.0, f32(1.0 / np.where(scale < 2.0 ** -126, 1.0, scale)))
        codes = np.minimum(np.round(f32(f32(x - least[..., None]) * inverse[..., None])), 15)
    codes = np.where(bad[..., None], 0, np.nan_to_num(codes)).astype(np.int64)
    return codes, np.where(bad, np.nan, scale), np.where(bad, np.nan, least)


def held(x, dtype):
    """The values that the cache stands for after it has been given x."""
    codes, scale, offset = hold(x, dtype)
    return codes * scale[..., None] + offset[..., None]


def decode(block, page, D, numbers):
    """(key codes [page, D], value codes [page, D]) of one head's block of bytes, and its numbers as they are given [page, 4]."""
    block = np.asarray(block, np.uint8)
    keys, values = np.zeros((page, D), np.int64), np.zeros((page, D), np.int64)
    for t in range(page):
        for d in range(D):
            keys[t, d] = block[t * (D // 2) + d // 2] >> (4 * (d % 2)) & 15
            unit, rest = divmod(d, 4)
            at = page * (D // 2) + (t // 2) * D + 4 * unit + 2 * (t % 2) + rest // 2
            values[t, d] = block[at] >> (4 * (d % 2)) & 15
    return keys, values, numbers


def attend(q, k, v, lengths, scale, gamma_b=None, limit=None, hidden=None):
    """q [B, G1, HQ, D]; k, v: lists of [tokens, heads, D] held keys and values
    of each sequence, in order.  Row i sees tokens 0 .. lengths[b] + i that are
    below `limit` and not `hidden[b]`.  Returns (out, lse, size, spread): size
    bounds what a score is summed from, spread what an output is."""
    q = np.asarray(q, np.float64)
    B, G1, HQ, D = q.shape
    out, spread = np.zeros_like(q), np.zeros_like(q)
    lse, size = np.zeros((B, G1, HQ)), np.zeros((B, G1, HQ))
    for b in range(B):
        kb, vb = np.asarray(k[b], np.float64), np.asarray(v[b], np.float64)
        group = HQ // kb.shape[1]
        for i in range(G1 if gamma_b is None else int(np.clip(gamma_b[b], -1, G1 - 1)) + 1):
            n = max(int(lengths[b]), 0) + i + 1
            if limit is not None:
                n = min(n, limit)
            sees = np.arange(n)
            if hidden is not None:
                sees = sees[~hidden[b][:n]]
            for h in range(HQ):
                kk, vv = kb[sees, h // group], vb[sees, h // group]
                z = scale * (kk @ q[b, i, h])
                if not len(z):
                    lse[b, i, h] = -np.inf
                    continue
                m = z.max()
                w = np.exp(z - m)
                lse[b, i, h] = m + np.log(w.sum())
                w /= w.sum()
                out[b, i, h] = w @ vv
                size[b, i, h] = scale * (np.abs(q[b, i, h]).sum() * np.abs(kk).max())
                spread[b, i, h] = w @ np.abs(vv - vv.min(-1, keepdims=True)) + w @ np.abs(vv.min(-1))
    return out, lse, size, spread
