"""Float64 restatement of the operators on logits rows (include/specverify_rows.h)
for tests: plain numpy loops over rows, sharing no code with the CUDA path.

* ``adjust``: penalties for repeated tokens, biases and masks; the transforms
  a server applies to p and q alike before verification ("11.1 核心原理: Draft +
  Verify 与 Rejection Sampling", section 11.1.2).
* ``top``: a teacher's record - its k best log-probabilities and the log of
  the mass outside them.
* ``distill``: KL divergence of a student's row from such a record, and its
  gradient ("投机解码 Speculative Decoding", section 4.2: the draft is distilled
  toward the target).
"""

from __future__ import annotations

import numpy as np


def _lse(x):
    """ln sum exp of a float64 vector (-inf for an empty or all -inf one)."""
    m = np.max(x, initial=-np.inf)
    return m if m == -np.inf else m + np.log(np.sum(np.exp(x - m)))


def adjust(logits, *, draft=None, history=None, history_len=None, prompt_len=None, repetition=None, frequency=None,
           presence=None, bias_tokens=None, bias_values=None, mask=None, mask_index=None, gamma_b=None, out=None):
    """[B, G1, V] float64; rows behind gamma_b keep `out`'s values (zeros
    without it).  Also returns the size of what was summed for each element,
    for error bounds: |x after the repetition step| + |f c + p| + |bias|."""
    L = np.asarray(logits, np.float64)
    B, G1, V = L.shape
    res = np.zeros_like(L) if out is None else np.asarray(out, np.float64).copy()
    size = np.zeros_like(L)
    for b in range(B):
        g = G1 - 1 if gamma_b is None else int(np.clip(gamma_b[b], 0, G1 - 1))
        n1 = 0 if history is None else int(np.clip(history_len[b], 0, history.shape[1]))
        n0 = 0 if prompt_len is None else int(np.clip(prompt_len[b], 0, n1))
        prompt, made = set(), {}
        for j in range(n1):
            t = int(history[b][j])
            if 0 <= t < V:
                if j < n0:
                    prompt.add(t)
                else:
                    made[t] = made.get(t, 0) + 1
        bias = {}
        if bias_tokens is not None:
            for t, v in zip(bias_tokens[b], bias_values[b]):
                if 0 <= int(t) < V:
                    bias[int(t)] = float(v)          # the last entry of a token counts
        r = 1.0 if repetition is None else float(repetition[b])
        f = 0.0 if frequency is None else float(frequency[b])
        p = 0.0 if presence is None else float(presence[b])
        for i in range(g + 1):
            if i > 0 and draft is not None:
                t = int(draft[b][i - 1])
                if 0 <= t < V:
                    made[t] = made.get(t, 0) + 1
            x = L[b, i].copy()
            sz = np.zeros(V)
            for t in set(made) | prompt:
                x[t] = x[t] / r if x[t] > 0 else x[t] * r
                c = made.get(t, 0)
                sz[t] += abs(f * c) + abs(p) * (c > 0) + abs(x[t])
                x[t] -= f * c + (p if c > 0 else 0.0)
            for t, v in bias.items():
                sz[t] += abs(v) + abs(x[t])
                x[t] += v
            if mask is not None:
                mi = b * G1 + i if mask_index is None else int(mask_index[b][i])
                if mi >= len(mask):
                    x[:] = -np.inf
                elif mi >= 0:
                    words = np.asarray(mask[mi]).astype(np.int64) & 0xffffffff
                    v = np.arange(V)
                    x[(words[v // 32] >> (v % 32)) & 1 == 0] = -np.inf
            res[b, i], size[b, i] = x, sz
    return res, size


def top(logits, k, temperature):
    """(indices [R, k], logprobs [R, k], tail [R]) of rows [R, V]."""
    L = np.asarray(logits, np.float64)
    R, V = L.shape
    idx = np.full((R, k), -1, np.int64)
    lp = np.full((R, k), -np.inf)
    tail = np.full(R, -np.inf)
    for r in range(R):
        x = L[r]
        if np.any(np.isnan(x)) or np.any(x == np.inf) or np.all(x == -np.inf):
            lp[r], tail[r] = np.nan, np.nan
            continue
        order = np.argsort(-x, kind="stable")
        keep = order[:k]
        keep = keep[x[keep] > -np.inf]
        z = (x - np.max(x)) / temperature            # huge logits: their sum keeps its logarithm
        lse = _lse(z)
        idx[r, :len(keep)] = keep
        lp[r, :len(keep)] = z[keep] - lse
        rest = np.ones(V, bool)
        rest[keep] = False
        tail[r] = _lse(z[rest]) - lse
    return idx, lp, tail


def distill(student, indices, logprobs, tail, temperature, weight=None, want_grad=True):
    """(loss [R], gradient [R, V], scale [R, V]): scale holds, for each
    gradient element, the sum of the magnitudes its formula subtracts."""
    S = np.asarray(student, np.float64)
    R, V = S.shape
    loss, grad, scale = np.zeros(R), np.zeros((R, V)), np.zeros((R, V))
    for r in range(R):
        w = 1.0 if weight is None else float(weight[r])
        if w == 0.0:
            continue
        ids = np.asarray(indices[r], np.int64)
        ok = (ids >= 0) & (ids < V)
        ids, lp = ids[ok], np.asarray(logprobs[r], np.float64)[ok]
        t = -np.inf if tail is None else float(tail[r])
        vals = np.append(lp, t)
        if not np.any(np.isnan(vals)) and np.all(vals == -np.inf):
            continue                                   # nothing to learn from
        z = S[r] / temperature
        if np.any(np.isnan(vals)) or np.any(vals == np.inf) or np.any(np.isnan(z)) or np.any(z == np.inf) or \
                np.all(z == -np.inf):
            loss[r], grad[r], scale[r] = np.nan, np.nan, np.nan
            continue
        vals, z = vals - np.max(vals), (S[r] - np.max(S[r])) / temperature
        lnp = vals - _lse(vals)
        p = np.exp(lnp)
        lq = z - _lse(z)
        outside = np.ones(V, bool)
        outside[ids] = False
        lqt = _lse(lq[outside])
        mine = np.append(lq[ids], lqt)
        on = p > 0
        loss[r] = w * np.sum(p[on] * (lnp[on] - mine[on])) if np.all(mine[on] > -np.inf) else np.inf * w
        if not want_grad:
            continue
        q = np.exp(lq)
        g, sc = q.copy(), q.copy()
        for j, v in enumerate(ids):
            g[v] -= p[j]
            sc[v] += p[j]
        if p[-1] > 0 and lqt > -np.inf:
            share = np.where(outside, np.exp(lq - lqt + lnp[-1]), 0.0)
            g -= share
            sc += share
        elif lqt == -np.inf:
            g[outside] = 0.0
        grad[r], scale[r] = g * w / temperature, sc * abs(w) / temperature
    return loss, grad, scale
