"""Softmax scales and queries at the ends of their ranges (attend_kv4), against
the float64 restatement with the tolerances of test_gpu_cache.py."""

import numpy as np
import pytest
import torch

from oracle import cacheref
from test_gpu_cache import DEV, _Cache, _check, _i32, _q, sv  # noqa: F401
from test_gpu_cache_edges import _LongTables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("group", [4, 20, 40])
@pytest.mark.parametrize("power", [104, 108, 126])
def test_large_scales_of_small_queries(sv, power, group, far):
    """Scores of ordinary size from queries of 2^-126 to 2^-98 and scales to match, beside rows of zeros."""
    lengths = [70, 20]
    c = _Cache(sv, [n + 1 for n in lengths], 2, 128, 16, "bf16")
    q = _q(2, 1, 2 * group, 128, "bf16", size=1.0) * 2.0 ** -(power + 2)
    q = torch.where(q.abs() < 2.0 ** -126, 2.0 ** -126, q)        # (no subnormal ones)
    q[:, :, 1::4] = 0.0
    out, lse = (_LongTables(sv) if far else sv).attend_kv4(q, c.cache, c.table, _i32(lengths), 16, scale=2.0 ** power, return_lse=True)
    _check(out, lse, q, c, lengths, "bf16", scale=2.0 ** power)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [2, 40])
def test_rows_of_zeros_at_any_scale(sv, dtype, group):
    c = _Cache(sv, [50], 1, 64, 16, dtype)
    q = torch.zeros_like(_q(1, 1, group, 64, dtype))
    for scale in (2.0 ** -149, 2.0 ** -126, 1.0, 2.0 ** 100, 2.0 ** 127):
        out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([49]), 16, scale=scale, return_lse=True)
        _check(out, lse, q, c, [49], dtype, scale=scale)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("D, group", [(64, 3), (128, 13), (128, 20), (64, 40), (128, 36), (128, 64)])
def test_queries_are_exact_over_2_to_26(sv, D, group, far):
    """bfloat16 queries 2^26 below their row's largest element, which meets keys
    of 0: scores come from the small ones alone, with all of their bits."""
    n, page = 90, 16
    g = np.random.default_rng(D + group)
    q = (1 + g.integers(0, 128, (1, 1, group, D)) / 128) * 2.0 ** -26 * g.choice([-1, 1], (1, 1, group, D))
    k = g.integers(0, 16, (n + 1, 1, D)) / 8.0
    top = int(g.integers(0, D))
    q[..., top] = 1.0
    k[..., top], k[..., (top + 5) % D] = 0.0, 15 / 8.0
    c = _Cache(sv, [n + 1], 1, D, page, "bf16")
    p = np.arange(n + 1)
    slots = _i32((c.table[0].cpu().numpy()[p // page] * page + p % page)[None])
    x = torch.as_tensor(k).to(torch.bfloat16).to(DEV)[None]
    v = torch.as_tensor(c.v[0]).to(torch.bfloat16).to(DEV)[None]
    sv.append_kv4(x, v, slots, c.cache)
    back = sv.read_kv4(c.cache, slots, page, torch.bfloat16)[0]
    assert torch.equal(back, x)
    c.k[0], c.v[0] = k, cacheref.held(v[0].double().cpu().numpy(), "bf16")
    rows = torch.as_tensor(q).to(torch.bfloat16).to(DEV)
    assert np.array_equal(rows.double().cpu().numpy(), q)
    scale = 2.0 ** 22
    out, lse = (_LongTables(sv) if far else sv).attend_kv4(rows, c.cache, c.table, _i32([n]), page, scale=scale, return_lse=True)
    small = rows.clone()
    small[..., top] = 0.0                                          # (the same scores; their size is the small ones')
    _check(out, lse, small, c, [n], "bf16", scale=scale)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("group", [4, 20, 40, 64])
@pytest.mark.parametrize("keys, values", [(0, 100), (0, -100), (60, 98), (-60, -98)])
def test_large_and_small_keys_and_values(sv, keys, values, group, far):
    """Held values up to 2^100, with keys whose size the queries make up for."""
    n, page = 500, 16
    c = _Cache(sv, [n + 1], 1, 128, page, "bf16")
    p = np.arange(n + 1)
    slots = _i32((c.table[0].cpu().numpy()[p // page] * page + p % page)[None])
    x, v = (torch.as_tensor(a).to(torch.bfloat16).to(DEV)[None] for a in (c.k[0], c.v[0]))
    x, v = x * 2.0 ** keys, v / v.abs().max() * 2.0 ** values
    sv.append_kv4(x, v, slots, c.cache)
    c.k[0], c.v[0] = (cacheref.held(a[0].double().cpu().numpy(), "bf16") for a in (x, v))
    q = _q(1, 1, group, 128, "bf16", size=0.5) * 2.0 ** -keys
    out, lse = (_LongTables(sv) if far else sv).attend_kv4(q, c.cache, c.table, _i32([n]), page, return_lse=True)
    c.v[0] *= 2.0 ** -values
    _check(out.double() * 2.0 ** -values, lse, q, c, [n], "bf16")
