"""plan_round where sequences give back more pages than the free list has room
for: nothing is written behind it, the pages given last are dropped."""

import numpy as np
import pytest
import torch

from test_gpu_cache import DEV, _i32, _State, sv  # noqa: F401

pytestmark = pytest.mark.gpu

_SENTINEL = -77


# rows for one CTA with the slots, one CTA and a kernel for the slots, a cluster
@pytest.mark.parametrize("B, gamma", [(1, 3), (6, 5), (300, 8), (64, 600)])
@pytest.mark.parametrize("room", [0, 1, 5])
def test_giving_stops_at_the_pool(sv, B, gamma, room):
    page, N = 16, gamma // 16 + 12
    s = _State(B, N, B * N, page, 11 + B, 150)
    used = int(s.blocks.sum())
    # a free list that has `room` entries more than pages in it
    s.free_count = min(s.free_count, 2 * B * (gamma // 16 + 2) + 3)
    s.pool = s.free_count + room
    big = _i32(np.concatenate([s.free[:s.free_count], np.full(room + 64, _SENTINEL)]))
    s.free = s.free[:s.pool].copy()
    s.gpu[3], s.gpu[4] = big[:s.pool], _i32([s.free_count])
    given = used - int((-(-np.maximum(s.lengths - 120, 0) // page)).sum())
    assert given > room
    # tokens are taken back and nobody has rows: pages only come back
    s.round(sv, gamma, kept=np.full(B, -120), gamma_b=np.full(B, -1))
    assert s.free_count == s.pool and (big[s.pool:] == _SENTINEL).all()
    # and are taken again, from the list's top
    got = s.round(sv, gamma, kept=np.zeros(B, int))
    assert not got[2].any() and (got[0] >= 0).all() and (big[s.pool:] == _SENTINEL).all()
    # as many come back as there is room for, and others are taken in the same round
    ended = np.where(np.arange(B) % 2 == 0, -10 ** 6, 20)
    s.round(sv, gamma, kept=ended, gamma_b=np.where(ended < 0, -1, gamma))
    assert (big[s.pool:] == _SENTINEL).all()
