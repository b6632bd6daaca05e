"""Rounds in which sequences get no pages, handled as the header says: such a
sequence takes no part in the round's attention (gamma_b = -1 there) and the
next call keeps nothing for it."""

import numpy as np
import pytest
import torch

from test_gpu_cache import DEV, _i32, _model_rows, _q, sv  # noqa: F401

pytestmark = pytest.mark.gpu


class _World:
    """Two sequences whose keys, values and queries at a position depend on it alone."""

    def __init__(self, sv, pool, gamma):
        self.sv, self.B, self.gamma, self.page, heads, D = sv, 2, gamma, 16, 2, 64
        self.k, self.v = (_model_rows((self.B, 200, heads, D), s, "bf16") for s in (1, 2))
        self.q = _q(self.B, 200, 2 * heads, D, "bf16")
        self.state = [_i32(x) for x in (np.zeros(self.B), np.full((self.B, 12), -1), np.zeros(self.B), np.arange(pool), [pool])]
        self.cache = sv.alloc_kv4_cache(pool, heads, D, self.page, DEV)
        self.rejected = _model_rows((self.B, 200, heads, D), 3, "bf16")

    def round(self, kept, right):
        """One round; tokens behind the first `right` rows of a sequence are drafts that will be rejected."""
        lengths, table, blocks, free, count = self.state
        slots, positions, status = self.sv.plan_round(lengths, self.gamma, self.page, table, blocks, free, count, kept=kept)
        b, p = torch.arange(self.B, device=DEV)[:, None], positions.long()
        wrong = (torch.arange(self.gamma + 1, device=DEV) >= right[:, None])[..., None, None]
        k, v = (torch.where(wrong, self.rejected[b, p], x[b, p]) for x in (self.k, self.v))
        self.sv.append_kv4(k, v, slots, self.cache)
        ready = torch.where(status == 0, self.gamma, -1).to(torch.int32)
        out = self.sv.attend_kv4(self.q[b, p], self.cache, table, lengths, self.page, gamma_b=ready)
        return status, out, torch.where(status == 0, right, 0).to(torch.int32)


@pytest.mark.parametrize("gamma", [3, 7])
def test_sequences_without_pages_wait(sv, gamma):
    """Their rows are 0 and their state is that of their kept tokens; once there
    are pages they go on with the results of a batch that never waited."""
    ample, few = _World(sv, 24, gamma), _World(sv, 5, gamma)
    right = _i32([3, 2])
    want = {}                                            # (sequence, its length) -> the rows that are kept
    kept = None
    for _ in range(40):
        _, out, kept = ample.round(kept, right)
        for b in range(2):
            want[b, int(ample.state[0][b])] = out[b, :int(right[b])]
    kept, waited, went_on, held = None, 0, 0, [0, 0]
    for turn in range(30):
        status, out, kept = few.round(kept, right)
        lengths = few.state[0].tolist()
        for b in range(2):
            assert lengths[b] == held[b]
            if status[b]:
                waited += 1
                assert not out[b].any() and not kept[b]
            else:
                went_on += waited > 0
                assert torch.equal(out[b, :int(right[b])], want[b, lengths[b]])
            held[b] += int(kept[b])
        if (status != 0).any() and (status == 0).any() or held[0] > 40:
            # the other sequence ends: all of its pages come back
            other = int((status == 0).nonzero()[0]) if (status != 0).any() else 0
            kept[other], held[other] = -10 ** 6, 0
        if (few.state[0] > 60).any():
            break
    assert waited and went_on
