"""The cache operators where calls and sizes meet: every tile of rows and its
neighbours, references that rise along a sequence, page lookups far into it,
caches beyond 4 GB, threads, padded batches.  Against the float64 restatement
with the tolerances of test_gpu_cache.py, or bit for bit against another form
of the same call."""

import threading

import numpy as np
import pytest
import torch

import test_gpu_cache
from oracle import cacheref
from test_gpu_cache import DEV, DTYPES, _Cache, _check, _i32, _model_rows, _q, _State, sv  # noqa: F401

pytestmark = pytest.mark.gpu


# rows of a sequence and head: (gamma + 1) * group, around the ends of the tiles of 8, 16, 24, 32 .. 80 rows
@pytest.mark.parametrize("dtype, D", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("gamma, group", [(6, 1), (7, 1), (8, 1), (15, 1), (16, 1), (23, 1), (24, 1), (7, 4), (32, 1), (5, 8), (48, 1), (12, 4),
                                          (63, 1), (64, 1), (9, 8), (26, 3), (39, 4), (40, 4), (64, 5)])
def test_every_tile_of_rows(sv, dtype, D, gamma, group):
    lengths = [150, 3]
    c = _Cache(sv, [n + gamma + 1 for n in lengths], 2, D, 32, dtype, seed=gamma)
    q = _q(2, gamma + 1, 2 * group, D, dtype)
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 32, return_lse=True)
    _check(out, lse, q, c, lengths, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gamma, group, D", [(0, 8, 128), (3, 4, 128), (5, 4, 64), (4, 8, 128), (6, 8, 128), (8, 8, 128), (8, 8, 64)])
def test_references_rise_along_the_sequence(sv, dtype, gamma, group, D):
    """Keys point along the queries ever more, values grow with them: a row's
    largest term, and the largest value scale, come again and again."""
    n, page = 1400, 16
    c = _Cache(sv, [n + gamma + 1], 1, D, page, dtype, seed=3)
    q = _q(1, gamma + 1, group, D, dtype, size=0.5)
    along = q[:, :1, :1].double()
    p = np.arange(n + gamma + 1)
    rise = torch.as_tensor(p / n * 40.0, device=DEV)[None, :, None, None]
    k = (torch.as_tensor(c.k[0], device=DEV)[None] * 0.1 + along * rise).to(DTYPES[dtype])
    v = (torch.as_tensor(c.v[0], device=DEV)[None] * torch.exp2(rise / 4)).to(DTYPES[dtype])
    slots = _i32((c.table[0].cpu().numpy()[p // page] * page + p % page)[None])
    sv.append_kv4(k, v, slots, c.cache)
    c.k[0], c.v[0] = (cacheref.held(x[0].double().cpu().numpy(), dtype) for x in (k, v))
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([n]), page, return_lse=True)
    _check(out, lse, q, c, [n], dtype)
    # and falling: the first terms are the largest by far
    order = slots.flip(1).contiguous()
    sv.append_kv4(k, v, order, c.cache)
    c.k[0], c.v[0] = c.k[0][::-1], c.v[0][::-1]
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([n]), page, return_lse=True)
    _check(out, lse, q, c, [n], dtype)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("gamma, group", [(0, 4), (4, 8)])
def test_hidden_pages_far_into_a_sequence(sv, page, gamma, group):
    n = 7000
    c = _Cache(sv, [n + gamma + 1], 1, 128, page, "bf16", seed=page)
    table = c.table.cpu().numpy().copy()
    g = np.random.default_rng(page)
    gone = g.random(table.shape[1]) < 0.4
    gone[0] = False
    table[0, gone] = g.choice([-1, c.cache.shape[0], 2 ** 30, -2 ** 31], int(gone.sum()))
    hidden = [np.repeat(gone, page)[:n + gamma + 1]]
    q = _q(1, gamma + 1, group, 128, "bf16")
    out, lse = sv.attend_kv4(q, c.cache, _i32(table), _i32([n]), page, return_lse=True)
    _check(out, lse, q, c, [n], "bf16", hidden=hidden)


@pytest.mark.parametrize("gamma, group", [(0, 2), (5, 8)])
def test_first_pages_hidden(sv, gamma, group):
    """The rows' references come from the first tokens that are there, however far in they are."""
    n, page = 600, 16
    c = _Cache(sv, [n + gamma + 1, n + gamma + 1], 2, 64, page, "f16")
    table = c.table.cpu().numpy().copy()
    table[0, :20] = -1
    table[1, :35] = -1
    hidden = [np.arange(n + gamma + 1) < 320, np.arange(n + gamma + 1) < 560]
    q = _q(2, gamma + 1, 2 * group, 64, "f16", size=4.0)
    out, lse = sv.attend_kv4(q, c.cache, _i32(table), _i32([n, n]), page, return_lse=True)
    _check(out, lse, q, c, [n, n], "f16", hidden=hidden)


def test_cache_beyond_4_gb(sv):
    """Pages whose bytes begin behind 2^32, in every operator."""
    heads, D, page = 8, 128, 256
    pages = (5 << 30) // (heads * page * (D + 8))
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    cache = sv.alloc_kv4_cache(pages, heads, D, page, DEV)
    far = [pages - 1, 3, pages - 2]
    n = 2 * page + 100
    p = np.arange(n + 1)
    table = _i32([far])
    k, v = (_model_rows((1, n + 1, heads, D), s, "bf16") for s in (1, 2))
    slots = _i32((np.array(far)[p // page] * page + p % page)[None])
    sv.append_kv4(k, v, slots, cache)
    small = sv.alloc_kv4_cache(3, heads, D, page, DEV)
    near = _i32(p[None])
    sv.append_kv4(k, v, near, small)
    for a, b in zip(sv.read_kv4(cache, slots, page, torch.bfloat16), sv.read_kv4(small, near, page, torch.bfloat16)):
        assert torch.equal(a, b)
    for rows, group in ((1, 4), (1, 48)):
        q = _q(1, rows, heads * group, D, "bf16")
        a = sv.attend_kv4(q, cache, table, _i32([n]), page)
        assert torch.equal(a, sv.attend_kv4(q, small, _i32([[0, 1, 2]]), _i32([n]), page))


def test_rows_beyond_2_to_31_elements(sv):
    """Queries, keys and values whose last rows' elements begin behind 2^31."""
    B, G1, heads, D, page = 2, 1, 1, 64, 16
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    big = torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device=DEV)
    view = big.as_strided((B, G1, heads, D), (1 << 31, D, D, 1))
    rows = _model_rows((B, G1, heads, D), 3, "bf16")
    view.copy_(rows)
    cache, near = (sv.alloc_kv4_cache(2, heads, D, page, DEV) for _ in range(2))
    slots = _i32([[0], [16]])
    sv.append_kv4(view, view, slots, cache)
    sv.append_kv4(rows, rows, slots, near)
    assert torch.equal(cache, near)
    args = (cache, _i32([[0], [1]]), _i32([0, 0]), page)
    assert torch.equal(sv.attend_kv4(view, *args), sv.attend_kv4(rows, *args))


def test_many_heads(sv):
    """More segments than a small batch suggests, the largest head count."""
    c = _Cache(sv, [40], 1024, 64, 16, "bf16")
    q = _q(1, 1, 1024, 64, "bf16")
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([39]), 16, return_lse=True)
    _check(out, lse, q, c, [39], "bf16")


def test_large_padded_batch(sv):
    """A batch padded with sequences that take no part and hold no pages."""
    B, gamma = 5000, 2
    lengths, gamma_b = np.zeros(B, np.int64), np.full(B, -1)
    live = np.random.default_rng(2).choice(B, 40, replace=False)
    lengths[live], gamma_b[live] = np.random.default_rng(3).integers(0, 200, 40), gamma
    totals = np.where(gamma_b >= 0, lengths + gamma_b + 1, 0)
    c = _Cache(sv, list(totals), 1, 64, 16, "bf16", width=20)
    q = _q(B, gamma + 1, 2, 64, "bf16")
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, gamma_b=_i32(gamma_b), return_lse=True)
    idle = torch.as_tensor(gamma_b < 0, device=DEV)
    assert (out[idle] == 0).all() and (lse[idle] == 0).all()
    part = type("C", (), dict(k=[c.k[b] for b in live], v=[c.v[b] for b in live], D=64))
    _check(out[live], lse[live], q[live], part, lengths[live], "bf16")


def test_out_is_not_touched_where_nothing_is_computed(sv):
    """gamma_b = -1 for all: nothing is computed, a given tensor stays as it is."""
    for group in (1, 40):
        c = _Cache(sv, [10, 10], 1, 64, 16, "bf16")
        q = _q(2, 1, group, 64, "bf16")
        out = torch.full_like(q, 5.0)
        sv.attend_kv4(q, c.cache, c.table, _i32([9, 9]), 16, gamma_b=_i32([-1, -1]), out=out)
        assert (out == 5.0).all()
        assert (sv.attend_kv4(q, c.cache, c.table, _i32([9, 9]), 16, gamma_b=_i32([-1, -1])) == 0).all()


@pytest.mark.parametrize("group", [2, 20])
def test_out_takes_the_queries_place(sv, group):
    """In place: out is q itself (its elements are read before they are written)."""
    lengths = [900, 31]
    c = _Cache(sv, [n + 2 for n in lengths], 2, 128, 16, "bf16")
    q = _q(2, 2, 2 * group, 128, "bf16")
    want = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16)
    with pytest.raises((ValueError, sv.SvError)):
        sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, out=q)
    assert torch.equal(sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16), want)


def test_threads(sv):
    """Calls of several threads at once, each on a stream of its own, the kernels' first ones among them."""
    lengths = [700, 90]
    c = _Cache(sv, [n + 9 for n in lengths], 2, 128, 16, "bf16")
    shapes = [(1, 4), (2, 8), (5, 8), (9, 8)]
    qs = [_q(2, rows, 2 * group, 128, "bf16", seed=i) for i, (rows, group) in enumerate(shapes)]
    n = _i32(lengths)
    want = [sv.attend_kv4(q, c.cache, c.table, n, 16) for q in qs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    if not torch.equal(sv.attend_kv4(qs[i], c.cache, c.table, n, 16), want[i]):
                        bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(qs)) for _ in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_plan_on_another_stream_and_in_inference_mode(sv):
    s = _State(30, 10, 200, 16, 5, 100)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    s.round(sv, 4, stream=stream)
    with torch.inference_mode():
        s.round(sv, 3, kept=np.ones(30, int))
        c = sv.alloc_kv4_cache(4, 1, 64, 16, DEV)
        x = torch.randn(1, 1, 1, 64, device=DEV, dtype=torch.bfloat16)
        sv.append_kv4(x, x, _i32([[3]]), c)
        sv.attend_kv4(x, c, _i32([[0]]), _i32([3]), 16, out=torch.empty_like(x))
        state = [t.clone() for t in s.gpu]
        sv.plan_round(state[0], 2, 16, *state[1:])
    sv.plan_round(state[0], 2, 16, *state[1:])               # tensors without a version, outside


@pytest.mark.parametrize("rows", [2048, 2049, 4096, 4097, 32768, 32769, 65536, 65537, 70001])
def test_plan_around_its_forms(sv, rows):
    """Row counts around those at which the slots become a kernel of their own and the pages are moved by a cluster."""
    for B in (1, 3):
        s = _State(B, rows // 16 + 40, B * (rows // 16 + 40), 16, rows, 300)
        s.round(sv, rows // B)
        s.round(sv, rows // B, kept=np.full(B, rows // (2 * B)), gamma_b=np.full(B, rows // (3 * B)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gamma, group", [(0, 4), (3, 4), (4, 8)])
def test_rows_do_not_touch_each_other(sv, dtype, gamma, group):
    """A row of NaN, of infinities or of other sizes changes nothing in the rows beside it."""
    lengths = [300]
    c = _Cache(sv, [n + gamma + 1 for n in lengths], 1, 128, 16, dtype)
    q = _q(1, gamma + 1, group, 128, dtype)
    want, want_lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, return_lse=True)
    _check(want, want_lse, q, c, lengths, dtype)
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"), 2.0 ** 15, 2.0 ** -14)):
        x = q.clone()
        h = i % group
        if abs(bad) < 1e9:
            x[:, :, h] = x[:, :, h].sign() * bad
        else:
            x[:, :, h, i::7] = bad
        out, lse = sv.attend_kv4(x, c.cache, c.table, _i32(lengths), 16, return_lse=True)
        rest = [j for j in range(group) if j != h]
        part = type("C", (), dict(k=c.k, v=c.v, D=128))
        _check(out[:, :, rest].contiguous(), lse[:, :, rest], q[:, :, rest].contiguous(), part, lengths, dtype)
        if bad != bad or abs(bad) == float("inf"):
            assert out[:, :, h].isnan().all()


@pytest.mark.parametrize("group", [4, 40])
def test_rows_of_very_different_sizes(sv, group):
    """Queries 2^60 apart in one tile, each with a scale of scores of its own."""
    c = _Cache(sv, [200], 1, 64, 16, "bf16")
    q = _q(1, 1, group, 64, "bf16")
    q = q * torch.as_tensor(np.exp2(np.linspace(-60, 0, group)), device=DEV, dtype=torch.bfloat16)[:, None]
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([199]), 16, return_lse=True)
    _check(out, lse, q, c, [199], "bf16")


@pytest.mark.parametrize("D, heads", [(64, 1), (128, 3), (64, 5)])
@pytest.mark.parametrize("start", [0, 1, 15, 16, 31])
def test_append_neighbouring_slots(sv, D, heads, start):
    """Rows whose slots follow one another, from even and odd ones, over the
    ends of pages and of sequences: what lies beside them stays as it is."""
    for B, G1 in ((1, 1), (1, 2), (2, 1), (1, 3), (3, 2), (2, 5), (1, 17), (5, 3)):
        k, v = (_model_rows((B, G1, heads, D), s, "bf16") for s in (1, 2))
        slots = _i32(start + np.arange(B * G1).reshape(B, G1))
        cache = sv.alloc_kv4_cache(4, heads, D, 16, DEV)
        cache.fill_(0x5A)
        before = sv.read_kv4(cache, _i32(np.arange(64)), 16, torch.bfloat16)
        sv.append_kv4(k, v, slots, cache)
        after = sv.read_kv4(cache, _i32(np.arange(64)), 16, torch.bfloat16)
        for x, a, b in zip((k, v), before, after):
            want = a.double().cpu().numpy()
            rows = x.double().cpu().numpy().reshape(B * G1, heads, D)
            want[start:start + B * G1] = cacheref.to_model(cacheref.held(rows, "bf16"), "bf16")
            assert np.array_equal(b.double().cpu().numpy(), want)


# ------------------------------------------------------------------ few segments are joined in one launch, or with the workspace

_SHORT = 16640     # positions of a table up to which calls are joined in one launch


class _LongTables:
    """The package, with tables too long for the join in one launch."""

    def __init__(self, sv):
        self.sv = sv

    def __getattr__(self, name):
        return getattr(self.sv, name)

    def attend_kv4(self, q, cache, table, lengths, page, **kw):
        more = _SHORT // page + 1 - table.shape[1]
        if more > 0:
            table = torch.cat([table, table.new_full((len(table), more), -1)], 1)
        return self.sv.attend_kv4(q, cache, table, lengths, page, **kw)


@pytest.mark.parametrize("dtype, D", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("gamma, group", [(6, 1), (7, 1), (8, 1), (15, 1), (16, 1), (23, 1), (24, 1), (7, 4), (32, 1), (5, 8), (48, 1), (12, 4),
                                          (63, 1), (64, 1), (9, 8), (26, 3), (39, 4), (40, 4), (64, 5)])
def test_every_tile_of_rows_with_long_tables(sv, dtype, D, gamma, group):
    test_every_tile_of_rows(_LongTables(sv), dtype, D, gamma, group)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gamma, group, D", [(0, 1, 64), (0, 8, 128), (6, 1, 128), (7, 2, 64), (3, 4, 128), (8, 1, 128), (2, 8, 128), (22, 1, 64),
                                             (4, 8, 128), (6, 8, 128), (8, 8, 128), (8, 8, 64), (16, 3, 128)])
def test_long_tables(sv, dtype, gamma, group, D):
    far = _LongTables(sv)
    test_gpu_cache.test_attend(far, dtype, gamma, 2, group, D, 16, [150, 0, 63, 1, 700, 129])
    test_references_rise_along_the_sequence(far, dtype, gamma, group, D)
    if group > 1 and D == 128:
        test_rows_do_not_touch_each_other(far, dtype, gamma, group)


def test_long_tables_in_other_calls(sv):
    far = _LongTables(sv)
    for page in (16, 48, 64, 256):
        test_hidden_pages_far_into_a_sequence(far, page, 0, 4)
        test_hidden_pages_far_into_a_sequence(far, page, 4, 8)
    for gamma, group in ((0, 2), (5, 8)):
        test_first_pages_hidden(far, gamma, group)
    for group in (4, 40):
        test_rows_of_very_different_sizes(far, group)
    for group in (2, 8):
        test_gpu_cache.test_attend_nan_reaches_only_rows_that_see_it(far, 5, group)
    for gamma, group in ((3, 2), (8, 8)):
        test_gpu_cache.test_attend_ragged(far, gamma, group, True)
        test_gpu_cache.test_attend_ragged(far, gamma, group, False)
    test_gpu_cache.test_attend_length_below_zero(far)
    test_gpu_cache.test_attend_one_token_takes_all(far)
    for gamma, group in ((0, 4), (8, 8)):
        test_gpu_cache.test_attend_results_do_not_depend_on_the_run_or_workspace(far, gamma, group)
    test_gpu_cache.test_two_captured_rounds_on_one_workspace(far)
    test_gpu_cache.test_attend_strided_queries(far)
    for dtype in ("bf16", "f16"):
        for gamma in (0, 8):
            test_gpu_cache.test_attend_wide_range(far, dtype, gamma)


# (segments that fill the GPU once, and one sequence more)
@pytest.mark.parametrize("B, heads, gamma, group", [(76, 1, 0, 2), (77, 1, 0, 2), (38, 2, 7, 1), (49, 1, 3, 4), (50, 1, 3, 4), (33, 1, 2, 8), (34, 1, 2, 8),
                                                    (7, 7, 1, 7), (1, 33, 23, 1), (11, 1, 8, 8), (12, 1, 8, 8), (24, 1, 3, 8), (25, 1, 3, 8), (1, 3, 64, 4)])
@pytest.mark.parametrize("page, width", [(16, 1040), (16, 1041), (256, 65), (48, 346), (48, 347)])
def test_around_the_join_in_one_launch(sv, B, heads, gamma, group, page, width):
    g = np.random.default_rng(B + page)
    lengths = list(g.integers(0, 400, B))
    lengths[0] = 1100
    c = _Cache(sv, [n + gamma + 1 for n in lengths], heads, 64, page, "bf16", seed=B, width=width)
    q = _q(B, gamma + 1, heads * group, 64, "bf16")
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), page, return_lse=True)
    _check(out, lse, q, c, lengths, "bf16")


def test_whole_table_in_one_launch(sv):
    """As many tokens as a table of 16640 positions has, and lengths beyond it."""
    n, page = _SHORT - 1, 64
    c = _Cache(sv, [n + 1], 2, 128, page, "bf16")
    q = _q(1, 1, 8, 128, "bf16")
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([n]), page, return_lse=True)
    _check(out, lse, q, c, [n], "bf16")
    beyond, lse_beyond = sv.attend_kv4(q, c.cache, c.table, _i32([2 ** 31 - 1]), page, return_lse=True)
    assert torch.equal(beyond, out) and torch.equal(lse_beyond, lse)


@pytest.mark.parametrize("gamma, group, D, dtype", [(8, 8, 128, "bf16"), (15, 5, 64, "f16"), (4, 8, 128, "f16"), (6, 5, 128, "bf16")])
def test_ragged_tiles_in_one_launch(sv, gamma, group, D, dtype):
    """Sequences with fewer row tiles than others, down to none."""
    for gamma_b in ([gamma, -1], [0, gamma], [1, 2], [-1, -1], [gamma // 2, -9]):
        rows = np.clip(gamma_b, -1, gamma) + 1
        lengths = [333, 70]
        c = _Cache(sv, [n + max(int(r), 1) for n, r in zip(lengths, rows)], 2, D, 16, dtype)
        q = _q(2, gamma + 1, 2 * group, D, dtype)
        behind = torch.as_tensor(np.arange(gamma + 1) >= rows[:, None], device=DEV)
        for out in (None, torch.full_like(q, 3.0)):
            got, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, gamma_b=_i32(gamma_b), out=out, return_lse=True)
            assert (got[behind] == (0.0 if out is None else 3.0)).all() and (lse[behind] == 0).all()
            _check(torch.where(behind[..., None, None], 0.0, got), lse, q, c, lengths, dtype, gamma_b=gamma_b)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gamma, group, D", [(0, 2, 128), (3, 4, 128), (2, 8, 64), (3, 11, 128), (8, 8, 128), (8, 8, 64), (40, 4, 128)])
def test_small_terms_behind_hidden_pages(sv, far, dtype, gamma, group, D):
    """Scores far below 0 in the first tokens that are there, 0 to 3 steps in;
    rows of which some see one token, some none.  With long tables there are so
    many segments that a CTA has several steps of one."""
    page, S, B, heads = (32, _LongTables(sv), 24, 16) if far else (32, sv, 2, 2)
    for skip in (4, 8, 13):                                # (a step is 128 tokens)
        lengths = [skip * page - 1 - gamma // 2, skip * page + 70] * (B // 2)
        c = _Cache(sv, [n + gamma + 1 for n in lengths], heads, D, page, dtype, seed=skip)
        q = _q(B, gamma + 1, heads * group, D, dtype, size=0.05) + 1.0
        for b, n in enumerate(lengths):
            t = n + gamma + 1
            k = (torch.as_tensor(c.k[b], device=DEV)[None] * 0.05 - 32.0 / D ** 0.5).to(DTYPES[dtype])
            v = torch.as_tensor(c.v[b], device=DEV)[None].to(DTYPES[dtype])
            p = np.arange(t)
            sv.append_kv4(k.contiguous(), v.contiguous(), _i32((c.table[b].cpu().numpy()[p // page] * page + p % page)[None]), c.cache)
            c.k[b], c.v[b] = (cacheref.held(x[0].double().cpu().numpy(), dtype) for x in (k, v))
        table = c.table.clone()
        table[:, :skip] = -1
        hidden = [np.arange(n + gamma + 1) < skip * page for n in lengths]
        out, lse = S.attend_kv4(q, c.cache, table, _i32(lengths), page, return_lse=True)
        _check(out, lse, q, c, lengths, dtype, hidden=hidden)


def test_caches_that_are_none(sv):
    q = _q(1, 1, 2, 64, "bf16")
    i = _i32([[0]])
    for cache in (torch.zeros(2, 0, 16 * 72, dtype=torch.uint8, device=DEV), torch.zeros((), dtype=torch.uint8, device=DEV)):
        with pytest.raises(ValueError):
            sv.append_kv4(q, q, i, cache)
        with pytest.raises(ValueError):
            sv.read_kv4(cache, i, 16, torch.bfloat16)
        with pytest.raises(ValueError):
            sv.attend_kv4(q, cache, i, _i32([0]), 16)
    # one without pages holds nothing
    none = sv.alloc_kv4_cache(0, 2, 64, 16, DEV)
    sv.append_kv4(q, q, i, none)
    k, v = sv.read_kv4(none, i, 16, torch.bfloat16)
    assert not k.any() and not v.any()
    out, lse = sv.attend_kv4(q, none, i, _i32([5]), 16, return_lse=True)
    assert not out.any() and (lse == -float("inf")).all()


class _Filled:
    """The package, with caches that hold `byte` wherever nothing was written."""

    def __init__(self, sv, byte):
        self.sv, self.byte = sv, byte

    def __getattr__(self, name):
        return getattr(self.sv, name)

    def alloc_kv4_cache(self, *args, **kw):
        return self.sv.alloc_kv4_cache(*args, **kw).fill_(self.byte)


@pytest.mark.parametrize("byte", [0x7B, 0x7F, 0xFB, 0x00])     # large numbers of either sign, NaN or the largest, nothing
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gamma, group", [(0, 4), (3, 4), (4, 8), (8, 8)])
def test_unwritten_slots_hold_anything(sv, byte, dtype, gamma, group):
    lengths = [3, 150, 511]
    c = _Cache(_Filled(sv, byte), [n + gamma + 1 for n in lengths], 2, 128, 64, dtype, garbage=False)
    q = _q(3, gamma + 1, 2 * group, 128, dtype)
    for S in (sv, _LongTables(sv)):
        out, lse = S.attend_kv4(q, c.cache, c.table, _i32(lengths), 64, return_lse=True)
        _check(out, lse, q, c, lengths, dtype)
