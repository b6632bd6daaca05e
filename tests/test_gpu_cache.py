"""The operators on a round's key/value cache against the float64 restatement
(oracle/cacheref.py).

Bookkeeping and the 4-bit format are exact.  Attention's tolerances:

* a score z = scale (s (q . n) + o sum q): at most 16 tensor-core steps, each
  cutting off below 2^-23 of its sum, and a few float32 roundings; the sums
  are at most 3 |q|_1 max|k| (|s n| <= 2 max|k|, |o| <= max|k|): with `size` =
  scale |q|_1 max|k|, dz = 16 * 2^-23 * 3 size < 2^-17 size;
* a weight exp(z - max): 2 dz (its own score's and the sum's), and its
  rounding as an operand, half a step of float16 (2^-11) where the result is
  bfloat16, 2^-20 with both parts where it is float16;
* the sums over at most 512 tensor-core steps between joins, each cutting off
  below 2^-23 of what was summed: 512 * 2^-23 = 2^-14 of `spread` = sum w |s n|
  + |sum w o| (a bound: the sums are kept near the mean);
* the result's own half step (2^-8 bfloat16, 2^-11 float16).
"""

import numpy as np
import pytest
import torch

from oracle import cacheref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_46_gb300 as pkg

    pkg.load_library()
    return pkg


def _i32(x):
    return torch.as_tensor(np.asarray(x).astype(np.int32), device=DEV)


def _np(t):
    return t.detach().cpu().numpy()


# ------------------------------------------------------------------ bookkeeping

class _State:
    """A batch's lengths, pages and free list, on the GPU and for the restatement."""

    def __init__(self, B, N, pool, page, seed, longest):
        g = np.random.default_rng(seed)
        self.page, self.N, self.pool = page, N, pool
        self.lengths = g.integers(0, longest + 1, B)
        need = np.minimum(-(-self.lengths // page), N)
        while need.sum() > pool:
            need[g.integers(0, B)] = 0
        ids = g.permutation(pool)
        self.table = np.full((B, N), -1)
        used = 0
        for b in range(B):
            self.table[b, :need[b]] = ids[used:used + need[b]]
            used += need[b]
        self.blocks, self.free_count = need, pool - used
        self.free = np.concatenate([ids[used:], np.full(used, -1)]).astype(np.int64)
        self.gpu = [_i32(x) for x in (self.lengths, self.table, self.blocks, self.free, [self.free_count])]

    def round(self, sv, gamma, kept=None, gamma_b=None, **kw):
        lengths, table, blocks, free, count = self.gpu
        got = sv.plan_round(lengths, gamma, self.page, table, blocks, free, count, kept=None if kept is None else _i32(kept),
                            gamma_b=None if gamma_b is None else _i32(gamma_b), **kw)
        slots, positions, status, self.lengths, self.table, self.blocks, self.free, self.free_count = cacheref.plan(
            self.lengths, gamma, self.page, self.table, self.blocks, self.free, self.free_count, kept, gamma_b)
        torch.cuda.synchronize()
        for name, a, b in (("status", got[2], status), ("blocks", blocks, self.blocks), ("table", table, self.table),
                           ("lengths", lengths, self.lengths), ("slots", got[0], slots), ("positions", got[1], positions)):
            assert np.array_equal(_np(a), b), name
        assert int(count) == self.free_count
        assert np.array_equal(_np(free)[:self.free_count], self.free[:self.free_count])
        return got


@pytest.mark.parametrize("B, N, pool, page, longest, gamma", [
    (1, 4, 4, 16, 40, 0), (1, 1, 1, 16, 0, 15), (5, 9, 60, 16, 100, 4), (33, 12, 300, 32, 300, 8), (64, 300, 64 * 300, 16, 1, 4095),
    (257, 8, 1500, 256, 1800, 64), (1025, 6, 6000, 64, 300, 8), (8192, 5, 40000, 16, 60, 2), (3000, 40, 100000, 16, 500, 30)])
def test_plan_rounds_in_a_row(sv, B, N, pool, page, longest, gamma):
    s = _State(B, N, pool, page, B + gamma, longest)
    g = np.random.default_rng(7)
    for turn in range(6):
        gamma_b = None if turn % 3 == 0 else g.integers(-1, gamma + 1, B)
        kept = None if turn == 0 else g.integers(-9 if turn % 2 else 0, min(gamma, 20) + 2, B)
        if turn == 4:
            kept[::3] = -10 ** 6                       # ended: every page comes back
        s.round(sv, gamma, kept, gamma_b)
        assert len(set(s.free[:s.free_count]) | set(s.table[s.table >= 0])) == pool     # no page is lost or given twice


def test_plan_without_enough_pages(sv):
    s = _State(40, 50, 120, 16, 3, 30)
    s.lengths[:] = np.minimum(s.lengths, 30)
    got = s.round(sv, 200)
    status = _np(got[2])
    assert (status == sv.SV_PLAN_NO_PAGES).any() and (status == 0).any()
    # those that fit go on when others end
    kept = np.where(status == 0, -10 ** 6, 0)
    s.round(sv, 200, kept, np.where(status == 0, -1, 30))


def test_plan_too_long_and_counts_outside(sv):
    s = _State(6, 3, 40, 16, 3, 40)
    s.lengths[2] = 2 ** 31 - 2
    s.gpu[0][2] = 2 ** 31 - 2
    got = s.round(sv, 4, kept=[0, 0, 3, 0, 0, 0], gamma_b=[99, -99, 4, 4, 4, 4])
    assert int(got[2][2]) == sv.SV_PLAN_TOO_LONG
    # a count above its array means all of it, a negative one none
    i = torch.int32
    for count, blocks, has in ((99, 99, 2), (-5, -5, 0)):
        table, free = torch.tensor([[3, 4]], dtype=i, device=DEV), torch.tensor([0, 1, 2], dtype=i, device=DEV)
        blocks, count = torch.tensor([blocks], dtype=i, device=DEV), torch.tensor([count], dtype=i, device=DEV)
        lengths = torch.tensor([16], dtype=i, device=DEV)
        slots, _, status = sv.plan_round(lengths, 0, 16, table, blocks, free, count)
        assert int(status) == (0 if has else sv.SV_PLAN_NO_PAGES) and int(count) == (3 if has else 0)
        assert int(slots) == (4 * 16 if has else -1) and int(blocks) == has


def test_plan_with_foreign_page_ids(sv):
    i = torch.int32
    table = torch.tensor([[-7, 2 ** 30]], dtype=i, device=DEV)
    blocks, count = torch.tensor([2], dtype=i, device=DEV), torch.zeros(1, dtype=i, device=DEV)
    slots, positions, status = sv.plan_round(torch.tensor([14], dtype=i, device=DEV), 3, 16, table, blocks, table.new_zeros(0), count)
    assert slots.tolist() == [[-1] * 4] and positions.tolist() == [[14, 15, 16, 17]] and int(status) == 0


def test_plan_refuses(sv):
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    t = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    for bad in (dict(lengths=i.long()), dict(blocks=i[:3]), dict(block_table=t[:, :1].expand(4, 2)), dict(free_count=i),
                dict(gamma=-1), dict(kept=i[:2]), dict(gamma_b=i.float()), dict(lengths=t)):
        a = dict(lengths=i, gamma=2, page=16, block_table=t, blocks=i, free_blocks=i, free_count=i[:1], kept=None, gamma_b=None)
        a.update(bad)
        with pytest.raises(ValueError):
            sv.plan_round(a.pop("lengths"), a.pop("gamma"), a.pop("page"), a.pop("block_table"), a.pop("blocks"), a.pop("free_blocks"),
                          a.pop("free_count"), **a)
    with pytest.raises(sv.SvError):
        sv.plan_round(i, 2, 20, t, i, i, i[:1])


# ------------------------------------------------------------------ the format

def _model_rows(shape, seed, dtype, wild=False):
    g = np.random.default_rng(seed)
    x = g.normal(size=shape) + 2.0 * g.normal(size=shape[-1])
    if wild:
        x = x * np.exp2(g.integers(-10, 11, shape[:-1] + (1,)))
    return torch.as_tensor(x).to(DTYPES[dtype]).to(DEV)


def _blocks(cache, page, D, dtype):
    """Codes and numbers of every block: keys, values [pages, heads, page, D], numbers [pages, heads, page, 4]."""
    c = _np(cache)
    numbers = cache[..., page * D:].contiguous().view(DTYPES[dtype]).double().cpu().numpy().reshape(c.shape[:2] + (page, 4))
    keys, values = np.zeros(c.shape[:2] + (page, D), np.int64), np.zeros(c.shape[:2] + (page, D), np.int64)
    for p in range(c.shape[0]):
        for h in range(c.shape[1]):
            keys[p, h], values[p, h], _ = cacheref.decode(c[p, h], page, D, None)
    return keys, values, numbers


def _same(a, b):
    return np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(a)], b[~np.isnan(b)])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B, G1, heads, D, page", [(1, 1, 1, 64, 16), (1, 1, 8, 128, 16), (3, 5, 5, 64, 32), (2, 37, 3, 128, 48), (4, 9, 2, 128, 256)])
def test_append_and_read(sv, dtype, B, G1, heads, D, page):
    pages = (B * G1 + page - 1) // page + 2
    k, v = (_model_rows((B, G1, heads, D), s, dtype, wild=True) for s in (1, 2))
    g = np.random.default_rng(5)
    slots = g.permutation(pages * page)[:B * G1].reshape(B, G1)
    if B * G1 > 3:
        slots.flat[1], slots.flat[2], slots.flat[3] = -1, pages * page, -2 ** 31       # not written
        k[0, 1], v[0, 1] = 7.0, -7.0
    cache = sv.alloc_kv4_cache(pages, heads, D, page, DEV)
    cache.fill_(0xA5)
    before = cache.clone()
    assert sv.append_kv4(k, v, _i32(slots), cache) is cache
    keys, values, numbers = _blocks(cache, page, D, dtype)
    old_keys, old_values, old_numbers = _blocks(before, page, D, dtype)
    want = [np.zeros((B, G1, heads, D))] * 2
    untouched = np.ones((pages, page), bool)
    for x, codes, old, n, which in ((k, keys, old_keys, numbers, 0), (v, values, old_values, numbers, 2)):
        c, scale, offset = cacheref.hold(x.double().cpu().numpy(), dtype)
        for b in range(B):
            for i in range(G1):
                if 0 <= slots[b, i] < pages * page:
                    p, t = divmod(slots[b, i], page)
                    untouched[p, t] = False
                    assert np.array_equal(codes[p, :, t], c[b, i])
                    assert np.array_equal(n[p, :, t, which], scale[b, i]) and np.array_equal(n[p, :, t, which + 1], offset[b, i])
    for a, b in ((keys, old_keys), (values, old_values), (numbers, old_numbers)):
        assert _same(np.moveaxis(a, 1, 2)[untouched].astype(float), np.moveaxis(b, 1, 2)[untouched].astype(float))
    got = sv.read_kv4(cache, _i32(slots), page, DTYPES[dtype])
    there = (slots >= 0) & (slots < pages * page)
    for x, y in zip((k, v), got):
        want = cacheref.to_model(cacheref.held(x.double().cpu().numpy(), dtype), dtype) * there[..., None, None]
        assert y.shape == x.shape and y.dtype is x.dtype and np.array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_odd_rows(sv, dtype, D):
    """Constant rows, rows whose scale leaves the type, NaN and infinities (each in another lane's elements)."""
    big, tiny = (3.3e38, 2e-38) if dtype == "bf16" else (65504.0, 2.0 ** -24)
    rows = torch.randn(12, D, generator=torch.Generator().manual_seed(1)).double()
    rows[0] = 1.5
    rows[1] = 0.0
    rows[2, 0], rows[2, 1:] = big, -big
    rows[3] = tiny * (torch.arange(D) % 3)
    rows[4, 3] = float("nan")
    rows[5, D - 1] = float("inf")
    rows[6, D // 2] = -float("inf")
    rows[7] = rows[7] * tiny
    rows[8, 5], rows[8, 6] = float("inf"), -float("inf")
    rows[9] = 1e-3 * rows[9] + 100
    rows[10] = (torch.arange(D) % 2) * tiny * 15
    rows = rows.to(DTYPES[dtype])
    x = rows.view(12, 1, 1, D).to(DEV)
    y = x.flip(0).contiguous()
    cache = sv.alloc_kv4_cache(1, 1, D, 16, DEV)
    slots = torch.arange(12, dtype=torch.int32, device=DEV)[:, None]
    k, v = sv.read_kv4(sv.append_kv4(x, y, slots, cache), slots, 16, DTYPES[dtype])
    for a, b in ((x, k), (y, v)):
        want = cacheref.to_model(cacheref.held(a.double().cpu().numpy(), dtype), dtype)
        assert _same(b.double().cpu().numpy(), want)
    assert torch.equal(k[0], x[0]) and torch.equal(k[1], x[1]) and k[4:7].isnan().all()


@pytest.mark.parametrize("D, heads", [(128, 3), (64, 5)])
def test_append_strided(sv, D, heads):
    """Slices of the projections' common output, a transposed layout, and one row for all."""
    B, G1, page = 3, 6, 16
    both = _model_rows((B, G1, 6 * heads, D), 4, "bf16")
    k, v = both[:, :, 4 * heads:5 * heads], both[:, :, 5 * heads:]
    slots = torch.arange(B * G1, dtype=torch.int32, device=DEV).view(B, G1)
    a = sv.append_kv4(k, v, slots, sv.alloc_kv4_cache(2, heads, D, page, DEV))
    b = sv.append_kv4(k.contiguous(), v.contiguous(), slots, sv.alloc_kv4_cache(2, heads, D, page, DEV))
    assert torch.equal(a, b)
    kt = k.contiguous().transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(sv.append_kv4(kt, v, slots, sv.alloc_kv4_cache(2, heads, D, page, DEV)), b)
    one = k[:1, :1].expand(B, G1, heads, D)
    a = sv.append_kv4(one, one, slots, sv.alloc_kv4_cache(2, heads, D, page, DEV))
    b = sv.append_kv4(one.contiguous(), one.contiguous(), slots, sv.alloc_kv4_cache(2, heads, D, page, DEV))
    assert torch.equal(a, b)


def test_append_and_read_many_rows(sv):
    """Odd row counts over many CTAs, against elementary torch operations."""
    B, G1, heads, D, page = 7, 1111, 3, 128, 64
    k, v = (_model_rows((B, G1, heads, D), s, "bf16") for s in (1, 2))
    pages = B * G1 // page + 9
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:B * G1].view(B, G1).to(torch.int32).to(DEV)
    cache = sv.append_kv4(k, v, slots, sv.alloc_kv4_cache(pages, heads, D, page, DEV))
    for x, y in zip((k, v), sv.read_kv4(cache, slots, page, torch.bfloat16)):
        f = x.float()
        lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
        scale = ((hi - lo) / 15).bfloat16().float()
        want = torch.round((f - lo) * (1 / scale)).clamp(0, 15) * scale + lo
        assert torch.equal(y, want.bfloat16())


def test_store_refuses(sv):
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device=DEV)
    c, s = sv.alloc_kv4_cache(2, 2, 64, 16, DEV), torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for k, v, slots, cache in ((x, x[:1], s, c), (x, x.half(), s, c), (x[..., ::2], x[..., ::2], s, c), (x, x, s.long(), c),
                               (x, x, s[:1], c), (x, x, s, c[:, :1].contiguous()), (x, x, s, c[:, :, :72]), (x, x, s, c.half()),
                               (x[..., :32], x[..., :32], s, c), (x[:, :0], x[:, :0], s[:, :0], c), (x[0], x[0], s, c),
                               (x, x, s, sv.alloc_kv4_cache(2, 2, 128, 16, DEV)[:, :, :17 * 72].contiguous())):
        with pytest.raises(ValueError):
            sv.append_kv4(k, v, slots, cache)
    with pytest.raises(ValueError, match="no gradient"):
        sv.append_kv4(x.clone().requires_grad_(), x, s, c)
    shifted = torch.zeros(2 * 3 * 2 * 64 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(2, 3, 2, 64)
    with pytest.raises(sv.SvError):
        sv.append_kv4(shifted, x, s, c)
    for page, dtype in ((32, torch.bfloat16), (0, torch.bfloat16), (16, torch.float32)):
        with pytest.raises(ValueError):
            sv.read_kv4(c, s, page, dtype)


# ------------------------------------------------------------------ attention

class _Cache:
    """Sequences of random keys and values in shuffled pages of a cache."""

    def __init__(self, sv, totals, heads, D, page, dtype, seed=0, spare=1, width=0, wild=False, garbage=True):
        g = np.random.default_rng(seed)
        self.page, self.dtype, self.heads, self.D = page, dtype, heads, D
        need = [-(-t // page) for t in totals]
        N = max(need + [width])
        ids = g.permutation(sum(need) + spare)
        table = np.full((len(totals), N), -1)
        self.cache = sv.alloc_kv4_cache(len(ids), heads, D, page, DEV)
        if garbage:
            self.cache.fill_(0xFF)                       # NaN numbers wherever nothing is written
        self.k, self.v = [], []
        used = 0
        for b, t in enumerate(totals):
            table[b, :need[b]] = ids[used:used + need[b]]
            used += need[b]
            rows = [_model_rows((1, t, heads, D), 10 * seed + 2 * b + i, dtype, wild=wild) for i in range(2)] if t else None
            if not t:
                self.k.append(np.zeros((0, heads, D)))
                self.v.append(np.zeros((0, heads, D)))
                continue
            p = np.arange(t)
            slots = _i32((table[b, p // page] * page + p % page)[None])
            sv.append_kv4(*rows, slots, self.cache)
            self.k.append(cacheref.held(rows[0][0].double().cpu().numpy(), dtype))
            self.v.append(cacheref.held(rows[1][0].double().cpu().numpy(), dtype))
        self.table = _i32(table)


def _q(B, G1, HQ, D, dtype, seed=9, size=1.5):
    g = np.random.default_rng(seed)
    return torch.as_tensor(size * g.normal(size=(B, G1, HQ, D))).to(DTYPES[dtype]).to(DEV)


def _check(got, lse, q, c, lengths, dtype, scale=None, gamma_b=None, **kw):
    scale = 1 / np.sqrt(c.D) if scale is None else scale
    out, want_lse, size, spread = cacheref.attend(q.double().cpu().numpy(), c.k, c.v, lengths, scale, gamma_b, **kw)
    dz = 2.0 ** -17 * size[..., None]
    half, weight = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -20)
    bound = half * np.abs(out) + (2 * dz + weight + 2.0 ** -14) * spread + 1e-30
    if dtype == "f16":
        bound += 2.0 ** -25                              # results below the smallest normal
    off = np.abs(got.double().cpu().numpy() - out)
    assert (off <= bound).all(), (off / bound).max()
    if lse is not None:
        a = lse.double().cpu().numpy()
        assert np.array_equal(np.isinf(a), np.isinf(want_lse))
        fine = np.isfinite(a)
        a, w = a[fine], want_lse[fine]
        assert (np.abs(a - w) <= dz[..., 0][fine] + 2.0 ** -19 * (1 + np.abs(w))).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gamma, heads, group, D, page, lengths", [
    (0, 1, 1, 64, 16, [0]), (0, 1, 1, 128, 16, [1, 0, 15, 16, 17]), (0, 8, 4, 128, 16, [62, 63, 64, 65, 127, 700]),
    (0, 2, 16, 128, 64, [1000, 3]), (3, 3, 5, 64, 16, [250, 0, 77, 16]), (4, 2, 4, 128, 64, [513, 60, 64]),
    (8, 2, 8, 128, 32, [200, 31, 1500]), (8, 1, 8, 64, 48, [47, 48, 300]), (3, 2, 4, 128, 256, [255, 256, 257, 1]),
    (15, 1, 1, 128, 16, [100, 1]), (64, 1, 1, 64, 16, [40, 3]), (0, 1, 64, 128, 16, [333]), (64, 2, 2, 128, 16, [129]),
    (1, 5, 8, 128, 128, [2000, 127]), (2, 2, 11, 64, 16, [90]), (16, 1, 3, 128, 16, [1, 5])])
def test_attend(sv, dtype, gamma, heads, group, D, page, lengths):
    c = _Cache(sv, [n + gamma + 1 for n in lengths], heads, D, page, dtype, seed=gamma + heads)
    q = _q(len(lengths), gamma + 1, heads * group, D, dtype)
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), page, return_lse=True)
    _check(out, lse, q, c, lengths, dtype)
    alone = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), page)
    assert torch.equal(alone, out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend_long(sv, dtype):
    """Sequences that many CTAs share, next to short ones."""
    lengths = [20000, 5, 9000]
    c = _Cache(sv, [n + 2 for n in lengths], 2, 128, 64, dtype)
    q = _q(3, 2, 8, 128, dtype)
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 64, return_lse=True)
    _check(out, lse, q, c, lengths, dtype)


def test_attend_many_short(sv):
    """More segments than CTAs, segments cut anywhere."""
    lengths = list(np.random.default_rng(1).integers(0, 150, 300))
    c = _Cache(sv, [n + 3 for n in lengths], 3, 64, 16, "bf16")
    q = _q(300, 3, 6, 64, "bf16")
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, return_lse=True)
    _check(out, lse, q, c, lengths, "bf16")


@pytest.mark.parametrize("gamma, group", [(3, 2), (8, 8)])
@pytest.mark.parametrize("given", [False, True])
def test_attend_ragged(sv, gamma, group, given):
    lengths, gamma_b = [40, 100, 0, 77, 5, 260], [gamma, -1, 0, 1, -9, 99]
    rows = np.clip(gamma_b, -1, gamma) + 1
    c = _Cache(sv, [n + r for n, r in zip(lengths, rows)], 2, 64, 16, "bf16", width=30)
    q = _q(6, gamma + 1, 2 * group, 64, "bf16")
    q[1], q[4] = float("nan"), float("nan")
    out = torch.full_like(q, 3.0) if given else None
    got, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, gamma_b=_i32(gamma_b), out=out, return_lse=True)
    assert (got is out) == given
    behind = torch.as_tensor(np.arange(gamma + 1) >= rows[:, None], device=DEV)
    assert (got[behind] == (3.0 if given else 0.0)).all() and (lse[behind] == 0).all()
    _check(torch.where(behind[..., None, None], 0.0, got), lse, q.nan_to_num(), c, lengths, "bf16", gamma_b=gamma_b)


def test_attend_hidden_pages(sv):
    """Table entries that are no page hide their tokens; a table too narrow hides those behind it."""
    lengths, page = [100, 70, 33, 20], 16
    c = _Cache(sv, [n + 2 for n in lengths], 2, 128, page, "bf16")
    table = _np(c.table).copy()
    hidden = [np.zeros(n + 2, bool) for n in lengths]
    table[0, 2], table[0, 5], table[1, 0] = -1, c.cache.shape[0], 2 ** 31 - 1
    hidden[0][32:48] = hidden[0][80:96] = hidden[1][:16] = True
    table[2, :] = -5
    hidden[2][:] = True
    q = _q(4, 2, 4, 128, "bf16")
    out, lse = sv.attend_kv4(q, c.cache, _i32(table), _i32(lengths), page, return_lse=True)
    _check(out, lse, q, c, lengths, "bf16", hidden=hidden)
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all()
    narrow = _i32(table[:, :2])
    out, lse = sv.attend_kv4(q, c.cache, narrow, _i32(lengths), page, return_lse=True)
    _check(out, lse, q, c, lengths, "bf16", hidden=hidden, limit=32)
    out, lse = sv.attend_kv4(q, c.cache, narrow[:, :0].contiguous(), _i32(lengths), page, return_lse=True)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_attend_length_below_zero(sv):
    c = _Cache(sv, [3, 3], 1, 64, 16, "f16")
    q = _q(2, 3, 1, 64, "f16")
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([-7, 0]), 16, return_lse=True)
    _check(out, lse, q, c, [0, 0], "f16")


@pytest.mark.parametrize("gamma, group", [(5, 2), (5, 8)])
def test_attend_nan_reaches_only_rows_that_see_it(sv, gamma, group):
    """A held NaN at position lengths + i makes rows i.. NaN, not those before; an unwritten slot (NaN numbers) behind the last makes none."""
    n, page = 61, 16
    for which in (0, 1):
        c = _Cache(sv, [n + gamma + 1], 1, 128, page, "bf16", seed=which)
        q = _q(1, gamma + 1, group, 128, "bf16")
        p = n + 3
        rows = [_model_rows((1, 1, 1, 128), 5 + i, "bf16") for i in range(2)]
        rows[which][..., 7] = float("nan")
        slot = _i32([[int(c.table[0, p // page]) * page + p % page]])
        sv.append_kv4(*rows, slot, c.cache)
        out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([n]), page, return_lse=True)
        assert out[:, 3:].isnan().all() and not out[:, :3].isnan().any()
        assert lse[:, 3:].isnan().all() == (which == 0) and not lse[:, :3].isnan().any()
        keep = c.k[0][:, :], c.v[0][:, :]
        short = type("C", (), dict(k=[keep[0][:n + 3]], v=[keep[1][:n + 3]], D=128))
        _check(out[:, :3], lse[:, :3], q[:, :3], short, [n], "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gamma", [0, 8])
def test_attend_wide_range(sv, dtype, gamma):
    """Rows of keys and values whose sizes differ by 2^20, scores that grow along the sequence."""
    lengths = [400, 37]
    c = _Cache(sv, [n + gamma + 1 for n in lengths], 2, 64, 16, dtype, wild=True)
    q = _q(2, gamma + 1, 16, 64, dtype, size=0.02)
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, return_lse=True)
    _check(out, lse, q, c, lengths, dtype)
    q = q * torch.as_tensor(np.exp2(np.arange(16) - 12.0), device=DEV, dtype=q.dtype)[:, None]
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16, return_lse=True, scale=0.3)
    _check(out, lse, q, c, lengths, dtype, scale=float(np.float32(0.3)))


def test_attend_one_token_takes_all(sv):
    """Weights of 1 on a token with small values beside others with large ones."""
    D, page, n = 128, 16, 300
    c = _Cache(sv, [n + 1], 1, D, page, "bf16")
    q = _q(1, 1, 4, D, "bf16", size=6.0)
    p = 3
    k = (q[:, :, :1] * 4).contiguous()
    v = _model_rows((1, 1, 1, D), 8, "bf16") * 2.0 ** -9
    sv.append_kv4(k, v, _i32([[int(c.table[0, 0]) * page + p]]), c.cache)
    c.k[0][p], c.v[0][p] = (cacheref.held(x[0, 0].double().cpu().numpy(), "bf16") for x in (k, v))
    out, lse = sv.attend_kv4(q, c.cache, c.table, _i32([n]), page, return_lse=True)
    _check(out, lse, q, c, [n], "bf16")


@pytest.mark.parametrize("size", [1e30, 1e-30])
def test_attend_large_and_small_queries(sv, size):
    c = _Cache(sv, [50, 20], 1, 64, 16, "bf16")
    q = _q(2, 1, 3, 64, "bf16", size=size)
    out = sv.attend_kv4(q, c.cache, c.table, _i32([49, 19]), 16, scale=0.25 / size)
    _check(out, None, q, c, [49, 19], "bf16", scale=float(np.float32(0.25 / size)))


def test_attend_strided_queries(sv):
    lengths = [100, 45]
    c = _Cache(sv, [n + 3 for n in lengths], 3, 64, 16, "bf16")
    both = _q(2, 3, 12, 64, "bf16")
    q = both[:, :, 3:9]
    a = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 16)
    assert torch.equal(a, sv.attend_kv4(q.contiguous(), c.cache, c.table, _i32(lengths), 16))
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(a, sv.attend_kv4(qt, c.cache, c.table, _i32(lengths), 16))
    one = q[:1, :1].expand(2, 3, 6, 64)
    assert torch.equal(sv.attend_kv4(one, c.cache, c.table, _i32(lengths), 16),
                       sv.attend_kv4(one.contiguous(), c.cache, c.table, _i32(lengths), 16))


@pytest.mark.parametrize("gamma, group", [(0, 4), (8, 8)])
def test_attend_results_do_not_depend_on_the_run_or_workspace(sv, gamma, group):
    lengths = [3000, 64, 900]
    c = _Cache(sv, [n + gamma + 1 for n in lengths], 2, 128, 64, "bf16")
    q = _q(3, gamma + 1, 2 * group, 128, "bf16")
    want = sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 64)
    w = sv.alloc_attend_workspace(gamma, 2, group, 128, DEV)
    for fill in (0, 0xFF):
        w.fill_(fill)
        for _ in range(5):
            assert torch.equal(sv.attend_kv4(q, c.cache, c.table, _i32(lengths), 64, workspace=w), want)


def test_attend_refuses(sv):
    c = _Cache(sv, [20, 30], 2, 64, 16, "bf16")
    q, n = _q(2, 1, 4, 64, "bf16"), _i32([19, 29])
    for bad in (dict(q=q.float()), dict(q=q[:, :, :3]), dict(q=q[..., ::2]), dict(q=q[:, :0]), dict(q=q[:1]), dict(q=q.cpu()), dict(page=32),
                dict(page=0), dict(lengths=n[:1]), dict(lengths=n.long()), dict(block_table=c.table[:1]), dict(block_table=c.table.t()),
                dict(gamma_b=n[:1]), dict(out=q[:1]), dict(out=q.half()), dict(cache=c.cache[0]), dict(workspace=n),
                dict(q=q.clone().requires_grad_())):
        a = dict(q=q, cache=c.cache, block_table=c.table, lengths=n, page=16)
        a.update(bad)
        with pytest.raises(ValueError):
            sv.attend_kv4(a.pop("q"), a.pop("cache"), a.pop("block_table"), a.pop("lengths"), a.pop("page"), **a)
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(sv.SvError):
            sv.attend_kv4(q, c.cache, c.table, n, 16, **bad)
    with torch.no_grad():
        sv.attend_kv4(q.clone().requires_grad_(), c.cache, c.table, n, 16)


def test_empty_calls(sv):
    c = sv.alloc_kv4_cache(0, 2, 64, 16, DEV)
    q, i = torch.zeros(0, 3, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    assert sv.attend_kv4(q, c, i.view(0, 1)[:, :1], i, 16).shape == q.shape
    sv.append_kv4(q[:, :, :2], q[:, :, :2], i.view(0, 3), c)
    assert sv.read_kv4(c, i, 16, torch.bfloat16)[0].shape == (0, 2, 64)
    slots, _, _ = sv.plan_round(i, 2, 16, i.view(0, 4), i, i, i.new_zeros(1))
    assert slots.shape == (0, 3)
    # a cache without pages: nothing to see
    out, lse = sv.attend_kv4(torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV), c, i.new_zeros(1, 3), i.new_zeros(1) + 9, 16, return_lse=True)
    assert (out == 0).all() and (lse == -np.inf).all()


# ------------------------------------------------------------------ streams, graphs, versions

def test_other_streams_and_dropped_inputs(sv):
    lengths = [500, 33]
    c = _Cache(sv, [n + 3 for n in lengths], 2, 128, 16, "bf16")
    q, n = _q(2, 3, 8, 128, "bf16"), _i32(lengths)
    want = sv.attend_kv4(q, c.cache, c.table, n, 16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(4):
        mine = q.clone()
        s.wait_stream(torch.cuda.current_stream())
        got.append(sv.attend_kv4(mine, c.cache, c.table, n, 16, stream=s))
        del mine
        torch.randn(2, 3, 8, 128, device=DEV)
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    with pytest.raises(TypeError):
        sv.attend_kv4(q, c.cache, c.table, n, 16, s)


def test_versions(sv):
    c = _Cache(sv, [20], 1, 64, 16, "bf16")
    q, out = _q(1, 1, 1, 64, "bf16"), torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device=DEV)
    before = out._version, c.cache._version
    sv.attend_kv4(q, c.cache, c.table, _i32([19]), 16, out=out)
    sv.append_kv4(q, q, _i32([[3]]), c.cache)
    assert out._version > before[0] and c.cache._version > before[1]
    s = _State(2, 3, 6, 16, 0, 20)
    before = [t._version for t in s.gpu]
    s.round(sv, 2)
    assert all(t._version > v for t, v in zip(s.gpu, before))


def test_two_captured_rounds_on_one_workspace(sv):
    """Whole rounds in two graphs that share a workspace, replayed in turn, against the eager calls."""
    B, gamma, heads, group, D, page = 3, 2, 2, 4, 128, 16

    def make(seed):
        s = _State(B, 40, 130, page, seed, 300)
        cache = sv.alloc_kv4_cache(130, heads, D, page, DEV)
        rows = [_model_rows((B, gamma + 1, heads, D), seed + i, "bf16") for i in range(2)]
        t = max(s.lengths)
        old = [_model_rows((B, t, heads, D), seed + 2 + i, "bf16") for i in range(2)]
        p = np.arange(t)
        slots = np.where(p < s.lengths[:, None], np.take_along_axis(s.table, np.minimum(p // page, 39)[None].repeat(B, 0), 1) * page + p % page, -1)
        sv.append_kv4(*old, _i32(slots), cache)
        return s, cache, rows, _q(B, gamma + 1, heads * group, D, "bf16", seed)

    def step(s, cache, rows, q, w):
        lengths, table, blocks, free, count = s
        slots, _, _ = sv.plan_round(lengths, gamma, page, table, blocks, free, count, kept=kept)
        sv.append_kv4(*rows, slots, cache)
        return sv.attend_kv4(q, cache, table, lengths, page, workspace=w)

    kept = _i32([1, 0, 3])
    w = sv.alloc_attend_workspace(gamma, heads, group, D, DEV)
    worlds = [make(10), make(20)]
    eager = []
    for s, cache, rows, q in worlds:
        state, cc = [t.clone() for t in s.gpu], cache.clone()
        eager.append([step(state, cc, rows, q, None) for _ in range(4)])
    graphs, outs = [], []
    for s, cache, rows, q in worlds:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs.append(step(s.gpu, cache, rows, q, w))
        graphs.append(graph)
    for turn in range(4):
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], eager[i][turn]), (turn, i)


# ------------------------------------------------------------------ a run of them together

def test_rounds_of_a_small_model(sv):
    """Greedy speculative decoding of a one-layer model over the cache gives
    the tokens that one token at a time without drafts gives, whatever the
    drafts are; rejected drafts leave nothing behind."""
    B, gamma, heads, group, D, page, V, steps = 3, 3, 2, 2, 64, 16, 512, 12
    g = torch.Generator(device=DEV).manual_seed(2)
    emb = torch.randn(V, heads * D, generator=g, device=DEV, dtype=torch.bfloat16)
    pos = torch.randn(400, heads * D, generator=g, device=DEV, dtype=torch.bfloat16)
    wq = torch.randn(heads * D, heads * group * D, generator=g, device=DEV, dtype=torch.bfloat16) / 6
    head = torch.randn(heads * group * D, V, generator=g, device=DEV, dtype=torch.bfloat16)
    prompts = torch.randint(0, V, (B, 20), generator=g, device=DEV, dtype=torch.int32)

    def rows(tokens, positions):
        x = emb[tokens.long()] + pos[positions.long()]
        kv = x.view(*tokens.shape, heads, D)
        return (x.double() @ wq.double()).to(torch.bfloat16).view(*tokens.shape, heads * group, D), kv

    class World:
        def __init__(self):
            N = 12
            self.lengths = torch.zeros(B, dtype=torch.int32, device=DEV)
            self.table = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
            self.blocks = torch.zeros(B, dtype=torch.int32, device=DEV)
            self.free = torch.arange(B * N, dtype=torch.int32, device=DEV)
            self.count = torch.full((1,), B * N, dtype=torch.int32, device=DEV)
            self.cache = sv.alloc_kv4_cache(B * N, heads, D, page, DEV)
            self.kept = None

        def logits(self, tokens):
            slots, positions, status = sv.plan_round(self.lengths, tokens.shape[1] - 1, page, self.table, self.blocks, self.free,
                                                     self.count, kept=self.kept)
            assert not status.any()
            q, kv = rows(tokens, positions)
            sv.append_kv4(kv, kv.flip(-1).contiguous(), slots, self.cache)
            outs = [sv.attend_kv4(q[:, i:i + 1], self.cache, self.table, self.lengths + i, page) for i in range(tokens.shape[1])] \
                if tokens.shape[1] > 65 else [sv.attend_kv4(q, self.cache, self.table, self.lengths, page)]
            out = torch.cat(outs, 1).reshape(B, tokens.shape[1], -1)
            return (out.double() @ head.double()).float()

    plain, last, want = World(), prompts, []
    for _ in range(steps * (gamma + 1)):
        last = plain.logits(last)[:, -1:].argmax(-1).to(torch.int32)
        want.append(last)
        plain.kept = torch.full((B,), prompts.shape[1] if len(want) == 1 else 1, dtype=torch.int32, device=DEV)
    want = torch.cat(want, 1)
    world = World()
    last = world.logits(prompts)[:, -1].argmax(-1).to(torch.int32)
    world.kept = torch.full((B,), prompts.shape[1], dtype=torch.int32, device=DEV)
    got = [[int(t)] for t in last]
    for turn in range(steps):
        draft = torch.randint(0, V, (B, gamma), generator=g, device=DEV, dtype=torch.int32)
        for b in range(B):                                 # some drafts are right for a while
            n = (turn + b) % (gamma + 1)
            draft[b, :n] = want[b, len(got[b]):len(got[b]) + n]
        logits = world.logits(torch.cat([last[:, None], draft], 1))
        tokens, n_accepted, _ = sv.verify_greedy(logits.contiguous(), draft)
        world.kept = sv.truncate_emitted(tokens, n_accepted)
        for b in range(B):
            got[b] += tokens[b, :int(world.kept[b])].tolist()
        last = torch.tensor([x[-1] for x in got], dtype=torch.int32, device=DEV)
    for b in range(B):
        n = min(len(got[b]), want.shape[1])
        assert n > steps and got[b][:n] == want[b, :n].tolist()
