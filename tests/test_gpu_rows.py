"""The operators on logits rows on the GPU against the float64 oracle
(oracle/rowsref.py).

Tolerances count roundings (u = 2^-24, the half step of float32; h = half a
step of the rows' type):

* adjust: the result is rounded once to the rows' type (h |x|), after at most
  four float32 roundings of what the formula sums (4 u of the sum of their
  magnitudes, which the oracle returns).
* a sum of exponentials over a row: each term is off by at most 4 u (the
  exponential instruction's 2^-22) and by u D from its argument, D the largest
  distance of a logit from the row's maximum in units of the temperature; a
  thread adds at most 32 terms in one chain (32 u).  So a logarithm of such a
  sum is off by at most (40 + D) u, called s below.
* top: a log-probability is off by s and half its own step, as is the tail
  (numerator and denominator: 2 s).
* distill: the loss by 2 s (the tail's and the row's sums) and half its step;
  a gradient element by (3 s + 16 u) of the magnitudes its formula subtracts
  (returned by the oracle) and h of itself.
"""

import math

import numpy as np
import pytest
import torch

from oracle import rowsref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from speculative_decoding_verification_46_gb300 import build

    build.build_library()
    import speculative_decoding_verification_46_gb300 as pkg

    pkg.load_library()
    return pkg


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def _half(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def _tiny(dtype):
    """Half the smallest step of the type (float16's subnormals; float32's are flushed)."""
    return {"f16": 2.0 ** -25, "bf16": 2.0 ** -126, "f32": 2.0 ** -126}[dtype]


def _assert_close(got, want, tol, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and not np.isinf(got[~inf]).any(), what
    ok = np.isfinite(want)
    excess = np.abs(got[ok] - want[ok]) - np.broadcast_to(tol, want.shape)[ok]
    assert excess.size == 0 or excess.max() <= 0, f"{what}: {excess.max():.3e} over the tolerance"


# ------------------------------------------------------------------ adjust

def _adjust_inputs(seed, B, G, V, dtype, H=40, NB=5, M=3, ragged=False):
    g = torch.Generator().manual_seed(seed)
    L = (torch.randn(B, G + 1, V, generator=g) * 4).to(DTYPES[dtype])
    few = max(1, V // 8)                                     # tokens repeat
    a = dict(
        draft=torch.randint(-1, few + 1, (B, G), generator=g, dtype=torch.int32),
        history=torch.randint(-2, few + 2, (B, H), generator=g, dtype=torch.int32),
        history_len=torch.randint(-1, H + 2, (B,), generator=g, dtype=torch.int32),
        prompt_len=torch.randint(-1, H + 2, (B,), generator=g, dtype=torch.int32),
        repetition=1 + torch.rand(B, generator=g), frequency=torch.randn(B, generator=g), presence=torch.randn(B, generator=g),
        bias_tokens=torch.randint(-1, V + 1, (B, NB), generator=g, dtype=torch.int32),
        bias_values=torch.randn(B, NB, generator=g) * 3)
    a["history"][:, ::5] = V - 1
    if NB > 2:
        a["bias_tokens"][:, 0] = a["history"][:, 0]
        a["bias_tokens"][:, 2] = a["bias_tokens"][:, 1]      # listed twice: the later value counts
    if M:
        W = (V + 31) // 32
        a["mask"] = torch.randint(-2 ** 31, 2 ** 31, (M, W), generator=g).to(torch.int32)
        a["mask"][0] = -1
        if M > 1:
            a["mask"][1] = 0                                 # nothing allowed
        a["mask_index"] = torch.randint(-1, M + 1, (B, G + 1), generator=g, dtype=torch.int32)
    if ragged:
        a["gamma_b"] = torch.randint(-1, G + 2, (B,), generator=g, dtype=torch.int32)
    return L, a


def _check_adjust(sv, L, a, dtype, inplace=False, out_fill=None):
    B, G1, V = L.shape
    dev = {k: v.to(DEV) for k, v in a.items()}
    x = L.to(DEV)
    fill = None
    if inplace:
        out = sv.adjust_logits(x, out=x, **dev)
        assert out is x
        fill = _np(L)
    elif out_fill is not None:
        out = torch.full_like(x, out_fill)
        assert sv.adjust_logits(x, out=out, **dev) is out
        fill = np.full(L.shape, out_fill)
    else:
        out = sv.adjust_logits(x, **dev)
    torch.cuda.synchronize()
    if not inplace:
        assert torch.equal(x.cpu().view(torch.uint8), L.view(torch.uint8)), "the input was written"
    want, size = rowsref.adjust(_np(L), out=fill, **{k: _np(v) for k, v in a.items()})
    got = _np(out)
    # untouched elements are copies
    same = (size == 0) & ~np.isneginf(want)
    assert np.array_equal(got[same], want[same], equal_nan=True)
    _assert_close(got, want, 4 * U * size + _half(dtype) * np.abs(np.where(np.isfinite(want), want, 0)) + _tiny(dtype), "adjust")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 33, 64, 255, 1000, 4097])
@pytest.mark.parametrize("G", [0, 3])
def test_adjust_sizes(sv, dtype, V, G):
    L, a = _adjust_inputs(V * 10 + G, 3, G, V, dtype)
    _check_adjust(sv, L, a, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [9, 1003, 8193, 20000])
@pytest.mark.parametrize("mode", ["new", "inplace", "given"])
def test_adjust_ragged_and_in_place(sv, dtype, V, mode):
    L, a = _adjust_inputs(V + 1, 5, 4, V, dtype, H=700, NB=40, ragged=True)
    _check_adjust(sv, L, a, dtype, inplace=mode == "inplace", out_fill=7.0 if mode == "given" else None)


def test_adjust_mask_table_without_rows(sv):
    """A negative index allows everything, one beyond the table nothing, also
    where the table has no rows."""
    L = torch.randn(2, 2, 70, device=DEV)
    mi = torch.tensor([[-1, 0], [3, -1]], dtype=torch.int32, device=DEV)
    got = sv.adjust_logits(L, mask=torch.zeros(0, 3, dtype=torch.int32, device=DEV), mask_index=mi)
    assert torch.equal(got, torch.where((mi < 0)[..., None], L, torch.full_like(L, -math.inf)))
    with pytest.raises(ValueError):
        sv.adjust_logits(L, mask=torch.zeros((), dtype=torch.int32, device=DEV), mask_index=mi)


@pytest.mark.parametrize("only", ["mask", "bias", "repetition", "frequency", "presence", "draft", "prompt", "none", "dense_mask"])
@pytest.mark.parametrize("inplace", [False, True])
def test_adjust_parts_alone(sv, only, inplace):
    B, G, V = 2, 2, 2051
    L, a = _adjust_inputs(11, B, G, V, "bf16", H=300)
    counts = ("draft", "history", "history_len", "prompt_len")
    keep = {"mask": ("mask", "mask_index"), "bias": ("bias_tokens", "bias_values"), "repetition": counts + ("repetition",),
            "frequency": counts + ("frequency",), "presence": counts + ("presence",), "draft": ("draft", "repetition", "presence"),
            "prompt": ("history", "history_len", "repetition"), "none": ("draft", "history", "history_len"),
            "dense_mask": ()}[only]
    a = {k: a[k] for k in keep}
    if only == "dense_mask":
        a["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B * (G + 1), (V + 31) // 32),
                                  generator=torch.Generator().manual_seed(1)).to(torch.int32)
    if only == "none":                                       # counting without a penalty changes nothing
        x = L.to(DEV)
        got = sv.adjust_logits(x, out=x if inplace else None, **{k: v.to(DEV) for k, v in a.items()})
        assert torch.equal(got.cpu(), L)
        return
    _check_adjust(sv, L, a, "bf16", inplace=inplace)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_adjust_special_values(sv, dtype):
    """Infinities and NaN in rows, masked and not, and the type's lowest value."""
    V = 100
    L = torch.zeros(1, 2, V)
    L[0, :, 0], L[0, :, 1], L[0, :, 2], L[0, :, 3] = math.inf, -math.inf, math.nan, -0.0
    L = L.to(DTYPES[dtype])
    L[0, :, 4] = torch.finfo(DTYPES[dtype]).min
    L[0, :, 50:] = L[0, :, :50]
    words = np.zeros((1, 4), np.uint32)
    words[0, 0], words[0, 1] = 0xffffffff, 0x3ffff          # tokens 0 .. 49
    a = dict(history=torch.arange(V, dtype=torch.int32)[None], history_len=torch.tensor([V], dtype=torch.int32),
             repetition=torch.tensor([1.5]), mask=torch.from_numpy(words.view(np.int32)),
             mask_index=torch.zeros(1, 2, dtype=torch.int32))
    got = _np(sv.adjust_logits(L.to(DEV), **{k: v.to(DEV) for k, v in a.items()}))
    assert np.isneginf(got[:, :, 50:]).all()
    assert (got[:, :, 0] == np.inf).all() and np.isneginf(got[:, :, 1]).all() and np.isnan(got[:, :, 2]).all()
    assert (got[:, :, 3] == 0).all()
    # lowest * 1.5 is below every finite value of the type
    assert np.isneginf(got[:, :, 4]).all() and (got[:, :, 5:50] == 0).all()


def test_adjust_long_history_and_many_drafts(sv):
    V, G = 300, 64
    L, a = _adjust_inputs(2, 2, G, V, "f32", H=70001, NB=1024)
    a["draft"][:] = 5
    _check_adjust(sv, L, a, "f32")


@pytest.mark.parametrize("H", [128, 1000, 6148, 9001])
def test_adjust_prompt_ends_anywhere(sv, H):
    """Prompts and histories that end inside, at and beside the runs of tokens
    that a warp counts at once."""
    V, ends = 500, [0, 1, 127, 128, 129, 255, 256, 257, 640, 6143, 6144, 6145, 9000]
    pairs = [(a, b) for a in ends for b in ends if a <= b <= H]
    L, a = _adjust_inputs(H, len(pairs), 1, V, "f32", H=H, M=0)
    a["prompt_len"] = torch.tensor([p[0] for p in pairs], dtype=torch.int32)
    a["history_len"] = torch.tensor([p[1] for p in pairs], dtype=torch.int32)
    _check_adjust(sv, L, a, "f32")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [40, 1000, 1003, 13000, 13001])
@pytest.mark.parametrize("G", [0, 8, 33])
@pytest.mark.parametrize("mode", ["new", "inplace"])
def test_adjust_masks_alone(sv, dtype, V, G, mode):
    L, a = _adjust_inputs(V + G, 2, G, V, dtype, M=7, ragged=True)
    a = {k: a[k] for k in ("mask", "mask_index", "gamma_b")}
    a["mask"][2] &= a["mask"][3] & a["mask"][4] & a["mask"][5]      # few allowed
    L[0, 0, :: 3] = float("nan")
    L[1, 0, 1 :: 5] = float("inf")
    _check_adjust(sv, L, a, dtype, inplace=mode == "inplace", out_fill=3.0 if mode == "new" else None)


def test_adjust_large_vocabulary_offsets(sv):
    """More than 2^31 elements: the last row's tokens are reached."""
    V, B = (1 << 24), 130
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    x = torch.zeros(B, 1, V, dtype=torch.bfloat16, device=DEV)
    hist = torch.tensor([[V - 1, 3]] * B, dtype=torch.int32, device=DEV)
    n = torch.full((B,), 2, dtype=torch.int32, device=DEV)
    pres = torch.full((B,), 2.0, device=DEV)
    sv.adjust_logits(x, history=hist, history_len=n, presence=pres, out=x)
    assert (x[:, 0, V - 1] == -2).all() and (x[:, 0, 3] == -2).all() and int((x[B - 1] != 0).sum()) == 2


# ------------------------------------------------------------------ top logits

def _spread(z):
    """The largest distance from the row's maximum in units of the temperature."""
    fin = np.isfinite(z)
    d = np.where(fin, z, -np.inf).max(-1) - np.where(fin, z, np.inf).min(-1)
    return np.where(np.isfinite(d), d, 0.0)


def _check_top(sv, L, k, T, dtype, **kw):
    idx, lp, tail = (_np(t) for t in sv.top_logits(L.to(DEV), k, T, **kw))
    V = L.shape[-1]
    rows = _np(L).reshape(-1, V)
    want_i, want_lp, want_t = rowsref.top(rows, k, T)
    assert np.array_equal(idx.reshape(-1, k), want_i)
    s = (40 + _spread(rows / T)) * U
    _assert_close(lp.reshape(-1, k), want_lp, s[:, None] + U * np.abs(np.where(np.isfinite(want_lp), want_lp, 0)), "logprobs")
    _assert_close(tail.reshape(-1), want_t, 2 * s + U * np.abs(np.where(np.isfinite(want_t), want_t, 0)), "tail")


@pytest.fixture(params=["toprow", "topslice"])
def top_path(request, monkeypatch):
    """Both kernels at every size: one CTA per row, and slices of rows."""
    monkeypatch.setenv("SPECVERIFY_PATH", request.param)
    return request.param


def _top_rows(seed, R, V, dtype, ties=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, V, generator=g) * 2.5
    if ties:
        x = torch.round(x * 2) / 2
    return x.to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 100, 255, 1024, 5003, 40000])
@pytest.mark.parametrize("k", [1, 8, 63])
def test_top_sizes(sv, top_path, dtype, V, k):
    _check_top(sv, _top_rows(V + k, 3, V, dtype), k, 0.8, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("k", [128, 129, 256, 300, 513, 1000, 1024])
@pytest.mark.parametrize("V", [1500, 33000])
def test_top_wide_records(sv, top_path, dtype, k, V):
    _check_top(sv, _top_rows(k, 2, V, dtype), k, 1.0, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("kind", ["ties", "constant", "two_values", "negative_ties", "zeros"])
@pytest.mark.parametrize("V", [60, 5000, 70000])
@pytest.mark.parametrize("k", [5, 200])
def test_top_ties(sv, top_path, dtype, kind, V, k):
    """Ties at the k-th value, up to rows with more ties than a slice's buffer."""
    x = _top_rows(V, 2, V, dtype, ties=True)
    if kind == "constant":
        x.fill_(-3.0)
    if kind == "two_values":
        x = torch.where(x > 0, 1.0, -1.0).to(x.dtype)
    if kind == "negative_ties":
        x = -x.abs() - 1
    if kind == "zeros":
        x = torch.where(x > 0, 0.0, -0.0).to(x.dtype)        # one value, whatever its sign
    _check_top(sv, x, k, 1.0, dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [50, 4000, 40001])
def test_top_masked_and_bad_rows(sv, top_path, dtype, V):
    x = _top_rows(4, 8, V, dtype)
    x[1, 3:] = -math.inf                                     # fewer than k tokens
    x[2] = -math.inf
    x[3, V // 2] = math.nan
    x[4, V - 1] = math.inf
    x[5] = torch.finfo(x.dtype).min                          # the type's lowest value is a value
    x[6, ::2] = -math.inf
    x[7, : V - 1] = -math.inf                                # a single token
    if dtype != "f16":
        x[0, 0], x[0, 1] = 300.0, -300.0                     # nearly all mass on one token
    _check_top(sv, x, 20, 1.0, dtype)


@pytest.mark.parametrize("T", [0.05, 1.0, 20.0])
def test_top_temperatures_and_small_tails(sv, top_path, T):
    """A tail of 1e-30 keeps its relative accuracy."""
    x = _top_rows(6, 4, 3000, "f32")
    x[:, 7] += 60 * T
    _check_top(sv, x, 3, T, "f32")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("k", [3, 64, 700])
@pytest.mark.parametrize("kind", ["rising", "falling", "late", "steps"])
def test_top_ordered_rows(sv, top_path, dtype, k, kind):
    """Rows whose order makes every step bring better tokens than the last."""
    V = 60001
    x = torch.sort(_top_rows(k, 2, V, "f32"), -1).values
    if kind == "falling":
        x = x.flip(-1)
    if kind == "late":
        x = torch.cat([x[:, : V // 2].flip(-1), x[:, V // 2:]], -1)
    if kind == "steps":
        x = torch.floor(x * 2) / 2                           # rising, in runs of ties
    _check_top(sv, x.to(DTYPES[dtype]), k, 1.0, dtype)


@pytest.mark.parametrize("T", [1e-6, 1e-30, 1e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_top_extreme_temperatures(sv, top_path, dtype, T):
    x = _top_rows(12, 3, 9000, dtype)
    x[1] *= 1e20
    x[2] = torch.finfo(x.dtype).min
    idx, lp, tail = (_np(t) for t in sv.top_logits(x.to(DEV), 6, T))
    want_i, want_lp, want_t = rowsref.top(_np(x), 6, T)
    assert np.array_equal(idx, want_i)
    # logits / T reach 1e50: float32 results beyond its range are -inf, the
    # others are off by half a step; exponents that small weigh nothing
    big = np.abs(want_lp) > 3.4e38
    assert np.array_equal(np.isneginf(lp), big | np.isneginf(want_lp))
    ok = ~np.isneginf(lp)
    D = np.minimum(_spread(_np(x) / T), 120)[:, None]        # terms below e^-120 of the sum do not count
    np.testing.assert_array_less(np.abs(lp - want_lp)[ok], np.broadcast_to((40 + D) * U, lp.shape)[ok] + U * np.abs(want_lp[ok]) + 1e-30)
    assert not np.isnan(tail).any()


def test_top_workspace_of_many_rows_serves_fewer(sv):
    x = _top_rows(3, 400, 2500, "bf16")
    ws = sv.alloc_top_logits_workspace(400, 2500, 7, DEV)
    for rows in (400, 1, 20, 151, 152, 60, 400):
        _check_top(sv, x[:rows], 7, 1.0, "bf16", workspace=ws)
        assert int(ws.count_nonzero()) == 0


def test_top_shapes_workspace_and_outputs(sv):
    x = _top_rows(3, 12, 2500, "bf16").view(2, 2, 3, 2500)
    ws = sv.alloc_top_logits_workspace(12, 2500, 40, DEV)
    for k in (40, 7, 40):
        _check_top(sv, x, k, 1.0, "bf16", workspace=ws)
        assert int(ws.count_nonzero()) == 0, "the workspace is not left zero-filled"
    outs = (torch.empty(12, 5, dtype=torch.int32, device=DEV), torch.empty(12, 5, device=DEV), torch.empty(12, device=DEV))
    got = sv.top_logits(x.view(12, 2500).to(DEV), 5, outputs=outs)
    assert all(a is b for a, b in zip(got, outs))
    one = sv.top_logits(x[0, 0, 0].to(DEV), 5)
    assert one[0].shape == (5,) and one[2].shape == () and torch.equal(one[0], got[0][0])
    empty = sv.top_logits(x.view(12, 2500)[:0].to(DEV), 5)
    assert empty[0].shape == (0, 5)


def test_top_large_rows(sv, top_path):
    _check_top(sv, _top_rows(8, 1, (1 << 24) - 3, "bf16"), 50, 1.0, "bf16")
    _check_top(sv, _top_rows(9, 2, 152064, "f32"), 64, 1.0, "f32")
    _check_top(sv, _top_rows(10, 700, 9001, "bf16"), 17, 1.0, "bf16")


# ------------------------------------------------------------------ distill

@pytest.fixture(params=["distillpipe", "distillrow"])
def distill_path(request, monkeypatch):
    """Both kernels at every size: a persistent pipeline over rows, and a cluster per row."""
    monkeypatch.setenv("SPECVERIFY_PATH", request.param)
    return request.param


def _record(seed, R, V, k, tail, unique=True):
    g = torch.Generator().manual_seed(seed)
    if unique:
        idx = torch.stack([torch.randperm(V, generator=g)[:k] for _ in range(R)]).to(torch.int32)
        if idx.shape[1] < k:
            idx = torch.cat([idx, torch.full((R, k - idx.shape[1]), -1, dtype=torch.int32)], 1)
    else:
        idx = torch.randint(-1, max(2, V // 3), (R, k), generator=g, dtype=torch.int32)
    lp = torch.randn(R, k, generator=g) * 2
    return idx, lp, torch.randn(R, generator=g) + 2 if tail else None


def _forms(sv, S, idx, lp, tail, T, w, form):
    d = [None if t is None else t.to(DEV) for t in (idx, lp, tail, w)]
    x = S.to(DEV, copy=True)
    if form == "fused":
        loss, grad = sv.distill_loss_grad(x, d[0], d[1], d[2], T, weight=d[3])
        assert torch.equal(x.view(torch.uint8), S.to(DEV).view(torch.uint8)), "the student was written"
    elif form == "inplace":
        loss, grad = sv.distill_loss_grad(x, d[0], d[1], d[2], T, weight=d[3], out_grad=x)
        assert grad is x
    else:
        x.requires_grad_()
        loss = sv.distill_loss(x, d[0], d[1], d[2], T, weight=d[3])
        (grad,) = torch.autograd.grad(loss.sum(), x)
    torch.cuda.synchronize()
    return loss, grad


def _check_distill(sv, S, idx, lp, tail, T, dtype, w=None, form="fused"):
    loss, grad = _forms(sv, S, idx, lp, tail, T, w, form)
    want_l, want_g, scale = rowsref.distill(_np(S), _np(idx), _np(lp), _np(tail), T, _np(w))
    s = (40 + _spread(_np(S) / T)) * U
    aw = 1.0 if w is None else np.abs(_np(w))
    # the listed tokens' own terms: two-float weights, double differences: u of each term's magnitude
    mag = aw * (1 + np.abs(np.where(np.isfinite(_np(lp)), _np(lp), 0)).max(-1))
    fin = np.where(np.isfinite(want_l), want_l, 0)
    _assert_close(_np(loss), want_l, 2 * s * aw + U * (np.abs(fin) + mag), "loss")
    assert grad.dtype == S.dtype
    fg = np.where(np.isfinite(want_g), want_g, 0)
    _assert_close(_np(grad), want_g, (3 * s + 16 * U)[:, None] * scale + _half(dtype) * np.abs(fg) * (1 + 1e-3) + _tiny(dtype),
                  "gradient")


def _student(seed, R, V, dtype):
    return (torch.randn(R, V, generator=torch.Generator().manual_seed(seed)) * 2.5).to(DTYPES[dtype])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 100, 255, 1024, 5003])
@pytest.mark.parametrize("k", [1, 8])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("form", ["fused", "autograd"])
def test_distill_sizes(sv, distill_path, dtype, V, k, tail, form):
    if tail and V <= k:
        pytest.skip("no token is left for the tail (tested by itself)")
    idx, lp, t = _record(V + k, 3, V, k, tail)
    _check_distill(sv, _student(V, 3, V, dtype), idx, lp, t, 0.7, dtype, form=form)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [40000, 70001, 152064, 300007])
@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_distill_large_rows(sv, distill_path, dtype, V, form):
    """Rows over several CTAs of a cluster, and beyond its registers."""
    idx, lp, t = _record(V, 2, V, 64, True)
    idx[0, :4] = torch.tensor([0, V - 1, V // 2, 32768], dtype=torch.int32)
    _check_distill(sv, _student(V, 2, V, dtype), idx, lp, t, 1.0, dtype, form=form)


@pytest.mark.parametrize("k", [33, 512, 513, 1000, 1024])
@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_distill_wide_records(sv, distill_path, k, form):
    idx, lp, t = _record(k, 4, 3001, k, True)
    _check_distill(sv, _student(k, 4, 3001, "bf16"), idx, lp, t, 2.0, "bf16", form=form)


@pytest.mark.parametrize("V", [20, 40000])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_distill_tokens_listed_twice_and_ignored(sv, distill_path, V, tail, form):
    idx, lp, t = _record(3, 6, V, 12, tail, unique=False)
    idx[1, 4:9] = idx[1, 3]
    idx[2] = 5
    idx[3, ::2], idx[3, 1] = -7, V + 5
    _check_distill(sv, _student(1, 6, V, "f32"), idx, lp, t, 1.0, "f32", form=form)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_distill_empty_masked_and_bad_rows(sv, distill_path, dtype, form):
    V, k = 2003, 6
    S = _student(2, 14, V, dtype)
    idx, lp, t = _record(2, 14, V, k, True)
    inf, nan = math.inf, math.nan
    idx[0], t[0] = -1, -inf                                  # nothing to learn from
    idx[1] = V                                               # only the tail: one outcome, loss 0
    lp[2], t[2] = -inf, -inf
    S[3, ::2] = -inf
    S[3, idx[3].long()] = 1.0                                # masked student tokens the teacher does not list
    S[4, idx[4, 0].long()] = -inf                            # a listed one: infinite loss
    S[5] = -inf
    S[6, 100] = nan
    S[7, idx[7, 2].long()] = nan
    S[8, 5] = inf
    lp[9, 1] = nan
    t[10] = nan
    lp[11, 0], t[11] = -inf, -inf                            # a listed token of no weight, no tail mass
    keep = torch.zeros(V, dtype=torch.bool)
    keep[idx[12].long()] = True
    S[12, ~keep] = -inf                                      # no student mass outside the list
    S[13] = torch.finfo(S.dtype).min                         # the type's lowest value everywhere: uniform
    _check_distill(sv, S, idx, lp, t, 1.0, dtype, form=form)
    t[12] = -inf
    _check_distill(sv, S, idx, lp, t, 1.0, dtype, form=form)
    _check_distill(sv, S[11:13], idx[11:13], lp[11:13], None, 1.0, dtype, form=form)


@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_distill_weights(sv, distill_path, form):
    """Weight 0 rows are not read (they hold NaN) and give zeros; others scale."""
    V = 5000
    S = _student(5, 5, V, "f32")
    idx, lp, t = _record(5, 5, V, 9, True)
    S[1], lp[2], w = math.nan, math.nan, torch.tensor([0.5, 0.0, 0.0, -2.0, 1e-3])
    _check_distill(sv, S, idx, lp, t, 1.0, "f32", w=w, form=form)


@pytest.mark.parametrize("R, V, dtype, k", [(1000, 700, "bf16", 16), (333, 40001, "f16", 100), (200, 70000, "f32", 256),
                                            (160, 131000, "f32", 33), (155, 152064, "bf16", 7), (40, 262143, "bf16", 64)])
@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_distill_many_rows(sv, distill_path, R, V, dtype, k, form):
    """More rows than clusters fit at once, a third of them of weight 0, some
    with nothing to learn from, tokens listed twice here and there.  Rows are
    checked against the oracle in part (the first, the last and a spread)."""
    S = torch.randn(R, V, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).mul_(2.5).to(DTYPES[dtype])
    g = torch.Generator().manual_seed(R)
    idx = torch.randint(0, V, (R, k), generator=g, dtype=torch.int32)
    idx[1::7, -1] = idx[1::7, 0]
    idx[2::11] = -1
    lp, t = torch.randn(R, k, generator=g) * 2, torch.randn(R, generator=g) + 2
    t[2::22] = -math.inf
    w = torch.rand(R, generator=g) + 0.1
    w[::3] = 0.0
    w[R - 1] = 1.0
    pick = torch.unique(torch.cat([torch.arange(0, 4), torch.arange(R - 4, R), torch.linspace(0, R - 1, 40).long()]))
    want_S = S[pick.to(DEV)].cpu()
    loss, grad = _forms(sv, S, idx, lp, t, 1.3, w, form)
    zero = (w == 0).to(DEV)
    assert not loss[zero].any() and not grad[zero].any()
    want_l, want_g, scale = rowsref.distill(_np(want_S), _np(idx[pick]), _np(lp[pick]), _np(t[pick]), 1.3, _np(w[pick]))
    s, aw = (40 + _spread(_np(want_S) / 1.3)) * U, _np(w[pick])
    _assert_close(_np(loss)[pick], want_l, 2 * s * aw + U * (np.abs(want_l) + aw * (1 + np.abs(_np(lp[pick])).max(-1))), "loss")
    _assert_close(_np(grad[pick.to(DEV)]), want_g, (3 * s + 16 * U)[:, None] * scale + _half(dtype) * np.abs(want_g) * (1 + 1e-3) +
                  _tiny(dtype), "gradient")


@pytest.mark.parametrize("T", [1e-6, 1e-30, 1e4])
@pytest.mark.parametrize("form", ["fused", "autograd"])
def test_distill_extreme_temperatures(sv, distill_path, T, form):
    """Exponents out of float32's range weigh nothing; nothing becomes NaN."""
    V = 3000
    S = _student(3, 3, V, "f32")
    S[1] *= 1e18
    idx, lp, t = _record(3, 3, V, 4, True)
    idx[:, 0] = S.argmax(-1).int()                           # the student's only mass at low temperatures
    lp[:, 1:], t[:] = -math.inf, -math.inf                   # which is also the teacher's
    loss, grad = _forms(sv, S, idx, lp, t, T, None, form)
    want_l, want_g, _ = rowsref.distill(_np(S), _np(idx), _np(lp), _np(t), T)
    # the listed token holds all the teacher's mass: loss = -ln q there, a sum's logarithm
    s = (40 + np.minimum(_spread(_np(S) / T), 120)) * U
    _assert_close(_np(loss), want_l, 2 * s + U * np.abs(want_l), "loss")
    assert np.isfinite(_np(grad)).all()
    np.testing.assert_allclose(_np(grad), want_g, rtol=0, atol=float((3 * s.max() + 32 * U) / T))


def test_distill_nothing_outside_the_list(sv, distill_path):
    """k covers the vocabulary: without a tail mass the loss is an ordinary
    divergence, with one it is infinite (no token could carry it)."""
    S = _student(1, 2, 6, "f32")
    idx, lp, t = _record(1, 2, 6, 6, True)
    t[0] = -math.inf
    _check_distill(sv, S, idx, lp, t, 1.0, "f32", form="fused")
    _check_distill(sv, S, idx, lp, t, 1.0, "f32", form="autograd")


def test_distill_upstream_gradients_and_shapes(sv, distill_path):
    """Row gradients of any size reach the student, also as an expanded view."""
    V = 900
    S = _student(8, 6, V, "f32").view(2, 3, V)
    idx, lp, t = _record(8, 6, V, 7, True)
    x = S.to(DEV).requires_grad_()
    loss = sv.distill_loss(x, idx.view(2, 3, 7).to(DEV), lp.view(2, 3, 7).to(DEV), t.view(2, 3).to(DEV), 0.9)
    assert loss.shape == (2, 3)
    up = torch.tensor([[1.0, 0.0, -2.0], [0.25, 1e-4, 3.0]])
    (grad,) = torch.autograd.grad(loss, x, up.to(DEV))
    _, want, scale = rowsref.distill(_np(S).reshape(6, V), _np(idx), _np(lp), _np(t), 0.9)
    u = up.reshape(6, 1).double().numpy()
    s = (40 + _spread(_np(S).reshape(6, V) / 0.9)) * U
    _assert_close(_np(grad).reshape(6, V), want * u, (3 * s + 16 * U)[:, None] * scale * np.abs(u) + U * np.abs(want * u) * 2 + 2.0 ** -126,
                  "gradient")
    with torch.no_grad():
        assert not sv.distill_loss(x, idx.view(2, 3, 7).to(DEV), lp.view(2, 3, 7).to(DEV)).requires_grad
    e = sv.distill_loss(x[:0], idx.view(2, 3, 7)[:0].to(DEV), lp.view(2, 3, 7)[:0].to(DEV))
    assert e.shape == (0, 3)


def test_distill_gradient_against_differences(sv, distill_path):
    """The gradient against differences of the library's own loss (float32):
    with step e the quotient is off by at most 2 (loss error) / (2 e) plus
    e^2 / 6 of a third derivative below 1 / T^3."""
    V, T, e = 50, 1.0, 0.02
    S = _student(4, 1, V, "f32")
    idx, lp, t = _record(4, 1, V, 5, True)
    d = [v.to(DEV) for v in (idx, lp, t)]
    _, grad = sv.distill_loss_grad(S.to(DEV), *d, T)
    both = S.repeat(2 * V, 1)
    both[torch.arange(V), torch.arange(V)] += e
    both[V + torch.arange(V), torch.arange(V)] -= e
    step = (both[torch.arange(V), torch.arange(V)].double() - both[V + torch.arange(V), torch.arange(V)].double())
    loss = sv.distill_loss(both.to(DEV), *(v.expand(2 * V, *v.shape[1:]).contiguous() for v in d), T).cpu().double()
    quotient = (loss[:V] - loss[V:]) / step
    tol = 2 * (2 * (40 + 20) * U + 8 * U) / (2 * e) + e * e / 6
    assert float((grad.cpu().double()[0] - quotient).abs().max()) <= tol


# ------------------------------------------------------------------ as they are called

def test_refusals_of_the_wrappers(sv):
    L = torch.zeros(2, 3, 64, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    bad = [
        lambda: sv.adjust_logits(L[0]), lambda: sv.adjust_logits(L.transpose(0, 1)), lambda: sv.adjust_logits(L.double()),
        lambda: sv.adjust_logits(L, draft=torch.zeros(2, 3, **i32)), lambda: sv.adjust_logits(L, draft=torch.zeros(2, 2, device=DEV)),
        lambda: sv.adjust_logits(L, history=torch.zeros(2, 4, **i32)), lambda: sv.adjust_logits(L, repetition=torch.ones(2)),
        lambda: sv.adjust_logits(L, bias_tokens=torch.zeros(2, 4, **i32)), lambda: sv.adjust_logits(L, mask_index=torch.zeros(2, 3, **i32)),
        lambda: sv.adjust_logits(L, mask=torch.zeros(5, 2, **i32)), lambda: sv.adjust_logits(L, mask=torch.zeros(6, 3, **i32)),
        lambda: sv.adjust_logits(L, out=torch.zeros(2, 3, 64, dtype=torch.half, device=DEV)),
        lambda: sv.top_logits(L, 0), lambda: sv.top_logits(L, 1025), lambda: sv.top_logits(L[..., ::2], 4),
        lambda: sv.top_logits(L, 4, workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
        lambda: sv.distill_loss(L, torch.zeros(2, 4, **i32), torch.zeros(2, 4, device=DEV)),
        lambda: sv.distill_loss(L, torch.zeros(2, 3, 4, **i32), torch.zeros(2, 3, 4, device=DEV, requires_grad=True)),
        lambda: sv.distill_loss_grad(L, torch.zeros(2, 3, 4, **i32), torch.zeros(2, 3, 4, device=DEV), torch.zeros(2, device=DEV)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    big = torch.zeros(3, 3, 64, device=DEV).view(-1)
    with pytest.raises(sv.SvError):                          # out overlaps the input
        sv.adjust_logits(big[:384].view(2, 3, 64), out=big[64:448].view(2, 3, 64), presence=torch.ones(2, device=DEV))
    with pytest.raises(sv.SvError):
        sv.top_logits(L, 4, temperature=0.0)
    with pytest.raises(sv.SvError):
        sv.top_logits(L, 4, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(sv.SvError):
        sv.distill_loss(L, torch.zeros(2, 3, 4, **i32), torch.zeros(2, 3, 4, device=DEV), temperature=-1.0)


def test_loss_without_a_gradient_is_the_same(sv):
    """No autograd node where nobody asks for a gradient; forward-mode
    differentiation is refused, not dropped."""
    x = torch.randn(5, 300, device=DEV)
    idx, lp, tail = sv.top_logits(torch.randn(5, 300, device=DEV), 9)
    want = sv.distill_loss(x.clone().requires_grad_(), idx, lp, tail)
    assert want.requires_grad
    with torch.no_grad():
        off = sv.distill_loss(x.clone().requires_grad_(), idx, lp, tail)
    for got in (sv.distill_loss(x, idx, lp, tail), off):
        assert not got.requires_grad and torch.equal(got, want.detach())
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises((RuntimeError, NotImplementedError)):
            sv.distill_loss(torch.autograd.forward_ad.make_dual(x, torch.ones_like(x)), idx, lp, tail)


def test_double_backward_is_refused(sv):
    x = torch.randn(1, 40, device=DEV, requires_grad=True)
    loss = sv.distill_loss(x, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, 1, device=DEV))
    (g,) = torch.autograd.grad(loss.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_empty_batches(sv):
    assert sv.adjust_logits(torch.zeros(0, 3, 64, device=DEV)).shape == (0, 3, 64)
    idx, lp = torch.zeros(0, 4, dtype=torch.int32, device=DEV), torch.zeros(0, 4, device=DEV)
    loss, grad = sv.distill_loss_grad(torch.zeros(0, 64, device=DEV), idx, lp)
    assert loss.shape == (0,) and grad.shape == (0, 64)


def _round(seed=0, B=6, G=4, V=4096, k=16):
    g = torch.Generator().manual_seed(seed)
    target = torch.randn(B, G + 1, V, generator=g) * 2
    draft_logits = target[:, :G] + 0.7 * torch.randn(B, G, V, generator=g)
    return (target.to(torch.bfloat16), draft_logits.to(torch.bfloat16), torch.randint(0, V, (B, 30), generator=g, dtype=torch.int32),
            torch.rand(B, G + 1, generator=g), g)


def test_a_round_with_all_of_them(sv):
    """A round as a server that also trains its drafter runs it: the teacher's
    record of the raw target rows, the same constraints on target and draft
    rows, the verify step, and the drafter's loss on its rows.  The verify
    step's tokens must be allowed by the grammar, and match its oracle on the
    oracle's constrained rows."""
    from oracle import svref

    target, ql, hist, uni, g = _round()
    B, G1, V = target.shape
    G, k = G1 - 1, 16
    mask = (torch.rand(2, V // 32, 32, generator=g) < 0.3)
    words = (mask.long() << torch.arange(32)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    mi = torch.randint(-1, 2, (B, 1), generator=g, dtype=torch.int32).expand(B, G1).contiguous()
    lens = torch.full((B,), 30, dtype=torch.int32)
    con = dict(history=hist, history_len=lens, prompt_len=lens // 3, repetition=torch.full((B,), 1.2),
               frequency=torch.full((B,), 0.3), presence=torch.full((B,), 0.2), mask=words)
    dcon = {n: v.to(DEV) for n, v in con.items()}

    idx, lp, tail = sv.top_logits(target[:, :G].contiguous().to(DEV), k)
    # the drafts a drafter under the same constraints would make (its row i stands behind d_0 .. d_{i-1})
    drafts = torch.zeros(B, G, dtype=torch.int32)
    qrows = None
    for i in range(G):
        qrows = sv.adjust_logits(ql.to(DEV), draft=drafts[:, :G - 1].contiguous().to(DEV), mask_index=mi[:, :G].contiguous().to(DEV), **dcon)
        drafts[:, i] = qrows[:, i].float().argmax(-1).int().cpu()
    p = sv.adjust_logits(target.to(DEV), draft=drafts.to(DEV), mask_index=mi.to(DEV), **dcon)
    tokens, n, a, status = sv.verify_sample_qlogits(p, qrows, drafts.to(DEV), uni.to(DEV), 0.9)
    x = ql.to(DEV).requires_grad_()
    loss = sv.distill_loss(x, idx, lp, tail)
    loss.mean().backward()

    assert not status.any()
    tokens = tokens.cpu()
    for b in range(B):
        for t in tokens[b][tokens[b] >= 0].tolist():
            assert mi[b, 0] < 0 or mask[mi[b, 0]].view(-1)[t]
    ref = svref.verify_sample_qlogits(_np(p).astype(np.float32), _np(qrows).astype(np.float32), drafts.numpy(), uni.numpy(), 0.9)
    sure = ~ref["boundary"]
    assert np.array_equal(tokens.numpy()[sure], ref["out_tokens"][sure])
    want_l, want_g, scale = rowsref.distill(_np(ql).reshape(B * G, V), _np(idx).reshape(-1, k), _np(lp).reshape(-1, k),
                                            _np(tail).reshape(-1), 1.0)
    np.testing.assert_allclose(_np(loss).reshape(-1), want_l, rtol=0, atol=2 * 70 * U + 8 * U)
    _assert_close(_np(x.grad).reshape(B * G, V), want_g / (B * G),
                  ((3 * 70 + 20) * U) * scale / (B * G) + 2.0 ** -8 * np.abs(want_g) / (B * G) * 1.001 + 1e-38, "gradient")


def test_streams_and_graphs(sv):
    """Calls on a side stream, and captured and replayed on new inputs: the
    results of the eager calls, bit for bit."""
    target, ql, hist, _, _ = _round(3)
    t, q = target.to(DEV), ql.to(DEV)
    lens = torch.full((6,), 30, dtype=torch.int32, device=DEV)
    con = dict(history=hist.to(DEV), history_len=lens, presence=torch.ones(6, device=DEV))
    ws = sv.alloc_top_logits_workspace(24, 4096, 16, DEV)
    rows = t[:, :4].contiguous()

    def calls(**kw):
        adj = sv.adjust_logits(t, **con, **kw)
        rec = sv.top_logits(rows, 16, workspace=ws, **kw)
        loss, grad = sv.distill_loss_grad(q, *rec, **kw)
        return [adj, *rec, loss, grad]

    eager = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = calls(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    t.copy_(torch.roll(t, 1, -1))
    rows.copy_(torch.roll(rows, 1, -1))
    q.copy_(q * 1.5)
    graph.replay()
    torch.cuda.synchronize()
    again = calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, again))
    assert not torch.equal(held[-1], eager[-1])


def test_training_step_captured_while_an_eager_graph_lives(sv):
    """The fused call leaves no autograd graph, so it is captured beside a live
    eager one of the same student; the eager backward still runs afterwards."""
    idx, lp, t = (v.to(DEV) for v in _record(1, 8, 3000, 10, True))
    x = _student(1, 8, 3000, "f32").to(DEV).requires_grad_()
    live = sv.distill_loss(x, idx, lp, t).sum()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grad = sv.distill_loss_grad(x.detach(), idx, lp, t)
    graph.replay()
    live.backward()
    torch.cuda.synchronize()
    assert abs(float((loss.sum() - live).detach())) <= 8 * 140 * U
    # two forms of one formula: each within the tolerance of the same value
    assert float((grad - x.grad).abs().max()) <= 2 * (3 * 70 + 16) * U


def test_writes_into_given_tensors_are_seen_by_autograd(sv):
    """A graph that saved a tensor refuses its backward pass after a call has
    written over it; a gradient in place of the student likewise."""
    x = torch.randn(2, 1, 64, device=DEV, requires_grad=True)
    y = (x * 1).view(2, 1, 64)
    saved = (y * y).sum()
    pres, hist, n = torch.ones(2, device=DEV), torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    with torch.no_grad():
        sv.adjust_logits(y, history=hist, history_len=n, presence=pres, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.backward()
    idx, lp = torch.zeros(2, 4, dtype=torch.int32, device=DEV), torch.zeros(2, 4, device=DEV)
    s = torch.randn(2, 64, device=DEV, requires_grad=True)
    t = s * 1
    loss = sv.distill_loss(t, idx, lp).sum()
    sv.distill_loss_grad(t.detach(), idx, lp, out_grad=t.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():                             # no versions there, and none needed
        z = torch.randn(2, 1, 64, device=DEV)
        sv.adjust_logits(z, history=hist, history_len=n, presence=pres, out=z)


def test_a_workspace_by_default_and_two_streams_at_once(sv):
    """Calls on two streams at the same time, each with its own workspace,
    give what they give alone."""
    a, b = _top_rows(1, 40, 60000, "bf16").to(DEV), _top_rows(2, 40, 60000, "bf16").to(DEV)
    idx, lp, t = (v.to(DEV) for v in _record(5, 200, 30000, 20, True))
    S = _student(5, 200, 30000, "bf16").to(DEV)
    alone = [sv.top_logits(a, 30), sv.top_logits(b, 30), sv.distill_loss_grad(S, idx, lp, t), sv.distill_loss_grad(S, idx, lp, t)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = [sv.top_logits(a, 30, stream=s1), sv.top_logits(b, 30, stream=s2), sv.distill_loss_grad(S, idx, lp, t, stream=s1),
               sv.distill_loss_grad(S, idx, lp, t, stream=s2)]
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for g, w in zip(got, alone) for u, v in zip(g, w))
    assert sv.alloc_top_logits_workspace(3, 1000, 4).is_cuda


def test_results_do_not_depend_on_the_run(sv):
    """No sum's order depends on the schedule: repeated calls agree bit for bit."""
    L, a = _adjust_inputs(5, 8, 4, 20000, "f32", H=3000, NB=100)
    dev = {k: v.to(DEV) for k, v in a.items()}
    x = L.to(DEV)
    idx, lp, t = (v.to(DEV) for v in _record(1, 40, 20000, 50, True, unique=False))
    first = None
    for _ in range(4):
        adj = sv.adjust_logits(x, **dev).nan_to_num(nan=1e9)
        rec = sv.top_logits(x, 50)
        loss, grad = sv.distill_loss_grad(x.view(40, 20000), idx, lp, t)
        got = [adj, *rec, loss, grad]
        if first is not None:
            assert all(torch.equal(u, v) for u, v in zip(got, first))
        first = got
