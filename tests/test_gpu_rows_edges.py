"""The operators on logits rows on the GPU where calls meet: in place beside
other CTAs, long common offsets, wide temperatures, threads, streams and waits
that give up.  Against the float64 oracle with the tolerances of
test_gpu_rows.py, or bit for bit against another form of the same call."""

import os
import subprocess
import sys

import pytest
import torch

from test_gpu_rows import (DEV, DTYPES, _check_distill, _check_top, _forms, _record, _student, _top_rows,  # noqa: F401
                           distill_path, sv, top_path)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ in place

@pytest.mark.parametrize("dtype, V, k", [("bf16", 130001, 1024), ("bf16", 152064, 300), ("f16", 40000, 600), ("f32", 70000, 1000),
                                         ("f32", 152064, 64), ("bf16", 300007, 40)])
def test_distill_in_place_with_tokens_listed_twice_in_every_slice(sv, dtype, V, k):
    """A cluster's CTAs count a token listed twice once without looking at the
    row again, which other CTAs turn into the gradient meanwhile: in place the
    results are those of a separate tensor, bit for bit."""
    R = 200
    S = torch.randn(R, V, generator=torch.Generator(device=DEV).manual_seed(k), device=DEV).mul_(2.5).to(DTYPES[dtype])
    g = torch.Generator().manual_seed(V)
    idx = torch.randint(0, V, (R, k), generator=g, dtype=torch.int32)
    idx[:, k // 2:] = idx[:, :k - k // 2].flip(1)             # every token of the first half again, all over the row
    lp, t = (torch.randn(R, k, generator=g) * 2).to(DEV), (torch.randn(R, generator=g) + 2).to(DEV)
    idx = idx.to(DEV)
    want = sv.distill_loss_grad(S, idx, lp, t, 1.3)
    for _ in range(10):
        x = S.clone()
        loss, grad = sv.distill_loss_grad(x, idx, lp, t, 1.3, out_grad=x)
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])


@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
@pytest.mark.parametrize("k", [12, 700])
def test_distill_tokens_listed_twice_in_wide_rows(sv, distill_path, form, k):
    S = _student(2, 3, 60000, "f32")
    idx, lp, t = _record(4, 3, 60000, k, True)
    idx[:, 1::2] = idx[:, 0::2]
    _check_distill(sv, S, idx, lp, t, 1.0, "f32", form=form)


def test_the_gradient_in_place_of_rows_that_a_model_made(sv):
    """Rows that require a gradient turn into it, and it is handed on to what
    made them: the parameters' gradients are those of the autograd form."""
    R, D, V = 40, 64, 3000
    g = torch.Generator(device=DEV).manual_seed(4)
    h, W0 = torch.randn(R, D, generator=g, device=DEV), torch.randn(D, V, generator=g, device=DEV) / 8
    idx, lp, t = (x.to(DEV) for x in _record(4, R, V, 12, True))
    grads = []
    for fused in (False, True):
        W = W0.clone().requires_grad_()
        rows = h @ W
        if fused:
            _, grad = sv.distill_loss_grad(rows, idx, lp, t, out_grad=rows)
            assert grad is rows
            rows.backward(grad.detach())
        else:
            sv.distill_loss(rows, idx, lp, t).sum().backward()
        grads.append(W.grad)
    # two forms of one formula, each within (3 s + 16 u) of its magnitudes (at most 2 an element), summed over the rows
    tol = R * 2 * (3 * (40 + 60) + 16) * 2.0 ** -24 * float(h.abs().max())
    assert float((grads[0] - grads[1]).abs().max()) <= tol


# ------------------------------------------------------------------ large common offsets

@pytest.mark.parametrize("offset", [0.0, 100.0, 1e4, -1e4, 2e5, 3e6, -3e6, 5545177.0, -5545177.0, 6e6])
@pytest.mark.parametrize("order", ["rising", "as_they_come", "falling"])
@pytest.mark.parametrize("T, k", [(1.0, 3), (1.0, 300), (0.7, 20)])
def test_top_rows_with_a_common_offset(sv, top_path, offset, order, T, k):
    """The mass outside keeps its accuracy where every step of a row raises the
    maximum, whatever the logits have in common (beyond 8e6 T / log2(e), about
    5.5e6, terms are formed another way, and rows rise across that border)."""
    x = _top_rows(11, 3, 60001, "f32")
    if order != "as_they_come":
        x = torch.sort(x, -1, descending=order == "falling").values
    _check_top(sv, x + offset, k, T, "f32")


@pytest.mark.parametrize("dtype, offset", [("bf16", 200.0), ("bf16", -3000.0), ("f16", 1000.0), ("f16", -200.0)])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_top_16_bit_rows_with_a_common_offset(sv, top_path, dtype, offset, order):
    x = torch.sort(_top_rows(12, 3, 100003, "f32"), -1, descending=order == "falling").values
    _check_top(sv, (x + offset).to(DTYPES[dtype]), 40, 0.8, dtype)


# ------------------------------------------------------------------ wide temperatures

@pytest.mark.parametrize("T", [100.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("below", [0.5, 2.0, 10.0, 60.0])
@pytest.mark.parametrize("form", ["fused", "autograd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_listed_tokens_far_below_at_high_temperatures(sv, distill_path, T, below, form, dtype):
    """A listed logit far below the row's maximum still has weight where the
    temperature is as large."""
    S = (_student(7, 4, 2000, "f32") * T / 8).to(DTYPES[dtype])
    idx, lp, t = _record(7, 4, 2000, 9, True)
    idx[3, 5] = idx[3, 4]
    S[torch.arange(4)[:, None], idx.long()] = (S.float().max() - below * T * (1 + torch.rand(4, 9))).to(DTYPES[dtype])
    _check_distill(sv, S, idx, lp, t, T, dtype, form=form)


# ------------------------------------------------------------------ bad teachers

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("k", [6, 300])
@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_distill_bad_teacher_of_a_student_without_mass_outside(sv, distill_path, dtype, k, form):
    """A teacher's NaN or +inf makes the whole row NaN, also where the student
    has nothing outside the list to move."""
    V = 2003
    S = _student(3, 6, V, dtype)
    idx, lp, t = _record(3, 6, V, k, True)
    outside = torch.ones(6, V, dtype=torch.bool).scatter_(1, idx.long(), False)
    S[outside] = -float("inf")
    lp[0, 2], lp[1, 0], t[2], t[3], t[4] = float("nan"), float("inf"), float("nan"), float("inf"), -float("inf")
    _check_distill(sv, S, idx, lp, t, 1.0, dtype, form=form)
    _check_distill(sv, S[:2], idx[:2], lp[:2], None, 1.0, dtype, form=form)


# ------------------------------------------------------------------ threads

_HARNESS = """
#include <atomic>
#include <cstdint>
#include <thread>
#include <vector>
typedef int (*adjust_fn)(int, int, int, const void*, int, void*, const int32_t*, const int32_t*, const int32_t*, int, const int32_t*,
                         const int32_t*, const float*, const float*, const float*, const int32_t*, const float*, int, const uint32_t*,
                         int, const int32_t*, void*);
// n threads, each on its own stream and output; at every step they start together
extern "C" int refused(adjust_fn call, int n, int B, int V, int dtype, const void* x, void** out, const int32_t* tokens,
                       const float* values, void** stream) {
  std::atomic<int> here{0}, bad{0};
  std::vector<std::thread> threads;
  for (int i = 0; i < n; ++i)
    threads.emplace_back([&, i] {
      for (int step = 0; step < 1024 / n; ++step) {
        here.fetch_add(1);
        while (here.load() < n * (step + 1)) {}
        if (call(B, 0, V, x, dtype, out[i], 0, 0, 0, 0, 0, 0, 0, 0, 0, tokens, values, step * n + n - i, 0, 0, 0, stream[i]) != 0) ++bad;
      }
    });
  for (auto& t : threads) t.join();
  return bad;
}
"""

_THREADS = """
import ctypes, sys
sys.path.insert(0, {root!r})
import torch
import speculative_decoding_verification_46_gb300 as sv

# many sequences of one full tile each, and lists that grow from call to call: every call needs more shared memory
# than all steps before, a little more or less than those beside it
B, V, n = 512, 6144, 8
x = torch.zeros(B, 1, V, dtype=torch.{dtype}, device="cuda")
outs = [torch.empty_like(x) for _ in range(n)]
streams = [torch.cuda.Stream() for _ in range(n)]
tokens, values = torch.full((B * 1024,), -1, dtype=torch.int32, device="cuda"), torch.zeros(B * 1024, device="cuda")
torch.cuda.synchronize()
call = ctypes.cast(sv._rows._lib().sv_adjust_logits, ctypes.c_void_p)
many = lambda values: (ctypes.c_void_p * n)(*values)
refused = ctypes.CDLL({harness!r}).refused
refused.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 4 + [ctypes.c_void_p] * 5
print(refused(call, n, B, V, sv._rows._TORCH_DTYPE[x.dtype], x.data_ptr(), many(o.data_ptr() for o in outs), tokens.data_ptr(),
              values.data_ptr(), many(s.cuda_stream for s in streams)))
torch.cuda.synchronize()
assert all(torch.equal(o, x) for o in outs)
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_calls_of_many_threads_that_need_more_and_more_shared_memory(sv, tmp_path, dtype):
    """Threads whose calls need different amounts of shared memory, more than
    any call before: none takes another's away (in a process of its own, where
    no earlier call has asked for the most)."""
    (tmp_path / "harness.cpp").write_text(_HARNESS)
    harness = str(tmp_path / "harness.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-o", harness, str(tmp_path / "harness.cpp")], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", _THREADS.format(root=root, dtype=dtype, harness=harness)], capture_output=True, text=True,
                         timeout=240)
    assert out.returncode == 0, out.stderr
    assert int(out.stdout) == 0, f"{out.stdout.strip()} of 1024 calls were refused"


# ------------------------------------------------------------------ waits that run out

@pytest.mark.parametrize("R, V, dtype, k, stop", [(300, 70000, "f32", 33, 2), (400, 40001, "bf16", 8, 5), (400, 40001, "bf16", 8, 0),
                                                  (160, 152064, "f16", 200, 4), (3, 900, "f32", 5, 0), (300, 70000, "f32", 33, 1000)])
@pytest.mark.parametrize("form", ["fused", "inplace", "autograd"])
def test_rows_of_a_pipeline_that_gives_up_are_nan_throughout(sv, monkeypatch, R, V, dtype, k, stop, form):
    """One warp of each cluster leaves at the cluster's row `stop` and the
    waits of the others run out: a row is what it always is, or NaN in its loss
    and all of its gradient, never a part of either; and the next call is as
    usual."""
    S = torch.randn(R, V, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).mul_(2.5).to(DTYPES[dtype])
    idx, lp, t = _record(R, R, V, k, True)
    idx[1::7, -1] = idx[1::7, 0]
    w = torch.rand(R, generator=torch.Generator().manual_seed(2)) + 0.1
    w[2::5] = 0.0
    want = _forms(sv, S, idx, lp, t, 1.1, w, form)
    monkeypatch.setenv("SPECVERIFY_PATH", f"distillstop{stop}")
    loss, grad = _forms(sv, S, idx, lp, t, 1.1, w, form)
    lost = loss.isnan()
    assert torch.equal(loss[~lost], want[0][~lost]) and torch.equal(grad[~lost], want[1][~lost])
    assert int(lost.sum()) == R if stop == 0 else not lost.any() if stop == 1000 else 0 < int(lost.sum())
    if form == "autograd":
        lost &= (w != 0).to(DEV)                              # the backward pass asks the weight first
    assert grad[lost].isnan().all()
    monkeypatch.delenv("SPECVERIFY_PATH")
    again = _forms(sv, S, idx, lp, t, 1.1, w, form)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


# ------------------------------------------------------------------ streams

def test_inputs_may_be_dropped_after_a_call_on_another_stream(sv):
    """Memory of inputs that the caller lets go of is not handed out again
    while the given stream has yet to read it."""
    R, V, k = 48, 50000, 9
    g = torch.Generator(device=DEV).manual_seed(3)
    made = dict(logits=torch.randn(R, 1, V, generator=g, device=DEV),
                history=torch.randint(0, V, (R, 3000), generator=g, device=DEV, dtype=torch.int32),
                history_len=torch.full((R,), 3000, device=DEV, dtype=torch.int32), presence=torch.rand(R, generator=g, device=DEV),
                bias_tokens=torch.randint(0, V, (R, 500), generator=g, device=DEV, dtype=torch.int32),
                bias_values=torch.randn(R, 500, generator=g, device=DEV),
                mask=torch.randint(-2 ** 31, 2 ** 31, (R, (V + 31) // 32), generator=g, device=DEV).to(torch.int32))
    idx, lp, t = (x.to(DEV) for x in _record(2, R, V, k, True))
    record = dict(indices=idx, logprobs=lp, tail=t, weight=torch.rand(R, generator=g, device=DEV))
    calls = [lambda a, **kw: [sv.adjust_logits(**a, **kw)], lambda a, **kw: list(sv.top_logits(a["logits"], k, **kw)),
             lambda a, **kw: list(sv.distill_loss_grad(a["logits"].view(R, V), **{n: a[n] for n in record}, **kw))]
    for call, names in zip(calls, (made, ["logits"], ["logits", *record])):
        inputs = {n: made[n] if n in made else record[n] for n in names}
        want = call(dict(inputs))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        copies = {n: x.clone() for n, x in inputs.items()}
        sizes = [(x.shape, x.dtype) for x in copies.values()]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        got = call(copies, stream=side)
        copies.clear()
        for _ in range(3):                                    # what is allocated now must not be what they were
            [torch.zeros(shape, dtype=dtype, device=DEV) for shape, dtype in sizes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ more than 2^31 elements

@pytest.mark.parametrize("V", [128256, 128003])
def test_rows_beyond_32_bit_offsets(sv, V):
    """The last rows of a tensor of more than 2^31 elements are what they are
    in a tensor of their own (from a row on that starts at the same place of a
    16-byte vector), in every operator."""
    R, n, k = 17000, 200, 20
    assert R * V > 2 ** 31 and (R - n) * V % 8 == 0
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(R, V, dtype=torch.bfloat16, device=DEV)
    for r in range(0, R, 1000):
        x[r:r + 1000] = torch.randn(1000, V, generator=g, device=DEV) * 2.5
    last = x[R - n:].clone()
    h = torch.randint(0, V, (R, 100), generator=g, device=DEV, dtype=torch.int32)
    lens, pen = torch.full((R,), 100, device=DEV, dtype=torch.int32), torch.rand(R, generator=g, device=DEV) + 0.5
    at = slice(R - n, None)

    def adjust(rows, part):
        return sv.adjust_logits(rows.unsqueeze(1), history=h[part].contiguous(), history_len=lens[part].contiguous(),
                                repetition=pen[part].contiguous(), presence=pen[part].contiguous()).squeeze(1)

    assert torch.equal(adjust(x, slice(None))[at], adjust(last, at))
    rec, own = sv.top_logits(x, k), sv.top_logits(last, k)
    assert all(torch.equal(a[at], b) for a, b in zip(rec, own))
    w = torch.rand(R, generator=g, device=DEV)
    loss, grad = sv.distill_loss_grad(x, *rec, 1.2, weight=w)
    want = sv.distill_loss_grad(last, *own, 1.2, weight=w[at].contiguous())
    assert torch.equal(loss[at], want[0]) and torch.equal(grad[at], want[1])
    del grad
    sv.distill_loss_grad(x, *rec, 1.2, weight=w, out_grad=x)
    assert torch.equal(x[at], want[1])
    x[at] = last
    y, z = x.requires_grad_(), last.clone().requires_grad_()
    (a,) = torch.autograd.grad(sv.distill_loss(y, *rec, 1.2, weight=w).sum(), y)
    (b,) = torch.autograd.grad(sv.distill_loss(z, *own, 1.2, weight=w[at].contiguous()).sum(), z)
    assert torch.equal(a[at], b)


def test_wide_records_beyond_32_bit_offsets(sv):
    """The same for the form with a cluster per row (lists above 256 tokens)."""
    R, n, k, V = 17000, 40, 300, 128256
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.empty(R, V, dtype=torch.bfloat16, device=DEV)
    for r in range(0, R, 1000):
        x[r:r + 1000] = torch.randn(1000, V, generator=g, device=DEV) * 2.5
    idx = torch.randint(0, V, (R, k), generator=g, device=DEV, dtype=torch.int32)
    lp, at = torch.randn(R, k, generator=g, device=DEV), slice(R - n, None)
    want = sv.distill_loss_grad(x[at].clone(), idx[at].contiguous(), lp[at].contiguous())
    loss, _ = sv.distill_loss_grad(x, idx, lp, out_grad=x)
    assert torch.equal(loss[at], want[0]) and torch.equal(x[at], want[1])
