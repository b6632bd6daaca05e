"""The operators on logits rows on the GPU where calls meet: in place beside
other CTAs, long common offsets, wide temperatures, threads, streams and waits
that give up.  Against the float64 oracle with the tolerances of
test_gpu_rows.py, or bit for bit against another form of the same call."""

import pytest
import torch

from test_gpu_rows import DEV, DTYPES, _check_distill, _record, _student, distill_path, sv  # noqa: F401

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
