"""The operators on logits rows: the library exports what its header declares,
and the host refuses bad arguments before any CUDA call (these run without a
GPU; the addresses are never dereferenced)."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_46_gb300 import build

    build.build_library()
    import speculative_decoding_verification_46_gb300 as pkg

    pkg.load_library()
    return pkg


def test_exports_every_declared_symbol(sv):
    text = open(os.path.join(ROOT, "include", "specverify_rows.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(sv_\w+)\s*\(", text))
    assert names == {"sv_adjust_logits", "sv_top_logits_workspace_bytes", "sv_top_logits", "sv_distill_forward",
                     "sv_distill_backward", "sv_distill_loss_grad"}
    lib = ctypes.CDLL(sv.load_library()._name)
    for n in names:
        assert hasattr(lib, n), n
    for name in ("SV_MAX_HISTORY", "SV_MAX_BIAS", "SV_DISTILL_STAT_WORDS"):
        value = re.search(rf"#define\s+{name}\s+(.+)", text).group(1)
        assert eval(value) == getattr(sv, name), name


def _adjust(sv, **kw):
    a = dict(B=4, gamma=3, V=100, logits=A, dtype=sv.SV_DTYPE_BF16, out=A + (1 << 20), draft=A + 8192, gamma_b=None,
             history=A + 12288, H=16, history_len=A + 16384, prompt_len=None, repetition=A + 20480, frequency=None,
             presence=None, bias_tokens=None, bias_values=None, NB=0, mask=None, M=0, mask_index=None, stream=None)
    a.update(kw)
    return sv.sv_adjust_logits(*a.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(gamma=-1), dict(gamma=65), dict(V=0), dict(V=(1 << 24) + 1),
                                dict(B=(1 << 24), gamma=1), dict(dtype=5), dict(logits=None), dict(out=None),
                                dict(logits=A + 2), dict(out=A + (1 << 20) + 8), dict(out=A + 16), dict(H=-1),
                                dict(H=(1 << 23) + 1), dict(history_len=None), dict(NB=-1), dict(NB=1025),
                                dict(NB=2), dict(NB=2, bias_tokens=A), dict(M=-1), dict(M=(1 << 24) + 1),
                                dict(mask=A, M=15), dict(mask=A, M=17)])
def test_adjust_refuses(sv, kw):
    assert _adjust(sv, **kw) == sv.SV_ERR_INVALID_ARG


def test_adjust_empty_calls(sv):
    assert _adjust(sv, B=0, logits=None, out=None) == sv.SV_OK
    # in place with nothing to apply: nothing is launched
    assert _adjust(sv, out=A, repetition=None) == sv.SV_OK
    assert _adjust(sv, out=A, history=None, H=0, draft=None) == sv.SV_OK


def _top(sv, **kw):
    a = dict(R=4, V=100, logits=A, dtype=sv.SV_DTYPE_BF16, k=8, temperature=1.0, indices=A + 4096, logprobs=A + 8192,
             tail=A + 12288, workspace=A + 16384, nbytes=1 << 30, stream=None)
    a.update(kw)
    return sv.sv_top_logits(*a.values())


@pytest.mark.parametrize("kw", [dict(R=-1), dict(R=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1), dict(dtype=3),
                                dict(k=0), dict(k=1025), dict(temperature=0.0), dict(temperature=-1.0),
                                dict(temperature=float("nan")), dict(temperature=float("inf")),
                                dict(temperature=1e-45), dict(logits=None), dict(logits=A + 8), dict(indices=None),
                                dict(logprobs=None), dict(tail=None)])
def test_top_refuses(sv, kw):
    assert _top(sv, **kw) == sv.SV_ERR_INVALID_ARG


def test_top_workspace(sv):
    need = sv.sv_top_logits_workspace_bytes(4, 100, 8)
    assert need > 0 and need % 256 == 0
    assert _top(sv, nbytes=need - 1) == sv.SV_ERR_WORKSPACE
    assert _top(sv, workspace=None) == sv.SV_ERR_WORKSPACE
    assert _top(sv, workspace=A + 4) == sv.SV_ERR_WORKSPACE
    assert _top(sv, R=0, logits=None, workspace=None, nbytes=0) == sv.SV_OK
    for bad in [(-1, 100, 8), (4, 0, 8), (4, 100, 0), (4, 100, 1025)]:
        assert sv.sv_top_logits_workspace_bytes(*bad) == 0
    # a list for every slice of a row; many rows need none
    assert sv.sv_top_logits_workspace_bytes(20, 152064, 64) >= 20 * 10 * 64 * 8
    assert sv.sv_top_logits_workspace_bytes(2304, 152064, 64) == 256


def _distill(sv, which, **kw):
    a = dict(R=4, V=100, student=A, dtype=sv.SV_DTYPE_F32, indices=A + 8192, logprobs=A + 12288, tail=A + 16384, k=8,
             temperature=1.0, weight=None, loss=A + 20480, stats=A + 24576, grad_loss=A + 28672, stride=1,
             grad=A + 32768)
    a.update(kw)
    head = [a[n] for n in ("R", "V", "student", "dtype", "indices", "logprobs")]
    if which == "forward":
        return sv.sv_distill_forward(*head, a["tail"], a["k"], a["temperature"], a["weight"], a["loss"], a["stats"], None)
    if which == "backward":
        return sv.sv_distill_backward(*head, a["k"], a["temperature"], a["weight"], a["stats"], a["grad_loss"], a["stride"],
                                      a["grad"], None)
    return sv.sv_distill_loss_grad(*head, a["tail"], a["k"], a["temperature"], a["weight"], a["loss"], a["grad"], None)


@pytest.mark.parametrize("which", ["forward", "backward", "loss_grad"])
@pytest.mark.parametrize("kw", [dict(R=-1), dict(R=(1 << 24) + 1), dict(V=0), dict(V=(1 << 24) + 1), dict(dtype=-1),
                                dict(k=0), dict(k=1025), dict(temperature=0.0), dict(temperature=float("nan")),
                                dict(student=None), dict(student=A + 4), dict(indices=None), dict(logprobs=None)])
def test_distill_refuses(sv, which, kw):
    assert _distill(sv, which, **kw) == sv.SV_ERR_INVALID_ARG


@pytest.mark.parametrize("which, kw", [("forward", dict(loss=None)), ("forward", dict(stats=A + 4)),
                                       ("backward", dict(stats=None)), ("backward", dict(grad_loss=None)),
                                       ("backward", dict(grad=None)), ("backward", dict(stride=-1)), ("backward", dict(stride=2)), ("backward", dict(grad=A + 16)),
                                       ("backward", dict(grad=A + 32772)), ("loss_grad", dict(loss=None)),
                                       ("loss_grad", dict(grad=None)), ("loss_grad", dict(grad=A + 1584)),
                                       ("loss_grad", dict(grad=A + 32776))])
def test_distill_refuses_by_form(sv, which, kw):
    assert _distill(sv, which, **kw) == sv.SV_ERR_INVALID_ARG


def test_distill_empty(sv):
    for which in ("forward", "backward", "loss_grad"):
        assert _distill(sv, which, R=0, student=None, indices=None, logprobs=None, loss=None, stats=None, grad=None,
                        grad_loss=None) == sv.SV_OK


def test_wrappers_refuse_cpu_tensors(sv):
    L = torch.zeros(2, 3, 16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.adjust_logits(L)
    with pytest.raises(ValueError, match="CUDA"):
        sv.top_logits(L, 4)
    idx, lp = torch.zeros(2, 3, 4, dtype=torch.int32), torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="CUDA"):
        sv.distill_loss(L, idx, lp)
    with pytest.raises(ValueError, match="CUDA"):
        sv.distill_loss_grad(L, idx, lp)
