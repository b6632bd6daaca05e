"""The operators on a round's key/value cache: the library exports what its
header declares, and the host refuses bad arguments before any CUDA call (these
run without a GPU; the addresses are never dereferenced)."""

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
    text = open(os.path.join(ROOT, "include", "specverify_cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(sv_\w+)\s*\(", text))
    assert names == {"sv_plan_round", "sv_append_kv4", "sv_read_kv4", "sv_attend_kv4_workspace_bytes", "sv_attend_kv4"}
    lib = ctypes.CDLL(sv.load_library()._name)
    for n in names:
        assert hasattr(lib, n) and hasattr(sv, n), n
    defined = re.findall(r"#define\s+(SV_(?:MAX|PLAN)_\w+)\s+(.+)", text)
    assert len(defined) == 8
    for name, value in defined:
        assert eval(value) == getattr(sv, name), name


def _plan(sv, **kw):
    a = dict(B=4, gamma=3, page=16, N=8, pool=32, lengths=A, kept=None, gamma_b=None, block_table=A, blocks=A, free_blocks=A,
             free_count=A, slots=A, positions=A, status=A, stream=None)
    a.update(kw)
    return sv.sv_plan_round(*a.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=8193), dict(gamma=-1), dict(gamma=1 << 24), dict(B=8192, gamma=4096),
                                dict(page=0), dict(page=8), dict(page=24), dict(page=272), dict(N=-1), dict(pool=-1),
                                dict(B=1024, N=(1 << 20) + 1), dict(N=(1 << 26) + 1), dict(pool=(1 << 26) + 1),
                                dict(lengths=None), dict(block_table=None), dict(blocks=None), dict(free_blocks=None),
                                dict(free_count=None), dict(slots=None), dict(positions=None), dict(status=None)])
def test_plan_refuses(sv, kw):
    assert _plan(sv, **kw) == sv.SV_ERR_INVALID_ARG


def test_empty_calls(sv):
    assert _plan(sv, B=0, lengths=None) == sv.SV_OK
    assert _append(sv, B=0, k=None) == sv.SV_OK
    assert _append(sv, pages=0, cache=None) == sv.SV_OK
    assert _read(sv, R=0, k=None) == sv.SV_OK
    assert _attend(sv, B=0, q=None, workspace=None) == sv.SV_OK


def _append(sv, **kw):
    a = dict(B=4, gamma=3, heads=2, D=64, page=16, pages=8, k=A, k_strides=(512, 128, 64), v=A + 65536, v_strides=(512, 128, 64),
             dtype=sv.SV_DTYPE_BF16, slots=A, cache=A + (1 << 20), stream=None)
    a.update(kw)
    return sv.sv_append_kv4(*a.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(gamma=-1), dict(B=1 << 20, gamma=16), dict(heads=0), dict(heads=1025), dict(D=96),
                                dict(D=256), dict(page=15), dict(page=512), dict(pages=-1), dict(pages=(1 << 26) + 1),
                                dict(k=None), dict(v=None), dict(slots=None), dict(cache=None), dict(k=A + 8), dict(v=A + 2),
                                dict(cache=A + (1 << 20) + 8), dict(cache=A), dict(cache=A + 65536 + 128), dict(cache=A - 16), dict(dtype=0), dict(dtype=7), dict(k_strides=None), dict(v_strides=None),
                                dict(k_strides=(512, 132, 64)), dict(v_strides=(512, -128, 64))])
def test_append_refuses(sv, kw):
    assert _append(sv, **kw) == sv.SV_ERR_INVALID_ARG


def _read(sv, **kw):
    a = dict(R=16, heads=2, D=64, page=16, pages=8, cache=A, dtype=sv.SV_DTYPE_F16, slots=A, k=A + (1 << 20), v=A + (1 << 21), stream=None)
    a.update(kw)
    return sv.sv_read_kv4(*a.values())


@pytest.mark.parametrize("kw", [dict(R=-1), dict(R=(1 << 24) + 1), dict(heads=0), dict(D=32), dict(page=20), dict(pages=-1),
                                dict(cache=None), dict(cache=A + 4), dict(dtype=0), dict(slots=None), dict(k=None),
                                dict(v=None), dict(k=A + (1 << 20) + 2), dict(v=A + (1 << 21) + 8), dict(k=A),
                                dict(v=A + 1024), dict(v=A + (1 << 20) + 4080)])
def test_read_refuses(sv, kw):
    assert _read(sv, **kw) == sv.SV_ERR_INVALID_ARG


def _attend(sv, **kw):
    a = dict(B=4, gamma=3, heads=2, G=4, D=64, page=16, pages=8, N=4, q=A, q_strides=(2048, 512, 64), dtype=sv.SV_DTYPE_BF16, cache=A + (1 << 21),
             block_table=A, lengths=A, gamma_b=None, scale=0.125, out=A + (1 << 20), lse=None, fill=0, workspace=A, nbytes=1 << 40, stream=None)
    a.update(kw)
    return sv.sv_attend_kv4(*a.values())


@pytest.mark.parametrize("kw", [dict(B=-1), dict(gamma=-1), dict(gamma=65), dict(heads=0), dict(G=0), dict(G=65), dict(D=72),
                                dict(page=0), dict(pages=-1), dict(N=-1), dict(N=(1 << 26) + 1), dict(q=None), dict(q=A + 8),
                                dict(q_strides=None), dict(q_strides=(2048, 516, 64)), dict(dtype=0), dict(cache=None),
                                dict(cache=A + (1 << 21) + 1), dict(block_table=None), dict(lengths=None), dict(scale=0.0),
                                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38),
                                dict(out=None), dict(out=A + (1 << 20) + 4), dict(out=A), dict(out=A + 16320),
                                dict(out=A + (1 << 21))])
def test_attend_refuses(sv, kw):
    assert _attend(sv, **kw) == sv.SV_ERR_INVALID_ARG


def test_attend_workspace(sv):
    need = sv.sv_attend_kv4_workspace_bytes(3, 2, 4, 64)
    assert need > 0
    assert _attend(sv, nbytes=need - 1) == sv.SV_ERR_WORKSPACE
    assert _attend(sv, workspace=None) == sv.SV_ERR_WORKSPACE
    assert _attend(sv, workspace=A + 4) == sv.SV_ERR_WORKSPACE
    for bad in [(-1, 2, 4, 64), (65, 2, 4, 64), (3, 0, 4, 64), (3, 2, 0, 64), (3, 2, 65, 64), (3, 2, 4, 80)]:
        assert sv.sv_attend_kv4_workspace_bytes(*bad) == 0


def test_wrappers_refuse_cpu_tensors(sv):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.plan_round(i, 3, 16, torch.zeros(4, 2, dtype=torch.int32), i, i, i[:1])
    x = torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 2, 16 * 72, dtype=torch.uint8)
    s = torch.zeros(4, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.append_kv4(x, x, s, c)
    with pytest.raises(ValueError, match="CUDA"):
        sv.read_kv4(c, s, 16, torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.attend_kv4(x, c, s, i, 16)
    with pytest.raises(ValueError, match="dtype"):
        sv.append_kv4(x.float(), x.float(), s, c)
    with pytest.raises(ValueError, match="dtype"):
        sv.read_kv4(c, s, 16, torch.float32)
    with pytest.raises(ValueError, match="no gradient"):
        sv.attend_kv4(x.clone().requires_grad_(), c, s, i, 16)
    with pytest.raises(sv.SvError):
        sv.alloc_kv4_cache(4, 2, 96)
    with pytest.raises(sv.SvError):
        sv.alloc_kv4_cache(4, 2, 64, page=20)
