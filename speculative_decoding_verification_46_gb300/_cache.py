"""ctypes binding of the operators on a round's paged key/value cache
(include/specverify_cache.h): the bookkeeping between two rounds, keys and
values into 4-bit pages and back, and the attention of a round's rows over
them.

As in ``_binding``: the functions named like the C entry points take raw
integers; the others take torch CUDA tensors, check them, allocate the outputs
and pass their addresses.  There is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._binding import (_TORCH_DTYPE, SV_ERR_INVALID_ARG, SV_OK, SvError, _addr, _c_float, _c_int, _c_ptr, _c_size,
                       _need_cuda, load_library)
from ._rows import _handle, _need, _need_constants, _on, _read_on, _written

SV_MAX_PLAN_SEQUENCES = 8192
SV_MAX_CACHE_PAGE = 256
SV_MAX_CACHE_SLOTS = 1 << 30
SV_MAX_CACHE_ROWS = 1 << 24
SV_MAX_CACHE_HEADS = 1024
SV_MAX_CACHE_GROUP = 64
SV_PLAN_NO_PAGES = 1
SV_PLAN_TOO_LONG = 2

_Strides = ctypes.c_int64 * 3


def _as_strides(s):
    return s if s is None or isinstance(s, _Strides) else _Strides(*s)


_declared = None   # the library object whose signatures are declared


def _lib():
    global _declared
    lib = load_library()
    if _declared is not lib:          # (as in _rows: asked of the object at hand)
        s = ctypes.POINTER(ctypes.c_int64)
        lib.sv_plan_round.argtypes = [_c_int] * 5 + [_c_ptr] * 11
        lib.sv_plan_round.restype = _c_int
        lib.sv_append_kv4.argtypes = [_c_int] * 6 + [_c_ptr, s, _c_ptr, s, _c_int, _c_ptr, _c_ptr, _c_ptr]
        lib.sv_append_kv4.restype = _c_int
        lib.sv_read_kv4.argtypes = [_c_int] * 5 + [_c_ptr, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr]
        lib.sv_read_kv4.restype = _c_int
        lib.sv_attend_kv4_workspace_bytes.argtypes = [_c_int] * 4
        lib.sv_attend_kv4_workspace_bytes.restype = _c_size
        lib.sv_attend_kv4.argtypes = [_c_int] * 8 + [_c_ptr, s, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_float,
                                                     _c_ptr, _c_ptr, _c_int, _c_ptr, _c_size, _c_ptr]
        lib.sv_attend_kv4.restype = _c_int
        _declared = lib
    return lib


# ------------------------------------------------------------ raw C entry points

def sv_plan_round(B, gamma, page, N, pool, lengths, kept, gamma_b, block_table, blocks, free_blocks, free_count, slots,
                  positions, status, stream) -> int:
    return int(_lib().sv_plan_round(B, gamma, page, N, pool, lengths, kept, gamma_b, block_table, blocks, free_blocks,
                                    free_count, slots, positions, status, stream))


def sv_append_kv4(B, gamma, heads, D, page, pages, k, k_strides, v, v_strides, dtype, slots, cache, stream) -> int:
    return int(_lib().sv_append_kv4(B, gamma, heads, D, page, pages, k, _as_strides(k_strides), v,
                                    _as_strides(v_strides), dtype, slots, cache, stream))


def sv_read_kv4(R, heads, D, page, pages, cache, dtype, slots, k, v, stream) -> int:
    return int(_lib().sv_read_kv4(R, heads, D, page, pages, cache, dtype, slots, k, v, stream))


def sv_attend_kv4_workspace_bytes(gamma: int, heads: int, G: int, D: int) -> int:
    return int(_lib().sv_attend_kv4_workspace_bytes(gamma, heads, G, D))


def sv_attend_kv4(B, gamma, heads, G, D, page, pages, N, q, q_strides, dtype, cache, block_table, lengths, gamma_b,
                  scale, out, lse, fill, workspace, workspace_bytes, stream) -> int:
    return int(_lib().sv_attend_kv4(B, gamma, heads, G, D, page, pages, N, q, _as_strides(q_strides), dtype,
                                    cache, block_table, lengths, gamma_b, scale, out, lse, fill, workspace,
                                    workspace_bytes, stream))


# ------------------------------------------------------------ torch wrappers

_MODEL_TYPES = (torch.bfloat16, torch.float16)
_i32 = torch.int32


def _need_model_rows(name, t):
    """[B, gamma+1, heads, D] of the model's type with contiguous elements."""
    if t.dtype not in _MODEL_TYPES:
        raise ValueError(f"unsupported {name} dtype {t.dtype}: bfloat16 or float16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, gamma+1, heads, D], got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _strides_of(t):
    """Strides of the first three dimensions (0 where there is one element, which may have any)."""
    b, i, h, _ = t.stride()
    if (b | i | h) & 7:
        return _Strides(*(st if n > 1 else 0 for n, st in zip(t.shape, (b, i, h))))
    return _Strides(b, i, h)


def _all_written(*tensors):
    """The caller's tensors have been written (see _written)."""
    try:
        torch.autograd.graph.increment_version(tensors)
    except RuntimeError:                     # some were made in inference mode and have no version
        for t in tensors:
            _written(t)


def _page_of(cache, page, D, heads, device):
    """Checks a cache [pages, heads, page * (D + 8)] and returns its pages."""
    if cache.dtype is not torch.uint8 or not cache.is_cuda or not cache.is_contiguous() or cache.dim() != 3:
        _need_cuda("cache", cache, torch.uint8)
        raise ValueError(f"cache must be [pages, heads, page * (D + 8)], got {tuple(cache.shape)}")
    if cache.device != device:
        raise ValueError(f"cache is on {cache.device}, the rows on {device}")
    if page < 16 or page > SV_MAX_CACHE_PAGE or page % 16:
        raise ValueError(f"page must be a multiple of 16 in 16..{SV_MAX_CACHE_PAGE}, got {page}")
    if D not in (64, 128):
        raise ValueError(f"head size must be 64 or 128, got {D}")
    if cache.shape[2] != page * (D + 8):
        raise ValueError(f"a block of {page} tokens with {D} channels has {page * (D + 8)} bytes, cache's {cache.shape[2]}")
    if cache.shape[1] < 1:
        raise ValueError("cache has no heads")
    if heads is not None and cache.shape[1] != heads:
        raise ValueError(f"cache has {cache.shape[1]} heads, the rows {heads}")
    return cache.shape[0]


def alloc_kv4_cache(pages: int, heads: int, D: int, page: int = 64, device=None) -> torch.Tensor:
    """A zero-filled cache [pages, heads, page * (D + 8)] uint8 (a zero-filled slot holds zeros)."""
    if D not in (64, 128) or page < 16 or page > SV_MAX_CACHE_PAGE or page % 16 or pages < 0 or heads < 1 or \
            heads > SV_MAX_CACHE_HEADS or pages * page > SV_MAX_CACHE_SLOTS:
        raise SvError(SV_ERR_INVALID_ARG, "alloc_kv4_cache")
    return torch.zeros(pages, heads, page * (D + 8), dtype=torch.uint8, device="cuda" if device is None else device)


def plan_round(lengths, gamma, page, block_table, blocks, free_blocks, free_count, *, kept=None, gamma_b=None,
               stream=None):
    """The bookkeeping between two rounds, in place on the state (sv_plan_round).

    lengths [B] int32 (tokens with valid keys and values) moves by kept [B]
    int32 (tokens of the last round that stay: n_accepted + 1, or what
    truncate_emitted returns; negative: taken back).  block_table [B, N] int32
    and blocks [B] int32 (each sequence's pages and their number) give back the
    pages that only rejected drafts used and take those that the next round
    needs, free_blocks [pool] int32 and free_count [1] int32 (the free pages,
    the last taken first) the other way round.  The next round has gamma
    drafts, or gamma_b [B] int32 of them (-1: the sequence takes no part).  All
    contiguous CUDA tensors on one device.  Returns (slots [B, gamma+1] int32,
    -1 behind a sequence's last row; positions [B, gamma+1] int32; status [B]
    int32, SV_PLAN_ bits: such a sequence got no pages and no slots, but its
    length has moved; give attend_kv4 gamma_b = -1 for it, and the next call
    kept = 0).  stream: as in adjust_logits.
    """
    dev = lengths.device
    B = lengths.shape[0] if lengths.dim() == 1 else -1
    N = block_table.shape[1] if block_table.dim() == 2 else 0
    pool = free_blocks.numel()
    gamma, page = int(gamma), int(page)
    _need_cuda("lengths", lengths, _i32)
    if B < 0:
        raise ValueError(f"lengths must be [B], got {tuple(lengths.shape)}")
    _need("block_table", block_table, _i32, (B, N), dev)
    _need("blocks", blocks, _i32, (B,), dev)
    _need("free_blocks", free_blocks, _i32, (pool,), dev)
    _need("free_count", free_count, _i32, (1,), dev)
    _need("kept", kept, _i32, (B,), dev)
    _need("gamma_b", gamma_b, _i32, (B,), dev)
    if gamma < 0 or B * (gamma + 1) > SV_MAX_CACHE_ROWS:
        raise ValueError(f"gamma must be at least 0 and B * (gamma + 1) at most {SV_MAX_CACHE_ROWS}, got {gamma}")
    with _on(dev, stream):
        if stream is not None:
            _read_on(stream, lengths, block_table, blocks, free_blocks, free_count, kept, gamma_b)
        slots = torch.empty((B, gamma + 1), dtype=_i32, device=dev)
        positions = torch.empty((B, gamma + 1), dtype=_i32, device=dev)
        status = torch.empty(B, dtype=_i32, device=dev)
        st = _lib().sv_plan_round(B, gamma, page, N, pool, lengths.data_ptr(), _addr(kept), _addr(gamma_b),
                                  block_table.data_ptr(), blocks.data_ptr(), free_blocks.data_ptr(),
                                  free_count.data_ptr(), slots.data_ptr(), positions.data_ptr(), status.data_ptr(),
                                  _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_plan_round")
    _all_written(lengths, block_table, blocks, free_blocks, free_count)
    return slots, positions, status


def append_kv4(k, v, slots, cache, *, stream=None):
    """Keys and values [B, gamma+1, heads, D] (bfloat16 / float16; any strides
    that are multiples of 8 elements, the last dimension contiguous) into the
    slots [B, gamma+1] int32 of a cache, quantised to 4 bits (sv_append_kv4);
    rows whose slot is negative or outside the cache are not written, and no
    slot may be given twice.  Returns cache.  No gradient is formed: outside
    torch.no_grad() tensors that require one are refused.  stream: as in
    adjust_logits.
    """
    _need_constants("k v", k, v)
    _need_model_rows("k", k)
    _need_model_rows("v", v)
    if v.shape != k.shape or v.dtype is not k.dtype or v.device != k.device:
        raise ValueError(f"v must be like k: {tuple(k.shape)} {k.dtype} on {k.device}, got {tuple(v.shape)} {v.dtype} on {v.device}")
    B, G1, heads, D = k.shape
    dev = k.device
    _need("slots", slots, _i32, (B, G1), dev)
    if D not in (64, 128):
        raise ValueError(f"head size must be 64 or 128, got {D}")
    page = cache.shape[-1] // (D + 8) if cache.dim() else 0
    pages = _page_of(cache, page, D, heads, dev)
    if G1 < 1:
        raise ValueError("k has no rows: [B, gamma+1, heads, D] with gamma >= 0")
    with _on(dev, stream):
        if stream is not None:
            _read_on(stream, k, v, slots, cache)
        st = _lib().sv_append_kv4(B, G1 - 1, heads, D, page, pages, k.data_ptr(), _strides_of(k), v.data_ptr(),
                                  _strides_of(v), _TORCH_DTYPE[k.dtype], slots.data_ptr(), cache.data_ptr(),
                                  _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_append_kv4")
    _written(cache)
    return cache


def read_kv4(cache, slots, page, dtype, *, stream=None):
    """What slots [...] int32 of a cache hold (sv_read_kv4): (k, v) [..., heads,
    D] of the model's type that was appended (`dtype`), 0 where a slot is
    negative or outside the cache.  stream: as in adjust_logits."""
    page = int(page)
    dev = slots.device
    if dtype not in _MODEL_TYPES:
        raise ValueError(f"unsupported dtype {dtype}: bfloat16 or float16")
    _need("slots", slots, _i32, slots.shape, dev)
    if cache.dim() != 3 or page < 1:
        raise ValueError(f"cache must be [pages, heads, page * (D + 8)], got {tuple(cache.shape)} and page {page}")
    D = cache.shape[2] // page - 8
    heads = cache.shape[1]
    pages = _page_of(cache, page, D, None, dev)
    with _on(dev, stream):
        if stream is not None:
            _read_on(stream, cache, slots)
        k = torch.empty((*slots.shape, heads, D), dtype=dtype, device=dev)
        v = torch.empty((*slots.shape, heads, D), dtype=dtype, device=dev)
        st = _lib().sv_read_kv4(slots.numel(), heads, D, page, pages, cache.data_ptr(), _TORCH_DTYPE[dtype],
                                slots.data_ptr(), k.data_ptr(), v.data_ptr(), _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_read_kv4")
    return k, v


def alloc_attend_workspace(gamma: int, heads: int, group: int, D: int, device=None) -> torch.Tensor:
    """A workspace for attend_kv4 on rounds of up to `gamma` drafts (any batch; kept by the caller, one per concurrent call)."""
    device = torch.device("cuda" if device is None else device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        if sv_attend_kv4_workspace_bytes(gamma, heads, group, D) == 0:
            raise SvError(SV_ERR_INVALID_ARG, "sv_attend_kv4_workspace_bytes")
        n = max(sv_attend_kv4_workspace_bytes(g, heads, group, D) for g in range(gamma + 1))
    return torch.empty(n, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=256)
def _attend_workspace_bytes(gamma, heads, group, D, device_index):
    """(of the current device, whose index is passed: its SMs count)"""
    return sv_attend_kv4_workspace_bytes(gamma, heads, group, D)


def attend_kv4(q, cache, block_table, lengths, page, *, gamma_b=None, scale=None, out=None, return_lse=False,
               workspace=None, stream=None):
    """Attention of a round's rows over the 4-bit cache (sv_attend_kv4).

    q [B, gamma+1, query heads, D] (bfloat16 / float16, the type of the rows
    that were appended; any strides that are multiples of 8 elements, the last
    dimension contiguous); the query heads share the cache's heads in equal
    groups of neighbours.  Row i of sequence b sees the positions 0 ..
    lengths[b] + i through block_table [B, N] int32: lengths [B] int32 counts
    the tokens before the round, whose own tokens have been appended; table
    entries that are no page hide their tokens.  (Few short sequences are
    served faster where the table has no more columns than they have pages: up
    to 16640 positions are one launch.)  gamma_b [B] int32: a ragged
    round, rows behind a sequence's last are not computed (-1: none is).
    scale: 1 / sqrt(D) by default.  Returns out [B, gamma+1, query heads, D],
    with return_lse also the logarithm of each row's sum [B, gamma+1, query
    heads] float32; a row that sees nothing is 0 (and -inf).  Rows behind
    gamma_b are 0 in new tensors and stay as they are in a given `out`.
    workspace: from alloc_attend_workspace.  No gradient is formed: outside
    torch.no_grad() tensors that require one are refused.  stream: as in
    adjust_logits.
    """
    _need_constants("q out", q, out)
    _need_model_rows("q", q)
    B, G1, HQ, D = q.shape
    dev = q.device
    page = int(page)
    pages = _page_of(cache, page, D, None, dev)
    heads = cache.shape[1]
    if HQ < 1 or HQ % heads:
        raise ValueError(f"{HQ} query heads do not share {heads} heads equally")
    if G1 < 1:
        raise ValueError("q has no rows: [B, gamma+1, query heads, D] with gamma >= 0")
    N = block_table.shape[1] if block_table.dim() == 2 else 0
    _need("block_table", block_table, _i32, (B, N), dev)
    _need("lengths", lengths, _i32, (B,), dev)
    _need("gamma_b", gamma_b, _i32, (B,), dev)
    _need("out", out, q.dtype, (B, G1, HQ, D), dev)
    if workspace is not None:
        _need_cuda("workspace", workspace, torch.uint8)
        if workspace.device != dev:
            raise ValueError(f"workspace is on {workspace.device}, the rows on {dev}")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    given = out
    with _on(dev, stream):
        if stream is not None:
            _read_on(stream, q, cache, block_table, lengths, gamma_b, out, workspace)
        if out is None:
            out = torch.empty((B, G1, HQ, D), dtype=q.dtype, device=dev)
        lse = None
        if return_lse:
            # rows behind gamma_b: 0, which the kernel writes only where `out` is new too
            make = torch.zeros if given is not None and gamma_b is not None else torch.empty
            lse = make((B, G1, HQ), dtype=torch.float32, device=dev)
        if workspace is None:
            n = _attend_workspace_bytes(G1 - 1, heads, HQ // heads, D, dev.index)
            if n == 0:
                raise SvError(SV_ERR_INVALID_ARG, "sv_attend_kv4")
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        st = _lib().sv_attend_kv4(B, G1 - 1, heads, HQ // heads, D, page, pages, N, q.data_ptr(), _strides_of(q),
                                  _TORCH_DTYPE[q.dtype], cache.data_ptr(), block_table.data_ptr(), lengths.data_ptr(),
                                  _addr(gamma_b), scale, out.data_ptr(), _addr(lse), given is None,
                                  workspace.data_ptr(), workspace.numel(), _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_attend_kv4")
    if given is not None:
        _written(out)
    return (out, lse) if return_lse else out
