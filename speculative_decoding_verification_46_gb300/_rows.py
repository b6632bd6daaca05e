"""ctypes binding of the operators on logits rows (include/specverify_rows.h):
penalties, biases and masks before the verify step; a teacher's top logits and
distillation of the draft from them.

As in ``_binding``: the functions named like the C entry points take raw
integers; the others take torch CUDA tensors, check them, allocate the outputs
and pass their addresses.  There is no fallback.
"""

from __future__ import annotations

import torch
from torch.autograd import forward_ad

from ._binding import (_TORCH_DTYPE, SV_ERR_INVALID_ARG, SV_OK, SvError, _addr, _c_float, _c_int, _c_ptr, _c_size,
                       _need_cuda, load_library)

SV_MAX_HISTORY = 1 << 23
SV_MAX_BIAS = 1024
SV_DISTILL_STAT_WORDS = 8

_declared = None   # the library object whose signatures are declared


def _lib():
    global _declared
    lib = load_library()
    # Threads whose first calls meet may each have loaded an object of their
    # own: what is declared is asked of the object at hand (a call without
    # signatures would pass addresses as 32-bit integers).
    if _declared is not lib:
        lib.sv_adjust_logits.argtypes = [_c_int, _c_int, _c_int, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int,
                                         _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_ptr, _c_int,
                                         _c_ptr, _c_ptr]
        lib.sv_adjust_logits.restype = _c_int
        lib.sv_top_logits_workspace_bytes.argtypes = [_c_int, _c_int, _c_int]
        lib.sv_top_logits_workspace_bytes.restype = _c_size
        lib.sv_top_logits.argtypes = [_c_int, _c_int, _c_ptr, _c_int, _c_int, _c_float, _c_ptr, _c_ptr, _c_ptr, _c_ptr,
                                      _c_size, _c_ptr]
        lib.sv_top_logits.restype = _c_int
        lib.sv_distill_forward.argtypes = [_c_int, _c_int, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_float,
                                           _c_ptr, _c_ptr, _c_ptr, _c_ptr]
        lib.sv_distill_forward.restype = _c_int
        lib.sv_distill_backward.argtypes = [_c_int, _c_int, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_int, _c_float, _c_ptr,
                                            _c_ptr, _c_ptr, _c_int, _c_ptr, _c_ptr]
        lib.sv_distill_backward.restype = _c_int
        lib.sv_distill_loss_grad.argtypes = [_c_int, _c_int, _c_ptr, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_float,
                                             _c_ptr, _c_ptr, _c_ptr, _c_ptr]
        lib.sv_distill_loss_grad.restype = _c_int
        _declared = lib
    return lib


# ------------------------------------------------------------ raw C entry points

def sv_adjust_logits(B, gamma, V, logits, dtype, out, draft_tokens, gamma_b, history, H, history_len, prompt_len,
                     repetition, frequency, presence, bias_tokens, bias_values, NB, mask, M, mask_index, stream) -> int:
    return int(_lib().sv_adjust_logits(B, gamma, V, logits, dtype, out, draft_tokens, gamma_b, history, H, history_len,
                                       prompt_len, repetition, frequency, presence, bias_tokens, bias_values, NB, mask,
                                       M, mask_index, stream))


def sv_top_logits_workspace_bytes(R: int, V: int, k: int) -> int:
    return int(_lib().sv_top_logits_workspace_bytes(R, V, k))


def sv_top_logits(R, V, logits, dtype, k, temperature, indices, logprobs, tail, workspace, workspace_bytes,
                  stream) -> int:
    return int(_lib().sv_top_logits(R, V, logits, dtype, k, float(temperature), indices, logprobs, tail, workspace,
                                    workspace_bytes, stream))


def sv_distill_forward(R, V, student, dtype, indices, logprobs, tail, k, temperature, weight, loss, stats,
                       stream) -> int:
    return int(_lib().sv_distill_forward(R, V, student, dtype, indices, logprobs, tail, k, float(temperature), weight,
                                         loss, stats, stream))


def sv_distill_backward(R, V, student, dtype, indices, logprobs, k, temperature, weight, stats, grad_loss,
                        grad_loss_stride, grad, stream) -> int:
    return int(_lib().sv_distill_backward(R, V, student, dtype, indices, logprobs, k, float(temperature), weight, stats,
                                          grad_loss, grad_loss_stride, grad, stream))


def sv_distill_loss_grad(R, V, student, dtype, indices, logprobs, tail, k, temperature, weight, loss, grad,
                         stream) -> int:
    return int(_lib().sv_distill_loss_grad(R, V, student, dtype, indices, logprobs, tail, k, float(temperature), weight,
                                           loss, grad, stream))


# ------------------------------------------------------------ torch wrappers

def _need(name, t, dtype, shape, device):
    """t is None, or a contiguous CUDA tensor of this type and shape on `device`."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    _need_cuda(name, t, dtype)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the rows on {device}")


def _need_rows(name, t):
    _need_cuda(name, t)
    if t.dtype not in _TORCH_DTYPE:
        raise ValueError(f"unsupported {name} dtype {t.dtype}")


def _need_constants(names, *tensors):
    """Nobody asks for a gradient that goes through these (or None): none is formed."""
    forward, wanted = forward_ad._current_level >= 0, torch.is_grad_enabled()
    if not (forward or wanted):
        return
    for i, t in enumerate(tensors):
        if t is not None and ((t.requires_grad and wanted) or (forward and forward_ad.unpack_dual(t).tangent is not None)):
            raise ValueError(f"no gradient is formed for {names.split()[i]}: detach it")


class _Here:
    """The device is current already: nothing to enter or leave."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(device, stream):
    """A context for `stream` (or the device's current stream) with the rows'
    device current; what is allocated inside belongs to that stream.  The
    caller orders `stream` behind what makes the inputs."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the rows on {device}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device.index:
        return torch.cuda.device(device)
    return _HERE


def _read_on(stream, *tensors):
    """The caller may drop these (or None) as soon as the call returns: their
    memory is not handed out again before `stream` has come to this point."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _written(t):
    """The caller's tensor has been written: autograd graphs that saved it must notice."""
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


def _handle(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def adjust_logits(logits, *, draft=None, history=None, history_len=None, prompt_len=None, repetition=None,
                  frequency=None, presence=None, bias_tokens=None, bias_values=None, mask=None, mask_index=None,
                  gamma_b=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on the rows of a
    round, before the verify step (sv_adjust_logits).

    logits [B, gamma+1, V] (float32 / bfloat16 / float16): row i stands behind
    the sequence's history and its drafts d_0 .. d_{i-1}.  draft [B, gamma]
    int32; history [B, H] int32 with history_len [B] int32 and prompt_len [B]
    int32 (the first prompt_len tokens are the prompt: they count for the
    repetition penalty only); repetition, frequency and presence [B] float32;
    bias_tokens [B, N] int32 (negative: unused) with bias_values [B, N]
    float32; mask [M, ceil(V / 32)] int32 words, bit v % 32 of word v // 32 set
    where token v is allowed, with mask_index [B, gamma+1] int32 (negative: no
    mask), or without it one mask row per logits row (M = B * (gamma+1));
    gamma_b [B] int32: a ragged round, the rows behind a sequence's last are
    not touched.  All contiguous CUDA tensors on one device; what is None is
    off.  out: where to write (logits itself: in place); by default a new
    tensor, whose untouched rows hold zeros.  Returns out.  No gradient is
    formed: outside torch.no_grad() tensors that require one are refused.
    stream: where to run, by default the device's current stream; the caller
    orders it behind what makes the inputs, and may drop them after the call.
    """
    _need_constants("logits repetition frequency presence bias_values out", logits, repetition, frequency, presence,
                    bias_values, out)
    if logits.dim() != 3:
        raise ValueError(f"logits must be [B, gamma+1, V], got {tuple(logits.shape)}")
    B, G1, V = logits.shape
    dev = logits.device
    _need_rows("logits", logits)
    if G1 < 1:
        raise ValueError("logits has no rows: [B, gamma+1, V] with gamma >= 0")
    H = history.shape[1] if history is not None and history.dim() == 2 else 0
    NB = bias_tokens.shape[1] if bias_tokens is not None and bias_tokens.dim() == 2 else 0
    M = mask.shape[0] if mask is not None and mask.dim() == 2 else 0
    i32, f32 = torch.int32, torch.float32
    _need("draft", draft, i32, (B, G1 - 1), dev)
    _need("history", history, i32, (B, H), dev)
    _need("history_len", history_len, i32, (B,), dev)
    _need("prompt_len", prompt_len, i32, (B,), dev)
    _need("repetition", repetition, f32, (B,), dev)
    _need("frequency", frequency, f32, (B,), dev)
    _need("presence", presence, f32, (B,), dev)
    _need("bias_tokens", bias_tokens, i32, (B, NB), dev)
    _need("bias_values", bias_values, f32, (B, NB), dev)
    _need("mask", mask, i32, (M, (V + 31) // 32), dev)
    _need("mask_index", mask_index, i32, (B, G1), dev)
    _need("gamma_b", gamma_b, i32, (B,), dev)
    _need("out", out, logits.dtype, (B, G1, V), dev)
    if history is not None and history_len is None:
        raise ValueError("history needs history_len")
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values go together")
    if mask_index is not None and mask is None:
        raise ValueError("mask_index needs mask")
    if mask is not None and mask_index is None and M != B * G1:
        raise ValueError(f"without mask_index the mask has one row per logits row: {B * G1}, got {M}")
    # a table without rows has no address, and NULL would allow every token:
    # any other address says that the table is there (with M = 0 it is not read)
    table = _addr(mask_index) if mask_index is not None and M == 0 else _addr(mask)
    given = out
    with _on(dev, stream):
        _read_on(stream, logits, draft, history, history_len, prompt_len, repetition, frequency, presence, bias_tokens,
                 bias_values, mask, mask_index, gamma_b, out)
        if out is None:
            out = torch.zeros_like(logits) if gamma_b is not None else torch.empty_like(logits)
        st = sv_adjust_logits(B, G1 - 1, V, _addr(logits), _TORCH_DTYPE[logits.dtype], _addr(out), _addr(draft),
                              _addr(gamma_b), _addr(history), H, _addr(history_len), _addr(prompt_len),
                              _addr(repetition), _addr(frequency), _addr(presence), _addr(bias_tokens),
                              _addr(bias_values), NB, table, M, _addr(mask_index), _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_adjust_logits")
    if given is not None:
        _written(given)
    return out


def alloc_top_logits_workspace(rows: int, V: int, k: int, device=None) -> torch.Tensor:
    """A zero-filled device workspace large enough for top_logits on up to `rows` rows."""
    device = torch.device("cuda" if device is None else device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        n = sv_top_logits_workspace_bytes(rows, V, k)
        if n == 0:
            raise SvError(SV_ERR_INVALID_ARG, "sv_top_logits_workspace_bytes")
        # fewer rows than SMs are taken in slices and need more than many rows do
        sms = torch.cuda.get_device_properties(device).multi_processor_count
        n = max([n] + [sv_top_logits_workspace_bytes(r, V, k) for r in range(1, min(rows, sms + 1))])
    return torch.zeros(n, dtype=torch.uint8, device=device)


def top_logits(logits, k, temperature=1.0, *, workspace=None, stream=None, outputs=None):
    """The record of teacher rows that distillation reads (sv_top_logits).

    logits [..., V] (float32 / bfloat16 / float16, contiguous, CUDA).  Returns
    (indices [..., k] int32, logprobs [..., k] float32, tail [...] float32):
    each row's k best tokens by (logit descending, index ascending), their
    log-probabilities under softmax(logits / temperature), and the log of the
    mass outside them.  A row of fewer than k tokens above -inf is padded with
    index -1.  workspace: from alloc_top_logits_workspace, kept by the caller
    (one per concurrent call).  outputs: (indices, logprobs, tail) to write
    into.  No gradient is formed: outside torch.no_grad() tensors that require
    one are refused.  stream: as in adjust_logits.
    """
    _need_constants("logits indices logprobs tail", logits, *(outputs or ()))
    _need_rows("logits", logits)
    if logits.dim() < 1:
        raise ValueError("logits must be [..., V]")
    k = int(k)
    lead, V = tuple(logits.shape[:-1]), logits.shape[-1]
    R, dev = logits.numel() // max(V, 1), logits.device
    if workspace is not None:
        _need_cuda("workspace", workspace, torch.uint8)
        if workspace.device != dev:
            raise ValueError(f"workspace is on {workspace.device}, the rows on {dev}")
    if outputs is not None:
        for name, t, dt, shape in zip(("indices", "logprobs", "tail"), outputs, (torch.int32, torch.float32, torch.float32),
                                      (lead + (k,), lead + (k,), lead)):
            _need(name, t, dt, shape, dev)
    if not 1 <= k <= 1024:
        raise ValueError(f"k must be in 1..1024, got {k}")
    given = outputs
    with _on(dev, stream):
        _read_on(stream, logits, workspace, *(outputs or ()))
        if outputs is None:
            outputs = (torch.empty(lead + (k,), dtype=torch.int32, device=dev),
                       torch.empty(lead + (k,), dtype=torch.float32, device=dev),
                       torch.empty(lead, dtype=torch.float32, device=dev))
        if workspace is None:
            n = sv_top_logits_workspace_bytes(R, V, k)
            if n == 0:
                raise SvError(SV_ERR_INVALID_ARG, "sv_top_logits")
            workspace = torch.zeros(n, dtype=torch.uint8, device=dev)
        indices, logprobs, tail = outputs
        st = sv_top_logits(R, V, _addr(logits), _TORCH_DTYPE[logits.dtype], k, temperature, _addr(indices),
                           _addr(logprobs), _addr(tail), _addr(workspace), workspace.numel(), _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_top_logits")
    for t in given or ():
        _written(t)
    return indices, logprobs, tail


def _check_distill(student, indices, logprobs, tail, weight):
    _need_constants("logprobs tail weight", logprobs, tail, weight)
    _need_rows("student", student)
    if student.dim() < 1 or indices.dim() < 1:
        raise ValueError("student must be [..., V] and indices [..., k]")
    lead, dev = tuple(student.shape[:-1]), student.device
    k = indices.shape[-1]
    _need("indices", indices, torch.int32, lead + (k,), dev)
    _need("logprobs", logprobs, torch.float32, lead + (k,), dev)
    _need("tail", tail, torch.float32, lead, dev)
    _need("weight", weight, torch.float32, lead, dev)
    V = student.shape[-1]
    return student.numel() // max(V, 1), V, k


def _distill_forward(student, indices, logprobs, tail, temperature, weight, keep_stats):
    R, V, k = student.numel() // max(student.shape[-1], 1), student.shape[-1], indices.shape[-1]
    dev = student.device
    with _on(dev, None):
        loss = torch.empty(student.shape[:-1], dtype=torch.float32, device=dev)
        stats = torch.empty(R, SV_DISTILL_STAT_WORDS, dtype=torch.float32, device=dev) if keep_stats else None
        st = sv_distill_forward(R, V, _addr(student), _TORCH_DTYPE[student.dtype], _addr(indices), _addr(logprobs),
                                _addr(tail), k, temperature, _addr(weight), _addr(loss), _addr(stats), _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_distill_forward")
    return loss, stats


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, student, indices, logprobs, tail, temperature, weight):
        loss, stats = _distill_forward(student, indices, logprobs, tail, temperature, weight, ctx.needs_input_grad[0])
        ctx.save_for_backward(student, indices, logprobs, weight, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        student, indices, logprobs, weight, stats = ctx.saved_tensors
        if stats is None:
            return (None,) * 6
        R, V, k = student.numel() // student.shape[-1], student.shape[-1], indices.shape[-1]
        with _on(student.device, None):
            # a sum of the losses hands back one value, expanded
            stride = 0 if not any(grad_loss.stride()) else 1
            if stride:
                grad_loss = grad_loss.contiguous()
            grad = torch.empty_like(student)
            st = sv_distill_backward(R, V, _addr(student), _TORCH_DTYPE[student.dtype], _addr(indices),
                                     _addr(logprobs), k, ctx.temperature, _addr(weight), _addr(stats),
                                     _addr(grad_loss), stride, _addr(grad), _handle(student.device))
        if st != SV_OK:
            raise SvError(st, "sv_distill_backward")
        return grad, None, None, None, None, None


def distill_loss(student, indices, logprobs, tail=None, temperature=1.0, *, weight=None):
    """The loss of a student's rows against a teacher's record, differentiable
    in `student` (sv_distill_forward, sv_distill_backward).

    student [..., V] (float32 / bfloat16 / float16); indices [..., k] int32 and
    logprobs [..., k] float32 as top_logits returns them (indices outside the
    vocabulary are ignored); tail [...] float32 adds the outcome "any token not
    listed", None renormalises the teacher over the listed tokens; weight [...]
    float32 scales each row's loss, and a row of weight 0 may hold anything.  Returns
    the rows' losses [...] float32: weight * KL(teacher || student), both at
    `temperature`.  The gradient has the student's type.  Runs on the current
    stream.  A backward pass into a leaf's .grad that is captured into a CUDA
    graph wants no eager autograd graph of that leaf alive (PyTorch's engine
    ends the process otherwise); distill_loss_grad has no such condition.
    """
    _check_distill(student, indices, logprobs, tail, weight)
    temperature = float(temperature)
    # nobody asks for a gradient: no node is made (20 rows of 1024: 16 us
    # against 22).  A forward-mode one is refused by the node.
    if not (student.requires_grad and torch.is_grad_enabled()) and forward_ad._current_level < 0:
        return _distill_forward(student, indices, logprobs, tail, temperature, weight, False)[0]
    return _DistillLoss.apply(student, indices, logprobs, tail, temperature, weight)


def distill_loss_grad(student, indices, logprobs, tail=None, temperature=1.0, *, weight=None, out_grad=None,
                      stream=None):
    """Loss and gradient from one pass over the student's rows
    (sv_distill_loss_grad): returns (loss [...] float32, gradient of loss.sum()
    with respect to student).  out_grad: where the gradient goes (student
    itself: in place).  Arguments as distill_loss; nothing is recorded for
    autograd (student.backward(grad) hands the gradient on to what made the
    student), so it can be captured into a CUDA graph whatever autograd graphs
    are alive.  stream: as in adjust_logits.
    """
    _need_constants("out_grad", None if out_grad is student else out_grad)
    if forward_ad._current_level >= 0:
        with torch.no_grad():                # a tangent would be dropped; backward mode is documented above
            _need_constants("student", student)
    R, V, k = _check_distill(student, indices, logprobs, tail, weight)
    dev = student.device
    _need("out_grad", out_grad, student.dtype, student.shape, dev)
    with _on(dev, stream):
        _read_on(stream, student, indices, logprobs, tail, weight, out_grad)
        loss = torch.empty(student.shape[:-1], dtype=torch.float32, device=dev)
        grad = torch.empty_like(student, requires_grad=False) if out_grad is None else out_grad
        st = sv_distill_loss_grad(R, V, _addr(student), _TORCH_DTYPE[student.dtype], _addr(indices), _addr(logprobs),
                                  _addr(tail), k, temperature, _addr(weight), _addr(loss), _addr(grad), _handle(dev))
    if st != SV_OK:
        raise SvError(st, "sv_distill_loss_grad")
    if out_grad is not None:
        _written(out_grad)
    return loss, grad
