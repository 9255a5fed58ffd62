"""Logits operators for torch tensors: log probabilities of given tokens with entropy and top
alternatives, and distillation from a teacher's top logits, each with its gradient.

torch supplies device memory, the current stream and, where asked for, autograd; every step of
the arithmetic runs in the library's kernels (include/argreduce.h states the semantics). Logits
are float32, float16 or bfloat16 on the GPU, shape [..., cols]; the leading dimensions are rows,
and rows may be further apart than cols (a slice of a padded vocabulary, or of one position per
sequence, needs no copy).

``token_logprobs`` and ``distill_loss`` take part in autograd when the logits require a
gradient; they have no forward-mode derivative and refuse logits that carry a tangent.
``token_logprobs_grad``, ``distill_loss_grad`` and ``distill_step`` are the same gradients as plain
calls, which take no part in autograd and can also be captured into a graph.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad as _forward_ad

from . import binding as B

TOP_MAX = 64         # alternatives per row (ARGREDUCE_TOP_MAX)
TEACHER_MAX = 1024   # teacher entries per row (ARGREDUCE_TEACHER_MAX)
_ENTROPY_APART = 0x61706172  # ARGREDUCE_ENTROPY_APART

_F32, _I64 = torch.float32, torch.int64
_CODES = {torch.float32: B.F32, torch.float16: B.F16, torch.bfloat16: B.BF16}


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns. ``stats`` (float32 [4, rows]) is what token_logprobs_grad
    takes: the log probabilities and entropies once more, and two rows of its own. It reads none of
    the memory of logprob and entropy, which may be written over."""

    logprob: torch.Tensor
    entropy: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]
    top_tokens: Optional[torch.Tensor]
    stats: torch.Tensor


class DistillLoss(NamedTuple):
    """What distill_loss returns. ``stats`` (float32 [5, rows]) is what distill_loss_grad takes;
    the loss is its first row in the logits' leading shape."""

    loss: torch.Tensor
    stats: torch.Tensor


def _rows(logits):
    """(format code, rows, cols, row stride) of the logits, or a refusal."""
    if not logits.is_cuda:
        raise ValueError("the logits operators run on the GPU only; got a CPU tensor")
    code = _CODES.get(logits.dtype)
    if code is None:
        raise B.ArgreduceError(-2, f"logits of {logits.dtype}")
    shape, strides = logits.shape, logits.stride()
    if len(shape) == 0:
        raise ValueError("logits need at least one dimension")
    cols = shape[-1]
    if cols == 0:
        raise ValueError("logits need at least one column")
    if strides[-1] != 1 and cols != 1:
        raise ValueError("the last dimension of the logits must be contiguous")
    if len(shape) == 2:
        return code, shape[0], cols, strides[0]
    rows, stride = 1, None
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif rows > 0 and s != stride * rows:
            raise ValueError("the leading dimensions of the logits must be rows of one stride")
        rows *= n
    return code, rows, cols, cols if stride is None else stride


def _same(t, name: str, like, dtype, shape) -> None:
    """An input array: contiguous, of this type and shape, on the logits' device."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == like.get_device():
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}; got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}; got {tuple(t.shape)}")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}; got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _temperature(t) -> float:
    t = float(t)
    if not 2.0 ** -60 <= t <= 2.0 ** 60:
        raise ValueError(f"temperature must lie in [2^-60, 2^60]; got {t}")
    return t


_tuple = tuple.__new__
# The current device and its current stream's handle, as cheaply as torch gives them
# (torch.cuda.current_stream(...).cuda_stream takes 2 us, a tenth of a small call).
_device = torch._C._cuda_getDevice
_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(logits) -> bool:
    """Whether the logits are on another device than the current one. Plans and launches go by the
    current device: such a call is made again with the logits' device current."""
    return logits.device.index != _device()


def _scratch(need: int, what: str, given, device):
    """(address, bytes, owner) of scratch for a call."""
    if given is not None:
        B._check_buffer(given, "scratch", device)
    if need == 0:
        return 0, 0, None
    if need == B.SIZE_MAX:
        raise B.ArgreduceError(-3, what)
    if given is None or given.numel() * given.element_size() < need:
        given = torch.empty(need, dtype=torch.uint8, device=device)
    return given.data_ptr(), given.numel() * given.element_size(), given


class _Calls:
    """The library's logits entry points, looked up when the first of them is needed."""

    def __getattr__(self, name):
        f = B.entry_point("argreduce_" + name)
        setattr(self, name, f)
        return f


_call = _Calls()


def _failed(rc: int, what: str, rows, cols, stride):
    return B.ArgreduceError(rc, f"argreduce_{what}(rows={rows}, cols={cols}, row_stride={stride})")


def _refuse_captured_autograd(logits) -> None:
    """An autograd graph recorded while a HIP graph is captured can share gradient accumulators
    with an eager one, which ends the process when the engine joins their streams."""
    if logits.is_cuda and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("autograd through the logits operators cannot be captured: call "
                           "token_logprobs_grad, distill_loss_grad or distill_step in the capture")


def _refuse_tangent(logits) -> None:
    """In forward mode: a dual tensor need not require a gradient, and its tangent would be lost
    without a word."""
    if _forward_ad.unpack_dual(logits).tangent is not None:
        raise NotImplementedError("the logits operators have no forward-mode derivative")


# ---------------------------------------------------------------------------------------
# token_logprobs


def _logprobs(logits, tokens, temperature, entropy, top, scratch, apart=False):
    """(stats, top_logprobs, top_tokens, entropy): with `apart` the entropy in memory that the
    gradient does not read, else None."""
    code, rows, cols, stride = _rows(logits)
    lead = (rows,) if logits.dim() == 2 else logits.shape[:-1]
    _same(tokens, "tokens", logits, _I64, lead)
    temperature = _temperature(temperature)
    if not 0 <= top <= TOP_MAX:
        raise ValueError(f"top must lie in 0..{TOP_MAX}; got {top}")
    device = logits.device
    if device.index != _device():
        with torch.cuda.device(device):
            return _logprobs(logits, tokens, temperature, entropy, top, scratch, apart)
    ent = lp = tok = None
    lp_ptr = tok_ptr = sptr = sbytes = 0
    if entropy and apart:
        buf = torch.empty(5, rows, dtype=_F32, device=device)
        stats, ent, entropy = buf.as_strided((4, rows), (rows, 1)), buf[4], _ENTROPY_APART
    else:
        stats = torch.empty(4, rows, dtype=_F32, device=device)
    if top:
        lp = torch.empty(*lead, top, dtype=_F32, device=device)
        tok = torch.empty(*lead, top, dtype=_I64, device=device)
        lp_ptr, tok_ptr = lp.data_ptr(), tok.data_ptr()
    need = _call.logprobs_scratch_bytes(rows, cols, code)
    if need or scratch is not None:
        sptr, sbytes, scratch = _scratch(need, "argreduce_logprobs", scratch, device)
    rc = _call.logprobs(logits.data_ptr(), code, rows, cols, stride, tokens.data_ptr(), temperature,
                        entropy, top, stats.data_ptr(), lp_ptr, tok_ptr, sptr, sbytes,
                        _stream(device.index))
    if rc:
        raise _failed(rc, "logprobs", rows, cols, stride)
    return stats, lp, tok, ent


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, entropy, top, scratch):
        stats, lp, tok, _ = _logprobs(logits, tokens, temperature, entropy, top, scratch)
        ctx.save_for_backward(logits, tokens, stats)
        ctx.temperature, ctx.entropy = temperature, entropy
        # outputs of their own: a view of stats would carry its gradient to the other rows
        lead = logits.shape[:-1]
        logprob = stats[0].view(lead).clone()
        ent = stats[1].view(lead).clone() if entropy else None
        ctx.mark_non_differentiable(*[t for t in (lp, tok, stats) if t is not None])
        ctx.set_materialize_grads(False)
        return logprob, ent, lp, tok, stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logprob, g_entropy, *_):
        logits, tokens, stats = ctx.saved_tensors
        _refuse_captured_autograd(logits)
        if g_logprob is None and g_entropy is None:
            return (None,) * 6
        lead = logits.shape[:-1]
        if g_logprob is None:
            g_logprob = torch.zeros(lead, dtype=torch.float32, device=logits.device)
        grad = token_logprobs_grad(logits, tokens, stats, g_logprob.contiguous(),
                                   None if g_entropy is None else g_entropy.contiguous(),
                                   temperature=ctx.temperature)
        return grad, None, None, None, None, None


def token_logprobs(logits, tokens, *, temperature: float = 1.0, entropy: bool = False, top: int = 0,
                   scratch=None) -> TokenLogprobs:
    """Log probability of one given token per row, ``ln softmax(logits / temperature)[token]``.

    logits [..., cols] (float32, float16, bfloat16); tokens int64, the logits' leading shape. A
    negative token leaves its row out (0, no gradient). entropy: also the entropy of each row's
    distribution. top: also the ``top`` most likely tokens and their log probabilities, most
    likely first, ties to the lower token; rows with fewer unmasked logits end in token -1.

    Differentiable in logprob and entropy (float32) when the logits require a gradient."""
    if _forward_ad._current_level >= 0:
        _refuse_tangent(logits)
    if logits.requires_grad and torch.is_grad_enabled():
        _refuse_captured_autograd(logits)
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, temperature, bool(entropy), top,
                                                   scratch))
    stats, lp, tok, ent = _logprobs(logits, tokens, temperature, bool(entropy), top, scratch, True)
    if logits.dim() == 2:  # (a named tuple's own constructor takes twice the time)
        return _tuple(TokenLogprobs, (stats[0], ent, lp, tok, stats))
    lead = logits.shape[:-1]
    return TokenLogprobs(stats[0].view(lead), None if ent is None else ent.view(lead), lp, tok, stats)


def _new_grad(logits):
    return torch.empty(*logits.shape, dtype=logits.dtype, device=logits.device)


def _check_grad(logits, rows, cols, stride, out, **others):
    """The caller's gradient tensor, which shares no memory with the logits or the other arguments,
    all contiguous (the kernels read them while they write it)."""
    B._check_buffer(out, "out", logits.device, logits.dtype, logits.numel())
    if out.shape != logits.shape:
        raise ValueError(f"out must have shape {tuple(logits.shape)}; got {tuple(out.shape)}")
    size, x, g = logits.element_size(), logits.data_ptr(), out.data_ptr()
    if rows > 0 and g < x + ((rows - 1) * stride + cols) * size and x < g + rows * cols * size:
        raise ValueError("out must not overlap the logits")
    for name, t in others.items():
        if t is not None and g < t.data_ptr() + t.numel() * t.element_size() and \
                t.data_ptr() < g + rows * cols * size:
            raise ValueError(f"out must not overlap {name}")
    return out


def token_logprobs_grad(logits, tokens, stats, grad_logprob, grad_entropy=None, *,
                        temperature: float = 1.0, out=None):
    """Gradient of ``(grad_logprob * logprob + grad_entropy * entropy).sum()`` with respect to the
    logits, in their type and shape (contiguous; ``out``, if given, is such a tensor, apart from
    every argument's memory). stats is that of the forward call on the same logits, tokens and temperature, made with
    ``entropy=True`` if grad_entropy is given; grad_logprob and grad_entropy are float32 in the
    logits' leading shape."""
    code, rows, cols, stride = _rows(logits)
    lead = logits.shape[:-1]
    _same(tokens, "tokens", logits, torch.int64, lead)
    _same(stats, "stats", logits, torch.float32, (4, rows))
    _same(grad_logprob, "grad_logprob", logits, torch.float32, lead)
    if grad_entropy is not None:
        _same(grad_entropy, "grad_entropy", logits, torch.float32, lead)
    temperature = _temperature(temperature)
    out = _new_grad(logits) if out is None else _check_grad(
        logits, rows, cols, stride, out, tokens=tokens, stats=stats, grad_logprob=grad_logprob,
        grad_entropy=grad_entropy)
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return token_logprobs_grad(logits, tokens, stats, grad_logprob, grad_entropy,
                                       temperature=temperature, out=out)
    rc = _call.logprobs_grad(
        logits.data_ptr(), code, rows, cols, stride, tokens.data_ptr(), temperature,
        stats.data_ptr(), grad_logprob.data_ptr(),
        0 if grad_entropy is None else grad_entropy.data_ptr(), out.data_ptr(),
        _stream(logits.device.index))
    if rc:
        raise _failed(rc, "logprobs_grad", rows, cols, stride)
    return out


# ---------------------------------------------------------------------------------------
# distill_loss


def _teacher(logits, teacher_tokens, teacher_logits) -> int:
    k = teacher_tokens.shape[-1] if teacher_tokens.dim() else 0
    if not 1 <= k <= TEACHER_MAX:
        raise ValueError(f"a row must have 1..{TEACHER_MAX} teacher entries; got {k}")
    shape = logits.shape[:-1] + (k,)
    _same(teacher_tokens, "teacher_tokens", logits, torch.int64, shape)
    _same(teacher_logits, "teacher_logits", logits, torch.float32, shape)
    return k


def _distill(logits, teacher_tokens, teacher_logits, temperature, scratch):
    code, rows, cols, stride = _rows(logits)
    k = _teacher(logits, teacher_tokens, teacher_logits)
    temperature = _temperature(temperature)
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return _distill(logits, teacher_tokens, teacher_logits, temperature, scratch)
    device = logits.device
    stats = torch.empty(5, rows, dtype=torch.float32, device=device)
    need = _call.distill_scratch_bytes(rows, cols, code)
    sptr, sbytes, scratch = _scratch(need, "argreduce_distill", scratch, device)
    rc = _call.distill(logits.data_ptr(), code, rows, cols, stride, k, teacher_tokens.data_ptr(),
                       teacher_logits.data_ptr(), temperature, stats.data_ptr(), sptr, sbytes,
                       _stream(device.index))
    if rc:
        raise _failed(rc, "distill", rows, cols, stride)
    return stats


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_tokens, teacher_logits, temperature, scratch):
        stats = _distill(logits, teacher_tokens, teacher_logits, temperature, scratch)
        ctx.save_for_backward(logits, teacher_tokens, teacher_logits, stats)
        ctx.temperature = temperature
        ctx.mark_non_differentiable(stats)
        ctx.set_materialize_grads(False)
        return stats[0].view(logits.shape[:-1]).clone(), stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss, _):
        if g_loss is None:
            return (None,) * 5
        logits, teacher_tokens, teacher_logits, stats = ctx.saved_tensors
        _refuse_captured_autograd(logits)
        grad = distill_loss_grad(logits, teacher_tokens, teacher_logits, stats, g_loss.contiguous(),
                                 temperature=ctx.temperature)
        return grad, None, None, None, None


def distill_loss(logits, teacher_tokens, teacher_logits, *, temperature: float = 1.0,
                 scratch=None) -> DistillLoss:
    """Divergence KL(q || p) per row of the student's distribution p = softmax(logits /
    temperature) from the teacher's q, the softmax at the same temperature over its k entries.

    teacher_tokens [..., k] int64 (negative: absent) and teacher_logits [..., k] float32 (logits or
    log probabilities; -inf: no weight), such as token_logprobs(teacher, ..., top=k) returns. A row
    without an entry of weight has loss 0. The loss is not multiplied by temperature ** 2.

    Differentiable in the loss when the logits require a gradient; the teacher is a constant."""
    if _forward_ad._current_level >= 0:
        _refuse_tangent(logits)
    if logits.requires_grad and torch.is_grad_enabled():
        _refuse_captured_autograd(logits)
        return DistillLoss(*_DistillLoss.apply(logits, teacher_tokens, teacher_logits, temperature,
                                               scratch))
    stats = _distill(logits, teacher_tokens, teacher_logits, temperature, scratch)
    return DistillLoss(stats[0] if logits.dim() == 2 else stats[0].view(logits.shape[:-1]), stats)


def distill_loss_grad(logits, teacher_tokens, teacher_logits, stats, grad_loss, *,
                      temperature: float = 1.0, out=None):
    """Gradient of ``(grad_loss * loss).sum()`` with respect to the logits, in their type and shape
    (contiguous; ``out``, if given, is such a tensor, apart from every argument's memory). stats is
    that of the forward call on the same inputs; grad_loss is float32 in the logits' leading shape."""
    code, rows, cols, stride = _rows(logits)
    k = _teacher(logits, teacher_tokens, teacher_logits)
    _same(stats, "stats", logits, torch.float32, (5, rows))
    _same(grad_loss, "grad_loss", logits, torch.float32, logits.shape[:-1])
    temperature = _temperature(temperature)
    out = _new_grad(logits) if out is None else _check_grad(
        logits, rows, cols, stride, out, teacher_tokens=teacher_tokens, teacher_logits=teacher_logits,
        stats=stats, grad_loss=grad_loss)
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return distill_loss_grad(logits, teacher_tokens, teacher_logits, stats, grad_loss,
                                     temperature=temperature, out=out)
    rc = _call.distill_grad(
        logits.data_ptr(), code, rows, cols, stride, k, teacher_tokens.data_ptr(),
        teacher_logits.data_ptr(), temperature, stats.data_ptr(), grad_loss.data_ptr(),
        out.data_ptr(), _stream(logits.device.index))
    if rc:
        raise _failed(rc, "distill_grad", rows, cols, stride)
    return out


def distill_step(logits, teacher_tokens, teacher_logits, weights, *, temperature: float = 1.0,
                 out=None, scratch=None):
    """(loss, grad): the loss of every row, and the gradient of ``(weights * loss).sum()`` with
    respect to the logits, in one call that reads the logits from memory once. For a training step
    whose row weights (float32, the logits' leading shape) do not depend on the loss. out: as for
    distill_loss_grad."""
    code, rows, cols, stride = _rows(logits)
    k = _teacher(logits, teacher_tokens, teacher_logits)
    _same(weights, "weights", logits, torch.float32, logits.shape[:-1])
    temperature = _temperature(temperature)
    out = _new_grad(logits) if out is None else _check_grad(
        logits, rows, cols, stride, out, teacher_tokens=teacher_tokens, teacher_logits=teacher_logits,
        weights=weights, scratch=scratch)
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return distill_step(logits, teacher_tokens, teacher_logits, weights,
                                temperature=temperature, out=out, scratch=scratch)
    device = logits.device
    stats = torch.empty(5, rows, dtype=torch.float32, device=device)
    need = _call.distill_scratch_bytes(rows, cols, code)
    sptr, sbytes, scratch = _scratch(need, "argreduce_distill_step", scratch, device)
    rc = _call.distill_step(
        logits.data_ptr(), code, rows, cols, stride, k, teacher_tokens.data_ptr(),
        teacher_logits.data_ptr(), temperature, weights.data_ptr(), stats.data_ptr(),
        out.data_ptr(), sptr, sbytes, _stream(device.index))
    if rc:
        raise _failed(rc, "distill_step", rows, cols, stride)
    return (stats[0] if logits.dim() == 2 else stats[0].view(logits.shape[:-1])), out
