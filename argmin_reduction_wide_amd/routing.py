"""Expert routing for torch tensors: the choice of experts per token from a router's logits, with weights,
per-expert counts and two losses that train the router, and the gradient.

torch supplies device memory, the current stream and, where asked for, autograd; the arithmetic runs in
the library's kernels (include/argreduce.h states the semantics). ``route_experts`` takes part in
autograd when the logits require a gradient; ``route_experts_grad`` is the same gradient as a plain call,
which can also be captured into a graph.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd import forward_ad as _forward_ad

from . import binding as B
from .beams import _contiguous, _results
from .logits import (_F32, _I64, _Calls, _check_grad, _device, _elsewhere, _new_grad, _refuse_tangent, _rows, _same,
                     _stream, _tuple)

EXPERTS_MAX = 1024   # experts of a router (ARGREDUCE_EXPERTS_MAX)
ROUTE_TOP_MAX = 64   # experts chosen per token (ARGREDUCE_ROUTE_TOP_MAX)

_call = _Calls()


class RouteExperts(NamedTuple):
    """What route_experts returns, for logits [..., tokens, experts]: weights (float32) and experts
    (int64), [..., tokens, top]; counts (int64 [..., experts]), how many tokens chose each expert; tokens
    (int64 [...]), how many there are; the losses balance and z (float32 [...]). ``totals`` is what
    route_experts_grad takes; without autograd counts, tokens, balance and z lie in its memory, and an in-place write
    to one of the five is one to all of them for autograd."""

    weights: torch.Tensor
    experts: torch.Tensor
    counts: torch.Tensor
    tokens: torch.Tensor
    balance: torch.Tensor
    z: torch.Tensor
    totals: torch.Tensor


def _router(logits, top):
    """(format code, groups, tokens, experts, row stride, leading shape) of the logits, or a refusal."""
    code, rows, experts, stride = _rows(logits)
    if logits.dim() < 2:
        raise ValueError("logits need dimensions for tokens and experts")
    if experts > EXPERTS_MAX:
        raise ValueError(f"a router must have 1..{EXPERTS_MAX} experts; got {experts}")
    if not 1 <= top <= min(experts, ROUTE_TOP_MAX):
        raise ValueError(f"top must lie in 1..{min(experts, ROUTE_TOP_MAX)}; got {top}")
    shape = tuple(logits.shape)  # (a slice or sum of torch's own sizes takes five times as long)
    lead, tokens = shape[:-2], shape[-2]
    groups = 1
    for n in lead:
        groups *= n
    return code, groups, tokens, experts, stride, lead


def _refuse_captured_autograd(logits) -> None:
    """An autograd graph recorded while a HIP graph is captured can share gradient accumulators
    with an eager one, which ends the process when the engine joins their streams."""
    if logits.is_cuda and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("autograd through route_experts cannot be captured: call route_experts_grad in the "
                           "capture")


def _route(logits, top, live, renormalize, scratch, apart=False) -> RouteExperts:
    """apart: the weights in memory of their own (a write to them by the caller would count as one to what
    the backward pass saves)."""
    code, groups, tokens, experts, stride, lead = _router(logits, top)
    if live is not None:
        _same(live, "live", logits, torch.bool, lead + (tokens,))
    device = logits.device
    if device.index != _device():
        with torch.cuda.device(device):
            return _route(logits, top, live, renormalize, scratch, apart)
    shape = lead + (tokens, top)
    # totals (counts, tokens: 8 bytes each, balance and z: 4 each, one after another), experts (8) and weights (4)
    per, n = groups * (experts + 2), groups * tokens * top
    need = _call.route_scratch_bytes(groups, tokens, experts, code)
    out, sptr, sbytes, scratch = _results(per + n + (0 if apart else (n + 1) // 2), need, "argreduce_route", scratch,
                                          device)
    strides, floats = _contiguous(shape), out.view(_F32)
    totals = out.as_strided((per,), (1,))
    # (.data: to autograd tensors of their own, so that a write to one is no write to another)
    chosen = out.as_strided(shape, strides, per).data
    weights = torch.empty(shape, dtype=_F32, device=device) if apart else \
        floats.as_strided(shape, strides, 2 * (per + n)).data
    rc = _call.route(logits.data_ptr(), code, groups, tokens, experts, stride,
                     0 if live is None else live.data_ptr(), top, bool(renormalize), weights.data_ptr(),
                     chosen.data_ptr(), totals.data_ptr(), sptr, sbytes, _stream(device.index))
    if rc:
        raise B.ArgreduceError(rc, f"argreduce_route(groups={groups}, tokens={tokens}, experts={experts}, "
                                   f"row_stride={stride}, top={top})")
    n = groups * experts
    each, columns = _contiguous(lead), lead + (experts,)
    return _tuple(RouteExperts, (
        weights, chosen, out.as_strided(columns, _contiguous(columns)),
        out.as_strided(lead, each, n), floats.as_strided(lead, each, 2 * (n + groups)),
        floats.as_strided(lead, each, 2 * n + 3 * groups), totals))


class _RouteExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top, live, renormalize, scratch):
        r = _route(logits, top, live, renormalize, scratch, True)
        ctx.save_for_backward(logits, r.experts, r.totals)
        ctx.renormalize = renormalize
        # outputs of their own, which may be written over, and no views of what the backward pass reads
        out = (r.weights, r.experts.clone(), r.counts.clone(), r.tokens.clone(), r.balance.clone(), r.z.clone(),
               r.totals)
        ctx.mark_non_differentiable(out[1], out[2], out[3], out[6])
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_weights, _e, _c, _t, g_balance, g_z, _totals):
        logits, experts, totals = ctx.saved_tensors
        _refuse_captured_autograd(logits)
        if g_weights is None and g_balance is None and g_z is None:
            return (None,) * 5
        plain = [None if g is None else g.contiguous() for g in (g_weights, g_balance, g_z)]
        grad = _grad(logits, experts, totals, *plain, None, ctx.renormalize, None)
        return grad, None, None, None, None


def route_experts(logits, top: int, *, live=None, renormalize: bool = False, scratch=None) -> RouteExperts:
    """The ``top`` experts of every token with weights, and what trains the router.

    logits [..., tokens, experts] (float32, float16, bfloat16; rows may lie further apart than experts;
    -inf: not available); every leading index is a group of tokens with counts and losses of its own.
    live: bool [..., tokens], False leaves a token out (experts -1, weights 0, no part in the rest).
    With p = softmax(logits): experts are the largest p, largest first, ties to the lower expert; weights
    their p, with renormalize divided by their sum; balance ``experts / (top * n**2) * sum_e counts_e
    sum_t p_te`` over the n tokens of a group (1 when evenly spread); z the mean square of
    ``logsumexp(logits)``.

    Differentiable in weights, balance and z when the logits require a gradient."""
    if _forward_ad._current_level >= 0:
        _refuse_tangent(logits)
    if logits.requires_grad and torch.is_grad_enabled():
        _refuse_captured_autograd(logits)
        return RouteExperts(*_RouteExperts.apply(logits, top, live, bool(renormalize), scratch))
    return _route(logits, top, live, bool(renormalize), scratch)


def _grad(logits, experts, totals, grad_weights, grad_balance, grad_z, live, renormalize, out):
    top = experts.shape[-1] if experts.dim() else 0
    code, groups, tokens, cols, stride, lead = _router(logits, top)
    shape = lead + (tokens, top)
    _same(experts, "experts", logits, _I64, shape)
    _same(totals, "totals", logits, _I64, (groups * (cols + 2),))
    if live is not None:
        _same(live, "live", logits, torch.bool, lead + (tokens,))
    if grad_weights is not None:
        _same(grad_weights, "grad_weights", logits, _F32, shape)
    if grad_balance is not None:
        _same(grad_balance, "grad_balance", logits, _F32, lead)
    if grad_z is not None:
        _same(grad_z, "grad_z", logits, _F32, lead)
    out = _new_grad(logits) if out is None else _check_grad(
        logits, groups * tokens, cols, stride, out, experts=experts, totals=totals, grad_weights=grad_weights,
        grad_balance=grad_balance, grad_z=grad_z, live=live)
    if _elsewhere(logits):
        with torch.cuda.device(logits.device):
            return _grad(logits, experts, totals, grad_weights, grad_balance, grad_z, live, renormalize, out)
    at = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    rc = _call.route_grad(logits.data_ptr(), code, groups, tokens, cols, stride, top, bool(renormalize),
                          experts.data_ptr(), totals.data_ptr(), at(grad_weights), at(grad_balance), at(grad_z),
                          out.data_ptr(), _stream(logits.device.index))
    if rc:
        raise B.ArgreduceError(rc, f"argreduce_route_grad(groups={groups}, tokens={tokens}, experts={cols}, "
                                   f"row_stride={stride}, top={top})")
    return out


def route_experts_grad(logits, routed: RouteExperts, grad_weights=None, grad_balance=None, grad_z=None, *, live=None,
                       renormalize: bool = False, out=None):
    """Gradient of ``(grad_weights * weights).sum() + (grad_balance * balance + grad_z * z).sum()`` with
    respect to the logits, in their type and shape (contiguous; ``out``, if given, is such a tensor, apart
    from every argument's memory). routed is what route_experts returned for the same logits, live and
    renormalize (its experts, counts and tokens are read; tokens left out are those without an expert);
    grad_weights float32 [..., tokens, top], grad_balance and grad_z float32 [...], each or None."""
    return _grad(logits, routed.experts, routed.totals, grad_weights, grad_balance, grad_z, live, renormalize, out)
