"""Beam search for torch tensors: the step that chooses a search's continuations from the model's
logits, and the reordering of the states (key-value caches, token histories) that the model keeps for
every beam.

torch supplies device memory and the current stream; the arithmetic runs in the library's kernels
(include/argreduce.h states the semantics). Both calls can be captured into a graph.
"""
from __future__ import annotations

import ctypes
from bisect import bisect_left
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad as _forward_ad

from . import binding as B
from .logits import (_F32, _I64, _Calls, _device, _elsewhere, _refuse_tangent, _rows, _same, _scratch, _stream,
                     _temperature, _tuple)

BEAM_MAX = 64  # beams of a group, and candidates kept (ARGREDUCE_BEAM_MAX)

_call = _Calls()


class BeamStep(NamedTuple):
    """What beam_step returns, each [..., width]: scores (float32), the beam each value comes from and
    its token (int64), and, with an end_token, whether it is finished (bool). Where a group has fewer
    values the rest is -inf, -1, -1 and False."""

    scores: torch.Tensor
    parents: torch.Tensor
    tokens: torch.Tensor
    ended: Optional[torch.Tensor]


def beam_step(logits, scores, width: Optional[int] = None, *, temperature: float = 1.0, ended=None,
              end_token: Optional[int] = None, scratch=None) -> BeamStep:
    """The ``width`` best continuations of every group of beams (as many as there are beams, if not
    given): the largest ``scores[b] + ln softmax(logits[b] / temperature)[v]`` over beams b and tokens
    v, largest first, equal values by beam and then by token.

    logits [..., beams, cols] (float32, float16, bfloat16; rows may lie further apart than cols; -inf:
    not allowed), scores float32 [..., beams]: the beams' sums of log probabilities (-inf: no such
    beam, as all but the first are at a search's start). ended: bool [..., beams], beams that are
    finished; such a beam offers its own score once, with the token ``end_token``, and its logits are
    not read. With an end_token the result says which of the chosen are finished.

    Takes no part in autograd; logits or scores that require a gradient are refused unless gradients
    are off."""
    if _forward_ad._current_level >= 0:
        _refuse_tangent(logits)
        _refuse_tangent(scores)
    if torch.is_grad_enabled() and (logits.requires_grad or scores.requires_grad):
        raise RuntimeError("beam_step has no gradient: call it under torch.no_grad() or on detached tensors")
    code, rows, cols, stride = _rows(logits)
    if logits.dim() < 2:
        raise ValueError("logits need dimensions for beams and columns")
    lead = tuple(logits.shape)[:-1]  # (a slice or sum of torch's own sizes takes five times as long)
    beams = lead[-1]
    if not 1 <= beams <= BEAM_MAX:
        raise ValueError(f"a group must have 1..{BEAM_MAX} beams; got {beams}")
    width = beams if width is None else width
    if not 1 <= width <= BEAM_MAX:
        raise ValueError(f"width must lie in 1..{BEAM_MAX}; got {width}")
    _same(scores, "scores", logits, _F32, lead)
    ended_ptr = 0
    if ended is not None:
        _same(ended, "ended", logits, torch.bool, lead)
        if end_token is None:
            raise ValueError("beams that are finished need an end_token")
        ended_ptr = ended.data_ptr()
    end = -1 if end_token is None else end_token
    if end_token is not None and not 0 <= end_token < cols:
        raise ValueError(f"end_token must lie in 0..{cols - 1}; got {end_token}")
    temperature = _temperature(temperature)
    device = logits.device
    if device.index != _device():
        with torch.cuda.device(device):
            return beam_step(logits, scores, width, temperature=temperature, ended=ended, end_token=end_token,
                             scratch=scratch)
    groups = rows // beams
    n = groups * width
    # parents, tokens (8 bytes each), scores (4) and ended (1), one after another
    need = _call.beam_scratch_bytes(groups, beams, cols, code, width)
    out, sptr, sbytes, scratch = _results(2 * n + (5 * n + 7) // 8, need, "argreduce_beam_step", scratch, device)
    rc = _call.beam_step(logits.data_ptr(), code, groups, beams, cols, stride, scores.data_ptr(), ended_ptr,
                         end, temperature, width, out.data_ptr(), sptr, sbytes, _stream(device.index))
    if rc:
        raise B.ArgreduceError(rc, f"argreduce_beam_step(groups={groups}, beams={beams}, cols={cols}, "
                                   f"row_stride={stride}, width={width})")
    shape = lead[:-1] + (width,)
    strides = _contiguous(shape)
    # (.data: to autograd tensors of their own, so that a write to one is no write to another)
    parents = out.as_strided(shape, strides)
    tokens = out.as_strided(shape, strides, n).data
    values = out.view(_F32).as_strided(shape, strides, 4 * n).data
    flags = None
    if end_token is not None:
        flags = out.view(torch.bool).as_strided(shape, strides, 20 * n).data
    return _tuple(BeamStep, (values, parents, tokens, flags))


def _results(words: int, need: int, what: str, scratch, device):
    """(words of 8 bytes, scratch's address, bytes and owner) for a call. Scratch of at most 32 KiB or an eighth of
    the results lies behind them (an allocation takes the host 1.5 us); results would keep more of it alive."""
    if scratch is None and 0 < need <= max(32768, words):
        more = (need + 7) // 8
        out = torch.empty(words + more, dtype=_I64, device=device)
        return out, out.data_ptr() + 8 * words, 8 * more, out
    out = torch.empty(words, dtype=_I64, device=device)
    if need or scratch is not None:
        return out, *_scratch(need, what, scratch, device)
    return out, 0, 0, None


def _contiguous(shape):
    """Strides of a contiguous tensor."""
    d = len(shape)
    if d == 3:
        return (shape[1] * shape[2], shape[2], 1)
    if d == 2:
        return (shape[1], 1)
    if d == 1:
        return (1,)
    strides, n = [], 1
    for s in reversed(shape):
        strides.append(n)
        n *= s
    return tuple(reversed(strides))


def _state(t, groups: int, beams: int, dim) -> B.argreduce_state_t:
    """One state tensor as the library addresses it, or a refusal."""
    size = t.element_size()
    rest = list(zip(t.shape[2:], t.stride()[2:]))
    positions, position_stride = (1, 0)
    before, after = [], rest
    if dim is not None:
        before, (positions, position_stride), after = rest[:dim - 2], rest[dim - 2], rest[dim - 1:]

    def merged(dims, run):
        """Sizes and strides of `dims` as one dimension: (elements, stride of the last)."""
        n, stride = 1, run
        for k, (size_k, stride_k) in enumerate(reversed([d for d in dims if d[0] != 1])):
            if k == 0:
                stride = stride_k
            elif stride_k != stride * n:
                return None
            n *= size_k
        return n, stride

    inner = merged(after, 1)
    outer = merged(before, 1)
    if inner is None or inner[1] != 1:
        raise ValueError("a state's dimensions after the positions (all, without them) must be contiguous")
    if outer is None:
        raise ValueError("a state's dimensions between beams and positions must be rows of one stride")
    return B.argreduce_state_t(t.data_ptr(), t.stride(0) * size, t.stride(1) * size, outer[0],
                               outer[1] * size, positions, position_stride * size, inner[0] * size)


def _span(t):
    """[first, last) byte that a tensor's elements lie in."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


class BeamStates:
    """The states of a search's beams, reordered together in one launch.

    states: a tensor or several, of any element types, each [groups, beams, ...], on one GPU. dim: the
    dimension (of every tensor, 2 or above or counted from the end) that holds the positions of a cache, or
    None if there are none. The dimensions after the positions must be contiguous, and those between
    beams and positions rows of one stride: [groups, beams, heads, positions, size] and [groups, beams,
    positions, heads, size] are both fine, and so are slices of longer caches.

    The tensors are held, not copied: they must keep their memory (no ``resize_`` or ``set_``), and may
    share no memory with each other. Autograd does not see the move: a state that a graph has saved must
    not be reordered before that graph's backward pass.

    Made once, outside of a graph capture: it checks the tensors on the host and copies a table of them to the
    GPU, and waits for that (21 us for one tensor, 77 for 16, 201 for 48). A program whose caches are new tensors
    in every step pays it in every step. A graph that captured a reordering reads this object's memory, which
    must live as long as the graph."""

    def __init__(self, states, *, dim: Optional[int] = None):
        states = [states] if isinstance(states, torch.Tensor) else list(states)
        if not states:
            raise ValueError("at least one state is needed")
        first = states[0]
        for t in states:
            if not t.is_cuda or t.device != first.device:
                raise ValueError("states must lie on one GPU")
            if t.dim() < 2 or t.shape[:2] != first.shape[:2]:
                raise ValueError("states must have the same shape [groups, beams, ...] in front")
            if t.requires_grad:
                raise ValueError("states are changed in place and cannot require a gradient")
        self.groups, self.beams = first.shape[:2]
        if not 1 <= self.beams <= BEAM_MAX:
            raise ValueError(f"a group must have 1..{BEAM_MAX} beams; got {self.beams}")
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("BeamStates cannot be made in a capture: make it before")
        self.states, self.device = states, first.device
        used = [t for t in states if t.numel()]
        spans = sorted(_span(t) for t in used)
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("states must not overlap (pass interleaved ones as one tensor)")
        self._starts, self._ends = [a[0] for a in spans], [a[1] for a in spans]
        table = (B.argreduce_state_t * max(1, len(used)))()
        for i, t in enumerate(used):
            d = dim
            if d is not None:
                d = d + t.dim() if d < 0 else d
                if not 2 <= d < t.dim():
                    raise ValueError(f"dim must name a dimension after the beams; got {dim} of {t.dim()}")
            table[i] = _state(t, self.groups, self.beams, d)
        self._plan = B.argreduce_reorder_plan(table, self.groups, self.beams) if used else None
        if used:
            host = torch.frombuffer(bytearray(bytes(table)), dtype=torch.int64)
            self._table = host.to(self.device)
            self._streams = {_stream(self.device.index)}  # those the table's memory is known to be used on

    def reorder(self, parents, *, first=None, last=None) -> None:
        """Every beam becomes a copy of its parent as that was before the call: ``state[g, b] =
        state[g, parents[g, b]]``, in place. parents int64 of groups * beams elements, [..., beams]
        (beam_step's, with as many candidates as beams); one outside 0..beams - 1 leaves its beam as it is.

        first, last: only positions first <= t < last move, each None (all), an int or an int64 tensor
        [groups] on the GPU. Positions that all of a group's beams share (a prompt) or that are not filled
        yet need no move. Beams that stay cost nothing."""
        groups, beams = self.groups, self.beams
        shape = parents.shape
        if parents.dtype is not _I64 or len(shape) == 0 or shape[-1] != beams or parents.numel() != groups * beams:
            raise ValueError(f"parents must be int64 [..., {beams}] of {groups * beams} elements; got "
                             f"{parents.dtype} {tuple(shape)}")
        if parents.device != self.device or not parents.is_contiguous():
            raise ValueError(f"parents must be contiguous and on {self.device}")
        if self._plan is None:
            return
        self._apart(parents, "parents")
        first_ptr, first_value = self._positions(first, "first", 0)
        last_ptr, last_value = self._positions(last, "last", 1 << 62)
        if self.device.index != _device():
            with torch.cuda.device(self.device):
                return self.reorder(parents, first=first, last=last)
        stream = _stream(self.device.index)
        if stream not in self._streams:
            self._table.record_stream(torch.cuda.current_stream())
            self._streams.add(stream)
        rc = _call.reorder(ctypes.addressof(self._plan), self._table.data_ptr(), parents.data_ptr(), first_ptr,
                           last_ptr, first_value, last_value, stream)
        if rc:
            raise B.ArgreduceError(rc, f"argreduce_reorder(tensors={len(self.states)}, groups={groups}, beams={beams})")

    def _apart(self, t, name: str) -> None:
        """What the kernel reads while it moves the states lies in none of them."""
        start = t.data_ptr()
        i = bisect_left(self._starts, start + 8 * t.numel())  # states that begin before t's end
        if i and self._ends[i - 1] > start:
            raise ValueError(f"{name} must lie apart from the states")

    def _positions(self, given, name: str, default: int):
        """(address, value) of a bound."""
        if given is None:
            return 0, default
        if isinstance(given, torch.Tensor):
            if given.dtype is not _I64 or given.numel() != self.groups or given.device != self.device or \
                    not given.is_contiguous():
                raise ValueError(f"{name} must be a number or contiguous int64 [{self.groups}] on {self.device}")
            self._apart(given, name)
            return given.data_ptr(), 0
        return 0, min(max(int(given), 0), 1 << 62)
