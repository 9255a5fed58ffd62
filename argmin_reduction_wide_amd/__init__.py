"""MI355X (gfx950) ArgMax / ArgMin (last or middle axis), cummax / cummin with indices, and
operators on logits over the last axis: token log probabilities and distillation, beam search's
step and reordering, expert routing.

The computation runs in the HIP library ``libargreduce.so`` (C ABI: include/argreduce.h);
``binding`` marshals arguments into it. Importing this package loads nothing; the library
is loaded on first use and its absence is an error, never a fallback.
"""
from .binding import (  # noqa: F401
    ArgreduceError,
    argmax,
    argmin,
    argreduce_axis,
    argreduce_axis_plan,
    argreduce_axis_scratch_bytes,
    argreduce_beam_out_bytes,
    argreduce_beam_plan,
    argreduce_beam_scratch_bytes,
    argreduce_beam_step,
    argreduce_debug_force_path,
    argreduce_debug_set_capacity,
    argreduce_distill,
    argreduce_distill_grad,
    argreduce_distill_plan,
    argreduce_distill_scratch_bytes,
    argreduce_distill_step,
    argreduce_lastaxis,
    argreduce_logprobs,
    argreduce_logprobs_grad,
    argreduce_logprobs_plan,
    argreduce_logprobs_scratch_bytes,
    argreduce_plan,
    argreduce_reorder,
    argreduce_reorder_plan,
    argreduce_route,
    argreduce_route_grad,
    argreduce_route_plan,
    argreduce_route_scratch_bytes,
    argreduce_route_totals_bytes,
    argreduce_scan_lastaxis,
    argreduce_scan_plan,
    argreduce_scan_scratch_bytes,
    argreduce_scratch_bytes,
    cummax,
    cummin,
)

# The logits operators are defined in terms of torch (autograd among it), which the rest of the
# package imports on first use only: they are looked up when first named.
_TORCH = {"logits": ("DistillLoss", "TokenLogprobs", "distill_loss", "distill_loss_grad", "distill_step",
                     "token_logprobs", "token_logprobs_grad"),
          "beams": ("BeamStates", "BeamStep", "beam_step"),
          "routing": ("RouteExperts", "route_experts", "route_experts_grad")}


def __getattr__(name):
    for module, names in _TORCH.items():
        if name in names:
            from importlib import import_module

            m = import_module("." + module, __name__)
            for n in names:
                globals()[n] = getattr(m, n)
            return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted(set(globals()).union(*_TORCH.values()))
