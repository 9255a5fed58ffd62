"""Results of plain calls as tensors of a program: written over in place where autograd has kept another one."""
import pytest
import torch

import argmin_reduction_wide_amd as ar
from gpu_helpers import announce

pytestmark = pytest.mark.gpu


def test_weights_written_after_the_experts_were_used():
    """A router that is not trained, experts that are: the gather keeps the expert numbers for its backward pass, and
    the weights are scaled in place after it."""
    announce("route_experts: weights in place after a gather by the experts")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 30, 16, device="cuda", generator=g)
    each = torch.randn(2, 30, 16, device="cuda", generator=g).requires_grad_()
    r = ar.route_experts(x, 3)
    want = r.weights.clone() * 0.5
    out = each.gather(-1, r.experts)
    r.weights.mul_(0.5)
    (out * r.weights).sum().backward()
    grad = torch.zeros_like(x).scatter_(-1, r.experts, want)
    assert torch.equal(each.grad, grad)


def test_scores_written_after_the_tokens_were_used():
    announce("beam_step: scores in place after a lookup by the tokens")
    g = torch.Generator(device="cuda").manual_seed(2)
    for cols in (50, 9000):
        x, s = torch.randn(2, 4, cols, device="cuda", generator=g), torch.zeros(2, 4, device="cuda")
        table = torch.randn(cols, 5, device="cuda", generator=g).requires_grad_()
        r = ar.beam_step(x, s, end_token=1)
        parents = r.parents.clone()
        out = table[r.tokens]
        r.scores.sub_(1.0)
        r.ended.logical_not_()
        out.sum().backward()
        want = torch.zeros(cols, device="cuda").index_add_(0, r.tokens.flatten(), torch.ones(8, device="cuda"))
        assert torch.equal(table.grad, want[:, None].expand(cols, 5)) and torch.equal(r.parents, parents)


def test_experts_written_after_the_weights_were_used():
    announce("route_experts: experts in place after a product with the weights")
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(2, 30, 16, device="cuda", generator=g)
    scale = torch.ones(3, device="cuda", requires_grad=True)
    r = ar.route_experts(x, 3)
    want = r.weights.sum((0, 1))
    out = r.weights * scale
    r.experts.clamp_(min=0)
    r.counts.zero_()
    out.sum().backward()
    assert torch.equal(scale.grad, want)


def test_weights_times_a_parameter_in_place():
    """The other results do not become part of the graph."""
    announce("route_experts: weights times a parameter in place")
    x = torch.randn(2, 30, 16, device="cuda")
    scale = torch.full((3,), 0.5, device="cuda", requires_grad=True)
    r = ar.route_experts(x, 3)
    want = r.weights.clone()
    r.weights.mul_(scale)
    assert not any(t.requires_grad for t in (r.experts, r.counts, r.tokens, r.balance, r.z, r.totals))
    r.weights.sum().backward()
    assert torch.equal(scale.grad, want.sum((0, 1)))


def test_tokens_written_after_the_parents_were_used():
    announce("beam_step: tokens in place after a gather by the parents")
    g = torch.Generator(device="cuda").manual_seed(4)
    for cols in (50, 9000):
        x, s = torch.randn(2, 4, cols, device="cuda", generator=g), torch.zeros(2, 4, device="cuda")
        hidden = torch.randn(2, 4, 5, device="cuda", generator=g).requires_grad_()
        r = ar.beam_step(x, s)
        want = torch.zeros(2, 4, device="cuda").scatter_add_(1, r.parents, torch.ones(2, 4, device="cuda"))
        out = hidden.gather(1, r.parents[..., None].expand(2, 4, 5))
        r.tokens.clamp_(min=3)
        out.sum().backward()
        assert torch.equal(hidden.grad, want[..., None].expand(2, 4, 5))


def test_experts_written_after_the_counts_were_used():
    announce("route_experts: experts in place after a product with the counts")
    x = torch.randn(2, 30, 16, device="cuda")
    load = torch.ones(2, 16, device="cuda", requires_grad=True)
    r = ar.route_experts(x, 3)
    out = load * r.counts
    r.experts.clamp_(min=1)
    out.sum().backward()
    assert torch.equal(load.grad, r.counts.float())
