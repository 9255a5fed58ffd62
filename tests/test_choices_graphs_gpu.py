"""Captured steps of beam search and routings whose scratch other kernels of the same graph write into between its
replays: every replay gives what an eager call gives."""
import pytest
import torch

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def step(groups, beams, cols, width, dtype):
    def make(gen):
        x = torch.randn(groups, beams, cols, device="cuda", generator=gen).to(DT[dtype])
        return x, -torch.rand(groups, beams, device="cuda", generator=gen)

    def call(inputs, scratch=None):
        return ar.beam_step(*inputs, width, end_token=1, scratch=scratch)

    return make, call, B.argreduce_beam_scratch_bytes(groups, beams, cols, dtype, width), groups


def route(groups, tokens, experts, top, dtype):
    def make(gen):
        return (torch.randn(groups, tokens, experts, device="cuda", generator=gen).to(DT[dtype]),)

    def call(inputs, scratch=None):
        return ar.route_experts(*inputs, top, scratch=scratch)[:6]

    return make, call, B.argreduce_route_scratch_bytes(groups, tokens, experts, dtype), groups


CALLS = {"step 1x4x32000": lambda: step(1, 4, 32000, 4, "f32"), "step 1x8x202048": lambda: step(1, 8, 202048, 16, "bf16"),
         "step 16x5x32001": lambda: step(16, 5, 32001, 5, "f16"), "step 300x3x700": lambda: step(300, 3, 700, 3, "f32"),
         "route 16x1000x64": lambda: route(16, 1000, 64, 2, "f16"), "route 3x5000x513": lambda: route(3, 5000, 513, 4, "f32"),
         "route 1x60000x64": lambda: route(1, 60000, 64, 6, "bf16")}  # the last: several sets of workgroups


def replay_and_compare(make, call, graph, static, results, what):
    gen = torch.Generator(device="cuda").manual_seed(9)
    for i in range(6):
        inputs = make(gen)
        for a, b in zip(static, inputs):
            a.copy_(b)
        want = call(inputs)
        for t in results:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(results, want)):
            assert torch.equal(a, b), (what, i, k)


@pytest.mark.parametrize("name", list(CALLS))
def test_scratch_written_over_between_replays(name):
    make, call, need, groups = CALLS[name]()
    # a word, a line, all words that are kept per group, half, the end, everything
    for a, b in [(0, 8), (0, 512), (0, 8 * groups), (8 * groups, 16 * groups), (0, need // 2), (need // 2, need), (0, need)]:
        b = min(b, need)
        if a >= b:
            continue
        announce(f"{name} scratch bytes [{a}, {b}) of {need} written over in the graph")
        static = make(torch.Generator(device="cuda").manual_seed(1))
        scratch = torch.full((need + 16,), 3, dtype=torch.uint8, device="cuda")
        assert scratch.data_ptr() % 16 == 0
        call(static)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results = call(static, scratch)
            scratch[a:b].fill_(90)
        replay_and_compare(make, call, graph, static, results, (name, a, b))


@pytest.mark.parametrize("name", list(CALLS))
def test_results_dropped_inside_of_a_graph(name):
    """The memory of a call's scratch goes to the next tensor of the capture, which holds the same in every replay."""
    make, call, need, groups = CALLS[name]()
    for words in (1, 2, groups, 64, 224, 4096):
        announce(f"{name} results dropped, {words} words in their place")
        static = make(torch.Generator(device="cuda").manual_seed(1))
        call(static)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = call(static)
            results = [t.clone() for t in r]
            del r
            others = [torch.full((words,), 5, dtype=torch.int64, device="cuda") for _ in range(4)]
        replay_and_compare(make, call, graph, static, results, (name, words))
        assert all((t == 5).all() for t in others)


@pytest.mark.parametrize("name", list(CALLS))
def test_scratch_moved_within_itself_between_replays(name):
    """What a launch has left in one word of scratch, another one holds at the next replay."""
    make, call, need, groups = CALLS[name]()
    for shift in (8, 16, 8 * groups, 16 * groups, need // 16 * 8):
        announce(f"{name} scratch moved on by {shift} of {need} bytes in the graph")
        static = make(torch.Generator(device="cuda").manual_seed(1))
        scratch = torch.full((need + 16,), 3, dtype=torch.uint8, device="cuda")
        call(static)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results = call(static, scratch)
            scratch.copy_(scratch.roll(shift))
        replay_and_compare(make, call, graph, static, results, (name, shift))
