"""Beam search's step and reordering on the GPU against the plain 64-bit reference (choices_reference.py): special
rows, ties, layouts, streams, graphs, bounds of buffers, and a search as a program runs it."""
import math

import numpy as np
import pytest
import torch

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B
import choices_reference as C
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf


@pytest.fixture
def capacity():
    yield B.argreduce_debug_set_capacity
    B.argreduce_debug_set_capacity(0)


def host(t):
    return t.detach().double().cpu().numpy()


def make_logits(rng, groups, beams, cols, dtype, std=2.0):
    """Ordinary rows and, from group to group, special ones: masked, empty, constant, the lowest value, NaN, +inf, a
    few values only, beams with equal rows."""
    x = rng.normal(size=(groups, beams, cols)) * std
    low = torch.finfo(DT[dtype]).min
    for g in range(groups):
        b = g % beams
        kind = g % 10
        if kind == 1:
            x[g, b, rng.random(cols) < 0.5] = -INF
        elif kind == 2:
            x[g, b] = -INF
        elif kind == 3:
            x[g, b] = 0.25
        elif kind == 4:
            x[g, b] = low
        elif kind == 5:
            x[g, b, rng.random(cols) < 0.5] = low
        elif kind == 6:
            x[g, b, int(rng.integers(cols))] = math.nan
        elif kind == 7:
            x[g, b, int(rng.integers(cols))] = INF
        elif kind == 8:
            x[g] = rng.integers(0, 3, size=(beams, cols))
        elif kind == 9:
            x[g] = x[g, 0]
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def make_scores(rng, groups, beams):
    s = -rng.random((groups, beams)).cumsum(axis=1) * 3 - 2
    for g in range(groups):
        if g % 10 == 9:
            s[g] = s[g, 0]             # ties across beams
        if g % 4 == 3:
            s[g, 1:] = -INF            # a search's start
        if g % 7 == 5:
            s[g, g % beams] = (math.nan, INF, -INF)[g % 3]
    return torch.from_numpy(s).float().cuda()


def check(x, scores, width, temperature=1.0, ended=None, end=None, **kw):
    """One call against the reference, group by group."""
    r = ar.beam_step(x, scores, width, temperature=temperature, ended=ended, end_token=end, **kw)
    torch.cuda.synchronize()
    beams, cols = x.shape[-2:]
    xs, ss = host(x).reshape(-1, beams, cols), host(scores).reshape(-1, beams)
    es = None if ended is None else ended.cpu().numpy().reshape(-1, beams)
    width = beams if width is None else width
    assert r.scores.shape == r.parents.shape == r.tokens.shape == x.shape[:-2] + (width,)
    got = [host(t).reshape(-1, width) for t in (r.scores, r.parents, r.tokens)]
    for g in range(len(xs)):
        want = C.beam_values(xs[g], ss[g], None if es is None else es[g], end, temperature)
        C.check_beam_group([t[g] for t in got], want, width, f"group {g}")
    if end is None:
        assert r.ended is None
    else:
        assert r.ended.dtype == torch.bool and torch.equal(r.ended, r.tokens == end)
    return r


SHAPES = [(1, 1, 1, 1), (5, 3, 2, 3), (21, 4, 7, 4), (11, 1, 64, 5), (21, 5, 65, 10), (11, 3, 129, 64), (11, 4, 500, 4),
          (11, 2, 1025, 17), (11, 6, 2049, 6), (10, 3, 4100, 33), (3, 7, 8200, 14), (2, 4, 16411, 4), (1, 64, 300, 64),
          (2, 33, 2100, 40), (10, 4, 1000, 9), (10, 8, 500, 8), (10, 16, 60, 20), (10, 30, 60, 64), (10, 64, 16, 64),
          (300, 3, 700, 3), (40, 7, 3001, 7)]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("groups,beams,cols,width", SHAPES)
def test_step(dtype, groups, beams, cols, width):
    rng = np.random.default_rng(groups * 1000 + cols + beams)
    temperature = [1.0, 0.7, 3.0][cols % 3]
    announce(f"beam_step {dtype} [{groups},{beams},{cols}] width {width} T={temperature}")
    x = make_logits(rng, groups, beams, cols, dtype)
    scores = make_scores(rng, groups, beams)
    check(x, scores, width, temperature)
    ended = torch.from_numpy(rng.random((groups, beams)) < 0.4).cuda()
    check(x, scores, width, temperature, ended, cols // 2)
    check(x, scores, None, temperature, None, cols - 1)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("cap", [2048, 256 * 2048])
@pytest.mark.parametrize("groups,beams,cols", [(4, 3, 6000), (2, 4, 20001), (1, 2, 70001), (1, 1, 262144)])
def test_every_path(capacity, dtype, cap, groups, beams, cols):
    """A small simulated device takes a workgroup per row where the real one splits the rows."""
    rng = np.random.default_rng(cols)
    capacity(cap)
    for width in (1, 4, 64):
        plan = B.argreduce_beam_plan(groups, beams, cols, dtype, width)
        announce(f"beam_step {dtype} [{groups},{beams},{cols}] width {width} capacity {cap}: path {plan['path']} "
                 f"slices {plan['blocks_per_row']}")
        x = make_logits(rng, groups, beams, cols, dtype)
        check(x, make_scores(rng, groups, beams), width, 0.9)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("beams,cols,width", [(5, 520, 3), (12, 1031, 24), (3, 1999, 64), (12, 2056, 12), (7, 4090, 20),
                                              (64, 515, 64), (5, 64 * 32 + 1, 7)])
def test_a_wavefront_per_row(capacity, dtype, beams, cols, width):
    """Rows of up to 512 vectors, more of them than the (simulated) device has compute units; a join of up to 64 lists
    that all count, and of hundreds of candidates."""
    capacity(2048)
    announce(f"beam_step {dtype} rows by wavefronts [3,{beams},{cols}] width {width}")
    rng = np.random.default_rng(cols)
    plan = B.argreduce_beam_plan(3, beams, cols, dtype, width)
    assert plan["block_threads"] == 64 or cols * (4 if dtype == "f32" else 2) > 16 * 512 or plan["path"] == B.PATH_SUBWAVE
    wide = torch.full((3, beams, cols + 5), float("nan"), dtype=DT[dtype], device="cuda")
    wide[..., :cols] = make_logits(rng, 3, beams, cols, dtype)
    ended = torch.from_numpy(rng.random((3, beams)) < 0.3).cuda()
    check(wide[..., :cols], make_scores(rng, 3, beams), width, 0.8, ended, cols - 1)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("beams,cols,width", [(8, 4090, 8), (6, 9001, 24), (16, 2100, 64), (12, 20400, 5)])
def test_many_rows_in_one_pass(capacity, dtype, beams, cols, width):
    """Longer rows, sixteen and more per compute unit of the (simulated) device: a wavefront each, in one pass."""
    capacity(2048)
    announce(f"beam_step {dtype} many rows in one pass [3,{beams},{cols}] width {width}")
    rng = np.random.default_rng(cols)
    plan = B.argreduce_beam_plan(3, beams, cols, dtype, width)
    vecs = -(-cols * (4 if dtype == "f32" else 2) // 16)
    assert plan["block_threads"] == 64 or vecs > 2560
    wide = torch.full((3, beams, cols + 5), float("nan"), dtype=DT[dtype], device="cuda")
    wide[..., :cols] = make_logits(rng, 3, beams, cols, dtype)
    wide[0, :, :cols - 1:2] = 1.0  # ties
    ended = torch.from_numpy(rng.random((3, beams)) < 0.3).cuda()
    check(wide[..., :cols], make_scores(rng, 3, beams), width, 0.8, ended, cols - 1)


@pytest.mark.parametrize("cap", [2048, 256 * 2048])
@pytest.mark.parametrize("cols", [40, 500, 3000, 140000])
def test_tied_rows(capacity, cap, cols):
    """Rows whose ties put far more elements at the border than any buffer holds, and equal rows."""
    capacity(cap)
    announce(f"beam_step ties cols={cols} capacity {cap}")
    rng = np.random.default_rng(7)
    x = np.zeros((4, 4, cols))
    x[0, 1] = np.arange(cols)
    x[0, 2] = -np.arange(cols)
    x[0, 3] = np.arange(cols) // 64
    x[1] = rng.integers(0, 2, size=cols)     # four equal rows
    x[2, :, 0::2] = -0.0
    x[3, :, cols // 2:] = -INF
    scores = torch.full((4, 4), -1.0).cuda()
    for dtype in sorted(DT):
        t = torch.from_numpy(x).to(DT[dtype]).cuda()
        if dtype == "f16":
            t = t.clamp(min=-60000.0, max=60000.0).masked_fill(torch.isinf(torch.from_numpy(x).cuda()), -INF)
        for width in (4, 64):
            check(t, scores, width)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("offset", [1, 3, 5])
@pytest.mark.parametrize("cols,pad", [(50, 14), (64, 0), (1000, 1), (3001, 7), (9001, 8)])
def test_strides_and_alignment(dtype, offset, cols, pad):
    groups, beams = 5, 3
    rng = np.random.default_rng(offset * cols)
    announce(f"beam_step strides {dtype} cols={cols} pad={pad} offset={offset}")
    rows = groups * beams
    buf = torch.full((rows * (cols + pad) + offset + 16,), 1e4, dtype=DT[dtype], device="cuda")
    x = buf[offset:offset + rows * (cols + pad)].view(groups, beams, cols + pad)[..., :cols]
    x.copy_(make_logits(rng, groups, beams, cols, dtype))
    scores = make_scores(rng, groups, beams)
    check(x, scores, 7)
    check(x.view(groups, 1, beams, cols + pad)[..., :cols] if pad == 0 else x, scores.view(groups, 1, beams)
          if pad == 0 else scores, 7)
    sixteenth = torch.full((scores.numel() + 3,), 9.0, device="cuda")[3:].view(groups, beams)
    sixteenth.copy_(scores)
    assert torch.equal(ar.beam_step(x, sixteenth, 7).tokens, ar.beam_step(x, scores, 7).tokens)


def test_leading_dimensions_and_one_group():
    rng = np.random.default_rng(4)
    announce("beam_step leading dimensions")
    x = torch.from_numpy(rng.normal(size=(2, 3, 4, 50))).float().cuda()
    s = torch.from_numpy(-rng.random((2, 3, 4))).float().cuda()
    r = check(x, s, 5)
    flat = ar.beam_step(x.view(6, 4, 50), s.view(6, 4), 5)
    assert torch.equal(r.tokens.view(6, 5), flat.tokens) and r.tokens.shape == (2, 3, 5)
    one = ar.beam_step(x[0, 0], s[0, 0], 5)
    assert one.tokens.shape == (5,) and torch.equal(one.tokens, r.tokens[0, 0]) and torch.equal(one.scores, r.scores[0, 0])
    assert ar.beam_step(x[:0], s[:0], 5).scores.shape == (0, 3, 5)


def test_rows_that_do_not_count_are_not_read():
    """Dead and finished beams' logits may be anything, and outside of memory even: here NaN."""
    announce("beam_step dead beams")
    x = torch.randn(3, 4, 3000, device="cuda")
    s = torch.tensor([-1.0, -2.0, -3.0, -4.0], device="cuda").repeat(3, 1)
    ended = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    ended[:, 2] = True
    s[:, 1] = -INF
    want = ar.beam_step(x, s, 6, ended=ended, end_token=7)
    x[:, 1:3] = math.nan
    got = ar.beam_step(x, s, 6, ended=ended, end_token=7)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    s[:] = -INF
    none = ar.beam_step(x, s, 6)
    assert (none.parents == -1).all() and (none.tokens == -1).all() and (none.scores == -INF).all()


@pytest.mark.parametrize("temperature", [2.0 ** -60, 1e-3, 0.1, 1e3, 2.0 ** 60])
def test_extreme_temperatures(temperature):
    announce(f"beam_step T={temperature}")
    rng = np.random.default_rng(3)
    for dtype in sorted(DT):
        x = torch.from_numpy(rng.normal(size=(3, 3, 700))).to(DT[dtype]).cuda()
        check(x, make_scores(rng, 3, 3), 8, temperature)


@pytest.mark.parametrize("dtype", sorted(DT))
def test_close_values_of_many_groups(dtype):
    """Selections of many groups against 64-bit torch, to what the bounds allow."""
    announce(f"beam_step many groups {dtype}")
    g = torch.Generator(device="cuda").manual_seed(5)
    for groups, beams, cols in ((3000, 4, 64), (300, 6, 5000), (20, 4, 33000)):
        x = (torch.randn(groups, beams, cols, device="cuda", generator=g) * 2.5).to(DT[dtype])
        s = -torch.rand(groups, beams, device="cuda", generator=g) * 4
        r = ar.beam_step(x, s, beams, temperature=0.9)
        lp = torch.log_softmax(x.double() / 0.9, -1) + s.double()[..., None]
        want = lp.flatten(1).topk(beams, 1).values
        at = lp.flatten(1).gather(1, r.parents * cols + r.tokens)
        # a chosen value is at most two bounds below the one that belongs there; 3 E|z| < 100
        tol = C.U * (100 + C.R.adds(cols))
        assert (want - at).abs().max() < 2 * tol
        assert (r.scores.double() - at).abs().max() < tol + C.U * 40
        pairs = (r.parents * cols + r.tokens).sort(1).values
        assert (pairs[:, 1:] != pairs[:, :-1]).all()


def test_offsets_beyond_32_bits():
    stride, cols = 2 ** 30 + 8, 1000
    announce("beam_step offsets beyond 32 bits")
    buf = torch.empty(5 * stride + cols, dtype=torch.float16, device="cuda")
    x = buf.as_strided((3, 2, cols), (2 * stride, stride, 1))
    rng = np.random.default_rng(3)
    x.copy_(torch.from_numpy(rng.normal(size=(3, 2, cols))).half().cuda())
    check(x, make_scores(rng, 3, 2), 4)


@pytest.mark.parametrize("soff", [0, 1, 13])
def test_scratch_and_output_bounds(soff):
    """Nothing is written outside of scratch and outputs, whatever scratch holds and wherever it starts."""
    announce(f"beam_step bounds offset {soff}")
    for groups, beams, cols, width in ((7, 3, 200, 5), (2, 2, 40000, 64), (3, 4, 9000, 9)):
        x, s = torch.randn(groups, beams, cols, device="cuda"), torch.zeros(groups, beams, device="cuda")
        want = ar.beam_step(x, s, width)
        need = B.argreduce_beam_scratch_bytes(groups, beams, cols, "f32", width)
        n = B.argreduce_beam_out_bytes(groups, width)
        for fill in (0, 255, 90):
            scratch = torch.full((need + soff + 64,), fill, dtype=torch.uint8, device="cuda")
            out = torch.full((n + 64,), 77, dtype=torch.uint8, device="cuda")
            rc = B.argreduce_beam_step(x.data_ptr(), "f32", groups, beams, cols, cols, s.data_ptr(), 0, -1, 1.0, width,
                                       out.data_ptr(), scratch.data_ptr() + soff, need,
                                       torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert rc == 0 and (out[n:] == 77).all()
            assert (scratch[:soff] == fill).all() and (scratch[soff + need:] == fill).all()
            assert torch.equal(out[:8 * groups * width].view(torch.int64).view(groups, width), want.parents)
            assert torch.equal(out[8 * groups * width:16 * groups * width].view(torch.int64).view(groups, width),
                               want.tokens)
            assert torch.equal(out[16 * groups * width:20 * groups * width].view(torch.float32).view(groups, width),
                               want.scores)


@pytest.mark.parametrize("groups,beams,cols,width", [(40, 4, 64, 4), (3, 4, 40000, 8), (600, 4, 5000, 4), (1, 8, 202048, 16)])
def test_same_bits_streams_and_graphs(groups, beams, cols, width):
    announce(f"beam_step [{groups},{beams},{cols}] repeated, on two streams, captured")
    g = torch.Generator(device="cuda").manual_seed(cols)
    xs = [torch.randn(groups, beams, cols, device="cuda", generator=g) for _ in range(2)]
    ss = [torch.rand(groups, beams, device="cuda", generator=g) for _ in range(2)]
    want = [ar.beam_step(x, s, width, end_token=1) for x, s in zip(xs, ss)]
    same = lambda a, b: all(torch.equal(u, v) for u, v in zip(a, b))  # noqa: E731
    for _ in range(5):
        assert same(ar.beam_step(xs[0], ss[0], width, end_token=1), want[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(ar.beam_step(xs[k], ss[k], width, end_token=1))
    torch.cuda.synchronize()
    assert all(same(r, want[k]) for k in range(2) for r in got[k])
    x, s = xs[0].clone(), ss[0].clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = ar.beam_step(x, s, width, end_token=1)
        graphs.append((graph, r))
    for i in range(6):
        x.copy_(xs[i % 2])
        s.copy_(ss[i % 2])
        ar.beam_step(xs[1], ss[1], width)
        graphs[i % 2][0].replay()
        torch.cuda.synchronize()
        assert same(graphs[i % 2][1], want[i % 2])


def test_graphs_that_share_a_scratch():
    """Steps and routings of several shapes in one scratch, captured and eager in turn, one stream."""
    announce("one scratch for graphs of several calls")
    gen = torch.Generator(device="cuda").manual_seed(3)
    scratch = torch.randint(0, 256, (1 << 21,), dtype=torch.uint8, device="cuda", generator=gen)
    calls = []
    for groups, beams, cols, width in ((1, 4, 32000, 4), (3, 4, 40000, 8), (2, 8, 3000, 20), (300, 3, 700, 3)):
        x = torch.randn(groups, beams, cols, device="cuda", generator=gen)
        s = torch.rand(groups, beams, device="cuda", generator=gen)
        calls.append(lambda x=x, s=s, w=width: ar.beam_step(x, s, w, scratch=scratch)[:3])
    for tokens, experts in ((4001, 64), (700, 300)):
        x = torch.randn(2, tokens, experts, device="cuda", generator=gen)
        calls.append(lambda x=x: ar.route_experts(x, 4, scratch=scratch)[:6])
    want = [f() for f in calls]
    torch.cuda.synchronize()
    graphs = []
    for f in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = f()
        graphs.append((graph, r))
    for i in (0, 4, 1, 1, 2, 5, 3, 0, 0, 5, 4, 2, 1, 3, 0):
        for t in graphs[i][1]:
            t.zero_()
        graphs[i][0].replay()
        graphs[(i + 1) % len(graphs)][0].replay()
        eager = calls[i]()
        for a, b, c in zip(graphs[i][1], want[i], eager):
            assert torch.equal(a, b) and torch.equal(c, b), i


def test_outputs_may_be_written_over():
    announce("beam_step outputs")
    x, s = torch.randn(3, 4, 100, device="cuda"), torch.zeros(3, 4, device="cuda")
    want = [t.clone() for t in ar.beam_step(x, s, 5, end_token=0)]
    for k in range(4):
        r = ar.beam_step(x, s, 5, end_token=0)
        r[k].zero_()
        for j in range(4):
            assert torch.equal(r[j], torch.zeros_like(r[j]) if j == k else want[j])


def test_step_refusals():
    announce("beam_step refusals")
    x, s = torch.zeros(2, 4, 16, device="cuda"), torch.zeros(2, 4, device="cuda")
    e = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    bad = [(x.double(), s, {}), (x[..., ::2], s, {}), (x, s.double(), {}), (x, s[:1], {}), (x, s.cpu(), {}),
           (x, s.t().contiguous().t(), {}), (x[0, 0], s[0, 0], {}), (x, s, dict(width=0)), (x, s, dict(width=65)),
           (x, s, dict(temperature=0.0)), (x, s, dict(temperature=math.nan)), (x, s, dict(end_token=16)),
           (x, s, dict(end_token=-1)), (x, s, dict(ended=e)), (x, s, dict(ended=e.byte(), end_token=1)),
           (x, s, dict(ended=e[:1], end_token=1)), (x[..., :0], s, {}), (torch.zeros(2, 65, 8, device="cuda"),
                                                                        torch.zeros(2, 65, device="cuda"), {}),
           (x, s, dict(scratch=torch.zeros(8, dtype=torch.uint8))), (x.transpose(0, 1), s, {})]
    for logits, scores, kw in bad:
        with pytest.raises((ValueError, ar.ArgreduceError)):
            ar.beam_step(logits, scores, **kw)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------------------
# Reordering

DTYPES = [torch.float32, torch.float16, torch.bfloat16, torch.float64, torch.int64, torch.uint8, torch.bool]


def bits(t):
    """A tensor's bytes as numpy, [.., element bytes]."""
    return t.detach().contiguous().view(torch.uint8).view(*t.shape, t.element_size()).cpu().numpy()


def fill(rng, t):
    raw = rng.integers(0, 2 if t.dtype == torch.bool else 256, size=(*t.shape, t.element_size()), dtype=np.uint8)
    t.copy_(torch.from_numpy(raw).view(t.dtype).view(t.shape))


def make_parents(rng, groups, beams):
    p = rng.integers(0, beams, size=(groups, beams))
    for g in range(groups):
        if g % 5 == 1:
            p[g] = np.arange(beams)                    # nothing moves
        elif g % 5 == 2:
            p[g] = np.roll(np.arange(beams), 1)        # a cycle
        elif g % 5 == 3:
            p[g] = 0
        elif g % 5 == 4:
            p[g, rng.random(beams) < 0.4] = (-1, beams, 2 ** 40, -2 ** 62)[g % 4]
    return p


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 11, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda d: str(d)[6:])
def test_reorder(dtype, beams):
    """Layouts of every kind in one call, with spans per group, numbers, and none."""
    groups = 6
    rng = np.random.default_rng(beams)
    announce(f"reorder {dtype} beams={beams}")
    p = make_parents(rng, groups, beams)
    parents = torch.from_numpy(p).cuda()
    first = rng.integers(-2, 9, size=groups)
    last = rng.integers(-1, 30, size=groups)
    spans = [(None, None), (3, None), (None, 11), (-4, 10 ** 12), (7, 5),
             (torch.from_numpy(first).cuda(), torch.from_numpy(last).cuda()), (2, torch.from_numpy(last).cuda())]
    for dim, shapes in ((3, [(3, 19, 5), (2, 7, 16), (1, 23, 1)]), (2, [(19, 3, 5), (8, 64), (21,)]), (None, [(), (7,), (5, 3)])):
        states = [torch.empty(groups, beams, *s, dtype=dtype, device="cuda") for s in shapes]
        if dim == 3:
            wide = torch.empty(groups, beams + 1, 3, 40, 6, dtype=dtype, device="cuda")
            states.append(wide[:, 1:, :, 5:25])        # a slice of a longer cache
        for t in states:
            fill(rng, t)
        handle = ar.BeamStates(states, dim=dim)
        for a, b in spans:
            before = [bits(t) for t in states]
            handle.reorder(parents, first=a, last=b)
            torch.cuda.synchronize()
            for t, old in zip(states, before):
                n = t.shape[dim] if dim is not None else 1
                lo = np.full(groups, 0 if a is None else a) if not torch.is_tensor(a) else a.cpu().numpy()
                hi = np.full(groups, n if b is None else b) if not torch.is_tensor(b) else b.cpu().numpy()
                want = C.reorder(old, p, dim, lo, hi)
                assert np.array_equal(bits(t), want), (dim, t.shape, a, b)


@pytest.mark.parametrize("shape,dim,offset", [((3, 4, 2, 50, 65), 3, 1), ((3, 4, 50, 2, 13), 2, 3), ((2, 5, 1, 9, 7), 3, 5),
                                              ((3, 4, 1000), None, 7)])
def test_reorder_leaves_the_rest(shape, dim, offset):
    """Memory around and between the states is left as it was: odd addresses, gaps, positions outside."""
    announce(f"reorder bounds {shape} offset {offset}")
    rng = np.random.default_rng(offset)
    for dtype in (torch.uint8, torch.float16, torch.float32):
        n = math.prod(shape)
        buf = torch.randint(0, 100, (2 * n + 2 * offset + 64,), device="cuda").to(dtype)
        strides = [1] * len(shape)
        for k in range(len(shape) - 2, -1, -1):
            strides[k] = strides[k + 1] * shape[k + 1]
        strides[0] += 5
        t = buf.as_strided(shape, strides, offset)
        p = make_parents(rng, *shape[:2])
        lo, hi = (None, None) if dim is None else (1, 8)
        model = buf.cpu().clone()
        view = model.as_strided(shape, strides, offset)
        view.copy_(torch.from_numpy(C.reorder(view.numpy(), p, dim, [lo or 0] * shape[0], [hi or 1] * shape[0])))
        ar.BeamStates(t, dim=dim).reorder(torch.from_numpy(p).cuda(), first=lo, last=hi)
        torch.cuda.synchronize()
        assert torch.equal(buf.cpu(), model), dtype


def test_reorder_of_large_states():
    """Offsets past 32 bits, and more units than lanes."""
    announce("reorder large")
    t = torch.empty(2, 3, 4, 200000, 1024, dtype=torch.uint8, device="cuda")  # 4.9 GB, 2.4 GB apart
    for g in range(2):
        for b in range(3):
            t[g, b] = 10 * g + b + 1
    t[1, 2, 3, 199999] = 99
    ar.BeamStates(t, dim=3).reorder(torch.tensor([[1, 2, 0], [2, 1, 1]], device="cuda"), first=150000)
    torch.cuda.synchronize()
    assert t[:, :, :, :150000].flatten(2).amin(2).tolist() == [[1, 2, 3], [11, 12, 13]]
    assert t[:, :, :, :150000].flatten(2).amax(2).tolist() == [[1, 2, 3], [11, 12, 13]]
    assert t[0, :, :, 150000:].flatten(1).amin(1).tolist() == [2, 3, 1] == t[0, :, :, 150000:].flatten(1).amax(1).tolist()
    assert (t[1, 0, 3, 199999] == 99).all() and (t[1, 0, :3, 150000:] == 13).all() and (t[1, 2, :, 150000:] == 12).all()


def test_reorder_empty_and_many():
    announce("reorder empty, many tensors")
    e = torch.empty(0, 4, 5, device="cuda")
    ar.BeamStates(e).reorder(torch.empty(0, 4, dtype=torch.int64, device="cuda"))
    z = torch.empty(3, 4, 0, 5, device="cuda")
    ar.BeamStates([z, z], dim=2).reorder(torch.zeros(3, 4, dtype=torch.int64, device="cuda"))
    states = [torch.full((2, 2, 3), float(i), device="cuda") for i in range(300)]
    for i, s in enumerate(states):
        s[:, 1] = -float(i)
    ar.BeamStates(states).reorder(torch.tensor([1, 1, 0, 0], device="cuda").view(2, 2))
    torch.cuda.synchronize()
    for i, s in enumerate(states):
        assert (s[0] == -float(i)).all() and (s[1] == float(i)).all()


def test_reorder_streams_and_graphs():
    announce("reorder captured")
    rng = np.random.default_rng(1)
    states = [torch.randn(5, 4, 3, 40, 16, device="cuda") for _ in range(3)]
    handle = ar.BeamStates(states, dim=3)
    parents = torch.zeros(5, 4, dtype=torch.int64, device="cuda")
    last = torch.zeros(5, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        handle.reorder(parents, first=2, last=last)
    side = torch.cuda.Stream()
    for i in range(6):
        p, hi = rng.integers(0, 4, size=(5, 4)), rng.integers(0, 41, size=5)
        parents.copy_(torch.from_numpy(p))
        last.copy_(torch.from_numpy(hi))
        before = [t.cpu().numpy().copy() for t in states]
        torch.cuda.synchronize()
        if i % 2:
            graph.replay()
        else:
            with torch.cuda.stream(side):
                handle.reorder(parents, first=2, last=last)
        torch.cuda.synchronize()
        for t, old in zip(states, before):
            assert np.array_equal(t.cpu().numpy(), C.reorder(old, p, 3, [2] * 5, hi))


def test_reorder_refusals():
    announce("reorder refusals")
    t = torch.zeros(2, 4, 3, 8, 5, device="cuda")
    for bad, kw in [([t, t], {}), ([t, t[:, :, 1:]], {}), (t[:, :, :, :, ::2], {}), (t.transpose(3, 4), dict(dim=3)),
                    (t[0, 0, 0, 0], {}), (t, dict(dim=1)), (t, dict(dim=5)), (t, dict(dim=-4)), ([t, t.cpu()], {}),
                    (t.expand(3, 2, 4, 3, 8, 5)[0:1].squeeze(0).expand(2, 4, 3, 8, 5)[:, :1].expand(2, 4, 3, 8, 5), {}),
                    (torch.zeros(2, 65, 3, device="cuda"), {}), (torch.zeros(2, 4, device="cuda", requires_grad=True), {}),
                    ([t, torch.zeros(3, 4, 2, device="cuda")], {})]:
        with pytest.raises((ValueError, ar.ArgreduceError)):
            ar.BeamStates(bad, **kw)
    handle = ar.BeamStates(t, dim=3)
    p = torch.zeros(2, 4, dtype=torch.int64, device="cuda")
    n = torch.zeros(2, dtype=torch.int64, device="cuda")
    for parents, kw in [(p.int(), {}), (p[:1], {}), (p.cpu(), {}), (p.t(), {}), (p.t().contiguous().t(), {}),
                        (p.view(8), {}), (p, dict(first=n.int())), (p, dict(last=n[:1])), (p, dict(first=n.cpu())),
                        (p, dict(last=torch.zeros(4, dtype=torch.int64, device="cuda")[::2]))]:
        with pytest.raises(ValueError):
            handle.reorder(parents, **kw)
    torch.cuda.synchronize()


def test_parents_inside_of_the_states_are_refused():
    """A call would change what its other workgroups still read."""
    announce("reorder by its own states")
    tokens = torch.zeros(3, 4, dtype=torch.int64, device="cuda")
    both = torch.zeros(2, 4, 8, 3, dtype=torch.int64, device="cuda")
    handle = ar.BeamStates([both[0, :3, :4], tokens, both[1, :3, :4]])
    p = torch.zeros(3, 4, dtype=torch.int64, device="cuda")
    handle.reorder(p)
    for bad in (tokens, both.view(-1)[:12].view(3, 4), both.view(-1)[90:102].view(3, 4)):
        with pytest.raises(ValueError, match="parents must lie apart"):
            handle.reorder(bad)
    caches = ar.BeamStates(both.view(3, 4, 16), dim=2)
    for name in ("first", "last"):
        with pytest.raises(ValueError, match=f"{name} must lie apart"):
            caches.reorder(p, **{name: both.view(-1)[189:]})
    caches.reorder(tokens, last=p[:, 0].contiguous())
    torch.cuda.synchronize()


def test_states_made_in_a_capture_are_refused():
    announce("states in a capture")
    t = torch.zeros(3, 4, 5, device="cuda")
    refused = False
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.add_(1)
        try:
            ar.BeamStates(t)
        except RuntimeError as e:
            refused = "capture" in str(e)
    graph.replay()
    torch.cuda.synchronize()
    assert refused and (t == 1).all()


def test_states_dropped_while_another_stream_moves_them():
    """The table that the kernel reads is not given to another tensor before the kernel has run."""
    announce("states dropped early")
    t = torch.arange(4.0, device="cuda").expand(2, 4).contiguous()
    p = torch.full((2, 4), 3, device="cuda")
    handle = ar.BeamStates(t)
    address, size = handle._table.data_ptr(), handle._table.numel() * 8
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        handle.reorder(p)
    del handle
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]
    waiting = not side.query()
    assert all(o.data_ptr() != address for o in others) or not waiting
    torch.cuda.synchronize()
    assert (t == 3).all()


def test_calls_without_the_fast_module(monkeypatch):
    """The same bits through ctypes alone."""
    announce("ctypes")
    import argmin_reduction_wide_amd.beams as module
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(3, 4, 9001, device="cuda", generator=g)
    scores = torch.randn(3, 4, device="cuda", generator=g)
    ended = torch.tensor([[True, False, False, True]] * 3, device="cuda")
    states = torch.randn(3, 4, 2, 20, 8, device="cuda", generator=g)

    def work():
        t = states.clone()
        r = ar.beam_step(x, scores, temperature=0.7, ended=ended, end_token=11)
        ar.BeamStates(t, dim=3).reorder(r.parents, first=2, last=15)
        return [*r, t]

    fast = work()

    class Ctypes:
        def __getattr__(self, name):
            return getattr(B.lib(), "argreduce_" + name)

    monkeypatch.setattr(module, "_call", Ctypes())
    for a, b in zip(fast, work()):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------
# A search


def test_run_together():
    """A beam search over a model whose logits come from its cache, by a router's experts: histories and caches that
    are reordered stay those of their own sequences, scores are the sums of log probabilities, and a finished beam
    stays as it is."""
    announce("a search with a router, step and reordering")
    g = torch.Generator(device="cuda").manual_seed(2)
    groups, beams, cols, size, experts, steps = 5, 4, 300, 16, 8, 9
    embed = torch.randn(cols, size, device="cuda", generator=g)
    gate = torch.randn(size, experts, device="cuda", generator=g)
    heads = torch.randn(experts, size, cols, device="cuda", generator=g)
    cache = torch.zeros(groups, beams, 1, steps, size, device="cuda")
    history = torch.full((groups, beams, steps), -1, dtype=torch.int64, device="cuda")
    caches, histories = ar.BeamStates(cache, dim=3), ar.BeamStates(history, dim=2)
    scores = torch.full((groups, beams), -INF, device="cuda")
    scores[:, 0] = 0.0
    ended = torch.zeros(groups, beams, dtype=torch.bool, device="cuda")
    tokens = torch.randint(0, cols, (groups, 1), device="cuda", generator=g).expand(groups, beams).contiguous()
    start, end = tokens.clone(), 17

    def model(context):  # [.., size] -> logits
        r = ar.route_experts(context @ gate, 2, renormalize=True)
        each = torch.stack([context @ h for h in heads], dim=-2)  # [.., experts, cols]
        chosen = each.gather(-2, r.experts[..., None].expand(*r.experts.shape, cols))
        out = (chosen * r.weights[..., None]).sum(-2) * 0.1
        out[..., end] += 2.0
        return out

    total, mixed = None, False
    for t in range(steps):
        cache[:, :, 0, t] = embed[tokens.clamp(min=0)]
        context = cache[:, :, 0, :t + 1].mean(2)
        logits = model(context)
        r = ar.beam_step(logits, scores, ended=ended, end_token=end)
        caches.reorder(r.parents, last=t + 1)
        histories.reorder(r.parents, last=t)
        total = r.scores.double().cpu()
        scores, tokens, ended = r.scores, r.tokens, r.ended
        history[:, :, t] = tokens
        mixed |= bool(ended.any()) and not bool(ended.all())
    assert mixed  # finished beams among the others
    for i in range(groups):
        for b in range(beams):
            seq = history[i, b].tolist()
            assert -1 not in seq
            # this sequence alone, its cache and its score
            past, value = [int(start[i, b])], 0.0
            for t, token in enumerate(seq):
                rows = embed[torch.tensor(past, device="cuda")]
                assert torch.equal(cache[i, b, 0, :t + 1], rows), (i, b, t)
                if t and seq[t - 1] == end:
                    assert token == end
                else:
                    lp = torch.log_softmax(model(rows.mean(0)[None, None])[0, 0].double(), 0)
                    value += float(lp[token])
                past.append(token)
            assert abs(value - float(total[i, b])) < 1e-4
        assert len({tuple(history[i, b].tolist()) for b in range(beams)}) == beams
        assert (total[i, 1:] <= total[i, :-1]).all()
