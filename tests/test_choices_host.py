"""Beam search and expert routing on the host (CPU only): argument checks before any GPU call, the fast-call
module against ctypes, plans and scratch, the states' layouts, and the refusals of the torch functions."""
import ctypes

import numpy as np
import pytest
import torch

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B
import choices_reference as C

MI355X_THREADS = 256 * 2048
FAKE = 1 << 20  # an aligned, never-dereferenced address
INT32_MAX = 2 ** 31 - 1


@pytest.fixture
def lib():
    h = B.lib()
    B.argreduce_debug_set_capacity(MI355X_THREADS)
    yield h
    B.argreduce_debug_set_capacity(0)


def both(lib, name, *args):
    a, b = getattr(lib, name)(*args), getattr(B.fast(), name)(*args)
    assert a == b
    return a


# x, dtype, groups, beams, cols, row_stride, scores, ended, end_token, temperature, width, out, scratch, bytes, stream
STEP = (FAKE, B.F32, 2, 4, 100, 100, FAKE, 0, -1, 1.0, 4, FAKE, 0, 0, 0)


@pytest.mark.parametrize("at,value,status", [
    (0, 0, -1), (0, FAKE + 2, -1), (0, FAKE | 1 << 50, -1), (1, B.F64, -2), (1, 77, -2), (2, -1, -1), (2, 0, 0),
    (2, INT32_MAX, -3), (2, INT32_MAX // 256 + 1, -3), (3, 0, -1), (3, 65, -1), (4, 0, -1), (4, 1 << 31, -3),
    (5, 99, -1), (5, -100, -1), (5, 1 << 32, -3), (6, 0, -1), (6, FAKE + 2, -1), (7, FAKE, -1), (7, 1 << 50, -1),
    (8, 100, -1), (9, 0.0, -1), (9, -1.0, -1), (9, float("nan"), -1), (9, float("inf"), -1), (9, 2.0 ** 61, -1),
    (9, 1e300, -1), (10, 0, -1), (10, 65, -1), (11, 0, -1), (11, FAKE + 4, -1)])
def test_step_arguments(lib, at, value, status):
    args = list(STEP)
    args[at] = value
    assert both(lib, "argreduce_beam_step", *args) == status


def test_step_scratch(lib):
    assert B.argreduce_beam_scratch_bytes(2, 4, 100, "f32", 4) == 0  # a wavefront per group
    args = list(STEP)
    args[4:6] = [9000, 9000]
    need = B.argreduce_beam_scratch_bytes(2, 4, 9000, "f32", 4)
    lists = 4 * B.argreduce_beam_plan(2, 4, 9000, "f32", 4)["blocks_per_row"]
    assert need == 15 + 2 * 8 * (2 + lists * (3 + 4))
    for ptr, size in [(0, need), (FAKE, need - 1), (0, 0)]:
        assert both(lib, "argreduce_beam_step", *args[:12], ptr, size, 0) == -4
    assert B.argreduce_beam_out_bytes(3, 5) == 15 * 21
    for bad in [(-1, 4), (2, 0), (2, 65), (1 << 31, 1)]:
        assert B.argreduce_beam_out_bytes(*bad) == B.SIZE_MAX
    for bad in [(-1, 4, 8, "f32", 4), (2, 0, 8, "f32", 4), (2, 4, 0, "f32", 4), (2, 4, 8, "f64", 4),
                (2, 4, 8, "f32", 0), (2, 65, 8, "f32", 4)]:
        assert B.argreduce_beam_scratch_bytes(*bad) == B.SIZE_MAX
        with pytest.raises(ar.ArgreduceError):
            B.argreduce_beam_plan(*bad)
    assert lib.argreduce_beam_plan(2, 4, 8, B.F32, 4, None) == -1


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_step_plans(lib, dtype):
    """Every plan's lists fit the join, its grid the launch, and its scratch is what the size call says."""
    paths = set()
    for groups in (0, 1, 2, 16, 300, 60000):
        for beams in (1, 2, 5, 8, 63, 64):
            for cols in (1, 31, 64, 1000, 5000, 32000, 202048, 1 << 24, INT32_MAX):
                p = B.argreduce_beam_plan(groups, beams, cols, dtype, 7)
                assert p["scratch_bytes"] == B.argreduce_beam_scratch_bytes(groups, beams, cols, dtype, 7)
                assert 1 <= beams * p["blocks_per_row"] <= 256
                assert p["grid_blocks"] * p["block_threads"] < 1 << 32
                assert p["grid_rows"] >= groups * beams
                paths.add(p["path"])
    assert paths == {B.PATH_SUBWAVE, B.PATH_BLOCK, B.PATH_SPLIT}


# x, dtype, groups, tokens, experts, row_stride, live, top, renormalize, weights, chosen, totals, scratch, bytes, stream
ROUTE = (FAKE, B.F32, 2, 30, 16, 16, 0, 2, 0, FAKE, FAKE, FAKE, 0, 0, 0)
# x, dtype, groups, tokens, experts, row_stride, top, renormalize, chosen, totals, g_weights, g_balance, g_z, grad, stream
GRAD = (FAKE, B.F32, 2, 30, 16, 16, 2, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0)
ROUTER = [(0, 0, -1), (0, FAKE + 2, -1), (0, FAKE | 1 << 50, -1), (1, B.F64, -2), (2, -1, -1), (2, 0, 0), (3, -1, -1),
          (2, 1 << 31, -3), (3, 1 << 31, -3), (3, 1 << 30, -3), (4, 0, -1), (4, 1025, -1), (5, 15, -1), (5, 1 << 32, -3)]


@pytest.mark.parametrize("at,value,status", ROUTER + [
    (6, 1 << 50, -1), (7, 0, -1), (7, 17, -1), (7, -3, -1), (9, 0, -1), (9, FAKE + 2, -1), (10, 0, -1),
    (10, FAKE + 4, -1), (11, 0, -1), (11, FAKE + 4, -1)])
def test_route_arguments(lib, at, value, status):
    args = list(ROUTE)
    args[at] = value
    assert both(lib, "argreduce_route", *args) == status


@pytest.mark.parametrize("at,value,status", ROUTER + [
    (3, 0, 0), (6, 0, -1), (6, 17, -1), (8, 0, -1), (8, FAKE + 4, -1), (9, 0, -1), (9, FAKE + 4, -1), (10, FAKE + 2, -1),
    (11, FAKE + 1, -1), (12, FAKE + 3, -1), (13, 0, -1), (13, FAKE + 2, -1)])
def test_route_grad_arguments(lib, at, value, status):
    args = list(GRAD)
    args[at] = value
    assert both(lib, "argreduce_route_grad", *args) == status


def test_route_scratch_and_plans(lib):
    for dtype in ("f32", "f16", "bf16"):
        for groups in (0, 1, 3, 100, 5000):
            for tokens in (0, 1, 31, 4096, 100000):
                for experts in (1, 2, 7, 8, 9, 64, 100, 256, 513, 1024):
                    p = B.argreduce_route_plan(groups, tokens, experts, dtype)
                    need = B.argreduce_route_scratch_bytes(groups, tokens, experts, dtype)
                    assert need == p["scratch_bytes"]
                    assert (need == 0) == (p["grid_blocks"] == max(1, groups))
                    vw = 4 if dtype == "f32" else 8
                    assert p["lanes_per_row"] * p["unroll"] * vw >= experts
                    assert p["grid_blocks"] % max(1, groups) == 0
                    assert p["grid_blocks"] // max(1, groups) <= 64 * 64
                    if need and groups:
                        for ptr, size in [(0, need), (FAKE, need - 1)]:
                            args = (FAKE, B.DTYPE_NAMES[dtype], groups, tokens, experts, experts, 0, 1, 0, FAKE, FAKE,
                                    FAKE, ptr, size, 0)
                            assert both(lib, "argreduce_route", *args) == -4
    assert B.argreduce_route_totals_bytes(3, 10) == 3 * (80 + 16)
    for bad in [(-1, 10), (1, 0), (1, 1025), (1 << 31, 1)]:
        assert B.argreduce_route_totals_bytes(*bad) == B.SIZE_MAX
    for bad in [(-1, 1, 8, "f32"), (1, -1, 8, "f32"), (1, 1, 0, "f32"), (1, 1, 1025, "f32"), (1, 1, 8, "f64"),
                (1 << 16, 1 << 16, 8, "f32")]:
        assert B.argreduce_route_scratch_bytes(*bad) == B.SIZE_MAX
        with pytest.raises(ar.ArgreduceError):
            B.argreduce_route_plan(*bad)
    assert lib.argreduce_route_plan(1, 1, 8, B.F32, None) == -1


def state(**kw):
    s = dict(base=FAKE, group_stride=4000, beam_stride=1000, outer=2, outer_stride=500, positions=10, position_stride=50,
             inner=50)
    s.update(kw)
    return B.argreduce_state_t(**s)


def plan_of(*states, groups=3, beams=4):
    return B.argreduce_reorder_plan((B.argreduce_state_t * len(states))(*states), groups, beams)


@pytest.mark.parametrize("kw,code", [
    (dict(base=0), -1), (dict(base=1 << 50), -1), (dict(outer=0), -1), (dict(positions=-1), -1), (dict(inner=0), -1),
    (dict(beam_stride=999), -1),          # beams that overlap
    (dict(beam_stride=0), -1), (dict(group_stride=3999), -1), (dict(outer_stride=499), -1),
    (dict(position_stride=49), -1), (dict(position_stride=-50), -1), (dict(group_stride=1 << 47), -1),
    (dict(outer=1 << 20, outer_stride=1 << 20, positions=1 << 12, beam_stride=1 << 42, group_stride=1 << 45), -3)])
def test_states_that_are_refused(lib, kw, code):
    with pytest.raises(ar.ArgreduceError) as e:
        plan_of(state(), state(**kw))
    assert e.value.code == code


def test_reorder_plan_and_arguments(lib):
    p = plan_of(state(), state(positions=7, inner=20, position_stride=50))
    assert (p.tensors, p.beams, p.groups, p.positions, p.position_bytes) == (2, 4, 3, 10, 100)
    plan_of(state(positions=0))
    plan_of(state(position_stride=100000, group_stride=800, beam_stride=200, outer_stride=100))  # positions outermost
    for groups, beams in [(-1, 4), (3, 0), (3, 65)]:
        with pytest.raises(ar.ArgreduceError):
            plan_of(state(), groups=groups, beams=beams)
    assert lib.argreduce_reorder_plan(None, 1, 1, 1, ctypes.byref(p)) == -1
    a = ctypes.addressof(p)
    good = (a, FAKE, FAKE, 0, 0, 0, 1 << 40, 0)
    for at, value, status in [(0, 0, -1), (1, 0, -1), (1, FAKE + 4, -1), (2, 0, -1), (2, FAKE + 4, -1), (3, FAKE + 4, -1),
                              (4, FAKE + 4, -1), (6, 0, 0), (6, -5, 0), (5, 10, 0), (5, 1 << 50, 0)]:
        args = list(good)
        args[at] = value
        assert both(lib, "argreduce_reorder", *args) == status
    none = B.argreduce_reorder_t(1, 4, 0, 10, 100)  # no groups
    assert both(lib, "argreduce_reorder", ctypes.addressof(none), 0, 0, 0, 0, 0, 9, 0) == 0
    for bad in [(0, 4, 3, 10, 100), (4097, 4, 3, 10, 100), (1, 65, 3, 10, 100), (1, 4, -1, 10, 100), (1, 4, 3, -1, 100),
                (1, 4, 3, 10, 0)]:
        wrong = B.argreduce_reorder_t(*bad)
        assert both(lib, "argreduce_reorder", ctypes.addressof(wrong), *good[1:]) == -1


def test_fast_module_checks_its_arguments():
    fast = B.fast()
    for name, args in (("argreduce_beam_step", STEP), ("argreduce_route", ROUTE), ("argreduce_route_grad", GRAD)):
        with pytest.raises(TypeError):
            getattr(fast, name)(*args[:-1])
        with pytest.raises(OverflowError):
            getattr(fast, name)(args[0], 1 << 40, *args[2:])
    with pytest.raises(TypeError):
        fast.argreduce_reorder(1)
    with pytest.raises(ValueError):
        fast.bind_choices(0, 0, 0, 0, 0, 0)


def test_names_and_limits():
    assert {"beam_step", "BeamStates", "BeamStep", "route_experts", "route_experts_grad", "token_logprobs"} <= set(dir(ar))
    assert ar.beam_step is ar.beams.beam_step and ar.route_experts is ar.routing.route_experts
    text = open(B.LIB_PATH.replace("libargreduce.so", "../include/argreduce.h")).read()
    for name, value in (("BEAM_MAX", ar.beams.BEAM_MAX), ("EXPERTS_MAX", ar.routing.EXPERTS_MAX),
                        ("ROUTE_TOP_MAX", ar.routing.ROUTE_TOP_MAX)):
        assert f"#define ARGREDUCE_{name} {value}\n" in text
    assert ctypes.sizeof(B.argreduce_state_t) == 64


@pytest.mark.parametrize("shape,strides,dim,want", [
    ((2, 3, 4, 50, 8), None, 3, (4, 400, 50, 8, 8)),
    ((2, 3, 50, 4, 8), None, 2, (1, None, 50, 32, 32)),
    ((2, 3, 4, 50, 8), (4800, 1600, 400, 8, 1), 3, (4, 400, 50, 8, 8)),          # longer caches
    ((2, 3, 2, 4, 50, 8), None, 4, (8, 400, 50, 8, 8)),
    ((2, 3, 7), None, None, (1, None, 1, None, 7)),
    ((2, 3, 7), None, 2, (1, None, 7, 1, 1)),
    ((2, 3), None, None, (1, None, 1, None, 1)),
    ((2, 3, 4, 1, 8), None, 3, (4, 8, 1, None, 8)),
    ((50, 2, 3, 4, 8), "positions first", 2, (1, None, 50, None, 32))])
def test_layouts(shape, strides, dim, want):
    n = 200000
    buf = torch.zeros(n, dtype=torch.int16)
    if strides == "positions first":
        t = torch.zeros(shape, dtype=torch.int16).permute(1, 2, 0, 3, 4)
    elif strides is None:
        t = torch.zeros(shape, dtype=torch.int16)
    else:
        t = buf.as_strided(shape, strides)
    s = ar.beams._state(t, 2, 3, dim)
    outer, outer_stride, positions, position_stride, inner = want
    assert (s.outer, s.positions, s.inner) == (outer, positions, 2 * inner)
    if outer_stride is not None:
        assert s.outer_stride == 2 * outer_stride
    if position_stride is not None:
        assert s.position_stride == 2 * position_stride
    assert (s.group_stride, s.beam_stride) == (2 * t.stride(0), 2 * t.stride(1))


def test_layouts_that_are_refused():
    t = torch.zeros(2, 3, 4, 50, 8)
    for bad, dim in [(t.transpose(3, 4), 3), (t[..., ::2], 3), (t[:, :, :, :, 1::2], None),
                     (torch.zeros(2, 3, 4, 5, 50, 8)[:, :, :, :3], 4)]:
        with pytest.raises(ValueError):
            ar.beams._state(bad, 2, 3, dim)


def test_torch_functions_refuse_cpu_tensors():
    x, s = torch.zeros(2, 4, 16), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="GPU"):
        ar.beam_step(x, s)
    with pytest.raises(ValueError, match="GPU"):
        ar.BeamStates(torch.zeros(2, 4, 8))
    with pytest.raises(ValueError, match="at least one"):
        ar.BeamStates([])
    with pytest.raises(ValueError, match="GPU"):
        ar.route_experts(x, 2)
    with pytest.raises(ValueError, match="GPU"):
        ar.route_experts(x.requires_grad_(), 2)
    r = ar.RouteExperts(*[torch.zeros(2, 4, 2)] * 7)
    with pytest.raises(ValueError, match="GPU"):
        ar.route_experts_grad(x.detach(), r)


def test_gradients_and_tangents_are_refused():
    from torch.autograd import forward_ad

    x, s = torch.zeros(2, 4, 16, requires_grad=True), torch.zeros(2, 4)
    with pytest.raises(RuntimeError, match="no gradient"):
        ar.beam_step(x, s)
    with pytest.raises(RuntimeError, match="no gradient"):
        ar.beam_step(x.detach(), s.clone().requires_grad_())
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        ar.beam_step(x, s)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x.detach(), torch.ones(2, 4, 16))
        for f in (lambda: ar.beam_step(dual, s), lambda: ar.route_experts(dual, 2),
                  lambda: ar.beam_step(x.detach(), forward_ad.make_dual(s, torch.ones(2, 4)))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                f()


def test_reference_of_the_step():
    """The reference against torch's own log softmax, and its own order on ties and ended beams."""
    rng = np.random.default_rng(0)
    x, s = rng.normal(size=(3, 20)), np.array([-1.0, -2.0, -np.inf])
    want = C.beam_values(x, s, None, None, 0.7)
    lp = torch.log_softmax(torch.from_numpy(x) / 0.7, 1) + torch.from_numpy(s)[:, None]
    top = lp.flatten().topk(10)
    assert [c[1] * 20 + c[2] for c in want[:10]] == top.indices.tolist() and len(want) == 40
    assert np.allclose([c[0] for c in want[:10]], top.values)
    x[1] = x[0]
    s[1] = s[0]
    want = C.beam_values(x, s, [False, False, True], 5, 0.7)
    assert [c[1] for c in want[:4]] == [0, 1, 0, 1] and len(want) == 40
    assert (C.beam_values(x, np.array([-1.0, -np.inf, -0.5]), [False, False, True], 5, 0.7)[0][1:3]) == (2, 5)


def test_reference_of_the_routing():
    """Gradients of the reference against torch's autograd in 64 bits."""
    rng = np.random.default_rng(1)
    for renormalize in (False, True):
        x = rng.normal(size=(9, 7))
        x[2, 3] = -np.inf
        live = np.array([True] * 8 + [False])
        group = C.route_group(x, live, 3, renormalize)
        gw, gb, gz = rng.normal(size=(9, 3)), 0.7, -0.3
        t = torch.from_numpy(x).requires_grad_()
        at = torch.from_numpy(np.where(group["experts"] < 0, 0, group["experts"]))
        p = torch.softmax(t, 1) * torch.from_numpy(live)[:, None]
        w = p.gather(1, at)
        if renormalize:
            w = torch.softmax(t.gather(1, at), 1) * torch.from_numpy(live)[:, None]
        counts = torch.from_numpy(group["counts"]).double()
        balance = 7 / (3 * 64) * (counts * p.sum(0)).sum()
        z = (torch.logsumexp(t, 1) ** 2 * torch.from_numpy(live)).sum() / 8
        assert np.allclose(w.detach(), group["weights"])
        assert abs(balance.item() - group["balance"]) < 1e-12 and abs(z.item() - group["z"]) < 1e-12
        target = (w * torch.from_numpy(gw)).sum() + gb * balance + gz * z
        want = torch.autograd.grad(target, t)[0].numpy()
        for k in range(9):
            d, tol = C.route_grad_token(group, k, renormalize, gw[k], gb, gz, "f32")
            assert np.allclose(np.nan_to_num(want[k]), d, atol=1e-13), k
            assert (tol >= 0).all()


def test_reference_of_the_reordering():
    rng = np.random.default_rng(2)
    s = rng.normal(size=(2, 3, 4, 6))
    parents = np.array([[1, 1, 0], [2, -1, 9]])
    got = C.reorder(s, parents, 3, [1, 0], [4, 99])
    assert np.array_equal(got[0, 0, :, 1:4], s[0, 1, :, 1:4]) and np.array_equal(got[0, 0, :, 4:], s[0, 0, :, 4:])
    assert np.array_equal(got[1, 0], s[1, 2]) and np.array_equal(got[1, 1:], s[1, 1:])
