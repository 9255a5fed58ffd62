"""The logits operators on the host (CPU only): argument checks before any GPU call, the fast-call
module against ctypes, plans and scratch, and the refusals of the torch functions."""
import ctypes

import pytest
import torch

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B

MI355X_THREADS = 256 * 2048
FAKE = 1 << 20  # an aligned, never-dereferenced address
INT32_MAX = 2 ** 31 - 1


@pytest.fixture
def lib():
    h = B.lib()
    B.argreduce_debug_set_capacity(MI355X_THREADS)
    yield h
    B.argreduce_debug_set_capacity(0)


# (x, dtype, rows, cols, row_stride) and the status it gives
LOGITS = [
    ((FAKE, B.F32, -1, 8, 8), -1),
    ((FAKE, B.F32, 2, 0, 8), -1),
    ((FAKE, B.F64, 2, 8, 8), -2),
    ((FAKE, B.I32, 2, 8, 8), -2),
    ((FAKE, 9, 2, 8, 8), -2),
    ((FAKE, B.F32, 2, 1 << 31, 1 << 31), -3),
    ((FAKE, B.F32, 1 << 31, 8, 8), -3),
    ((FAKE, B.F32, 2, 8, 1 << 32), -3),
    ((FAKE, B.F32, 2, 8, 7), -1),          # rows that overlap
    ((FAKE, B.F32, 2, 8, -8), -1),
    ((0, B.F32, 2, 8, 8), -1),
    ((FAKE + 2, B.F32, 2, 8, 8), -1),
    ((FAKE + 1, B.BF16, 2, 8, 8), -1),
    ((FAKE | 1 << 50, B.F32, 2, 8, 8), -1),  # not a device address
    ((0, B.F32, 0, 8, 8), 0),
]
CALLS = {
    "argreduce_logprobs": (FAKE, 1.0, 1, 2, FAKE, FAKE, FAKE, 0, 0, 0),
    "argreduce_logprobs_grad": (FAKE, 1.0, FAKE, FAKE, FAKE, FAKE, 0),
    "argreduce_distill": (3, FAKE, FAKE, 1.0, FAKE, 0, 0, 0),
    "argreduce_distill_grad": (3, FAKE, FAKE, 1.0, FAKE, FAKE, FAKE, 0),
    "argreduce_distill_step": (3, FAKE, FAKE, 1.0, FAKE, FAKE, FAKE, 0, 0, 0),
}
GOOD = (FAKE, B.F32, 2, 8, 8)
# Arguments after the logits that are refused: (call, position, value)
BAD = [("argreduce_logprobs", 0, 0), ("argreduce_logprobs", 0, FAKE + 4), ("argreduce_logprobs", 1, 0.0),
       ("argreduce_logprobs", 1, -1.0), ("argreduce_logprobs", 1, float("nan")),
       ("argreduce_logprobs", 1, float("inf")), ("argreduce_logprobs", 1, 2.0 ** 61),
       ("argreduce_logprobs", 3, -1), ("argreduce_logprobs", 3, 65), ("argreduce_logprobs", 4, 0),
       ("argreduce_logprobs", 4, FAKE + 2), ("argreduce_logprobs", 5, 0),
       ("argreduce_logprobs", 6, 0), ("argreduce_logprobs", 6, FAKE + 4),
       ("argreduce_logprobs_grad", 0, 0), ("argreduce_logprobs_grad", 1, 0.0),
       ("argreduce_logprobs_grad", 2, 0), ("argreduce_logprobs_grad", 3, 0),
       ("argreduce_logprobs_grad", 4, FAKE + 1), ("argreduce_logprobs_grad", 5, 0),
       ("argreduce_logprobs_grad", 5, FAKE + 2),
       ("argreduce_distill", 0, 0), ("argreduce_distill", 0, 1025), ("argreduce_distill", 1, 0),
       ("argreduce_distill", 1, FAKE + 4), ("argreduce_distill", 2, FAKE + 2),
       ("argreduce_distill", 3, 0.0), ("argreduce_distill", 4, 0),
       ("argreduce_distill_grad", 0, 0), ("argreduce_distill_grad", 4, 0),
       ("argreduce_distill_grad", 5, 0), ("argreduce_distill_grad", 6, 0),
       ("argreduce_distill_grad", 6, FAKE + 2),
       ("argreduce_distill_step", 0, -1), ("argreduce_distill_step", 4, 0),
       ("argreduce_distill_step", 5, 0), ("argreduce_distill_step", 6, 0)]


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("logits,status", LOGITS)
def test_logits_arguments(lib, name, logits, status):
    args = logits + CALLS[name]
    assert getattr(lib, name)(*args) == status
    assert getattr(B.fast(), name)(*args) == status


@pytest.mark.parametrize("name,at,value", BAD)
def test_other_arguments(lib, name, at, value):
    rest = list(CALLS[name])
    rest[at] = value
    assert getattr(lib, name)(*GOOD, *rest) == -1
    assert getattr(B.fast(), name)(*GOOD, *rest) == -1


@pytest.mark.parametrize("name", ["argreduce_logprobs", "argreduce_distill", "argreduce_distill_step"])
def test_scratch_too_small(lib, name):
    big = (FAKE, B.F32, 1, 202048, 202048)
    need = getattr(B, ("argreduce_logprobs" if "logprobs" in name else "argreduce_distill") +
                   "_scratch_bytes")(1, 202048, B.F32)
    assert 15 < need < 64 * 1024
    rest = list(CALLS[name])
    for ptr, size in [(0, need), (FAKE, need - 1), (0, 0)]:
        rest[-3:] = [ptr, size, 0]
        assert getattr(lib, name)(*big, *rest) == -4


@pytest.mark.parametrize("which", ["logprobs", "distill"])
def test_scratch_depends_on_the_shape_and_stays_small(lib, which):
    f = getattr(B, f"argreduce_{which}_scratch_bytes")
    plan = getattr(B, f"argreduce_{which}_plan")
    paths = set()
    for dtype in (B.F32, B.F16, B.BF16):
        for rows in (0, 1, 3, 64, 1000, 1 << 20):
            for cols in (1, 31, 64, 1000, 5000, 32000, 202048, 1 << 24, INT32_MAX):
                need = f(rows, cols, dtype)
                p = plan(rows, cols, dtype)
                assert p["scratch_bytes"] == need < 1 << 20
                assert (p["path"] == B.PATH_SPLIT) == (need > 0) == (p["dispatches"] == 2)
                assert p["grid_blocks"] * p["block_threads"] < 1 << 32
                paths.add(p["path"])
    assert paths == {B.PATH_SUBWAVE, B.PATH_BLOCK, B.PATH_SPLIT}
    for bad in [(-1, 8, B.F32), (2, 0, B.F32), (2, 8, B.F64), (2, 1 << 31, B.F32)]:
        assert f(*bad) == B.SIZE_MAX
        with pytest.raises(ar.ArgreduceError):
            plan(*bad)
    assert getattr(lib, f"argreduce_{which}_plan")(2, 8, B.F32, None) == -1


def test_a_grid_too_large_is_refused(lib):
    # more workgroups of a row each than a launch holds
    args = (FAKE, B.F32, INT32_MAX, 1 << 20, 1 << 20)
    for name, rest in CALLS.items():
        assert getattr(lib, name)(*args, *rest) == -3


def test_fast_module_checks_its_arguments():
    fast = B.fast()
    assert fast is not None
    with pytest.raises(TypeError):
        fast.argreduce_logprobs(*GOOD)
    with pytest.raises(TypeError):
        fast.argreduce_logprobs(*GOOD, FAKE, "1.0", *CALLS["argreduce_logprobs"][2:])
    with pytest.raises(OverflowError):
        fast.argreduce_logprobs(*GOOD, FAKE, 1.0, 1, 1 << 40, *CALLS["argreduce_logprobs"][4:])
    with pytest.raises(OverflowError):
        fast.argreduce_distill(*GOOD, 1 << 33, *CALLS["argreduce_distill"][1:])
    with pytest.raises(ValueError):
        fast.bind_logits(0, 0, 0, 0, 0, 0, 0)
    with pytest.raises(TypeError):
        fast.bind_logits(1)
    assert fast.argreduce_logprobs_scratch_bytes(1, 0, B.F32) == B.SIZE_MAX


def test_torch_functions_refuse_cpu_tensors():
    x, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    ids, v, w = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3), torch.zeros(2)
    with pytest.raises(ValueError, match="GPU"):
        ar.token_logprobs(x, t)
    with pytest.raises(ValueError, match="GPU"):
        ar.token_logprobs_grad(x, t, torch.zeros(4, 2), w)
    with pytest.raises(ValueError, match="GPU"):
        ar.distill_loss(x, ids, v)
    with pytest.raises(ValueError, match="GPU"):
        ar.distill_loss_grad(x, ids, v, torch.zeros(5, 2), w)
    with pytest.raises(ValueError, match="GPU"):
        ar.distill_step(x, ids, v, w)


def test_package_names():
    assert {"token_logprobs", "distill_step", "argmax"} <= set(dir(ar))
    assert ar.token_logprobs is ar.logits.token_logprobs
    with pytest.raises(AttributeError):
        ar.no_such_name
    text = open(B.LIB_PATH.replace("libargreduce.so", "../include/argreduce.h")).read()
    assert f"#define ARGREDUCE_TOP_MAX {ar.logits.TOP_MAX} " in text
    assert f"#define ARGREDUCE_TEACHER_MAX {ar.logits.TEACHER_MAX} " in text
    assert ctypes.sizeof(B.argreduce_plan_t) > 0


def test_the_stride_of_a_single_row_does_not_matter(lib):
    """Refused for what follows it (too many alternatives), not for a stride that nothing reads."""
    args = list((FAKE, B.F32, 1, 8, 1 << 40) + CALLS["argreduce_logprobs"])
    args[8] = 65
    assert lib.argreduce_logprobs(*args) == -1


def test_rows_times_columns_past_64_bits(lib):
    args = (FAKE, B.F32, INT32_MAX, INT32_MAX, INT32_MAX) + CALLS["argreduce_logprobs"]
    assert lib.argreduce_logprobs(*args) == -3


# (call, rows, cols, dtype, k) whose own launches hold fewer than 2^32 threads, though those of the
# gradient as a call of its own (the first two), or a workgroup or wavefront per row, would not
WIDE_BUT_FINE = [("argreduce_distill", 1 << 23, 4104, B.F32, 3), ("argreduce_distill", 1 << 28, 64, B.F16, 3),
                 ("argreduce_distill_step", 1 << 23, 4104, B.F32, 3),
                 ("argreduce_distill_step", 1 << 28, 64, B.F16, 3),
                 ("argreduce_distill_step", 1 << 26, 264, B.F16, 1),
                 ("argreduce_distill_step", 1 << 24, 5000, B.F16, 64),
                 ("argreduce_distill_step", 1 << 24, 264, B.BF16, 1024)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would run on these addresses")
@pytest.mark.parametrize("name,rows,cols,dtype,k", WIDE_BUT_FINE)
def test_a_call_is_refused_for_its_own_launches_only(lib, name, rows, cols, dtype, k):
    """Without a GPU such a call gets as far as its launch, which fails."""
    rest = (k,) + CALLS[name][1:]
    assert getattr(lib, name)(FAKE, dtype, rows, cols, cols, *rest) == -5
    assert B.argreduce_distill_scratch_bytes(rows, cols, dtype) == 0
    if name == "argreduce_distill":
        assert B.argreduce_distill_plan(rows, cols, dtype)["grid_blocks"] > 0


@pytest.mark.parametrize("rows,cols,stride,dtype", [(INT32_MAX, 1 << 20, 1 << 20, B.F32),
                                                    (1 << 15, 8, 1 << 31, B.F32), (1 << 16, 8, 1 << 31, B.BF16),
                                                    (INT32_MAX, 8, (1 << 32) - 1, B.F16)])
def test_logits_beyond_the_address_space(lib, rows, cols, stride, dtype):
    for name, rest in CALLS.items():
        assert getattr(lib, name)(FAKE, dtype, rows, cols, stride, *rest) == -3


def test_a_gradient_with_too_large_a_grid_is_refused(lib):
    for name in ("argreduce_logprobs_grad", "argreduce_distill_grad"):
        assert getattr(lib, name)(FAKE, B.F32, 1 << 23, 4104, 4104, *CALLS[name]) == -3


def test_the_fifth_row_of_statistics_is_named_alike():
    text = open(B.LIB_PATH.replace("libargreduce.so", "../include/argreduce.h")).read()
    import argmin_reduction_wide_amd.logits as L
    assert f"#define ARGREDUCE_ENTROPY_APART {L._ENTROPY_APART:#x}\n" in text


@pytest.mark.parametrize("requires_grad", [False, True])
def test_forward_mode_is_refused(requires_grad):
    """Logits with a tangent, also where autograd is off; without one, and after the level, the calls
    get as far as their other checks."""
    from torch.autograd import forward_ad

    x, t = torch.zeros(2, 8, requires_grad=requires_grad), torch.zeros(2, dtype=torch.int64)
    ids, v = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones(2, 8))
        for f in (lambda y: ar.token_logprobs(y, t), lambda y: ar.distill_loss(y, ids, v)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                f(dual)
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                f(dual)
            with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
                f(x)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        ar.token_logprobs(x, t)


def test_function_transforms_are_refused():
    t = torch.zeros(2, dtype=torch.int64)
    f = lambda y: ar.token_logprobs(y, t).logprob.sum()
    with pytest.raises(NotImplementedError, match="forward-mode"):
        torch.func.jvp(f, (torch.zeros(2, 8),), (torch.ones(2, 8),))
    for transform in (torch.func.grad(f), torch.func.jacfwd(f)):
        with pytest.raises((RuntimeError, ValueError)):
            transform(torch.zeros(2, 8))


def test_cpu_logits_that_require_a_gradient_are_refused_alike():
    """With or without a GPU in the machine: no HIP call comes before the refusal."""
    x, t = torch.zeros(2, 8, requires_grad=True), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        ar.token_logprobs(x, t)
    with pytest.raises(ValueError, match="GPU"):
        ar.distill_loss(x, t.view(2, 1), torch.zeros(2, 1))


@pytest.mark.parametrize("temperature", [1e39, -1e39, 1e300, float("inf"), float("nan"), 1e-300])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_temperatures_beyond_a_float_are_refused_by_status(lib, name, temperature):
    rest = list(CALLS[name])
    rest[1 if "logprobs" in name else 3] = temperature
    assert getattr(lib, name)(*GOOD, *rest) == -1
    assert getattr(B.fast(), name)(*GOOD, *rest) == -1
