"""Plans of beam search and expert routing on the host (CPU only) against what is launched: workgroups' sizes, the limit
of a launch's grid, and which path is reported for what."""
import pytest

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B

MI355X_THREADS = 256 * 2048
FAKE = 1 << 20  # an aligned, never-dereferenced address
ROUTE_THREADS = 512


@pytest.fixture
def lib():
    h = B.lib()
    B.argreduce_debug_set_capacity(MI355X_THREADS)
    yield h
    B.argreduce_debug_set_capacity(0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_route_plans_name_the_launch(lib, dtype):
    for experts in (1, 4, 8, 64, 256, 1000):
        for groups, tokens in [(1, 1), (1, 32), (3, 5000), (16, 4096), (300, 1000), (1, 2 ** 31 - 1), (2 ** 23 - 1, 1),
                               (2 ** 23 - 1, 200)]:
            p = B.argreduce_route_plan(groups, tokens, experts, dtype)
            assert p["block_threads"] == ROUTE_THREADS
            assert p["grid_blocks"] * p["block_threads"] < 1 << 32, (groups, tokens, experts)
            assert p["outputs_per_block"] == ROUTE_THREADS // p["lanes_per_row"]
            assert p["grid_rows"] == p["grid_blocks"] * p["outputs_per_block"]


@pytest.mark.parametrize("groups,tokens", [(2 ** 23, 1), (9_000_000, 1), (2 ** 23, 0), (2 ** 24 - 1, 100), (2 ** 31 - 1, 1)])
def test_routings_of_too_many_groups_are_refused(lib, groups, tokens):
    """Before anything is enqueued, in both directions and by both bindings."""
    with pytest.raises(ar.ArgreduceError) as e:
        B.argreduce_route_plan(groups, tokens, 8, "bf16")
    assert e.value.code == -3
    assert B.argreduce_route_scratch_bytes(groups, tokens, 8, "bf16") == B.SIZE_MAX
    route = (FAKE, B.BF16, groups, tokens, 8, 8, 0, 2, 0, FAKE, FAKE, FAKE, 0, 0, 0)
    grad = (FAKE, B.BF16, groups, tokens, 8, 8, 2, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0)
    for h in (lib, B.fast()):
        assert h.argreduce_route(*route) == -3
        assert h.argreduce_route_grad(*grad) == (-3 if tokens else 0)


def test_step_paths_are_what_the_header_says(lib):
    text = " ".join(open(B.LIB_PATH.replace("libargreduce.so", "../include/argreduce.h")).read().split()).replace("* ", "")
    at = text.index("The plan of argreduce_beam_step")
    text = text[at:text.index("*/", at)]
    for words in ("SUBWAVE (a wavefront per group of beams, four to a workgroup)", "block_threads 64 a wavefront per row",
                  "SPLIT (a workgroup per slice"):
        assert words in text
    p = B.argreduce_beam_plan(2048, 4, 64, "f16", 4)
    assert (p["path"], p["block_threads"], p["grid_blocks"], p["scratch_bytes"]) == (B.PATH_SUBWAVE, 256, 512, 0)
    assert p["outputs_per_block"] == 16  # rows of four groups
    p = B.argreduce_beam_plan(2000, 12, 1000, "f16", 12)
    assert (p["path"], p["block_threads"], p["grid_blocks"]) == (B.PATH_BLOCK, 64, 24000)
    p = B.argreduce_beam_plan(2000, 8, 6000, "f16", 8)
    assert (p["path"], p["block_threads"], p["grid_blocks"]) == (B.PATH_BLOCK, 64, 16000)
    p = B.argreduce_beam_plan(256, 8, 128256, "bf16", 8)
    assert (p["path"], p["block_threads"], p["grid_blocks"]) == (B.PATH_BLOCK, 512, 2048)
    p = B.argreduce_beam_plan(1, 8, 202048, "bf16", 16)
    assert p["path"] == B.PATH_SPLIT and p["grid_blocks"] == 8 * p["blocks_per_row"]
