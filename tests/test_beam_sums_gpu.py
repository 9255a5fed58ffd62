"""The error of the logarithm of a beam's sum, which decides between close continuations of different beams."""
import numpy as np
import pytest
import torch

import argmin_reduction_wide_amd as ar
import choices_reference as C
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# groups, cols of the step's kernels: a wavefront per group; per row; slices that join; one pass by 64 lanes, by a
# workgroup, and in slices
PATHS = [(3000, 64), (3000, 1000), (200, 32000), (3, 32000), (5000, 6000), (2000, 40000), (100, 202048)]


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("groups,cols", PATHS)
def test_error_of_a_beams_sum(dtype, groups, cols):
    """A score that is -ln p of the best token leaves a value next to 0, where binary32 is fine: the result is the error
    of ln s. Every row is within the derived bound (choices_reference.py). Independent roundings, one of 2^-24 / sqrt 3
    for each addition, leave 2^-24 sqrt(2 / 3) from the last ones (those of 2, 4, 8 ... lanes average out) and as
    much again from the terms and the merges: less than 2^-23 in the root of the mean square."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    errors, worst = [], 0.0
    while sum(len(e) for e in errors) < 200:
        x = (torch.randn(groups, 1, cols, device="cuda", generator=gen) * 2.5).to(DT[dtype])
        for temperature in (1.0, 0.7):
            z = x.double() / temperature
            z -= z.amax(-1, keepdim=True)
            p = z.exp()
            s = p.sum(-1)
            scores = s.log().float()
            r = ar.beam_step(x, scores, 1, temperature=temperature)
            e = (r.scores.double() - (scores.double() - s.log())).flatten()
            mean = -(p * z).sum(-1).div(s).flatten()
            bound = C.U * (3 * mean / np.log(2.0) + C.R.adds(cols) + 2) + 1e-14
            worst = max(worst, (e.abs() / bound).max().item())
            errors.append(e)
            del z, p
    e = torch.cat(errors)
    announce(f"beam_step {dtype} [{groups},1,{cols}]: ln s off by {e.square().mean().sqrt().item():.2e} (root of the mean "
             f"square), {e.mean().item():.2e} (mean), {e.abs().max().item():.2e} at most, {worst:.3f} of the bound")
    assert worst <= 1.0
    assert e.square().mean().sqrt().item() < 2.0 ** -23
