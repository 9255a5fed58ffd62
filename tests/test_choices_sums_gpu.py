"""What the sums behind the choices lose: routing's totals where nothing but the joining of workgroups can round."""
import numpy as np
import pytest
import torch

import argmin_reduction_wide_amd as ar
import argmin_reduction_wide_amd.binding as B
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
INF = float("inf")


def sets(groups, tokens, experts, dtype):
    """How many sets of 64 workgroups a group's sums are joined from."""
    return -(-B.argreduce_route_plan(groups, tokens, experts, dtype)["grid_blocks"] // groups // 64)


@pytest.mark.parametrize("groups,tokens", [(1, 60000), (2, 30000), (3, 20000)])
def test_z_is_rounded_once(groups, tokens):
    """One expert is available to each token, its logit an odd number up to 255: z's terms are integers, and a
    workgroup's sum of up to 236 of them is below 2^24, so that it is exact. Between workgroups sums are in binary64,
    exact too, and the quotient by the number of tokens is rounded once more, to binary32."""
    announce(f"route z of [{groups},{tokens},8]")
    assert sets(groups, tokens, 8, "f32") > 1
    gen = torch.Generator(device="cuda").manual_seed(groups)
    for seed in range(8):
        value = 2 * torch.randint(0, 128, (groups, tokens, 1), device="cuda", generator=gen) + 1
        at = torch.randint(0, 8, (groups, tokens, 1), device="cuda", generator=gen)
        x = torch.full((groups, tokens, 8), -INF, device="cuda").scatter_(2, at, value.float())
        r = ar.route_experts(x, 1)
        total = value.square().sum(dim=(1, 2)).tolist()
        assert r.z.tolist() == [float(np.float32(t / tokens)) for t in total], seed


def test_balance_is_rounded_once():
    """A token's probability of expert 0 is 1 or 1 / 512, and all choose it. Of 2048 tokens to a workgroup the sum is a
    multiple of 1 / 512 of 21 bits, exact; of all of a group it has 27 bits, exact in binary64. Products and n^2 stay
    below 2^53, the quotient is rounded, and then the result."""
    groups, tokens, experts = 2, 1 << 18, 512
    announce(f"route balance of [{groups},{tokens},{experts}]")
    assert sets(groups, tokens, experts, "f16") > 1
    gen = torch.Generator(device="cuda").manual_seed(4)
    alone = torch.rand(groups, tokens, device="cuda", generator=gen) < 0.7
    x = torch.zeros(groups, tokens, experts, dtype=torch.float16, device="cuda")
    x[..., 1:].masked_fill_(alone[..., None], -INF)
    for seed in range(40):
        live = torch.rand(groups, tokens, device="cuda", generator=gen) < 0.9
        r = ar.route_experts(x, 1, live=live)
        n, ones = live.sum(1), (alone & live).sum(1)
        assert torch.equal(r.tokens, n) and torch.equal(r.counts[:, 0], n)
        # E / n^2 * n * (ones + (n - ones) / 512)
        want = [k * (o * experts + k - o) / (k * k) for k, o in zip(n.tolist(), ones.tolist())]
        assert r.balance.tolist() == [float(np.float32(v)) for v in want], seed
