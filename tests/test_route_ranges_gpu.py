"""Routing of tokens to experts where 32 bits do not hold what the choice or the gradient needs, against
the definitions in 64 bits: biases far larger than the scores, scores near and below fp32's smallest,
groups of a single expert. Bars as in test_experts_gpu.py.
"""
import numpy as np
import pytest
import torch

import tiled_gemm_gemv_amd as mm
from gpu_helpers import require_gpu
from test_experts_gpu import DT, U, best_first, check_route, gradient, half_step, scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    mm.load()
    return d


def on(a, dev, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DT[dtype]).to(dev)


# --------------------------------------------------------------------- groups, large biases

# the kernel for four tokens a wave, for one by groups, for one by experts
@pytest.mark.parametrize("T,E,groups,top_groups", [(3000, 32, 8, 4), (1500, 96, 32, 9), (700, 512, 8, 3), (5, 256, 16, 6)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [32.0, 1000.0, 1e5])
def test_groups_of_cancelling_biases(dev, T, E, groups, top_groups, scoring, size):
    """A group's two best have biases of opposite sign: their sum is that of the scores, which their
    rounding to fp32, 2^-24 of the bias each, may change by more than the sums are apart."""
    rng = np.random.default_rng(E + groups)
    x = on(0.3 + 1e-4 * rng.standard_normal((T, E)), dev)
    bias = np.full((groups, E // groups), -2 * size, np.float32)
    bias[0::2, 0], bias[0::2, 1] = size, -size
    bias[1::2, :2] = 0
    bias = torch.from_numpy(bias.reshape(-1))
    how = dict(scoring=scoring, groups=groups, top_groups=top_groups, group_top=2, renormalize=True)
    got = mm.route_topk(x, 2 * top_groups, bias=bias.to(dev), **how)
    check_route(x, got, bias=bias.double().numpy(), **how)


def test_groups_told_by_a_known_sum(dev):
    """Sums 1.0748106 and 1.0747726; of summands rounded to fp32, 1.0747681 and 1.0747726."""
    x = on([[0.03452131, 0.26628694, 0.8659476, -0.5284826]], dev)
    bias = torch.tensor([1000.0, -1000.0, 0.0, 0.0])
    how = dict(scoring="sigmoid", groups=2, top_groups=1, group_top=2)
    got = mm.route_topk(x, 2, bias=bias.to(dev), **how)
    assert got[1].tolist() == [[0, 1]]
    check_route(x, got, bias=bias.double().numpy(), **how)


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("top_groups", [1, 2, 3])
@pytest.mark.parametrize("E", [8, 34, 400])
def test_groups_past_the_range_of_32_bits(dev, E, top_groups, group_top):
    """Sums of two biases beyond the largest fp32 value, of either sign."""
    rng = np.random.default_rng(E)
    groups, per = (17, 2) if E == 34 else (4, E // 4)
    x = on(rng.standard_normal((20, E)), dev)
    bias = np.full((groups, per), -3.1e38)
    bias[:4, :2] = [[-3.0e38, -2.9e38], [-2.0e38, -2.1e38], [3.3e38, 3.0e38], [3.2e38, 3.3e38]]
    bias = torch.from_numpy(bias.reshape(-1).astype(np.float32))
    how = dict(scoring="sigmoid", groups=groups, top_groups=top_groups, group_top=group_top)
    got = mm.route_topk(x, 2, bias=bias.to(dev), **how)
    check_route(x, got, bias=bias.double().numpy(), **how)
