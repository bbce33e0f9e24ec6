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


# ------------------------------------------------------------ gradient of renormalised weights

def differences(x, experts, dw, scoring, scale, e, h):
    """The derivative of sum w_j dw_j with respect to x[e] from two values of it; weights from logarithms
    of scores, which do not leave any range."""
    def value(v):
        l = v[experts] if scoring == "softmax" else -np.logaddexp(0, -v[experts])
        w = np.exp(l - l.max())
        return scale * (w / w.sum() * dw).sum()
    up, down = x.copy(), x.copy()
    up[e] += h
    down[e] -= h
    return (value(up) - value(down)) / (2 * h)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("level", [-80, -88, -92, -95, -100, -104, -110, -200, -700])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 6), (130, 12), (1024, 32)])
def test_grad_of_small_scores(dev, E, k, level, scoring, dtype):
    """Scores around and below fp32's smallest, 2^-126 and 2^-149, whose shares are ordinary numbers: all
    of a sigmoid's; a softmax's but the first expert's, which a bias keeps from being chosen."""
    rng = np.random.default_rng(E - level)
    T = 7
    x = level + rng.standard_normal((T, E))
    if scoring == "softmax":
        x[:, 0] = 0
    x = on(x, dev, dtype)
    bias = torch.ones(E)
    bias[0] = -1.0
    w, experts, _, _ = mm.route_topk(x, k, scoring=scoring, renormalize=True, scale=1.5, bias=bias.to(dev))
    assert bool((w.double().sum(dim=1) - 1.5).abs().max() <= 1e-6) and bool((experts > 0).all())
    dw = on(rng.standard_normal((T, k)), dev)
    got = mm.route_topk_grad(x, experts, dw, scoring=scoring, renormalize=True, scale=1.5)
    xh, eh, dh = x.cpu().double().numpy(), experts.cpu().numpy(), dw.cpu().double().numpy()
    want, size = gradient(xh, eh, dh, scoring, True, 1.5)
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= (E + 32) * U * size + half_step(want, DT[dtype]) + 1e-38).all()
    for t in (0, T - 1):
        for e in (0, eh[t, 0], eh[t, -1]):
            # a term h^2 |third derivative| <= 1e-8 size, and 2^-53 level / h of the values
            assert abs(differences(xh[t], eh[t], dh[t], scoring, 1.5, e, 1e-4) - want[t, e]) <= 1e-7 * max(1, size[t].max())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_grad_where_scores_vanish_or_are_none(dev, scoring):
    """Rows whose chosen scores are 0 in 64 bits too, whose weights then are 0; masked ones; NaN."""
    x = np.full((6, 10), -1000.0)
    x[:, 0] = 0 if scoring == "softmax" else -1000
    x[1] = -np.inf
    x[2, 2:] = -np.inf
    x[2, :2] = -95, -95.5
    x[4] = np.linspace(-1, 1, 10)
    x[5] = np.linspace(-1, 1, 10)
    x[5, 9] = np.nan
    experts = torch.tensor([[3, 4], [-1, -1], [1, -1], [1, 5], [7, 8], [9, 2]], dtype=torch.int32, device=dev)
    dw = torch.ones(6, 2, device=dev)
    dw[:, 0] = -2
    dw[4, 1] = float("nan")
    got = mm.route_topk_grad(on(x, dev), experts, dw, scoring=scoring, renormalize=True).cpu()
    assert bool((got[:4] == 0).all())  # one chosen expert's share is 1 whatever its logit
    assert bool(torch.isnan(got[4, 7:9]).all()) and bool(torch.isnan(got[5, [9, 2]]).all())
    if scoring == "softmax":
        assert bool(torch.isnan(got[4:]).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_grad_of_odd_experts_renormalised(dev, scoring):
    """Entries that are no expert add nothing; one that stands twice counts twice."""
    rng = np.random.default_rng(5)
    x = on(rng.standard_normal((3, 10)) - 100, dev)
    experts = torch.tensor([[-1, 4, 10], [2, 2, 7], [-5, 2 ** 30, -1]], dtype=torch.int32, device=dev)
    dw = on(rng.standard_normal((3, 3)), dev)
    got = mm.route_topk_grad(x, experts, dw, scoring=scoring, renormalize=True).cpu().double().numpy()
    want, size = gradient(x.cpu().double().numpy(), experts.cpu().numpy(), dw.cpu().double().numpy(), scoring, True, 1.0)
    assert (np.abs(got - want) <= 42 * U * size + 1e-38).all()


# ------------------------------------------------------------------ groups of a single expert

def routed_alone(x, k, scoring, bias, top_groups, renormalize):
    """experts and weights where each expert is a group, whose value is the sum of the one it has."""
    T, E = x.shape
    s = scores(x, scoring)
    experts, weights = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        c = s[t] + bias if bias is not None else x[t]
        dead = np.isneginf(x[t]) | np.isneginf(c)
        value = np.where(dead, -np.inf, c if bias is not None else s[t])
        kept = best_first(value)[:top_groups]
        c = np.where(dead | ~np.isin(np.arange(E), kept), -np.inf, c)
        order = [e for e in best_first(c) if not np.isneginf(c[e])][:k]
        experts[t, :len(order)] = order
        w = s[t][order]
        weights[t, :len(order)] = w / w.sum() if renormalize and w.sum() != 0 else w
    return experts, weights


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,top_groups,k", [(2, 1, 1), (12, 4, 2), (16, 3, 3), (17, 5, 4), (40, 30, 20), (64, 8, 8)])
def test_groups_of_one_expert(dev, E, top_groups, k, biased, scoring, dtype):
    rng = np.random.default_rng(E + k)
    x = rng.standard_normal((60, E)) * 1.5
    x[3] = -np.inf
    x[4, 1:] = -np.inf
    x[5] = 40 + np.arange(E) % 3  # a sigmoid of 1 in 64 bits: equal groups, the lower index first
    if scoring == "sigmoid":
        x[6, E // 2] = np.nan  # done in 64 bits throughout
        x[7, E - 1] = np.inf
    x = on(x, dev, dtype)
    bias = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)) if biased else None
    got = mm.route_topk(x, k, scoring=scoring, bias=bias.to(dev) if biased else None, groups=E, top_groups=top_groups,
                        group_top=2, renormalize=True)
    experts, weights = routed_alone(x.cpu().double().numpy(), k, scoring, bias.double().numpy() if biased else None,
                                    top_groups, True)
    assert np.array_equal(got[1].cpu().numpy(), experts)
    w = got[0].cpu().double().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(weights))
    assert (np.abs(w - weights) <= 2 * U * np.abs(weights) + 2.0 ** -150)[~np.isnan(weights)].all()
