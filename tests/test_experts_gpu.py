"""GPU parity of the routing of tokens to experts, its gradient, and the tokens' rows to the experts'
order and back, against their definitions in 64 bits; and a layer of experts made of them.

Bars, from the number formats:
* Experts, rows and offsets are equal: the choice is made in 64 bits on both sides, and equal values
  go to the lower index. (Two scores that differ by less than 2^-50 of themselves could fall either
  way; the inputs' spacing, 2^-24 and more, keeps them apart.)
* Weights are 64-bit values rounded to fp32, a scale of fp32: within 2^-24 of the value, one more for
  the order of the sums. A softmax that is not renormalised divides by a sum of fp32 exponentials:
  each off by 2^-23 (one unit) and, from its argument l - m rounded to fp32, by |l - m| 2^-24; weighted
  by the softmax p the latter add up to sum p (m - l) <= log E <= 7 (the entropy is at most log E) of
  2^-24; with the additions, log2 E + 6 + E / 64 of at most 2^-24 each, at most 32 in all.
* The logits' gradient is computed in fp32 from sums of up to E terms, each off by a few 2^-24: within
  (E + 32) 2^-24 of the sum of the terms' magnitudes, and half a step of the output type.
* Rows: copies are equal; sums of k products in fp32 within (k + 1) 2^-24 of the sum of magnitudes, dot
  products of D within (D + 1) 2^-24 of it, single products one rounding; plus half a step of the
  output type, eps / 2 of the value (fp16 also 2^-25).
"""
import numpy as np
import pytest
import torch

import tiled_gemm_gemv_amd as mm
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    mm.load()
    return d


def half_step(values, dtype):
    if dtype == torch.float32:
        return np.abs(values) * U
    half = np.abs(values) * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -8)
    return half + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def scores(x, scoring):
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1 / (1 + np.exp(-x))
        m = x.max(axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0, m)
        e = np.exp(x - m)
        total = e.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0, e / np.where(total == 0, 1, total))


def best_first(v):
    """Indices by falling value, NaN first, equal ones by index (a list of one token's values)."""
    return sorted(range(len(v)), key=lambda e: (0, 0, e) if np.isnan(v[e]) else (1, -v[e], e))


def routed(x, k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=False, scale=1.0):
    """weights, experts, rows and offsets from the definition; x float64."""
    T, E = x.shape
    s = scores(x, scoring)
    weights, experts = np.zeros((T, k)), np.full((T, k), -1)
    for t in range(T):
        c = s[t] + bias if bias is not None else x[t].copy()
        dead = np.isneginf(x[t]) | np.isneginf(c)
        c = np.where(dead, -np.inf, c)
        if groups > 1:
            basis = c if bias is not None or group_top == 1 else np.where(dead, -np.inf, s[t])
            value = []
            for g in range(groups):
                part = basis[g * (E // groups):(g + 1) * (E // groups)]
                order = best_first(part)[:group_top]
                value.append(sum(part[i] for i in order) if len(order) == group_top else -np.inf)
            kept = best_first(np.array(value))[:top_groups]
            c = np.where(np.isin(np.arange(E) // (E // groups), kept), c, -np.inf)
        order = [e for e in best_first(c) if not np.isneginf(c[e])][:k]
        experts[t, :len(order)] = order
        w = s[t][order]
        if renormalize:
            w = w / w.sum() if w.sum() != 0 else 0 * w
        weights[t, :len(order)] = scale * w
    flat = [(e, i) for i, e in enumerate(experts.reshape(-1)) if e >= 0]
    rows = np.full(T * k, -1)
    for r, (_, i) in enumerate(sorted(flat)):
        rows[i] = r
    offsets = np.array([sum(1 for e, _ in flat if e < n) for n in range(E + 1)]) if E < 100 else \
        np.concatenate([[0], np.cumsum(np.bincount([e for e, _ in flat], minlength=E))])
    return weights, experts, rows.reshape(T, k), offsets


def check_route(x, got, **how):
    k = got[0].shape[1]
    weights, experts, rows, offsets = routed(x.cpu().double().numpy(), k, **how)
    assert got[0].dtype == torch.float32 and got[1].dtype == got[2].dtype == torch.int32 and got[3].dtype == torch.int64
    assert np.array_equal(got[1].cpu().numpy(), experts)
    assert np.array_equal(got[2].cpu().numpy(), rows)
    assert np.array_equal(got[3].cpu().numpy(), offsets)
    w = got[0].cpu().double().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(weights))
    # below 2^-126 fp32 has steps of 2^-149 (sigmoid(-200) = 1.4e-87 rounds to 0): half of one
    units = 2 if how.get("renormalize") or how.get("scoring") == "sigmoid" or how.get("bias") is not None else 36
    assert (np.abs(w - weights) <= units * U * np.abs(weights) + 2.0 ** -150)[~np.isnan(weights)].all()


def logits_of(rng, T, E, dtype, dev, spread=1.5):
    return torch.from_numpy((rng.standard_normal((T, E)) * spread).astype(np.float32)).to(DT[dtype]).to(dev)


CASES = [
    (1, 1, 1, {}),
    (1, 64, 8, dict(renormalize=True)),
    (3, 5, 5, dict(scoring="sigmoid")),
    (7, 60, 6, {}),
    (8, 64, 1, dict(scoring="sigmoid", renormalize=True, scale=2.5)),
    (64, 65, 4, dict(renormalize=True)),
    (65, 8, 2, {}),
    (100, 128, 8, dict(groups=4, top_groups=2)),
    (130, 96, 6, dict(groups=8, top_groups=3, group_top=2)),
    (200, 256, 8, dict(scoring="sigmoid", groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5)),
    (63, 160, 6, dict(scoring="sigmoid", groups=5, top_groups=5, group_top=1)),
    (129, 12, 2, dict(groups=12, top_groups=4, group_top=2)),
    (33, 512, 10, {}),
    (17, 1000, 32, dict(scoring="sigmoid", renormalize=True)),
    (1, 1024, 32, dict(groups=64, top_groups=8, group_top=2)),
    (1500, 40, 3, dict(scoring="sigmoid")),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_route(dev, case, biased, dtype):
    T, E, k, how = CASES[case]
    rng = np.random.default_rng(case)
    x = logits_of(rng, T, E, dtype, dev)
    how = dict(how)
    bias = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32)) if biased else None
    got = mm.route_topk(x, k, bias=bias.to(dev) if biased else None, **how)
    check_route(x, got, bias=bias.double().numpy() if biased else None, **how)


@pytest.mark.parametrize("how", [{}, dict(scoring="sigmoid"), dict(groups=4, top_groups=2, group_top=2),
                                 dict(groups=4, top_groups=1, renormalize=True),
                                 dict(scoring="sigmoid", groups=4, top_groups=3, renormalize=True)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_ties_and_specials(dev, how, biased):
    """Rows that leave few or no experts, equal logits, infinities, NaN and values far apart."""
    E, k = 24, 6
    inf, nan = float("inf"), float("nan")
    rng = np.random.default_rng(4)
    x = logits_of(rng, 80, E, "f32", dev)
    x[0] = -inf
    x[1] = -inf
    x[1, 7] = 1.0
    x[2, 3:] = -inf
    x[3] = 0.5                       # all equal
    x[4, ::2] = 1.0
    x[4, 1::2] = -1.0
    x[5, 4], x[5, 9] = nan, nan
    x[6, 10] = nan
    x[6, :8] = -inf
    x[7] = torch.linspace(-60, 60, E, device=dev)
    x[8] = (torch.arange(E, device=dev) - 12) * 2e37
    x[9] = torch.finfo(torch.float32).min  # the type's lowest value is no mask
    x[10] = -200.0
    x[11] = 0.0
    x[11, ::3] = -0.0                # equal to 0
    x[12, 5] = inf
    x[70:] = -inf
    bias = None
    if biased:
        bias = torch.zeros(E)
        bias[2], bias[11] = -inf, 0.25
    got = mm.route_topk(x, k, bias=None if bias is None else bias.to(dev), **how)
    check_route(x, got, bias=None if bias is None else bias.double().numpy(), **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_large(dev, dtype):
    """Many workgroups, some experts much liked, padded tokens at the end; strided logits."""
    T, E, k = 5000, 128, 8
    rng = np.random.default_rng(11)
    whole = logits_of(rng, T, E + 9, dtype, dev)
    x = whole[:, 5:5 + E]
    x[:, 17] += 6
    x[4500:] = -float("inf")
    how = dict(scoring="sigmoid", groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5)
    bias = torch.from_numpy((0.05 * rng.standard_normal(E)).astype(np.float32))
    got = mm.route_topk(x, k, bias=bias.to(dev), **how)
    check_route(x, got, bias=bias.double().numpy(), **how)
    work = mm.route_topk_workspace(T, E, k, dev)
    assert work.numel() == mm.mm_route_topk_workspace_bytes(T, E, k) > 0
    again = mm.route_topk(x, k, bias=bias.to(dev), workspace=work, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    with pytest.raises(mm.MMError, match="workspace smaller"):
        mm.route_topk(x, k, workspace=work[:16])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = mm.route_topk(x, k, bias=bias.to(dev), stream=side, **how)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, other))


@pytest.mark.parametrize("how", [{}, dict(scoring="sigmoid", groups=4, top_groups=2, group_top=2)])
def test_route_close_scores(dev, how):
    """Neighbouring fp32 logits: scores a few 2^-25 apart, which fp32 sums do not tell."""
    T, E, k = 300, 64, 8
    rng = np.random.default_rng(12)
    base = rng.standard_normal((T, 1)).astype(np.float32)
    steps = rng.integers(-3, 4, (T, E))
    x = np.where(steps > 0, np.nextafter(base, np.float32(9)), np.where(steps < 0, np.nextafter(base, np.float32(-9)), base))
    x = torch.from_numpy(np.ascontiguousarray(x.astype(np.float32))).to(dev)
    bias = torch.zeros(E)
    got = mm.route_topk(x, k, bias=bias.to(dev), **how)
    check_route(x, got, bias=bias.double().numpy(), **how)


def test_route_empty(dev):
    for T, E, k in ((0, 8, 2), (5, 8, 0), (0, 0, 0), (3, 0, 0)):
        w, e, r, o = mm.route_topk(torch.randn(T, E, device=dev), k)
        assert w.shape == e.shape == r.shape == (T, k)
        assert o.shape == (E + 1,) and bool((o == 0).all())
        g = mm.route_topk_grad(torch.randn(T, E, device=dev), e, w)
        assert g.shape == (T, E) and bool((g == 0).all())


# ------------------------------------------------------------------------------- gradient

def gradient(x, experts, dw, scoring, renormalize, scale):
    """(dlogits, the sum of its terms' magnitudes) from the definition, float64."""
    T, E = x.shape
    s = scores(x, scoring)
    d, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        g, gs = np.zeros(E), np.zeros(E)
        slots = [j for j, e in enumerate(experts[t]) if 0 <= e < E]
        total = sum(s[t][experts[t][j]] for j in slots)
        for j in slots:
            e = experts[t][j]
            if renormalize:
                if total != 0:
                    mean = sum(dw[t][i] * s[t][experts[t][i]] / total for i in slots)
                    big = sum(abs(dw[t][i]) * s[t][experts[t][i]] / total for i in slots)
                    g[e] += scale * (dw[t][j] - mean) / total
                    gs[e] += abs(scale) * (abs(dw[t][j]) + big) / total
            else:
                g[e] += scale * dw[t][j]
                gs[e] += abs(scale * dw[t][j])
        if scoring == "sigmoid":
            d[t], size[t] = s[t] * (1 - s[t]) * g, s[t] * (1 - s[t]) * gs
        else:
            d[t] = s[t] * (g - (s[t] * g).sum())
            size[t] = s[t] * (gs + (s[t] * gs).sum())
    return d, size


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (5, 60, 6), (67, 130, 4), (3, 1024, 32), (9, 300, 1)])
def test_route_grad(dev, T, E, k, renormalize, scoring, dtype):
    rng = np.random.default_rng(T + E + k)
    whole = logits_of(rng, T, E + 3, dtype, dev)
    x = whole[:, 2:2 + E]
    if T > 4:
        x[1] = -float("inf")
        x[2, 2:] = -float("inf")
    w, experts, _, _ = mm.route_topk(x, k, scoring=scoring, renormalize=renormalize, scale=1.5)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(dev)
    got = mm.route_topk_grad(x, experts, dw, scoring=scoring, renormalize=renormalize, scale=1.5)
    assert got.dtype == x.dtype
    d, size = gradient(x.cpu().double().numpy(), experts.cpu().numpy(), dw.cpu().double().numpy(), scoring, renormalize, 1.5)
    err = np.abs(got.cpu().double().numpy() - d)
    assert (err <= (E + 32) * U * size + half_step(d, DT[dtype]) + 1e-38).all()
    # the formula against differences of the definition's weights, at one token
    t, h = T // 2, 1e-6
    base = x.cpu().double().numpy()[t:t + 1]
    chosen = [j for j in range(k) if experts[t, j] >= 0]
    for e in ([0, E // 2, E - 1] + [int(experts[t, j]) for j in chosen[:2]]):
        if np.isneginf(base[0, e]):
            continue
        sides = []
        for sign in (1, -1):
            v = base.copy()
            v[0, e] += sign * h
            s = scores(v, scoring)[0]
            wv = np.array([s[int(experts[t, j])] for j in chosen])
            wv = 1.5 * (wv / wv.sum() if renormalize else wv)
            sides.append((wv * dw[t].cpu().double().numpy()[chosen]).sum())
        assert abs((sides[0] - sides[1]) / (2 * h) - d[t, e]) <= 1e-8 + 1e-6 * size[t, e]


def test_route_grad_odd_experts(dev):
    """Entries that are no expert add nothing; one that stands twice counts twice."""
    x = torch.randn(3, 10, device=dev)
    experts = torch.tensor([[-1, 4, 10], [2, 2, 7], [-5, 2 ** 30, -1]], dtype=torch.int32, device=dev)
    dw = torch.randn(3, 3, device=dev)
    for scoring in ("softmax", "sigmoid"):
        got = mm.route_topk_grad(x, experts, dw, scoring=scoring).cpu().double().numpy()
        d, size = gradient(x.cpu().double().numpy(), experts.cpu().numpy(), dw.cpu().double().numpy(), scoring, False, 1.0)
        assert (np.abs(got - d) <= 42 * U * size + 1e-38).all()


# ----------------------------------------------------------------------------------- rows

def slots_of(rng, T, k, total, dev):
    """Random distinct rows below total, some slots without one (-1 and beyond the rows)."""
    rows = rng.permutation(max(total, T * k))[:T * k].astype(np.int32)
    rows[rng.random(T * k) < 0.1] = -1
    return torch.from_numpy(rows.reshape(T, k)).to(dev)


ROWS = [(1, 1, 1, 1), (2, 3, 6, 7), (5, 2, 8, 64), (8, 8, 64, 4096), (3, 9, 40, 130), (17, 4, 68, 2049), (70, 1, 70, 100),
        (33, 6, 250, 777), (4, 32, 128, 5000), (300, 3, 850, 512), (130, 2, 260, 513), (1000, 9, 9000, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "i8", "u8"])
@pytest.mark.parametrize("T,k,total,D", ROWS)
def test_spread(dev, T, k, total, D, dtype):
    rng = np.random.default_rng(T + D)
    rows = slots_of(rng, T, k, total, dev)
    t = {"i8": torch.int8, "u8": torch.uint8}.get(dtype) or DT[dtype]
    for gap, offset in ((0, 0), (3, 1)):
        flat = torch.from_numpy(rng.integers(-100 if t != torch.uint8 else 0, 100, T * (D + gap) + offset)).to(t).to(dev)
        x = torch.as_strided(flat, (T, D), (D + gap, 1), offset)
        buf = torch.full((total * (D + gap) + offset + 9,), 101, dtype=t, device=dev)
        out = torch.as_strided(buf, (total, D), (D + gap, 1), offset)
        assert mm.spread_rows(x, rows, out=out) is out
        want = np.full((total, D), 101.0)
        for i, r in enumerate(rows.cpu().numpy().reshape(-1)):
            if 0 <= r < total:
                want[r] = x[i // k].cpu().double().numpy()
        assert np.array_equal(out.cpu().double().numpy(), want)
        out.fill_(101)
        assert bool((buf == 101).all())
    if rows.min() >= 0 and total == T * k:
        assert torch.equal(mm.spread_rows(x, rows)[rows[0, 0].long()], x[0])


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,total,D", ROWS)
def test_combine(dev, T, k, total, D, weighted, dtype, out):
    rng = np.random.default_rng(T + D + 1)
    rows = slots_of(rng, T, k, total, dev)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(dev) if weighted else None
    whole = logits_of(rng, total, D + 5, dtype, dev)
    y = whole[:, 3:3 + D]
    buf = torch.full((T, D + 7), float("nan"), dtype=DT[out], device=dev)
    mm.combine_rows(y, rows, w, out=buf[:, 1:1 + D])
    got = buf[:, 1:1 + D].cpu().double().numpy()
    v, r = y.cpu().double().numpy(), rows.cpu().numpy()
    want, size = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j in range(k):
            if 0 <= r[t, j] < total:
                c = float(w[t, j]) if weighted else 1.0
                want[t] += c * v[r[t, j]]
                size[t] += np.abs(c * v[r[t, j]])
    assert (np.abs(got - want) <= (k + 1) * U * size + half_step(want, DT[out]) * (1 + 2.0 ** -8)).all()
    assert bool(torch.isnan(buf[:, 0]).all()) and bool(torch.isnan(buf[:, 1 + D:]).all())


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,k,total,D", ROWS)
def test_combine_grad(dev, T, k, total, D, dtype, grad):
    rng = np.random.default_rng(T + D + 2)
    rows = slots_of(rng, T, k, total, dev)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(dev)
    y = logits_of(rng, total, D + 5, dtype, dev)[:, 3:3 + D]
    g = logits_of(rng, T, D + 1, grad, dev)[:, 1:]
    buf = torch.full((total, D + 7), float("nan"), dtype=DT[dtype], device=dev)
    dy, dw = mm.combine_rows_grad(g, y, rows, w, out=buf[:, 1:1 + D])
    v, r, gv, wv = y.cpu().double().numpy(), rows.cpu().numpy(), g.cpu().double().numpy(), w.cpu().double().numpy()
    want, dwant, size = np.full((total, D), np.nan), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= r[t, j] < total:
                want[r[t, j]] = wv[t, j] * gv[t]
                dwant[t, j] = v[r[t, j]] @ gv[t]
                size[t, j] = np.abs(v[r[t, j]]) @ np.abs(gv[t])
    got = dy.cpu().double().numpy()
    live = ~np.isnan(want)
    assert np.isnan(got[~live]).all()
    assert (np.abs(got - want)[live] <= (U * np.abs(want) + half_step(want, DT[dtype]) * (1 + 2.0 ** -8))[live]).all()
    assert (np.abs(dw.cpu().double().numpy() - dwant) <= (D + 1) * U * size).all()
    assert bool(torch.isnan(buf[:, 0]).all()) and bool(torch.isnan(buf[:, 1 + D:]).all())


@pytest.mark.parametrize("D", [2 ** 31 - 1, 2 ** 31 - 9])
def test_longest_rows(dev, D):
    """One token's row of 2^31 - 1 elements (and one whose last 8 are whole) and back, and its
    gradients; what lies behind stays as it is. Values and sums are exact."""
    x = torch.zeros((1, D), dtype=torch.bfloat16, device=dev)
    x[0, :70] = torch.arange(70, device=dev)
    x[0, -70:] = -torch.arange(70, device=dev).to(torch.bfloat16)
    rows = torch.tensor([[0]], dtype=torch.int32, device=dev)
    w = torch.full((1, 1), 0.5, device=dev)
    out = torch.full((D + 16,), 3.0, dtype=torch.bfloat16, device=dev)
    place = out[:D].view(1, D)

    def check(factor):
        assert torch.equal(place[0, :200], x[0, :200] * factor) and torch.equal(place[0, -200:], x[0, -200:] * factor)
        assert int((place != 0).sum()) == 138 and bool((out[D:] == 3).all())
        place.fill_(3)

    mm.spread_rows(x[:, :D // 2], rows, out=place[:, :D // 2])
    assert torch.equal(place[0, :D // 2], x[0, :D // 2]) and bool((place[0, D // 2:] == 3).all())  # 2^31 - 1 bytes at most
    mm.combine_rows(x, rows, out=place)
    check(1)
    mm.combine_rows(x, rows, w, out=place)
    check(0.5)
    _, dw = mm.combine_rows_grad(x, x, rows, w, out=place)
    check(0.5)
    assert dw.item() == 2 * sum(i * i for i in range(70))


def test_rows_empty(dev):
    rows = torch.zeros(0, 4, dtype=torch.int32, device=dev)
    assert mm.spread_rows(torch.zeros(0, 8, device=dev), rows).shape == (0, 8)
    assert mm.combine_rows(torch.zeros(0, 8, device=dev), rows).shape == (0, 8)
    none = torch.full((3, 2), -1, dtype=torch.int32, device=dev)
    w = torch.ones(3, 2, device=dev)
    assert bool((mm.combine_rows(torch.ones(0, 8, device=dev), none, w) == 0).all())
    assert bool((mm.combine_rows(torch.ones(4, 8, device=dev), none, w) == 0).all())
    assert bool((mm.combine_rows(torch.ones(4, 8, device=dev), none[:, :0].contiguous()) == 0).all())
    dy, dw = mm.combine_rows_grad(torch.ones(3, 8, device=dev), torch.ones(4, 8, device=dev), none, w,
                                  out=torch.full((4, 8), 7.0, device=dev))
    assert bool((dy == 7).all()) and bool((dw == 0).all())
    assert mm.combine_rows_grad(torch.ones(3, 0, device=dev), torch.ones(4, 0, device=dev), none, w)[1].eq(0).all()


# ---------------------------------------------------------------------- a layer of experts

def layer16(x, logits, w1, w2, k, how):
    """A layer of experts in 16 bits, its intermediate values kept for the backward pass."""
    weights, experts, rows, offsets = mm.route_topk(logits, k, **how)
    xs = mm.spread_rows(x, rows, out=torch.zeros(x.shape[0] * k, x.shape[1], dtype=x.dtype, device=x.device))
    h = mm.gemm16_grouped(xs, w1, offsets, out=torch.zeros(xs.shape[0], w1.shape[2], dtype=x.dtype, device=x.device))
    y = mm.gemm16_grouped(h, w2, offsets, out=torch.zeros(xs.shape[0], w2.shape[2], dtype=x.dtype, device=x.device))
    return (weights, experts, rows, offsets, xs, h, y), mm.combine_rows(y, rows, weights)


def test_layer_of_experts_trains(dev):
    """Router, spread, two grouped products and combine, forward and backward, against autograd of the
    definition in 64 bits. bf16 values are rounded between the products: half a step each, 2^-9 of the
    largest value, and sums average it; five roundings in a row stay within 2^-6 of the largest."""
    T, E, k, D, H = 50, 8, 2, 64, 96
    rng = np.random.default_rng(21)
    how = dict(scoring="softmax", renormalize=True, scale=1.0)
    x = logits_of(rng, T, D, "bf16", dev, 1.0)
    logits = logits_of(rng, T, E, "f32", dev)
    logits[-3:] = -float("inf")  # padded tokens
    w1, w2 = logits_of(rng, E * D, H, "bf16", dev, 0.1).view(E, D, H), logits_of(rng, E * H, D, "bf16", dev, 0.1).view(E, H, D)
    dout = logits_of(rng, T, D, "bf16", dev, 1.0)
    (weights, experts, rows, offsets, xs, h, y), out = layer16(x, logits, w1, w2, k, how)
    dy, dweights = mm.combine_rows_grad(dout, y, rows, weights, out=torch.zeros_like(y))
    dw2 = mm.gemm16_grouped_grad_b(h, dy, offsets)
    dh = mm.gemm16_grouped(dy, w2, offsets, trans_b=True, out=torch.zeros_like(h))
    dw1 = mm.gemm16_grouped_grad_b(xs, dh, offsets)
    dxs = mm.gemm16_grouped(dh, w1, offsets, trans_b=True, out=torch.zeros_like(xs))
    dx = mm.combine_rows(dxs, rows)
    dlogits = mm.route_topk_grad(logits, experts, dweights, **how)

    leaves = [v.cpu().double().requires_grad_() for v in (x, logits[:-3], w1, w2)]
    X, L, W1, W2 = leaves
    p = torch.softmax(L, dim=1)
    chosen = experts[:-3].cpu().long()
    w = p.gather(1, chosen)
    w = w / w.sum(dim=1, keepdim=True)
    want = torch.zeros(T, D, dtype=torch.float64)
    parts = []
    for t in range(T - 3):
        parts.append(sum(w[t, j] * (X[t] @ W1[chosen[t, j]] @ W2[chosen[t, j]]) for j in range(k)))
    want = torch.cat([torch.stack(parts), torch.zeros(3, D, dtype=torch.float64)])
    grads = torch.autograd.grad(want, leaves, dout.cpu().double())
    for name, got, ref in (("out", out, want), ("dx", dx, grads[0]), ("dlogits", dlogits[:-3], grads[1]),
                           ("dw1", dw1, grads[2]), ("dw2", dw2, grads[3])):
        err = (got.cpu().double() - ref.detach()).abs().max()
        assert err <= 2.0 ** -6 * ref.detach().abs().max(), (name, float(err), float(ref.detach().abs().max()))
    assert bool((out[-3:] == 0).all()) and bool((dx[-3:] == 0).all()) and bool((dlogits[-3:] == 0).all())


def test_layer_of_4_bit_experts(dev):
    """Router, 4-bit rows spread by code and scale, two grouped 4-bit products and combine: bit for bit
    what the parts give from the definitions' values (sums of 4-bit products within 1e-5)."""
    T, E, k, D, H = 30, 16, 4, 128, 192
    rng = np.random.default_rng(22)
    x = logits_of(rng, T, D, "bf16", dev, 1.0)
    logits = logits_of(rng, T, E, "bf16", dev)
    how = dict(scoring="sigmoid", renormalize=True, scale=2.0)
    weights, experts, rows, offsets = mm.route_topk(logits, k, **how)
    w = [mm.quantize_mx4(logits_of(rng, E * n, m, "f32", dev, 0.1)) for n, m in ((H, D), (D, H))]
    (b1, s1), (b2, s2) = [(q.view(E, n, m // 2), s.view(E, n, m // 32)) for (q, s), (n, m) in zip(w, ((H, D), (D, H)))]
    q, s = mm.quantize_mx4(x)
    qs, ss = mm.spread_rows(q, rows), mm.spread_rows(s, rows)
    h = mm.gemm_mx4_grouped(qs, b1, offsets, ss, s1)
    hq, hs = mm.quantize_mx4(h)
    y = mm.gemm_mx4_grouped(hq, b2, offsets, hs, s2)
    out = mm.combine_rows(y, rows, weights).cpu().double().numpy()
    x4 = mm.dequantize_mx4(q, s).cpu().double().numpy()
    v1 = mm.dequantize_mx4(b1.reshape(-1, D // 2), s1.reshape(-1, D // 32)).view(E, H, D).cpu().double().numpy()
    v2 = mm.dequantize_mx4(b2.reshape(-1, H // 2), s2.reshape(-1, H // 32)).view(E, D, H).cpu().double().numpy()
    h4 = mm.dequantize_mx4(hq, hs).cpu().double().numpy()
    r, e, c = rows.cpu().numpy(), experts.cpu().numpy(), weights.cpu().double().numpy()
    for t in range(T):
        want, size = np.zeros(D), np.zeros(D)
        for j in range(k):
            hv = x4[t] @ v1[e[t, j]].T
            assert (np.abs(h[r[t, j]].cpu().double().numpy() - hv) <= 1e-5 * (np.abs(x4[t]) @ np.abs(v1[e[t, j]]).T)).all()
            want += c[t, j] * (h4[r[t, j]] @ v2[e[t, j]].T)
            size += c[t, j] * (np.abs(h4[r[t, j]]) @ np.abs(v2[e[t, j]]).T)
        assert (np.abs(out[t] - want) <= 1.1e-5 * size).all()


def test_layer_captured_and_replayed(dev):
    """The layer's forward and backward in a graph, with eager work and waits between the replays."""
    T, E, k, D, H = 200, 16, 4, 64, 64
    rng = np.random.default_rng(23)
    how = dict(scoring="sigmoid", renormalize=True, scale=1.0)
    x, logits = logits_of(rng, T, D, "bf16", dev), logits_of(rng, T, E, "f32", dev)
    w1, w2 = logits_of(rng, E * D, H, "bf16", dev, 0.1).view(E, D, H), logits_of(rng, E * H, D, "bf16", dev, 0.1).view(E, H, D)
    dout = logits_of(rng, T, D, "bf16", dev)

    def step():
        (weights, experts, rows, offsets, xs, h, y), out = layer16(x, logits, w1, w2, k, how)
        dy, dweights = mm.combine_rows_grad(dout, y, rows, weights, out=torch.zeros_like(y))
        return out, rows, offsets, dy, dweights, mm.route_topk_grad(logits, experts, dweights, **how)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same call do not share what they work in
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = step()
        graphs.append((graph, result))
    for i in range(4):
        x.copy_(logits_of(rng, T, D, "bf16", dev))
        logits.copy_(logits_of(rng, T, E, "f32", dev))
        for graph, _ in graphs:
            graph.replay()
        want = step()
        torch.cuda.synchronize()
        for _, result in graphs:
            assert all(torch.equal(a, b) for a, b in zip(result, want)), i


# --------------------------------------------------------- sizes at the kernels' borders, far rows

@pytest.mark.parametrize("T,E,k,how", [
    (17, 64, 4, {}), (40, 200, 12, dict(renormalize=True)), (64, 33, 5, dict(scoring="sigmoid")),
    (50, 256, 13, {}), (50, 257, 8, {}), (70, 256, 12, dict(groups=16, top_groups=5, group_top=2)),
    (70, 136, 6, dict(groups=17, top_groups=3, group_top=2)), (1025, 48, 3, dict(renormalize=True)),
    (8192, 16, 2, {}), (8193, 16, 2, {}), (8200, 300, 2, {}), (9001, 130, 2, dict(groups=2)), (1000, 700, 3, {}),
    (16, 256, 8, {}), (17, 129, 7, {}), (64, 256, 8, dict(scoring="sigmoid", groups=8, top_groups=4, group_top=2)),
    (64, 128, 9, {}), (65, 128, 9, {})])
@pytest.mark.parametrize("biased", [False, True])
def test_route_borders(dev, T, E, k, how, biased):
    """Sizes on both sides of where another kernel or another number of launches takes over."""
    rng = np.random.default_rng(T + E)
    x = logits_of(rng, T, E, "f32", dev)
    x[T - T // 9:] = -float("inf")
    bias = torch.from_numpy((0.05 * rng.standard_normal(E)).astype(np.float32)) if biased else None
    got = mm.route_topk(x, k, bias=bias.to(dev) if biased else None, **how)
    check_route(x, got, bias=bias.double().numpy() if biased else None, **how)


@pytest.mark.parametrize("E", [100, 600])
@pytest.mark.parametrize("biased", [False, True])
def test_route_many_alike(dev, E, biased):
    """More experts next to the border than a token's candidates have room for, all equal or nearly:
    those tokens among others."""
    rng = np.random.default_rng(E)
    T, k = 90, 6
    x = rng.standard_normal((T, E)).astype(np.float32)
    x[::7] = 0.75
    near = np.nextafter(np.float32(0.75), np.float32(1)) if not biased else np.float32(0.75) + np.float32(2.0 ** -20)
    x[3::7] = np.where(rng.random((x[3::7].shape)) < 0.5, np.float32(0.75), near)
    x = torch.from_numpy(x).to(dev)
    bias = torch.zeros(E) if biased else None
    for how in (dict(scoring="sigmoid", renormalize=True), dict(groups=E // 50, top_groups=1, group_top=2, renormalize=True)):
        got = mm.route_topk(x, k, bias=bias.to(dev) if biased else None, **how)
        check_route(x, got, bias=bias.double().numpy() if biased else None, **how)


def test_rows_past_32_bits(dev):
    """Rows that start past 2^32 bytes."""
    D, total = 40000, 60000
    y = torch.zeros((total, D), dtype=torch.bfloat16, device=dev)
    rows = torch.tensor([[total - 1, 3], [-1, total - 2], [57000, total]], dtype=torch.int32, device=dev)
    x = torch.randn(3, D, device=dev).to(torch.bfloat16)
    mm.spread_rows(x, rows, out=y)
    w = torch.tensor([[1.0, 2.0], [4.0, 0.5], [-1.0, 8.0]], device=dev)
    out = mm.combine_rows(y, rows, w, out_dtype=torch.float32)
    assert torch.equal(out, x.float() * torch.tensor([[3.0], [0.5], [-1.0]], device=dev))
    dy, dw = mm.combine_rows_grad(x, y, rows, w, out=y.clone())
    for t, j, r in ((0, 0, total - 1), (0, 1, 3), (1, 1, total - 2), (2, 0, 57000)):
        assert torch.equal(dy[r], (x[t].float() * w[t, j]).to(torch.bfloat16))
    assert dw[1, 0] == 0 and dw[2, 1] == 0 and float(dw[0, 0]) > 0


def test_two_streams_at_once(dev):
    """The same calls on two streams side by side, each with a workspace of its own."""
    rng = np.random.default_rng(31)
    xs = [logits_of(rng, 3000, 96, "f32", dev) for _ in range(2)]
    how = dict(scoring="sigmoid", renormalize=True)
    want = [mm.route_topk(x, 6, **how) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(mm.route_topk(xs[i], 6, **how))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
