"""Every kernel of the 4-bit products, by name (asked of the library for the operands that the call
then gets), with K-steps even and odd in number, whole and partial; operands past 32 bits; and the
most rows there can be. Codes stand in buffers of other codes and scales among 255s, in whole words or
at odd bytes, since the choice depends on that.

Bars as in test_mx4_gpu.py, from the number formats.
"""
import os

import numpy as np
import pytest
import torch

import tiled_gemm_gemv_amd as mm
from test_mx4_gpu import DT, check, inside, operand, values
from tiled_gemm_gemv_amd import build as mm_build

FAKE = 1 << 40  # never dereferenced

ROWS = [f"rows {r}x{c}" for r in (16, 32, 64) for c in (16, 32)]
TILES = ["tile 64x64 in 4", "tile 64x64 in 2", "tile 128x128", "tile 256x256"]

# (kernel, groups (0: the plain product), rows, N, K, codes' rows at odd bytes)
CASES = [
    ("rows 16x16", 0, 1, 1, 32, False),
    ("rows 16x16", 0, 13, 100, 4128, True),
    ("rows 16x16", 2, 3, 70, 1312, False),
    ("rows 16x32", 0, 244, 1526, 32, False),
    ("rows 16x32", 3, 422, 1546, 32, True),
    ("rows 32x16", 0, 323, 244, 32, False),
    ("rows 32x16", 40, 416, 3, 96, False),
    ("rows 32x16", 12, 148, 2, 320, True),
    ("rows 32x32", 0, 1007, 737, 160, False),
    ("rows 32x32", 13, 265, 2500, 128, True),
    ("rows 64x16", 0, 299, 1222, 32, True),
    ("rows 64x16", 2, 750, 527, 32, False),
    ("rows 64x32", 0, 982, 1508, 32, False),
    ("rows 64x32", 19, 419, 2438, 576, False),
    ("tile 64x64 in 4", 0, 69, 2755, 2144, False),
    ("tile 64x64 in 4", 0, 270, 1168, 800, True),
    ("tile 64x64 in 4", 0, 130, 1100, 4096, False),
    ("tile 64x64 in 4", 3, 527, 542, 2176, False),
    ("tile 64x64 in 4", 2, 224, 928, 1216, True),
    ("tile 64x64 in 2", 0, 1540, 485, 288, False),
    ("tile 64x64 in 2", 0, 587, 1197, 288, True),
    ("tile 64x64 in 2", 0, 700, 1000, 1280, False),
    ("tile 64x64 in 2", 8, 1652, 451, 352, False),
    ("tile 64x64 in 2", 53, 1079, 247, 256, True),
    ("tile 64x64 in 2", 0, 2478, 415, 32, False),
    ("tile 64x64 in 2", 55, 2118, 352, 64, False),
    ("tile 64x64 in 2", 29, 1589, 385, 224, True),
    ("tile 128x128", 0, 481, 1577, 256, False),
    ("tile 128x128", 0, 2000, 1300, 1024, False),
    ("tile 128x128", 0, 2000, 1300, 1312, True),
    ("tile 128x128", 15, 2860, 399, 256, False),
    ("tile 128x128", 4, 793, 745, 256, True),
    ("tile 128x128", 0, 851, 916, 32, True),
    ("tile 128x128", 7, 1831, 419, 32, False),
    ("tile 128x128", 3, 2726, 567, 32, False),
    ("tile 128x128", 0, 951, 1608, 160, False),
    ("tile 128x128", 2, 1013, 2660, 96, True),
    ("tile 256x256", 0, 2974, 2925, 544, False),
    ("tile 256x256", 0, 2858, 2911, 864, True),
    ("tile 256x256", 0, 3100, 2900, 256, False),
    ("tile 256x256", 0, 3100, 2900, 512, False),
    ("tile 256x256", 0, 3100, 2900, 768, False),
    ("tile 256x256", 0, 3100, 2900, 1024, False),
    ("tile 256x256", 0, 3100, 2900, 1312, False),
    ("tile 256x256", 16, 2811, 2712, 288, False),
    ("tile 256x256", 3, 3000, 3001, 1568, False),
    ("tile 256x256", 0, 2960, 2959, 64, False),
    ("tile 256x256", 0, 2991, 2925, 32, True),
    ("tile 256x256", 7, 2827, 2717, 96, False),
    ("tile 256x256", 22, 2935, 2210, 64, True),
]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mm_build.LIB):
        mm_build.build()
    return mm.load()


def selected(groups, M, N, K, a, lda, sa, ld_as, b, ldb, stride_b, sb, ld_bs, stride_bs):
    if groups == 0:
        cfg = mm.mm_gemm_mx4_select(M, N, K, a, lda, sa, ld_as, b, ldb, sb, ld_bs)
    else:
        cfg = mm.mm_gemm_mx4_grouped_select(groups, M, N, K, a, lda, sa, ld_as, b, ldb, stride_b, sb, ld_bs, stride_bs)
    return None if cfg < 0 else mm.mm_gemm_grouped_config_name(cfg)


def test_cases_cover_the_table():
    assert {c[0] for c in CASES} == set(ROWS + TILES)


def test_calls_without_a_kernel():
    assert selected(0, 0, 5, 64, FAKE, 32, FAKE, 2, FAKE, 32, 0, FAKE, 2, 0) is None       # no rows
    assert selected(0, 4, 5, 48, FAKE, 24, FAKE, 2, FAKE, 24, 0, FAKE, 2, 0) is None       # refused
    assert selected(0, 4, 5, 64, None, 32, FAKE, 2, FAKE, 32, 0, FAKE, 2, 0) is None
    assert selected(0, 4, 5, 64, FAKE, 32, FAKE, 1, FAKE, 32, 0, FAKE, 2, 0) is None
    assert selected(5000, 4, 5, 64, FAKE, 32, FAKE, 2, FAKE, 32, 160, FAKE, 2, 10) is None
    assert selected(0, 2 ** 31 - 1, 1, 32, FAKE, 16, FAKE, 1, FAKE, 16, 0, FAKE, 1, 0) == "any 64x64"


@pytest.fixture(scope="module")
def dev():
    from gpu_helpers import require_gpu
    return require_gpu()


def counts_of(groups, rows):
    """Uneven groups, an empty one among many."""
    weight = [(3 * g + 1) % 7 + (0 if g == 1 and groups > 2 else 1) for g in range(groups)]
    if groups > 2:
        weight[1] = 0
    count = [rows * w // sum(weight) for w in weight]
    count[0] += rows - sum(count)
    return count


@pytest.mark.gpu
@pytest.mark.parametrize("spread,out", [(0, "f32"), (5, "bf16")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_kernel(dev, case, spread, out):
    name, groups, M, N, K, odd = CASES[case]
    rng = np.random.default_rng(case)
    gap = 1 if odd else 0
    a, sa, av = operand(rng, (M,), K, spread, dev, gap, 3 * gap, gap, gap)
    shape = (N,) if groups == 0 else (groups, N)
    b, sb, bv = operand(rng, shape, K, spread, dev, gap, 3 * gap, gap, gap)
    if not odd and groups:  # `operand` leaves 3 bytes between the groups
        pad = torch.empty((groups, N * (K // 2) + 16), dtype=torch.uint8, device=dev)
        whole = pad[:, :N * (K // 2)].view(groups, N, K // 2)
        whole.copy_(b)
        b = whole

    def strides(t):
        return (t.stride(-2) if t.shape[-2] > 1 else t.shape[-1], t.stride(0) if t.dim() == 3 else 0)

    got_name = selected(groups, M, N, K, a, strides(a)[0], sa, strides(sa)[0], b, *strides(b), sb, *strides(sb))
    assert got_name == name
    buf, y = inside((M, N), DT[out], 3, 1, dev, float("nan"))
    want, S = np.empty((M, N)), np.zeros((M, N))

    def call(out):
        if groups == 0:
            return mm.gemm_mx4(a, b, sa, sb, out=out)
        return mm.gemm_mx4_grouped(a, b, torch.tensor(off, device=dev), sa, sb, out=out)

    if groups == 0:
        call(y)
        want = av @ bv.T
        S = np.abs(av) @ np.abs(bv).T if spread else S
    else:
        off = np.concatenate([[0], np.cumsum(counts_of(groups, M))])
        call(y)
        for g in range(groups):
            lo, hi = off[g], off[g + 1]
            want[lo:hi] = av[lo:hi] @ bv[g].T
            if spread:
                S[lo:hi] = np.abs(av[lo:hi]) @ np.abs(bv[g]).T
    check(y.cpu().double().numpy(), want, S, not spread, DT[out])
    for _ in range(4):  # the same bits every time
        assert torch.equal(call(torch.empty_like(y)), y)
    y.fill_(float("nan"))
    assert bool(torch.isnan(buf).all())


@pytest.mark.gpu
def test_operands_past_32_bits(dev):
    """Rows 2^24 bytes apart (row 300 starts past 2^32), of codes and of scales; groups 2^32 bytes apart."""
    rng = np.random.default_rng(3)
    M, N, K, ld = 300, 140, 512, 1 << 24
    a, sa, av = operand(rng, (M,), K, 0, dev)
    b, sb, bv = operand(rng, (N,), K, 0, dev)
    buf = torch.empty(M * ld, dtype=torch.uint8, device=dev)
    far = torch.as_strided(buf, (M, K // 2), (ld, 1))
    scales = torch.as_strided(buf, (M, K // 32), (ld, 1), 4096)
    far.copy_(a)
    scales.copy_(sa)
    want = av @ bv.T
    check(mm.gemm_mx4(far, b, scales, sb).cpu().double().numpy(), want, None, True, torch.float32)
    check(mm.gemm_mx4(b, far, sb, scales).cpu().double().numpy(), want.T, None, True, torch.float32)
    group = (1 << 32) + 64
    del far, scales, buf
    buf = torch.empty(group + (1 << 20), dtype=torch.uint8, device=dev)
    b2 = torch.as_strided(buf, (2, N, K // 2), (group, K // 2, 1))
    s2 = torch.as_strided(buf, (2, N, K // 32), (group, K // 32, 1), 1 << 18)
    b2[0], b2[1], s2[0], s2[1] = b, b.flip(0), sb, sb.flip(0)
    off = torch.tensor([0, 120, M], device=dev)
    got = mm.gemm_mx4_grouped(a, b2, off, sa, s2).cpu().double().numpy()
    check(got, np.concatenate([want[:120], want[120:, ::-1]]), None, True, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("name,N,K", [("tile 64x64 in 2", 33, 2048), ("tile 128x128", 100, 512), ("tile 256x256", 256, 2048)])
def test_last_row_past_32_bits(dev, name, N, K):
    """Matrices whose last row starts past 2^32 bytes, 100 rows on, in either place: the rows of a tile
    at the matrix' start go on past its 100th."""
    rng = np.random.default_rng(K + N)
    M, ld, distinct = 65536 + 100, 1 << 16, 701
    a, sa, av = operand(rng, (distinct,), K, 0, dev)
    b, sb, bv = operand(rng, (N,), K, 0, dev)
    at = torch.arange(M, device=dev) * 7 % distinct  # rows of `a` and none like its neighbours
    buf = torch.empty(M * ld, dtype=torch.uint8, device=dev)
    far = torch.as_strided(buf, (M, K // 2), (ld, 1))
    far.copy_(a[at])
    scales = sa[at]
    k2 = K // 2
    assert selected(0, M, N, K, far, ld, scales, K // 32, b, k2, 0, sb, K // 32, 0) == name
    assert selected(0, N, M, K, b, k2, sb, K // 32, far, ld, 0, scales, K // 32, 0) == name
    want = torch.from_numpy(av @ bv.T).float().to(dev)[at]  # fp32: exact
    assert torch.equal(mm.gemm_mx4(far, b, scales, sb), want)
    assert torch.equal(mm.gemm_mx4(b, far, sb, scales), want.t())


@pytest.mark.gpu
def test_most_rows(dev):
    """2^31 - 1 rows of one block: element 0 of each row against element 0 of one column, 1.5 or 6."""
    M = 2 ** 31 - 1
    a = torch.zeros((M, 16), dtype=torch.uint8, device=dev)
    code = torch.randint(0, 16, (M,), dtype=torch.uint8, device=dev)
    a[:, 0] = code
    sa = torch.full((M, 1), 126, dtype=torch.uint8, device=dev)
    b = torch.zeros((3, 1, 16), dtype=torch.uint8, device=dev)
    b[:, 0, 0] = torch.tensor([3, 7, 11], dtype=torch.uint8)  # 1.5, 6, -1.5
    sb = torch.full((3, 1, 1), 128, dtype=torch.uint8, device=dev)
    table = torch.from_numpy(values(np.arange(16, dtype=np.uint8)[:, None].repeat(16, 1), np.full((16, 1), 127, np.uint8))[:, 0])
    table = table.to(dev).to(torch.bfloat16)
    off = torch.tensor([0, M - 33, M - 3, M], device=dev)
    got = mm.gemm_mx4_grouped(a, b, off, sa, sb, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    del a
    step = 1 << 28
    for g, (lo, hi, w) in enumerate([(0, M - 33, 1.5), (M - 33, M - 3, 6.0), (M - 3, M, -1.5)]):
        for at in range(lo, hi, step):
            part = code[at:min(at + step, hi)].int()
            assert torch.equal(got[at:min(at + step, hi), 0], table[part] * w), (g, at)
