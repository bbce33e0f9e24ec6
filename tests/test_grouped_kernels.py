"""Every kernel of the grouped and the 8-bit products, by name: which one a call runs is asked of the
library (`..._select`), on the CPU for the table's completeness and on the GPU with the operands
that the call then gets. The operands stand in buffers with NaN (99 for 8-bit integers) in every
gap, their rows at whole 4-byte words or at odd elements, since the choice depends on that.

Bars as in test_grouped_gpu.py, from the number formats.
"""
import os

import numpy as np
import pytest
import torch

import tiled_gemm_gemv_amd as mm
from test_grouped_gpu import (DT, check, check_i8, draw, host64, int8, ranges, reference, reference_grad_b, scales)
from tiled_gemm_gemv_amd import build as mm_build

FAKE = 1 << 40  # never dereferenced

ROW = ["row x16", "row x32"]
NARROW = [f"rows {r}x{c}" for r in (16, 32, 64) for c in (16, 32)]        # rows of B along k
WIDE = ["rows 16x32", "rows 32x32"] + [f"rows {r}x{c}" for r in (16, 32, 64) for c in (64, 128)]  # across k
TILES = ["tile 64x64 in 4", "tile 64x64 in 2", "tile 128x128", "tile 256x256"]
# What calls can get. (Rows of B along k: "any" only within 1024 of 2^31, as in test_most_rows.)
KERNELS = {"kn": ["any 64x64"] + WIDE + TILES, "nk": ROW[:1] + NARROW + TILES, "grad": ["any 64x64"] + TILES,
           "i8": ROW + NARROW + TILES, "i8g": ROW + NARROW + TILES}

# (call, kernel, groups, rows in groups, rows before and after them, N, K, rows at odd elements)
CASES = [
    ("grad", "any 64x64", 6, 301, 0, 0, 5, 70, False),
    ("grad", "any 64x64", 5, 200, 1, 2, 131, 7, True),
    ("grad", "tile 64x64 in 4", 3, 847, 0, 3, 70, 77, False),
    ("grad", "tile 64x64 in 4", 3, 710, 0, 0, 92, 74, True),
    ("grad", "tile 64x64 in 2", 3, 406, 1, 2, 261, 276, False),
    ("grad", "tile 64x64 in 2", 3, 528, 0, 0, 142, 195, True),
    ("grad", "tile 128x128", 3, 5, 0, 0, 130, 78, False),
    ("grad", "tile 128x128", 3, 4, 0, 3, 130, 70, True),
    ("grad", "tile 256x256", 90, 2, 0, 3, 290, 129, False),
    ("grad", "tile 256x256", 74, 1, 0, 0, 390, 129, True),
    ("i8", "row x16", 1, 1, 0, 0, 17, 4588, False),
    ("i8", "row x16", 1, 1, 0, 0, 17, 4218, True),
    ("i8", "row x32", 1, 1, 0, 0, 35, 1108, False),
    ("i8", "row x32", 1, 1, 0, 0, 38, 1046, True),
    ("i8", "rows 16x16", 1, 2, 0, 0, 17, 86, False),
    ("i8", "rows 16x16", 1, 15, 0, 0, 39, 73, True),
    ("i8", "rows 16x32", 1, 1016, 0, 0, 374, 77, False),
    ("i8", "rows 16x32", 1, 204, 0, 0, 2117, 116, True),
    ("i8", "rows 32x16", 1, 161, 0, 0, 466, 77, False),
    ("i8", "rows 32x16", 1, 351, 0, 0, 242, 70, True),
    ("i8", "rows 32x32", 1, 762, 0, 0, 995, 142, False),
    ("i8", "rows 32x32", 1, 750, 0, 0, 1043, 129, True),
    ("i8", "rows 64x16", 1, 295, 0, 0, 1218, 76, False),
    ("i8", "rows 64x16", 1, 226, 0, 0, 759, 180, True),
    ("i8", "rows 64x32", 1, 460, 0, 0, 3045, 82, False),
    ("i8", "rows 64x32", 1, 995, 0, 0, 1506, 87, True),
    ("i8", "tile 64x64 in 4", 1, 464, 0, 0, 657, 1044, False),
    ("i8", "tile 64x64 in 4", 1, 529, 0, 0, 550, 479, True),
    ("i8", "tile 64x64 in 2", 1, 790, 0, 0, 966, 149, False),
    ("i8", "tile 64x64 in 2", 1, 707, 0, 0, 643, 260, True),
    ("i8", "tile 128x128", 1, 924, 0, 0, 838, 78, False),
    ("i8", "tile 128x128", 1, 390, 0, 0, 818, 339, True),
    ("i8", "tile 256x256", 1, 4251, 0, 0, 1933, 108, False),
    ("i8", "tile 256x256", 1, 2360, 0, 0, 3347, 99, True),
    ("i8g", "row x16", 64, 8, 0, 3, 165, 4777, False),
    ("i8g", "row x16", 48, 9, 1, 2, 44, 4358, True),
    ("i8g", "row x16", 10, 1, 0, 3, 20, 4777, False),
    ("i8g", "row x32", 64, 12, 1, 2, 333, 2048, False),
    ("i8g", "row x32", 64, 8, 0, 0, 36, 1531, True),
    ("i8g", "row x32", 3, 1, 0, 0, 36, 1324, False),
    ("i8g", "rows 16x16", 3, 2, 0, 0, 17, 86, False),
    ("i8g", "rows 16x16", 3, 3, 0, 3, 17, 107, True),
    ("i8g", "rows 16x32", 5, 1830, 1, 2, 412, 70, False),
    ("i8g", "rows 16x32", 5, 551, 0, 3, 886, 95, True),
    ("i8g", "rows 32x16", 4, 852, 0, 0, 102, 70, False),
    ("i8g", "rows 32x16", 3, 732, 0, 3, 126, 78, True),
    ("i8g", "rows 32x32", 169, 1503, 0, 3, 279, 83, False),
    ("i8g", "rows 32x32", 3, 3663, 1, 2, 209, 129, True),
    ("i8g", "rows 64x16", 3, 1472, 0, 0, 259, 75, False),
    ("i8g", "rows 64x16", 3, 954, 1, 2, 182, 196, True),
    ("i8g", "rows 64x32", 41, 1411, 0, 0, 1706, 139, False),
    ("i8g", "rows 64x32", 31, 612, 1, 2, 1453, 141, True),
    ("i8g", "tile 64x64 in 4", 3, 1199, 1, 2, 231, 1318, False),
    ("i8g", "tile 64x64 in 4", 3, 362, 0, 3, 665, 468, True),
    ("i8g", "tile 64x64 in 2", 4, 2064, 1, 2, 430, 76, False),
    ("i8g", "tile 64x64 in 2", 5, 1360, 0, 0, 481, 148, True),
    ("i8g", "tile 128x128", 3, 1901, 1, 2, 426, 79, False),
    ("i8g", "tile 128x128", 3, 1783, 1, 2, 353, 125, True),
    ("i8g", "tile 256x256", 6, 3003, 0, 3, 2570, 74, False),
    ("i8g", "tile 256x256", 59, 4941, 1, 2, 941, 71, True),
    ("kn", "any 64x64", 4, 70, 0, 2, 1, 333, False),
    ("kn", "any 64x64", 3, 131, 1, 0, 1, 70, True),
    ("kn", "rows 16x32", 3, 2, 0, 0, 36, 94, False),
    ("kn", "rows 16x32", 3, 2, 0, 3, 34, 79, True),
    ("kn", "rows 16x64", 4, 567, 0, 3, 155, 71, False),
    ("kn", "rows 16x64", 4, 500, 0, 3, 149, 84, True),
    ("kn", "rows 16x128", 7, 1569, 0, 3, 137, 86, False),
    ("kn", "rows 16x128", 11, 423, 0, 3, 676, 74, True),
    ("kn", "rows 16x128", 64, 40, 1, 2, 1003, 200, False),
    ("kn", "rows 32x32", 3, 839, 0, 0, 234, 407, False),
    ("kn", "rows 32x32", 3, 156, 0, 3, 1026, 195, True),
    ("kn", "rows 32x64", 3, 540, 0, 3, 410, 396, False),
    ("kn", "rows 32x64", 8, 589, 0, 3, 319, 228, True),
    ("kn", "rows 32x128", 50, 685, 0, 0, 591, 131, False),
    ("kn", "rows 32x128", 15, 205, 0, 3, 2119, 71, True),
    ("kn", "rows 64x64", 3, 35, 1, 2, 2459, 1501, False),
    ("kn", "rows 64x128", 15, 388, 1, 2, 4491, 580, False),
    ("kn", "tile 64x64 in 4", 3, 71, 0, 0, 71, 820, False),
    ("kn", "tile 64x64 in 4", 3, 42, 0, 3, 76, 342, True),
    ("kn", "tile 64x64 in 2", 3, 1429, 0, 3, 138, 74, False),
    ("kn", "tile 64x64 in 2", 5, 1012, 1, 2, 197, 75, True),
    ("kn", "tile 128x128", 3, 1222, 1, 2, 231, 126, False),
    ("kn", "tile 128x128", 110, 1253, 0, 0, 263, 70, True),
    ("kn", "tile 256x256", 5, 4768, 0, 3, 1674, 70, False),
    ("kn", "tile 256x256", 5, 1655, 0, 0, 4379, 93, True),
    ("nk", "row x16", 64, 10, 0, 3, 131, 2304, False),
    ("nk", "row x16", 32, 6, 1, 2, 53, 2049, True),
    ("nk", "row x16", 5, 2, 0, 0, 27, 2103, False),
    ("nk", "rows 16x16", 64, 8, 1, 2, 260, 1024, False),
    ("nk", "rows 16x16", 64, 12, 0, 0, 67, 777, True),
    ("nk", "rows 16x16", 7, 3, 0, 0, 35, 869, False),
    ("nk", "rows 16x16", 3, 5, 1, 2, 17, 73, False),
    ("nk", "rows 16x16", 3, 3, 1, 2, 17, 70, True),
    ("nk", "rows 16x32", 3, 316, 1, 2, 1460, 117, False),
    ("nk", "rows 16x32", 3, 302, 0, 3, 1498, 70, True),
    ("nk", "rows 32x16", 3, 953, 0, 3, 95, 76, False),
    ("nk", "rows 32x16", 6, 66, 0, 3, 17, 366, True),
    ("nk", "rows 32x32", 70, 998, 0, 3, 483, 70, False),
    ("nk", "rows 32x32", 5, 1353, 1, 2, 575, 78, True),
    ("nk", "rows 64x16", 3, 1147, 0, 0, 229, 135, False),
    ("nk", "rows 64x16", 3, 390, 0, 3, 445, 85, True),
    ("nk", "rows 64x32", 185, 4367, 0, 0, 166, 185, False),
    ("nk", "rows 64x32", 216, 3777, 0, 0, 134, 131, True),
    ("nk", "tile 64x64 in 4", 3, 828, 1, 2, 293, 707, False),
    ("nk", "tile 64x64 in 4", 3, 244, 1, 2, 866, 237, True),
    ("nk", "tile 64x64 in 2", 3, 1186, 0, 0, 427, 188, False),
    ("nk", "tile 64x64 in 2", 3, 832, 1, 2, 666, 105, True),
    ("nk", "tile 128x128", 4, 1440, 1, 2, 1388, 83, False),
    ("nk", "tile 128x128", 3, 546, 0, 0, 662, 118, True),
    ("nk", "tile 256x256", 5, 2684, 0, 0, 2906, 91, False),
    ("nk", "tile 256x256", 9, 4482, 0, 3, 1652, 77, True),
]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mm_build.LIB):
        mm_build.build()
    return mm.load()


def row_stride(cols, odd, size):
    """A leading dimension with a gap of 3 to 6 elements: odd, or of whole 4-byte words."""
    ld = cols + 3
    while ld % 2 == 0 if odd else ld % 2 or ld * size % 4:
        ld += 1
    return ld


def embed(t, odd, fill):
    """A copy of the matrix (or stack of matrices) t inside a buffer of `fill`, its rows row_stride
    apart, the matrices 4 elements more than their rows; starts at 4 bytes, or at one element."""
    size, (rows, cols) = t.element_size(), t.shape[-2:]
    ld, start = row_stride(cols, odd, size), 1 if odd else 4 // size
    step = rows * ld + 4
    buf = torch.full((start + (t.shape[0] if t.dim() == 3 else 1) * step,), fill, dtype=t.dtype, device=t.device)
    view = torch.as_strided(buf, tuple(t.shape), (ld, 1) if t.dim() == 2 else (step, ld, 1), start)
    view.copy_(t)
    return buf, view


def select(op, groups, M, N, K, A, lda, B, ldb, stride_b):
    if op == "grad":
        cfg = mm.mm_gemm_h16_grouped_grad_b_select(groups, M, N, K, A, lda, B, ldb)
    elif op == "i8":
        cfg = mm.mm_gemm_i8_select(M, N, K, A, lda, B, ldb)
    elif op == "i8g":
        cfg = mm.mm_gemm_i8_grouped_select(groups, M, N, K, A, lda, B, ldb, stride_b)
    else:
        cfg = mm.mm_gemm_h16_grouped_select(groups, M, N, K, A, lda, B, ldb, stride_b, int(op == "nk"))
    return mm.mm_gemm_grouped_config_name(cfg)


def counts_of(groups, rows):
    """Rows of each group, uneven; the last group has two rows at least."""
    rng = np.random.default_rng(1000 * groups + rows)
    weight = rng.exponential(size=groups)
    counts = rng.multinomial(max(rows - 2, 0), weight / weight.sum())
    counts[-1] += min(rows, 2)
    return counts


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_case_selects_its_kernel(case):
    op, kernel, groups, rows, lead, tail, N, K, odd = case
    size = 1 if op in ("i8", "i8g") else 2
    start = FAKE + (size if odd else 4)
    M = lead + rows + tail
    lda = row_stride(K, odd, size) if M > 1 else K
    cols, b_rows = (N, K) if op in ("kn", "grad") else (K, N)
    ldb = row_stride(cols, odd, size)
    assert select(op, groups, M, N, K, start, lda, start, ldb, b_rows * ldb + 4) == kernel


def test_every_kernel_has_cases():
    names = [mm.mm_gemm_grouped_config_name(i) for i in range(mm.mm_gemm_grouped_num_configs())]
    assert all(names) and len(set(names)) == len(names)
    assert set().union(*KERNELS.values()) == set(names)
    assert mm.mm_gemm_grouped_config_name(-1) is None and mm.mm_gemm_grouped_config_name(len(names)) is None
    for op, kernels in KERNELS.items():
        assert set(kernels) == {c[1] for c in CASES if c[0] == op}, op


def test_choices_stay_in_the_table():
    # sizes spread over the whole range, aligned and not: never a kernel outside the call's list
    rng = np.random.default_rng(1)
    for _ in range(20000):
        groups, M, N, K = (int(np.exp(rng.uniform(0, np.log(top)))) for top in (4096, 1 << 17, 1 << 16, 1 << 16))
        op, gap = ("kn", "nk", "grad", "i8", "i8g")[rng.integers(5)], int(rng.integers(0, 3))
        cols, b_rows = (N, K) if op in ("kn", "grad") else (K, N)
        name = select(op, groups, M, N, K, FAKE, K + gap, FAKE, cols + gap, b_rows * (cols + gap))
        assert name in KERNELS[op], (op, groups, M, N, K, gap, name)


def test_one_row_meets_one_group():
    # one row in one group is the dense product of one row, whatever the sizes
    for N in (1, 32, 777, 4096, 14336):
        for K in (64, 1000, 1331, 2048, 4096, 7000):
            dense = mm.mm_gemm_i8_select(1, N, K, FAKE, K, FAKE, K)
            assert mm.mm_gemm_i8_grouped_select(1, 1, N, K, FAKE, K, FAKE, K, N * K) == dense, (N, K)
    assert select("i8g", 1, 1, 14336, 4096, FAKE, 4096, FAKE, 4096, 0) == "row x16"
    assert select("nk", 1, 1, 14336, 4096, FAKE, 4096, FAKE, 4096, 0) == "row x16"


@pytest.mark.parametrize("groups,rows", [(2, 1), (3, 1), (3, 2), (4, 2), (8, 1), (8, 2), (64, 8)])
def test_few_rows_among_few_groups(groups, rows):
    # rows at random fall into G (1 - (1 - 1/G)^M) of G groups; with M little above that, about one row
    # to a group is what the call is taken for
    expected = groups * (1 - (1 - 1 / groups) ** rows)
    assert rows <= 1.25 * expected
    for op in ("nk", "i8g"):
        name = select(op, groups, rows, 4096, 4096, FAKE, 4096, FAKE, 4096, 4096 * 4096)
        assert name == "row x16", (op, name)


@pytest.mark.parametrize("groups,rows", [(1, 2), (2, 2), (3, 3), (8, 5), (64, 40)])
def test_more_rows_than_groups_they_fall_into(groups, rows):
    assert rows > 1.25 * groups * (1 - (1 - 1 / groups) ** rows)
    for op in ("nk", "i8g"):
        assert select(op, groups, rows, 4096, 4096, FAKE, 4096, FAKE, 4096, 4096 * 4096) not in ROW


def test_calls_without_a_kernel():
    grouped, grad = mm.mm_gemm_h16_grouped_select, mm.mm_gemm_h16_grouped_grad_b_select
    assert grouped(2, 4, 5, 8, FAKE, 8, FAKE, 5, 40, 0) >= 0
    assert grouped(2, 4, 5, 8, FAKE, 7, FAKE, 5, 40, 0) == -1      # lda
    assert grouped(2, 4, 5, 8, FAKE, 8, FAKE, 5, 40, 2) == -1      # trans_b
    assert grouped(2, 4, 5, 8, None, 8, FAKE, 5, 40, 0) == -1      # A is NULL
    assert grouped(4097, 4, 5, 8, FAKE, 8, FAKE, 5, 40, 0) == -1
    assert grouped(0, 4, 5, 8, FAKE, 8, FAKE, 5, 40, 0) == -1      # these enqueue nothing
    assert grouped(2, 0, 5, 8, FAKE, 8, FAKE, 5, 40, 0) == -1
    assert grouped(2, 4, 0, 8, FAKE, 8, FAKE, 1, 40, 0) == -1
    assert grouped(2, 4, 5, 0, None, 1, None, 5, 0, 0) >= 0        # zeros are written
    assert grad(2, 0, 5, 8, None, 8, None, 5) >= 0
    assert grad(2, 4, 5, 0, None, 1, FAKE, 5) == -1
    assert mm.mm_gemm_i8_select(4, 5, 1 << 17, FAKE, 1 << 17, FAKE, 1 << 17) == -1
    assert mm.mm_gemm_i8_select(4, 5, 8, FAKE, 8, FAKE, 8) >= 0
    assert mm.mm_gemm_i8_grouped_select(2, 4, 5, 8, FAKE, 8, FAKE, 8, -1) == -1
    assert mm.mm_gemm_i8_grouped_select(2, 4, 5, 8, FAKE, 8, FAKE, 8, 40) >= 0


def selected(op, groups, M, N, K, A, B):
    lda = A.stride(0) if M > 1 else K  # as the front ends pass it on
    return select(op, groups, M, N, K, A, lda, B, B.stride(-2), B.stride(0) if B.dim() == 3 else 0)


@pytest.fixture(scope="module")
def dev(lib):
    from gpu_helpers import require_gpu
    return require_gpu()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out,dist", [("bf16", "f32", "int"), ("f16", "f16", "normal")])
@pytest.mark.parametrize("case", [c for c in CASES if c[0] in ("kn", "nk")], ids=lambda c: "-".join(map(str, c)))
def test_grouped16_on(dev, case, dtype, out, dist):
    op, kernel, groups, rows, lead, tail, N, K, odd = case
    off, trans, nan = ranges(counts_of(groups, rows), lead), op == "nk", float("nan")
    M = off[-1] + tail
    A = draw(1, (M, K), dist, dtype, dev)
    B = draw(2, (groups, N, K) if trans else (groups, K, N), dist, dtype, dev)
    A[:lead], A[off[-1]:] = nan, nan
    want, S = reference(A, B, off, trans)
    _, Av = embed(A, odd, nan)
    _, Bv = embed(B, odd, nan)
    buf, C = embed(torch.full((M, N), nan, dtype=DT[out], device=dev), odd, nan)
    assert selected(op, groups, M, N, K, Av, Bv) == kernel
    mm.gemm16_grouped(Av, Bv, torch.tensor(off, device=dev), trans_b=trans, out=C)
    torch.cuda.synchronize()
    check(host64(C), want, S, dist, DT[out])
    C.fill_(nan)
    assert torch.isnan(buf).all().item(), "wrote outside C"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out,dist", [("bf16", "f32", "int"), ("f16", "f16", "normal")])
@pytest.mark.parametrize("case", [c for c in CASES if c[0] == "grad"], ids=lambda c: "-".join(map(str, c)))
def test_grad_b_on(dev, case, dtype, out, dist):
    _, kernel, groups, rows, lead, tail, N, K, odd = case
    off, nan = ranges(counts_of(groups, rows), lead), float("nan")
    M = off[-1] + tail
    A, G = draw(1, (M, K), dist, dtype, dev), draw(2, (M, N), dist, dtype, dev)
    for t in (A, G):
        t[:lead], t[off[-1]:] = nan, nan
    want, S = reference_grad_b(A, G, off)
    _, Av = embed(A, odd, nan)
    _, Gv = embed(G, odd, nan)
    buf, D = embed(torch.full((groups, K, N), nan, dtype=DT[out], device=dev), odd, nan)
    assert selected("grad", groups, M, N, K, Av, Gv) == kernel
    mm.gemm16_grouped_grad_b(Av, Gv, torch.tensor(off, device=dev), out=D)
    torch.cuda.synchronize()
    check(host64(D), want, S, dist, DT[out])
    D.fill_(nan)
    assert torch.isnan(buf).all().item(), "wrote outside D"


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case", [c for c in CASES if c[0] in ("i8", "i8g")], ids=lambda c: "-".join(map(str, c)))
def test_i8_on(dev, case, out):
    op, kernel, groups, rows, lead, tail, N, K, odd = case
    off, nan = ranges(counts_of(groups, rows), lead), float("nan")
    M = off[-1] + tail
    A, B = int8(1, (M, K), dev), int8(2, (groups, N, K), dev)
    sa, sb = scales(3, M, dev), scales(4, (groups, N), dev)
    a, b, ha, hb = host64(A), host64(B), host64(sa), host64(sb)
    want = np.full((M, N), np.nan)
    for g in range(groups):
        lo, hi = off[g], off[g + 1]
        want[lo:hi] = (a[lo:hi] @ b[g].T) * ha[lo:hi, None] * hb[g]
    _, Av = embed(A, odd, 99)
    _, Bv = embed(B, odd, 99)
    buf, C = embed(torch.full((M, N), nan, dtype=DT[out], device=dev), odd, nan)
    assert selected(op, groups, M, N, K, Av, Bv[0] if op == "i8" else Bv) == kernel
    if op == "i8":
        mm.gemm_i8(Av, Bv[0], sa, sb[0], out=C)
    else:
        mm.gemm_i8_grouped(Av, Bv, torch.tensor(off, device=dev), sa, sb, out=C)
    torch.cuda.synchronize()
    check_i8(host64(C), want, DT[out])
    C.fill_(nan)
    assert torch.isnan(buf).all().item(), "wrote outside C"


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,counts", [(5, 6, [3, 0, 4]), (72, 40, [3, 0, 40]), (333, 264, [100, 1, 0, 70]), (1030, 520, [300, 129])])
def test_grad_b_into_matrices_row_by_row(dev, N, K, counts):
    off, groups, nan = ranges(counts), len(counts), float("nan")
    A, G = draw(1, (off[-1], K), "int", "bf16", dev), draw(2, (off[-1], N), "int", "bf16", dev)
    want, S = reference_grad_b(A, G, off)
    offsets = torch.tensor(off, device=dev)
    for gap in (0, 3):
        buf = torch.full((K, groups, N + gap), nan, device=dev)
        D = buf[:, :, :N].transpose(0, 1)
        assert mm.gemm16_grouped_grad_b(A, G, offsets, out=D) is D
        torch.cuda.synchronize()
        check(host64(D), want, S, "int", torch.float32)
        D.fill_(nan)
        assert torch.isnan(buf).all().item(), "wrote outside the matrices"
    with pytest.raises(ValueError, match="overlap"):  # rows of two matrices share elements
        mm.gemm16_grouped_grad_b(A, G, offsets, out=torch.as_strided(buf, (groups, K, N), (N - 1, groups * N, 1)))
