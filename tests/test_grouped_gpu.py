"""GPU parity of the products grouped by expert (16-bit forward and gradients, 8-bit integers),
the 8-bit product and the quantisation of rows, against their definitions in 64 bits.

Bars, from the number formats:
* 16-bit products: every product is exact in fp32. Integer inputs in [-4, 4] have sums below
  2^24, so fp32 outputs are bit-exact and 16-bit outputs are the exact sums rounded to nearest
  even. Random inputs: fp32 sums within 1e-5 sum |a b| (the bar of the plain 16-bit GEMM), and a
  16-bit output adds half a step, eps / 2 of the value (fp16 also 2^-25, half its smallest step).
* 8-bit products: the integer sum is exact; rounding it to fp32 and two multiplications are off
  by 3 2^-24 of the value, (1 + 2^-24)^3 - 1 < 4 2^-24, plus half a step of the output type.
* Quantisation: integers equal; the scale within 2^-24 (one rounding).
"""
import numpy as np
import pytest
import torch

import tiled_gemm_gemv_amd as mm
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    mm.load()
    return d


def rounding(values, dtype):
    """Half a step of dtype at the given float64 values."""
    if dtype == torch.float32:
        return np.zeros_like(values)
    half = np.abs(values) * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -10)
    return half + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def draw(seed, shape, dist, dtype, dev, scale=1.0):
    rng = np.random.default_rng(seed)
    if dist == "int":
        a = rng.integers(-4, 5, shape).astype(np.float32)
    else:
        a = (rng.standard_normal(shape) * scale).astype(np.float32)
    return torch.from_numpy(a).to(DT.get(dtype, dtype)).to(dev)


def padded(t, gap, offset, fill):
    """A copy of the matrix (or stack of matrices) t with `gap` extra elements per row, `offset`
    elements before it and 5 after each matrix, all of them `fill`; unit column stride."""
    rows, cols = t.shape[-2:]
    ld = cols + gap
    if t.dim() == 2:
        buf = torch.full((offset + max(rows, 1) * ld + 16,), fill, dtype=t.dtype, device=t.device)
        view = torch.as_strided(buf, (rows, cols), (ld, 1), offset)
    else:
        step = max(rows, 1) * ld + 5
        buf = torch.full((offset + t.shape[0] * step + 16,), fill, dtype=t.dtype, device=t.device)
        view = torch.as_strided(buf, tuple(t.shape), (step, ld, 1), offset)
    view.copy_(t)
    return buf, view


def host64(t):
    return t.cpu().double().numpy()


def ranges(counts, lead=0):
    off = np.concatenate([[0], np.cumsum(counts)]) + lead
    return [int(v) for v in off]


def reference(A, B, off, trans):
    """The rows' products and the sums of magnitudes, float64; NaN rows where no group is."""
    a, b = host64(A), host64(B)
    n = b.shape[1] if trans else b.shape[2]
    C, S = np.full((a.shape[0], n), np.nan), np.zeros((a.shape[0], n))
    for g in range(b.shape[0]):
        lo, hi = off[g], off[g + 1]
        w = b[g].T if trans else b[g]
        C[lo:hi] = a[lo:hi] @ w
        S[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w)
    return C, S


def check(got, want, S, dist, dtype):
    """got against want (float64) where want is not NaN; NaN there must be NaN in got."""
    live = ~np.isnan(want)
    assert np.isnan(got[~live]).all(), "an element that should be NaN or untouched is not"
    assert not np.isnan(got[live]).any(), "NaN in the result"
    if dist == "int":
        rounded = torch.from_numpy(want).to(dtype).double().numpy()
        assert np.array_equal(got[live], rounded[live]), np.abs(got - rounded)[live].max()
    else:
        tol = 1e-5 * S + rounding(want, dtype) * (1 + 2.0 ** -8)
        err = np.abs(got - want)
        assert (err[live] <= tol[live]).all(), float((err[live] / np.maximum(tol[live], 1e-300)).max())


# (rows of each group, rows before the first, rows after the last, N, K)
CASES = [
    ([1], 0, 0, 1, 1),
    ([1], 0, 0, 16, 16),
    ([3, 0, 2], 1, 2, 7, 5),
    ([1, 1, 1, 1], 0, 0, 64, 128),
    ([0, 0, 5, 0], 0, 3, 40, 64),
    ([1, 2, 0, 8], 0, 0, 256, 256),
    ([16, 17, 15, 1], 3, 0, 136, 96),
    ([33, 0, 64, 31, 2], 0, 5, 130, 200),
    ([64, 65, 63, 1], 0, 0, 128, 192),
    ([100, 28, 0, 1, 127], 2, 1, 264, 320),
    ([300], 0, 0, 257, 777),
    ([129, 255, 1], 0, 0, 333, 129),
    ([257, 256, 0, 300], 0, 7, 512, 256),
    ([700, 3, 600], 0, 0, 776, 520),
    ([40], 0, 0, 1000, 33),
    ([2, 3], 0, 0, 31, 4099),
    ([5, 1, 7], 0, 0, 2048, 1024),
    ([1], 0, 0, 130, 2000),
    ([0, 1, 1, 0], 1, 1, 37, 1024),
    ([1, 0, 0, 1, 1, 1], 0, 0, 100, 4500),
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype,out,dist", [("bf16", "f32", "int"), ("bf16", "bf16", "normal"),
                                            ("f16", "f16", "int"), ("f16", "f32", "normal")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_grouped16(dev, case, dtype, out, dist, trans):
    counts, lead, tail, N, K = CASES[case]
    off = ranges(counts, lead)
    M = off[-1] + tail
    A = draw(10 + case, (M, K), dist, dtype, dev)
    B = draw(50 + case, (len(counts), N, K) if trans else (len(counts), K, N), dist, dtype, dev)
    A[:lead] = float("nan")      # rows of no group are not read into any other row
    A[off[-1]:] = float("nan")
    for g, c in enumerate(counts):
        if c == 0:
            B[g] = float("nan")  # nor an empty group's matrix
    want, S = reference(A, B, off, trans)
    offsets = torch.tensor(off, device=dev)
    # packed operands, then rows apart by odd amounts at odd starts, NaN in every gap
    C = mm.gemm16_grouped(A, B, offsets, trans_b=trans, out_dtype=DT[out],
                          out=torch.full((M, N), float("nan"), dtype=DT[out], device=dev))
    torch.cuda.synchronize()
    check(host64(C), want, S, dist, DT[out])
    _, Av = padded(A, 3, 1, float("nan"))
    _, Bv = padded(B, 5, 3, float("nan"))
    buf, Cv = padded(torch.full((M, N), float("nan"), dtype=DT[out], device=dev), 7, 1, float("nan"))
    mm.gemm16_grouped(Av, Bv, offsets, trans_b=trans, out=Cv)
    torch.cuda.synchronize()
    check(host64(Cv), want, S, dist, DT[out])
    Cv.fill_(float("nan"))
    assert torch.isnan(buf).all().item(), "wrote outside C"


def reference_grad_b(A, G, off):
    a, g = host64(A), host64(G)
    E = len(off) - 1
    D, S = np.zeros((E, a.shape[1], g.shape[1])), np.zeros((E, a.shape[1], g.shape[1]))
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        D[e] = a[lo:hi].T @ g[lo:hi]
        S[e] = np.abs(a[lo:hi]).T @ np.abs(g[lo:hi])
    return D, S


@pytest.mark.parametrize("dtype,out,dist", [("bf16", "f32", "int"), ("bf16", "bf16", "normal"),
                                            ("f16", "f16", "int"), ("f16", "f32", "normal")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_grad_b(dev, case, dtype, out, dist):
    counts, lead, tail, N, K = CASES[case]
    K = min(K, 800)  # here an output size; long sums are those of test_grad_b_long
    off = ranges(counts, lead)
    M = off[-1] + tail
    A = draw(110 + case, (M, K), dist, dtype, dev)
    G = draw(150 + case, (M, N), dist, dtype, dev)
    for t in (A, G):
        t[:lead] = float("nan")
        t[off[-1]:] = float("nan")
    want, S = reference_grad_b(A, G, off)
    offsets = torch.tensor(off, device=dev)
    D = mm.gemm16_grouped_grad_b(A, G, offsets, out=torch.full(want.shape, float("nan"), dtype=DT[out], device=dev))
    torch.cuda.synchronize()
    check(host64(D), want, S, dist, DT[out])
    _, Av = padded(A, 3, 1, float("nan"))
    _, Gv = padded(G, 5, 3, float("nan"))
    buf, Dv = padded(torch.full(want.shape, float("nan"), dtype=DT[out], device=dev), 7, 1, float("nan"))
    mm.gemm16_grouped_grad_b(Av, Gv, offsets, out=Dv)
    torch.cuda.synchronize()
    check(host64(Dv), want, S, dist, DT[out])
    Dv.fill_(float("nan"))
    assert torch.isnan(buf).all().item(), "wrote outside D"


@pytest.mark.parametrize("counts", [[5000], [2049, 0, 3000, 1]])
def test_grad_b_long(dev, counts):
    off = ranges(counts)
    A, G = (draw(s, (off[-1], c), "int", "bf16", dev) for s, c in ((1, 96), (2, 200)))
    want, S = reference_grad_b(A, G, off)
    D = mm.gemm16_grouped_grad_b(A, G, torch.tensor(off, device=dev))
    torch.cuda.synchronize()
    check(host64(D), want, S, "int", torch.float32)


def test_many_groups(dev):
    # more groups than one wave holds lanes, most of them empty or of one row
    rng = np.random.default_rng(5)
    for groups in (64, 65, 128, 300):
        counts = rng.choice([0, 0, 1, 2, 40], groups)
        off = ranges(counts)
        M = off[-1]
        A, B = draw(1, (M, 72), "int", "bf16", dev), draw(2, (groups, 72, 88), "int", "bf16", dev)
        offsets = torch.tensor(off, device=dev)
        want, S = reference(A, B, off, False)
        C = mm.gemm16_grouped(A, B, offsets)
        torch.cuda.synchronize()
        check(host64(C), want, S, "int", torch.float32)
        G = draw(3, (M, 88), "int", "bf16", dev)
        want, S = reference_grad_b(A, G, off)
        D = mm.gemm16_grouped_grad_b(A, G, offsets)
        torch.cuda.synchronize()
        check(host64(D), want, S, "int", torch.float32)


def test_most_groups(dev):
    # 4096 groups, a few of them with rows, at both ends too
    counts = np.zeros(4096, int)
    for g, c in ((0, 3), (63, 1), (64, 70), (1000, 17), (4094, 1), (4095, 130)):
        counts[g] = c
    off = ranges(counts)
    A, W = draw(1, (off[-1], 64), "int", "bf16", dev), draw(2, (1, 64, 72), "int", "bf16", dev)
    offsets = torch.tensor(off, device=dev)
    C = mm.gemm16_grouped(A, W.expand(4096, 64, 72), offsets)
    torch.cuda.synchronize()
    assert np.array_equal(host64(C), host64(A) @ host64(W[0]))
    D = mm.gemm16_grouped_grad_b(A, A[:, :16], offsets)
    torch.cuda.synchronize()
    D = host64(D)
    assert not D[counts == 0].any()
    for g in np.flatnonzero(counts):
        a = host64(A)[off[g]:off[g + 1]]
        assert np.array_equal(D[g], a.T @ a[:, :16]), g


# Shapes of many tiles: those of 256 x 256 (and 128 x 128) with whole and partial K-steps, one K-step,
# groups of one row, of a whole number of tiles, ending in a tile's first and second half, and N that
# is no multiple of 8. References in float64 on the GPU.
MANY_TILES = [
    ([1500, 1, 0, 700, 1895], 4100, 136),
    ([300, 3000, 256, 129], 4096, 777),
    ([4096], 4095, 64),
    ([2048, 2048 + 127], 4001, 1024),
    ([3990, 13], 4096, 128),
    ([4090], 4096, 136),
    ([3850], 4000, 192),
    ([3969], 4089, 333),
]


def close(got, want, S, dist):
    """got (any type) against float64 want on the GPU, as check() does on the host."""
    if got.numel() == 0:  # an empty group's rows
        return
    if dist == "int":
        assert torch.equal(got.double(), want.to(got.dtype).double())
        return
    tol = 1e-5 * S
    if got.dtype != torch.float32:
        tol = tol + want.abs() * (torch.finfo(got.dtype).eps / 2 * (1 + 2.0 ** -7)) + 2.0 ** -25
    worst = ((got.double() - want).abs() / tol).nan_to_num(nan=1e30).max().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("dtype,out,dist", [("bf16", "bf16", "normal"), ("f16", "f32", "int"), ("bf16", "f16", "int")])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("case", range(len(MANY_TILES)))
def test_grouped16_many_tiles(dev, case, trans, dtype, out, dist):
    counts, N, K = MANY_TILES[case]
    off = ranges(counts)
    gen = torch.Generator(device=dev).manual_seed(case)

    def make(*shape):
        if dist == "int":
            return torch.randint(-2, 3, shape, generator=gen, device=dev).to(DT[dtype])
        return torch.randn(shape, generator=gen, device=dev).to(DT[dtype])

    A, B = make(off[-1], K), make(len(counts), N, K) if trans else make(len(counts), K, N)
    C = mm.gemm16_grouped(A, B, torch.tensor(off, device=dev), trans_b=trans, out_dtype=DT[out])
    for g in range(len(counts)):
        a, w = A[off[g]:off[g + 1]].double(), B[g].double()
        w = w.t().contiguous() if trans else w
        close(C[off[g]:off[g + 1]], a @ w, a.abs() @ w.abs(), dist)


@pytest.mark.parametrize("dtype,out,dist", [("bf16", "bf16", "normal"), ("f16", "f32", "int")])
@pytest.mark.parametrize("counts,N,K", [([130, 0, 700], 2050, 2048), ([64, 1, 200, 66], 2304, 1928), ([1500], 4097, 4200),
                                        ([3000, 5, 127], 2056, 2185)])
def test_grad_b_many_tiles(dev, counts, N, K, dtype, out, dist):
    off = ranges(counts)
    gen = torch.Generator(device=dev).manual_seed(K)

    def make(*shape):
        if dist == "int":
            return torch.randint(-2, 3, shape, generator=gen, device=dev).to(DT[dtype])
        return torch.randn(shape, generator=gen, device=dev).to(DT[dtype])

    A, G = make(off[-1], K), make(off[-1], N)
    D = mm.gemm16_grouped_grad_b(A, G, torch.tensor(off, device=dev), out_dtype=DT[out])
    for g in range(len(counts)):
        a, b = A[off[g]:off[g + 1]].double().t().contiguous(), G[off[g]:off[g + 1]].double()
        close(D[g], a @ b, a.abs() @ b.abs(), dist)


# Sizes of about one tile of 128 x 128 for each CU, and of fewer tiles of 64 x 64 than CUs with sums of
# few and many K-steps (parts of a sum in one workgroup that are empty, whole and partial).
FEW_TILES = [
    ([1500], 2000, 300), ([700, 0, 400], 4000, 136), ([2000, 0, 100], 2100, 333), ([1048, 1], 2048, 512),
    ([100, 28], 4096, 520), ([200], 777, 1531), ([60, 0, 131], 1000, 2049), ([256], 2048, 4096), ([70], 520, 100),
    ([33, 64], 1030, 190), ([300], 1024, 8192), ([65, 1, 190], 600, 257),
]


@pytest.mark.parametrize("dtype,out,dist", [("bf16", "bf16", "normal"), ("f16", "f32", "int")])
@pytest.mark.parametrize("case", range(len(FEW_TILES)))
def test_few_tiles(dev, case, dtype, out, dist):
    counts, N, K = FEW_TILES[case]
    off = ranges(counts)
    offsets = torch.tensor(off, device=dev)
    gen = torch.Generator(device=dev).manual_seed(100 + case)

    def make(*shape):
        if dist == "int":
            return torch.randint(-2, 3, shape, generator=gen, device=dev).to(DT[dtype])
        return torch.randn(shape, generator=gen, device=dev).to(DT[dtype])

    A, B, G = make(off[-1], K), make(len(counts), K, N), make(off[-1], N)
    Bt = B.transpose(1, 2).contiguous()
    C = mm.gemm16_grouped(A, B, offsets, out_dtype=DT[out])
    Ct = mm.gemm16_grouped(A, Bt, offsets, trans_b=True, out_dtype=DT[out])
    D = mm.gemm16_grouped_grad_b(A, G, offsets, out_dtype=DT[out])
    # the same numbers with the sum over K in the gradient: long sums for few tiles
    turned = mm.gemm16_grouped_grad_b(A.t().contiguous(), B[0], torch.tensor([0, K], device=dev), out_dtype=DT[out])
    a, w = A.double(), B[0].double()
    close(turned[0], a @ w, a.abs() @ w.abs(), dist)
    for g in range(len(counts)):
        a, w, d = A[off[g]:off[g + 1]].double(), B[g].double(), G[off[g]:off[g + 1]].double()
        if counts[g]:
            close(C[off[g]:off[g + 1]], a @ w, a.abs() @ w.abs(), dist)
            close(Ct[off[g]:off[g + 1]], a @ w, a.abs() @ w.abs(), dist)
        at = a.t().contiguous()
        close(D[g], at @ d, at.abs() @ d.abs(), dist)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(FEW_TILES)))
def test_i8_few_tiles(dev, case, out):
    counts, N, K = FEW_TILES[case]
    M, off = sum(counts), ranges(counts)
    a, b, sa, sb = int8(1, (M, K), dev), int8(2, (len(counts), N, K), dev), scales(3, M, dev), scales(4, (len(counts), N), dev)
    got = mm.gemm_i8_grouped(a, b, torch.tensor(off, device=dev), sa, sb, out_dtype=DT[out])
    one = mm.gemm_i8(a, b[0], sa, sb[0], out_dtype=DT[out])
    torch.cuda.synchronize()
    ha, hb, hsa, hsb = host64(a), host64(b), host64(sa), host64(sb)
    check_i8(host64(one), (ha @ hb[0].T) * hsa[:, None] * hsb[0], DT[out])
    for g in range(len(counts)):
        lo, hi = off[g], off[g + 1]
        check_i8(host64(got)[lo:hi], (ha[lo:hi] @ hb[g].T) * hsa[lo:hi, None] * hsb[g], DT[out])


# Matrices of few columns, whole pieces of 8 and others, in each of a tile's quadrants.
@pytest.mark.parametrize("dtype,out,dist", [("bf16", "bf16", "normal"), ("f16", "f32", "int")])
@pytest.mark.parametrize("N,K", [(9, 8), (100, 17), (127, 200), (130, 64), (131, 255), (250, 2000), (4000, 241), (8, 3000),
                                 (199, 2100), (1030, 121), (65, 63)])
def test_narrow_matrices(dev, N, K, dtype, out, dist):
    counts = [300, 0, 70, 800]
    off = ranges(counts)
    offsets = torch.tensor(off, device=dev)
    A, B, G = draw(1, (off[-1], K), dist, dtype, dev), draw(2, (len(counts), K, N), dist, dtype, dev), draw(
        3, (off[-1], N), dist, dtype, dev)
    C = mm.gemm16_grouped(A, B, offsets, out_dtype=DT[out])
    buf, D = padded(torch.zeros((len(counts), K, N), dtype=DT[out], device=dev), 3, 5, float("nan"))
    mm.gemm16_grouped_grad_b(A, G, offsets, out=D)
    torch.cuda.synchronize()
    check(host64(C), *reference(A, B, off, False), dist, DT[out])
    check(host64(D), *reference_grad_b(A, G, off), dist, DT[out])
    D.fill_(float("nan"))
    assert torch.isnan(buf).all().item(), "wrote outside the matrices"


# Inner sizes below one K-step of the tiles (64 16-bit elements, 128 bytes), from one 16-byte piece on,
# with NaN beyond the rows' ends and before their starts.
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype,out,dist", [("bf16", "bf16", "normal"), ("f16", "f32", "int")])
@pytest.mark.parametrize("counts,N,K", [([700, 0, 1, 300], 520, 40), ([3000], 2056, 8), ([129, 600], 1000, 33),
                                        ([2000, 130], 264, 63), ([255, 1, 257], 1000, 9), ([900], 777, 7)])
def test_grouped16_short_inner_sizes(dev, counts, N, K, dtype, out, dist, trans):
    off = ranges(counts)
    A0, B0 = draw(1, (off[-1], K), dist, dtype, dev), draw(2, (len(counts), N, K) if trans else (len(counts), K, N), dist,
                                                           dtype, dev)
    _, A = padded(A0, 3, 5, float("nan"))
    _, B = padded(B0, 5, 3, float("nan"))
    want, S = reference(A0, B0, off, trans)
    for a, b in ((A, B), (A0, B0)):
        got = mm.gemm16_grouped(a, b, torch.tensor(off, device=dev), trans_b=trans, out_dtype=DT[out])
        torch.cuda.synchronize()
        check(host64(got), want, S, dist, DT[out])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(2000, 4100, 16), (1500, 1000, 17), (700, 777, 100), (3000, 520, 127), (129, 5000, 31),
                                   (1000, 1000, 15)])
def test_i8_short_inner_sizes(dev, M, N, K, out):
    a, b, sa, sb = int8(1, (M, K), dev), int8(2, (N, K), dev), scales(3, M, dev), scales(4, N, dev)
    want = (host64(a) @ host64(b).T) * host64(sa)[:, None] * host64(sb)
    _, av = padded(a, 3, 7, 99)
    _, bv = padded(b, 9, 1, 99)
    for x, y in ((av, bv), (a, b)):
        got = mm.gemm_i8(x, y, sa, sb, out_dtype=DT[out])
        torch.cuda.synchronize()
        check_i8(host64(got), want, DT[out])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 128), (3000, 5003, 777), (4225, 4096, 1024), (8192, 2049, 130),
                                   (3850, 4090, 256), (3969, 4000, 300)])
def test_i8_many_tiles(dev, M, N, K, out):
    A, B = int8(1, (M, K), dev), int8(2, (N, K), dev)
    sa, sb = scales(3, M, dev), scales(4, N, dev)
    C = mm.gemm_i8(A, B, sa, sb, out_dtype=DT[out])
    want = (A.double() @ B.double().t().contiguous()) * sa.double()[:, None] * sb.double()
    half = 0 if out == "f32" else torch.finfo(DT[out]).eps / 2 * (1 + 2.0 ** -20)
    err = (C.double() - want).abs()
    assert (err <= want.abs() * (4 * 2.0 ** -24 + half)).all().item()


def test_i8_no_inner_size(dev):
    # the empty sum: zero times the scales
    sa, sb = scales(3, 5, dev), scales(4, 40, dev)
    sa[2] = float("nan")
    e = torch.empty((5, 0), dtype=torch.int8, device=dev), torch.empty((40, 0), dtype=torch.int8, device=dev)
    C = mm.gemm_i8(*e, sa, sb, out=torch.full((5, 40), 7.0, device=dev))
    torch.cuda.synchronize()
    assert torch.isnan(C[2]).all().item() and (C[[0, 1, 3, 4]] == 0).all().item()
    C = mm.gemm_i8_grouped(e[0], e[1][None], torch.tensor([1, 5], device=dev), sa, sb[None],
                           out=torch.full((5, 40), 7.0, device=dev))
    torch.cuda.synchronize()
    assert (C[0] == 7).all().item() and torch.isnan(C[2]).all().item() and (C[[1, 3, 4]] == 0).all().item()


def test_shared_matrix_and_no_inner_size(dev):
    # group stride 0 shares B; K = 0 gives zero rows, rows of no group untouched
    A, B = draw(1, (70, 128), "int", "f16", dev), draw(2, (1, 128, 96), "int", "f16", dev)
    off = [0, 30, 30, 69]
    want, S = reference(A, B.expand(3, 128, 96), off, False)
    want[69:] = np.nan
    C = mm.gemm16_grouped(A, B.expand(3, 128, 96), torch.tensor(off, device=dev),
                          out=torch.full((70, 96), float("nan"), device=dev))
    torch.cuda.synchronize()
    check(host64(C), want, S, "int", torch.float32)
    out = torch.full((70, 96), float("nan"), device=dev)
    mm.gemm16_grouped(A[:, :0], B[:, :0].expand(3, 0, 96), torch.tensor(off, device=dev), out=out)
    torch.cuda.synchronize()
    assert (out[:69] == 0).all().item() and torch.isnan(out[69:]).all().item()
    D = mm.gemm16_grouped_grad_b(A[:0], draw(3, (0, 96), "int", "f16", dev), torch.zeros(4, dtype=torch.int64, device=dev))
    torch.cuda.synchronize()
    assert D.shape == (3, 128, 96) and (D == 0).all().item()


@pytest.mark.parametrize("N,K", [(96, 200), (264, 512)])
def test_offsets_outside_the_rows(dev, N, K):
    # entries beyond [0, M] count as the bound, an end below its start is an empty group;
    # nothing outside C's M rows is written
    M = 300
    A, B = draw(1, (M, K), "int", "bf16", dev), draw(2, (4, K, N), "int", "bf16", dev)
    buf, C = padded(torch.full((M, N), float("nan"), device=dev), 0, 0, float("nan"))
    mm.gemm16_grouped(A, B, torch.tensor([-5, 100, 100, 1 << 40, 1 << 41], device=dev), out=C)
    torch.cuda.synchronize()
    want, S = reference(A, B, [0, 100, 100, 300, 300], False)
    check(host64(C), want, S, "int", torch.float32)
    mm.gemm16_grouped(A, B, torch.tensor([200, 100, 50, 40, -(1 << 50)], device=dev), out=C.fill_(float("nan")))
    D = mm.gemm16_grouped_grad_b(A, A[:, :64], torch.tensor([200, 100, 50, 40, 1 << 60], device=dev))
    torch.cuda.synchronize()
    assert torch.isnan(C).all().item()
    want, S = reference_grad_b(A, A[:, :64], [200, 200, 200, 200, 300])
    want[3], S[3] = reference_grad_b(A, A[:, :64], [40, 300])[0][0], 0
    check(host64(D), want, S, "int", torch.float32)
    C.fill_(float("nan"))
    assert torch.isnan(buf).all().item()


def test_specials_stay_in_their_rows(dev):
    # an infinity or NaN in one row of A makes that row's products non-finite and no others,
    # whatever the partial k step (K = 200, 777) or the group's partial tile reads beside it
    for K, N in [(200, 130), (777, 264), (64, 64), (1024, 512)]:
        counts = [5, 40, 130, 260]
        off = ranges(counts)
        for trans in (False, True):
            A = draw(7, (off[-1], K), "normal", "bf16", dev)
            B = draw(8, (4, N, K) if trans else (4, K, N), "normal", "bf16", dev)
            bad = [4, 5, 44, 174, 175, off[-1] - 1]
            for i, r in enumerate(bad):
                A[r, (i * 37) % K] = float("nan") if i % 2 else float("inf")
                A[r, K - 1] = float("inf")
            C = mm.gemm16_grouped(A, B, torch.tensor(off, device=dev), trans_b=trans)
            torch.cuda.synchronize()
            c = host64(C)
            assert not np.isfinite(c[bad]).any()
            rest = np.delete(np.arange(off[-1]), bad)
            want, S = reference(A[rest], B, ranges([4, 38, 129, 258]), trans)
            check(c[rest], want, S, "normal", torch.float32)


def test_grad_specials_stay_in_their_group(dev):
    counts = [5, 40, 130, 0, 260]
    off = ranges(counts)
    A, G = draw(7, (off[-1], 72), "int", "bf16", dev), draw(8, (off[-1], 264), "int", "bf16", dev)
    G[off[1]:off[2]] = float("nan")
    A[off[3]:off[5]] = float("inf")
    D = host64(mm.gemm16_grouped_grad_b(A, G, torch.tensor(off, device=dev)))
    want, _ = reference_grad_b(A, G, off)
    for g in (0, 2, 3):
        assert np.array_equal(D[g], want[g])
    assert np.isnan(D[1]).all() and not np.isfinite(D[4]).any()


# ------------------------------------------------------------------------- 8-bit integers

def int8(seed, shape, dev, lo=-128):
    return torch.from_numpy(np.random.default_rng(seed).integers(lo, 128, shape).astype(np.int8)).to(dev)


def scales(seed, shape, dev):
    return torch.from_numpy((np.random.default_rng(seed).random(shape) * 0.02 + 1e-3).astype(np.float32)).to(dev)


def check_i8(got, want, dtype):
    live = ~np.isnan(want)
    assert np.isnan(got[~live]).all()
    tol = np.abs(want) * 4 * 2.0 ** -24 + rounding(want, dtype) * (1 + 2.0 ** -20)
    err = np.abs(got - want)
    assert (err[live] <= tol[live]).all(), float((err[live] / np.maximum(tol[live], 1e-300)).max())


I8_SHAPES = [(1, 1, 1), (1, 16, 16), (1, 33, 1024), (1, 70, 2049), (1, 515, 9000), (3, 5, 7), (1, 256, 512), (2, 100, 128), (8, 136, 384), (16, 264, 200),
             (17, 64, 128), (33, 130, 777), (64, 128, 256), (65, 300, 129), (100, 257, 1000), (129, 131, 640),
             (256, 256, 256), (300, 520, 1024), (700, 300, 2049), (513, 1031, 130)]


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", I8_SHAPES)
def test_i8(dev, shape, out):
    M, N, K = shape
    A, B = int8(1, (M, K), dev), int8(2, (N, K), dev)
    sa, sb = scales(3, M, dev), scales(4, N, dev)
    want = (host64(A) @ host64(B).T) * host64(sa)[:, None] * host64(sb)
    got = mm.gemm_i8(A, B, sa, sb, out_dtype=DT[out])
    torch.cuda.synchronize()
    check_i8(host64(got), want, DT[out])
    _, Av = padded(A, 3, 1, 99)
    _, Bv = padded(B, 1, 3, -77)
    buf, Cv = padded(torch.full((M, N), float("nan"), dtype=DT[out], device=dev), 3, 1, float("nan"))
    mm.gemm_i8(Av, Bv, sa, sb, out=Cv)
    torch.cuda.synchronize()
    check_i8(host64(Cv), want, DT[out])
    Cv.fill_(float("nan"))
    assert torch.isnan(buf).all().item(), "wrote outside C"


@pytest.mark.parametrize("M,N", [(1, 40), (40, 64), (300, 260)])
def test_i8_largest_sums(dev, M, N):
    # every value -128 and K at its limit: the sum is K 2^14 = 2^31 - 2^14, still exact in 32 bits
    K = (1 << 17) - 1
    A = torch.full((M, K), -128, dtype=torch.int8, device=dev)
    B = torch.full((N, K), -128, dtype=torch.int8, device=dev)
    got = mm.gemm_i8(A, B, torch.ones(M, device=dev), torch.ones(N, device=dev))
    torch.cuda.synchronize()
    assert (got == float(np.float32(K * 16384))).all().item()
    B[:, ::2] = 127
    got = mm.gemm_i8(A, B, torch.ones(M, device=dev), torch.ones(N, device=dev))
    torch.cuda.synchronize()
    s = -128 * 127 * ((K + 1) // 2) + 128 * 128 * (K // 2)
    assert (got == float(np.float32(s))).all().item()


def test_i8_scales_propagate(dev):
    A, B = int8(1, (40, 256), dev), int8(2, (70, 256), dev)
    A[5] = 0
    sa, sb = scales(3, 40, dev), scales(4, 70, dev)
    sa[3], sa[5], sb[7] = float("nan"), float("nan"), 0.0
    got = host64(mm.gemm_i8(A, B, sa, sb))
    assert np.isnan(got[[3, 5]]).all()
    keep = np.delete(np.arange(40), [3, 5])
    assert (got[keep][:, 7] == 0).all() and np.isfinite(got[keep]).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_i8_grouped(dev, case, out):
    counts, lead, tail, N, K = CASES[case]
    off = ranges(counts, lead)
    M = off[-1] + tail
    A, B = int8(10 + case, (M, K), dev), int8(50 + case, (len(counts), N, K), dev)
    sa, sb = scales(3, M, dev), scales(4, (len(counts), N), dev)
    a, b = host64(A), host64(B)
    want = np.full((M, N), np.nan)
    for g in range(len(counts)):
        lo, hi = off[g], off[g + 1]
        want[lo:hi] = (a[lo:hi] @ b[g].T) * host64(sa)[lo:hi, None] * host64(sb)[g]
    offsets = torch.tensor(off, device=dev)
    out_t = torch.full((M, N), float("nan"), dtype=DT[out], device=dev)
    got = mm.gemm_i8_grouped(A, B, offsets, sa, sb, out=out_t)
    torch.cuda.synchronize()
    check_i8(host64(got), want, DT[out])
    _, Av = padded(A, 3, 1, 99)
    _, Bv = padded(B, 1, 3, -77)
    buf, Cv = padded(out_t.fill_(float("nan")), 3, 1, float("nan"))
    mm.gemm_i8_grouped(Av, Bv, offsets, sa, sb, out=Cv)
    torch.cuda.synchronize()
    check_i8(host64(Cv), want, DT[out])
    Cv.fill_(float("nan"))
    assert torch.isnan(buf).all().item(), "wrote outside C"


# ---------------------------------------------------------------------------- quantisation

def quantize_reference(x):
    v = host64(x)
    top = np.abs(v).max(axis=1) if v.shape[1] else np.zeros(v.shape[0])
    q = np.rint(v * 127.0 / np.where(top > 0, top, 1.0)[:, None])
    return q, top / 127.0


def check_quantize(x, q, s):
    want_q, want_s = quantize_reference(x)
    assert np.array_equal(q.cpu().numpy(), want_q), np.abs(q.cpu().numpy() - want_q).max()
    # one rounding to fp32 (below 2^-126: half the smallest step)
    assert (np.abs(host64(s) - want_s) <= np.maximum(want_s * 2.0 ** -24, 2.0 ** -150)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (2, 255), (4, 256), (7, 1000), (1, 4096), (9, 4104),
                                       (3, 8192), (2, 14336), (3, 40000), (1025, 96)])
def test_quantize(dev, dtype, rows, cols):
    x = draw(rows * 7 + cols, (rows, cols), "normal", dtype, dev, scale=3.0)
    q, s = mm.quantize_i8(x)
    torch.cuda.synchronize()
    check_quantize(x, q, s)
    _, xv = padded(x, 5, 3, float("nan"))
    buf, qv = padded(torch.zeros((rows, cols), dtype=torch.int8, device=dev), 3, 1, 55)
    mm.quantize_i8(xv, out=qv, scale=s.zero_())
    torch.cuda.synchronize()
    check_quantize(x, qv, s)
    qv.fill_(55)
    assert (buf == 55).all().item(), "wrote outside Q"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_ties_and_neighbours(dev, dtype):
    # amax = 127 2^e: the quotients are the integers and halves themselves; in fp32 also the
    # values next to each half
    rows = []
    for e in (0, -6, 3):
        h = np.arange(-127, 127.5, 0.5)
        v = [h * 2.0 ** e]
        if dtype == "f32":
            f = (h * 2.0 ** e).astype(np.float32)
            v += [np.nextafter(f, np.float32(1e9))[:-2], np.nextafter(f, np.float32(-1e9))[2:]]
        rows.append(np.concatenate(v))
    n = len(rows[0])
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).to(dev).to(DT[dtype])
    assert x.shape == (3, n)
    q, s = mm.quantize_i8(x)
    torch.cuda.synchronize()
    check_quantize(x, q, s)


def test_quantize_every_16_bit_value(dev):
    # every finite value of a 16-bit type up to amax, over several amax
    for dtype, tops in ((torch.bfloat16, [1.0, 1.9921875, 3.3e38, 1e-38, 9.2e-41, 253.0]),
                        (torch.float16, [1.0, 65504.0, 0.333, 6e-8, 6.1e-5])):
        bits = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16)
        v = torch.cat([bits, bits | -32768]).view(dtype)
        for top in tops:
            t = torch.tensor(top, dtype=dtype)
            x = torch.where(v.abs() <= t, v, t.expand_as(v))[None].to(dev)
            q, s = mm.quantize_i8(x)
            torch.cuda.synchronize()
            check_quantize(x, q, s)


def test_quantize_extreme_scales(dev):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((8, 777))
    for i, e in enumerate([-149, -140, -126, -61, -59, 0, 100, 126]):
        x[i] = x[i] / np.abs(x[i]).max() * 2.0 ** e * (1.9 if e > -149 else 1.0)
    t = torch.from_numpy(x.astype(np.float32)).to(dev)
    q, s = mm.quantize_i8(t)
    torch.cuda.synchronize()
    check_quantize(t, q, s)


def test_quantize_rows_of_zeros_and_specials(dev):
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for cols in (5, 300, 9000):
            x = torch.ones((6, cols), dtype=dtype, device=dev)
            x[0] = 0
            x[1] = -0.0
            x[2, cols - 1] = float("nan")
            x[3, 0] = float("inf")
            x[4, cols // 2] = -float("inf")
            q, s = mm.quantize_i8(x, out=torch.full((6, cols), 9, dtype=torch.int8, device=dev))
            torch.cuda.synchronize()
            assert (q[:5] == 0).all().item() and (q[5] == 127).all().item()
            assert (s[:2] == 0).all().item() and torch.isnan(s[2:5]).all().item()
    q, s = mm.quantize_i8(torch.ones((3, 0), device=dev), scale=torch.ones(3, device=dev))
    torch.cuda.synchronize()
    assert q.shape == (3, 0) and (s == 0).all().item()


# ------------------------------------------------------------- offsets past 32 bits, streams

def test_offsets_past_32_bits(dev):
    # group strides and leading dimensions that put operands past 2^32 bytes
    K, N = 136, 72
    far = (1 << 31) + 8
    B = torch.empty(2 * far + K * N, dtype=torch.bfloat16, device=dev)
    Bs = torch.as_strided(B, (3, K, N), (far, N, 1))
    Bs.copy_(draw(2, (3, K, N), "int", "bf16", dev))
    A = draw(1, (40, K), "int", "bf16", dev)
    off = [0, 3, 20, 40]
    want, S = reference(A, Bs.contiguous(), off, False)
    got = mm.gemm16_grouped(A, Bs, torch.tensor(off, device=dev))
    torch.cuda.synchronize()
    check(host64(got), want, S, "int", torch.float32)
    D = torch.as_strided(B, (3, K, N), (far, N, 1))
    G = draw(3, (40, N), "int", "bf16", dev)
    mm.gemm16_grouped_grad_b(A, G, torch.tensor(off, device=dev), out=D)
    torch.cuda.synchronize()
    check(host64(D.contiguous()), reference_grad_b(A, G, off)[0], 0, "int", torch.bfloat16)
    del B, Bs, D
    # rows 2^24 bytes apart: row 300 starts past 2^32
    M, ld = 300, 1 << 24
    buf = torch.empty(M * ld, dtype=torch.int8, device=dev)
    Av = torch.as_strided(buf, (M, 256), (ld, 1))
    Av.copy_(int8(1, (M, 256), dev))
    W = int8(2, (130, 256), dev)
    sa, sb = scales(3, M, dev), scales(4, 130, dev)
    want = (host64(Av.contiguous()) @ host64(W).T) * host64(sa)[:, None] * host64(sb)
    got = mm.gemm_i8(Av, W, sa, sb)
    torch.cuda.synchronize()
    check_i8(host64(got), want, torch.float32)
    got = mm.gemm_i8(W, Av, sb, sa)
    torch.cuda.synchronize()
    check_i8(host64(got), want.T, torch.float32)


def test_most_rows(dev):
    # 2^31 - 1 rows: tile counts and row numbers at the end of 32 bits. One column and one inner
    # element, so each output is one product, exact in bf16 (8-bit values by powers of two).
    M = 2 ** 31 - 1
    a8 = torch.randint(-128, 128, (M, 1), dtype=torch.int8, device=dev)
    A = a8.to(torch.bfloat16)
    B = torch.tensor([[[2.0]], [[0.5]], [[-4.0]]], dtype=torch.bfloat16, device=dev)
    off = torch.tensor([0, M - 33, M - 3, M], device=dev)
    for trans in (False, True):
        C = mm.gemm16_grouped(A, B, off, trans_b=trans, out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        for g, (lo, hi) in enumerate([(0, M - 33), (M - 33, M - 3), (M - 3, M)]):
            assert torch.equal(C[lo:hi], A[lo:hi] * B[g]), (trans, g)
        del C
    s, one = torch.full((M,), 0.25, device=dev), torch.ones(1, device=dev)
    C = mm.gemm_i8(a8, torch.ones((1, 1), dtype=torch.int8, device=dev), s, one, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(C, A * 0.25)


SUBNORMAL = [([1, 2, 0, 1], 1100, 600), ([20, 0, 9, 30], 200, 264), ([300, 200], 520, 192), ([40, 3], 31, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts,N,K", SUBNORMAL)
def test_subnormal_inputs_and_outputs(dev, counts, N, K, trans, dtype):
    """Subnormal inputs count in full (sums of integers, so exact), and so do fp16 outputs below 2^-14
    (multiples of 2^-24 with magnitude at most 16 K 2^-24 < 2^-9: rounded, by `check`'s bar)."""
    E, M = len(counts), sum(counts)
    off = ranges(counts)
    offsets = torch.tensor(off, device=dev)
    Bi = draw(2, (E, N, K) if trans else (E, K, N), "int", dtype, dev)
    Ai, Gi = draw(1, (M, K), "int", dtype, dev), draw(3, (M, N), "int", dtype, dev)
    small, large = (2.0 ** -133, 2.0 ** 40) if dtype == "bf16" else (2.0 ** -24, 2.0 ** 6)

    def times(t, factor):  # exact
        return (t.cpu().double() * factor).to(t.dtype).to(dev)

    want, S = reference(Ai, Bi, off, trans)
    got = mm.gemm16_grouped(times(Ai, small), times(Bi, large), offsets, trans_b=trans)
    d = mm.gemm16_grouped_grad_b(times(Ai, large), times(Gi, small), offsets)
    torch.cuda.synchronize()
    check(host64(got) / (small * large), want, S, "int", torch.float32)
    check(host64(d) / (small * large), reference_grad_b(Ai, Gi, off)[0], 0, "int", torch.float32)
    if dtype == "f16":
        got = mm.gemm16_grouped(times(Ai, 2.0 ** -14), times(Bi, 2.0 ** -10), offsets, trans_b=trans, out_dtype=torch.float16)
        torch.cuda.synchronize()
        check(host64(got), want * 2.0 ** -24, S * 2.0 ** -24, "int", torch.float16)


def moe(dev, tokens, experts, top, d, f, seed):
    """Routing of a layer of experts: the sorted token rows, offsets and matrices."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((tokens, experts), generator=g) + torch.linspace(0, 1.5, experts)
    choice = logits.topk(top, dim=1).indices.flatten()
    order = torch.argsort(choice, stable=True)
    counts = torch.bincount(choice, minlength=experts)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    x = torch.randn((tokens, d), generator=g)
    up = torch.randn((experts, d, f), generator=g) / d ** 0.5
    down = torch.randn((experts, f, d), generator=g) / f ** 0.5
    return x, order // top, offsets, up, down


@pytest.mark.parametrize("tokens,experts,top,d,f", [(1, 8, 2, 256, 384), (50, 6, 2, 200, 136), (400, 8, 2, 256, 520)])
def test_layer_of_experts_and_its_gradient(dev, tokens, experts, top, d, f):
    """Up projection, square (an activation whose gradient is exact to write down), down
    projection and the gradients of the whole layer, against the same in float64 from the same
    bf16 values at each stage, and against differences."""
    x, rows, offsets, up, down = moe(dev, tokens, experts, top, d, f, 11)
    bf = torch.bfloat16
    xs, up, down = x[rows].to(bf).to(dev), up.to(bf).to(dev), down.to(bf).to(dev)
    off = offsets.to(dev)
    h = mm.gemm16_grouped(xs, up, off, out_dtype=bf)
    a = (h.float() ** 2).to(bf)
    y = mm.gemm16_grouped(a, down, off)
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(1)).to(bf).to(dev)
    da = mm.gemm16_grouped(dy, down, off, trans_b=True)
    ddown = mm.gemm16_grouped_grad_b(a, dy, off)
    dh = (2 * h.float() * da).to(bf)
    dx = mm.gemm16_grouped(dh, up, off, trans_b=True)
    dup = mm.gemm16_grouped_grad_b(xs, dh, off)
    torch.cuda.synchronize()
    o = offsets.tolist()
    for got, (want, S), dtype in ((h, reference(xs, up, o, False), bf), (y, reference(a, down, o, False), torch.float32),
                                  (da, reference(dy, down, o, True), torch.float32),
                                  (dx, reference(dh, up, o, True), torch.float32),
                                  (ddown, reference_grad_b(a, dy, o), torch.float32),
                                  (dup, reference_grad_b(xs, dh, o), torch.float32)):
        check(host64(got), want, S, "normal", dtype)
    # differences: the loss sum(dy y) moves along a direction v of `up` by <dup, v>. In exact
    # arithmetic the loss is quadratic in `up`, so a central difference has no error of its own;
    # h, a and dh are bf16 roundings (2^-8 of the value each), which bounds what is left.
    v = torch.randn(up.shape, generator=torch.Generator().manual_seed(2)).double().numpy()
    X, U, W, DY = host64(xs), host64(up), host64(down), host64(dy)
    slope = mags = 0.0
    for g in range(experts):
        lo, hi = o[g], o[g + 1]

        def loss(U_g):
            return (DY[lo:hi] * ((X[lo:hi] @ U_g) ** 2 @ W[g])).sum()

        slope += (loss(U[g] + v[g]) - loss(U[g] - v[g])) / 2
        # the terms of <dup, v> before they cancel: 2 |dy| |w| |h| |x v|
        mags += 2 * (np.abs(DY[lo:hi]) @ np.abs(W[g]).T * np.abs(X[lo:hi] @ U[g]) * np.abs(X[lo:hi] @ v[g])).sum()
    got = (host64(dup) * v).sum()
    assert abs(got - slope) <= mags * (2 * 2.0 ** -8 + 1e-4), (got, slope, mags)


def test_layer_of_8_bit_experts(dev):
    """Weights quantised per output channel, tokens per row, both grouped products in 8 bits; each
    stage against float64 on the integers that stage was given."""
    x, rows, offsets, up, down = moe(dev, 90, 8, 2, 256, 392, 12)
    off, o = offsets.to(dev), offsets.tolist()
    xs = x[rows].to(torch.bfloat16).to(dev)
    w_up, w_down = (w.transpose(1, 2).contiguous().to(dev) for w in (up, down))  # groups x N x K

    def quantize_weights(w):
        q, s = mm.quantize_i8(w.view(-1, w.shape[2]))
        check_quantize(w.view(-1, w.shape[2]), q, s)
        return q.view(w.shape), s.view(w.shape[:2])

    (q_up, s_up), (q_down, s_down) = quantize_weights(w_up), quantize_weights(w_down)

    def stage(t, q_w, s_w, dtype):
        q, s = mm.quantize_i8(t)
        y = mm.gemm_i8_grouped(q, q_w, off, s, s_w, out_dtype=dtype)
        torch.cuda.synchronize()
        check_quantize(t, q, s)
        want = np.zeros(tuple(y.shape))
        for g in range(8):
            lo, hi = o[g], o[g + 1]
            want[lo:hi] = (host64(q[lo:hi]) @ host64(q_w[g]).T) * host64(s)[lo:hi, None] * host64(s_w[g])
        check_i8(host64(y), want, dtype)
        return y

    h = stage(xs, q_up, s_up, torch.bfloat16)
    y = stage(torch.relu(h), q_down, s_down, torch.float32)
    # and the whole stays near the layer in float64: each operand's rounding is at most half a
    # step of amax / 127, so a product of K terms is off by at most
    # sum (|x| dw + |w| dx + dx dw), dx, dw those half steps
    X, W = host64(xs), w_up.cpu().double().numpy()
    H = host64(h)
    for g in range(8):
        lo, hi = o[g], o[g + 1]
        dx = np.abs(X[lo:hi]).max(axis=1, keepdims=True) / 254 if hi > lo else np.zeros((0, 1))
        dw = np.abs(W[g]).max(axis=1, keepdims=True) / 254
        bound = (np.abs(X[lo:hi]) + dx) @ np.ones_like(W[g].T) * dw.T + dx * np.abs(W[g]).sum(axis=1)
        want = X[lo:hi] @ W[g].T
        assert (np.abs(H[lo:hi] - want) <= bound * 1.001 + np.abs(want) * 2.0 ** -8 * 1.01).all()
    assert torch.isfinite(y).all().item()


def test_streams_and_graph_replays(dev):
    """Two streams at once, then a captured graph of every operator replayed with other inputs and
    other offsets in the same buffers, each replay against the eager calls."""
    E, K, N, M = 5, 264, 200, 330
    bf = torch.bfloat16
    A, B, G = draw(1, (M, K), "normal", bf, dev), draw(2, (E, K, N), "normal", bf, dev), draw(3, (M, N), "normal", bf, dev)
    Wq, Ws = int8(4, (E, N, K), dev), scales(5, (E, N), dev)
    off = torch.tensor(ranges([40, 0, 100, 60, 130]), device=dev)

    def all_calls():
        q, s = mm.quantize_i8(A)
        return [mm.gemm16_grouped(A, B, off, out_dtype=bf), mm.gemm16_grouped(G, B, off, trans_b=True),
                mm.gemm16_grouped_grad_b(A, G, off), q, s, mm.gemm_i8(q, Wq[1], s, Ws[1]),
                mm.gemm_i8_grouped(q, Wq, off, s, Ws, out_dtype=bf)]

    eager = all_calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for st in streams:
        with torch.cuda.stream(st):
            results.append(all_calls())
    for st in streams:
        st.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_calls()
    for counts in ([40, 0, 100, 60, 130], [330, 0, 0, 0, 0], [1, 2, 3, 4, 320], [66] * 5):
        A.copy_(draw(sum(counts) + counts[0], (M, K), "normal", bf, dev))
        off.copy_(torch.tensor(ranges(counts)))
        graph.replay()
        torch.cuda.synchronize()
        eager = all_calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))


def test_front_end_refusals(dev):
    A, B = draw(1, (8, 32), "int", "bf16", dev), draw(2, (2, 32, 16), "int", "bf16", dev)
    off = torch.tensor([0, 3, 8], device=dev)
    with pytest.raises(TypeError):
        mm.gemm16_grouped(A, B.half(), off)
    with pytest.raises(ValueError, match="inner"):
        mm.gemm16_grouped(A, B, off, trans_b=True)
    with pytest.raises(TypeError, match="int64"):
        mm.gemm16_grouped(A, B, off.int())
    with pytest.raises(ValueError, match="groups"):
        mm.gemm16_grouped(A, B, off[:2])
    with pytest.raises(ValueError, match="cpu"):
        mm.gemm16_grouped(A, B, off.cpu())
    with pytest.raises(ValueError, match="3-D"):
        mm.gemm16_grouped(A, B[0], off)
    with pytest.raises(TypeError, match="out_dtype"):
        mm.gemm16_grouped(A, B, off, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        mm.gemm16_grouped(A, B, off, out=torch.empty((8, 16), dtype=torch.float64, device=dev))
    with pytest.raises(TypeError, match="out_dtype"):
        mm.gemm16_grouped(A, B, off, out=torch.empty((8, 16), device=dev), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shape"):
        mm.gemm16_grouped(A, B, off, out=torch.empty((8, 15), device=dev))
    with pytest.raises(ValueError, match="row counts"):
        mm.gemm16_grouped_grad_b(A, A[:7], off)
    with pytest.raises(ValueError, match="overlap"):
        mm.gemm16_grouped_grad_b(A, A, off, out=torch.empty((1, 32, 32), device=dev).expand(2, 32, 32))
    q, s = mm.quantize_i8(A)
    w = torch.zeros((4, 32), dtype=torch.int8, device=dev)
    with pytest.raises(ValueError, match="a_scale"):
        mm.gemm_i8(q, w, s[:7], torch.ones(4, device=dev))
    with pytest.raises(TypeError, match="b_scale"):
        mm.gemm_i8(q, w, s, torch.ones(4, dtype=torch.float64, device=dev))
    with pytest.raises(ValueError, match="inner"):
        mm.gemm_i8(q, w[:, :31], s, torch.ones(4, device=dev))
    with pytest.raises(ValueError, match="b_scale"):
        mm.gemm_i8_grouped(q, w[None].expand(2, 4, 32), off, s, torch.ones(4, device=dev))
    with pytest.raises(ValueError, match="shape"):
        mm.quantize_i8(A, out=w)
    torch.cuda.synchronize()
