"""GPU parity of the 4-bit block format: quantisation, the values of the codes, and the products
(plain and grouped), against their definitions in 64 bits.

Bars, from the number formats:
* Codes and scales are equal to the definition's; values of codes are exact in fp32 and bf16.
* Products of two codes' values are exact in fp32. Codes with scale 127 are multiples of 1/2 up to 6,
  so sums of up to 4096 products are multiples of 1/4 below 2^18: fp32 outputs are bit-exact and
  16-bit outputs are the exact sums rounded to nearest even. With random scales fp32 sums lie
  within 1e-5 sum |a b| (the bar of the 16-bit products); a 16-bit output adds half a step, eps / 2 of
  the value (fp16 also 2^-25, half its smallest step).
"""
import numpy as np
import pytest
import torch

import tiled_gemm_gemv_amd as mm
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
TABLE = np.concatenate([VALUES, -VALUES])


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    mm.load()
    return d


def quantized(x):
    """Codes (one to an element, whole blocks) and scales of a float64 matrix, from the definition."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    y = np.zeros((rows, blocks * 32))
    y[:, :cols] = x
    y = y.reshape(rows, blocks, 32)
    codes, scales = np.zeros(y.shape, np.uint8), np.zeros((rows, blocks), np.uint8)
    for i in range(rows):
        for b in range(blocks):
            v = y[i, b]
            top = np.abs(v).max()
            if not np.isfinite(v).all():
                scales[i, b] = 255
                continue
            if top == 0:
                e = -127
            else:
                e = max(int(np.frexp(top)[1]) - 1 - 2, -127)
            scales[i, b] = e + 127
            q = np.minimum(np.abs(v) / 2.0 ** e, 6.0)
            d = np.abs(q[:, None] - VALUES[None, :])
            least = d.min(axis=1, keepdims=True)
            near = d == least  # two of them halfway: the even code
            n = np.argmax(near & (~(near.sum(axis=1, keepdims=True) > 1) | (np.arange(8) % 2 == 0)), axis=1)
            codes[i, b] = n + 8 * np.signbit(v)
    return codes.reshape(rows, -1), scales


def packed(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpacked(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def values(q, s):
    """The values of packed codes and scales, float64 (NaN where the scale is 255)."""
    power = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return TABLE[unpacked(q)] * np.repeat(power, 32, axis=1)


def inside(shape, dtype, gap, offset, dev, fill):
    """A view of the shape with `gap` extra elements per row, `offset` elements into a filled buffer."""
    rows, cols = shape[-2:]
    ld = cols + gap
    step = max(rows, 1) * ld + 3
    count = 1 if len(shape) == 2 else shape[0]
    buf = torch.full((offset + count * step + 32,), fill, dtype=dtype, device=dev)
    strides = (ld, 1) if len(shape) == 2 else (step, ld, 1)
    return buf, torch.as_strided(buf, tuple(shape), strides, offset)


def same(x, q, s):
    codes, scales = quantized(x)
    assert np.array_equal(s, scales), np.argwhere(s != scales)[:5]
    got = unpacked(q)
    # the sign of a zero does not matter
    bad = (got != codes) & ~((got % 8 == 0) & (codes % 8 == 0))
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], codes[bad][:5])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 7), (3, 31), (1, 32), (5, 33), (4, 40), (7, 100), (33, 65), (16, 777),
                                       (3, 1024), (2, 2080), (130, 352), (1, 8193)])
def test_quantize(dev, rows, cols, dtype):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = torch.from_numpy((rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 13, (rows, 1)))).astype(np.float32))
    x = x.to(DT[dtype]).to(dev)
    q, s = mm.quantize_mx4(x)
    blocks = (cols + 31) // 32
    assert q.shape == (rows, 16 * blocks) and s.shape == (rows, blocks)
    want = x.cpu().double().numpy()
    same(want, q.cpu().numpy(), s.cpu().numpy())
    back = mm.dequantize_mx4(q, s, cols=cols, out_dtype=DT[dtype])
    assert np.array_equal(back.cpu().double().numpy(), values(q.cpu().numpy(), s.cpu().numpy())[:, :cols])


@pytest.mark.parametrize("dtype,gap,offset", [("bf16", 3, 1), ("f16", 1, 5), ("f32", 2, 3)])
def test_quantize_strides(dev, dtype, gap, offset):
    rows, cols = 19, 150
    rng = np.random.default_rng(3)
    _, x = inside((rows, cols), DT[dtype], gap, offset, dev, float("nan"))
    x.copy_(torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)))
    qbuf, q = inside((rows, 80), torch.uint8, 3, 5, dev, 0x77)
    sbuf, s = inside((rows, 5), torch.uint8, 2, 1, dev, 0x77)
    mm.quantize_mx4(x, out=q, scale=s)
    same(x.cpu().double().numpy(), q.cpu().numpy(), s.cpu().numpy())
    assert (qbuf != 0x77).sum() <= q.numel() and (sbuf != 0x77).sum() <= s.numel()
    for buf, view in ((qbuf, q), (sbuf, s)):
        kept = buf.clone()
        torch.as_strided(kept, view.shape, view.stride(), view.storage_offset()).fill_(0x77)
        assert bool((kept == 0x77).all())
    obuf, out = inside((rows, cols), DT[dtype], gap, offset, dev, float("nan"))
    mm.dequantize_mx4(q, s, cols=cols, out=out)
    assert np.array_equal(out.cpu().double().numpy(), values(q.cpu().numpy(), s.cpu().numpy())[:, :cols])
    out.fill_(float("nan"))
    assert bool(torch.isnan(obuf).all())


def test_quantize_every_bf16(dev):
    """Every 16-bit pattern: finite ones next to a largest element of each of four powers, and as they
    come (blocks of 32 neighbours, infinities and NaN among them)."""
    bits = np.arange(65536, dtype=np.uint32)
    x = (bits << 16).view(np.float32).reshape(-1, 32)
    t = torch.from_numpy(x.copy()).to(dev)
    for v in (t, t.to(torch.bfloat16)):
        q, s = mm.quantize_mx4(v)
        same(x.astype(np.float64), q.cpu().numpy(), s.cpu().numpy())


def test_quantize_borders(dev):
    """Quotients at and next to every halfway point, for powers over the whole range of fp32."""
    out = []
    for e in [-149, -140, -130, -129, -128, -127, -126, -125, -120, -64, -1, 0, 1, 60, 100, 122, 123, 124, 125]:
        row = []
        for top in (4.0, 5.0, 6.0, 7.0, 7.9999995):
            block = [top]
            for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                block += [m, -m, np.nextafter(np.float32(m), np.float32(0)), -np.nextafter(np.float32(m), np.float32(8))]
            block += [0.0, -0.0, np.float32(1e-30)]
            row += [np.float64(v) * 2.0 ** e for v in block]
        out.append(row)
    x = np.array(out).astype(np.float32)
    q, s = mm.quantize_mx4(torch.from_numpy(x).to(dev))
    same(x.astype(np.float64), q.cpu().numpy(), s.cpu().numpy())


def test_quantize_specials(dev):
    x = torch.zeros(4, 96, device=dev)
    x[0, 5], x[1, 40], x[2, 95] = float("inf"), float("-inf"), float("nan")
    x[:, 64:67] = torch.tensor([1.0, -3.4028235e38, 1e-45], device=dev)
    q, s = mm.quantize_mx4(x)
    same(x.cpu().double().numpy(), q.cpu().numpy(), s.cpu().numpy())
    back = mm.dequantize_mx4(q, s)
    assert bool(torch.isnan(back[0, :32]).all()) and not torch.isnan(back[0, 32:]).any()
    for shape in ((0, 32), (3, 0), (0, 0)):
        q, s = mm.quantize_mx4(torch.empty(shape, device=dev))
        assert q.shape == (shape[0], (shape[1] + 31) // 32 * 16) and s.shape == (shape[0], (shape[1] + 31) // 32)
        assert mm.dequantize_mx4(q, s, cols=shape[1]).shape == shape


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_values_of_every_code_and_scale(dev, dtype):
    s = np.arange(256, dtype=np.uint8)[:, None]
    q = np.tile(np.arange(16, dtype=np.uint8), (256, 1)) | (np.arange(16, dtype=np.uint8)[::-1] << 4)
    out = mm.dequantize_mx4(torch.from_numpy(q).to(dev), torch.from_numpy(s).to(dev), out_dtype=DT[dtype])
    want = torch.from_numpy(values(q, s)).float()  # 6 2^127 is beyond fp32
    want = want.to(DT[dtype]).double().numpy()
    got = out.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


# ------------------------------------------------------------------------------- products

def operand(rng, shape, k, spread, dev, gap=0, offset=0, sgap=0, soffset=0):
    """Random codes and scales: (codes view, scales view, float64 values)."""
    q = rng.integers(0, 256, tuple(shape) + (k // 2,), dtype=np.uint8)
    s = (127 + (rng.integers(-spread, spread + 1, tuple(shape) + (k // 32,)) if spread else 0) *
         np.ones(tuple(shape) + (k // 32,), np.int64)).astype(np.uint8)
    _, qv = inside(q.shape, torch.uint8, gap, offset, dev, 0x77)
    _, sv = inside(s.shape, torch.uint8, sgap, soffset, dev, 0xff)  # NaN around the scales
    qv.copy_(torch.from_numpy(q))
    sv.copy_(torch.from_numpy(s))
    flat = values(q.reshape(-1, k // 2), s.reshape(-1, max(k // 32, 1))[:, :k // 32]) if k and q.size else np.zeros((0, k))
    return qv, sv, flat.reshape(tuple(shape) + (k,))


def check(got, want, S, exact, dtype):
    live = ~np.isnan(want)
    assert np.isnan(got[~live]).all(), "an element that should be NaN or untouched is not"
    assert not np.isnan(got[live]).any(), "NaN in the result"
    if exact:
        rounded = torch.from_numpy(want).to(dtype).double().numpy()
        assert np.array_equal(got[live], rounded[live]), np.abs(got - rounded)[live].max()
        return
    half = 0.0
    if dtype != torch.float32:
        half = np.abs(want) * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -8) + (2.0 ** -25 if dtype == torch.float16 else 0)
    err, tol = np.abs(got - want), 1e-5 * S + half
    assert (err[live] <= tol[live]).all(), float((err[live] / np.maximum(tol[live], 1e-300)).max())


SHAPES = [(1, 1, 32), (1, 16, 64), (3, 5, 96), (2, 33, 128), (5, 40, 160), (1, 100, 256), (17, 64, 288), (16, 130, 512),
          (33, 257, 320), (64, 128, 1024), (100, 200, 2080), (130, 300, 544), (257, 129, 768), (300, 520, 4096),
          (1, 1000, 4096), (4, 2050, 1056), (600, 777, 256), (1, 4100, 224), (40, 96, 4064), (1, 77, 8224)]


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("spread", [0, 6])
@pytest.mark.parametrize("shape", SHAPES)
def test_gemm(dev, shape, spread, out):
    M, N, K = shape
    rng = np.random.default_rng(M + 10 * N + 100 * K + spread)
    a, sa, av = operand(rng, (M,), K, spread, dev)
    b, sb, bv = operand(rng, (N,), K, spread, dev)
    scale = 1.0
    if out == "f16" and spread:  # sums inside the type's range
        sa -= 6
        scale = 2.0 ** -6
    got = mm.gemm_mx4(a, b, sa, sb, out_dtype=DT[out])
    want, S = av @ bv.T * scale, np.abs(av) @ np.abs(bv).T * scale
    if out == "f16":
        want = np.where(np.abs(want) < 65504, want, np.sign(want) * np.inf)
        live = np.isfinite(want)
        check(np.where(live, got.cpu().double().numpy(), 0), np.where(live, want, 0), S, not spread, DT[out])
    else:
        check(got.cpu().double().numpy(), want, S, not spread, DT[out])


@pytest.mark.parametrize("shape", [(1, 300, 992), (9, 64, 352), (40, 130, 1024), (200, 260, 544), (300, 300, 1312),
                                   (1, 513, 4096)])
@pytest.mark.parametrize("gap,offset,sgap,soffset", [(16, 16, 4, 4), (1, 3, 1, 1), (5, 2, 3, 2), (0, 1, 0, 3), (8, 8, 2, 0)])
def test_gemm_strides(dev, shape, gap, offset, sgap, soffset):
    M, N, K = shape
    rng = np.random.default_rng(M + N + K + gap)
    a, sa, av = operand(rng, (M,), K, 0, dev, gap, offset, sgap, soffset)
    b, sb, bv = operand(rng, (N,), K, 0, dev, gap, offset, sgap, soffset)
    buf, out = inside((M, N), torch.float32, gap, offset, dev, float("nan"))
    mm.gemm_mx4(a, b, sa, sb, out=out)
    check(out.cpu().double().numpy(), av @ bv.T, None, True, torch.float32)
    out.fill_(float("nan"))
    assert bool(torch.isnan(buf).all())


@pytest.mark.parametrize("shape", [(1, 64, 512), (1, 200, 4096), (20, 100, 288), (130, 256, 1024), (300, 513, 1056)])
def test_gemm_nan_scales(dev, shape):
    """A block of scale 255 makes its row (column) of the result NaN and nothing else."""
    M, N, K = shape
    rng = np.random.default_rng(K)
    a, sa, av = operand(rng, (M,), K, 3, dev)
    b, sb, bv = operand(rng, (N,), K, 3, dev)
    for at, (t, v) in (((M // 2, K // 32 - 1), (sa, av)), ((N // 3, 0), (sb, bv)), ((N - 1, K // 64), (sb, bv))):
        t[at] = 255
        v[at[0], 32 * at[1]:32 * at[1] + 32] = np.nan
    got = mm.gemm_mx4(a, b, sa, sb).cpu().double().numpy()
    check(got, av @ bv.T, np.abs(np.nan_to_num(av)) @ np.abs(np.nan_to_num(bv)).T, False, torch.float32)


def test_gemm_extreme_scales(dev):
    """Powers at both ends: 2^-127 2^127 = 1, and products beyond fp32 are infinities."""
    K = 512
    rng = np.random.default_rng(1)
    for M, N in ((1, 40), (40, 70), (140, 140)):
        a, sa, av = operand(rng, (M,), K, 0, dev)
        b, sb, bv = operand(rng, (N,), K, 0, dev)
        sa.fill_(0), sb.fill_(254)
        check(mm.gemm_mx4(a, b, sa, sb).cpu().double().numpy(), av @ bv.T, None, True, torch.float32)
        a.fill_(0x77), b.fill_(0x77), sa.fill_(200), sb.fill_(200)
        assert bool(torch.isinf(mm.gemm_mx4(a, b, sa, sb)).all())


def test_gemm_zero_sizes(dev):
    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=dev)
    assert mm.gemm_mx4(zeros(0, 16), zeros(4, 16), zeros(0, 1), zeros(4, 1)).shape == (0, 4)
    assert mm.gemm_mx4(zeros(4, 16), zeros(0, 16), zeros(4, 1), zeros(0, 1)).shape == (4, 0)
    out = torch.full((3, 5), float("nan"), device=dev)
    mm.gemm_mx4(zeros(3, 0), zeros(5, 0), zeros(3, 0), zeros(5, 0), out=out)
    assert bool((out == 0).all())


# (rows of each group, rows before the first, rows after the last, N, K)
GROUPS = [
    ([1], 0, 0, 16, 32),
    ([3, 0, 2], 1, 2, 7, 96),
    ([1, 1, 1, 1], 0, 0, 64, 256),
    ([0, 0, 5, 0], 0, 3, 40, 64),
    ([16, 17, 15, 1], 3, 0, 136, 288),
    ([33, 0, 64, 31, 2], 0, 5, 130, 512),
    ([100, 28, 0, 1, 127], 2, 1, 264, 640),
    ([129, 255, 1], 0, 0, 333, 1056),
    ([257, 256, 0, 300], 0, 7, 512, 1024),
    ([700, 3, 600], 0, 0, 776, 544),
    ([1, 0, 0, 1, 1, 1], 0, 0, 100, 4512),
    ([1, 0, 1, 0, 0, 1, 0, 2], 0, 1, 2048, 2048),
    ([5, 1, 7], 0, 0, 2048, 1024),
    ([40, 2], 0, 0, 1000, 96),
]


@pytest.mark.parametrize("out,spread", [("f32", 0), ("bf16", 5), ("f16", 0)])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped(dev, case, out, spread):
    counts, lead, tail, N, K = GROUPS[case]
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    M = off[-1] + tail
    rng = np.random.default_rng(case)
    a, sa, av = operand(rng, (M,), K, spread, dev)
    b, sb, bv = operand(rng, (len(counts), N), K, spread, dev, 16, 16)
    sa[:lead] = 255          # rows of no group are not read into any other row
    sa[off[-1]:] = 255
    for g, c in enumerate(counts):
        if c == 0:
            sb[g] = 255      # nor an empty group's matrix
    buf, y = inside((M, N), DT[out], 3, 1, dev, float("nan"))
    mm.gemm_mx4_grouped(a, b, torch.tensor(off, device=dev), sa, sb, out=y)
    want, S = np.full((M, N), np.nan), np.zeros((M, N))
    for g in range(len(counts)):
        lo, hi = off[g], off[g + 1]
        want[lo:hi], S[lo:hi] = av[lo:hi] @ bv[g].T, np.abs(av[lo:hi]) @ np.abs(bv[g]).T
    check(y.cpu().double().numpy(), want, S, not spread, DT[out])
    y.fill_(float("nan"))
    assert bool(torch.isnan(buf).all())


def test_grouped_bad_offsets_stay_inside(dev):
    """Offsets outside the rows and falling ones: nothing outside out is written, rows of no group stay."""
    rng = np.random.default_rng(5)
    M, N, K = 70, 90, 512
    a, sa, _ = operand(rng, (M,), K, 0, dev)
    b, sb, _ = operand(rng, (4, N), K, 0, dev)
    for off in ([-5, 10, 10, 2 ** 40, 2 ** 41], [60, 20, 20, 5, 1], [70, 70, 70, 70, 70], [-9, -8, -7, -6, -5]):
        buf, y = inside((M, N), torch.float32, 2, 3, dev, float("nan"))
        mm.gemm_mx4_grouped(a, b, torch.tensor(off, device=dev), sa, sb, out=y)
        torch.cuda.synchronize()
        if off[0] in (70, -9, 60):
            assert bool(torch.isnan(y).all())
        y.fill_(float("nan"))
        assert bool(torch.isnan(buf).all())


def test_captured_and_replayed(dev):
    """Quantisation and a grouped product in a graph: replays follow new inputs and offsets."""
    rng = np.random.default_rng(8)
    M, N, K = 48, 160, 1024
    x = torch.randn(M, K, device=dev)
    b, sb, bv = operand(rng, (3, N), K, 2, dev)
    off = torch.tensor([0, 10, 10, 48], device=dev)
    q, s = mm.quantize_mx4(x)
    y = torch.zeros(M, N, device=dev)
    mm.gemm_mx4_grouped(q, b, off, s, sb, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mm.quantize_mx4(x, out=q, scale=s)
        mm.gemm_mx4_grouped(q, b, off, s, sb, out=y)
    for step in range(4):
        x.copy_(torch.randn(M, K, device=dev) * (step + 1))
        off.copy_(torch.tensor([0, 5 * step, 30, 48], device=dev))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        q2, s2 = mm.quantize_mx4(x)
        want = mm.gemm_mx4_grouped(q2, b, off, s2, sb, out=torch.zeros(M, N, device=dev))
        assert torch.equal(y, want)


def test_other_stream(dev):
    rng = np.random.default_rng(9)
    a, sa, av = operand(rng, (30,), 512, 0, dev)
    b, sb, bv = operand(rng, (50,), 512, 0, dev)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = mm.gemm_mx4(a, b, sa, sb, stream=stream)
    stream.synchronize()
    check(got.cpu().double().numpy(), av @ bv.T, None, True, torch.float32)


@pytest.mark.parametrize("exponent", [-120, 0, 5, 127])
def test_quantize_every_bf16_below(dev, exponent):
    """Every 16-bit pattern below 2^(exponent + 1) in size, in blocks whose largest element is 2^exponent or
    another of its binade: all quotients from there down to 0, the halfway points among them."""
    x = (np.arange(65536, dtype=np.uint32) << 16).view(np.float32)
    x = x[np.abs(x.astype(np.float64)) < 2.0 ** (exponent + 1)]
    x = np.concatenate([x, np.zeros(-len(x) % 31, np.float32)])
    x = np.random.default_rng(0).permutation(x).reshape(-1, 31)
    x = np.concatenate([np.full((len(x), 1), 2.0 ** exponent, np.float32), x], axis=1)
    t = torch.from_numpy(x).to(dev)
    for v in (t, t.to(torch.bfloat16)):
        q, s = mm.quantize_mx4(v)
        assert bool((s == max(exponent - 2, -127) + 127).all())
        same(x.astype(np.float64), q.cpu().numpy(), s.cpu().numpy())
