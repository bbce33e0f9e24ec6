"""CPU checks of the entry points of the routing, the experts' rows and the 4-bit blocks: argument
checks that return before any HIP call, empty calls that enqueue nothing, workspace sizes, and the
tensor front ends' refusals. No kernel is launched."""
import os

import pytest
import torch

import tiled_gemm_gemv_amd as mm
from tiled_gemm_gemv_amd import build as mm_build

FAKE = 1 << 40  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(mm_build.LIB):
        mm_build.build()
    return mm.load()


def quantize(rows=4, cols=70, X=FAKE, x_type=0, ldx=70, Q=FAKE, ldq=48, scale=FAKE, ld_scale=3):
    mm.mm_quantize_mx4(rows, cols, X, x_type, ldx, Q, ldq, scale, ld_scale, stream=0)


def dequantize(rows=4, cols=70, X=FAKE, x_type=0, ldx=70, Q=FAKE, ldq=48, scale=FAKE, ld_scale=3):
    mm.mm_dequantize_mx4(rows, cols, Q, ldq, scale, ld_scale, X, x_type, ldx, stream=0)


def gemm(M=4, N=5, K=64, A=FAKE, lda=32, sa=FAKE, ld_as=2, B=FAKE, ldb=32, sb=FAKE, ld_bs=2, C=FAKE, c_type=0, ldc=5):
    mm.mm_gemm_mx4(M, N, K, A, lda, sa, ld_as, B, ldb, sb, ld_bs, C, c_type, ldc, stream=0)


def grouped(groups=2, M=4, N=5, K=64, offsets=FAKE, A=FAKE, lda=32, sa=FAKE, ld_as=2, B=FAKE, ldb=32, stride_b=160,
            sb=FAKE, ld_bs=2, stride_bs=10, C=FAKE, c_type=0, ldc=5):
    mm.mm_gemm_mx4_grouped(groups, M, N, K, offsets, A, lda, sa, ld_as, B, ldb, stride_b, sb, ld_bs, stride_bs, C,
                           c_type, ldc, stream=0)


def route(T=4, E=12, k=3, logits=FAKE, type=0, ld=12, scoring=0, bias=None, groups=1, top_groups=1, group_top=1,
          renormalize=0, scale=1.0, weights=FAKE, experts=FAKE, rows=FAKE, offsets=FAKE, workspace=None, size=0):
    mm.mm_route_topk(T, E, k, logits, type, ld, scoring, bias, groups, top_groups, group_top, renormalize, scale,
                     weights, experts, rows, offsets, workspace, size, stream=0)


def route_grad(T=4, E=12, k=3, logits=FAKE, type=0, ld=12, scoring=0, renormalize=0, scale=1.0, experts=FAKE,
               dweights=FAKE, dlogits=FAKE, ldd=12):
    mm.mm_route_topk_grad(T, E, k, logits, type, ld, scoring, renormalize, scale, experts, dweights, dlogits, ldd,
                          stream=0)


def spread(T=4, k=2, row_bytes=10, X=FAKE, ldx=10, rows=FAKE, total=8, Y=FAKE, ldy=10):
    mm.mm_spread_rows(T, k, row_bytes, X, ldx, rows, total, Y, ldy, stream=0)


def combine(T=4, k=2, D=10, Y=FAKE, y_type=0, ldy=10, total=8, rows=FAKE, weights=None, C=FAKE, c_type=0, ldc=10):
    mm.mm_combine_rows(T, k, D, Y, y_type, ldy, total, rows, weights, C, c_type, ldc, stream=0)


def combine_grad(T=4, k=2, D=10, G=FAKE, g_type=0, ldg=10, Y=FAKE, y_type=0, ldy=10, total=8, rows=FAKE, weights=FAKE,
                 dY=FAKE, lddy=10, dweights=FAKE):
    mm.mm_combine_rows_grad(T, k, D, G, g_type, ldg, Y, y_type, ldy, total, rows, weights, dY, lddy, dweights, stream=0)


BAD = [(call, change, why) for call in (quantize, dequantize) for change, why in [
    (dict(rows=-1), "negative size"),
    (dict(cols=1 << 31, ldx=1 << 31, ldq=1 << 31, ld_scale=1 << 31), "size above"),
    (dict(x_type=3), "type"),
    (dict(ldx=69), "ldx"),
    (dict(ldq=47), "ldq"),
    (dict(ld_scale=2), "ld_scale"),
    (dict(X=None), "X is NULL"),
    (dict(Q=None), "Q is NULL"),
    (dict(scale=None), "scale is NULL"),
    (dict(X=FAKE + 2), "aligned"),
    (dict(X=FAKE + 1, x_type=1), "aligned"),
    (dict(rows=1 << 30, ldx=1 << 40), "extent"),
    (dict(rows=1 << 30, ldq=1 << 40), "extent"),
    (dict(rows=1 << 30, ld_scale=1 << 40), "extent"),
]] + [(call, change, why) for call in (gemm, grouped) for change, why in [
    (dict(K=48), "multiple of 32"),
    (dict(K=-32), "negative size"),
    (dict(M=-1), "negative size"),
    (dict(N=1 << 31, ldc=1 << 31), "size above"),
    (dict(lda=31), "lda < max(1, K / 2)"),
    (dict(ldb=31), "ldb < max(1, K / 2)"),
    (dict(ldc=4), "ldc"),
    (dict(ld_as=1), "a_scale < max"),
    (dict(ld_bs=1), "b_scale < max"),
    (dict(c_type=3), "output type"),
    (dict(A=None), "A is NULL"),
    (dict(B=None), "B is NULL"),
    (dict(C=None), "C is NULL"),
    (dict(sa=None), "a_scale is NULL"),
    (dict(sb=None), "b_scale is NULL"),
    (dict(C=FAKE + 2), "aligned"),
    (dict(M=1 << 30, lda=1 << 40), "A extent"),
    (dict(M=1 << 30, ld_as=1 << 40), "a_scale extent"),
    (dict(N=1 << 30, ldb=1 << 40, ldc=1 << 30), "B extent"),
    (dict(N=1 << 30, ld_bs=1 << 40, ldc=1 << 30), "b_scale extent"),
]] + [
    (grouped, dict(groups=-1), "negative size"),
    (grouped, dict(groups=4097), "4096 groups"),
    (grouped, dict(offsets=None), "offsets is NULL"),
    (grouped, dict(offsets=FAKE + 4), "offsets not 8-byte"),
    (grouped, dict(stride_b=-1), "negative group stride"),
    (grouped, dict(stride_bs=-1), "negative group stride"),
    (grouped, dict(groups=3, stride_b=1 << 61), "B extent"),
    (grouped, dict(groups=3, stride_bs=1 << 61), "b_scale extent"),
] + [(call, change, why) for call in (route, route_grad) for change, why in [
    (dict(T=-1), "negative size"),
    (dict(E=1025, ld=1025), "1024 experts"),
    (dict(E=100, ld=100, k=33), "32 experts"),
    (dict(k=13), "more experts to a token than there are"),
    (dict(T=1 << 30), "T k above"),
    (dict(type=3), "type of the logits"),
    (dict(scoring=2), "scoring"),
    (dict(renormalize=2), "renormalize"),
    (dict(ld=11), "ld < max"),
    (dict(logits=None), "logits is NULL"),
    (dict(logits=FAKE + 2), "aligned"),
    (dict(ld=1 << 62), "logits extent"),
    (dict(experts=None), "experts is NULL"),
    (dict(experts=FAKE + 1), "aligned"),
]] + [
    (route, dict(groups=0), "groups outside"),
    (route, dict(groups=65), "groups outside"),
    (route, dict(groups=5), "multiple of groups"),
    (route, dict(groups=4, top_groups=0), "top_groups"),
    (route, dict(groups=4, top_groups=5), "top_groups"),
    (route, dict(groups=4, top_groups=2, group_top=3), "group_top"),
    (route, dict(groups=6, top_groups=1), "kept groups"),
    (route, dict(weights=None), "weights is NULL"),
    (route, dict(rows=None), "rows is NULL"),
    (route, dict(offsets=None), "offsets is NULL"),
    (route, dict(offsets=FAKE + 4), "offsets not 8-byte"),
    (route, dict(bias=FAKE + 2), "aligned"),
    (route, dict(T=100000), "workspace is NULL"),
    (route, dict(T=100000, workspace=FAKE + 4, size=1 << 30), "16-byte aligned"),
    (route, dict(T=100000, workspace=FAKE, size=16), "workspace smaller"),
    (route_grad, dict(dweights=None), "dweights is NULL"),
    (route_grad, dict(dlogits=None), "dlogits is NULL"),
    (route_grad, dict(ldd=11), "ldd"),
    (route_grad, dict(dlogits=FAKE + 1, type=1), "aligned"),
    (route_grad, dict(ldd=1 << 62), "dlogits extent"),
] + [(call, change, why) for call in (spread, combine, combine_grad) for change, why in [
    (dict(T=-1), "negative size"),
    (dict(total=-1), "negative size"),
    (dict(total=1 << 31), "size above"),
    (dict(T=1 << 30, k=2), "T k above"),
    (dict(k=1025), "1024 slots"),
    (dict(T=1, k=(1 << 31) - 1), "1024 slots"),
    (dict(rows=None), "rows is NULL"),
    (dict(rows=FAKE + 2), "rows not 4-byte"),
    (dict(Y=None), "Y is NULL"),
    (dict(ldy=9), "ldy"),
    (dict(ldy=1 << 62), "Y extent"),
]] + [
    (spread, dict(X=None), "X is NULL"),
    (spread, dict(ldx=9), "ldx"),
    (spread, dict(row_bytes=1 << 31, ldx=1 << 31, ldy=1 << 31), "size above"),
    (combine, dict(C=None), "C is NULL"),
    (combine, dict(ldc=9), "ldc"),
    (combine, dict(y_type=4), "input type"),
    (combine, dict(c_type=-1), "output type"),
    (combine, dict(weights=FAKE + 1), "aligned"),
    (combine, dict(C=FAKE + 1, c_type=1), "aligned"),
    (combine_grad, dict(G=None), "G is NULL"),
    (combine_grad, dict(dY=None), "dY is NULL"),
    (combine_grad, dict(weights=None), "weights is NULL"),
    (combine_grad, dict(dweights=None), "dweights is NULL"),
    (combine_grad, dict(lddy=9), "lddy"),
    (combine_grad, dict(ldg=9), "ldg"),
    (combine_grad, dict(g_type=9), "input type"),
    (combine_grad, dict(G=FAKE + 2), "aligned"),
]


@pytest.mark.parametrize("call,change,why", BAD)
def test_refused(call, change, why):
    with pytest.raises(mm.MMError) as e:
        call(**change)
    assert e.value.status == mm.MM_ERR_INVALID_ARG
    assert why in str(e.value)


@pytest.mark.parametrize("call,change", [
    (quantize, dict(rows=0, X=None, Q=None, scale=None)),
    (dequantize, dict(cols=0, ldx=1, ldq=1, ld_scale=1, X=None, Q=None, scale=None)),
    (gemm, dict(M=0, A=None, sa=None, C=None)),
    (gemm, dict(N=0, ldc=1, B=None, sb=None, C=None)),
    (grouped, dict(groups=0, offsets=None, A=None, B=None, C=None, sa=None, sb=None)),
    (route_grad, dict(T=0, logits=None, experts=None, dweights=None, dlogits=None)),
    (spread, dict(T=0, X=None, rows=None, Y=None)),
    (spread, dict(total=0, X=None, Y=None)),
    (spread, dict(row_bytes=0, X=None, Y=None)),
    (combine, dict(T=0, rows=None, C=None, Y=None)),
    (combine, dict(D=0, C=None, Y=None)),
    (combine_grad, dict(k=0, rows=None, G=None, Y=None, dY=None, weights=None, dweights=None)),
])
def test_empty_calls_enqueue_nothing(call, change):
    call(**change)  # no device here: a launch would raise


def test_workspace_sizes():
    ws = mm.mm_route_topk_workspace_bytes
    assert ws(0, 8, 2) == ws(100, 8, 0) == ws(1, 64, 8) == 0
    assert ws(-1, 8, 2) == ws(4, 1025, 2) == ws(4, 64, 33) == ws(4, 8, 9) == ws(1 << 30, 8, 4) == -1
    assert ws(100000, 256, 8) > 0 and ws(100000, 256, 8) % 4 == 0
    with pytest.raises(ValueError, match="invalid sizes"):
        mm.route_topk_workspace(4, 8, 9, "cpu")


def test_front_ends_refuse_host_tensors_and_wrong_types():
    u8 = torch.zeros(4, 16, dtype=torch.uint8)
    s = torch.zeros(4, 1, dtype=torch.uint8)
    x, rows = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    off = torch.tensor([0, 4])
    for call, args in ((mm.quantize_mx4, (x,)), (mm.dequantize_mx4, (u8, s)), (mm.gemm_mx4, (u8, u8, s, s)),
                       (mm.gemm_mx4_grouped, (u8, u8[None], off, s, s[None])), (mm.route_topk, (x, 2)),
                       (mm.route_topk_grad, (x, rows, torch.zeros(4, 2))), (mm.spread_rows, (x, rows)),
                       (mm.combine_rows, (x, rows)), (mm.combine_rows_grad, (x, x, rows, torch.zeros(4, 2)))):
        with pytest.raises(ValueError, match="GPU"):
            call(*args)
    for call, args in ((mm.quantize_mx4, (x.double(),)), (mm.dequantize_mx4, (u8.char(), s)),
                       (mm.gemm_mx4, (u8.short(), u8, s, s)), (mm.route_topk, (x.double(), 2)),
                       (mm.spread_rows, (x.double(), rows)), (mm.combine_rows, (x.char(), rows))):
        with pytest.raises(TypeError):
            call(*args)
