"""CPU checks of the grouped and the 8-bit products' entry points: argument checks that return
before any HIP call, empty calls that enqueue nothing, and the tensor front ends' refusals.
No kernel is launched."""
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


def grouped(name="bf16", groups=2, M=4, N=5, K=8, offsets=FAKE, A=FAKE, lda=8, B=FAKE, ldb=5, stride_b=40,
            trans_b=0, C=FAKE, c_type=0, ldc=5):
    getattr(mm, f"mm_gemm_{name}_grouped")(groups, M, N, K, offsets, A, lda, B, ldb, stride_b, trans_b, C,
                                           c_type, ldc, stream=0)


def grad_b(name="bf16", groups=2, M=4, N=5, K=8, offsets=FAKE, A=FAKE, lda=8, G=FAKE, ldg=5, D=FAKE, d_type=0,
           ldd=5, stride_d=40):
    getattr(mm, f"mm_gemm_{name}_grouped_grad_b")(groups, M, N, K, offsets, A, lda, G, ldg, D, d_type, ldd,
                                                  stride_d, stream=0)


def i8(M=4, N=5, K=8, A=FAKE, lda=8, sa=FAKE, B=FAKE, ldb=8, sb=FAKE, C=FAKE, c_type=0, ldc=5):
    mm.mm_gemm_i8(M, N, K, A, lda, sa, B, ldb, sb, C, c_type, ldc, stream=0)


def i8_grouped(groups=2, M=4, N=5, K=8, offsets=FAKE, A=FAKE, lda=8, sa=FAKE, B=FAKE, ldb=8, stride_b=40, sb=FAKE,
               C=FAKE, c_type=0, ldc=5):
    mm.mm_gemm_i8_grouped(groups, M, N, K, offsets, A, lda, sa, B, ldb, stride_b, sb, C, c_type, ldc, stream=0)


def quantize(rows=4, cols=8, X=FAKE, x_type=0, ldx=8, Q=FAKE, ldq=8, scale=FAKE):
    mm.mm_quantize_i8(rows, cols, X, x_type, ldx, Q, ldq, scale, stream=0)


BAD = [
    (grouped, dict(groups=-1), "negative size"),
    (grouped, dict(M=-1), "negative size"),
    (grouped, dict(groups=4097), "4096 groups"),
    (grouped, dict(M=1 << 31), "size above"),
    (grouped, dict(N=1 << 31, ldb=1 << 31, ldc=1 << 31), "size above"),
    (grouped, dict(lda=7), "lda"),
    (grouped, dict(ldb=4), "ldb < max(1, N)"),
    (grouped, dict(trans_b=1, ldb=7), "ldb < max(1, K)"),
    (grouped, dict(trans_b=2), "trans_b"),
    (grouped, dict(ldc=4), "ldc"),
    (grouped, dict(c_type=3), "output type"),
    (grouped, dict(c_type=-1), "output type"),
    (grouped, dict(stride_b=-1), "negative group stride"),
    (grouped, dict(offsets=None), "offsets is NULL"),
    (grouped, dict(offsets=FAKE + 4), "offsets not 8-byte"),
    (grouped, dict(A=None), "A is NULL"),
    (grouped, dict(B=None), "B is NULL"),
    (grouped, dict(C=None), "C is NULL"),
    (grouped, dict(A=FAKE + 1), "aligned"),
    (grouped, dict(B=FAKE + 1), "aligned"),
    (grouped, dict(C=FAKE + 2), "aligned"),
    (grouped, dict(C=FAKE + 1, c_type=1), "aligned"),
    (grouped, dict(M=1 << 30, lda=1 << 40), "A extent"),
    (grouped, dict(stride_b=1 << 62), "B extent"),
    (grouped, dict(groups=3, stride_b=1 << 60), "B extent"),
    (grad_b, dict(K=-1), "negative size"),
    (grad_b, dict(lda=7), "lda"),
    (grad_b, dict(ldg=4), "ldg"),
    (grad_b, dict(ldd=4), "ldd"),
    (grad_b, dict(stride_d=-1), "negative group stride"),
    (grad_b, dict(G=None), "G is NULL"),
    (grad_b, dict(D=None), "D is NULL"),
    (grad_b, dict(offsets=None), "offsets is NULL"),
    (grad_b, dict(d_type=7), "output type"),
    (grad_b, dict(groups=3, stride_d=1 << 60), "D extent"),
    (i8, dict(K=-1), "negative size"),
    (i8, dict(K=1 << 17, lda=1 << 17, ldb=1 << 17), "K above"),
    (i8, dict(ldb=7), "ldb"),
    (i8, dict(sa=None), "a_scale is NULL"),
    (i8, dict(sb=None), "b_scale is NULL"),
    (i8, dict(sa=FAKE + 2), "scales"),
    (i8, dict(C=FAKE + 1, c_type=2), "aligned"),
    (i8, dict(c_type=5), "output type"),
    (i8, dict(M=0, ldc=1), "ldc"),
    (i8_grouped, dict(groups=4097), "4096 groups"),
    (i8_grouped, dict(offsets=None), "offsets is NULL"),
    (i8_grouped, dict(stride_b=-8), "negative group stride"),
    (i8_grouped, dict(sb=None), "b_scale is NULL"),
    (quantize, dict(rows=-1), "negative size"),
    (quantize, dict(cols=1 << 31, ldx=1 << 31, ldq=1 << 31), "size above"),
    (quantize, dict(x_type=3), "input type"),
    (quantize, dict(ldx=7), "ldx"),
    (quantize, dict(ldq=7), "ldq"),
    (quantize, dict(X=None), "X is NULL"),
    (quantize, dict(Q=None), "Q is NULL"),
    (quantize, dict(scale=None), "scale is NULL"),
    (quantize, dict(X=FAKE + 2), "aligned"),
    (quantize, dict(X=FAKE + 1, x_type=1), "aligned"),
    (quantize, dict(rows=1 << 30, ldx=1 << 40), "extent"),
]


@pytest.mark.parametrize("call,change,why", BAD)
def test_refused(call, change, why):
    with pytest.raises(mm.MMError) as e:
        call(**change)
    assert e.value.status == mm.MM_ERR_INVALID_ARG
    assert why in str(e.value)


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_both_formats_check(name):
    for call in (grouped, grad_b):
        with pytest.raises(mm.MMError, match="lda"):
            call(name=name, lda=1)


@pytest.mark.parametrize("call,change", [
    (grouped, dict(groups=0, offsets=None, A=None, B=None, C=None)),
    (grouped, dict(M=0, A=None, C=None)),
    (grouped, dict(N=0, ldb=1, ldc=1, B=None, C=None)),
    (grad_b, dict(groups=0, offsets=None, A=None, G=None, D=None)),
    (grad_b, dict(N=0, ldg=1, ldd=1, G=None, D=None)),
    (grad_b, dict(K=0, lda=1, A=None, D=None)),
    (i8, dict(M=0, A=None, sa=None, C=None)),
    (i8, dict(N=0, ldc=1, B=None, sb=None, C=None)),
    (i8_grouped, dict(groups=0, offsets=None, A=None, B=None, C=None, sa=None, sb=None)),
    (quantize, dict(rows=0, X=None, Q=None, scale=None)),
])
def test_empty_calls_enqueue_nothing(call, change):
    call(**change)  # no device here: a launch would raise


def test_front_ends_refuse_host_tensors_and_wrong_types():
    a16, b16 = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 5, dtype=torch.bfloat16)
    off = torch.tensor([0, 2, 4])
    with pytest.raises(ValueError, match="GPU"):
        mm.gemm16_grouped(a16, b16, off)
    with pytest.raises(ValueError, match="GPU"):
        mm.gemm16_grouped_grad_b(a16, torch.zeros(4, 5, dtype=torch.bfloat16), off)
    with pytest.raises(TypeError):
        mm.gemm16_grouped(a16.float(), b16, off)
    a8, b8 = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(5, 8, dtype=torch.int8)
    with pytest.raises(ValueError, match="GPU"):
        mm.gemm_i8(a8, b8, torch.ones(4), torch.ones(5))
    with pytest.raises(TypeError):
        mm.gemm_i8(a8.short(), b8, torch.ones(4), torch.ones(5))
    with pytest.raises(ValueError, match="GPU"):
        mm.gemm_i8_grouped(a8, b8[None], torch.tensor([0, 4]), torch.ones(4), torch.ones(1, 5))
    with pytest.raises(ValueError, match="GPU"):
        mm.quantize_i8(torch.zeros(4, 8))
    with pytest.raises(TypeError):
        mm.quantize_i8(torch.zeros(4, 8, dtype=torch.float64))


def test_matrices_apart():
    """The check of an output's strides against a count of the elements' addresses."""
    for count in (2, 3, 5):
        for rows in (1, 2, 3):
            for cols in (1, 2, 4):
                for stride in range(0, 14):
                    for ld in range(cols, 25):
                        at = {g * stride + i * ld + j for g in range(count) for i in range(rows) for j in range(cols)}
                        if mm._apart(count, stride, rows, ld, cols):
                            assert len(at) == count * rows * cols, (count, stride, rows, ld, cols)
    assert mm._apart(3, 20, 4, 5, 5) and not mm._apart(3, 19, 4, 5, 5)    # one after the other
    assert mm._apart(3, 5, 4, 15, 5) and not mm._apart(3, 5, 4, 14, 5)    # row by row in turn
    assert not mm._apart(2, 0, 4, 100, 5)
