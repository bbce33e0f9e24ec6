"""Empty operands through the tensor front ends: their strides are arbitrary (a slice, an expanded or
a transposed tensor may hold any) and nothing uses them. An empty inner size gives zeros."""
import pytest
import torch

import tiled_gemm_gemv_amd as mm
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

STRIDES = [(1, 1), (0, 1), (3, 5), (7, 0), (0, 0)]


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    mm.load()
    return d


def empty(rows, cols, strides, dtype, dev):
    assert rows == 0 or cols == 0
    return torch.empty_strided((rows, cols), strides, dtype=dtype, device=dev)


@pytest.mark.parametrize("strides", STRIDES)
def test_empty_inner_size_gives_zeros(dev, strides):
    for fn, dtypes in ((mm.gemm, [torch.float32]), (mm.gemm16, [torch.bfloat16, torch.float16])):
        for dtype in dtypes:
            A, B = empty(4, 0, strides, dtype, dev), empty(0, 5, strides, dtype, dev)
            buf = torch.full((5, 7), float("nan"), device=dev)
            out = fn(A, B, out=buf[:4, :5])
            torch.cuda.synchronize()
            assert (out == 0).all().item()
            out.fill_(float("nan"))
            assert torch.isnan(buf).all().item(), "wrote outside out"
    A, B = (torch.empty_strided(s, (9,) + strides, device=dev) for s in ((2, 4, 0), (2, 0, 5)))
    out = mm.gemm_batched(A, B, out=torch.full((2, 4, 5), float("nan"), device=dev))
    torch.cuda.synchronize()
    assert (out == 0).all().item()


@pytest.mark.parametrize("strides", STRIDES)
def test_empty_outputs(dev, strides):
    for fn, dtype in ((mm.gemm, torch.float32), (mm.gemm16, torch.bfloat16)):
        full = torch.ones((3, 5), dtype=dtype, device=dev)
        for A, B, shape in ((empty(0, 3, strides, dtype, dev), full, (0, 5)),
                            (full.t().contiguous(), empty(3, 0, strides, dtype, dev), (5, 0)),
                            (empty(0, 0, strides, dtype, dev), empty(0, 5, strides, dtype, dev), (0, 5))):
            assert fn(A, B).shape == shape
            out = empty(*shape, strides, torch.float32, dev)
            assert fn(A, B, out=out) is out
    torch.cuda.synchronize()


def test_strides_of_others_still_count(dev):
    A, B = torch.ones((4, 3), device=dev), torch.ones((3, 5), device=dev)
    with pytest.raises(ValueError, match="unit column stride"):
        mm.gemm(A, B.t().contiguous().t())
    with pytest.raises(ValueError, match="row stride"):
        mm.gemm(A[:1].expand(4, 3), B)
