"""fp32 GEMM and GEMV on one AMD Instinct MI355X, through libmm's C ABI.

The functions named like the C entry points (mm_gemm_f32, mm_gemv_f32, ...)
marshal their arguments and call libmm.so; every step of the computation runs in
the library's HIP kernels. Pointer arguments accept a device address (int) or a
torch tensor on the GPU; `stream` accepts a hipStream_t address (int), a
torch.cuda.Stream, or None for torch's current stream on the current device.

gemm(A, B, out=None), gemv(A, x, out=None), conv2d(x, w, ...), gemm16_grouped(A, B, offsets),
gemm_i8(A, B, a_scale, b_scale), gemm_mx4(A, B, a_scale, b_scale), route_topk(logits, k)
etc. are conveniences for torch tensors: they check dtypes, devices and strides (not those of
empty tensors, which are arbitrary), allocate the output with torch when none is given, and call the C entry points. PyTorch
only provides device memory and streams here.

There is no fallback: if libmm.so is missing or fails to load, every call raises.
Build it with `python -m tiled_gemm_gemv_amd.build`.
"""
import ctypes
import os

# the library build.py writes (not imported from there, so that `python -m
# tiled_gemm_gemv_amd.build` runs the module once)
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmm.so")

MM_OK = 0
MM_ERR_INVALID_ARG = 1
MM_ERR_NO_DEVICE = 2
MM_ERR_LAUNCH = 3


class MMError(RuntimeError):
    """A libmm call returned a non-zero status."""

    def __init__(self, status, where, detail=""):
        self.status = status
        text = _lib_or_none().mm_status_string(status).decode() if _lib_or_none() else str(status)
        msg = f"{where}: {text} (status {status})"
        if detail:
            msg += f": {detail}"
        super().__init__(msg)


_lib = None
_torch = None  # once a front end has been called; an import statement takes 0.1 us of each function


def _lib_or_none():
    return _lib


def _import_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libmm.so (once). Raises OSError if it is missing or cannot be loaded."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise OSError(f"{_LIB_PATH} is not built; run `python -m tiled_gemm_gemv_amd.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.mm_gemm_f32.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.mm_gemm_f32.restype = ci
    lib.mm_gemm_f32_config.argtypes = [ci, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.mm_gemm_f32_config.restype = ci
    lib.mm_gemm_f32_num_configs.argtypes = []
    lib.mm_gemm_f32_num_configs.restype = ci
    lib.mm_gemm_f32_config_name.argtypes = [ci]
    lib.mm_gemm_f32_config_name.restype = ctypes.c_char_p
    lib.mm_gemm_f32_select.argtypes = [i64, i64, i64]
    lib.mm_gemm_f32_select.restype = ci
    lib.mm_gemm_f32_batched.argtypes = [i64, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64,
                                        i64, vp]
    lib.mm_gemm_f32_batched.restype = ci
    for name in ("mm_gemm_bf16", "mm_gemm_f16"):
        getattr(lib, name).argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
        getattr(lib, name).restype = ci
    for name in ("mm_gemm_bf16_config", "mm_gemm_f16_config"):
        getattr(lib, name).argtypes = [ci, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
        getattr(lib, name).restype = ci
    lib.mm_gemm_h16_num_configs.argtypes = []
    lib.mm_gemm_h16_num_configs.restype = ci
    lib.mm_gemm_h16_config_name.argtypes = [ci]
    lib.mm_gemm_h16_config_name.restype = ctypes.c_char_p
    lib.mm_gemm_h16_select.argtypes = [i64, i64, i64]
    lib.mm_gemm_h16_select.restype = ci
    lib.mm_gemv_f32.argtypes = [i64, i64, vp, vp, vp, vp]
    lib.mm_gemv_t_f32.argtypes = [i64, i64, vp, vp, vp, vp]
    lib.mm_gemv_t_f32.restype = ci
    lib.mm_gemm_f32_workspace_bytes.argtypes = [i64, i64, i64]
    lib.mm_gemm_f32_workspace_bytes.restype = i64
    lib.mm_gemm_f32_ws.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.mm_gemm_f32_ws.restype = ci
    lib.mm_gemm_f32_ws_static.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    lib.mm_gemm_f32_ws_static.restype = ci
    lib.mm_gemv_t_f32_workspace_bytes.argtypes = [i64, i64]
    lib.mm_gemv_t_f32_workspace_bytes.restype = i64
    lib.mm_gemv_t_f32_ws.argtypes = [i64, i64, vp, vp, vp, vp, i64, vp]
    lib.mm_gemv_t_f32_ws.restype = ci
    lib.mm_gemv_f32.restype = ci
    conv_args = [i64] * 13 + [vp, vp, vp, vp]
    lib.mm_conv2d_f32.argtypes = conv_args
    lib.mm_conv2d_f32.restype = ci
    lib.mm_conv2d_f32_config.argtypes = [ci] + conv_args
    lib.mm_conv2d_f32_config.restype = ci
    lib.mm_conv2d_out_dim.argtypes = [i64] * 5
    lib.mm_conv2d_out_dim.restype = i64
    lib.mm_conv2d_f32_num_configs.argtypes = []
    lib.mm_conv2d_f32_num_configs.restype = ci
    lib.mm_conv2d_f32_config_name.argtypes = [ci]
    lib.mm_conv2d_f32_config_name.restype = ctypes.c_char_p
    lib.mm_conv2d_f32_select.argtypes = [i64] * 13
    lib.mm_conv2d_f32_select.restype = ci
    for name in ("mm_gemm_bf16_grouped", "mm_gemm_f16_grouped"):
        getattr(lib, name).argtypes = [i64] * 4 + [vp, vp, i64, vp, i64, i64, ci, vp, ci, i64, vp]
        getattr(lib, name).restype = ci
    for name in ("mm_gemm_bf16_grouped_grad_b", "mm_gemm_f16_grouped_grad_b"):
        getattr(lib, name).argtypes = [i64] * 4 + [vp, vp, i64, vp, i64, vp, ci, i64, i64, vp]
        getattr(lib, name).restype = ci
    lib.mm_quantize_i8.argtypes = [i64, i64, vp, ci, i64, vp, i64, vp, vp]
    lib.mm_quantize_i8.restype = ci
    lib.mm_gemm_i8.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, ci, i64, vp]
    lib.mm_gemm_i8.restype = ci
    lib.mm_gemm_i8_grouped.argtypes = [i64] * 4 + [vp, vp, i64, vp, vp, i64, i64, vp, vp, ci, i64, vp]
    lib.mm_gemm_i8_grouped.restype = ci
    lib.mm_quantize_mx4.argtypes = [i64, i64, vp, ci, i64, vp, i64, vp, i64, vp]
    lib.mm_dequantize_mx4.argtypes = [i64, i64, vp, i64, vp, i64, vp, ci, i64, vp]
    lib.mm_gemm_mx4.argtypes = [i64] * 3 + [vp, i64, vp, i64, vp, i64, vp, i64, vp, ci, i64, vp]
    lib.mm_gemm_mx4_grouped.argtypes = [i64] * 4 + [vp, vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp, ci, i64, vp]
    lib.mm_gemm_mx4_select.argtypes = [i64] * 3 + [vp, i64, vp, i64, vp, i64, vp, i64]
    lib.mm_gemm_mx4_grouped_select.argtypes = [i64] * 4 + [vp, i64, vp, i64, vp, i64, i64, vp, i64, i64]
    f32 = ctypes.c_float
    lib.mm_route_topk_workspace_bytes.argtypes = [i64, i64, i64]
    lib.mm_route_topk_workspace_bytes.restype = i64
    lib.mm_route_topk.argtypes = [i64] * 3 + [vp, ci, i64, ci, vp, i64, i64, i64, ci, f32, vp, vp, vp, vp, vp, i64, vp]
    lib.mm_route_topk_grad.argtypes = [i64] * 3 + [vp, ci, i64, ci, ci, f32, vp, vp, vp, i64, vp]
    lib.mm_spread_rows.argtypes = [i64] * 3 + [vp, i64, vp, i64, vp, i64, vp]
    lib.mm_combine_rows.argtypes = [i64] * 3 + [vp, ci, i64, i64, vp, vp, vp, ci, i64, vp]
    lib.mm_combine_rows_grad.argtypes = [i64] * 3 + [vp, ci, i64, vp, ci, i64, i64, vp, vp, vp, i64, vp, vp]
    for name in ("mm_quantize_mx4", "mm_dequantize_mx4", "mm_gemm_mx4", "mm_gemm_mx4_grouped", "mm_gemm_mx4_select",
                 "mm_gemm_mx4_grouped_select", "mm_route_topk", "mm_route_topk_grad", "mm_spread_rows",
                 "mm_combine_rows", "mm_combine_rows_grad"):
        getattr(lib, name).restype = ci
    lib.mm_gemm_grouped_num_configs.argtypes = []
    lib.mm_gemm_grouped_num_configs.restype = ci
    lib.mm_gemm_grouped_config_name.argtypes = [ci]
    lib.mm_gemm_grouped_config_name.restype = ctypes.c_char_p
    lib.mm_gemm_h16_grouped_select.argtypes = [i64] * 4 + [vp, i64, vp, i64, i64, ci]
    lib.mm_gemm_h16_grouped_grad_b_select.argtypes = [i64] * 4 + [vp, i64, vp, i64]
    lib.mm_gemm_i8_select.argtypes = [i64] * 3 + [vp, i64, vp, i64]
    lib.mm_gemm_i8_grouped_select.argtypes = [i64] * 4 + [vp, i64, vp, i64, i64]
    for name in ("mm_gemm_h16_grouped_select", "mm_gemm_h16_grouped_grad_b_select", "mm_gemm_i8_select",
                 "mm_gemm_i8_grouped_select"):
        getattr(lib, name).restype = ci
    lib.mm_status_string.argtypes = [ci]
    lib.mm_status_string.restype = ctypes.c_char_p
    lib.mm_last_error.argtypes = []
    lib.mm_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


# ----------------------------------------------------------------- marshalling

def _addr(p):
    """Device address of an int, None or torch tensor."""
    if p is None:
        return None
    if isinstance(p, int):
        return p or None
    if hasattr(p, "data_ptr"):
        return p.data_ptr() or None
    raise TypeError(f"expected a device address or a tensor, got {type(p).__name__}")


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(s, int):
        return s or None
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream or None
    raise TypeError(f"expected a stream address or torch.cuda.Stream, got {type(s).__name__}")


def _check(status, where):
    if status != MM_OK:
        raise MMError(status, where, load().mm_last_error().decode())


# ------------------------------------------------------- C entry points by name

def mm_gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    """C = A x B (row-major, leading dimensions lda, ldb, ldc). Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f32(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                           _stream(stream)), "mm_gemm_f32")


def mm_gemm_f32_config(cfg, M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    """mm_gemm_f32 with tile configuration `cfg` forced. Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f32_config(cfg, M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                                  _stream(stream)), "mm_gemm_f32_config")


def mm_gemm_f32_batched(batch, M, N, K, A, lda, stride_a, B, ldb, stride_b, C, ldc, stride_c,
                        stream=None):
    """C_b = A_b x B_b for b < batch, operands offset by b * stride. Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f32_batched(batch, M, N, K, _addr(A), lda, stride_a, _addr(B), ldb,
                                   stride_b, _addr(C), ldc, stride_c, _stream(stream)),
           "mm_gemm_f32_batched")


def mm_gemm_bf16(M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    """C (fp32) = A x B with bf16 A and B. Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_bf16(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                            _stream(stream)), "mm_gemm_bf16")


def mm_gemm_f16(M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    """C (fp32) = A x B with fp16 A and B. Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f16(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                           _stream(stream)), "mm_gemm_f16")


def mm_gemm_bf16_config(cfg, M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    lib = load()
    _check(lib.mm_gemm_bf16_config(cfg, M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                                   _stream(stream)), "mm_gemm_bf16_config")


def mm_gemm_f16_config(cfg, M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    lib = load()
    _check(lib.mm_gemm_f16_config(cfg, M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                                  _stream(stream)), "mm_gemm_f16_config")


def mm_gemm_h16_num_configs():
    return load().mm_gemm_h16_num_configs()


def mm_gemm_h16_config_name(cfg):
    name = load().mm_gemm_h16_config_name(cfg)
    return name.decode() if name is not None else None


def mm_gemm_h16_select(M, N, K):
    return load().mm_gemm_h16_select(M, N, K)


def mm_gemv_f32(M, N, A, x, y, stream=None):
    """y = A x (A M x N with packed rows). Raises MMError."""
    lib = load()
    _check(lib.mm_gemv_f32(M, N, _addr(A), _addr(x), _addr(y), _stream(stream)), "mm_gemv_f32")


def mm_gemv_t_f32(M, N, A, x, y, stream=None):
    """y = A^T x (A M x N with packed rows, x of M, y of N). Raises MMError."""
    lib = load()
    _check(lib.mm_gemv_t_f32(M, N, _addr(A), _addr(x), _addr(y), _stream(stream)),
           "mm_gemv_t_f32")


def mm_gemm_f32_workspace_bytes(M, N, K):
    """Bytes of workspace mm_gemm_f32_ws needs for (M, N, K); -1 for invalid sizes."""
    return load().mm_gemm_f32_workspace_bytes(M, N, K)


def mm_gemm_f32_ws(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, stream=None):
    """C = A B, splitting K across workgroups through `workspace` where that pays.
    Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f32_ws(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc, _addr(workspace),
                              workspace_bytes, _stream(stream)), "mm_gemm_f32_ws")


def mm_gemm_f32_ws_static(M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    """mm_gemm_f32_ws with the library's static device scratch (MM_STATIC_SCRATCH_BYTES per
    GPU) as its workspace: allocates nothing. Calls that overlap on one GPU race.
    Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f32_ws_static(M, N, K, _addr(A), lda, _addr(B), ldb, _addr(C), ldc,
                                     _stream(stream)), "mm_gemm_f32_ws_static")


MM_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024  # as include/mm.h defines it


def mm_gemv_t_f32_workspace_bytes(M, N):
    """Bytes of workspace mm_gemv_t_f32_ws needs for (M, N); -1 for invalid sizes."""
    return load().mm_gemv_t_f32_workspace_bytes(M, N)


def mm_gemv_t_f32_ws(M, N, A, x, y, workspace, workspace_bytes, stream=None):
    """y = A^T x reading A along whole rows, partial sums in `workspace`. Raises MMError."""
    lib = load()
    _check(lib.mm_gemv_t_f32_ws(M, N, _addr(A), _addr(x), _addr(y), _addr(workspace), workspace_bytes,
                                _stream(stream)), "mm_gemv_t_f32_ws")


def mm_gemm_f32_num_configs():
    return load().mm_gemm_f32_num_configs()


def mm_gemm_f32_config_name(cfg):
    name = load().mm_gemm_f32_config_name(cfg)
    return name.decode() if name is not None else None


def mm_gemm_f32_select(M, N, K):
    return load().mm_gemm_f32_select(M, N, K)


def mm_conv2d_f32(N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, x, w, y, stream=None):
    """2-D convolution, x N x C x H x W, w K x C x R x S, y N x K x P x Q (packed).
    Raises MMError."""
    lib = load()
    _check(lib.mm_conv2d_f32(N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, _addr(x), _addr(w),
                             _addr(y), _stream(stream)), "mm_conv2d_f32")


def mm_conv2d_f32_config(cfg, N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, x, w, y, stream=None):
    lib = load()
    _check(lib.mm_conv2d_f32_config(cfg, N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, _addr(x),
                                    _addr(w), _addr(y), _stream(stream)), "mm_conv2d_f32_config")


def mm_conv2d_out_dim(in_, filter_, stride, pad, dil):
    return load().mm_conv2d_out_dim(in_, filter_, stride, pad, dil)


def mm_conv2d_f32_num_configs():
    return load().mm_conv2d_f32_num_configs()


def mm_conv2d_f32_config_name(cfg):
    name = load().mm_conv2d_f32_config_name(cfg)
    return name.decode() if name is not None else None


def mm_conv2d_f32_select(N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw):
    return load().mm_conv2d_f32_select(N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw)


MM_TYPE_F32 = 0   # element types, as include/mm.h defines them
MM_TYPE_BF16 = 1
MM_TYPE_F16 = 2


def mm_gemm_bf16_grouped(groups, M, N, K, offsets, A, lda, B, ldb, stride_b, trans_b, C, c_type, ldc,
                         stream=None):
    """C rows of group g = A rows of group g x B_g (bf16 A and B). Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_bf16_grouped(groups, M, N, K, _addr(offsets), _addr(A), lda, _addr(B), ldb,
                                    stride_b, trans_b, _addr(C), c_type, ldc, _stream(stream)),
           "mm_gemm_bf16_grouped")


def mm_gemm_f16_grouped(groups, M, N, K, offsets, A, lda, B, ldb, stride_b, trans_b, C, c_type, ldc,
                        stream=None):
    """C rows of group g = A rows of group g x B_g (fp16 A and B). Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f16_grouped(groups, M, N, K, _addr(offsets), _addr(A), lda, _addr(B), ldb,
                                   stride_b, trans_b, _addr(C), c_type, ldc, _stream(stream)),
           "mm_gemm_f16_grouped")


def mm_gemm_bf16_grouped_grad_b(groups, M, N, K, offsets, A, lda, G, ldg, D, d_type, ldd, stride_d,
                                stream=None):
    """D_g = (A rows of group g)^T x (G rows of group g) (bf16 A and G). Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_bf16_grouped_grad_b(groups, M, N, K, _addr(offsets), _addr(A), lda, _addr(G),
                                           ldg, _addr(D), d_type, ldd, stride_d, _stream(stream)),
           "mm_gemm_bf16_grouped_grad_b")


def mm_gemm_f16_grouped_grad_b(groups, M, N, K, offsets, A, lda, G, ldg, D, d_type, ldd, stride_d,
                               stream=None):
    """D_g = (A rows of group g)^T x (G rows of group g) (fp16 A and G). Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_f16_grouped_grad_b(groups, M, N, K, _addr(offsets), _addr(A), lda, _addr(G),
                                          ldg, _addr(D), d_type, ldd, stride_d, _stream(stream)),
           "mm_gemm_f16_grouped_grad_b")


def mm_quantize_i8(rows, cols, X, x_type, ldx, Q, ldq, scale, stream=None):
    """Rows of X to 8-bit integers Q with a scale each. Raises MMError."""
    lib = load()
    _check(lib.mm_quantize_i8(rows, cols, _addr(X), x_type, ldx, _addr(Q), ldq, _addr(scale),
                              _stream(stream)), "mm_quantize_i8")


def mm_gemm_i8(M, N, K, A, lda, a_scale, B, ldb, b_scale, C, c_type, ldc, stream=None):
    """C = diag(a_scale) (A x B^T) diag(b_scale), 8-bit A (M x K) and B (N x K). Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_i8(M, N, K, _addr(A), lda, _addr(a_scale), _addr(B), ldb, _addr(b_scale),
                          _addr(C), c_type, ldc, _stream(stream)), "mm_gemm_i8")


def mm_gemm_i8_grouped(groups, M, N, K, offsets, A, lda, a_scale, B, ldb, stride_b, b_scale, C, c_type,
                       ldc, stream=None):
    """mm_gemm_i8 with rows of A in groups, a B_g and scales for each group. Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_i8_grouped(groups, M, N, K, _addr(offsets), _addr(A), lda, _addr(a_scale),
                                  _addr(B), ldb, stride_b, _addr(b_scale), _addr(C), c_type, ldc,
                                  _stream(stream)), "mm_gemm_i8_grouped")


def mm_quantize_mx4(rows, cols, X, x_type, ldx, Q, ldq, scale, ld_scale, stream=None):
    """Rows of X to 4-bit codes Q with a scale for each block of 32. Raises MMError."""
    lib = load()
    _check(lib.mm_quantize_mx4(rows, cols, _addr(X), x_type, ldx, _addr(Q), ldq, _addr(scale), ld_scale,
                               _stream(stream)), "mm_quantize_mx4")


def mm_dequantize_mx4(rows, cols, Q, ldq, scale, ld_scale, X, x_type, ldx, stream=None):
    """The values of 4-bit codes Q and their scales. Raises MMError."""
    lib = load()
    _check(lib.mm_dequantize_mx4(rows, cols, _addr(Q), ldq, _addr(scale), ld_scale, _addr(X), x_type, ldx,
                                 _stream(stream)), "mm_dequantize_mx4")


def mm_gemm_mx4(M, N, K, A, lda, a_scale, ld_as, B, ldb, b_scale, ld_bs, C, c_type, ldc, stream=None):
    """C = A x B^T of 4-bit A (M x K) and B (N x K) with a scale for each block of 32. Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_mx4(M, N, K, _addr(A), lda, _addr(a_scale), ld_as, _addr(B), ldb, _addr(b_scale), ld_bs,
                           _addr(C), c_type, ldc, _stream(stream)), "mm_gemm_mx4")


def mm_gemm_mx4_grouped(groups, M, N, K, offsets, A, lda, a_scale, ld_as, B, ldb, stride_b, b_scale, ld_bs,
                        stride_bs, C, c_type, ldc, stream=None):
    """mm_gemm_mx4 with rows of A in groups, a B_g and scales for each group. Raises MMError."""
    lib = load()
    _check(lib.mm_gemm_mx4_grouped(groups, M, N, K, _addr(offsets), _addr(A), lda, _addr(a_scale), ld_as, _addr(B),
                                   ldb, stride_b, _addr(b_scale), ld_bs, stride_bs, _addr(C), c_type, ldc,
                                   _stream(stream)), "mm_gemm_mx4_grouped")


MM_ROUTE_SOFTMAX = 0  # scorings, as include/mm.h defines them
MM_ROUTE_SIGMOID = 1


def mm_route_topk_workspace_bytes(T, E, k):
    """Bytes of workspace mm_route_topk needs for (T, E, k); -1 for invalid sizes."""
    return load().mm_route_topk_workspace_bytes(T, E, k)


def mm_route_topk(T, E, k, logits, type, ld, scoring, bias, groups, top_groups, group_top, renormalize, scale,
                  weights, experts, rows, offsets, workspace, workspace_bytes, stream=None):
    """The k best of E experts for each of T tokens, their weights and the rows' order. Raises MMError."""
    lib = load()
    _check(lib.mm_route_topk(T, E, k, _addr(logits), type, ld, scoring, _addr(bias), groups, top_groups, group_top,
                             renormalize, scale, _addr(weights), _addr(experts), _addr(rows), _addr(offsets),
                             _addr(workspace), workspace_bytes, _stream(stream)), "mm_route_topk")


def mm_route_topk_grad(T, E, k, logits, type, ld, scoring, renormalize, scale, experts, dweights, dlogits, ldd,
                       stream=None):
    """The logits' gradient from that of the weights. Raises MMError."""
    lib = load()
    _check(lib.mm_route_topk_grad(T, E, k, _addr(logits), type, ld, scoring, renormalize, scale, _addr(experts),
                                  _addr(dweights), _addr(dlogits), ldd, _stream(stream)), "mm_route_topk_grad")


def mm_spread_rows(T, k, row_bytes, X, ldx, rows, total, Y, ldy, stream=None):
    """Y[rows[t][j]] = X[t], rows of bytes. Raises MMError."""
    lib = load()
    _check(lib.mm_spread_rows(T, k, row_bytes, _addr(X), ldx, _addr(rows), total, _addr(Y), ldy, _stream(stream)),
           "mm_spread_rows")


def mm_combine_rows(T, k, D, Y, y_type, ldy, total, rows, weights, C, c_type, ldc, stream=None):
    """C[t] = sum over j of weights[t][j] Y[rows[t][j]]. Raises MMError."""
    lib = load()
    _check(lib.mm_combine_rows(T, k, D, _addr(Y), y_type, ldy, total, _addr(rows), _addr(weights), _addr(C), c_type,
                               ldc, _stream(stream)), "mm_combine_rows")


def mm_combine_rows_grad(T, k, D, G, g_type, ldg, Y, y_type, ldy, total, rows, weights, dY, lddy, dweights,
                         stream=None):
    """Gradients of mm_combine_rows with respect to Y and the weights. Raises MMError."""
    lib = load()
    _check(lib.mm_combine_rows_grad(T, k, D, _addr(G), g_type, ldg, _addr(Y), y_type, ldy, total, _addr(rows),
                                    _addr(weights), _addr(dY), lddy, _addr(dweights), _stream(stream)),
           "mm_combine_rows_grad")


def mm_gemm_grouped_num_configs():
    """Number of kernels of the grouped, the 8-bit and the 4-bit products."""
    return load().mm_gemm_grouped_num_configs()


def mm_gemm_grouped_config_name(cfg):
    """Name of kernel `cfg` of the grouped, the 8-bit and the 4-bit products, None outside the
    table."""
    name = load().mm_gemm_grouped_config_name(cfg)
    return name.decode() if name is not None else None


def mm_gemm_h16_grouped_select(groups, M, N, K, A, lda, B, ldb, stride_b, trans_b):
    """Kernel that mm_gemm_bf16_grouped and mm_gemm_f16_grouped run (-1: none)."""
    return load().mm_gemm_h16_grouped_select(groups, M, N, K, _addr(A), lda, _addr(B), ldb, stride_b, trans_b)


def mm_gemm_h16_grouped_grad_b_select(groups, M, N, K, A, lda, G, ldg):
    """Kernel that mm_gemm_bf16_grouped_grad_b and mm_gemm_f16_grouped_grad_b run (-1: none)."""
    return load().mm_gemm_h16_grouped_grad_b_select(groups, M, N, K, _addr(A), lda, _addr(G), ldg)


def mm_gemm_i8_select(M, N, K, A, lda, B, ldb):
    """Kernel that mm_gemm_i8 runs (-1: none)."""
    return load().mm_gemm_i8_select(M, N, K, _addr(A), lda, _addr(B), ldb)


def mm_gemm_i8_grouped_select(groups, M, N, K, A, lda, B, ldb, stride_b):
    """Kernel that mm_gemm_i8_grouped runs (-1: none)."""
    return load().mm_gemm_i8_grouped_select(groups, M, N, K, _addr(A), lda, _addr(B), ldb, stride_b)


def mm_gemm_mx4_select(M, N, K, A, lda, a_scale, ld_as, B, ldb, b_scale, ld_bs):
    """Kernel that mm_gemm_mx4 runs (-1: none)."""
    return load().mm_gemm_mx4_select(M, N, K, _addr(A), lda, _addr(a_scale), ld_as, _addr(B), ldb, _addr(b_scale), ld_bs)


def mm_gemm_mx4_grouped_select(groups, M, N, K, A, lda, a_scale, ld_as, B, ldb, stride_b, b_scale, ld_bs, stride_bs):
    """Kernel that mm_gemm_mx4_grouped runs (-1: none)."""
    return load().mm_gemm_mx4_grouped_select(groups, M, N, K, _addr(A), lda, _addr(a_scale), ld_as, _addr(B), ldb,
                                             stride_b, _addr(b_scale), ld_bs, stride_bs)


def mm_status_string(status):
    return load().mm_status_string(status).decode()


def mm_last_error():
    return load().mm_last_error().decode()


# ----------------------------------------------------- torch-tensor front ends

def _on_device(device, **tensors):
    """Raise ValueError unless every given tensor is on `device` (a host tensor's address
    handed to a kernel would fault the GPU)."""
    for name, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _workspace_bytes(ws, device):
    """Size in bytes of a workspace tensor, which must be contiguous and on `device`."""
    if not hasattr(ws, "data_ptr"):
        raise TypeError(f"workspace must be a torch.Tensor, got {type(ws).__name__}")
    if ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, the operands on {device}")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws.numel() * ws.element_size()


def _matrix(t, name, dtypes=None):
    torch = _torch or _import_torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtypes = dtypes or (torch.float32,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    if rows == 0 or cols == 0:  # the strides of an empty tensor are arbitrary, and nothing uses them
        return max(cols, 1)
    ld, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows == 1:
        return cols
    if ld < cols:
        raise ValueError(f"{name} row stride {ld} is below its width {cols}")
    return ld


def gemm_workspace(M, N, K, device):
    """A device buffer of the size mm_gemm_f32_ws needs for (M, N, K) (None if none)."""
    import torch
    n = mm_gemm_f32_workspace_bytes(M, N, K)
    if n < 0:
        raise ValueError(f"invalid sizes {M} x {N} x {K}")
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def gemm(A, B, out=None, config=None, stream=None, workspace=None):
    """out = A @ B for fp32 GPU tensors (any row strides, unit column stride). With
    `workspace` (a device tensor of at least mm_gemm_f32_workspace_bytes bytes, e.g. from
    gemm_workspace) it runs mm_gemm_f32_ws; with workspace="static", mm_gemm_f32_ws_static
    (the library's own device scratch; calls that overlap on one GPU race)."""
    import torch
    lda = _matrix(A, "A")
    ldb = _matrix(B, "B")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)}")
    if B.device != A.device:
        raise ValueError("A and B are on different devices")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, N)}")
    ldc = _matrix(out, "out")
    _on_device(A.device, out=out)
    if workspace is not None and config is not None:
        raise ValueError("a workspace and a forced config do not go together")
    with torch.cuda.device(A.device):
        if isinstance(workspace, str):
            if workspace != "static":
                raise ValueError(f"workspace must be a tensor or 'static', got {workspace!r}")
            mm_gemm_f32_ws_static(M, N, K, A, lda, B, ldb, out, ldc, stream)
        elif workspace is not None:
            mm_gemm_f32_ws(M, N, K, A, lda, B, ldb, out, ldc, workspace,
                           _workspace_bytes(workspace, A.device), stream)
        elif config is None:
            mm_gemm_f32(M, N, K, A, lda, B, ldb, out, ldc, stream)
        else:
            mm_gemm_f32_config(config, M, N, K, A, lda, B, ldb, out, ldc, stream)
    return out


def gemm_batched(A, B, out=None, stream=None):
    """out[b] = A[b] @ B[b] for 3-D fp32 GPU tensors (batch, rows, cols) whose last
    dimension has unit stride; a batch stride of 0 (e.g. from expand) shares an operand."""
    import torch
    for t, name in ((A, "A"), (B, "B")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.dim() != 3:
            raise TypeError(f"{name} must be a 3-D float32 tensor")
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on the GPU")
    batch, M, K = A.shape
    batch2, K2, N = B.shape
    if batch2 != batch or K2 != K:
        raise ValueError(f"shapes differ: {tuple(A.shape)} x {tuple(B.shape)}")
    if out is None:
        out = torch.empty((batch, M, N), dtype=torch.float32, device=A.device)
    lda = _matrix(A[0] if batch else A.new_empty((M, K)), "A")
    ldb = _matrix(B[0] if batch else B.new_empty((K, N)), "B")
    ldc = _matrix(out[0] if batch else out.new_empty((M, N)), "out")
    _on_device(A.device, B=B, out=out)
    with torch.cuda.device(A.device):
        mm_gemm_f32_batched(batch, M, N, K, A, lda, A.stride(0), B, ldb, B.stride(0), out, ldc,
                            out.stride(0), stream)
    return out


def gemm16(A, B, out=None, config=None, stream=None):
    """out (fp32) = A @ B for bf16 or fp16 GPU tensors A and B of the same dtype."""
    import torch
    lda = _matrix(A, "A", (torch.bfloat16, torch.float16))
    ldb = _matrix(B, "B", (A.dtype,))
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)}")
    if B.device != A.device:
        raise ValueError("A and B are on different devices")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, N)}")
    ldc = _matrix(out, "out")
    _on_device(A.device, out=out)
    bf = A.dtype == torch.bfloat16
    with torch.cuda.device(A.device):
        if config is None:
            (mm_gemm_bf16 if bf else mm_gemm_f16)(M, N, K, A, lda, B, ldb, out, ldc, stream)
        else:
            (mm_gemm_bf16_config if bf else mm_gemm_f16_config)(config, M, N, K, A, lda, B, ldb,
                                                                 out, ldc, stream)
    return out


def gemv(A, x, out=None, stream=None):
    """out = A @ x for an fp32 GPU matrix with packed rows and a contiguous vector."""
    import torch
    _matrix(A, "A")
    M, N = A.shape
    if not A.is_contiguous():
        raise ValueError("A must have packed rows (contiguous)")
    if x.dtype != torch.float32 or x.dim() != 1 or x.shape[0] != N or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous float32 vector of {N} entries")
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=A.device)
    if out.dtype != torch.float32 or tuple(out.shape) != (M,) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous float32 vector of {M} entries")
    _on_device(A.device, x=x, out=out)
    with torch.cuda.device(A.device):
        mm_gemv_f32(M, N, A, x, out, stream)
    return out


def gemv_t_workspace(M, N, device):
    """A device buffer of the size mm_gemv_t_f32_ws needs for (M, N) (None if none)."""
    import torch
    n = mm_gemv_t_f32_workspace_bytes(M, N)
    if n < 0:
        raise ValueError(f"invalid sizes {M} x {N}")
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def gemv_t(A, x, out=None, workspace=None, stream=None):
    """out = A.T @ x for an fp32 GPU matrix with packed rows and a contiguous vector.
    With `workspace` (a device tensor of at least mm_gemv_t_f32_workspace_bytes bytes,
    e.g. from gemv_t_workspace) it runs mm_gemv_t_f32_ws."""
    import torch
    _matrix(A, "A")
    M, N = A.shape
    if not A.is_contiguous():
        raise ValueError("A must have packed rows (contiguous)")
    if x.dtype != torch.float32 or x.dim() != 1 or x.shape[0] != M or not x.is_contiguous():
        raise ValueError(f"x must be a contiguous float32 vector of {M} entries")
    if out is None:
        out = torch.empty(N, dtype=torch.float32, device=A.device)
    if out.dtype != torch.float32 or tuple(out.shape) != (N,) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous float32 vector of {N} entries")
    _on_device(A.device, x=x, out=out)
    with torch.cuda.device(A.device):
        if workspace is None:
            mm_gemv_t_f32(M, N, A, x, out, stream)
        else:
            mm_gemv_t_f32_ws(M, N, A, x, out, workspace, _workspace_bytes(workspace, A.device), stream)
    return out


def conv2d(x, w, stride=(1, 1), pad=(0, 0), dilation=(1, 1), out=None, config=None, stream=None):
    """out = the 2-D convolution of x (N x C x H x W) with w (K x C x R x S), both
    contiguous fp32 GPU tensors; out is N x K x P x Q (allocated if not given)."""
    import torch
    for t, name in ((x, "x"), (w, "w")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.dim() != 4:
            raise TypeError(f"{name} must be a 4-D float32 tensor")
        if t.device.type != "cuda" or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous GPU tensor")
    if w.device != x.device:
        raise ValueError("x and w are on different devices")
    N, C, H, W = x.shape
    K, C2, R, S = w.shape
    if C2 != C:
        raise ValueError(f"channel counts differ: x has {C}, w has {C2}")
    (sh, sw), (ph, pw), (dh, dw) = stride, pad, dilation
    P = mm_conv2d_out_dim(H, R, sh, ph, dh)
    Q = mm_conv2d_out_dim(W, S, sw, pw, dw)
    if P < 1 or Q < 1:
        raise ValueError("invalid convolution geometry (the filter must fit the padded input)")
    if out is None:
        out = torch.empty((N, K, P, Q), dtype=torch.float32, device=x.device)
    if (out.dtype != torch.float32 or tuple(out.shape) != (N, K, P, Q) or not out.is_contiguous()
            or out.device != x.device):
        raise ValueError(f"out must be a contiguous float32 tensor of shape {(N, K, P, Q)}")
    with torch.cuda.device(x.device):
        if config is None:
            mm_conv2d_f32(N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, x, w, out, stream)
        else:
            mm_conv2d_f32_config(config, N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, x, w, out,
                                 stream)
    return out


def _run(name, device, stream, *args):
    """Call the C entry point `name` with `args` and the stream, `device` (an index) current."""
    torch = _torch or _import_torch()
    fn = getattr(_lib or load(), name)
    # the current stream's address without a Stream object around it (2.9 us of a 12 us call)
    s = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == device:  # as torch.cuda.current_device(), initialised with the tensors
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            status = fn(*args, s)
    if status != MM_OK:
        _check(status, name)


def _mm_type(dtype, name):
    """MM_TYPE_* of a torch dtype."""
    torch = _torch or _import_torch()
    if dtype is torch.float32:
        return MM_TYPE_F32
    if dtype is torch.bfloat16:
        return MM_TYPE_BF16
    if dtype is torch.float16:
        return MM_TYPE_F16
    raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")


def _same_device(t, name, device):
    """Raise ValueError unless the tensor is on the GPU with index `device`."""
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


def _stack(t, name, dtypes):
    """Leading dimension and group stride of a 3-D tensor of matrices."""
    torch = _torch or _import_torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D (groups, rows, columns)")
    _, rows, cols = t.shape
    stride_g, ld, unit = t.stride()
    if t.numel() == 0:  # the strides of an empty tensor are arbitrary, and nothing uses them
        return max(cols, 1), 0
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows == 1:
        ld = cols
    if ld < cols:
        raise ValueError(f"{name} row stride {ld} is below its width {cols}")
    return ld, stride_g


def _apart(count, stride, rows, ld, cols):
    """Whether `count` rows x cols matrices, `stride` elements apart, share no element: each ends before
    the next begins, or all their rows i lie between one matrix' row i and its row i + 1."""
    return stride >= (rows - 1) * ld + cols or (stride >= cols and ld >= (count - 1) * stride + cols)


def _offsets(t, groups, device):
    torch = _torch or _import_torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int64:
        raise TypeError("offsets must be an int64 tensor")
    if t.dim() != 1 or t.shape[0] != groups + 1 or not t.is_contiguous():
        raise ValueError(f"offsets must be contiguous, with groups + 1 = {groups + 1} entries")
    _same_device(t, "offsets", device)


def _scale(t, shape, name, device):
    torch = _torch or _import_torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32:
        raise TypeError(f"{name} must be a float32 tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {shape}")
    _same_device(t, name, device)


def _output(out, out_dtype, shape, like):
    """(the output tensor, its MM_TYPE_*, leading dimension, group stride): `out` if given (its dtype
    must be out_dtype where that is given too), else a new one of out_dtype (float32 by default)."""
    torch = _torch or _import_torch()
    if out is None:
        dtype = torch.float32 if out_dtype is None else out_dtype
        c_type = _mm_type(dtype, "out_dtype")
        cols = max(shape[-1], 1)
        new = like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
        return new, c_type, cols, shape[-2] * cols
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch.Tensor")
    c_type = _mm_type(out.dtype, "out")
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    if out.shape != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {shape}")
    _same_device(out, "out", like.get_device())
    if len(shape) == 2:
        return out, c_type, _matrix(out, "out", (out.dtype,)), 0
    return (out, c_type) + _stack(out, "out", (out.dtype,))


def gemm16_grouped(A, B, offsets, trans_b=False, out=None, out_dtype=None, stream=None):
    """Products of rows grouped by expert: rows offsets[g] <= i < offsets[g + 1] of out are those
    rows of A (M x K) times B[g], for bf16 or fp16 GPU tensors of the same dtype. B is
    groups x K x N, or groups x N x K with trans_b (B[g] is then transposed); any row and group
    strides, unit column stride. offsets is an int64 GPU tensor of groups + 1 entries that do
    not decrease; the host never reads it. out is float32, bfloat16 or float16 (out_dtype,
    float32 by default); its rows of no group are left as they are (uninitialised if out was
    not given). The gradient with respect to A is gemm16_grouped(dout, B, offsets, not trans_b)."""
    torch = _torch or _import_torch()
    lda = _matrix(A, "A", (torch.bfloat16, torch.float16))
    ldb, stride_b = _stack(B, "B", (A.dtype,))
    device = A.get_device()
    M, K = A.shape
    groups, K2, N = B.shape
    if trans_b:
        K2, N = N, K2
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)}")
    _same_device(B, "B", device)
    _offsets(offsets, groups, device)
    out, c_type, ldc, _ = _output(out, out_dtype, (M, N), A)
    name = "mm_gemm_bf16_grouped" if A.dtype is torch.bfloat16 else "mm_gemm_f16_grouped"
    _run(name, device, stream, groups, M, N, K, offsets.data_ptr(), A.data_ptr(), lda, B.data_ptr(), ldb,
         stride_b, 1 if trans_b else 0, out.data_ptr(), c_type, ldc)
    return out


def gemm16_grouped_grad_b(A, G, offsets, out=None, out_dtype=None, stream=None):
    """The gradient of gemm16_grouped(A, B, offsets) with respect to B from the gradient G of its
    output: out[g] = A[lo:hi].T @ G[lo:hi] over the rows lo = offsets[g] .. hi = offsets[g + 1]
    (zeros for an empty group), groups x K x N. For B stored groups x N x K (trans_b) exchange A
    and G. A, G: bf16 or fp16 of the same dtype; out float32 (default), bfloat16 or float16, its
    matrices one after the other or row by row in turn (a transposed K x groups x N)."""
    import torch
    lda = _matrix(A, "A", (torch.bfloat16, torch.float16))
    ldg = _matrix(G, "G", (A.dtype,))
    device = A.get_device()
    M, K = A.shape
    M2, N = G.shape
    if M2 != M:
        raise ValueError(f"row counts differ: {tuple(A.shape)}, {tuple(G.shape)}")
    _same_device(G, "G", device)
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be a 1-D tensor of groups + 1 entries")
    groups = offsets.shape[0] - 1
    _offsets(offsets, groups, device)
    out, d_type, ldd, stride_d = _output(out, out_dtype, (groups, K, N), A)
    if groups > 1 and K > 0 and N > 0 and not _apart(groups, stride_d, K, ldd, N):
        raise ValueError("the matrices of out overlap (neither one after the other nor row by row in turn)")
    name = "mm_gemm_bf16_grouped_grad_b" if A.dtype is torch.bfloat16 else "mm_gemm_f16_grouped_grad_b"
    _run(name, device, stream, groups, M, N, K, offsets.data_ptr(), A.data_ptr(), lda, G.data_ptr(), ldg,
         out.data_ptr(), d_type, ldd, stride_d)
    return out


def quantize_i8(x, out=None, scale=None, stream=None):
    """(q, scale): the rows of x (float32, bfloat16 or float16) as int8 with q[i] * scale[i] ~ x[i],
    scale[i] = max |x[i]| / 127; values are rounded to the nearest integer, halves to even."""
    torch = _torch or _import_torch()
    ldx = _matrix(x, "x", (torch.float32, torch.bfloat16, torch.float16))
    device = x.get_device()
    rows, cols = x.shape
    if out is None:
        out, ldq = x.new_empty((rows, cols), dtype=torch.int8), max(cols, 1)
    else:
        ldq = _matrix(out, "out", (torch.int8,))
        if out.shape != x.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(rows, cols)}")
        _same_device(out, "out", device)
    if scale is None:
        scale = x.new_empty(rows, dtype=torch.float32)
    else:
        _scale(scale, (rows,), "scale", device)
    _run("mm_quantize_i8", device, stream, rows, cols, x.data_ptr(), _mm_type(x.dtype, "x"), ldx, out.data_ptr(),
         ldq, scale.data_ptr())
    return out, scale


def gemm_i8(A, B, a_scale, b_scale, out=None, out_dtype=None, stream=None):
    """out[i][j] = a_scale[i] b_scale[j] sum_k A[i][k] B[j][k] for int8 GPU tensors A (M x K) and
    B (N x K), any row strides; out float32 (default), bfloat16 or float16."""
    torch = _torch or _import_torch()
    lda = _matrix(A, "A", (torch.int8,))
    ldb = _matrix(B, "B", (torch.int8,))
    device = A.get_device()
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)} transposed")
    _same_device(B, "B", device)
    _scale(a_scale, (M,), "a_scale", device)
    _scale(b_scale, (N,), "b_scale", device)
    out, c_type, ldc, _ = _output(out, out_dtype, (M, N), A)
    _run("mm_gemm_i8", device, stream, M, N, K, A.data_ptr(), lda, a_scale.data_ptr(), B.data_ptr(), ldb,
         b_scale.data_ptr(), out.data_ptr(), c_type, ldc)
    return out


def gemm_i8_grouped(A, B, offsets, a_scale, b_scale, out=None, out_dtype=None, stream=None):
    """gemm_i8 with rows grouped by expert: B groups x N x K, b_scale groups x N, offsets as for
    gemm16_grouped; rows of no group are left as they are."""
    torch = _torch or _import_torch()
    lda = _matrix(A, "A", (torch.int8,))
    ldb, stride_b = _stack(B, "B", (torch.int8,))
    device = A.get_device()
    M, K = A.shape
    groups, N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)} transposed")
    _same_device(B, "B", device)
    _offsets(offsets, groups, device)
    _scale(a_scale, (M,), "a_scale", device)
    _scale(b_scale, (groups, N), "b_scale", device)
    out, c_type, ldc, _ = _output(out, out_dtype, (M, N), A)
    _run("mm_gemm_i8_grouped", device, stream, groups, M, N, K, offsets.data_ptr(), A.data_ptr(), lda,
         a_scale.data_ptr(), B.data_ptr(), ldb, stride_b, b_scale.data_ptr(), out.data_ptr(), c_type, ldc)
    return out


def _bytes_matrix(t, shape, name, device):
    """Leading dimension of a uint8 matrix of the given shape."""
    torch = _torch or _import_torch()
    if isinstance(t, torch.Tensor) and t.dtype is torch.uint8 and t.shape == shape and t.get_device() == device:
        rows, cols = shape
        if rows > 1 and cols > 1:  # the common case, with few questions
            ld, unit = t.stride()
            if unit == 1 and ld >= cols:
                return ld
    ld = _matrix(t, name, (torch.uint8,))
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    _same_device(t, name, device)
    return ld


def quantize_mx4(x, out=None, scale=None, stream=None):
    """(q, scale): the rows of x (float32, bfloat16 or float16) in 4-bit floating point (values 0, 0.5,
    1, 1.5, 2, 3, 4 and 6 with a sign) and blocks of 32 along the row with a power of two each. q is
    uint8, rows x 16 ceil(cols / 32), two elements to a byte, the even one low (the last block filled
    up with zeros); scale is uint8, rows x ceil(cols / 32), the exponent + 127. An element is x / 2^e
    rounded to the nearest value, halves to the even code, e = floor(log2 max |x|) - 2 in its block."""
    torch = _torch or _import_torch()
    ldx = _matrix(x, "x", (torch.float32, torch.bfloat16, torch.float16))
    device = x.get_device()
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    if out is None:
        out, ldq = x.new_empty((rows, 16 * blocks), dtype=torch.uint8), max(16 * blocks, 1)
    else:
        ldq = _bytes_matrix(out, (rows, 16 * blocks), "out", device)
    if scale is None:
        scale, lds = out.new_empty((rows, blocks)), max(blocks, 1)
    else:
        lds = _bytes_matrix(scale, (rows, blocks), "scale", device)
    _run("mm_quantize_mx4", device, stream, rows, cols, x.data_ptr(), _mm_type(x.dtype, "x"), ldx, out.data_ptr(), ldq,
         scale.data_ptr(), lds)
    return out, scale


def dequantize_mx4(q, scale, cols=None, out=None, out_dtype=None, stream=None):
    """The values that quantize_mx4's codes and scales stand for: rows x cols (all elements of the
    blocks by default) of out_dtype, float32 (default), bfloat16 (both exact) or float16."""
    torch = _torch or _import_torch()
    ldq = _matrix(q, "q", (torch.uint8,))
    device = q.get_device()
    rows, width = q.shape
    if width % 16:
        raise ValueError(f"q has rows of {width} bytes, no multiple of 16")
    if cols is None:
        cols = 2 * width
    if (cols + 31) // 32 * 16 != width:
        raise ValueError(f"{cols} columns do not fit rows of {width // 16} blocks")
    lds = _bytes_matrix(scale, (rows, width // 16), "scale", device)
    out, x_type, ldx, _ = _output(out, out_dtype, (rows, cols), q)
    _run("mm_dequantize_mx4", device, stream, rows, cols, q.data_ptr(), ldq, scale.data_ptr(), lds, out.data_ptr(),
         x_type, ldx)
    return out


def gemm_mx4(A, B, a_scale, b_scale, out=None, out_dtype=None, stream=None):
    """out[i][j] = sum_k a[i][k] b[j][k] of the values of quantize_mx4's codes A (M x K / 2 bytes) and B
    (N x K / 2) with scales M x K / 32 and N x K / 32, all uint8, any row strides; out float32
    (default), bfloat16 or float16."""
    torch = _torch or _import_torch()
    lda = _matrix(A, "A", (torch.uint8,))
    ldb = _matrix(B, "B", (torch.uint8,))
    device = A.get_device()
    M, K = A.shape
    N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)} transposed")
    if K % 16:
        raise ValueError(f"rows of {K} bytes, no multiple of 16")
    _same_device(B, "B", device)
    ld_as = _bytes_matrix(a_scale, (M, K // 16), "a_scale", device)
    ld_bs = _bytes_matrix(b_scale, (N, K // 16), "b_scale", device)
    out, c_type, ldc, _ = _output(out, out_dtype, (M, N), A)
    _run("mm_gemm_mx4", device, stream, M, N, 2 * K, A.data_ptr(), lda, a_scale.data_ptr(), ld_as, B.data_ptr(), ldb,
         b_scale.data_ptr(), ld_bs, out.data_ptr(), c_type, ldc)
    return out


def gemm_mx4_grouped(A, B, offsets, a_scale, b_scale, out=None, out_dtype=None, stream=None):
    """gemm_mx4 with rows grouped by expert: B groups x N x K / 2, b_scale groups x N x K / 32, offsets as
    for gemm16_grouped (and as route_topk returns them); rows of no group are left as they are."""
    torch = _torch or _import_torch()
    lda = _matrix(A, "A", (torch.uint8,))
    ldb, stride_b = _stack(B, "B", (torch.uint8,))
    device = A.get_device()
    M, K = A.shape
    groups, N, K2 = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: {tuple(A.shape)} x {tuple(B.shape)} transposed")
    if K % 16:
        raise ValueError(f"rows of {K} bytes, no multiple of 16")
    _same_device(B, "B", device)
    _offsets(offsets, groups, device)
    ld_as = _bytes_matrix(a_scale, (M, K // 16), "a_scale", device)
    ld_bs, stride_bs = _stack(b_scale, "b_scale", (torch.uint8,))
    if b_scale.shape != (groups, N, K // 16):
        raise ValueError(f"b_scale has shape {tuple(b_scale.shape)}, expected {(groups, N, K // 16)}")
    _same_device(b_scale, "b_scale", device)
    out, c_type, ldc, _ = _output(out, out_dtype, (M, N), A)
    _run("mm_gemm_mx4_grouped", device, stream, groups, M, N, 2 * K, offsets.data_ptr(), A.data_ptr(), lda,
         a_scale.data_ptr(), ld_as, B.data_ptr(), ldb, stride_b, b_scale.data_ptr(), ld_bs, stride_bs, out.data_ptr(),
         c_type, ldc)
    return out


def _scoring(name):
    if name == "softmax":
        return MM_ROUTE_SOFTMAX
    if name == "sigmoid":
        return MM_ROUTE_SIGMOID
    raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {name!r}")


def _slots(t, shape, dtype, name, device):
    """Check a packed tensor with an entry for each slot of each token."""
    torch = _torch or _import_torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {tuple(shape)}")
    _same_device(t, name, device)


def _allocating_for(stream, device):
    """A context whose allocations belong to `stream`, so that what is freed while work on that stream
    still uses it is handed out again on that stream only."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        address = _stream(stream)
        stream = torch.cuda.ExternalStream(address, device=device) if address else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def route_topk_workspace(T, E, k, device):
    """A device buffer of the size mm_route_topk needs for (T, E, k) (None if none)."""
    import torch
    n = mm_route_topk_workspace_bytes(T, E, k)
    if n < 0:
        raise ValueError(f"invalid sizes: {T} tokens, {k} of {E} experts")
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def route_topk(logits, k, scoring="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=False,
               scale=1.0, workspace=None, stream=None):
    """(weights, experts, rows, offsets): the k best of E experts for each row of logits (T x E; float32,
    bfloat16 or float16), and the order of their rows. Scores are the softmax or the sigmoid of the
    logits; experts are chosen by score + bias (float32, E entries), with groups > 1 among the
    top_groups groups of E / groups neighbours whose group_top (1 or 2) best add up highest (a single
    expert's own value, where a group has no more); equal ones by the lower index. weights (T x k,
    float32) are the chosen scores times scale, with renormalize divided by their sum. experts (T x k,
    int32) holds -1 where none is left (logits of -inf are never chosen: give padded tokens only
    those). rows (T x k, int32) numbers the slots by expert, token and slot, -1 without an expert, and
    offsets (E + 1, int64) says where each expert's rows begin, as the grouped products take it.
    workspace: a device tensor of mm_route_topk_workspace_bytes bytes (e.g. from
    route_topk_workspace); allocated for the call if not given."""
    torch = _torch or _import_torch()
    ld = _matrix(logits, "logits", (torch.float32, torch.bfloat16, torch.float16))
    device = logits.get_device()
    T, E = logits.shape
    how = _scoring(scoring)
    if bias is not None:
        _scale(bias, (E,), "bias", device)
    need = (_lib or load()).mm_route_topk_workspace_bytes(T, E, k)
    if need < 0:
        raise ValueError(f"invalid sizes: {T} tokens, {k} of {E} experts")
    if workspace is not None:
        size = _workspace_bytes(workspace, logits.device)
    elif need > 0:
        with _allocating_for(stream, logits.device):
            workspace, size = logits.new_empty(need, dtype=torch.uint8), need
    else:
        size = 0
    weights = logits.new_empty((T, k), dtype=torch.float32)
    experts = logits.new_empty((T, k), dtype=torch.int32)
    rows = torch.empty_like(experts)
    offsets = logits.new_empty(E + 1, dtype=torch.int64)
    _run("mm_route_topk", device, stream, T, E, k, logits.data_ptr(), _mm_type(logits.dtype, "logits"), ld, how,
         None if bias is None else bias.data_ptr(), groups, top_groups, group_top, 1 if renormalize else 0, scale,
         weights.data_ptr(), experts.data_ptr(), rows.data_ptr(), offsets.data_ptr(),
         None if workspace is None else workspace.data_ptr(), size)
    return weights, experts, rows, offsets


def route_topk_grad(logits, experts, dweights, scoring="softmax", renormalize=False, scale=1.0, out=None, stream=None):
    """The gradient of route_topk's weights with respect to the logits, T x E of the logits' dtype, from
    dweights (T x k, float32) and the experts that route_topk returned."""
    torch = _torch or _import_torch()
    ld = _matrix(logits, "logits", (torch.float32, torch.bfloat16, torch.float16))
    device = logits.get_device()
    T, E = logits.shape
    how = _scoring(scoring)
    if not isinstance(experts, torch.Tensor) or experts.dim() != 2:
        raise TypeError("experts must be a 2-D tensor")
    k = experts.shape[1]
    _slots(experts, (T, k), torch.int32, "experts", device)
    _slots(dweights, (T, k), torch.float32, "dweights", device)
    out, _, ldd, _ = _output(out, logits.dtype, (T, E), logits)
    _run("mm_route_topk_grad", device, stream, T, E, k, logits.data_ptr(), _mm_type(logits.dtype, "logits"), ld, how,
         1 if renormalize else 0, scale, experts.data_ptr(), dweights.data_ptr(), out.data_ptr(), ldd)
    return out


def _token_slots(rows):
    """(T, k) of a router's rows."""
    torch = _torch or _import_torch()
    if not isinstance(rows, torch.Tensor) or rows.dim() != 2:
        raise TypeError("rows must be a 2-D tensor")
    return rows.shape


def spread_rows(x, rows, out=None, stream=None):
    """out[rows[t][j]] = x[t]: the tokens' rows in the experts' order. x is T x D of any of float32,
    bfloat16, float16, int8 and uint8, rows T x k int32 as route_topk returns it (k at most 1024); entries
    outside out's rows are none. out has T k rows if it is not given; those that nothing names are left as they are
    (uninitialised if out was not given). The gradient is combine_rows without weights."""
    torch = _torch or _import_torch()
    dtypes = (torch.float32, torch.bfloat16, torch.float16, torch.int8, torch.uint8)
    ldx = _matrix(x, "x", dtypes)
    device = x.get_device()
    T, k = _token_slots(rows)
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, rows {T}")
    _slots(rows, (T, k), torch.int32, "rows", device)
    D, size = x.shape[1], x.element_size()
    if out is None:
        out, ldo = x.new_empty((T * k, D)), max(D, 1)
    else:
        ldo = _matrix(out, "out", (x.dtype,))
        if out.shape[1] != D:
            raise ValueError(f"out has {out.shape[1]} columns, x {D}")
        _same_device(out, "out", device)
    _run("mm_spread_rows", device, stream, T, k, D * size, x.data_ptr(), ldx * size, rows.data_ptr(), out.shape[0],
         out.data_ptr(), ldo * size)
    return out


def combine_rows(y, rows, weights=None, out=None, out_dtype=None, stream=None):
    """out[t] = sum_j weights[t][j] y[rows[t][j]]: the experts' outputs y (float32, bfloat16 or float16)
    back to the tokens. rows T x k int32 as route_topk returns it (k at most 1024; entries outside y's
    rows add nothing), weights T x k float32 or None for the plain sum; out T x D, float32 (default), bfloat16 or
    float16."""
    torch = _torch or _import_torch()
    ldy = _matrix(y, "y", (torch.float32, torch.bfloat16, torch.float16))
    device = y.get_device()
    T, k = _token_slots(rows)
    _slots(rows, (T, k), torch.int32, "rows", device)
    if weights is not None:
        _slots(weights, (T, k), torch.float32, "weights", device)
    total, D = y.shape
    out, c_type, ldc, _ = _output(out, out_dtype, (T, D), y)
    _run("mm_combine_rows", device, stream, T, k, D, y.data_ptr(), _mm_type(y.dtype, "y"), ldy, total, rows.data_ptr(),
         None if weights is None else weights.data_ptr(), out.data_ptr(), c_type, ldc)
    return out


def combine_rows_grad(dout, y, rows, weights, out=None, stream=None):
    """(dy, dweights): the gradients of combine_rows(y, rows, weights) from that of its output (T x D,
    float32, bfloat16 or float16): dy[rows[t][j]] = weights[t][j] dout[t], of y's shape and dtype (out
    if given), rows that nothing names left as they are (uninitialised if out was not given);
    dweights[t][j] = <y[rows[t][j]], dout[t]>, float32."""
    torch = _torch or _import_torch()
    types = (torch.float32, torch.bfloat16, torch.float16)
    ldg = _matrix(dout, "dout", types)
    ldy = _matrix(y, "y", types)
    device = y.get_device()
    _same_device(dout, "dout", device)
    T, k = _token_slots(rows)
    total, D = y.shape
    if dout.shape != (T, D):
        raise ValueError(f"dout has shape {tuple(dout.shape)}, expected {(T, D)}")
    _slots(rows, (T, k), torch.int32, "rows", device)
    _slots(weights, (T, k), torch.float32, "weights", device)
    y_type = _mm_type(y.dtype, "y")
    out, _, lddy, _ = _output(out, y.dtype, (total, D), y)
    dweights = y.new_empty((T, k), dtype=torch.float32)
    _run("mm_combine_rows_grad", device, stream, T, k, D, dout.data_ptr(), _mm_type(dout.dtype, "dout"), ldg,
         y.data_ptr(), y_type, ldy, total, rows.data_ptr(), weights.data_ptr(), out.data_ptr(), lddy,
         dweights.data_ptr())
    return out, dweights
