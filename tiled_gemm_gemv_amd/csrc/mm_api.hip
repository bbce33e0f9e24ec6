// mm_api.hip -- the C ABI of libmm (declared in include/mm.h): host-side argument
// checks, shape -> kernel configuration, launch, and status codes.
#include <stdint.h>
#include <stdio.h>

#include "mm.h"
#include "mm_internal.h"

namespace {

thread_local char g_last_error[256] = "";

void set_error(const char *what, hipError_t e)
{
    snprintf(g_last_error, sizeof g_last_error, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
}

void set_error_text(const char *what)
{
    snprintf(g_last_error, sizeof g_last_error, "%s", what);
}

int from_hip(const char *what, hipError_t e)
{
    if (e == hipSuccess) return MM_OK;
    set_error(what, e);
    if (e == hipErrorNoDevice || e == hipErrorInsufficientDriver) return MM_ERR_NO_DEVICE;
    return MM_ERR_LAUNCH;
}

int invalid(const char *why)
{
    set_error_text(why);
    return MM_ERR_INVALID_ARG;
}

constexpr int64_t kMaxDim = 0x7fffffff;

// Byte extent of a rows x cols matrix with row stride ld is
// 4 * ((rows - 1) * ld + cols); true if that fits in int64 (rows, cols >= 1).
bool extent_fits(int64_t rows, int64_t cols, int64_t ld)
{
    const int64_t limit = INT64_MAX / 4;
    if (ld > 0 && rows - 1 > (limit - cols) / ld) return false;
    return true;
}

int check_gemm_dims(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc)
{
    if (M < 0 || N < 0 || K < 0) return invalid("negative size");
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return invalid("size above 2^31 - 1");
    if (lda < (K > 1 ? K : 1)) return invalid("lda < max(1, K)");
    if (ldb < (N > 1 ? N : 1)) return invalid("ldb < max(1, N)");
    if (ldc < (N > 1 ? N : 1)) return invalid("ldc < max(1, N)");
    return MM_OK;
}

// elem: bytes per element of A and B (4 for fp32, 2 for the 16-bit formats).
int check_gemm(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *B,
               int64_t ldb, const float *C, int64_t ldc, int elem = 4)
{
    const int d = check_gemm_dims(M, N, K, lda, ldb, ldc);
    if (d != MM_OK) return d;
    if (M > 0 && K > 0 && !A) return invalid("A is NULL");
    if (K > 0 && N > 0 && !B) return invalid("B is NULL");
    if (M > 0 && N > 0 && !C) return invalid("C is NULL");
    if ((uintptr_t)A % elem || (uintptr_t)B % elem || (uintptr_t)C % 4)
        return invalid("pointer not aligned to its element size");
    if (M > 0 && K > 0 && !extent_fits(M, K, lda)) return invalid("A extent overflows");
    if (K > 0 && N > 0 && !extent_fits(K, N, ldb)) return invalid("B extent overflows");
    if (M > 0 && N > 0 && !extent_fits(M, N, ldc)) return invalid("C extent overflows");
    return MM_OK;
}

int run_gemm(int cfg, int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
             int64_t ldb, float *C, int64_t ldc, void *stream)
{
    const int st = check_gemm(M, N, K, A, lda, B, ldb, C, ldc);
    if (st != MM_OK) return st;
    if (M == 0 || N == 0) return MM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) return from_hip("zero fill launch", mm::zero_fill_launch(C, M, N, ldc, s));
    mm::GemmArgs a;
    a.A = A;
    a.B = B;
    a.C = C;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    if (cfg < 0 && mm::gemm_split2_ok(M, N, K)) return from_hip("gemm launch", mm::gemm_split2_launch(a, s));
    if (cfg < 0) cfg = mm::gemm_select_config(M, N, K);
    return from_hip("gemm launch", mm::gemm_launch(cfg, a, s));
}

// Batched: every problem's extent and its offset b * stride must fit, strides >= 0.
int run_gemm_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const float *A, int64_t lda,
                     int64_t sa, const float *B, int64_t ldb, int64_t sb, float *C, int64_t ldc,
                     int64_t sc, void *stream)
{
    if (batch < 0) return invalid("negative batch");
    if (batch > 65535) return invalid("batch above 65535");
    if (sa < 0 || sb < 0 || sc < 0) return invalid("negative batch stride");
    if (batch == 0) return check_gemm_dims(M, N, K, lda, ldb, ldc);  // pointers may be NULL
    const int st = check_gemm(M, N, K, A, lda, B, ldb, C, ldc);
    if (st != MM_OK) return st;
    if (M == 0 || N == 0) return MM_OK;
    const int64_t limit = INT64_MAX / 8;
    if ((batch - 1) > 0 && (sa > limit / (batch - 1) || sb > limit / (batch - 1) ||
                            sc > limit / (batch - 1)))
        return invalid("batch offset overflows");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) {
        for (int64_t b = 0; b < batch; ++b) {
            const int r = from_hip("zero fill launch", mm::zero_fill_launch(C + b * sc, M, N, ldc, s));
            if (r != MM_OK) return r;
        }
        return MM_OK;
    }
    mm::GemmArgs a;
    a.A = A;
    a.B = B;
    a.C = C;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.batch = (int)batch;
    a.sa = sa;
    a.sb = sb;
    a.sc = sc;
    return from_hip("batched gemm launch",
                    mm::gemm_launch(mm::gemm_select_config(M, N, K, batch), a, s));
}

int run_gemm16(int cfg, bool bf16, int64_t M, int64_t N, int64_t K, const uint16_t *A,
               int64_t lda, const uint16_t *B, int64_t ldb, float *C, int64_t ldc, void *stream)
{
    const int st = check_gemm(M, N, K, A, lda, B, ldb, C, ldc, 2);
    if (st != MM_OK) return st;
    if (M == 0 || N == 0) return MM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) return from_hip("zero fill launch", mm::zero_fill_launch(C, M, N, ldc, s));
    if (cfg < 0) cfg = mm::gemm16_select_config(M, N, K);
    return from_hip("gemm16 launch", mm::gemm16_launch(cfg, bf16, A, lda, B, ldb, C, ldc, (int)M,
                                                       (int)N, (int)K, s));
}

constexpr int64_t kConvMaxGeom = int64_t(1) << 29;

// Output extent along one axis, or -1 (arguments as for mm_conv2d_out_dim).
int64_t conv_out_dim(int64_t in, int64_t filter, int64_t stride, int64_t pad, int64_t dil)
{
    if (in < 0 || filter < 1 || stride < 1 || pad < 0 || dil < 1) return -1;
    if (in >= kConvMaxGeom || filter >= kConvMaxGeom || stride >= kConvMaxGeom ||
        pad >= kConvMaxGeom || dil >= kConvMaxGeom)
        return -1;
    const int64_t span = dil * (filter - 1);  // < 2^58
    const int64_t padded = in + 2 * pad;
    if (span >= kConvMaxGeom || padded >= kConvMaxGeom) return -1;
    if (padded - span - 1 < 0) return -1;
    return (padded - span - 1) / stride + 1;
}

// Checks a convolution's arguments and fills `a`. Returns MM_OK, or the error; *work
// is false when there is no output element (nothing to enqueue).
int check_conv(int64_t N, int64_t C, int64_t H, int64_t W, int64_t K, int64_t R, int64_t S,
               int64_t sh, int64_t sw, int64_t ph, int64_t pw, int64_t dh, int64_t dw,
               const float *x, const float *w, const float *y, bool check_pointers,
               mm::ConvArgs &a, bool &work)
{
    work = false;
    if (N < 0 || C < 0 || H < 0 || W < 0 || K < 0) return invalid("negative size");
    if (R < 1 || S < 1) return invalid("filter size below 1");
    if (sh < 1 || sw < 1) return invalid("stride below 1");
    if (ph < 0 || pw < 0) return invalid("negative padding");
    if (dh < 1 || dw < 1) return invalid("dilation below 1");
    const int64_t P = conv_out_dim(H, R, sh, ph, dh), Q = conv_out_dim(W, S, sw, pw, dw);
    if (P < 0 || Q < 0) {
        if (H + 2 * ph >= kConvMaxGeom || W + 2 * pw >= kConvMaxGeom || R >= kConvMaxGeom ||
            S >= kConvMaxGeom || dh >= kConvMaxGeom || dw >= kConvMaxGeom ||
            sh >= kConvMaxGeom || sw >= kConvMaxGeom || dh * (R - 1) >= kConvMaxGeom ||
            dw * (S - 1) >= kConvMaxGeom)
            return invalid("convolution geometry above 2^29");
        return invalid("filter does not fit the padded input");
    }
    if (K > kMaxDim || N > kMaxDim || C > kMaxDim) return invalid("size above 2^31 - 1");
    const int64_t HW = H * W, PQ = P * Q;  // each below 2^58
    const int64_t kMaxImage = (int64_t(1) << 30) - 1;
    if (C > 0 && HW > kMaxImage / C) return invalid("C * H * W above 2^30 - 1");
    // P * Q <= (H + 2 ph)(W + 2 pw), so this also keeps P * Q below 2^30
    if ((H + 2 * ph) * (W + 2 * pw) > kMaxImage) return invalid("padded plane above 2^30 - 1");
    if (C > 0 && R * S > kMaxDim / C) return invalid("C * R * S above 2^31 - 1");
    const int64_t limit = INT64_MAX / 4;
    const int64_t CHW = C * HW, CRS = C * R * S;
    if (N > 0 && CHW > limit / N) return invalid("x extent overflows");
    if (K > 0 && PQ > 0 && N > limit / K / PQ) return invalid("y extent overflows");
    if (check_pointers) {
        const bool has_x = N > 0 && CHW > 0, has_w = K > 0 && CRS > 0, has_y = N > 0 && K > 0;
        if (has_x && !x) return invalid("x is NULL");
        if (has_w && !w) return invalid("w is NULL");
        if (has_y && !y) return invalid("y is NULL");
        if ((uintptr_t)x % 4 || (uintptr_t)w % 4 || (uintptr_t)y % 4)
            return invalid("pointer not aligned to its element size");
    }
    a.N = N;
    a.C = C;
    a.H = H;
    a.W = W;
    a.K = K;
    a.R = R;
    a.S = S;
    a.sh = sh;
    a.sw = sw;
    a.ph = ph;
    a.pw = pw;
    a.dh = dh;
    a.dw = dw;
    a.P = P;
    a.Q = Q;
    a.x = x;
    a.w = w;
    a.y = const_cast<float *>(y);
    work = N > 0 && K > 0;  // P, Q >= 1 here
    return MM_OK;
}

int run_conv(int cfg, int64_t N, int64_t C, int64_t H, int64_t W, int64_t K, int64_t R,
             int64_t S, int64_t sh, int64_t sw, int64_t ph, int64_t pw, int64_t dh, int64_t dw,
             const float *x, const float *w, float *y, void *stream)
{
    mm::ConvArgs a;
    bool work;
    const int st = check_conv(N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, x, w, y, true, a, work);
    if (st != MM_OK || !work) return st;
    return from_hip("conv2d launch", mm::conv_launch(cfg, a, static_cast<hipStream_t>(stream)));
}

// Largest K of the 8-bit products: sums of K products of magnitude up to 2^14 fit 32 bits.
constexpr int64_t kMaxKInt8 = (int64_t(1) << 17) - 1;
constexpr int64_t kMaxGroups = 4096;  // a workgroup finds its group among them by itself

bool type_ok(int t) { return t == MM_TYPE_F32 || t == MM_TYPE_BF16 || t == MM_TYPE_F16; }
int type_size(int t) { return t == MM_TYPE_F32 ? 4 : 2; }

// Byte extent of `count` rows x cols matrices, `stride` elements apart, fits in int64.
bool strided_extent_fits(int64_t count, int64_t stride, int64_t rows, int64_t cols, int64_t ld)
{
    if (!extent_fits(rows, cols, ld)) return false;
    const int64_t one = (rows - 1) * ld + cols, limit = INT64_MAX / 4;
    return count <= 1 || stride <= (limit - one) / (count - 1);
}

// Checks of the grouped products; rows mode and gradient mode differ in the operands' shapes.
// offsets == nullptr with dense == true: the product of one group of all rows.
int check_group(const mm::GroupArgs &a, int64_t groups, int64_t M, int64_t N, int64_t K, bool dense)
{
    if (groups < 0 || M < 0 || N < 0 || K < 0) return invalid("negative size");
    if (groups > kMaxGroups) return invalid("more than 4096 groups");
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return invalid("size above 2^31 - 1");
    const bool i8 = a.elem == mm::GroupElem::I8;
    if (i8 && K > kMaxKInt8) return invalid("K above 2^17 - 1 (sums of 8-bit products fit 32 bits up to there)");
    if (!type_ok(a.c_type)) return invalid("unknown output type");
    // A is M x K; B_g is K x N, or N x K transposed; in gradient mode B is the M x N gradient
    // and C_g is K x N
    const int64_t b_rows = a.grad ? M : a.trans_b ? N : K, b_cols = a.grad ? N : a.trans_b ? K : N;
    const int64_t c_rows = a.grad ? K : M, b_count = a.grad ? 1 : groups, c_count = a.grad ? groups : 1;
    const bool mx4 = a.elem == mm::GroupElem::Mx4;  // K counts bytes
    if (a.lda < (K > 1 ? K : 1)) return invalid(mx4 ? "lda < max(1, K / 2)" : "lda < max(1, K)");
    if (a.ldb < (b_cols > 1 ? b_cols : 1))
        return invalid(mx4 ? "ldb < max(1, K / 2)" : a.grad ? "ldg < max(1, N)" : a.trans_b ? "ldb < max(1, K)" : "ldb < max(1, N)");
    if (a.ldc < (N > 1 ? N : 1)) return invalid(a.grad ? "ldd < max(1, N)" : "ldc < max(1, N)");
    if (a.stride_b < 0 || a.stride_c < 0) return invalid("negative group stride");
    if (groups == 0) return MM_OK;  // no rows belong to a group: pointers may be NULL
    const bool has_a = M > 0 && K > 0, has_b = b_rows > 0 && b_cols > 0, has_c = c_rows > 0 && N > 0;
    if (has_a && !a.A) return invalid("A is NULL");
    if (has_b && !a.B) return invalid(a.grad ? "G is NULL" : "B is NULL");
    if (has_c && !a.C) return invalid(a.grad ? "D is NULL" : "C is NULL");
    if (!dense && !a.offsets) return invalid("offsets is NULL");
    const int elem = mm::group_elem_size(a);
    if ((uintptr_t)a.A % elem || (uintptr_t)a.B % elem || (uintptr_t)a.C % type_size(a.c_type))
        return invalid("pointer not aligned to its element size");
    if ((uintptr_t)a.offsets % 8) return invalid("offsets not 8-byte aligned");
    if (i8) {
        if (M > 0 && !a.sa) return invalid("a_scale is NULL");
        if (N > 0 && !a.sb) return invalid("b_scale is NULL");
        if ((uintptr_t)a.sa % 4 || (uintptr_t)a.sb % 4) return invalid("scales not 4-byte aligned");
    }
    if (has_a && !extent_fits(M, K, a.lda)) return invalid("A extent overflows");
    if (has_b && !strided_extent_fits(b_count, a.stride_b, b_rows, b_cols, a.ldb))
        return invalid(a.grad ? "G extent overflows" : "B extent overflows");
    if (has_c && !strided_extent_fits(c_count, a.stride_c, c_rows, N, a.ldc))
        return invalid(a.grad ? "D extent overflows" : "C extent overflows");
    return MM_OK;
}

int run_group(mm::GroupArgs &a, int64_t groups, int64_t M, int64_t N, int64_t K, bool dense, void *stream)
{
    const int st = check_group(a, groups, M, N, K, dense);
    if (st != MM_OK) return st;
    if (groups == 0 || N == 0 || (a.grad ? K : M) == 0) return MM_OK;  // no output
    a.groups = (int)groups;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    return from_hip(a.grad ? "grouped gradient launch" : !dense ? "grouped gemm launch" : a.elem == mm::GroupElem::I8 ? "i8 gemm launch" : "mx4 gemm launch",
                    mm::group_launch(a, static_cast<hipStream_t>(stream)));
}

// The kernel of the call that `a` describes but for its offsets, outputs and scales; -1 if it is refused
// or launches nothing.
int select_group(mm::GroupArgs &a, int64_t groups, int64_t M, int64_t N, int64_t K, bool dense)
{
    static const int64_t present = 0;  // its address stands for the pointers that the choice does not use
    a.C = const_cast<int64_t *>(&present);
    a.offsets = dense ? nullptr : &present;
    a.sa = a.sb = reinterpret_cast<const float *>(&present);
    a.ldc = N > 1 ? N : 1;
    a.stride_c = 0;
    a.c_type = MM_TYPE_F32;
    if (check_group(a, groups, M, N, K, dense) != MM_OK) return -1;
    if (groups == 0 || N == 0 || (a.grad ? K : M) == 0) return -1;
    a.groups = (int)groups;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    return mm::group_select(a);
}

int run_grouped16(mm::GroupElem elem, int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets,
                  const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, int64_t stride_b, int trans_b,
                  void *C, int c_type, int64_t ldc, void *stream)
{
    if (trans_b != 0 && trans_b != 1) return invalid("trans_b is neither 0 nor 1");
    mm::GroupArgs a{};
    a.elem = elem;
    a.A = A;
    a.B = B;
    a.C = C;
    a.offsets = offsets;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.stride_b = stride_b;
    a.trans_b = trans_b == 1;
    a.c_type = c_type;
    return run_group(a, groups, M, N, K, false, stream);
}

int run_grouped16_grad_b(mm::GroupElem elem, int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets,
                         const uint16_t *A, int64_t lda, const uint16_t *G, int64_t ldg, void *D, int d_type,
                         int64_t ldd, int64_t stride_d, void *stream)
{
    mm::GroupArgs a{};
    a.elem = elem;
    a.grad = true;
    a.A = A;
    a.B = G;
    a.C = D;
    a.offsets = offsets;
    a.lda = lda;
    a.ldb = ldg;
    a.ldc = ldd;
    a.stride_c = stride_d;
    a.c_type = d_type;
    return run_group(a, groups, M, N, K, false, stream);
}

// The 4-bit products: the public K counts elements, the kernels' bytes of two of them.
int check_mx4(mm::GroupArgs &a, int64_t groups, int64_t M, int64_t N, int64_t K)
{
    if (K % 32) return invalid("K is no multiple of 32");
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim || groups < 0 || groups > kMaxGroups)
        return MM_OK;  // check_group names these
    const int64_t blocks = K / 32, least = blocks > 1 ? blocks : 1;
    if (a.ld_mxa < least) return invalid("ld of a_scale < max(1, K / 32)");
    if (a.ld_mxb < least) return invalid("ld of b_scale < max(1, K / 32)");
    if (a.stride_mxb < 0) return invalid("negative group stride");
    if (groups == 0 || K == 0) return MM_OK;
    if (M > 0 && !a.mxa) return invalid("a_scale is NULL");
    if (N > 0 && !a.mxb) return invalid("b_scale is NULL");
    if (M > 0 && !extent_fits(M, blocks, a.ld_mxa)) return invalid("a_scale extent overflows");
    if (N > 0 && !strided_extent_fits(groups, a.stride_mxb, N, blocks, a.ld_mxb))
        return invalid("b_scale extent overflows");
    return MM_OK;
}

mm::GroupArgs mx4_args(const int64_t *offsets, const uint8_t *A, int64_t lda, const uint8_t *a_scale, int64_t ld_as,
                       const uint8_t *B, int64_t ldb, int64_t stride_b, const uint8_t *b_scale, int64_t ld_bs,
                       int64_t stride_bs, void *C, int c_type, int64_t ldc)
{
    mm::GroupArgs a{};
    a.elem = mm::GroupElem::Mx4;
    a.trans_b = true;
    a.A = A;
    a.B = B;
    a.C = C;
    a.offsets = offsets;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.stride_b = stride_b;
    a.c_type = c_type;
    a.mxa = a_scale;
    a.mxb = b_scale;
    a.ld_mxa = ld_as;
    a.ld_mxb = ld_bs;
    a.stride_mxb = stride_bs;
    return a;
}

// Rows of 4-bit blocks: the sizes and addresses that both directions check.
int check_mx4_rows(int64_t rows, int64_t cols, const void *X, int x_type, int64_t ldx, const uint8_t *Q, int64_t ldq,
                   const uint8_t *scale, int64_t ld_scale)
{
    if (rows < 0 || cols < 0) return invalid("negative size");
    if (rows > kMaxDim || cols > kMaxDim) return invalid("size above 2^31 - 1");
    if (!type_ok(x_type)) return invalid("unknown type of X");
    const int64_t blocks = (cols + 31) / 32;
    if (ldx < (cols > 1 ? cols : 1)) return invalid("ldx < max(1, cols)");
    if (ldq < (blocks > 0 ? 16 * blocks : 1)) return invalid("ldq < max(1, 16 ceil(cols / 32))");
    if (ld_scale < (blocks > 0 ? blocks : 1)) return invalid("ld_scale < max(1, ceil(cols / 32))");
    if (rows == 0 || cols == 0) return MM_OK;
    if (!X) return invalid("X is NULL");
    if (!Q) return invalid("Q is NULL");
    if (!scale) return invalid("scale is NULL");
    if ((uintptr_t)X % type_size(x_type)) return invalid("pointer not aligned to its element size");
    if (!extent_fits(rows, cols, ldx) || !extent_fits(rows, 16 * blocks, ldq) || !extent_fits(rows, blocks, ld_scale))
        return invalid("extent overflows");
    return MM_OK;
}

int check_route(int64_t T, int64_t E, int64_t k, const void *logits, int type, int64_t ld, int scoring, int renormalize)
{
    if (T < 0 || E < 0 || k < 0) return invalid("negative size");
    if (E > mm::kRouteMaxExperts) return invalid("more than 1024 experts");
    if (k > mm::kRouteMaxTop) return invalid("more than 32 experts to a token");
    if (k > E) return invalid("more experts to a token than there are");
    if (T > kMaxDim || (k > 0 && T > kMaxDim / k)) return invalid("T k above 2^31 - 1");
    if (!type_ok(type)) return invalid("unknown type of the logits");
    if (scoring != MM_ROUTE_SOFTMAX && scoring != MM_ROUTE_SIGMOID) return invalid("unknown scoring");
    if (renormalize != 0 && renormalize != 1) return invalid("renormalize is neither 0 nor 1");
    if (ld < (E > 1 ? E : 1)) return invalid("ld < max(1, E)");
    if (T > 0 && E > 0 && !logits) return invalid("logits is NULL");
    if ((uintptr_t)logits % type_size(type)) return invalid("pointer not aligned to its element size");
    if (T > 0 && E > 0 && !extent_fits(T, E, ld)) return invalid("logits extent overflows");
    return MM_OK;
}

// A matrix of `rows` x `cols` elements of `size` bytes that is used where it has elements.
int check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int size, const char *null, const char *extent)
{
    if (rows == 0 || cols == 0) return MM_OK;
    if (!p) return invalid(null);
    if ((uintptr_t)p % size) return invalid("pointer not aligned to its element size");
    if (!extent_fits(rows, cols, ld)) return invalid(extent);
    return MM_OK;
}

int check_rows(int64_t T, int64_t k, int64_t D, int64_t total, const int32_t *rows)
{
    if (T < 0 || k < 0 || D < 0 || total < 0) return invalid("negative size");
    if (T > kMaxDim || D > kMaxDim || total > kMaxDim) return invalid("size above 2^31 - 1");
    if (k > mm::kRowsMaxSlots) return invalid("more than 1024 slots to a token");
    if (k > 0 && T > kMaxDim / k) return invalid("T k above 2^31 - 1");
    if (T > 0 && k > 0 && !rows) return invalid("rows is NULL");
    if ((uintptr_t)rows % 4) return invalid("rows not 4-byte aligned");
    return MM_OK;
}

}  // namespace

extern "C" {

int mm_gemm_f32(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
                int64_t ldb, float *C, int64_t ldc, void *stream)
{
    return run_gemm(-1, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int64_t mm_gemm_f32_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return -1;
    if (M == 0 || N == 0 || K == 0) return 0;
    return 4 * mm::gemm_split_ws_floats(M, N, K);
}

int mm_gemm_f32_ws(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
                   int64_t ldb, float *C, int64_t ldc, void *workspace, int64_t workspace_bytes, void *stream)
{
    const int64_t need = mm_gemm_f32_workspace_bytes(M, N, K);
    if (need > 0) {
        if (!workspace) return invalid("workspace is NULL");
        if ((uintptr_t)workspace % 16) return invalid("workspace not 16-byte aligned");
        if (workspace_bytes < need) return invalid("workspace smaller than mm_gemm_f32_workspace_bytes");
    }
    if (need <= 0) return run_gemm(-1, M, N, K, A, lda, B, ldb, C, ldc, stream);
    const int st = check_gemm(M, N, K, A, lda, B, ldb, C, ldc);
    if (st != MM_OK) return st;
    mm::GemmArgs a;
    a.A = A;
    a.B = B;
    a.C = C;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    return from_hip("split gemm launch", mm::gemm_split_launch(a, static_cast<float *>(workspace),
                                                                static_cast<hipStream_t>(stream)));
}

int mm_gemm_f32_ws_static(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
                          int64_t ldb, float *C, int64_t ldc, void *stream)
{
    const int64_t need = mm_gemm_f32_workspace_bytes(M, N, K);
    if (need <= 0) return run_gemm(-1, M, N, K, A, lda, B, ldb, C, ldc, stream);  // no scratch used
    const int st = check_gemm(M, N, K, A, lda, B, ldb, C, ldc);
    if (st != MM_OK) return st;
    if (need > MM_STATIC_SCRATCH_BYTES)
        return invalid("the K split of this shape needs more than the MM_STATIC_SCRATCH_BYTES of static scratch");
    mm::GemmArgs a;
    a.A = A;
    a.B = B;
    a.C = C;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    const int r = mm::gemm_split_static_launch(a, static_cast<hipStream_t>(stream));
    if (r != MM_OK) set_error_text(mm::static_ws_error());
    return r;
}

int mm_gemm_f32_config(int cfg, int64_t M, int64_t N, int64_t K, const float *A, int64_t lda,
                       const float *B, int64_t ldb, float *C, int64_t ldc, void *stream)
{
    if (cfg < 0 || cfg >= mm::gemm_num_configs()) return invalid("config index out of range");
    return run_gemm(cfg, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int mm_gemm_f32_num_configs(void) { return mm::gemm_num_configs(); }

const char *mm_gemm_f32_config_name(int cfg) { return mm::gemm_config_name(cfg); }

int mm_gemm_f32_select(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0) return 0;
    if (mm::gemm_split2_ok(M, N, K)) return mm::gemm_split2_config();
    return mm::gemm_select_config(M, N, K);
}

int mm_gemm_f32_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const float *A,
                        int64_t lda, int64_t stride_a, const float *B, int64_t ldb,
                        int64_t stride_b, float *C, int64_t ldc, int64_t stride_c, void *stream)
{
    return run_gemm_batched(batch, M, N, K, A, lda, stride_a, B, ldb, stride_b, C, ldc, stride_c,
                            stream);
}

int mm_gemm_bf16(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                 const uint16_t *B, int64_t ldb, float *C, int64_t ldc, void *stream)
{
    return run_gemm16(-1, true, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int mm_gemm_f16(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                const uint16_t *B, int64_t ldb, float *C, int64_t ldc, void *stream)
{
    return run_gemm16(-1, false, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int mm_gemm_bf16_config(int cfg, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                        const uint16_t *B, int64_t ldb, float *C, int64_t ldc, void *stream)
{
    if (cfg < 0 || cfg >= mm::gemm16_num_configs()) return invalid("config index out of range");
    return run_gemm16(cfg, true, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int mm_gemm_f16_config(int cfg, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                       const uint16_t *B, int64_t ldb, float *C, int64_t ldc, void *stream)
{
    if (cfg < 0 || cfg >= mm::gemm16_num_configs()) return invalid("config index out of range");
    return run_gemm16(cfg, false, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int mm_gemm_h16_num_configs(void) { return mm::gemm16_num_configs(); }

const char *mm_gemm_h16_config_name(int cfg) { return mm::gemm16_config_name(cfg); }

int mm_gemm_h16_select(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0) return 0;
    return mm::gemm16_select_config(M, N, K);
}

int mm_gemv_f32(int64_t M, int64_t N, const float *A, const float *x, float *y, void *stream)
{
    if (M < 0 || N < 0) return invalid("negative size");
    if (M > kMaxDim || N > kMaxDim) return invalid("size above 2^31 - 1");
    if (M > 0 && N > 0 && !A) return invalid("A is NULL");
    if (N > 0 && !x) return invalid("x is NULL");
    if (M > 0 && !y) return invalid("y is NULL");
    if ((uintptr_t)A % 4 || (uintptr_t)x % 4 || (uintptr_t)y % 4)
        return invalid("pointer not aligned to its element size");
    if (M > 0 && N > 0 && !extent_fits(M, N, N)) return invalid("A extent overflows");
    if (M == 0) return MM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (N == 0) return from_hip("zero fill launch", mm::zero_fill_launch(y, 1, M, M, s));
    mm::GemvArgs a;
    a.A = A;
    a.x = x;
    a.y = y;
    a.M = (int)M;
    a.N = (int)N;
    return from_hip("gemv launch", mm::gemv_launch(a, s));
}

int mm_gemv_t_f32(int64_t M, int64_t N, const float *A, const float *x, float *y, void *stream)
{
    if (M < 0 || N < 0) return invalid("negative size");
    if (M > kMaxDim || N > kMaxDim) return invalid("size above 2^31 - 1");
    if (M > 0 && N > 0 && !A) return invalid("A is NULL");
    if (M > 0 && !x) return invalid("x is NULL");
    if (N > 0 && !y) return invalid("y is NULL");
    if ((uintptr_t)A % 4 || (uintptr_t)x % 4 || (uintptr_t)y % 4)
        return invalid("pointer not aligned to its element size");
    if (M > 0 && N > 0 && !extent_fits(M, N, N)) return invalid("A extent overflows");
    if (N == 0) return MM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) return from_hip("zero fill launch", mm::zero_fill_launch(y, 1, N, N, s));
    mm::GemvArgs a;
    a.A = A;
    a.x = x;
    a.y = y;
    a.M = (int)M;
    a.N = (int)N;
    return from_hip("gemv_t launch", mm::gemv_t_launch(a, s));
}

int64_t mm_gemv_t_f32_workspace_bytes(int64_t M, int64_t N)
{
    if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return -1;
    if (M == 0 || N == 0) return 0;
    return 4 * mm::gemv_t_ws_floats(M, N);
}

int mm_gemv_t_f32_ws(int64_t M, int64_t N, const float *A, const float *x, float *y, void *workspace,
                     int64_t workspace_bytes, void *stream)
{
    const int64_t need = mm_gemv_t_f32_workspace_bytes(M, N);
    if (need > 0) {
        if (!workspace) return invalid("workspace is NULL");
        if ((uintptr_t)workspace % 16) return invalid("workspace not 16-byte aligned");
        if (workspace_bytes < need) return invalid("workspace smaller than mm_gemv_t_f32_workspace_bytes");
    }
    if (need <= 0) return mm_gemv_t_f32(M, N, A, x, y, stream);  // the checks and the strips kernel
    // same checks as mm_gemv_t_f32 (M, N >= 1 here)
    if (!A) return invalid("A is NULL");
    if (!x) return invalid("x is NULL");
    if (!y) return invalid("y is NULL");
    if ((uintptr_t)A % 4 || (uintptr_t)x % 4 || (uintptr_t)y % 4)
        return invalid("pointer not aligned to its element size");
    if (!extent_fits(M, N, N)) return invalid("A extent overflows");
    mm::GemvArgs a;
    a.A = A;
    a.x = x;
    a.y = y;
    a.M = (int)M;
    a.N = (int)N;
    return from_hip("gemv_t launch", mm::gemv_t_ws_launch(a, static_cast<float *>(workspace),
                                                            static_cast<hipStream_t>(stream)));
}

int mm_conv2d_f32(int64_t N, int64_t C, int64_t H, int64_t W, int64_t K, int64_t R, int64_t S,
                  int64_t sh, int64_t sw, int64_t ph, int64_t pw, int64_t dh, int64_t dw,
                  const float *x, const float *w, float *y, void *stream)
{
    return run_conv(-1, N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, x, w, y, stream);
}

int mm_conv2d_f32_config(int cfg, int64_t N, int64_t C, int64_t H, int64_t W, int64_t K,
                         int64_t R, int64_t S, int64_t sh, int64_t sw, int64_t ph, int64_t pw,
                         int64_t dh, int64_t dw, const float *x, const float *w, float *y,
                         void *stream)
{
    if (cfg < 0 || cfg >= mm::conv_num_configs()) return invalid("config index out of range");
    return run_conv(cfg, N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, x, w, y, stream);
}

int64_t mm_conv2d_out_dim(int64_t in, int64_t filter, int64_t stride, int64_t pad, int64_t dil)
{
    return conv_out_dim(in, filter, stride, pad, dil);
}

int mm_conv2d_f32_num_configs(void) { return mm::conv_num_configs(); }

const char *mm_conv2d_f32_config_name(int cfg) { return mm::conv_config_name(cfg); }

int mm_conv2d_f32_select(int64_t N, int64_t C, int64_t H, int64_t W, int64_t K, int64_t R,
                         int64_t S, int64_t sh, int64_t sw, int64_t ph, int64_t pw, int64_t dh,
                         int64_t dw)
{
    mm::ConvArgs a;
    bool work;
    if (check_conv(N, C, H, W, K, R, S, sh, sw, ph, pw, dh, dw, nullptr, nullptr, nullptr, false, a,
                   work) != MM_OK)
        return -1;
    return mm::conv_choose_config(a);
}

int mm_gemm_bf16_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets, const uint16_t *A,
                         int64_t lda, const uint16_t *B, int64_t ldb, int64_t stride_b, int trans_b, void *C,
                         int c_type, int64_t ldc, void *stream)
{
    return run_grouped16(mm::GroupElem::Bf16, groups, M, N, K, offsets, A, lda, B, ldb, stride_b, trans_b, C, c_type,
                         ldc, stream);
}

int mm_gemm_f16_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets, const uint16_t *A,
                        int64_t lda, const uint16_t *B, int64_t ldb, int64_t stride_b, int trans_b, void *C,
                        int c_type, int64_t ldc, void *stream)
{
    return run_grouped16(mm::GroupElem::F16, groups, M, N, K, offsets, A, lda, B, ldb, stride_b, trans_b, C, c_type,
                         ldc, stream);
}

int mm_gemm_bf16_grouped_grad_b(int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets,
                                const uint16_t *A, int64_t lda, const uint16_t *G, int64_t ldg, void *D, int d_type,
                                int64_t ldd, int64_t stride_d, void *stream)
{
    return run_grouped16_grad_b(mm::GroupElem::Bf16, groups, M, N, K, offsets, A, lda, G, ldg, D, d_type, ldd,
                                stride_d, stream);
}

int mm_gemm_f16_grouped_grad_b(int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets,
                               const uint16_t *A, int64_t lda, const uint16_t *G, int64_t ldg, void *D, int d_type,
                               int64_t ldd, int64_t stride_d, void *stream)
{
    return run_grouped16_grad_b(mm::GroupElem::F16, groups, M, N, K, offsets, A, lda, G, ldg, D, d_type, ldd,
                                stride_d, stream);
}

int mm_quantize_i8(int64_t rows, int64_t cols, const void *X, int x_type, int64_t ldx, int8_t *Q, int64_t ldq,
                   float *scale, void *stream)
{
    if (rows < 0 || cols < 0) return invalid("negative size");
    if (rows > kMaxDim || cols > kMaxDim) return invalid("size above 2^31 - 1");
    if (!type_ok(x_type)) return invalid("unknown input type");
    if (ldx < (cols > 1 ? cols : 1)) return invalid("ldx < max(1, cols)");
    if (ldq < (cols > 1 ? cols : 1)) return invalid("ldq < max(1, cols)");
    if (rows > 0 && cols > 0 && !X) return invalid("X is NULL");
    if (rows > 0 && cols > 0 && !Q) return invalid("Q is NULL");
    if (rows > 0 && !scale) return invalid("scale is NULL");
    if ((uintptr_t)X % type_size(x_type) || (uintptr_t)scale % 4)
        return invalid("pointer not aligned to its element size");
    if (rows > 0 && cols > 0 && !(extent_fits(rows, cols, ldx) && extent_fits(rows, cols, ldq)))
        return invalid("extent overflows");
    if (rows == 0) return MM_OK;
    mm::QuantArgs a;
    a.X = X;
    a.Q = Q;
    a.scale = scale;
    a.rows = rows;
    a.cols = cols;
    a.ldx = ldx;
    a.ldq = ldq;
    a.x_type = x_type;
    return from_hip("quantize launch", mm::quantize_launch(a, static_cast<hipStream_t>(stream)));
}

int mm_gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const float *a_scale, const int8_t *B,
               int64_t ldb, const float *b_scale, void *C, int c_type, int64_t ldc, void *stream)
{
    mm::GroupArgs a{};
    a.elem = mm::GroupElem::I8;
    a.trans_b = true;
    a.A = A;
    a.B = B;
    a.C = C;
    a.sa = a_scale;
    a.sb = b_scale;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.c_type = c_type;
    return run_group(a, 1, M, N, K, true, stream);
}

int mm_gemm_i8_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets, const int8_t *A,
                       int64_t lda, const float *a_scale, const int8_t *B, int64_t ldb, int64_t stride_b,
                       const float *b_scale, void *C, int c_type, int64_t ldc, void *stream)
{
    mm::GroupArgs a{};
    a.elem = mm::GroupElem::I8;
    a.trans_b = true;
    a.A = A;
    a.B = B;
    a.C = C;
    a.offsets = offsets;
    a.sa = a_scale;
    a.sb = b_scale;
    a.lda = lda;
    a.ldb = ldb;
    a.ldc = ldc;
    a.stride_b = stride_b;
    a.stride_sb = N;
    a.c_type = c_type;
    return run_group(a, groups, M, N, K, false, stream);
}

int mm_quantize_mx4(int64_t rows, int64_t cols, const void *X, int x_type, int64_t ldx, uint8_t *Q, int64_t ldq,
                    uint8_t *scale, int64_t ld_scale, void *stream)
{
    const int st = check_mx4_rows(rows, cols, X, x_type, ldx, Q, ldq, scale, ld_scale);
    if (st != MM_OK || rows == 0 || cols == 0) return st;
    const mm::Mx4Args a{const_cast<void *>(X), Q, scale, rows, cols, ldx, ldq, ld_scale, x_type};
    return from_hip("quantize launch", mm::mx4_quantize_launch(a, static_cast<hipStream_t>(stream)));
}

int mm_dequantize_mx4(int64_t rows, int64_t cols, const uint8_t *Q, int64_t ldq, const uint8_t *scale,
                      int64_t ld_scale, void *X, int x_type, int64_t ldx, void *stream)
{
    const int st = check_mx4_rows(rows, cols, X, x_type, ldx, Q, ldq, scale, ld_scale);
    if (st != MM_OK || rows == 0 || cols == 0) return st;
    const mm::Mx4Args a{X, const_cast<uint8_t *>(Q), const_cast<uint8_t *>(scale), rows, cols, ldx, ldq, ld_scale, x_type};
    return from_hip("dequantize launch", mm::mx4_dequantize_launch(a, static_cast<hipStream_t>(stream)));
}

int mm_gemm_mx4(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *a_scale, int64_t ld_as,
                const uint8_t *B, int64_t ldb, const uint8_t *b_scale, int64_t ld_bs, void *C, int c_type, int64_t ldc,
                void *stream)
{
    mm::GroupArgs a = mx4_args(nullptr, A, lda, a_scale, ld_as, B, ldb, 0, b_scale, ld_bs, 0, C, c_type, ldc);
    const int st = check_mx4(a, 1, M, N, K);
    return st != MM_OK ? st : run_group(a, 1, M, N, K / 2, true, stream);
}

int mm_gemm_mx4_grouped(int64_t groups, int64_t M, int64_t N, int64_t K, const int64_t *offsets, const uint8_t *A,
                        int64_t lda, const uint8_t *a_scale, int64_t ld_as, const uint8_t *B, int64_t ldb,
                        int64_t stride_b, const uint8_t *b_scale, int64_t ld_bs, int64_t stride_bs, void *C, int c_type,
                        int64_t ldc, void *stream)
{
    mm::GroupArgs a =
        mx4_args(offsets, A, lda, a_scale, ld_as, B, ldb, stride_b, b_scale, ld_bs, stride_bs, C, c_type, ldc);
    const int st = check_mx4(a, groups, M, N, K);
    return st != MM_OK ? st : run_group(a, groups, M, N, K / 2, false, stream);
}

int64_t mm_route_topk_workspace_bytes(int64_t T, int64_t E, int64_t k)
{
    if (T < 0 || E < 0 || k < 0 || E > mm::kRouteMaxExperts || k > mm::kRouteMaxTop || k > E || T > kMaxDim ||
        (k > 0 && T > kMaxDim / k))
        return -1;
    return T == 0 || k == 0 ? 0 : 4 * mm::route_ws_ints(T, (int)E, (int)k);
}

int mm_route_topk(int64_t T, int64_t E, int64_t k, const void *logits, int type, int64_t ld, int scoring,
                  const float *bias, int64_t groups, int64_t top_groups, int64_t group_top, int renormalize,
                  float scale, float *weights, int32_t *experts, int32_t *rows, int64_t *offsets, void *workspace,
                  int64_t workspace_bytes, void *stream)
{
    const int st = check_route(T, E, k, logits, type, ld, scoring, renormalize);
    if (st != MM_OK) return st;
    if (groups < 1 || groups > 64) return invalid("groups outside 1 .. 64");
    if (E % groups) return invalid("E is no multiple of groups");
    if (top_groups < 1 || top_groups > groups) return invalid("top_groups outside 1 .. groups");
    if (group_top != 1 && group_top != 2) return invalid("group_top is neither 1 nor 2");
    if (k > E / groups * top_groups) return invalid("more experts to a token than the kept groups have");
    const bool any = T > 0 && k > 0;
    if (any && !weights) return invalid("weights is NULL");
    if (any && !experts) return invalid("experts is NULL");
    if (any && !rows) return invalid("rows is NULL");
    if (!offsets) return invalid("offsets is NULL");
    if ((uintptr_t)offsets % 8) return invalid("offsets not 8-byte aligned");
    if ((uintptr_t)bias % 4 || (uintptr_t)weights % 4 || (uintptr_t)experts % 4 || (uintptr_t)rows % 4)
        return invalid("pointer not aligned to its element size");
    const int64_t need = mm_route_topk_workspace_bytes(T, E, k);
    if (need > 0) {
        if (!workspace) return invalid("workspace is NULL");
        if ((uintptr_t)workspace % 16) return invalid("workspace not 16-byte aligned");
        if (workspace_bytes < need) return invalid("workspace smaller than mm_route_topk_workspace_bytes");
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    // no rows: every expert's begin at 0 (the fill counts words)
    if (!any) return from_hip("zero fill launch", mm::zero_fill_launch(reinterpret_cast<float *>(offsets), 1, 2 * (E + 1), 2 * (E + 1), s));
    mm::RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.weights = weights;
    a.experts = experts;
    a.rows = rows;
    a.offsets = offsets;
    a.ws = static_cast<int *>(workspace);
    a.ld = ld;
    a.T = (int)T;
    a.E = (int)E;
    a.k = (int)k;
    a.groups = (int)groups;
    a.top_groups = (int)top_groups;
    a.group_top = (int)group_top;
    a.type = type;
    a.sigmoid = scoring == MM_ROUTE_SIGMOID;
    a.renormalize = renormalize == 1;
    a.scale = scale;
    return from_hip("route launch", mm::route_launch(a, s));
}

int mm_route_topk_grad(int64_t T, int64_t E, int64_t k, const void *logits, int type, int64_t ld, int scoring,
                       int renormalize, float scale, const int32_t *experts, const float *dweights, void *dlogits,
                       int64_t ldd, void *stream)
{
    const int st = check_route(T, E, k, logits, type, ld, scoring, renormalize);
    if (st != MM_OK) return st;
    if (ldd < (E > 1 ? E : 1)) return invalid("ldd < max(1, E)");
    const bool any = T > 0 && k > 0;
    if (any && !experts) return invalid("experts is NULL");
    if (any && !dweights) return invalid("dweights is NULL");
    if ((uintptr_t)experts % 4 || (uintptr_t)dweights % 4) return invalid("pointer not aligned to its element size");
    const int d = check_matrix(dlogits, T, E, ldd, type_size(type), "dlogits is NULL", "dlogits extent overflows");
    if (d != MM_OK || T == 0 || E == 0) return d;
    mm::RouteGradArgs a;
    a.logits = logits;
    a.experts = experts;
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.ld = ld;
    a.ldd = ldd;
    a.T = (int)T;
    a.E = (int)E;
    a.k = (int)k;
    a.type = type;
    a.sigmoid = scoring == MM_ROUTE_SIGMOID;
    a.renormalize = renormalize == 1;
    a.scale = scale;
    return from_hip("route gradient launch", mm::route_grad_launch(a, static_cast<hipStream_t>(stream)));
}

int mm_spread_rows(int64_t T, int64_t k, int64_t row_bytes, const void *X, int64_t ldx, const int32_t *rows,
                   int64_t total, void *Y, int64_t ldy, void *stream)
{
    int st = check_rows(T, k, row_bytes, total, rows);
    if (st != MM_OK) return st;
    if (ldx < (row_bytes > 1 ? row_bytes : 1)) return invalid("ldx < max(1, row_bytes)");
    if (ldy < (row_bytes > 1 ? row_bytes : 1)) return invalid("ldy < max(1, row_bytes)");
    const int64_t used = k > 0 && total > 0 ? T : 0;
    if ((st = check_matrix(X, used, row_bytes, ldx, 1, "X is NULL", "X extent overflows")) != MM_OK) return st;
    if ((st = check_matrix(Y, used > 0 ? total : 0, row_bytes, ldy, 1, "Y is NULL", "Y extent overflows")) != MM_OK) return st;
    if (used == 0 || row_bytes == 0) return MM_OK;
    mm::RowsArgs a{};
    a.x = X;
    a.out = Y;
    a.rows = rows;
    a.total = total;
    a.ldx = ldx;
    a.ldo = ldy;
    a.T = (int)T;
    a.k = (int)k;
    a.D = (int)row_bytes;
    return from_hip("spread rows launch", mm::spread_rows_launch(a, static_cast<hipStream_t>(stream)));
}

int mm_combine_rows(int64_t T, int64_t k, int64_t D, const void *Y, int y_type, int64_t ldy, int64_t total,
                    const int32_t *rows, const float *weights, void *C, int c_type, int64_t ldc, void *stream)
{
    int st = check_rows(T, k, D, total, rows);
    if (st != MM_OK) return st;
    if (!type_ok(y_type)) return invalid("unknown input type");
    if (!type_ok(c_type)) return invalid("unknown output type");
    if (ldy < (D > 1 ? D : 1)) return invalid("ldy < max(1, D)");
    if (ldc < (D > 1 ? D : 1)) return invalid("ldc < max(1, D)");
    if ((uintptr_t)weights % 4) return invalid("pointer not aligned to its element size");
    const int64_t used = T > 0 && k > 0 ? total : 0;
    if ((st = check_matrix(Y, used, D, ldy, type_size(y_type), "Y is NULL", "Y extent overflows")) != MM_OK) return st;
    if ((st = check_matrix(C, T, D, ldc, type_size(c_type), "C is NULL", "C extent overflows")) != MM_OK) return st;
    if (T == 0 || D == 0) return MM_OK;
    mm::RowsArgs a{};
    a.x = Y;
    a.out = C;
    a.rows = rows;
    a.weights = weights;
    a.total = total;
    a.ldx = ldy;
    a.ldo = ldc;
    a.T = (int)T;
    a.k = (int)k;
    a.D = (int)D;
    a.x_type = y_type;
    a.o_type = c_type;
    return from_hip("combine rows launch", mm::combine_rows_launch(a, static_cast<hipStream_t>(stream)));
}

int mm_combine_rows_grad(int64_t T, int64_t k, int64_t D, const void *G, int g_type, int64_t ldg, const void *Y,
                         int y_type, int64_t ldy, int64_t total, const int32_t *rows, const float *weights, void *dY,
                         int64_t lddy, float *dweights, void *stream)
{
    int st = check_rows(T, k, D, total, rows);
    if (st != MM_OK) return st;
    if (!type_ok(g_type) || !type_ok(y_type)) return invalid("unknown input type");
    if (ldg < (D > 1 ? D : 1)) return invalid("ldg < max(1, D)");
    if (ldy < (D > 1 ? D : 1)) return invalid("ldy < max(1, D)");
    if (lddy < (D > 1 ? D : 1)) return invalid("lddy < max(1, D)");
    const bool any = T > 0 && k > 0;
    if (any && !weights) return invalid("weights is NULL");
    if (any && !dweights) return invalid("dweights is NULL");
    if ((uintptr_t)weights % 4 || (uintptr_t)dweights % 4) return invalid("pointer not aligned to its element size");
    const int ys = type_size(y_type);
    if ((st = check_matrix(G, any ? T : 0, D, ldg, type_size(g_type), "G is NULL", "G extent overflows")) != MM_OK) return st;
    if ((st = check_matrix(Y, any ? total : 0, D, ldy, ys, "Y is NULL", "Y extent overflows")) != MM_OK) return st;
    if ((st = check_matrix(dY, any ? total : 0, D, lddy, ys, "dY is NULL", "dY extent overflows")) != MM_OK) return st;
    if (!any) return MM_OK;
    mm::RowsArgs a{};
    a.x = G;
    a.out = dY;
    a.y = Y;
    a.rows = rows;
    a.weights = weights;
    a.dweights = dweights;
    a.total = total;
    a.ldx = ldg;
    a.ldo = lddy;
    a.ldy = ldy;
    a.T = (int)T;
    a.k = (int)k;
    a.D = (int)D;
    a.x_type = g_type;
    a.y_type = y_type;
    return from_hip("combine rows gradient launch", mm::combine_rows_grad_launch(a, static_cast<hipStream_t>(stream)));
}

int mm_gemm_grouped_num_configs(void) { return mm::group_num_configs(); }
const char *mm_gemm_grouped_config_name(int cfg) { return mm::group_config_name(cfg); }

int mm_gemm_h16_grouped_select(int64_t groups, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                               const uint16_t *B, int64_t ldb, int64_t stride_b, int trans_b)
{
    if (trans_b != 0 && trans_b != 1) return -1;
    mm::GroupArgs a{};
    a.elem = mm::GroupElem::Bf16;
    a.A = A;
    a.B = B;
    a.lda = lda;
    a.ldb = ldb;
    a.stride_b = stride_b;
    a.trans_b = trans_b == 1;
    return select_group(a, groups, M, N, K, false);
}

int mm_gemm_h16_grouped_grad_b_select(int64_t groups, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                                      const uint16_t *G, int64_t ldg)
{
    mm::GroupArgs a{};
    a.elem = mm::GroupElem::Bf16;
    a.grad = true;
    a.A = A;
    a.B = G;
    a.lda = lda;
    a.ldb = ldg;
    return select_group(a, groups, M, N, K, false);
}

int mm_gemm_i8_select(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const int8_t *B, int64_t ldb)
{
    mm::GroupArgs a{};
    a.elem = mm::GroupElem::I8;
    a.trans_b = true;
    a.A = A;
    a.B = B;
    a.lda = lda;
    a.ldb = ldb;
    return select_group(a, 1, M, N, K, true);
}

int mm_gemm_i8_grouped_select(int64_t groups, int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda,
                              const int8_t *B, int64_t ldb, int64_t stride_b)
{
    mm::GroupArgs a{};
    a.elem = mm::GroupElem::I8;
    a.trans_b = true;
    a.A = A;
    a.B = B;
    a.lda = lda;
    a.ldb = ldb;
    a.stride_b = stride_b;
    a.stride_sb = N;
    return select_group(a, groups, M, N, K, false);
}

int mm_gemm_mx4_select(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const uint8_t *a_scale,
                       int64_t ld_as, const uint8_t *B, int64_t ldb, const uint8_t *b_scale, int64_t ld_bs)
{
    mm::GroupArgs a = mx4_args(nullptr, A, lda, a_scale, ld_as, B, ldb, 0, b_scale, ld_bs, 0, nullptr, 0, 0);
    return check_mx4(a, 1, M, N, K) != MM_OK ? -1 : select_group(a, 1, M, N, K / 2, true);
}

int mm_gemm_mx4_grouped_select(int64_t groups, int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda,
                               const uint8_t *a_scale, int64_t ld_as, const uint8_t *B, int64_t ldb, int64_t stride_b,
                               const uint8_t *b_scale, int64_t ld_bs, int64_t stride_bs)
{
    mm::GroupArgs a =
        mx4_args(nullptr, A, lda, a_scale, ld_as, B, ldb, stride_b, b_scale, ld_bs, stride_bs, nullptr, 0, 0);
    return check_mx4(a, groups, M, N, K) != MM_OK ? -1 : select_group(a, groups, M, N, K / 2, false);
}

const char *mm_status_string(int status)
{
    switch (status) {
    case MM_OK: return "ok";
    case MM_ERR_INVALID_ARG: return "invalid argument";
    case MM_ERR_NO_DEVICE: return "no HIP device";
    case MM_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown status";
    }
}

const char *mm_last_error(void) { return g_last_error; }

}  // extern "C"
