// mm_group_any.hip -- the grouped products and the 8-bit integer and 4-bit products for any shape,
// stride and alignment (see mm_group.h for the sums).
//
// One workgroup of 4 waves per 64 x 64 tile of C, each wave a 32 x 32 block. Per step the
// threads copy 64 bytes of k of both panels into LDS one element at a time (zeros outside
// the matrices), as rows of consecutive k whatever the operands' layout, so each MFMA operand
// is one 16-byte LDS read. Single elements make no demand on alignment or sizes, and bound
// the kernel (i8 8192 x 14336 x 4096 in 8.6 ms, 112 TOP/s; 4-bit 4.9 ms): it is the one for what the
// others do not take, a single column of matrices stored K x N, gradients of fewer than 8 rows or columns or with
// strides that put a K-step's rows past 2^32 bytes, and sizes within 1024 of 2^31. The choice among all
// of them is at the end of this file.
#include "mm_group.h"

namespace mm {
namespace {

constexpr int kTile = 64, kStepBytes = 64, kPitch = kStepBytes + 16;

// GRAD: gradient mode (A and B both with the sum running over rows). B_ROWS_K: B's rows run
// over k (B_g(k, j) at k ldb + j), otherwise over j.
template <class E, int OUT, bool GRAD, bool B_ROWS_K>
__global__ __launch_bounds__(256) void group_any_kernel(GroupArgs p)
{
    typedef typename E::T T;
    constexpr int BK = kStepBytes / (int)sizeof(T);
    __shared__ __attribute__((aligned(16))) char lds[2 * kTile * kPitch];

    const unsigned tiles_n = ((unsigned)p.N + kTile - 1) / kTile;
    int g, m0, m_end, k_lo, k_end, n0;
    const int64_t bid = linear_block();
    if constexpr (GRAD) {
        const unsigned tiles_m = ((unsigned)p.K + kTile - 1) / kTile;
        const int64_t per = (int64_t)tiles_m * tiles_n;
        if (bid >= per * p.groups) return;
        g = (int)(bid / per);
        const unsigned in = (unsigned)(bid - g * per);
        m0 = (int)(in / tiles_n) * kTile;
        n0 = (int)(in % tiles_n) * kTile;
        m_end = p.K;
        group_range(p.offsets, g, p.M, k_lo, k_end);
    } else {
        const RowTiles<kTile> tiles(p);
        if (bid >= (int64_t)tiles.total * tiles_n) return;
        RowTile t;
        if (!tiles.find(p, (unsigned)(bid / tiles_n), t)) return;
        g = t.g;
        m0 = t.row0;
        m_end = t.hi;
        n0 = (int)(bid % tiles_n) * kTile;
        k_lo = 0;
        k_end = p.K;
    }
    const T *A = static_cast<const T *>(p.A);
    const T *B = static_cast<const T *>(p.B) + (GRAD ? 0 : g * p.stride_b);

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    typename E::template Acc<32> acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0;

    T *As = reinterpret_cast<T *>(lds), *Bs = reinterpret_cast<T *>(lds + kTile * kPitch);
    constexpr int pitch = kPitch / (int)sizeof(T);
    for (int64_t k0 = k_lo; k0 < k_end; k0 += BK) {
        for (int e = tid; e < kTile * BK; e += 256) {
            const int i = GRAD ? e % kTile : e / BK, kk = GRAD ? e / kTile : e % BK;
            const int64_t m = (int64_t)m0 + i, k = k0 + kk;
            T v = 0;
            if (m < m_end && k < k_end) v = GRAD ? A[k * p.lda + m] : A[m * p.lda + k];
            As[i * pitch + kk] = v;
        }
        for (int e = tid; e < kTile * BK; e += 256) {
            const int j = B_ROWS_K ? e % kTile : e / BK, kk = B_ROWS_K ? e / kTile : e % BK;
            const int64_t n = (int64_t)n0 + j, k = k0 + kk;
            T v = 0;
            if (n < p.N && k < k_end) v = B_ROWS_K ? B[k * p.ldb + n] : B[n * p.ldb + k];
            Bs[j * pitch + kk] = v;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kStepBytes / 32; ++s) {
            const char *a = lds + (wm + (lane & 31)) * kPitch + 32 * s + 16 * (lane >> 5);
            const char *b = lds + (kTile + wn + (lane & 31)) * kPitch + 32 * s + 16 * (lane >> 5);
            const u32x4 x = *reinterpret_cast<const u32x4 *>(a), y = *reinterpret_cast<const u32x4 *>(b);
            if constexpr (is_mx<E>) {
                const int64_t m = (int64_t)m0 + wm + (lane & 31), n = (int64_t)n0 + wn + (lane & 31);
                const int64_t block = k0 / 16 + 2 * s + (lane >> 5);  // of zeros from K on: scale 1
                const bool inside = 16 * block < k_end;
                const unsigned sa = inside && m < m_end ? p.mxa[m * p.ld_mxa + block] : 127u;
                const unsigned sb = inside && n < p.N ? p.mxb[g * p.stride_mxb + n * p.ld_mxb + block] : 127u;
                acc = E::template mma<32, 0, 0>(x, sa, y, sb, acc);
            } else {
                acc = E::template mma<32>(x, y, acc);
            }
        }
        __syncthreads();
    }

    // lane l holds column l % 32 and rows 8 (r / 4) + 4 (l / 32) + r % 4, r = 0..15
    typedef typename OutType<OUT>::T O;
    O *C = static_cast<O *>(p.C) + (GRAD ? g * p.stride_c : 0);
    const int64_t n = (int64_t)n0 + wn + (lane & 31);
    if (n >= p.N) return;
    float sb = 1.f;
    if constexpr (E::INT8) sb = p.sb[g * p.stride_sb + n];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t m = (int64_t)m0 + wm + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (m >= m_end) continue;
        float v = (float)acc[r];
        if constexpr (E::INT8) v = v * p.sa[m] * sb;
        C[m * p.ldc + n] = (O)v;
    }
}

template <class E, bool GRAD, bool B_ROWS_K>
hipError_t launch_any(const GroupArgs &a, hipStream_t stream)
{
    const int64_t tiles_n = ((int64_t)a.N + kTile - 1) / kTile;
    const int64_t tiles_m = GRAD ? ((int64_t)a.K + kTile - 1) / kTile * a.groups : max_row_tiles(a, kTile);
    if (tiles_m > INT64_MAX / 2 / tiles_n) return hipErrorInvalidConfiguration;
    unsigned gx, gy;
    if (!grid_for(tiles_m * tiles_n, gx, gy)) return hipErrorInvalidConfiguration;
    const void *fn[3] = {reinterpret_cast<const void *>(&group_any_kernel<E, 0, GRAD, B_ROWS_K>),
                         reinterpret_cast<const void *>(&group_any_kernel<E, 1, GRAD, B_ROWS_K>),
                         reinterpret_cast<const void *>(&group_any_kernel<E, 2, GRAD, B_ROWS_K>)};
    GroupArgs arg = a;
    void *args[] = {&arg};
    return hipLaunchKernel(fn[a.c_type], dim3(gx, gy), dim3(256), args, 0, stream);
}

}  // namespace

hipError_t group_any_launch(const GroupArgs &a, hipStream_t stream)
{
    if (a.grad)
        return a.elem == GroupElem::F16 ? launch_any<ElemF16, true, true>(a, stream)
                                        : launch_any<ElemBf16, true, true>(a, stream);
    if (a.elem == GroupElem::I8) return launch_any<ElemI8, false, false>(a, stream);
    if (a.elem == GroupElem::Mx4) return launch_any<ElemMx4, false, false>(a, stream);
    if (a.elem == GroupElem::F16)
        return a.trans_b ? launch_any<ElemF16, false, false>(a, stream) : launch_any<ElemF16, false, true>(a, stream);
    return a.trans_b ? launch_any<ElemBf16, false, false>(a, stream) : launch_any<ElemBf16, false, true>(a, stream);
}

// The kernels by number: one workgroup's rows and columns, and how many parts of k it sums side by side.
// "Row": one row of a group, in columns of 8 or 4 to a wave.
namespace {

constexpr const char *kNames[] = {
    "any 64x64",
    "row x16", "row x32",
    "rows 16x16", "rows 16x32", "rows 16x64", "rows 16x128",
    "rows 32x16", "rows 32x32", "rows 32x64", "rows 32x128",
    "rows 64x16", "rows 64x32", "rows 64x64", "rows 64x128",
    "tile 64x64 in 4", "tile 64x64 in 2", "tile 128x128", "tile 256x256",
};
constexpr int kConfigs = sizeof kNames / sizeof kNames[0];
constexpr int kAny = 0, kRow = 1, kRows = 3, kTiles = 15;

int rows_config(int rows, int cols)
{
    if (rows == 1) return kRow + (cols == 32);
    const int r = rows == 16 ? 0 : rows == 32 ? 1 : 2, c = cols == 16 ? 0 : cols == 32 ? 1 : cols == 64 ? 2 : 3;
    return kRows + 4 * r + c;
}

constexpr GroupTileKind kTileKinds[] = {GroupTileKind::Small4, GroupTileKind::Small, GroupTileKind::Mid, GroupTileKind::Large};

}  // namespace

int group_num_configs() { return kConfigs; }
const char *group_config_name(int cfg) { return cfg >= 0 && cfg < kConfigs ? kNames[cfg] : nullptr; }

// The kernel whose modelled time is least among those that take the shape.
int group_select(const GroupArgs &a)
{
    int best = kAny;
    double time = 1e300;
    constexpr int largest = 0x7fffffff - 1024;  // row and column numbers of a tile fit an int
    if (a.M > largest || a.N > largest || a.K > largest) return kAny;
    if (!a.grad)
        for (int r : {1, 16, 32, 64}) {
            if (!group_rows_ok(a, r)) continue;
            const double t = group_rows_time(a, r);
            if (t < time) best = rows_config(r, group_rows_columns(a, r)), time = t;
        }
    for (int k = 0; k < 4; ++k) {
        if (!group_tile_ok(a, kTileKinds[k])) continue;
        const double t = group_tile_time(a, kTileKinds[k]);
        if (t < time) best = kTiles + k, time = t;
    }
    return best;
}

hipError_t group_launch(const GroupArgs &a, hipStream_t stream)
{
    const int cfg = group_select(a);
    if (cfg == kAny) return group_any_launch(a, stream);
    if (cfg >= kTiles) return group_tile_launch(a, kTileKinds[cfg - kTiles], stream);
    return group_rows_launch(a, cfg < kRows ? 1 : 16 << (cfg - kRows) / 4, stream);
}

}  // namespace mm
