// mm_group_rows.hip -- grouped, 8-bit and 4-bit products with few rows per group (decoding):
// see mm_group.h for the sums.
//
// With up to 16 RB rows to a group the product is a stream of B: 2 (1) bytes of B for every
// 2 x rows FLOP. B goes from memory straight into the registers that feed the MFMA, no LDS and no
// barrier in the loop, so every wave keeps its own loads in flight; all waves of a workgroup share
// the columns, each takes every W-th slice of k, and at the end their partial sums are added in LDS
// in wave order. v_mfma_f32_16x16x32_* and v_mfma_i32_16x16x64_i8 take 64 bytes of k: lane l
// supplies the 16 bytes at k byte 16 (l / 16) of row (column) l % 16.
//
//   B rows along k (stored N x K): lane l reads the 16 bytes of its column itself: 16 columns x
//     128 bytes of k per slice.
//   B rows across k (stored K x N): lane l reads CPL columns of each of the 8 rows 8 (l / 16) .. + 7
//     of a slice of 32 k; 16 CPL columns in all. The MFMA for column CPL i + c wants those 8 rows of
//     one column: a pair of rows is one v_perm_b32, 4 CPL of them for the lane's 8 CPL values.
// A's rows come from L2 (every workgroup of a group reads the same rows); rows past the group's end
// repeat its last row and are not stored.
//
// Bound by the stream of B from memory: 13 experts of 4096 x 2048 bf16 K x N, 16 rows, cold: 38 us,
// 5.7 TB/s (through 128 x 128 tiles 43). The same stored N x K 46 us, 4.7 TB/s: the MFMA's 16 pieces of
// 64 bytes.
//
// With one row to a group and B's rows along k, whole rows of B (1 KB per wave and load) stream
// faster than the MFMA's 16 pieces of 64 bytes, and the vector units keep up: each wave takes J
// columns, multiplies its lanes' 16-byte pieces with A's by dot products (v_dot4_i32_i8, or fp32
// multiply-adds of the 16-bit values) and adds the 64 lanes' sums at the end (fixed order). Cold, i8
// 1 x 14336 x 4096: 15.6 us through the MFMA, 12.1 this way; 8 rows for 8 of 64 groups of 4096 x 2048:
// 13.8 and 13.2 (with 4 rows at a time, in registers for fewer waves, 14.4 and 17.4, so only for one);
// the latter in bf16 23.5 us, 5.7 TB/s. Rows of one group each read its matrix, all but the first from
// L2 where they run side by side, so the choice takes this kernel for about one row to a group only.
//
// 4-bit blocks come as bytes of two codes, 16 to a block; their scales, 8 bytes a slice of a row, go
// straight into registers too, and a lane's byte for either MFMA step is picked by v_perm_b32. Cold, 1 x 4096
// x 4096: 4.7 us (64 x 64 tiles 5.1).
#include "mm_group.h"

namespace mm {
namespace {

// load16 for data read once (not kept in the caches).
__device__ __forceinline__ u32x4 load16_once(const char *p)
{
    typedef unsigned int Words __attribute__((ext_vector_type(4), aligned(1)));
    return __builtin_nontemporal_load(reinterpret_cast<const Words *>(p));
}

// Partial sums of the W waves added in wave order and stored. `mine` holds NC x 4 values per lane:
// value (c, r) is row 4 (lane / 16) + r, column COLS_C * (lane % 16) + c  (columns 16 c + lane % 16
// where COLS_C is 0).
template <class E, int W, int NC, int COLS_C>
__device__ __forceinline__ void join_and_store(const GroupArgs &p, const typename E::template Acc<16> (&mine)[NC], char *lds, int g,
                                               int row0, int row_end, int n0)
{
    typedef decltype(mine[0][0] + 0) V;
    V *part = reinterpret_cast<V *>(lds);  // [wave][row][column]
    constexpr int COLS = 16 * NC;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int col = COLS_C ? COLS_C * (lane & 15) + c : 16 * c + (lane & 15);
            part[(w * 16 + 4 * (lane >> 4) + r) * COLS + col] = mine[c][r];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * COLS; e += 64 * W) {
        const int row = row0 + e / COLS;
        const int64_t n = (int64_t)n0 + e % COLS;
        if (row >= row_end || n >= p.N) continue;
        V sum = part[e];
#pragma unroll
        for (int i = 1; i < W; ++i) sum += part[i * 16 * COLS + e];
        float v = (float)sum;
        if constexpr (E::INT8) v = v * p.sa[row] * p.sb[(int64_t)g * p.stride_sb + n];
        const int64_t at = (int64_t)row * p.ldc + n;
        if (p.c_type == 0) static_cast<float *>(p.C)[at] = v;
        else if (p.c_type == 1) static_cast<__bf16 *>(p.C)[at] = (__bf16)v;
        else static_cast<_Float16 *>(p.C)[at] = (_Float16)v;
    }
    __syncthreads();
}

// The workgroup's row tile (16 RB rows of a group) and strip of columns; false: none.
template <int ROWS>
__device__ __forceinline__ bool rows_tile(const GroupArgs &p, int cols, RowTile &t, int &n0)
{
    const unsigned strips = (unsigned)(((int64_t)p.N + cols - 1) / cols);
    const int64_t bid = linear_block();
    const int64_t rt = bid / strips;
    if (rt > 0x7fffffff || !RowTiles<ROWS>(p).find(p, (unsigned)rt, t)) return false;
    n0 = (int)((unsigned)(bid - rt * strips) * (unsigned)cols);
    t.g = __builtin_amdgcn_readfirstlane(t.g);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.hi = __builtin_amdgcn_readfirstlane(t.hi);
    return true;
}

// 8 scale bytes from any address.
__device__ __forceinline__ u32x2 load8(const unsigned char *p)
{
    struct __attribute__((packed)) Bytes {
        u32x2 v;
    };
    return reinterpret_cast<const Bytes *>(p)->v;
}

// B rows along k. W waves, 16 NB columns, slices of 128 bytes of k, J of them in flight.
template <class E, int RB, int NB, int W, int J>
__global__ __launch_bounds__(64 * W) void rows_kernel_d(GroupArgs p)
{
    typedef typename E::T T;
    __shared__ __attribute__((aligned(16))) char lds[W * 16 * 16 * NB * 4];
    RowTile t;
    int n0;
    if (!rows_tile<16 * RB>(p, 16 * NB, t, n0)) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t kb = (int64_t)p.K * sizeof(T);  // bytes along k
    const char *a[RB], *b[NB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
        a[i] = static_cast<const char *>(p.A) +
               (int64_t)min(t.row0 + 16 * i + (lane & 15), t.hi - 1) * p.lda * (int)sizeof(T) + 16 * (lane >> 4);
#pragma unroll
    for (int j = 0; j < NB; ++j)
        b[j] = static_cast<const char *>(p.B) +
               (t.g * p.stride_b + min((int64_t)n0 + 16 * j + (lane & 15), (int64_t)p.N - 1) * p.ldb) * (int)sizeof(T) +
               16 * (lane >> 4);
    typename E::template Acc<16> acc[RB][NB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = typename E::template Acc<16>{0, 0, 0, 0};
    // Mx4: a slice's 8 scale bytes of the same rows and columns; this lane's are number lane / 16 and 4 on
    const unsigned char *sa[RB], *sb[NB];
    const unsigned pick = (unsigned)(lane >> 4) * 0x0101u | 0x0c0c0400u;
    if constexpr (is_mx<E>) {
#pragma unroll
        for (int i = 0; i < RB; ++i) sa[i] = p.mxa + (int64_t)min(t.row0 + 16 * i + (lane & 15), t.hi - 1) * p.ld_mxa;
#pragma unroll
        for (int j = 0; j < NB; ++j)
            sb[j] = p.mxb + t.g * p.stride_mxb + min((int64_t)n0 + 16 * j + (lane & 15), (int64_t)p.N - 1) * p.ld_mxb;
    }
    // MFMA step h of a slice
    auto mma = [&](auto h, u32x4 x, unsigned sx, u32x4 y, unsigned sy, typename E::template Acc<16> c) {
        if constexpr (is_mx<E>) return E::template mma<16, decltype(h)::value, decltype(h)::value>(x, sx, y, sy, c);
        else return E::template mma<16>(x, y, c);
    };
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;

    const int64_t whole = kb / 128;  // whole slices; wave w takes w, w + W, ...
    u32x4 av[J][2][RB], bv[J][2][NB];
    u32x2 as[J][RB] = {}, bs[J][NB] = {};
    int64_t s = w;
    auto load = [&](int x, int64_t slice) {
        if constexpr (is_mx<E>) {
#pragma unroll
            for (int j = 0; j < NB; ++j) bs[x][j] = load8(sb[j] + slice * 8);
#pragma unroll
            for (int i = 0; i < RB; ++i) as[x][i] = load8(sa[i] + slice * 8);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < NB; ++j) bv[x][h][j] = load16(b[j] + slice * 128 + 64 * h);
#pragma unroll
            for (int i = 0; i < RB; ++i) av[x][h][i] = load16(a[i] + slice * 128 + 64 * h);
        }
    };
    auto multiply = [&](int x) {
        unsigned p[RB] = {}, q[NB] = {};
        if constexpr (is_mx<E>) {
#pragma unroll
            for (int i = 0; i < RB; ++i) p[i] = __builtin_amdgcn_perm(as[x][i][1], as[x][i][0], pick);
#pragma unroll
            for (int j = 0; j < NB; ++j) q[j] = __builtin_amdgcn_perm(bs[x][j][1], bs[x][j][0], pick);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = mma(H0(), av[x][0][i], p[i], bv[x][0][j], q[j], acc[i][j]);
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = mma(H1(), av[x][1][i], p[i], bv[x][1][j], q[j], acc[i][j]);
    };
    // J slices loaded ahead; a slice is multiplied, then its registers take the slice J further on
    if (whole > 0) {
#pragma unroll
        for (int x = 0; x < J; ++x) load(x, min(s + (int64_t)x * W, whole - 1));
        while (s < whole) {
#pragma unroll
            for (int x = 0; x < J; ++x) {
                if (s < whole) multiply(x);
                if (s + (int64_t)J * W < whole) load(x, s + (int64_t)J * W);
                s += W;
            }
        }
    }
    if (kb % 128 != 0 && whole % W == w) {  // the partial slice
        const int64_t at = whole * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int valid = (int)(kb - at) - 64 * h - 16 * (lane >> 4);
            u32x4 aa[RB];
            unsigned p[RB] = {}, q = 0;  // Mx4: of a block, 16 bytes; past the last zeros of scale 1
            const int64_t block = whole * 8 + 4 * h + (lane >> 4);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                aa[i] = load16_upto<T>(a[i] + at + 64 * h, valid, kb);
                if constexpr (is_mx<E>) p[i] = valid > 0 ? sa[i][block] : 127u;
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const u32x4 bb = load16_upto<T>(b[j] + at + 64 * h, valid, kb);
                if constexpr (is_mx<E>) q = valid > 0 ? sb[j][block] : 127u;
#pragma unroll
                for (int i = 0; i < RB; ++i) acc[i][j] = mma(H0(), aa[i], p[i], bb, q, acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
        join_and_store<E, W, NB, 0>(p, acc[i], lds, t.g, t.row0 + 16 * i, t.hi, n0);
}

// The CPL 16-bit values at p (any 2-byte alignment) in CPL / 2 words. They are read once, so not kept
// in the caches (13 experts of 4096 x 2048 bf16: 46.9 -> 41.7 us; the other layout, whose two loads
// share a cache line, loses by it).
template <int CPL>
__device__ __forceinline__ void load_columns(const char *p, unsigned (&v)[CPL / 2])
{
    typedef unsigned Words __attribute__((ext_vector_type(CPL / 2), aligned(2)));
    if constexpr (CPL == 2) {
        typedef unsigned One __attribute__((aligned(2)));
        v[0] = __builtin_nontemporal_load(reinterpret_cast<const One *>(p));
    } else {
        const Words x = __builtin_nontemporal_load(reinterpret_cast<const Words *>(p));
#pragma unroll
        for (int i = 0; i < CPL / 2; ++i) v[i] = x[i];
    }
}
// The last `cols` of them, moved to the front: value e becomes value e - (CPL - cols).
template <int CPL>
__device__ __forceinline__ void drop_columns(unsigned (&v)[CPL / 2], int cols)
{
    const int sh = 16 * (CPL - cols);
    if constexpr (CPL == 2) {
        v[0] >>= sh;
    } else if constexpr (CPL == 4) {
        const uint64_t x = (v[0] | (uint64_t)v[1] << 32) >> sh;
        v[0] = (unsigned)x;
        v[1] = (unsigned)(x >> 32);
    } else {
        const u32x4 x = __builtin_bit_cast(
            u32x4, __builtin_bit_cast(unsigned __int128, u32x4{v[0], v[1], v[2], v[3]}) >> sh);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = x[i];
    }
}

// B rows across k (16-bit elements). W waves, 16 CPL columns, slices of 32 k, J of them in flight.
template <class E, int RB, int CPL, int W, int J>
__global__ __launch_bounds__(64 * W) void rows_kernel_t(GroupArgs p)
{
    typedef typename E::T T;
    __shared__ __attribute__((aligned(16))) char lds[W * 16 * 16 * CPL * 4];
    RowTile t;
    int n0;
    if (!rows_tile<16 * RB>(p, 16 * CPL, t, n0)) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const T *a[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
        a[i] = static_cast<const T *>(p.A) + (int64_t)min(t.row0 + 16 * i + (lane & 15), t.hi - 1) * p.lda +
               8 * (lane >> 4);
    const int64_t col = (int64_t)n0 + CPL * (lane & 15);
    // a lane whose columns cross N reads the last CPL of the row and drops those before its own;
    // one past N reads them too, for columns that are not stored. N >= CPL.
    const bool full = (int64_t)n0 + 16 * CPL <= p.N;  // the strip's columns all exist
    const int cols = (int)(p.N - col < CPL && p.N > col ? p.N - col : CPL);
    const T *b = static_cast<const T *>(p.B) + t.g * p.stride_b + (int64_t)(8 * (lane >> 4)) * p.ldb +
                 min(col, (int64_t)p.N - CPL);
    typename E::template Acc<16> acc[RB][CPL];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int c = 0; c < CPL; ++c) acc[i][c] = typename E::template Acc<16>{0, 0, 0, 0};

    u32x4 av[J][RB];
    unsigned bv[J][8][CPL / 2];
    auto load = [&](int x, int slice) {
        const int64_t k0 = (int64_t)slice * 32;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            load_columns<CPL>(reinterpret_cast<const char *>(b + (k0 + r) * p.ldb), bv[x][r]);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) av[x][i] = load16(reinterpret_cast<const char *>(a[i] + k0));
    };
    auto multiply = [&](const u32x4 (&aa)[RB], unsigned (&bb)[8][CPL / 2]) {
        if (!full) {
#pragma unroll
            for (int r = 0; r < 8; ++r) drop_columns<CPL>(bb[r], cols);
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            u32x4 o;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o[q] = __builtin_amdgcn_perm(bb[2 * q + 1][c >> 1], bb[2 * q][c >> 1],
                                             (c & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int i = 0; i < RB; ++i) acc[i][c] = E::template mma<16>(aa[i], o, acc[i][c]);
        }
    };
    const int whole = p.K / 32;
    if (whole > 0) {
        int s = w;
#pragma unroll
        for (int x = 0; x < J; ++x) load(x, min(s + x * W, whole - 1));
        while (s < whole) {
#pragma unroll
            for (int x = 0; x < J; ++x) {
                if (s < whole) multiply(av[x], bv[x]);
                if (s < whole - J * W) load(x, s + J * W);
                s += W;
            }
        }
    }
    if (p.K % 32 != 0 && whole % W == w) {  // the partial slice
        const int64_t k0 = (int64_t)whole * 32;
        const int left = p.K - whole * 32 - 8 * (lane >> 4);  // of this lane's 8 k
        u32x4 aa[RB];
        unsigned bb[8][CPL / 2];
#pragma unroll
        for (int r = 0; r < 8; ++r) {  // rows from K on: row K - 1 read, zeros used
            load_columns<CPL>(reinterpret_cast<const char *>(b + (k0 + min(r, left - 1)) * p.ldb), bb[r]);
#pragma unroll
            for (int i = 0; i < CPL / 2; ++i) bb[r][i] = r < left ? bb[r][i] : 0u;
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
            aa[i] = load16_upto<T>(reinterpret_cast<const char *>(a[i] + k0), 2 * left, 2 * (int64_t)p.K);
        multiply(aa, bb);
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
        join_and_store<E, W, CPL, CPL>(p, acc[i], lds, t.g, t.row0 + 16 * i, t.hi, n0);
}

// acc + the products of the 16 bytes x and y.
template <class E>
__device__ __forceinline__ auto dot16(u32x4 x, u32x4 y, decltype(typename E::template Acc<16>()[0] + 0) acc)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const unsigned a = x[q], b = y[q];
        if constexpr (E::INT8) {
            acc = __builtin_amdgcn_sdot4((int)a, (int)b, acc, false);
        } else if constexpr (std::is_same_v<E, ElemBf16>) {
            acc = fmaf(__builtin_bit_cast(float, a << 16), __builtin_bit_cast(float, b << 16), acc);
            acc = fmaf(__builtin_bit_cast(float, a & 0xffff0000u), __builtin_bit_cast(float, b & 0xffff0000u), acc);
        } else {
            typedef _Float16 h2 __attribute__((ext_vector_type(2)));
            const h2 u = __builtin_bit_cast(h2, a), v = __builtin_bit_cast(h2, b);
            acc = fmaf((float)u[0], (float)v[0], acc);
            acc = fmaf((float)u[1], (float)v[1], acc);
        }
    }
    return acc;
}

// Sum over the lanes, in lane 63 (rows of 16 lanes first, then the rows' sums).
template <class V>
__device__ __forceinline__ V wave_sum(V v)
{
    auto step = [&](auto ctrl, auto rows) {
        v += __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value,
                                                               decltype(rows)::value, 0xf, false));
    };
    step(std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());  // row_shr 1, 2, 4, 8
    step(std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());  // row_bcast 15
    step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());  // row_bcast 31
    return v;
}

// B rows along k, one row of A per workgroup, 4 waves of J columns each, U KB of k at a time.
template <class E, int J, int U>
__global__ __launch_bounds__(256) void rows_kernel_dot(GroupArgs p)
{
    typedef typename E::T T;
    typedef decltype(typename E::template Acc<16>()[0] + 0) V;
    RowTile t;
    int n0;
    if (!rows_tile<1>(p, 4 * J, t, n0)) return;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t col0 = (int64_t)n0 + J * w;
    if (col0 >= p.N) return;  // a whole wave; there is no barrier
    const int64_t kb = (int64_t)p.K * sizeof(T);  // bytes along k
    const char *a = static_cast<const char *>(p.A) + (int64_t)t.row0 * p.lda * (int)sizeof(T) + 16 * lane, *b[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
        b[j] = static_cast<const char *>(p.B) +
               (t.g * p.stride_b + min(col0 + j, (int64_t)p.N - 1) * p.ldb) * (int)sizeof(T) + 16 * lane;
    V acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = 0;

    for (int64_t k0 = 0; k0 < kb; k0 += 1024 * U) {
        u32x4 av[U], bv[J][U];
        if (k0 + 1024 * U <= kb) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < J; ++j) bv[j][u] = load16_once(b[j] + k0 + 1024 * u);
#pragma unroll
            for (int u = 0; u < U; ++u) av[u] = load16(a + k0 + 1024 * u);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int valid = (int)(kb - k0) - 1024 * u - 16 * lane;
#pragma unroll
                for (int j = 0; j < J; ++j) bv[j][u] = load16_upto<T>(b[j] + k0 + 1024 * u, valid, kb);
                av[u] = load16_upto<T>(a + k0 + 1024 * u, valid, kb);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < J; ++j) acc[j] = dot16<E>(av[u], bv[j][u], acc[j]);
    }
    // lane j < J stores column col0 + j
    const int64_t n = col0 + lane;
    const bool live = lane < J && n < p.N;
    V mine = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int sum = __builtin_amdgcn_readlane(__builtin_bit_cast(int, wave_sum(acc[j])), 63);
        if (lane == j) mine = __builtin_bit_cast(V, sum);
    }
    if (!live) return;
    float v = (float)mine;
    if constexpr (E::INT8) v = v * p.sa[t.row0] * p.sb[(int64_t)t.g * p.stride_sb + n];
    const int64_t at = (int64_t)t.row0 * p.ldc + n;
    if (p.c_type == 0) static_cast<float *>(p.C)[at] = v;
    else if (p.c_type == 1) static_cast<__bf16 *>(p.C)[at] = (__bf16)v;
    else static_cast<_Float16 *>(p.C)[at] = (_Float16)v;
}

template <int ROWS>
hipError_t launch_rows(const void *fn, const GroupArgs &a, int cols, int waves, hipStream_t stream)
{
    const int64_t strips = ((int64_t)a.N + cols - 1) / cols, tiles = max_row_tiles(a, ROWS);
    if (tiles > INT64_MAX / strips) return hipErrorInvalidConfiguration;
    unsigned gx, gy;
    if (!grid_for(tiles * strips, gx, gy)) return hipErrorInvalidConfiguration;
    GroupArgs arg = a;
    void *args[] = {&arg};
    return hipLaunchKernel(fn, dim3(gx, gy), dim3(64 * waves), args, 0, stream);
}

template <class E, int RB, int NB, int W, int J>
hipError_t launch_d(const GroupArgs &a, hipStream_t stream)
{
    return launch_rows<16 * RB>(reinterpret_cast<const void *>(&rows_kernel_d<E, RB, NB, W, J>), a, 16 * NB, W, stream);
}

template <class E, int RB, int CPL, int W, int J>
hipError_t launch_t(const GroupArgs &a, hipStream_t stream)
{
    return launch_rows<16 * RB>(reinterpret_cast<const void *>(&rows_kernel_t<E, RB, CPL, W, J>), a, 16 * CPL, W, stream);
}

// Columns per workgroup: with many workgroups wide strips, which read A's rows less often; with few
// narrow ones, since one workgroup streams no more than about 40 GB/s. Measured at 16 rows: i8, 16
// groups of 4096 x 2048 38 us in strips of 16, 31 in strips of 32; one of 4096 x 4096 7.1 and 9.0.
// One row: 4 waves of 4 columns of 4 KB, or 8 of 2 KB of short 8-bit rows: 16 KB requested at once.
int strip_columns(const GroupArgs &a, int rows)
{
    if (rows == 1) return a.elem == GroupElem::I8 && a.K <= 2048 ? 32 : 16;
    const double tiles = expected_row_tiles(a, rows);
    if (a.trans_b) return tiles * ((a.N + 31) / 32) >= 768 ? 32 : 16;
    const double wide = tiles * ((a.N + 127) / 128);
    if (a.N < 4 || (rows <= 32 && wide < 64)) return 32;
    return a.N >= 8 && wide >= 192 ? 128 : 64;
}

template <class E>
hipError_t rows_dot(const GroupArgs &a, hipStream_t stream)
{
    if constexpr (E::INT8)
        if (strip_columns(a, 1) == 32)
            return launch_rows<1>(reinterpret_cast<const void *>(&rows_kernel_dot<E, 8, 2>), a, 32, 4, stream);
    return launch_rows<1>(reinterpret_cast<const void *>(&rows_kernel_dot<E, 4, 4>), a, 16, 4, stream);
}

template <class E>
hipError_t rows_d(const GroupArgs &a, int rows, hipStream_t stream)
{
    if constexpr (!is_mx<E>)
        if (rows == 1) return rows_dot<E>(a, stream);
    const bool wide = strip_columns(a, rows) == 32;
    if (rows == 16) return wide ? launch_d<E, 1, 2, 4, 2>(a, stream) : launch_d<E, 1, 1, 4, 4>(a, stream);
    if (rows == 32) return wide ? launch_d<E, 2, 2, 4, 2>(a, stream) : launch_d<E, 2, 1, 4, 4>(a, stream);
    return wide ? launch_d<E, 4, 2, 4, 2>(a, stream) : launch_d<E, 4, 1, 4, 2>(a, stream);
}

template <class E>
hipError_t rows_t(const GroupArgs &a, int rows, hipStream_t stream)
{
    const int cols = strip_columns(a, rows);
    if (rows == 16)
        return cols == 128  ? launch_t<E, 1, 8, 8, 1>(a, stream)
               : cols == 64 ? launch_t<E, 1, 4, 8, 4>(a, stream)
                            : launch_t<E, 1, 2, 8, 6>(a, stream);
    if (rows == 32)
        return cols == 128  ? launch_t<E, 2, 8, 8, 2>(a, stream)
               : cols == 64 ? launch_t<E, 2, 4, 8, 2>(a, stream)
                            : launch_t<E, 2, 2, 8, 4>(a, stream);
    return cols == 128 ? launch_t<E, 4, 8, 8, 1>(a, stream) : launch_t<E, 4, 4, 8, 2>(a, stream);
}

}  // namespace

bool group_rows_ok(const GroupArgs &a, int rows)
{
    // One row at a time: about one row to a group, since each row reads its matrix (one that several
    // rows share comes from L2 again), and of 8-bit elements 1 KB of it, of 16-bit ones more than 2.
    // Against the other kernels, cold, rows at random: 8-bit 0.6-1.2 times their time (5 rows, 27 groups
    // of 8496 x 6448: 45 us and 54); 16-bit 0.55-1.3 (one row of 6880 x 6064: 18 us and 32), up to 2 KB
    // 0.8-1.6 (2 rows, 3 groups of 2173 x 900: 8.6 us and 5.4), most of it in partial loads. 4-bit rows
    // never: unpacking and scaling them by vector instructions (8 rows for 8 of 64 groups of 4096 x 2048: 17
    // us, 10 through the MFMA).
    if (rows == 1)
        return a.trans_b && a.elem != GroupElem::Mx4 && a.M <= 1.25 * expected_groups(a) &&
               a.K >= (a.elem == GroupElem::I8 ? 1024 : 1025);
    return a.trans_b || a.N >= (rows == 64 ? 4 : 2);  // a lane's columns of B rows across k
}

// Fitted to some 200 shapes of all operators: a launch and one workgroup's start 4.5 us; the
// right-hand matrices from memory at 5.4 TB/s; what is read again, through L2, at 9 TB/s (5 with B's
// rows across k); 40 (24) GB/s per workgroup where they are few; and rounds of workgroups, each at least
// its latency and its sums' join.
double group_rows_time(const GroupArgs &a, int rows)
{
    const int es = group_elem_size(a);
    const double unaligned = aligned_words(a) ? 1.0 : 2.2;
    if (rows == 1) return 3.5 + a.M * (double)a.N * a.K * es / 5.8e6 * unaligned;
    const int cols = strip_columns(a, rows), rb = rows / 16;
    const double tiles = expected_row_tiles(a, rows) * (double)(((int64_t)a.N + cols - 1) / cols);
    const double mean = a.M / expected_groups(a), weights = expected_weight_bytes(a);
    const double bytes = tiles * (fmin(rows, mean) + cols) * (double)a.K * es;  // rows past a group's end are one row
    const double again = fmax(0.0, bytes - weights) / (a.trans_b ? 9e6 : 5e6);
    const double rate = !a.trans_b && cols == 32 ? 2.4e4 : 4e4;  // of one workgroup; 64-byte rows of B: less
    const double stream = fmax(weights / 5.4e6 + again, bytes / (rate * tiles)) * unaligned;
    const double rounds = a.trans_b ? ceil(tiles / 768) * (1.2 + 0.4 * rb) : ceil(tiles / 256) * (2 + 1.25 * rb);
    return 2.5 + fmax(2 + stream, rounds);
}

int group_rows_columns(const GroupArgs &a, int rows) { return strip_columns(a, rows); }

hipError_t group_rows_launch(const GroupArgs &a, int rows, hipStream_t stream)
{
    if (a.elem == GroupElem::I8) return rows_d<ElemI8>(a, rows, stream);
    if (a.elem == GroupElem::Mx4) return rows_d<ElemMx4>(a, rows, stream);
    if (a.trans_b)
        return a.elem == GroupElem::F16 ? rows_d<ElemF16>(a, rows, stream) : rows_d<ElemBf16>(a, rows, stream);
    return a.elem == GroupElem::F16 ? rows_t<ElemF16>(a, rows, stream) : rows_t<ElemBf16>(a, rows, stream);
}

}  // namespace mm
