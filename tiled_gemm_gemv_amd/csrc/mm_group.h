// mm_group.h -- shared by the kernels of the grouped products and of the 8-bit integer and
// 4-bit products (mm_group_tile.hip, mm_group_rows.hip, mm_group_any.hip): element types, loads of any
// alignment, the map from a workgroup to a tile of a group, and what the host expects of group
// sizes that it does not know.
//
// The sums. Rows lo_g <= i < hi_g of A (lo_g = offsets[g], hi_g = offsets[g + 1]) belong to
// group g:
//   rows mode      C[i][j] = s(i, j) sum over k < K of A[i][k] B_g(k, j)
//                  s = 1 for 16-bit elements, sa[i] sb_g[j] for 8-bit integers;
//                  B_g(k, j) = B[g stride_b + k ldb + j] or, "transposed",
//                  B[g stride_b + j ldb + k]; 4-bit elements come in blocks of 32 along k
//                  with a scale each, for A and B
//   gradient mode  C_g[p][j] = sum over lo_g <= i < hi_g of A[i][p] B[i][j]
//
// The offsets live in device memory and no host code reads them: the grid covers the most
// tiles that M rows in `groups` groups can need, and each workgroup finds its own tile. They
// are clamped to [0, M], and a group whose end is not above its start is empty, so whatever
// they hold no kernel leaves the rows of A and C.
#pragma once

#include <math.h>

#include <type_traits>

#include "mm_internal.h"

namespace mm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// An element type: its storage, and the MFMAs that multiply B = 32 rows by 32 columns over 32 bytes
// of k, or B = 16 by 16 over 64 bytes: lane l supplies the 16 bytes at k byte 16 (l / B) of row
// (column) l % B. Acc<B>: a lane's values of the block, of column l % B: rows 8 (r / 4) + 4 (l / 32)
// + r % 4, r < 16, for B = 32; rows 4 (l / 16) + r, r < 4, for B = 16.
template <int B, class V4, class V16>
using BlockAcc = std::conditional_t<B == 32, V16, V4>;

struct ElemBf16 {
    typedef unsigned short T;
    static constexpr bool INT8 = false;
    template <int B>
    using Acc = BlockAcc<B, f32x4, f32x16>;
    template <int B>
    static __device__ __forceinline__ Acc<B> mma(u32x4 a, u32x4 b, Acc<B> c)
    {
        const bf16x8 x = __builtin_bit_cast(bf16x8, a), y = __builtin_bit_cast(bf16x8, b);
        if constexpr (B == 32) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, c, 0, 0, 0);
        else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
    }
};
struct ElemF16 {
    typedef unsigned short T;
    static constexpr bool INT8 = false;
    template <int B>
    using Acc = BlockAcc<B, f32x4, f32x16>;
    template <int B>
    static __device__ __forceinline__ Acc<B> mma(u32x4 a, u32x4 b, Acc<B> c)
    {
        const f16x8 x = __builtin_bit_cast(f16x8, a), y = __builtin_bit_cast(f16x8, b);
        if constexpr (B == 32) return __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, c, 0, 0, 0);
        else return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
    }
};
// Sums of 8-bit products are exact in 32 bits: |sum| <= 2^14 K, and the host admits
// K <= 2^17 - 1.
struct ElemI8 {
    typedef signed char T;
    static constexpr bool INT8 = true;
    template <int B>
    using Acc = BlockAcc<B, i32x4, i32x16>;
    template <int B>
    static __device__ __forceinline__ Acc<B> mma(u32x4 a, u32x4 b, Acc<B> c)
    {
        const i32x4 x = __builtin_bit_cast(i32x4, a), y = __builtin_bit_cast(i32x4, b);
        if constexpr (B == 32) return __builtin_amdgcn_mfma_i32_32x32x32_i8(x, y, c, 0, 0, 0);
        else return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
    }
};

// 4-bit floating point in blocks of 32 along k with a power of two each: K counts bytes here, two
// elements to a byte, so that a block is 16 bytes of k, one lane's part of an MFMA operand, and
// everything that moves bytes is the 8-bit product's. The MFMA multiplies lane l's products by
// 2^(x - 127) 2^(y - 127), x and y the scale bytes number SA and SB of that lane's words sa and sb
// (255: NaN). Products are exact in fp32.
struct ElemMx4 {
    typedef unsigned char T;
    static constexpr bool INT8 = false;
    template <int B>
    using Acc = BlockAcc<B, f32x4, f32x16>;
    template <int B, int SA, int SB>
    static __device__ __forceinline__ Acc<B> mma(u32x4 a, unsigned sa, u32x4 b, unsigned sb, Acc<B> c)
    {
        typedef int i32x8 __attribute__((ext_vector_type(8)));  // the builtin's operand; 4-bit formats take half of it
        const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
        const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
        constexpr int fp4 = 4;  // the format's number
        if constexpr (B == 32)
            return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, fp4, fp4, SA, (int)sa, SB, (int)sb);
        else return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, fp4, fp4, SA, (int)sa, SB, (int)sb);
    }
};
template <class E>
constexpr bool is_mx = std::is_same_v<E, ElemMx4>;

// Output types (the public MM_TYPE_* values). fp32 sums are rounded once, to nearest even.
template <int OUT>
struct OutType;
template <>
struct OutType<0> {
    typedef float T;
};
template <>
struct OutType<1> {
    typedef __bf16 T;
};
template <>
struct OutType<2> {
    typedef _Float16 T;
};

// 16 bytes from any address (the device's unaligned access mode serves them)
__device__ __forceinline__ u32x4 load16(const char *p)
{
    struct __attribute__((packed)) Bytes {
        u32x4 v;
    };
    return reinterpret_cast<const Bytes *>(p)->v;
}

// The first `valid` bytes (a multiple of the element size) at p, zeros after; nothing past them is
// read. `row`: bytes from the start of p's row to the end of those bytes; with 16 or more the 16
// bytes that end there are read and shifted down, with fewer single elements.
template <class Elem>
__device__ __forceinline__ u32x4 load16_upto(const char *p, int valid, int64_t row)
{
    if (valid >= 16) return load16(p);
    u32x4 v = {0u, 0u, 0u, 0u};
    if (valid <= 0) return v;
    constexpr int es = sizeof(Elem);
    if (row >= 16) {
        const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, load16(p + valid - 16)) >> (8 * (16 - valid));
        return __builtin_bit_cast(u32x4, x);
    }
#pragma unroll
    for (int e = 0; e < 16 / es; ++e)
        if (e * es < valid) {
            const unsigned x = es == 1   ? (unsigned)*reinterpret_cast<const unsigned char *>(p + e)
                               : es == 2 ? (unsigned)*reinterpret_cast<const unsigned short *>(p + 2 * e)
                                         : *reinterpret_cast<const unsigned *>(p + 4 * e);
            v[e * es / 4] |= x << (8 * (e * es % 4));
        }
    return v;
}

// lo and hi of group g, clamped to [0, M].
__device__ __forceinline__ void group_range(const int64_t *offsets, int g, int M, int &lo, int &hi)
{
    const int64_t a = offsets[g], b = offsets[g + 1];
    lo = (int)(a < 0 ? 0 : a > M ? M : a);
    hi = (int)(b < 0 ? 0 : b > M ? M : b);
    if (hi < lo) hi = lo;
}

// Sum over the lanes up to this one: within rows of 16 lanes, then the rows' sums.
__device__ __forceinline__ unsigned wave_inclusive_sum(unsigned v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15: to rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31: to rows 2 and 3
    return v;
}

// A row tile of a group: rows row0 <= i < min(row0 + BM, hi) of group g.
struct RowTile {
    int g, row0, hi;
};

// The groups' BM-row tiles, numbered in group order, and where a tile is. Every wave of a workgroup
// builds it for itself (all values wave-uniform but `run`, `incl`, `lo`, `hi`): lane l counts the
// tiles of groups l R .. l R + R - 1, R = ceil(groups / 64), and a scan over the lanes gives the
// rest; up to 64 groups (R = 1) the lane keeps its group's range.
template <int BM>
struct RowTiles {
    unsigned total;       // tiles in all
    unsigned run, incl;   // tiles of this lane's groups, and of the lanes up to it
    int R, lo, hi;

    static __device__ __forceinline__ unsigned count(int lo, int hi)
    {
        return ((unsigned)(hi - lo) + (BM - 1)) / BM;  // not as int: up to 2^31 - 1 rows
    }

    __device__ __forceinline__ RowTiles(const GroupArgs &p)
    {
        if (!p.offsets) {
            total = count(0, p.M);
            return;
        }
        const int lane = threadIdx.x & 63;
        R = (p.groups + 63) / 64;
        run = 0;
        lo = hi = 0;
        for (int g = lane * R; g < min(lane * R + R, p.groups); ++g) {
            group_range(p.offsets, g, p.M, lo, hi);
            run += count(lo, hi);
        }
        incl = wave_inclusive_sum(run);
        total = __builtin_amdgcn_readlane(incl, 63);
    }

    // Tile number rt. False if there is none; never for rt < total of offsets that do not decrease.
    // Others may count more tiles than 32 bits hold: the rows returned are the group's all the same.
    __device__ __forceinline__ bool find(const GroupArgs &p, unsigned rt, RowTile &t) const
    {
        if (!p.offsets) {
            t.g = 0;
            t.row0 = (int)rt * BM;
            t.hi = p.M;
            return (int64_t)rt * BM < p.M;
        }
        unsigned long long above = __ballot(incl > rt);
        if (!above) return false;
        int l = __ffsll(above) - 1;
        unsigned first = __builtin_amdgcn_readlane(incl - run, l);  // the run's first tile
        int from = lo, to = hi;
        t.g = l;
        if (R > 1) {  // the run's groups, one per lane (R <= 64)
            const int i = threadIdx.x & 63, g = l * R + i;
            from = to = 0;
            if (i < R && g < p.groups) group_range(p.offsets, g, p.M, from, to);
            const unsigned c = count(from, to), upto = first + wave_inclusive_sum(c);
            above = __ballot(upto > rt);
            if (!above) return false;
            const int run0 = l * R;
            l = __ffsll(above) - 1;
            first = __builtin_amdgcn_readlane(upto - c, l);
            t.g = run0 + l;
        }
        t.hi = __builtin_amdgcn_readlane(to, l);
        const int64_t row0 = __builtin_amdgcn_readlane(from, l) + (int64_t)(rt - first) * BM;
        t.row0 = (int)row0;
        return rt >= first && row0 < t.hi;
    }
};

// What the host expects of group sizes that it does not know, for the choice of a kernel: groups
// with a row, BM-row tiles (a group's last tile half full on average), and the bytes of the
// right-hand matrices that are read. Rows fall into the groups at random: one of G groups stays empty
// with probability (1 - 1/G)^M, M >= 1 rows, so G (1 - (1 - 1/G)^M) have rows: 1 where M or G is 1.
inline double expected_groups(const GroupArgs &a)
{
    if (!a.offsets || a.groups == 1) return 1;
    return a.groups * -expm1(a.M * log1p(-1.0 / a.groups));
}
inline double expected_row_tiles(const GroupArgs &a, int bm)
{
    const double groups = expected_groups(a), mean = a.M / groups;
    if (!a.offsets || a.groups == 1 || bm == 1) return (double)(((int64_t)a.M + bm - 1) / bm);
    return groups * (mean > bm / 2 ? mean / bm + 0.5 : 1.0);
}
inline double expected_weight_bytes(const GroupArgs &a)
{
    return expected_groups(a) * a.N * (double)a.K * group_elem_size(a);
}

// Rows that start at 4-byte boundaries. Loads of others take about twice as long (measured on one
// shape with K = 1531 and 1536: 50 and 22 us through the rows kernel, 25 and 17 in 128 x 128 tiles).
inline bool aligned_words(const GroupArgs &a)
{
    const int es = group_elem_size(a);
    return (a.lda * es | a.ldb * es | a.stride_b * es | (int64_t)(uintptr_t)a.A | (int64_t)(uintptr_t)a.B) % 4 == 0;
}

// Most BM-row tiles that M rows in `groups` groups can need: whole tiles, and one partial
// tile for each group that has a row.
inline int64_t max_row_tiles(const GroupArgs &a, int bm)
{
    if (!a.offsets) return ((int64_t)a.M + bm - 1) / bm;
    return a.M / bm + (a.groups < a.M ? a.groups : a.M);
}

// Logical tile of workgroup bid: consecutive logical tiles on one XCD (workgroups are dealt
// to the 8 XCDs in turn), in groups of 8 row tiles that walk the tile columns together, so
// that an XCD's L2 serves both panels.
__device__ __forceinline__ void tile_of_group_block(unsigned bid, unsigned nblocks, unsigned tiles_m, unsigned tiles_n,
                                                    unsigned &tm, unsigned &tn)
{
    constexpr unsigned xcds = 8, group_m = 8;
    const unsigned q = nblocks / xcds, r = nblocks % xcds;
    const unsigned xcd = bid % xcds, slot = bid / xcds;
    const unsigned logical = (xcd < r) ? xcd * (q + 1) + slot : r * (q + 1) + (xcd - r) * q + slot;
    const unsigned per_group = group_m * tiles_n;
    const unsigned g = logical / per_group;
    const unsigned first_m = g * group_m;
    const unsigned gm = min(tiles_m - first_m, group_m);
    const unsigned in_g = logical - g * per_group;
    tm = first_m + in_g % gm;
    tn = in_g / gm;
}

}  // namespace
}  // namespace mm
