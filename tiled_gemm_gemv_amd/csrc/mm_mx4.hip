// mm_mx4.hip -- rows of a matrix to 4-bit floating point in blocks of 32 with a power of two each,
// and back.
//
// For block b of a row with amax = max |x|:  the power's exponent e = floor(log2 amax) - 2, stored
// as the byte e + 127 (at least 0; blocks of zeros: 0); element x / 2^e to the nearest of 0, 1/2, 1,
// 3/2, 2, 3, 4, 6 with x's sign, halfway to the one with the even code, above 6 to 6 (x / 2^e < 8).
// With the byte s the quotient is x 2^(127 - s), a multiplication by a normal power (s <= 252) and
// exact where it matters: |x| < 2^(s - 124), and a quotient that becomes subnormal is far below 1/4.
// The rounding is the conversion instruction's, with scale 1. A block with an infinity or a NaN gets
// the byte 255, which stands for NaN, and zeros: all its values are NaN. The largest magnitude is
// taken over the bits without their sign, as integers: there infinities and NaN are above every
// number.
//
// A lane takes 8 elements, so a block is a quad of lanes: the maximum takes two DPP steps. Bound by
// memory: each x is read once, each code written once, x past the caches. 8192 x 14336 bf16: 50 us (5.9
// TB/s), back 43 us (6.9 TB/s); x through the caches both together 113 instead of 92.
#include "mm_group.h"

namespace mm {
namespace {

typedef unsigned int AnyWords __attribute__((ext_vector_type(4), aligned(1)));  // at any address

constexpr int kUnit = 8;      // elements of a lane
constexpr int kUnits = 4;     // units of a lane, 256 apart
constexpr int kThreads = 256;

// Unit number i of this lane: its row and its place in the row; false past the last. Workgroups take
// consecutive units of the matrix, four to a block, row after row.
struct Units {
    int64_t row0, rows;
    unsigned first, per_row;
    __device__ __forceinline__ Units(int64_t rows_, int64_t cols) : rows(rows_)
    {
        per_row = (unsigned)((cols + 31) / 32) * 4;
        const int64_t u = linear_block() * (kThreads * kUnits);
        row0 = u / per_row;
        first = (unsigned)(u - row0 * per_row) + threadIdx.x;
    }
    __device__ __forceinline__ bool at(int i, int64_t &row, unsigned &unit) const
    {
        const unsigned u = first + kThreads * i, r = u / per_row;
        row = row0 + r;
        unit = u - r * per_row;
        return row < rows;
    }
};

// The 8 values of a unit, as fp32.
template <class X>
__device__ __forceinline__ void unpack(const u32x4 (&v)[sizeof(X) / 2], float (&x)[kUnit])
{
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
        if constexpr (sizeof(X) == 4) {
            const unsigned w = v[i / 4][i % 4];
            x[i] = __builtin_bit_cast(float, w);
        } else {
            const unsigned w = v[0][i / 2];
            x[i] = (float)__builtin_bit_cast(X, (unsigned short)(w >> (16 * (i & 1))));
        }
    }
}

template <class X>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(Mx4Args p)
{
    constexpr int V = sizeof(X) / 2;  // 16-byte loads of a unit
    const Units units(p.rows, p.cols);
    const int64_t row_bytes = p.cols * (int64_t)sizeof(X);
    u32x4 v[kUnits][V];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        int64_t row;
        unsigned unit;
        const bool live = units.at(i, row, unit);
        if (live && (int64_t)(unit + 1) * kUnit <= p.cols) {
            const AnyWords *x = reinterpret_cast<const AnyWords *>(static_cast<const X *>(p.X) + row * p.ldx + (int64_t)unit * kUnit);
#pragma unroll
            for (int c = 0; c < V; ++c) v[i][c] = __builtin_nontemporal_load(x + c);
            continue;
        }
        const char *x = static_cast<const char *>(p.X) + (row * p.ldx + (int64_t)unit * kUnit) * (int)sizeof(X);
        const int64_t left = live ? row_bytes - (int64_t)unit * kUnit * (int)sizeof(X) : 0;
#pragma unroll
        for (int c = 0; c < V; ++c)
            v[i][c] = load16_upto<X>(x + 16 * c, (int)max((int64_t)-1, min(left - 16 * c, (int64_t)16)), row_bytes);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        int64_t row;
        unsigned unit;
        const bool live = units.at(i, row, unit);
        float x[kUnit];
        unpack<X>(v[i], x);
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < kUnit; ++e) top = max(top, __builtin_bit_cast(unsigned, x[e]) & 0x7fffffffu);
        top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0xb1, 0xf, 0xf, false));  // quad: lanes 1 0 3 2
        top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0x4e, 0xf, 0xf, false));  // lanes 2 3 0 1
        const unsigned exponent = top >> 23;
        const bool finite = exponent < 255;
        const unsigned code = !finite ? 255u : exponent > 2 ? exponent - 2 : 0u;
        const float power = __builtin_bit_cast(float, (254u - min(code, 252u)) << 23);
        unsigned q = 0;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[0] * power, x[1] * power, 1.f, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[2] * power, x[3] * power, 1.f, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[4] * power, x[5] * power, 1.f, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, x[6] * power, x[7] * power, 1.f, 3);
        if (!finite) q = 0;
        if (!live) continue;
        struct __attribute__((packed)) Word {
            unsigned w;
        };
        reinterpret_cast<Word *>(p.Q + row * p.ldq + (int64_t)unit * 4)->w = q;
        if (unit % 4 == 0) p.scale[row * p.lds + unit / 4] = (unsigned char)code;
    }
}

template <class X>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(Mx4Args p)
{
    const Units units(p.rows, p.cols);
    struct __attribute__((packed)) Word {
        unsigned w;
    };
    unsigned q[kUnits], s[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        int64_t row;
        unsigned unit;
        q[i] = s[i] = 0;
        if (!units.at(i, row, unit)) continue;
        q[i] = reinterpret_cast<const Word *>(p.Q + row * p.ldq + (int64_t)unit * 4)->w;
        s[i] = p.scale[row * p.lds + unit / 4];
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        int64_t row;
        unsigned unit;
        if (!units.at(i, row, unit)) continue;
        const unsigned bits = s[i] == 255 ? 0x7fc00000u : s[i] == 0 ? 0x00400000u : s[i] << 23;
        const float power = __builtin_bit_cast(float, bits);
        float x[kUnit];
        auto pair = [&](auto v, int at) {
            x[at] = v[0] * power;
            x[at + 1] = v[1] * power;
        };
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 0), 0);
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 1), 2);
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 2), 4);
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 3), 6);
        const int64_t col = (int64_t)unit * kUnit;
        X *out = static_cast<X *>(p.X) + row * p.ldx + col;
        if (col + kUnit <= p.cols) {
            struct Eight {
                X v[kUnit];
            } o;
#pragma unroll
            for (int e = 0; e < kUnit; ++e) o.v[e] = (X)x[e];
            struct Words {
                u32x4 w[sizeof(X) / 2];
            };
            const Words words = __builtin_bit_cast(Words, o);
#pragma unroll
            for (int c = 0; c < (int)sizeof(X) / 2; ++c)
                __builtin_nontemporal_store(words.w[c], reinterpret_cast<AnyWords *>(out) + c);
        } else {
#pragma unroll
            for (int e = 0; e < kUnit; ++e)
                if (col + e < p.cols) out[e] = (X)x[e];
        }
    }
}

hipError_t launch(const void *fn, const Mx4Args &a, hipStream_t stream)
{
    const int64_t per_row = (a.cols + 31) / 32 * 4;
    if (a.rows > INT64_MAX / 2 / per_row) return hipErrorInvalidConfiguration;
    unsigned gx, gy;
    if (!grid_for((a.rows * per_row + kThreads * kUnits - 1) / (kThreads * kUnits), gx, gy))
        return hipErrorInvalidConfiguration;
    Mx4Args arg = a;
    void *args[] = {&arg};
    return hipLaunchKernel(fn, dim3(gx, gy), dim3(kThreads), args, 0, stream);
}

}  // namespace

hipError_t mx4_quantize_launch(const Mx4Args &a, hipStream_t stream)
{
    const void *fn[3] = {reinterpret_cast<const void *>(&mx4_quantize_kernel<float>),
                         reinterpret_cast<const void *>(&mx4_quantize_kernel<__bf16>),
                         reinterpret_cast<const void *>(&mx4_quantize_kernel<_Float16>)};
    return launch(fn[a.x_type], a, stream);
}

hipError_t mx4_dequantize_launch(const Mx4Args &a, hipStream_t stream)
{
    const void *fn[3] = {reinterpret_cast<const void *>(&mx4_dequantize_kernel<float>),
                         reinterpret_cast<const void *>(&mx4_dequantize_kernel<__bf16>),
                         reinterpret_cast<const void *>(&mx4_dequantize_kernel<_Float16>)};
    return launch(fn[a.x_type], a, stream);
}

}  // namespace mm
