// mm_quantize.hip -- rows of a matrix to 8-bit integers with one scale for each row.
//
// For row i with amax = max |x_ij|:  scale_i = amax / 127 (rounded to fp32),
// q_ij = 127 x_ij / amax rounded to the nearest integer, halves to the even one. The rounding is
// that of the exact quotient, although it is computed as r = x (127 / amax) in fp32, off by at most
// 2^-23 |r| (two roundings of half a step):
//   * 16-bit x and amax are m 2^e with m < 2^11. A quotient that is not itself a half lies at
//     least |254 m_x 2^d - (2n + 1) m_a| / (2 m_a) from the half n + 1/2 (d = e_x - e_a), and the
//     numerator is a nonzero multiple of 2^min(d, 0): more than 2^-19 of the quotient. Rounding r
//     to the nearest multiple of 8 steps (moving it by at most 4 2^-23 |r|) therefore takes every
//     exact half back to itself, and no other quotient across one.
//   * fp32: where r lies within 2^-22 |r| of a half, the quotient is taken in 64 bits: 127 x is
//     exact there, and by the same count a quotient that is not a half is at least 2^-32 of itself
//     away from it.
// amax below 2^-60 (127 / amax could overflow) is scaled by 2^64, as is x.
//
// A row of zeros gets scale 0; a row with an infinity or a NaN gets scale NaN and zeros, so that
// every product with it is NaN. The largest magnitude is taken over the bits without their sign, as
// integers: there infinities and NaN are above every number.
//
// Bound by memory: each x is read once, kept in registers between the two steps, each q written once:
// bf16 8192 x 14336 66 us, 5.3 TB/s read and written, fp32 102 us, 5.8 TB/s (the 64-bit quotients, for
// one element in some 10^5, do not show); 8 x 4096 3 and 4 us, the launch. Reading the rows twice
// and single elements took 224 and 15.6 us.
#include "mm_group.h"

namespace mm {
namespace {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// The elements of a 16-byte chunk.
template <class X>
struct Chunk {
    static constexpr int N = 16 / sizeof(X);
};

// |x| bits (as fp32) of the largest of the chunk's elements and `top`, which is in the form that
// top_bits turns into fp32 bits.
template <class X>
__device__ __forceinline__ unsigned chunk_top(u32x4 v, unsigned top)
{
    if constexpr (sizeof(X) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, v[i] & 0x7fffffffu);
    } else {  // two 16-bit maxima side by side
        u16x2 t = __builtin_bit_cast(u16x2, top);
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
        top = __builtin_bit_cast(unsigned, t);
    }
    return top;
}
template <class X>
__device__ __forceinline__ unsigned top_bits(unsigned top)
{
    if constexpr (sizeof(X) == 4) {
        return top;
    } else {
        const unsigned short m = (unsigned short)max(top & 0xffffu, top >> 16);
        return __builtin_bit_cast(unsigned, (float)__builtin_bit_cast(X, m));
    }
}

template <class X>
__device__ __forceinline__ float element(u32x4 v, int i)
{
    const unsigned word = v[sizeof(X) == 4 ? i : i >> 1];  // a copy: a bit cast of the element itself reads element 0
    if constexpr (sizeof(X) == 4) return __builtin_bit_cast(float, word);
    else return (float)__builtin_bit_cast(X, (unsigned short)(word >> (16 * (i & 1))));
}

struct Quotient {
    float amax, inv, c;  // c = 1, or 2^64 for a tiny amax; inv = 127 / (amax c), 0 for a row without scale
    __device__ Quotient(unsigned bits)
    {
        amax = __builtin_bit_cast(float, bits);
        c = amax < 0x1p-60f ? 0x1p64f : 1.f;
        inv = bits == 0 || bits >= 0x7f800000u ? 0.f : 127.f / (amax * c);
    }
    __device__ float scale() const { return amax < __builtin_inff() ? amax / 127.f : __builtin_nanf(""); }
    template <class X>
    __device__ __forceinline__ int of(float x) const
    {
        const float r = x * c * inv;
        if constexpr (sizeof(X) == 2) {
            return (int)rintf(__builtin_bit_cast(float, (__builtin_bit_cast(unsigned, r) + 4u) & ~7u));
        } else {
            const float n = rintf(r);
            // distance of r from the half next to it
            if (fabsf(0.5f - fabsf(r - n)) <= fabsf(r) * 0x1p-22f) return (int)rint((double)x * 127.0 / (double)amax);
            return (int)n;
        }
    }
};

// The first `n` of the chunk's quotients to q.
template <class X>
__device__ __forceinline__ void store_chunk(signed char *q, u32x4 v, const Quotient &k, bool live, int n)
{
    constexpr int N = Chunk<X>::N;
    unsigned words[N / 4];
#pragma unroll
    for (int w = 0; w < N / 4; ++w) {
        unsigned o = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) o |= ((unsigned)k.of<X>(element<X>(v, 4 * w + i)) & 0xffu) << (8 * i);
        words[w] = live ? o : 0u;
    }
    if (n >= N) {
        struct __attribute__((packed)) Out {
            unsigned w[N / 4];
        } o;
#pragma unroll
        for (int w = 0; w < N / 4; ++w) o.w[w] = words[w];
        *reinterpret_cast<Out *>(q) = o;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) q[i] = (signed char)(words[i / 4] >> (8 * (i & 3)));
    }
}

// The row's largest bits over its TPR threads (in the workgroup's 256 or TPR threads).
template <int TPR>
__device__ __forceinline__ unsigned row_max(unsigned bits, unsigned *part)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) bits = max(bits, (unsigned)__shfl_xor((int)bits, d));
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = bits;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) bits = max(bits, part[i]);
    }
    return bits;
}

// TPR threads per row, each with CH chunks of it in registers (cols <= TPR CH chunks); 256 / TPR
// rows per workgroup where TPR is 64.
template <class X, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void quantize_kernel(QuantArgs p)
{
    constexpr int N = Chunk<X>::N, RPW = TPR < 256 ? 256 / TPR : 1;
    __shared__ unsigned part[TPR / 64];
    const int64_t row = linear_block() * RPW + (RPW > 1 ? threadIdx.x / TPR : 0);
    if (row >= p.rows) return;  // whole waves; with RPW > 1 there is no barrier below
    const int t = threadIdx.x % TPR, cols = (int)p.cols;
    const char *x = reinterpret_cast<const char *>(static_cast<const X *>(p.X) + row * p.ldx);
    u32x4 v[CH];
    unsigned top = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (t + c * TPR) * N;
        v[c] = load16_upto<X>(x + (int64_t)col * (int)sizeof(X), (cols - col) * (int)sizeof(X), p.cols * sizeof(X));
        top = chunk_top<X>(v[c], top);
    }
    const Quotient k(row_max<TPR>(top_bits<X>(top), part));
    if (t == 0) p.scale[row] = k.scale();
    signed char *q = p.Q + row * p.ldq;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = (t + c * TPR) * N;
        if (col < cols) store_chunk<X>(q + col, v[c], k, k.inv != 0.f, cols - col);
    }
}

// Rows too long for the registers: read twice.
template <class X>
__global__ __launch_bounds__(1024) void quantize_long_kernel(QuantArgs p)
{
    constexpr int N = Chunk<X>::N;
    __shared__ unsigned part[16];
    const int64_t row = linear_block();
    if (row >= p.rows) return;
    const char *x = reinterpret_cast<const char *>(static_cast<const X *>(p.X) + row * p.ldx);
    signed char *q = p.Q + row * p.ldq;
    auto load = [&](int64_t col) {
        return load16_upto<X>(x + col * (int)sizeof(X), (int)min((int64_t)16, (p.cols - col) * (int64_t)sizeof(X)),
                              p.cols * sizeof(X));
    };
    unsigned top = 0;
    for (int64_t col = (int64_t)threadIdx.x * N; col < p.cols; col += 1024 * N) top = chunk_top<X>(load(col), top);
    const Quotient k(row_max<1024>(top_bits<X>(top), part));
    if (threadIdx.x == 0) p.scale[row] = k.scale();
    for (int64_t col = (int64_t)threadIdx.x * N; col < p.cols; col += 1024 * N)
        store_chunk<X>(q + col, load(col), k, k.inv != 0.f, (int)min((int64_t)N, p.cols - col));
}

template <class X, int TPR, int CH>
hipError_t launch(const QuantArgs &a, hipStream_t stream)
{
    constexpr int rpw = TPR < 256 ? 256 / TPR : 1;
    unsigned gx, gy;
    if (!grid_for((a.rows + rpw - 1) / rpw, gx, gy)) return hipErrorInvalidConfiguration;
    QuantArgs arg = a;
    void *args[] = {&arg};
    return hipLaunchKernel(reinterpret_cast<const void *>(&quantize_kernel<X, TPR, CH>), dim3(gx, gy),
                           dim3(TPR < 256 ? 256 : TPR), args, 0, stream);
}

// A row's threads: a wave (four rows to a workgroup) up to 128 chunks, else 256 with up to 8 chunks
// each, else 1024 (up to 64 KB of a row in registers); longer rows are read twice.
template <class X>
hipError_t quantize(const QuantArgs &a, hipStream_t stream)
{
    const int64_t chunks = (a.cols + Chunk<X>::N - 1) / Chunk<X>::N;
    if (chunks <= 64) return launch<X, 64, 1>(a, stream);
    if (chunks <= 128) return launch<X, 64, 2>(a, stream);
    if (chunks <= 256) return launch<X, 256, 1>(a, stream);
    if (chunks <= 512) return launch<X, 256, 2>(a, stream);
    if (chunks <= 1024) return launch<X, 256, 4>(a, stream);
    if (chunks <= 2048) return launch<X, 256, 8>(a, stream);
    if (chunks <= 4096) return launch<X, 1024, 4>(a, stream);
    unsigned gx, gy;
    if (!grid_for(a.rows, gx, gy)) return hipErrorInvalidConfiguration;
    QuantArgs arg = a;
    void *args[] = {&arg};
    return hipLaunchKernel(reinterpret_cast<const void *>(&quantize_long_kernel<X>), dim3(gx, gy), dim3(1024), args, 0,
                           stream);
}

}  // namespace

hipError_t quantize_launch(const QuantArgs &a, hipStream_t stream)
{
    if (a.x_type == 0) return quantize<float>(a, stream);
    return a.x_type == 1 ? quantize<__bf16>(a, stream) : quantize<_Float16>(a, stream);
}

}  // namespace mm
