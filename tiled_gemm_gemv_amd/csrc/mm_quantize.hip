// mm_quantize.hip -- rows of a matrix to 8-bit integers with one scale for each row.
//
// For row i with amax = max |x_ij|:  scale_i = amax / 127 (rounded to fp32),
// q_ij = 127 x_ij / amax rounded to the nearest integer, halves to the even one. The rounding
// is that of the exact quotient: r = x (127 / amax) in fp32 is off by at most 2^-23 |r|
// (two roundings of half a step), so it decides wherever it lies further than that from a
// half; nearer, the quotient is taken in 64 bits, where 127 x is exact and the rounded
// quotient lands on a half only if the exact one does: 127 x / amax = n + 1/2 + d with d != 0
// has |d| >= 2^-26 |x / amax| (x and amax have 24 significant bits), far above 2^-53 of the
// quotient. amax below 2^-60 (127 / amax could overflow) is scaled by 2^64, as is x.
//
// A row of zeros gets scale 0; a row with an infinity or a NaN gets scale NaN and zeros, so
// that every product with it is NaN.
#include "mm_group.h"

namespace mm {
namespace {

template <class X>
__device__ __forceinline__ float as_f32(X v)
{
    return (float)v;
}

__device__ __forceinline__ int quantize_one(float x, float amax, float inv, float c)
{
    const float r = x * c * inv;
    const float n = rintf(r);
    // distance of |r - n| from one half, against the error bound of r
    if (fabsf(0.5f - fabsf(r - n)) <= fabsf(r) * 0x1p-22f) return (int)rint((double)x * 127.0 / (double)amax);
    return (int)n;
}

// One workgroup per row: the row's largest magnitude, then its values.
template <class X>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs p)
{
    __shared__ float part[4];
    const int64_t row = linear_block();
    if (row >= p.rows) return;
    const X *x = static_cast<const X *>(p.X) + row * p.ldx;
    signed char *q = p.Q + row * p.ldq;
    float amax = 0.f;
    bool bad = false;
    for (int64_t j = threadIdx.x; j < p.cols; j += 256) {
        const float v = fabsf(as_f32(x[j]));
        bad |= !(v < __builtin_inff());
        amax = fmaxf(amax, v);
    }
    if (bad) amax = __builtin_inff();
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    const bool finite = amax < __builtin_inff();
    if (threadIdx.x == 0) p.scale[row] = finite ? amax / 127.f : __builtin_nanf("");
    const bool zero = !finite || amax == 0.f;
    const float c = amax < 0x1p-60f ? 0x1p64f : 1.f;
    const float inv = zero ? 0.f : 127.f / (amax * c);
    for (int64_t j = threadIdx.x; j < p.cols; j += 256)
        q[j] = zero ? 0 : (signed char)quantize_one(as_f32(x[j]), amax, inv, c);
}

}  // namespace

hipError_t quantize_launch(const QuantArgs &a, hipStream_t stream)
{
    unsigned gx, gy;
    if (!grid_for(a.rows, gx, gy)) return hipErrorInvalidConfiguration;
    const void *fn = a.x_type == 0   ? reinterpret_cast<const void *>(&quantize_kernel<float>)
                     : a.x_type == 1 ? reinterpret_cast<const void *>(&quantize_kernel<__bf16>)
                                     : reinterpret_cast<const void *>(&quantize_kernel<_Float16>);
    QuantArgs arg = a;
    void *args[] = {&arg};
    return hipLaunchKernel(fn, dim3(gx, gy), dim3(256), args, 0, stream);
}

}  // namespace mm
