// mm_expert_rows.hip -- tokens' rows to the experts' order and back.
//
// rows[t][j] is the row that slot j of token t has in the experts' order, from 0 on; an entry outside
// [0, total) is no row and adds nothing.
//   spread    out[rows[t][j]] = x[t]
//   combine   out[t] = sum over j of w[t][j] y[rows[t][j]]      (w = 1 where there are no weights)
//   gradient  of combine, from the gradient g of out: dy[rows[t][j]] = w[t][j] g[t],
//             dw[t][j] = sum over d of y[rows[t][j]][d] g[t][d]
// The gradient of spread is combine without weights. Sums are fp32, over j from 0 on, so results are
// deterministic; each output is rounded once.
//
// Bound by memory: a token's row is read (written) once for all its slots.
#include "mm_group.h"

namespace mm {
namespace {

// 16 bytes of a row as fp32 values.
template <class X>
struct Piece {
    static constexpr int N = 16 / sizeof(X);
    static __device__ __forceinline__ float get(u32x4 v, int i)
    {
        const unsigned w = v[sizeof(X) == 4 ? i : i / 2];
        if constexpr (sizeof(X) == 4) return __builtin_bit_cast(float, w);
        else return (float)__builtin_bit_cast(X, (unsigned short)(w >> (16 * (i & 1))));
    }
};

// 8 elements from column `col` of a row of D (zeros past it), as fp32.
template <class X>
__device__ __forceinline__ void load_eight(const void *base, int64_t at, int col, int D, float (&x)[8])
{
    constexpr int N = Piece<X>::N;
    const char *p = reinterpret_cast<const char *>(static_cast<const X *>(base) + at + col);
    const int64_t row_bytes = (int64_t)D * (int)sizeof(X);
#pragma unroll
    for (int c = 0; c < 8 / N; ++c) {
        const int64_t left = row_bytes - (int64_t)(col + c * N) * (int)sizeof(X);
        const u32x4 v = load16_upto<X>(p + 16 * c, (int)max((int64_t)-1, min(left, (int64_t)16)), row_bytes);
#pragma unroll
        for (int i = 0; i < N; ++i) x[c * N + i] = Piece<X>::get(v, i);
    }
}

template <class O>
__device__ __forceinline__ void store_eight(void *base, int64_t at, int col, int D, const float (&x)[8])
{
    O *out = static_cast<O *>(base) + at + col;
    if (col + 8 <= D) {
        struct __attribute__((packed)) Eight {
            O v[8];
        } o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = (O)x[e];
        *reinterpret_cast<Eight *>(out) = o;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < D) out[e] = (O)x[e];
    }
}

// Workgroup: token and 4 KB of its row.
__global__ __launch_bounds__(256) void spread_kernel(RowsArgs p, unsigned parts)
{
    const int64_t bid = linear_block(), t = bid / parts;
    if (t >= p.T) return;
    const int64_t at = (bid - t * parts) * 4096 + 16 * threadIdx.x;
    if (at >= p.D) return;
    const int valid = (int)min((int64_t)16, p.D - at);
    const u32x4 v = load16_upto<unsigned char>(static_cast<const char *>(p.x) + t * p.ldx + at, valid, p.D);
    for (int j = 0; j < p.k; ++j) {
        const int r = p.rows[t * p.k + j];
        if (r < 0 || r >= p.total) continue;
        char *out = static_cast<char *>(p.out) + r * p.ldo + at;
        if (valid == 16) {
            struct __attribute__((packed)) Bytes {
                u32x4 v;
            };
            reinterpret_cast<Bytes *>(out)->v = v;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < valid) out[i] = (char)(v[i / 4] >> (8 * (i % 4)));
        }
    }
}

// Workgroup: token and 2048 columns.
template <class X, class O>
__global__ __launch_bounds__(256) void combine_kernel(RowsArgs p, unsigned parts)
{
    const int64_t bid = linear_block(), t = bid / parts;
    if (t >= p.T) return;
    const int64_t first = (bid - t * parts) * 2048 + 8 * threadIdx.x;
    if (first >= p.D) return;
    const int col = (int)first;
    float sum[8] = {};
    for (int j = 0; j < p.k; ++j) {
        const int r = p.rows[t * p.k + j];
        if (r < 0 || r >= p.total) continue;
        const float w = p.weights ? p.weights[t * p.k + j] : 1.f;
        float x[8];
        load_eight<X>(p.x, r * p.ldx, col, p.D, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, x[e], sum[e]);
    }
    store_eight<O>(p.out, t * p.ldo, col, p.D, sum);
}

// Workgroup: token.
template <class G, class Y>
__global__ __launch_bounds__(256) void combine_grad_kernel(RowsArgs p)
{
    __shared__ float part[4][8];
    const int64_t t = linear_block();
    if (t >= p.T) return;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        float dot[8] = {};
        for (int64_t first = 8 * threadIdx.x; first < p.D; first += 2048) {
            const int col = (int)first;
            float g[8];
            load_eight<G>(p.x, t * p.ldx, col, p.D, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j0 + j >= p.k) break;
                const int r = p.rows[t * p.k + j0 + j];
                if (r < 0 || r >= p.total) continue;
                float y[8], d[8];
                load_eight<Y>(p.y, r * p.ldy, col, p.D, y);
                const float w = p.weights[t * p.k + j0 + j];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot[j] = fmaf(y[e], g[e], dot[j]);
                    d[e] = w * g[e];
                }
                store_eight<Y>(p.out, r * p.ldo, col, p.D, d);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) dot[j] += __shfl_xor(dot[j], d);
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][j] = dot[j];
        }
        __syncthreads();
        const int j = threadIdx.x;
        if (j < 8 && j0 + j < p.k) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) sum += part[w][j];
            p.dweights[t * p.k + j0 + j] = sum;
        }
    }
}

hipError_t launch(const void *fn, const RowsArgs &a, int64_t part, hipStream_t stream)
{
    const int64_t parts = part ? (a.D + part - 1) / part : 1;
    unsigned gx, gy;
    if (!grid_for(parts * a.T, gx, gy)) return hipErrorInvalidConfiguration;
    RowsArgs arg = a;
    unsigned n = (unsigned)parts;
    void *args[] = {&arg, &n};
    return hipLaunchKernel(fn, dim3(gx, gy), dim3(256), args, 0, stream);
}

// f(X()) with the type of number t (MM_TYPE_*).
template <class F>
auto with_type(int t, F &&f)
{
    if (t == 0) return f(float());
    if (t == 1) return f(__bf16());
    return f(_Float16());
}

}  // namespace

hipError_t spread_rows_launch(const RowsArgs &a, hipStream_t stream)
{
    return launch(reinterpret_cast<const void *>(&spread_kernel), a, 4096, stream);
}

hipError_t combine_rows_launch(const RowsArgs &a, hipStream_t stream)
{
    return with_type(a.x_type, [&](auto x) {
        return with_type(a.o_type, [&](auto o) {
            return launch(reinterpret_cast<const void *>(&combine_kernel<decltype(x), decltype(o)>), a, 2048, stream);
        });
    });
}

hipError_t combine_rows_grad_launch(const RowsArgs &a, hipStream_t stream)
{
    return with_type(a.x_type, [&](auto x) {
        return with_type(a.y_type, [&](auto y) {
            return launch(reinterpret_cast<const void *>(&combine_grad_kernel<decltype(x), decltype(y)>), a, 0, stream);
        });
    });
}

}  // namespace mm
