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
// Bound by memory: a token's row is read (written) once for all its slots, the experts' rows go past the
// caches. 8192 tokens, 4 slots, rows of 4096 bf16, read and written: spread 52 us (6.4 TB/s), combine 57
// (5.8), gradient 117 (5.1); through the caches combine took 79-93.
#include "mm_group.h"

namespace mm {
namespace {

typedef unsigned int AnyWords __attribute__((ext_vector_type(4), aligned(1)));  // at any address

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

// 8 elements from column `col` of a row of D (zeros past it): as loaded, and as fp32.
template <class X>
struct Eight {
    static constexpr int N = Piece<X>::N, V = 8 / N;
    u32x4 v[V];
    // not kept in the caches
    __device__ __forceinline__ void load_once(const void *base, int64_t at, int col, int D)
    {
        if (D - col < 8) return load(base, at, col, D);  // not col + 8, which may pass 2^31 - 1
        const char *p = reinterpret_cast<const char *>(static_cast<const X *>(base) + at + col);
#pragma unroll
        for (int c = 0; c < V; ++c) v[c] = __builtin_nontemporal_load(reinterpret_cast<const AnyWords *>(p) + c);
    }
    __device__ __forceinline__ void load(const void *base, int64_t at, int col, int D)
    {
        const char *p = reinterpret_cast<const char *>(static_cast<const X *>(base) + at + col);
        const int64_t row_bytes = (int64_t)D * (int)sizeof(X);
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int64_t left = row_bytes - (int64_t)(col + c * N) * (int)sizeof(X);
            v[c] = load16_upto<X>(p + 16 * c, (int)max((int64_t)-1, min(left, (int64_t)16)), row_bytes);
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return Piece<X>::get(v[i / N], i % N); }
};

// ONCE: not kept in the caches.
template <class O, bool ONCE = false>
__device__ __forceinline__ void store_eight(void *base, int64_t at, int col, int D, const float (&x)[8])
{
    O *out = static_cast<O *>(base) + at + col;
    if (D - col >= 8) {
        constexpr int W = sizeof(O) / 2;  // 16-byte pieces
        struct Row {
            O v[8];
        } o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o.v[e] = (O)x[e];
        struct Words {
            u32x4 w[W];
        };
        const Words words = __builtin_bit_cast(Words, o);
#pragma unroll
        for (int c = 0; c < W; ++c) {
            AnyWords *q = reinterpret_cast<AnyWords *>(out) + c;
            if constexpr (ONCE) __builtin_nontemporal_store(words.w[c], q);
            else *q = words.w[c];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < D) out[e] = (O)x[e];
    }
}

// This thread's token and its number in the token's threads. Wide rows: a workgroup has a token and
// the part'th of `parts` pieces of 256 threads' units. NARROW, rows of at most 64 threads' units: 2^shift
// threads to a token, the others of the workgroup to those behind it.
struct Place {
    int64_t t, unit;
};
template <bool NARROW>
__device__ __forceinline__ Place place_of(unsigned parts, int shift)
{
    const int64_t bid = linear_block();
    if constexpr (NARROW) {
        return {(bid << (8 - shift)) + (threadIdx.x >> shift), (int64_t)(threadIdx.x & ((1u << shift) - 1))};
    } else {
        const int64_t t = bid / parts;
        return {t, (bid - t * parts) * 256 + threadIdx.x};
    }
}

// 16 bytes of a token's row to a thread.
template <bool NARROW>
__global__ __launch_bounds__(256) void spread_kernel(RowsArgs p, unsigned parts, int shift)
{
    const Place place = place_of<NARROW>(parts, shift);
    const int64_t t = place.t, at = 16 * place.unit;
    if (t >= p.T || at >= p.D) return;
    const int valid = (int)min((int64_t)16, p.D - at);
    const u32x4 v = load16_upto<unsigned char>(static_cast<const char *>(p.x) + t * p.ldx + at, valid, p.D);
    for (int j = 0; j < p.k; ++j) {
        const int r = p.rows[t * p.k + j];
        if (r < 0 || r >= p.total) continue;
        char *out = static_cast<char *>(p.out) + r * p.ldo + at;
        if (valid == 16) {
            __builtin_nontemporal_store(v, reinterpret_cast<AnyWords *>(out));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < valid) out[i] = (char)(v[i / 4] >> (8 * (i % 4)));
        }
    }
}

constexpr int kSlots = 4;

// 8 columns of a token to a thread.
template <class X, class O, bool NARROW>
__global__ __launch_bounds__(256) void combine_kernel(RowsArgs p, unsigned parts, int shift)
{
    const Place place = place_of<NARROW>(parts, shift);
    const int64_t t = place.t, first = 8 * place.unit;
    if (t >= p.T || first >= p.D) return;
    const int col = (int)first;
    float sum[8] = {};
    // kSlots loads on their way at once (one after the other: 79-93 us for 8192 x 4 rows of 4096 bf16)
    for (int j0 = 0; j0 < p.k && p.total > 0; j0 += kSlots) {
        Eight<X> x[kSlots];
        float w[kSlots];
        bool live[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int64_t slot = t * p.k + min(j0 + j, p.k - 1);
            const int r = p.rows[slot];
            live[j] = j0 + j < p.k && r >= 0 && r < p.total;
            w[j] = p.weights ? p.weights[slot] : 1.f;
            x[j].load_once(p.x, live[j] ? r * p.ldx : 0, col, p.D);  // row 0 in the place of none, and not used
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
            if (live[j]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[j], x[j][e], sum[e]);
            }
    }
    store_eight<O>(p.out, t * p.ldo, col, p.D, sum);
}

// Wide: a workgroup to a token, narrow: 2^shift threads, 8 columns each at a time.
template <class G, class Y, bool NARROW>
__global__ __launch_bounds__(256) void combine_grad_kernel(RowsArgs p, unsigned, int shift)
{
    __shared__ float part[4][8];
    const Place place = place_of<NARROW>(1, shift);
    const int64_t t = place.t;
    if (t >= p.T) return;  // narrow: whole tokens, whose threads' sums are their own
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        float dot[8] = {};
        for (int64_t first = 8 * place.unit; first < p.D; first += 2048) {
            const int col = (int)first;
            Eight<G> g;
            g.load(p.x, t * p.ldx, col, p.D);
#pragma unroll
            for (int j1 = 0; j1 < 8; j1 += kSlots) {
                if (j0 + j1 >= p.k || p.total == 0) break;
                Eight<Y> y[kSlots];
                int row[kSlots];
#pragma unroll
                for (int j = 0; j < kSlots; ++j) {
                    const int r = p.rows[t * p.k + min(j0 + j1 + j, p.k - 1)];
                    row[j] = j0 + j1 + j < p.k && r >= 0 && r < p.total ? r : -1;
                    y[j].load_once(p.y, max(row[j], 0) * p.ldy, col, p.D);  // row 0 in the place of none, and not used
                }
#pragma unroll
                for (int j = 0; j < kSlots; ++j) {
                    if (row[j] < 0) continue;
                    const float w = p.weights[t * p.k + j0 + j1 + j];
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dot[j1 + j] = fmaf(y[j][e], g[e], dot[j1 + j]);
                        d[e] = w * g[e];
                    }
                    store_eight<Y, true>(p.out, row[j] * p.ldo, col, p.D, d);
                }
            }
        }
        if constexpr (NARROW) {
            for (int d = 1 << shift >> 1; d > 0; d >>= 1)
#pragma unroll
                for (int j = 0; j < 8; ++j) dot[j] += __shfl_xor(dot[j], d);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (place.unit == 0 && j0 + j < p.k) p.dweights[t * p.k + j0 + j] = dot[j];
            continue;
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

// `unit`: what a thread takes of a row. `split`: a wide row's pieces go to workgroups of their own.
// Narrow rows would leave most of a workgroup idle (65536 x 2 rows of 128 bf16: spread 7.4 us, combine 13, its
// gradient 23; with one token to a workgroup 26, 41 and 217).
hipError_t launch(const void *wide, const void *narrow, const RowsArgs &a, int unit, bool split, hipStream_t stream)
{
    const int64_t units = ((int64_t)a.D + unit - 1) / unit;
    int shift = 0;
    while (shift < 6 && (int64_t)1 << shift < units) ++shift;
    const bool few = units <= 64;
    const int64_t parts = few || !split ? 1 : (units + 255) / 256, tokens = few ? 256 >> shift : 1;
    unsigned gx, gy;
    if (!grid_for(parts * ((a.T + tokens - 1) / tokens), gx, gy)) return hipErrorInvalidConfiguration;
    RowsArgs arg = a;
    unsigned n = (unsigned)parts;
    void *args[] = {&arg, &n, &shift};
    return hipLaunchKernel(few ? narrow : wide, dim3(gx, gy), dim3(256), args, 0, stream);
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
    return launch(reinterpret_cast<const void *>(&spread_kernel<false>), reinterpret_cast<const void *>(&spread_kernel<true>),
                  a, 16, true, stream);
}

hipError_t combine_rows_launch(const RowsArgs &a, hipStream_t stream)
{
    return with_type(a.x_type, [&](auto x) {
        return with_type(a.o_type, [&](auto o) {
            return launch(reinterpret_cast<const void *>(&combine_kernel<decltype(x), decltype(o), false>),
                          reinterpret_cast<const void *>(&combine_kernel<decltype(x), decltype(o), true>), a, 8, true, stream);
        });
    });
}

hipError_t combine_rows_grad_launch(const RowsArgs &a, hipStream_t stream)
{
    return with_type(a.x_type, [&](auto x) {
        return with_type(a.y_type, [&](auto y) {
            return launch(reinterpret_cast<const void *>(&combine_grad_kernel<decltype(x), decltype(y), false>),
                          reinterpret_cast<const void *>(&combine_grad_kernel<decltype(x), decltype(y), true>), a, 8, false, stream);
        });
    });
}

}  // namespace mm
