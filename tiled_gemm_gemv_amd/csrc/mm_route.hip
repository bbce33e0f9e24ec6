// mm_route.hip -- routing of tokens to experts, the rows' order by expert, and the logits' gradient.
//
// Scores of token t: s_e = exp(l_e - m) / sum exp(l - m), m = max l, or s_e = 1 / (1 + exp(-l_e)).
// Experts are ranked by c_e = s_e + b_e, without a bias by l_e, which ranks them as s_e does; groups
// of E / G neighbouring experts by the sum of their group_top best c_e (without a bias and with
// group_top 2: s_e). The best top_groups groups are kept, then the best k experts in them; equal
// values go to the lowest index, NaN is above every number. An expert whose l_e or c_e is -inf is not
// chosen; slots left over get expert -1 and weight 0. w_j = scale s_j, or scale s_j / sum of the chosen s
// (0 where that is 0).
//
// The ranks are taken in 64 bits: with 16384 tokens and 256 experts some pair of neighbouring scores
// lies closer than 32-bit rounding, and the choice would go by it.
//
// The rows' order: slots by (expert, token, slot). Each workgroup routes 64 tokens, counts their slots
// for each expert and numbers them there; a scan over the workgroups' counts gives each expert's first
// row and each workgroup's first of it; the last kernel adds that to the slots' numbers. No atomics: the
// order is fixed.
#include "mm_group.h"

namespace mm {
namespace {

constexpr int kWaves = 16, kTokens = 64;  // of a workgroup of the first kernel

template <class X>
__device__ __forceinline__ float load_logit(const void *p, int64_t at)
{
    return (float)static_cast<const X *>(p)[at];
}

__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmax(v, __shfl_xor(v, d));
    return v;
}
template <class V>
__device__ __forceinline__ V wave_add(V v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Numbers in an order of unsigned integers, NaN above all; 0 is below every number (-inf is 2^52 - 1).
__device__ __forceinline__ uint64_t ordered(double v)
{
    if (v != v) return ~0ull;
    if (v == 0) v = 0;  // -0 and 0 are equal
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return b >> 63 ? ~b : b | 1ull << 63;
}
constexpr uint64_t kLowest = 0x000fffffffffffffull;  // ordered(-inf)

// The largest key of the wave and the lowest index that has it.
__device__ __forceinline__ void wave_best(uint64_t &key, int &index)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint64_t k = __shfl_xor(key, d);
        const int i = __shfl_xor(index, d);
        if (k > key || (k == key && i < index)) key = k, index = i;
    }
}

// Scores of this lane's experts lane + 64 r of one token.
template <int R>
__device__ __forceinline__ void token_scores(const RouteArgs &p, const float (&l)[R], double (&s)[R])
{
    const int lane = threadIdx.x & 63;
    if (p.sigmoid) {
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = 1.0 / (1.0 + exp(-(double)l[r]));
        return;
    }
    double m = -__builtin_inf();
    bool nan = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m = fmax(m, (double)l[r]);
        nan |= l[r] != l[r];
    }
    m = wave_max(m);
    if (m == -__builtin_inf()) m = 0;
    if (__any(nan)) m = __builtin_nan("");
    double sum = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        s[r] = lane + 64 * r < p.E ? exp((double)l[r] - m) : 0.0;
        sum += s[r];
    }
    sum = wave_add(sum);
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = sum == 0 ? 0.0 : s[r] / sum;
}

// Scores, choice and weights of token t by one wave; lane j < k returns the expert of slot j (-1: none).
template <class X, int R>
__device__ __forceinline__ int route_token(const RouteArgs &p, int64_t t)
{
    const int lane = threadIdx.x & 63;
    float l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = lane + 64 * r;
        l[r] = e < p.E ? load_logit<X>(p.logits, t * p.ld + e) : -__builtin_inff();
    }
    double s[R];
    token_scores<R>(p, l, s);
    uint64_t key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = lane + 64 * r;
        const bool dead = l[r] == -__builtin_inff();
        const double c = p.bias ? s[r] + (double)(e < p.E ? p.bias[e] : 0.f) : (double)l[r];
        key[r] = dead ? kLowest : ordered(c);
    }
    if (p.groups > 1) {
        const int per = p.E / p.groups;
        uint64_t mine = 0;  // lane g: group g's value
        for (int g = 0; g < p.groups; ++g) {
            double sum = 0;
            int taken = -1;
            for (int n = 0; n < p.group_top; ++n) {
                uint64_t best = 0;
                int index = 0x7fffffff;
                double value = -__builtin_inf();
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int e = lane + 64 * r;
                    const bool dead = l[r] == -__builtin_inff();
                    const double c = dead                                   ? -__builtin_inf()
                                     : p.bias                               ? s[r] + (double)(e < p.E ? p.bias[e] : 0.f)
                                     : p.group_top == 1                     ? (double)l[r]
                                                                            : s[r];
                    const uint64_t k = ordered(c);
                    if (e / per == g && e < p.E && e != taken && k > best) best = k, index = e, value = c;
                }
                const int own = index;
                wave_best(best, index);
                const unsigned long long who = __ballot(own == index);
                value = __shfl(value, who ? __ffsll(who) - 1 : 0);
                sum = n == 0 ? value : index == 0x7fffffff ? -__builtin_inf() : sum + value;
                taken = index;
            }
            if (lane == g) mine = ordered(sum);
        }
        unsigned long long kept = 0;
        for (int n = 0; n < p.top_groups; ++n) {
            uint64_t best = lane < p.groups && !(kept >> lane & 1) ? mine : 0;
            int index = lane;
            wave_best(best, index);
            kept |= 1ull << index;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = lane + 64 * r;
            if (e < p.E && !(kept >> (e / per) & 1)) key[r] = kLowest;
        }
    }
    int chosen = -1;
    double weight = 0;
    for (int j = 0; j < p.k; ++j) {
        uint64_t best = 0;
        int index = 0x7fffffff;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (key[r] > best) best = key[r], index = lane + 64 * r;
        wave_best(best, index);
        if (best <= kLowest) break;  // none left
        double score = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane + 64 * r == index) {
                key[r] = 0;
                score = s[r];
            }
        score = __shfl(score, index & 63);
        if (lane == j) chosen = index, weight = score;
    }
    if (p.renormalize) {
        double sum = 0;
        for (int j = 0; j < p.k; ++j) sum += __shfl(weight, j);
        weight = sum == 0 || chosen < 0 ? 0.0 : weight / sum;
    }
    if (lane < p.k) {
        p.weights[t * p.k + lane] = (float)(weight * (double)p.scale);
        p.experts[t * p.k + lane] = chosen;
    }
    return chosen;
}

// Exclusive sum over the workgroup's threads, in thread order, and the total.
template <int W>
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned *part, unsigned &total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const unsigned incl = wave_inclusive_sum(v);
    if (lane == 63) part[w] = incl;
    __syncthreads();
    unsigned before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        before += i < w ? part[i] : 0;
        total += part[i];
    }
    __syncthreads();
    return before + incl - v;
}

// 64 tokens: weights and experts; rows: each slot's number among the workgroup's of its expert; the
// experts' counts. ALL: the only workgroup, which finishes rows and offsets.
template <class X, int R, bool ALL>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs p)
{
    // a wave's tokens choose an expert once each at most
    __shared__ unsigned char count[kWaves][64 * R];
    __shared__ short slot[kTokens * kRouteMaxTop];
    __shared__ unsigned first[64 * R], part[kWaves];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t bid = linear_block(), t0 = bid * kTokens;
    constexpr int per_wave = kTokens / kWaves;
    if (t0 >= p.T) return;  // the whole workgroup
    for (int i = lane; i < 64 * R; i += 64) count[w][i] = 0;
    for (int i = 0; i < per_wave; ++i) {
        const int t = w * per_wave + i;
        const int chosen = t0 + t < p.T ? route_token<X, R>(p, t0 + t) : -1;
        if (lane < p.k) slot[t * p.k + lane] = (short)chosen;
    }
    __syncthreads();
    // numbers within the wave: a token's experts differ, so those of the tokens before
    const int slots = per_wave * p.k, base = w * slots;
    for (int c = 0; c < slots; c += 64) {
        const int i = c + lane, e = i < slots ? slot[base + i] : -1;
        unsigned long long same = __ballot(e >= 0);
        for (int b = 0; b < 10; ++b) {
            const unsigned long long set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        if (e >= 0) {
            const int before = __popcll(same & ((1ull << lane) - 1)), n = count[w][e];
            __builtin_amdgcn_wave_barrier();
            if (before == __popcll(same) - 1) count[w][e] = (unsigned char)(n + before + 1);
            p.rows[t0 * p.k + base + i] = n + before;  // of the slots in range: e >= 0
        }
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // of the waves before; this workgroup's count of expert e
    unsigned total_e = 0;
    const int e = threadIdx.x;
    if (e < 64 * R)
        for (int i = 0; i < kWaves; ++i) {
            const unsigned n = count[i][e];
            count[i][e] = (unsigned char)total_e;  // at most 64 - 4
            total_e += n;
        }
    if constexpr (ALL) {
        unsigned total;
        const unsigned at = block_scan<kWaves>(e < p.E ? total_e : 0, part, total);
        if (e < p.E) {
            first[e] = at;
            p.offsets[e] = at;
        }
        if (e == 0) p.offsets[p.E] = total;
    } else if (e < p.E) {
        p.ws[bid * p.E + e] = (int)total_e;
    }
    __syncthreads();
    for (int c = 0; c < slots; c += 64) {
        const int i = c + lane;
        if (i >= slots || t0 * p.k + base + i >= (int64_t)p.T * p.k) continue;
        const int x = slot[base + i];
        int *row = p.rows + t0 * p.k + base + i;
        *row = x < 0 ? -1 : *row + count[w][x] + (ALL ? (int)first[x] : 0);
    }
}

// The workgroups' counts -> their first rows; offsets. One workgroup; `blocks` of the kernel before.
__global__ __launch_bounds__(1024) void route_scan_kernel(RouteArgs p, int blocks)
{
    __shared__ unsigned sums[1024], part[16];
    // 1024 / W threads to an expert, W = E rounded up to a power of two
    int W = 1;
    while (W < p.E) W *= 2;
    const int parts = 1024 / W, e = threadIdx.x % W, q = threadIdx.x / W;
    const int lo = (int)((int64_t)blocks * q / parts), hi = (int)((int64_t)blocks * (q + 1) / parts);
    unsigned sum = 0;
    if (e < p.E)
        for (int b = lo; b < hi; ++b) sum += (unsigned)p.ws[(int64_t)b * p.E + e];
    sums[threadIdx.x] = sum;
    __syncthreads();
    unsigned before = 0, all = 0;
    for (int i = 0; i < parts; ++i) {
        const unsigned v = sums[i * W + e];
        before += i < q ? v : 0;
        all += v;
    }
    __syncthreads();
    unsigned total;
    const unsigned first = block_scan<16>(q == 0 ? all : 0, part, total);  // of thread e: expert e
    if (q == 0) sums[e] = first;
    __syncthreads();
    unsigned at = sums[e] + before;
    if (e < p.E) {
        if (q == 0) p.offsets[e] = first;
        for (int b = lo; b < hi; ++b) {
            int *c = p.ws + (int64_t)b * p.E + e;
            const unsigned n = (unsigned)*c;
            *c = (int)at;
            at += n;
        }
    }
    if (threadIdx.x == 0) p.offsets[p.E] = total;
}

__global__ __launch_bounds__(256) void route_rows_kernel(RouteArgs p)
{
    const int64_t i = linear_block() * 256 + threadIdx.x;
    if (i >= (int64_t)p.T * p.k) return;
    const int e = p.experts[i];
    if (e >= 0) p.rows[i] += p.ws[i / (kTokens * p.k) * p.E + e];
}

// dl_e of one token by one wave: with g_e the gradient of s_e (0 where e was not chosen),
// softmax s_e (g_e - sum over i of s_i g_i), sigmoid s_e (1 - s_e) g_e. For w_j = scale s_j,
// g = scale dw; renormalised, with S the sum of the chosen s: g_j = scale / S (dw_j - sum_i dw_i s_i / S).
template <class X, int R>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = linear_block() * 4 + (threadIdx.x >> 6);
    if (t >= p.T) return;
    float l[R], s[R], d[R], g[R];  // d: s (1 - s) of a sigmoid
    float m = -__builtin_inff();
    bool nan = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = lane + 64 * r;
        l[r] = e < p.E ? load_logit<X>(p.logits, t * p.ld + e) : -__builtin_inff();
        m = fmaxf(m, l[r]);
        nan |= l[r] != l[r];
        g[r] = 0;
    }
    float sum = 0;
    if (p.sigmoid) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float q = expf(-fabsf(l[r])), n = 1.f / (1.f + q);
            s[r] = l[r] < 0 ? q * n : n;
            d[r] = q * n * n;
        }
    } else {
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
        if (m == -__builtin_inff()) m = 0;
        if (__any(nan)) m = __builtin_nanf("");
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = lane + 64 * r < p.E ? expf(l[r] - m) : 0.f;
            sum += s[r];
        }
        sum = wave_add(sum);
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = sum == 0 ? 0.f : s[r] / sum;
    }
    // lane j: slot j
    int e = lane < p.k ? p.experts[t * p.k + lane] : -1;
    if (e < 0 || e >= p.E) e = -1;
    float dw = e >= 0 ? p.scale * p.dweights[t * p.k + lane] : 0.f, mine = 0;
    for (int j = 0; j < p.k; ++j) {
        const int of = __shfl(e, j);
        float v = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (of >= 0 && of >> 6 == r) v = s[r];
        v = __shfl(v, of & 63);
        if (lane == j && of >= 0) mine = v;
    }
    if (p.renormalize) {
        float total = wave_add(mine);
        const float mean = total == 0 ? 0.f : wave_add(dw * (mine / total));
        dw = total == 0 || e < 0 ? 0.f : (dw - mean) / total;
    }
    float dot = 0;
    for (int j = 0; j < p.k; ++j) {
        const int of = __shfl(e, j);
        const float v = __shfl(dw, j);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (of == lane + 64 * r) g[r] += v;
    }
    if (!p.sigmoid) {
#pragma unroll
        for (int r = 0; r < R; ++r) dot = fmaf(s[r], g[r], dot);
        dot = wave_add(dot);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = lane + 64 * r;
        if (i < p.E) static_cast<X *>(p.dlogits)[t * p.ldd + i] = (X)(p.sigmoid ? d[r] * g[r] : s[r] * (g[r] - dot));
    }
}

// f(X(), R) with the logits' type and the registers of E experts in a wave.
template <class F>
hipError_t with_route(int type, int E, F &&f)
{
    auto sized = [&](auto x) {
        if (E <= 64) return f(x, std::integral_constant<int, 1>());
        if (E <= 128) return f(x, std::integral_constant<int, 2>());
        if (E <= 256) return f(x, std::integral_constant<int, 4>());
        if (E <= 512) return f(x, std::integral_constant<int, 8>());
        return f(x, std::integral_constant<int, 16>());
    };
    if (type == 0) return sized(float());
    if (type == 1) return sized(__bf16());
    return sized(_Float16());
}

}  // namespace

int64_t route_ws_ints(int64_t T, int E, int k)
{
    (void)k;
    const int64_t blocks = (T + kTokens - 1) / kTokens;
    return blocks > 1 ? blocks * E : 0;
}

hipError_t route_launch(const RouteArgs &a, hipStream_t stream)
{
    RouteArgs arg = a;
    const int64_t blocks = ((int64_t)a.T + kTokens - 1) / kTokens;
    unsigned gx, gy;
    if (!grid_for(blocks, gx, gy)) return hipErrorInvalidConfiguration;
    void *args[] = {&arg};
    const hipError_t e = with_route(a.type, a.E, [&](auto x, auto r) {
        typedef decltype(x) X;
        constexpr int R = decltype(r)::value;
        const void *fn = blocks == 1 ? reinterpret_cast<const void *>(&route_kernel<X, R, true>)
                                     : reinterpret_cast<const void *>(&route_kernel<X, R, false>);
        return hipLaunchKernel(fn, dim3(gx, gy), dim3(64 * kWaves), args, 0, stream);
    });
    if (e != hipSuccess || blocks == 1) return e;
    int n = (int)blocks;
    void *scan_args[] = {&arg, &n};
    const hipError_t s = hipLaunchKernel(reinterpret_cast<const void *>(&route_scan_kernel), dim3(1), dim3(1024), scan_args,
                                         0, stream);
    if (s != hipSuccess) return s;
    if (!grid_for(((int64_t)a.T * a.k + 255) / 256, gx, gy)) return hipErrorInvalidConfiguration;
    return hipLaunchKernel(reinterpret_cast<const void *>(&route_rows_kernel), dim3(gx, gy), dim3(256), args, 0, stream);
}

hipError_t route_grad_launch(const RouteGradArgs &a, hipStream_t stream)
{
    RouteGradArgs arg = a;
    unsigned gx, gy;
    if (!grid_for(((int64_t)a.T + 3) / 4, gx, gy)) return hipErrorInvalidConfiguration;
    void *args[] = {&arg};
    return with_route(a.type, a.E, [&](auto x, auto r) {
        return hipLaunchKernel(reinterpret_cast<const void *>(&route_grad_kernel<decltype(x), decltype(r)::value>),
                               dim3(gx, gy), dim3(256), args, 0, stream);
    });
}

}  // namespace mm
