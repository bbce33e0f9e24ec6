// mm_route.hip -- routing of tokens to experts, the rows' order by expert, and the logits' gradient.
//
// Scores of token t: s_e = exp(l_e - m) / sum exp(l - m), m = max l, or s_e = 1 / (1 + exp(-l_e)).
// Experts are ranked by c_e = s_e + b_e, without a bias by l_e, which ranks them as s_e does; groups
// of E / G neighbouring experts by the sum of their group_top best c_e (without a bias and with
// group_top 2: s_e; of a single expert, its own). The best top_groups groups are kept, then the best k
// experts in them; equal values go to the lowest index, NaN is above every number. An expert whose l_e or
// c_e is -inf is not chosen; slots left over get expert -1 and weight 0. w_j = scale s_j, or scale s_j / sum
// of the chosen s (0 where that is 0).
//
// The ranks are those of 64-bit values: with 16384 tokens and 256 experts some pair of neighbouring
// scores lies closer than 32-bit rounding, and the choice would go by it. A wave takes four tokens, 16
// lanes each, or (more than 256 experts, 12 chosen or 16 groups) one. It computes c in 32 bits, off by at
// most `slack`, and picks the best one after the other by a 32-bit key of 22 leading bits and the index: k
// of them, and all others that could be above the k-th by slack and truncation. Those few, one to a lane,
// get their values in 64 bits and are put in that order. Where groups lie closer than their summands'
// slack, they are ranked in 64 bits; where values are NaN or infinite, or more experts than the token has
// lanes are that close, the token is done in 64 bits throughout.
//
// The rows' order: slots by (expert, token, slot). A workgroup routes 16 or 64 tokens; a token takes an expert
// once, so a 64-bit mask for each expert says which of them have it, and counts of its bits number the
// workgroup's slots. The workgroups' counts are added up over workgroups and experts (in the last
// kernel itself for up to 16 workgroups, else by one in between). No atomics but the masks' bits: the
// order is fixed.
//
// Many tokens are bound by instructions, some 2000 of a wave for four tokens of 256 experts, 8 of them
// chosen, and by waits for chains of maxima (0.46 of the waves' cycles): all three kernels for 16384 tokens,
// in a graph, 21-23 us, with groups and a bias 27 (one token to a wave 39), of 8 MB that could be read in 2.
// One token to a wave: 16384 tokens of 384 experts in groups 51 us, of 512 (10 chosen) 47, of 1024 (32
// chosen) 173; with so many experts the kernel keeps part of its values in memory. Few tokens are bound by
// the launches: 3 to 5 us each, three of them (4001 tokens of 60 experts 12 us in a graph; 8 tokens of 64
// experts: one launch, 5.5).
//
// Tokens done in 64 bits throughout take turns in their wave: 16384 tokens whose 256 logits are all equal
// 56 us, biased and in groups 147; of 512 experts 148. Biases of +-1000 (256 experts in 8 groups), which
// leave most choices to 64 bits: 119 us.
//
// The gradient takes a wave for a token: 16384 tokens of 64, 256 and 512 experts, 16-bit logits, 9, 14 and
// 20 us (4, 17 and 34 MB read and written), of 1024, fp32, 48 (134 MB); 4001 of 60, fp32, 4.4.
#include "mm_group.h"

namespace mm {
namespace {

constexpr int kWaves = 16;                // of a workgroup of the first kernel
constexpr int kTokens = 64;               // most tokens of a workgroup
constexpr int kFewBlocks = 16;            // workgroups whose counts the last kernel adds up by itself

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

// Largest value of the wave, in every lane.
__device__ __forceinline__ unsigned wave_max_u32(unsigned v)
{
    v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));  // row_shr 1, 2, 4, 8
    v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
    v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
    v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
    v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));  // row_bcast 15
    v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));  // row_bcast 31
    return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
}
// The largest key of the wave and the lowest index that has it.
__device__ __forceinline__ void wave_best(uint64_t &key, int &index)
{
    const unsigned hi = wave_max_u32((unsigned)(key >> 32));
    const bool top = (unsigned)(key >> 32) == hi;
    const unsigned lo = wave_max_u32(top ? (unsigned)key : 0u);
    index = (int)~wave_max_u32(top && (unsigned)key == lo ? ~(unsigned)index : 0u);
    key = (uint64_t)hi << 32 | lo;
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

// Scores, choice and weights of token t by one wave, all of it in 64 bits; lane j < k returns the expert
// of slot j (-1: none).
template <class X, int R>
__device__ __forceinline__ int route_token_exact(const RouteArgs &p, int64_t t)
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
                                     : p.sums                               ? s[r]
                                                                            : (double)l[r];
                    const uint64_t k = ordered(c);
                    if (e / per == g && e < p.E && e != taken && k > best) best = k, index = e, value = c;
                }
                const int own = index;
                wave_best(best, index);
                const unsigned long long who = __ballot(own == index);
                value = __shfl(value, who ? __ffsll(who) - 1 : 0);
                sum = n == 0 ? value : sum + value;
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

// The same for fp32, and back.
__device__ __forceinline__ unsigned ordered32(float v)
{
    if (v != v) return ~0u;
    const unsigned b = __builtin_bit_cast(unsigned, v + 0.f);  // -0 and 0 are equal
    return b >> 31 ? ~b : b | 1u << 31;
}
__device__ __forceinline__ float from_ordered32(unsigned u)
{
    return __builtin_bit_cast(float, u >> 31 ? u & 0x7fffffffu : ~u);
}

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v)
{
    auto step = [&](auto ctrl, auto rows) {
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value,
                                                                   decltype(rows)::value, 0xf, false));
    };
    step(std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());  // row_shr 1, 2, 4, 8
    step(std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());  // row_bcast 15
    step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());  // row_bcast 31
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ float readlane_f(float v, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ uint64_t readlane_u64(uint64_t v, int lane)
{
    return (uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (unsigned)__builtin_amdgcn_readlane((int)v, lane);
}

// How far c in 32 bits may be from c in 64. Sigmoid: the exponential is off by 2^-23 of itself and, from
// its argument times log2 e, by 1.5 |l| 2^-24, which makes 2^-25 and (s (1 - s) |l| <= 0.224) 2^-25.5 of s;
// 1 + exp and its reciprocal 3 2^-24 s: less than 2^-22. Softmax: the exponential 2^-23 of itself and
// |l - m| 2^-24 (0.37 at most of p |l - m|), sum and quotient 2^-24 each: less than 2^-22 too. The sum with
// the bias 2^-24 |c|.
__device__ __forceinline__ float slack(float c) { return 0x1p-22f + 0x1p-23f * fabsf(c); }

// The same for a group's value, first or (two) first + second: its summands' slack, however small the sum
// of summands of either sign is. Half of 2^-23 |c| is c's own rounding, the other half the sum's. A sum
// past fp32's range may be anything; one with -inf is -inf in 64 bits too.
template <class V>
__device__ __forceinline__ float group_slack(V first, V second, V value, bool two)
{
    if constexpr (sizeof(V) == 8) return 0.f;
    else if ((two ? second : first) == -__builtin_inff()) return 0.f;
    else if (!(fabsf(value) < __builtin_inff())) return __builtin_inff();
    else return slack(first) + (two ? slack(second) : 0.f);
}
// Whether values of 64 bits may stand in another order than `low`, the last kept group's, and `next`, the
// best other's: `off` is the largest slack of any group (a hundredth more for the rounding of these bounds).
__device__ __forceinline__ bool groups_close(float low, float next, float off)
{
    const float inf = __builtin_inff();
    return off == inf || (next > -inf && !(low - next > 2.01f * off));
}

// v of the lane that differs in the bit d (a lane of the other half of 2 d lanes, where those of a half
// are equal).
template <class V>
__device__ __forceinline__ V other_half(V v, int d)
{
    if constexpr (sizeof(V) == 8) {
        return __shfl_xor(v, d);
    } else {
        const int x = __builtin_bit_cast(int, v);
        int y;
        if (d == 1) y = __builtin_amdgcn_update_dpp(0, x, 0xb1, 0xf, 0xf, false);         // quad_perm 1 0 3 2
        else if (d == 2) y = __builtin_amdgcn_update_dpp(0, x, 0x4e, 0xf, 0xf, false);    // quad_perm 2 3 0 1
        else if (d == 4) y = __builtin_amdgcn_update_dpp(0, x, 0x141, 0xf, 0xf, false);   // row_half_mirror
        else if (d == 8) y = __builtin_amdgcn_update_dpp(0, x, 0x140, 0xf, 0xf, false);   // row_mirror
        else y = __shfl_xor(x, d);
        return __builtin_bit_cast(float, y);
    }
}
__device__ __forceinline__ float readlane(float v, int lane) { return readlane_f(v, lane); }
__device__ __forceinline__ double readlane(double v, int lane)
{
    return __builtin_bit_cast(double, readlane_u64(__builtin_bit_cast(uint64_t, v), lane));
}

// The kept groups, 2^shift lanes to a group, the bit of a group that of its first lane; at(e) is the
// value of expert e, no NaN. low, next: the last kept group's value and the first other's; off: group_slack,
// of the lane's group.
template <class V, class F>
__device__ __forceinline__ unsigned long long keep_groups(const RouteArgs &p, int per, int shift, F &&at, V &low, V &next,
                                                          float &off)
{
    const int lane = threadIdx.x & 63, g = lane >> shift, e0 = min(g, p.groups - 1) * per;
    const V none = -__builtin_inff();
    V first = none, second = none;
    for (int i = lane & ((1 << shift) - 1); i < per; i += 4 << shift) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x = i + (u << shift);
            const V v = x < per ? at(e0 + x) : none;
            second = fmax(second, fmin(first, v));
            first = fmax(first, v);
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        if (d < 1 << shift) {
            const V f = other_half(first, d), h = other_half(second, d);
            second = fmax(fmin(first, f), fmax(second, h));
            first = fmax(first, f);
        }
    const V value = p.group_top == 1 ? first : second == none ? none : first + second;
    off = group_slack(first, second, value, p.group_top == 2);
    int rank = 0;
    for (int i = 0; i < p.groups; ++i) {
        const V v = readlane(value, i << shift);
        rank += (v > value) | ((v == value) & (i < g));
    }
    const unsigned long long a = __ballot(rank == p.top_groups - 1 && g < p.groups);
    const unsigned long long b = __ballot(rank == p.top_groups && g < p.groups);
    low = a ? readlane(value, __ffsll(a) - 1) : none;
    next = b ? readlane(value, __ffsll(b) - 1) : none;
    return __ballot(g < p.groups && rank < p.top_groups);
}

// Sum of 64-bit values over the wave, in lane 63.
__device__ __forceinline__ double wave_sum64(double v)
{
    auto step = [&](auto ctrl, auto rows) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)b, decltype(ctrl)::value, decltype(rows)::value,
                                                                  0xf, false);
        const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), decltype(ctrl)::value,
                                                                  decltype(rows)::value, 0xf, false);
        v += __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    };
    step(std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());  // row_shr 1, 2, 4, 8
    step(std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());
    step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());  // row_bcast 15
    step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());  // row_bcast 31
    return v;
}

constexpr int kExact = -2;  // the token has to be done in 64 bits throughout

// Token t by one wave, `row` its LDS for E values, `bias` in LDS; lane j < k returns the expert of slot
// j (-1: none), or every lane kExact.
template <class X, int R>
__device__ __forceinline__ int route_token(const RouteArgs &p, int64_t t, const float (&l)[R], const int (&group)[R],
                                           int per, int shift, float *row, const float *bias)
{
    const int lane = threadIdx.x & 63;
    const float inf = __builtin_inff();
    const bool by_score = p.bias, sums = p.sums;
    // scores in 32 bits (softmax: without the quotient) where the choice or the sum needs them
    float m = 0.f, total32 = 1.f;
    float s[R];
    if (!p.sigmoid) {
        unsigned top = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) top = max(top, ordered32(l[r]));
        m = from_ordered32(wave_max_u32(top));
        if (m == -inf) m = 0.f;
        if (!(m < inf)) m = __builtin_nanf("");  // an infinite logit makes all scores NaN, as NaN does
    }
    const bool all_scores = !p.sigmoid && (by_score || !p.renormalize);
    double total = 1.0;
    if (by_score || sums || all_scores) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            s[r] = p.sigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-l[r])) : expf(l[r] - m);
    }
    if (all_scores) {
        if (by_score) {  // the quotient decides ranks: the sum in 64 bits
            double sum = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) sum += exp((double)l[r] - (double)m);
            total = wave_add(sum);
            total32 = (float)total;
        } else {
            float sum = s[0];
#pragma unroll
            for (int r = 1; r < R; ++r) sum += s[r];
            total = total32 = wave_sum(sum);
        }
    }
    bool exact = false;  // the token has to be done in 64 bits throughout
    float c[R];
    if (by_score) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float q = p.sigmoid ? s[r] : total32 == 0.f ? 0.f : s[r] / total32;
            const int e = lane + 64 * r;
            c[r] = l[r] == -inf || e >= p.E ? -inf : q + bias[e];
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) c[r] = l[r];
    }
    unsigned long long kept = ~0ull;  // the bit of a group: of its first lane, 2^shift lanes to a group
    if (p.groups > 1) {
        bool odd = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float v = by_score || !sums ? c[r] : l[r] == -inf ? -inf : s[r];
            odd |= !(v < inf);
            if (lane + 64 * r < p.E) row[lane + 64 * r] = v;
        }
        exact = __any(odd);
        __builtin_amdgcn_wave_barrier();
        float low, next, off;
        kept = keep_groups<float>(p, per, shift, [&](int e) { return row[e]; }, low, next, off);
        __builtin_amdgcn_wave_barrier();
        off = __builtin_bit_cast(float, wave_max_u32(__builtin_bit_cast(unsigned, off)));  // not negative
        if (!exact && p.top_groups < p.groups && (by_score || sums) && groups_close(low, next, off)) {
            // too close to tell: the same in 64 bits (softmax without a bias: without the quotient)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (lane + 64 * r < p.E) row[lane + 64 * r] = c[r] == -inf ? -inf : l[r];
            __builtin_amdgcn_wave_barrier();
            auto wide = [&](int e) {
                const double x = row[e];
                if (x == -__builtin_inf()) return x;
                double v = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)m);
                if (by_score) v = (all_scores ? total == 0 ? 0.0 : v / total : v) + (double)bias[e];
                return v;
            };
            double low64, next64;
            float none;
            kept = keep_groups<double>(p, per, shift, wide, low64, next64, none);
            __builtin_amdgcn_wave_barrier();
        }
    }
    // the picks' keys: 22 bits of c, then the lower index first; 0: not to be picked
    unsigned key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = lane + 64 * r;
        const bool live = c[r] != -inf && (p.groups == 1 || (kept >> group[r] & 1));
        key[r] = live ? (ordered32(c[r]) & ~1023u) | (unsigned)(1023 - e) : 0u;
        if (e < p.E) row[e] = l[r];
    }
    unsigned mine = 0, least = 0;
    int n = 0;
    for (; !exact; ++n) {
        unsigned best = key[0];
#pragma unroll
        for (int r = 1; r < R; ++r) best = max(best, key[r]);
        best = wave_max_u32(best);
        if (best <= least) break;  // none left, or none that could be above the k-th
        if (n == 64) {
            exact = true;
            break;
        }
        if (lane == n) mine = best;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (key[r] == best) key[r] = 0;
        if (n == p.k - 1) {
            if (by_score) {
                const float v = from_ordered32(best & ~1023u);
                exact = !(fabsf(v) < inf);
                least = (ordered32(v - 2 * slack(v)) & ~1023u) - 1;
            } else if (sizeof(X) == 2) {  // 16-bit logits are in the key whole
                ++n;
                break;
            } else {
                least = (best & ~1023u) - 1;
            }
        }
    }
    if (exact) return kExact;
    __builtin_amdgcn_wave_barrier();
    int index = lane < n ? 1023 - (int)(mine & 1023u) : -1;
    double score = 0;
    uint64_t rank_value = 0;
    if (lane < n) {
        const float x = row[index];
        score = p.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)m);
        if (all_scores) score = total == 0 ? 0.0 : score / total;
        rank_value = by_score ? ordered(score + (double)bias[index]) : (uint64_t)ordered32(x);
    }
    if (by_score || sizeof(X) == 4) {
        // in order? (32 bits almost always tell it)
        const uint64_t next = __shfl_down(rank_value, 1);
        const int next_index = __shfl_down(index, 1);
        if (__any(lane + 1 < n && (next > rank_value || (next == rank_value && next_index < index)))) {
            int place = 0;
            for (int i = 0; i < n; ++i) {
                const uint64_t v = readlane_u64(rank_value, i);
                const int e = __builtin_amdgcn_readlane(index, i);
                place += (v > rank_value) | ((v == rank_value) & (e < index));
            }
            // lane `place` takes this lane's: push
            const uint64_t bits = __builtin_bit_cast(uint64_t, score);
            const int to = 4 * (lane < n ? place : lane);
            index = __builtin_amdgcn_ds_permute(to, index);
            const unsigned lo = (unsigned)__builtin_amdgcn_ds_permute(to, (int)bits);
            const unsigned hi = (unsigned)__builtin_amdgcn_ds_permute(to, (int)(bits >> 32));
            score = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
        }
    }
    if (lane >= p.k || lane >= n) {
        index = -1;
        score = 0;
    }
    if (p.renormalize) {
        const double sum = __builtin_bit_cast(double, readlane_u64(__builtin_bit_cast(uint64_t, wave_sum64(score)), 63));
        score = sum == 0 || index < 0 ? 0.0 : score / sum;
    }
    if (lane < p.k) {
        p.weights[t * p.k + lane] = (float)(score * (double)p.scale);
        p.experts[t * p.k + lane] = index;
    }
    return index;
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

// p.tokens tokens: weights and experts; rows: each slot's number among the workgroup's of its expert; the
// experts' counts. ALL: the only workgroup, which finishes rows and offsets.
template <class X, int R, bool ALL>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs p)
{
    __shared__ unsigned mask[64 * R][2];  // the tokens that take an expert
    __shared__ short slot[kTokens * kRouteMaxTop];
    __shared__ float rows[kWaves][64 * R], bias[64 * R];
    __shared__ unsigned first[64 * R], part[kWaves];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, e = threadIdx.x;
    const int64_t t0 = linear_block() * p.tokens;
    if (t0 >= p.T) return;  // the whole workgroup
    if (e < 64 * R) {
        mask[e][0] = mask[e][1] = 0;
        bias[e] = p.bias && e < p.E ? p.bias[e] : 0.f;
    }
    __syncthreads();
    int group[R], shift = 0;  // the bit of an expert's group
    const int per = __builtin_amdgcn_readfirstlane(p.E / p.groups);
    while (2 * p.groups << shift <= 64) ++shift;
#pragma unroll
    for (int r = 0; r < R; ++r) group[r] = p.groups == 1 ? 0 : min((lane + 64 * r) / per, p.groups - 1) << shift;
    float l[R], ahead[R];
    auto load = [&](int t, float (&x)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = lane + 64 * r;
            x[r] = t < p.tokens && t0 + t < p.T && i < p.E ? load_logit<X>(p.logits, (t0 + t) * p.ld + i) : -__builtin_inff();
        }
    };
    auto keep = [&](int t, int chosen) {
        if (lane < p.k) {
            slot[t * p.k + lane] = (short)chosen;
            if (chosen >= 0) atomicOr(&mask[chosen][t >> 5], 1u << (t & 31));
        }
    };
    unsigned again = 0;  // of this wave's tokens, those to be done in 64 bits
    load(w, ahead);
    for (int i = 0; i < p.tokens / kWaves; ++i) {
        const int t = w + kWaves * i;
        if (t0 + t >= p.T) break;
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = ahead[r];
        load(t + kWaves, ahead);
        const int chosen = route_token<X, R>(p, t0 + t, l, group, per, shift, rows[w], bias);
        if (__builtin_amdgcn_readfirstlane(chosen) == kExact) again |= 1u << i;
        else keep(t, chosen);
    }
    for (int i = 0; again >> i; ++i)
        if (again >> i & 1) keep(w + kWaves * i, route_token_exact<X, R>(p, t0 + w + kWaves * i));
    __syncthreads();
    const unsigned count = e < p.E ? __popc(mask[e][0]) + __popc(mask[e][1]) : 0;
    if constexpr (ALL) {
        unsigned total;
        const unsigned at = block_scan<kWaves>(count, part, total);
        if (e < p.E) {
            first[e] = at;
            p.offsets[e] = at;
        }
        if (e == 0) p.offsets[p.E] = total;
        __syncthreads();
    } else if (e < p.E) {
        p.ws[linear_block() * p.E + e] = (int)count;
    }
    const int slots = (int)min((int64_t)p.tokens, p.T - t0) * p.k;
    for (int i = threadIdx.x; i < slots; i += 64 * kWaves) {
        const int x = slot[i], t = i / p.k;
        int row = -1;
        if (x >= 0) {
            row = t < 32 ? __popc(mask[x][0] & ((1u << t) - 1))
                         : __popc(mask[x][0]) + __popc(mask[x][1] & ((1u << (t - 32)) - 1));
            if (ALL) row += (int)first[x];
        }
        p.rows[t0 * p.k + i] = row;
    }
}

// ------------------------------------------------------------ four tokens to a wave
//
// Up to 256 experts, 12 of them chosen and 16 groups: a token takes a row of 16 lanes, lane q its experts
// q + 16 r, so that what is done for a token with one instruction is done for four, and maxima need four
// steps. The same steps as route_token; up to 16 candidates.
constexpr int kRowExperts = 256, kRowTop = 12, kRowGroups = 16;

// v of the lane I before this one in the row, in a circle.
template <int I>
__device__ __forceinline__ unsigned rotate(unsigned v)
{
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + I, 0xf, 0xf, false);  // row_ror
}
template <int I>
__device__ __forceinline__ float rotate(float v)
{
    return __builtin_bit_cast(float, rotate<I>(__builtin_bit_cast(unsigned, v)));
}
template <int I>
__device__ __forceinline__ uint64_t rotate(uint64_t v)
{
    return (uint64_t)rotate<I>((unsigned)(v >> 32)) << 32 | rotate<I>((unsigned)v);
}
template <int I>
__device__ __forceinline__ double rotate(double v)
{
    return __builtin_bit_cast(double, rotate<I>(__builtin_bit_cast(uint64_t, v)));
}
// f(I) for I = 1 .. 15.
template <int I = 1, class F>
__device__ __forceinline__ void each_other(F &&f)
{
    f(std::integral_constant<int, I>());
    if constexpr (I < 15) each_other<I + 1>(f);
}
// Maximum and sum of the row, in all its lanes.
__device__ __forceinline__ unsigned row_max(unsigned v)
{
    v = max(v, rotate<8>(v));
    v = max(v, rotate<4>(v));
    v = max(v, rotate<2>(v));
    return max(v, rotate<1>(v));
}
template <class V>
__device__ __forceinline__ V row_sum(V v)
{
    v += rotate<8>(v);
    v += rotate<4>(v);
    v += rotate<2>(v);
    return v + rotate<1>(v);
}

// As keep_groups, for each row's token; the bits of a group's lanes in the row.
template <class V, class F>
__device__ __forceinline__ unsigned row_keep_groups(const RouteArgs &p, int per, int shift, F &&at, V &value, int &rank,
                                                    float &off)
{
    const int lane = threadIdx.x & 63, q = lane & 15, g = q >> shift, e0 = min(g, p.groups - 1) * per;
    const V none = -__builtin_inff();
    V first = none, second = none;
    for (int i = q & ((1 << shift) - 1); i < per; i += 4 << shift) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x = i + (u << shift);
            const V v = x < per ? at(e0 + x) : none;
            second = fmax(second, fmin(first, v));
            first = fmax(first, v);
        }
    }
#pragma unroll
    for (int d = 1; d < 16; d *= 2)
        if (d < 1 << shift) {
            const V f = other_half(first, d), h = other_half(second, d);
            second = fmax(fmin(first, f), fmax(second, h));
            first = fmax(first, f);
        }
    value = p.group_top == 1 ? first : second == none ? none : first + second;
    off = group_slack(first, second, value, p.group_top == 2);
    int above = 0;  // lanes of better groups
    each_other([&](auto i) {
        constexpr int I = decltype(i)::value;
        const V v = rotate<I>(value);
        const int of = (int)rotate<I>((unsigned)g);
        above += (of < p.groups) & ((v > value) | ((v == value) & (of < g)));  // no branches
    });
    rank = above >> shift;
    return (unsigned)(__ballot(g < p.groups && rank < p.top_groups) >> (lane & 48)) & 0xffffu;
}

template <class X, int R, int W, bool ALL>
__global__ __launch_bounds__(64 * W) void route_rows_of_16_kernel(RouteArgs p)
{
    constexpr int tokens = 4 * W;
    static_assert(tokens <= 64 && 16 * R <= 64 * W, "a mask's bits; a thread for each expert");
    __shared__ unsigned mask[16 * R][2];  // the tokens that take an expert
    __shared__ short slot[tokens * kRowTop];
    __shared__ float rows[tokens][16 * R];
    __shared__ unsigned first[16 * R], part[W];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, q = lane & 15, tid = threadIdx.x;
    const int64_t t0 = linear_block() * tokens;
    if (t0 >= p.T) return;  // the whole workgroup
    if (tid < 16 * R) mask[tid][0] = mask[tid][1] = 0;
    const int token = 4 * w + (lane >> 4);  // in the workgroup
    const int64_t t = t0 + token;
    const float inf = __builtin_inff();
    float *row = rows[token];

    const bool by_score = p.bias, sums = p.sums;
    float l[R], c[R];
#pragma unroll
    for (int r = 0; r < R; ++r)  // no branches: the last one's in the place of others
        l[r] = load_logit<X>(p.logits, min(t, (int64_t)p.T - 1) * p.ld + min(q + 16 * r, p.E - 1));
    float bias[R];
    if (by_score) {
#pragma unroll
        for (int r = 0; r < R; ++r) bias[r] = p.bias[min(q + 16 * r, p.E - 1)];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (t >= p.T || q + 16 * r >= p.E) l[r] = -inf;
    float m = 0.f, total32 = 1.f;
    double total = 1.0;
    if (!p.sigmoid) {
        unsigned top = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) top = max(top, ordered32(l[r]));
        m = from_ordered32(row_max(top));
        if (m == -inf) m = 0.f;
        if (!(m < inf)) m = __builtin_nanf("");
    }
    const bool all_scores = !p.sigmoid && (by_score || !p.renormalize);
    float s[R];
    if (by_score || sums || all_scores) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            s[r] = p.sigmoid ? __builtin_amdgcn_rcpf(1.f + __expf(-l[r])) : expf(l[r] - m);
    }
    if (all_scores) {
        if (by_score) {
            double sum = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) sum += exp((double)l[r] - (double)m);
            total = row_sum(sum);
            total32 = (float)total;
        } else {
            float sum = s[0];
#pragma unroll
            for (int r = 1; r < R; ++r) sum += s[r];
            total = total32 = row_sum(sum);
        }
    }
    if (by_score) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float score = p.sigmoid ? s[r] : total32 == 0.f ? 0.f : s[r] / total32;
            c[r] = l[r] == -inf ? -inf : score + bias[r];
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) c[r] = l[r];
    }
    bool exact = false;  // the same in a row's lanes, like all below
    unsigned kept = 0xffffu;
    int shift = 0, per = p.E;
    unsigned inverse = 0;  // e / per = e inverse >> 16: e < 256 times less than 1 too much is below 2^16 / per
    if (p.groups > 1) {
        per = __builtin_amdgcn_readfirstlane(p.E / p.groups);
        inverse = __builtin_amdgcn_readfirstlane((65535 + per) / per);
        while (2 * p.groups << shift <= 16) ++shift;
        bool odd = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float v = by_score || !sums ? c[r] : l[r] == -inf ? -inf : s[r];
            odd |= !(v < inf);
            row[q + 16 * r] = v;
        }
        exact = (__ballot(odd) >> (lane & 48) & 0xffffu) != 0;
        __builtin_amdgcn_wave_barrier();
        float value, off;
        int rank;
        kept = row_keep_groups<float>(p, per, shift, [&](int e) { return row[e]; }, value, rank, off);
        __builtin_amdgcn_wave_barrier();
        if (p.top_groups < p.groups && (by_score || sums)) {
            const float low = from_ordered32(row_max(rank == p.top_groups - 1 && q >> shift < p.groups ? ordered32(value) : 0u));
            const float next = from_ordered32(row_max(rank == p.top_groups && q >> shift < p.groups ? ordered32(value) : 0u));
            off = __builtin_bit_cast(float, row_max(__builtin_bit_cast(unsigned, off)));  // not negative
            const bool close = !exact && groups_close(low, next, off);
            if (__any(close)) {
#pragma unroll
                for (int r = 0; r < R; ++r) row[q + 16 * r] = c[r] == -inf ? -inf : l[r];
                __builtin_amdgcn_wave_barrier();
                auto wide = [&](int e) {
                    const double x = row[e];
                    if (x == -__builtin_inf()) return x;
                    double v = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)m);
                    if (by_score) v = (all_scores ? total == 0 ? 0.0 : v / total : v) + (double)p.bias[e];
                    return v;
                };
                double value64;
                int rank64;
                float none;
                const unsigned kept64 = row_keep_groups<double>(p, per, shift, wide, value64, rank64, none);
                __builtin_amdgcn_wave_barrier();
                if (close) kept = kept64;
            }
        }
    }
    unsigned key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e = q + 16 * r;
        bool live = c[r] != -inf;
        if (p.groups > 1) live &= (kept >> ((e * inverse >> 16) << shift & 31) & 1) != 0;
        key[r] = live ? (ordered32(c[r]) & ~1023u) | (unsigned)(1023 - e) : 0u;
        row[e] = l[r];
    }
    unsigned mine = 0, least = 0;
    int n = 0;  // picks of the row's token
    for (int i = 0;; ++i) {
        unsigned best = key[0];
#pragma unroll
        for (int r = 1; r < R; ++r) best = max(best, key[r]);
        best = row_max(best);
        const bool live = best > least && !exact;
        if (!__any(live)) break;
        if (i == 16) {
            exact |= live;
            break;
        }
        if (live) {
            if (q == i) mine = best;
            n = i + 1;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (key[r] == best) key[r] = 0;
        if (i == p.k - 1) {
            if (by_score) {
                const float v = from_ordered32(best & ~1023u);
                exact |= live && !(fabsf(v) < inf);
                least = live ? (ordered32(v - 2 * slack(v)) & ~1023u) - 1 : ~0u;
            } else if (sizeof(X) == 2) {
                break;
            } else {
                least = live ? (best & ~1023u) - 1 : ~0u;
            }
        }
    }
    __builtin_amdgcn_wave_barrier();
    const bool has = q < n;
    int index = has ? 1023 - (int)(mine & 1023u) : -1;
    double score = 0;
    uint64_t rank_value = 0;
    if (has) {
        const float x = row[index];
        score = p.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)m);
        if (all_scores) score = total == 0 ? 0.0 : score / total;
        rank_value = by_score ? ordered(score + (double)p.bias[index]) : (uint64_t)ordered32(x);
    }
    if (by_score || sizeof(X) == 4) {
        const uint64_t next = rotate<15>(rank_value);  // of the lane after this one
        const int next_index = (int)rotate<15>((unsigned)index);
        if (__any((q + 1 < n) & ((next > rank_value) | ((next == rank_value) & (next_index < index))))) {
            int place = 0;
            each_other([&](auto i) {
                constexpr int I = decltype(i)::value;
                const uint64_t v = rotate<I>(rank_value);
                const int e = (int)rotate<I>((unsigned)index);
                place += (e >= 0) & ((v > rank_value) | ((v == rank_value) & (e < index)));
            });
            const uint64_t bits = __builtin_bit_cast(uint64_t, score);
            const int to = 4 * ((lane & 48) | (has ? place : q));
            index = __builtin_amdgcn_ds_permute(to, index);
            const unsigned lo = (unsigned)__builtin_amdgcn_ds_permute(to, (int)bits);
            const unsigned hi = (unsigned)__builtin_amdgcn_ds_permute(to, (int)(bits >> 32));
            score = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
        }
    }
    if (q >= p.k || q >= n) {
        index = -1;
        score = 0;
    }
    if (p.renormalize) {
        const double sum = row_sum(score);
        score = sum == 0 || index < 0 ? 0.0 : score / sum;
    }
    __syncthreads();  // the masks are clear
    auto keep = [&](int of, int j, int chosen) {
        slot[of * kRowTop + j] = (short)chosen;
        if (chosen >= 0) atomicOr(&mask[chosen][of >> 5], 1u << (of & 31));
    };
    if (q < p.k && t < p.T && !exact) {
        p.weights[t * p.k + q] = (float)(score * (double)p.scale);
        p.experts[t * p.k + q] = index;
        keep(token, q, index);
    }
    const unsigned long long again = __ballot(exact && t < p.T);
    for (int i = 0; i < 4; ++i)
        if (again >> (16 * i) & 1) {
            const int chosen = route_token_exact<X, (R + 3) / 4>(p, t0 + 4 * w + i);
            if (lane < p.k) keep(4 * w + i, lane, chosen);
        }
    __syncthreads();
    const unsigned count = tid < p.E ? __popc(mask[tid][0]) + __popc(mask[tid][1]) : 0;
    if constexpr (ALL) {
        unsigned all;
        const unsigned at = block_scan<W>(count, part, all);
        if (tid < p.E) {
            first[tid] = at;
            p.offsets[tid] = at;
        }
        if (tid == 0) p.offsets[p.E] = all;
        __syncthreads();
    } else if (tid < p.E) {
        p.ws[linear_block() * p.E + tid] = (int)count;
    }
    if (q < p.k && t < p.T) {
        const int x = slot[token * kRowTop + q];
        int r = -1;
        if (x >= 0) {
            r = token < 32 ? __popc(mask[x][0] & ((1u << token) - 1))
                           : __popc(mask[x][0]) + __popc(mask[x][1] & ((1u << (token - 32)) - 1));
            if (ALL) r += (int)first[x];
        }
        p.rows[t * p.k + q] = r;
    }
}

// The workgroups' counts of an expert -> those of the workgroups before; the experts' totals behind them.
// A workgroup takes 64 experts, 16 threads each.
__global__ __launch_bounds__(1024) void route_scan_kernel(RouteArgs p, int blocks)
{
    __shared__ unsigned sums[16][64];
    const int x = threadIdx.x & 63, q = threadIdx.x >> 6, e = blockIdx.x * 64 + x;
    const bool live = e < p.E;
    constexpr int U = 16;
    const int each = (blocks + 15) / 16, lo = min(q * each, blocks), hi = min(lo + each, blocks);
    unsigned v[U], sum = 0;
    auto load = [&](int b) {
#pragma unroll
        for (int i = 0; i < U; ++i) v[i] = live && b + i < hi ? (unsigned)p.ws[(int64_t)(b + i) * p.E + e] : 0u;
    };
    for (int b = lo; b < hi; b += U) {
        load(b);
#pragma unroll
        for (int i = 0; i < U; ++i) sum += v[i];
    }
    sums[q][x] = sum;
    __syncthreads();
    unsigned at = 0, all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        at += i < q ? sums[i][x] : 0;
        all += sums[i][x];
    }
    if (!live) return;
    if (q == 0) p.ws[(int64_t)blocks * p.E + e] = (int)all;
    for (int b = lo; b < hi; b += U) {
        if (each > U) load(b);  // else they are still there
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (b + i < hi) p.ws[(int64_t)(b + i) * p.E + e] = (int)at;
            at += v[i];
        }
    }
}

// A workgroup's tokens: rows from their numbers in it; offsets. FEW: the counts as route_kernel left
// them, else as the scan did.
template <bool FEW>
__global__ __launch_bounds__(1024) void route_rows_kernel(RouteArgs p, int blocks)
{
    __shared__ unsigned first[kRouteMaxExperts], part[16];
    const int64_t bid = linear_block();
    if (bid >= blocks) return;
    const int e = threadIdx.x;
    const int64_t s0 = bid * p.tokens * p.k;
    const int slots = (int)min((int64_t)p.tokens * p.k, (int64_t)p.T * p.k - s0);
    // the first slot of this thread, loaded ahead
    int x = -1, row = -1;
    if (e < slots) {
        x = p.experts[s0 + e];
        row = p.rows[s0 + e];
    }
    unsigned all = 0, before = 0;
    if (e < p.E) {
        if constexpr (FEW) {
#pragma unroll
            for (int b = 0; b < kFewBlocks; ++b) {
                const unsigned v = b < blocks ? (unsigned)p.ws[b * p.E + e] : 0u;
                before += b < bid ? v : 0u;
                all += v;
            }
        } else {
            before = (unsigned)p.ws[bid * p.E + e];
            all = (unsigned)p.ws[(int64_t)blocks * p.E + e];
        }
    }
    unsigned total;
    const unsigned at = block_scan<16>(all, part, total);
    if (e < p.E) {
        first[e] = at + before;
        if (bid == 0) p.offsets[e] = at;
    }
    if (bid == 0 && e == 0) p.offsets[p.E] = total;
    __syncthreads();
    if (x >= 0) p.rows[s0 + e] = row + (int)first[x];
    for (int i = e + 1024; i < slots; i += 1024) {
        const int y = p.experts[s0 + i];
        if (y >= 0) p.rows[s0 + i] += (int)first[y];
    }
}

// dl_e of one token by one wave: with g_e the gradient of s_e (0 where e was not chosen),
// softmax s_e (g_e - sum over i of s_i g_i), sigmoid s_e (1 - s_e) g_e. For w_j = scale s_j, g = scale dw.
// Renormalised, with S the sum of the chosen s and shares r_j = s_j / S: g_j = scale / S (dw_j - sum_i dw_i r_i),
// so that softmax's sum of s g vanishes and s_j g_j = scale r_j (dw_j - sum_i dw_i r_i). The shares are the
// weights that the token got, taken in 64 bits as there: the chosen s may be far below fp32's smallest.
template <class X, int R>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs p)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = linear_block() * 4 + (threadIdx.x >> 6);
    if (t >= p.T) return;
    float l[R], s[R], g[R];
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
    if (!p.sigmoid) {
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
        if (m == -__builtin_inff()) m = 0;
        if (__any(nan) || !(m < __builtin_inff())) m = __builtin_nanf("");  // all scores are NaN
    }
    // lane j: slot j
    int e = lane < p.k ? p.experts[t * p.k + lane] : -1;
    if (e < 0 || e >= p.E) e = -1;
    float dw = e >= 0 ? p.scale * p.dweights[t * p.k + lane] : 0.f;
    float rest = 0;  // softmax: what the sum of s g leaves to the experts not chosen, 0 or NaN
    if (p.renormalize) {
        const float x = e >= 0 ? load_logit<X>(p.logits, t * p.ld + e) : 0.f;
        const double score = e < 0 ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)m);
        const double total = wave_add(score);
        const float share = total == 0 ? 0.f : (float)(score / total);
        const float mean = total == 0 ? 0.f : wave_add(dw * share);
        const float q = expf(-fabsf(x)), not_s = x < 0 ? 1.f / (1.f + q) : q / (1.f + q);
        dw = total == 0 || e < 0 ? 0.f : share * (dw - mean) * (p.sigmoid ? not_s : 1.f);
        rest = p.sigmoid ? 0.f : 0.f * fabsf(mean) + 0.f * m;
    }
    for (int j = 0; j < p.k; ++j) {
        const int of = __shfl(e, j);
        const float v = __shfl(dw, j);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (of == lane + 64 * r) g[r] += v;
    }
    if (p.renormalize) {
#pragma unroll
        for (int r = 0; r < R; ++r) g[r] = l[r] != l[r] ? l[r] : g[r] + rest;
    } else if (p.sigmoid) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float q = expf(-fabsf(l[r])), n = 1.f / (1.f + q);
            g[r] *= q * n * n;
        }
    } else {
        float sum = 0, dot = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = lane + 64 * r < p.E ? expf(l[r] - m) : 0.f;
            sum += s[r];
        }
        sum = wave_add(sum);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = sum == 0 ? 0.f : s[r] / sum;
            dot = fmaf(s[r], g[r], dot);
        }
        dot = wave_add(dot);
#pragma unroll
        for (int r = 0; r < R; ++r) g[r] = s[r] * (g[r] - dot);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = lane + 64 * r;
        if (i < p.E) static_cast<X *>(p.dlogits)[t * p.ldd + i] = (X)g[r];
    }
}

// f(X()) with the type of number t (MM_TYPE_*).
template <class F>
void with_type(int t, F &&f)
{
    if (t == 0) f(float());
    else if (t == 1) f(__bf16());
    else f(_Float16());
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

// Whether a call takes four tokens to a wave.
static bool rows_of_16(int64_t E, int64_t k, int64_t groups) { return E <= kRowExperts && k <= kRowTop && groups <= kRowGroups; }

// Tokens of a workgroup. Four to a wave: 4 waves, so that more CUs take part, or 16 where all of them have
// work. Else one to a wave of 16, or four after each other (4001 tokens of 60 experts one by one: 15 us with
// 64 to a workgroup, 7 with 16). One workgroup saves a launch, which pays up to 64 tokens of at most 128
// experts (both kernels against one, in a graph: 32 of 64 experts 7.2 and 5.9 us, 64 of 128 8.5 and 9.2, 64 of
// 256 10.5 and 13.4, in groups 13.2 and 17.9).
static int tokens_of(int64_t T, int64_t E, int64_t k, int64_t groups)
{
    if (rows_of_16(E, k, groups)) return T <= 16 || (T <= 8192 && (T > 64 || E > 128)) ? 16 : 64;
    return T <= 32 || T > 8192 ? kTokens : kWaves;
}

int64_t route_ws_ints(int64_t T, int E, int k)
{
    int64_t ints = 0;  // the caller's groups may allow either
    for (int groups : {1, kRowGroups + 1}) {
        const int64_t tokens = tokens_of(T, E, k, groups), blocks = (T + tokens - 1) / tokens;
        const int64_t need = blocks > 1 ? (blocks + 1) * E : 0;
        ints = need > ints ? need : ints;
    }
    return ints;
}

hipError_t route_launch(const RouteArgs &a, hipStream_t stream)
{
    RouteArgs arg = a;
    arg.sums = a.groups > 1 && a.group_top == 2;
    arg.group_top = a.group_top < a.E / a.groups ? a.group_top : a.E / a.groups;  // a group's only expert: its own
    arg.tokens = tokens_of(a.T, a.E, a.k, a.groups);
    int blocks = (int)(((int64_t)a.T + arg.tokens - 1) / arg.tokens);
    unsigned gx, gy;
    if (!grid_for(blocks, gx, gy)) return hipErrorInvalidConfiguration;
    void *args[] = {&arg};
    const void *fn = nullptr;
    int threads = 64 * kWaves;
    if (rows_of_16(a.E, a.k, a.groups)) {
        threads = 16 * arg.tokens;
        with_type(a.type, [&](auto x) {
            auto sized = [&](auto r) {
                typedef decltype(x) X;
                constexpr int R = decltype(r)::value;
                if (arg.tokens == 16)
                    fn = blocks == 1 ? reinterpret_cast<const void *>(&route_rows_of_16_kernel<X, R, 4, true>)
                                     : reinterpret_cast<const void *>(&route_rows_of_16_kernel<X, R, 4, false>);
                else
                    fn = blocks == 1 ? reinterpret_cast<const void *>(&route_rows_of_16_kernel<X, R, 16, true>)
                                     : reinterpret_cast<const void *>(&route_rows_of_16_kernel<X, R, 16, false>);
            };
            if (a.E <= 64) sized(std::integral_constant<int, 4>());
            else if (a.E <= 128) sized(std::integral_constant<int, 8>());
            else sized(std::integral_constant<int, 16>());
        });
    } else {
        (void)with_route(a.type, a.E, [&](auto x, auto r) {
            typedef decltype(x) X;
            constexpr int R = decltype(r)::value;
            fn = blocks == 1 ? reinterpret_cast<const void *>(&route_kernel<X, R, true>)
                             : reinterpret_cast<const void *>(&route_kernel<X, R, false>);
            return hipSuccess;
        });
    }
    hipError_t e = hipLaunchKernel(fn, dim3(gx, gy), dim3(threads), args, 0, stream);
    if (e != hipSuccess || blocks == 1) return e;
    void *more[] = {&arg, &blocks};
    const bool few = blocks <= kFewBlocks;
    if (!few) {
        e = hipLaunchKernel(reinterpret_cast<const void *>(&route_scan_kernel), dim3((a.E + 63) / 64), dim3(1024), more, 0,
                            stream);
        if (e != hipSuccess) return e;
    }
    return hipLaunchKernel(few ? reinterpret_cast<const void *>(&route_rows_kernel<true>)
                               : reinterpret_cast<const void *>(&route_rows_kernel<false>),
                           dim3(gx, gy), dim3(1024), more, 0, stream);
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
