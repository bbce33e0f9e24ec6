// mm_group_tile.hip -- large tiles of the grouped products and of the 8-bit integer and 4-bit products
// (see mm_group.h for the sums), with panels moved HBM -> LDS by the LDS DMA.
//
// A group of waves computes a BM x BN tile of C (256 x 256 or 128 x 128 on 8 waves, 64 x 64 on 2;
// of the last, 2 or 4 groups in a workgroup share one tile's sums) in K-steps of 128 bytes of k (64
// 16-bit or 128 8-bit elements; v_mfma_*_16x16x* takes 64 bytes of k at once, 2 steps of it). The
// tile is four quadrants of RH x CH (halves lo, hi of its rows and columns); the waves stand in a
// GM x GN grid over each quadrant (2 x 4, 4 x 2 and 2 x 1), so a wave owns a QM x QN part of all
// four. A K-step is four phases, one quadrant each; every phase multiplies operands that are in
// registers and reads the half panel that a phase after it needs from LDS, between its MFMAs:
//   phase 0  A lo x B lo    reads B hi
//   phase 1  A lo x B hi    reads A hi
//   phase 2  A hi x B hi    reads A lo of the next K-step
//   phase 3  A hi x B lo    reads B lo of the next K-step, into the registers of B hi
// so each half panel is read from LDS once per K-step and wave, and the reads are spread evenly. A
// tile whose second half of rows holds none of C (the last of a group, often) goes without A hi:
//   phase 0  A lo x B lo    reads B hi
//   phase 1  A lo x B hi    reads A lo and B lo of the next K-step, A lo into the registers of A hi
//
// LDS holds two K-steps as half panels. The buffer of a half panel is free once every wave has
// read it; the DMA for the same half two K-steps on goes out one phase later, so six half panels
// are on their way while one is read. A phase has one barrier, a few MFMAs into it: before it a
// wave waits until its own loads of the half panel to be read have landed (vmcnt) and until its
// reads of the phase before are done (lgkmcnt), so that after it both hold for every wave.
//
// Operand layouts in LDS. k along the operand's rows ("D"): rows of 128 bytes, 16-byte chunk c of
// row r in slot c ^ swz(r), an MFMA operand is one 16-byte read. k across the rows ("T": B stored
// K x N, and both operands of the gradient): BK rows of 2 RH (2 CH) bytes as stored, an operand is
// two ds_read_b64_tr_b16 (which transpose 16 x 4 blocks within 16 lanes: lane i receives column i
// of the four rows that lanes 4c .. 4c + 3 addressed).
//
// Edges. Rows of A past the group's end, and rows of a D operand B past N, are clamped to the last
// one; they feed only elements that are not stored. The columns of a T operand that crosses the
// matrix' edge start earlier instead (every 16-byte chunk inside its row; elements of C left of the
// tile's origin belong to the tile before and are not stored again), or, with fewer columns than
// the tile, clamp to the row's last 16 bytes: the last chunk is moved back by what it would have
// crossed, and so are its elements of C, those that the chunk before holds too not being stored
// again. A partial K-step is run first and ends at the last k: it shares its first `ov` k with the
// next step (or, in a group of fewer rows than a K-step, reads rows before the group), and both
// panels are zeroed there once they have landed, so that those k add 0 x 0 whatever the memory
// holds. Outside the gradient a K below one K-step starts at k = 0, and its last, partial chunk
// ends at the last k instead: the k that it shares with the chunk before are zeroed, and all chunks
// after it.
//
// Bound by the matrix cores at the clock the power limit leaves (1.64-1.7 GHz; MFMAs busy 67% of it in
// i8 8192 x 14336 x 4096 and 75% in 8 bf16 experts of 14336 x 4096, 52-63% in a training batch's
// gradients and 8-bit experts, whose last rounds are uneven; no LDS bank conflicts). 256 x 256, one
// workgroup per CU: 1.35 us per K-step and round of 256 tiles; bf16 8192 x 14336 x 4096 682 us (1411
// TFLOP/s), i8 368-371 us (2.6 POP/s; medians of calls in a row, single runs 362-410; 435-458 in short
// runs under the profiler). 128 x 128, two per CU, for fewer tiles: i8 1000 x 1531 x 777 12 us. With
// fewer tiles than CUs a tile's panels bound it, which one CU takes from L2 at about 100 GB/s: 64 x 64
// tiles spread them over four times the CUs, and the groups of a workgroup keep enough loads on their
// way (operands in the caches, bf16 128 x 4096 x 4096 27.1 us in 128 x 128 tiles, 16.6 in 64 x 64; 256 x
// 2048 x 4096 26.9 and 14.8; two groups to a 128 x 128 tile no faster than one). Against that, same
// shapes: 32 x 32 MFMAs instead of 16 x 16 8-15% slower (they pass twice the accumulator bytes per
// product); 4 waves of 128 x 128 the same with 32 x 32 MFMAs; a phase's reads in front of its MFMAs 5-8%
// slower; workgroups that stay and load their next tile during the stores -1.7% to +8.6%.
//
// 4-bit elements (two to a byte, so a K-step is 256 of them, one 32-element block to a 16-byte chunk) take
// the same tiles with other phases (phase_mx), since their scales need registers too, and
// v_mfma_scale_f32_16x16x128, 10.3 ns of a SIMD against 7.8 for i8's of the same bytes. 8192 x 14336 x 4096:
// 255-276 us in long runs, 3.5-3.8 PFLOP/s (290-330, 2.9-3.3, in the first 40 calls after a pause, until the
// clock has settled), 230 registers, MFMAs busy 44% of the cycles at 1.7-2 GHz. Taken apart, of 255 us: without
// the scales' loads 9 us less, without spreading them to lanes another 16, without reading them 4, and with no
// loads at all 217 us. Of these the MFMAs alone are 148; an 8-wave tile's K-step also moves 192 KB of operands
// from LDS and 64 KB into it, 2048 cycles at 128 bytes each, as many as its MFMAs take, and the two overlap in
// part only. (32 x 32 x 64 MFMAs: 9% fewer cycles at a clock 8% lower, the same time.)
#include "mm_group.h"

namespace mm {
namespace {

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

template <class E_, bool AT_, bool BT_, int RH_, int CH_, int GM_, int GN_>
struct GroupTile {
    typedef E_ E;
    static constexpr bool AT = AT_, BT = BT_;
    static constexpr int RH = RH_, CH = CH_, GM = GM_, GN = GN_, BM = 2 * RH, BN = 2 * CH;
    static constexpr int WAVES = GM * GN, NT = 64 * WAVES;
    static constexpr int QM = RH / GM, QN = CH / GN;
    static constexpr int MB = 16, FM = QM / MB, FN = QN / MB;  // MFMA blocks of a wave's part
    static constexpr int KS = 2, ACC = 4;  // MFMA steps per K-step, values per lane and block
    static constexpr int ES = sizeof(typename E::T), BK = 128 / ES;
    static constexpr int A_HALF = RH * 128, B_HALF = CH * 128;  // bytes of a half panel
    static constexpr int STAGE = 2 * (A_HALF + B_HALF);
    // Mx4: the scales of two K-steps, 16 bytes of every row of B and A, come in one load per wave and lane,
    // with the first half panel of the even one. (8 bytes for each K-step: every 128-byte line of them
    // read twice as often, which took i8's 233 us for the same bytes of k to 373.)
    static constexpr bool MX = is_mx<E>;
    static constexpr int SC_PAIR = MX ? 16 * (BN + BM) : 0;  // bytes of LDS, two of them
    static constexpr int SC_SEGMENTS = (BN + BM) / 64;       // 64 rows each
    static_assert(!MX || SC_SEGMENTS <= WAVES, "one load brings all rows' scales");
    // Few blocks of A: a lane reads its row's 8 scale bytes itself for every block, and picks its own; else 64
    // rows are read at once and spread over the lanes (scales_of_lane). Words of a half's scales of A and B.
    static constexpr bool DIRECT = FM <= 2;
    static constexpr int SAW = DIRECT ? FM : 2, SBW = DIRECT ? FN : 1;
    static constexpr int GROUP_LDS = 2 * (STAGE + SC_PAIR);  // of a group of waves
    static constexpr int A_LD = A_HALF / 1024 / WAVES, B_LD = B_HALF / 1024 / WAVES;  // 1 KB loads per wave
    // offsets of the half panels in a stage
    static constexpr int A_OFF[2] = {0, A_HALF}, B_OFF[2] = {2 * A_HALF, 2 * A_HALF + B_HALF};
    static_assert(A_LD >= 1 && B_LD >= 1 && A_HALF % (1024 * WAVES) == 0 && B_HALF % (1024 * WAVES) == 0, "whole loads");
    static_assert(QM % MB == 0 && QN % MB == 0, "whole blocks");
    static_assert(GROUP_LDS <= 160 * 1024, "two stages in LDS");
    static constexpr bool SPLIT = RH == 128;  // one workgroup per CU: the last round's tiles may be split
    static_assert(FN == 2, "the epilogue exchanges two 16 x 16 blocks side by side");
    static_assert(!(AT || BT) || ES == 2, "transposed reads of 16-bit elements");
};

// D rows of 128 bytes: the 8 slots of one chunk over any 8 (16 on 64 banks) rows are distinct.
__device__ __forceinline__ int swz_d(int row) { return ((row >> 1) & 7) ^ ((row & 1) << 2); }

// T rows of W columns (2 W bytes): a transposed read touches 64 bytes of four consecutive rows (and
// of four more 8 rows on); XOR-ing the chunk index spreads them over the bank quarters. Rows of 128
// bytes (W = 64) span two quarters, chosen by the row's parity already; rows of 64 bytes (W = 32) all
// four.
template <int W>
__device__ __forceinline__ int swz_t(int krow)
{
    static_assert(W == 32 || W == 64 || W == 128, "rows of 4, 8 or 16 chunks: the permuted index stays inside the row");
    if constexpr (W == 32) return ((krow >> 3) & 1) * 2;
    else if constexpr (W == 64) return ((krow >> 1) & 1) * 4 ^ ((krow >> 3) & 1) * 2;
    else return (krow & 3) * 4 ^ ((krow >> 3) & 1) * 2;
}

// 16 bytes per lane from base + voff into LDS at lds_addr + 16 lane (lds_addr, base wave-uniform).
// The s_nop is the wait state that a load with LDS needs after the write of M0.
__device__ __forceinline__ void dma16(unsigned lds_addr, const void *base, unsigned voff)
{
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds_addr) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A lane's scale bytes as the MFMA takes them. `raw`: the 8 scale bytes (chunk c of the K-step in byte
// c) of the row that lane 16 s + r reads its operands' row r from in block s, s < 4. The operand of
// block i and MFMA step ks in lane 16 g + r is chunk 4 ks + g of row r; its scale becomes byte
// 2 (i / 2) + ks of word i % 2 (of B's two blocks: byte 2 i + ks of one word). Bytes change places with
// 16-lane rows in two steps: the 16-bit halves between the halves of the wave, then the bytes between
// neighbouring rows.
template <int W>
__device__ __forceinline__ void scales_of_lane(u32x2 raw, unsigned (&out)[W])
{
    const unsigned x = __builtin_amdgcn_perm(raw[1], raw[0], 0x05040100u);  // chunks 0 1 4 5
    const unsigned y = __builtin_amdgcn_perm(raw[1], raw[0], 0x07060302u);  // chunks 2 3 6 7
    const auto h = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    const unsigned p = __builtin_amdgcn_perm(h[1], h[0], 0x06040200u), q = __builtin_amdgcn_perm(h[1], h[0], 0x07050301u);
    const auto w = __builtin_amdgcn_permlane16_swap(p, q, false, false);
    if constexpr (W == 2) {
        out[0] = w[0];
        out[1] = w[1];
    } else {
        out[0] = __builtin_amdgcn_perm(w[1], w[0], 0x05040100u);
    }
}

// The MFMA of A's block i and B's block j in step ks (constants once unrolled), the operands exchanged.
template <class T, class Acc>
__device__ __forceinline__ Acc mma_scaled(u32x4 b, const unsigned (&sbs)[T::SBW], int j, u32x4 a,
                                          const unsigned (&sa)[T::SAW], int i, int ks, Acc c)
{
    typedef typename T::E E;
    const unsigned sb = sbs[T::DIRECT ? j : 0], y = sa[T::DIRECT ? i : i & 1];
    const int x_byte = T::DIRECT ? ks : 2 * j + ks, y_byte = T::DIRECT ? ks : 2 * (i >> 1) + ks;
    switch (4 * x_byte + y_byte) {  // the same step ks on both sides
    case 0: return E::template mma<16, 0, 0>(b, sb, a, y, c);
    case 2: return E::template mma<16, 0, 2>(b, sb, a, y, c);
    case 5: return E::template mma<16, 1, 1>(b, sb, a, y, c);
    case 7: return E::template mma<16, 1, 3>(b, sb, a, y, c);
    case 8: return E::template mma<16, 2, 0>(b, sb, a, y, c);
    case 10: return E::template mma<16, 2, 2>(b, sb, a, y, c);
    case 13: return E::template mma<16, 3, 1>(b, sb, a, y, c);
    default: return E::template mma<16, 3, 3>(b, sb, a, y, c);
    }
}

// Loads per wave of the S half panels after number n (n % 2P == N) of the order A lo, B lo, B hi,
// A hi, ...
// (P = 4; without A hi, P = 3). The first of an even K-step comes with scales.
template <class T, int N, int S, int P = 4>
constexpr int loads_after()
{
    int sum = 0;
    for (int i = 1; i <= S; ++i) {
        sum += ((N + i) % P == 0 || (N + i) % P == 3) ? T::A_LD : T::B_LD;
        if (T::MX && (N + i) % (2 * P) == 0) ++sum;
    }
    return sum;
}

// Wait until at most the min(later, S) half panels issued after number n are outstanding.
template <class T, int N, int S, int P = 4>
__device__ __forceinline__ void wait_halves(int later)
{
    if constexpr (S == 0) {
        wait_vm<0>();
    } else {
        if (later >= S) wait_vm<loads_after<T, N, S, P>()>();
        else wait_halves<T, N, S - 1, P>(later);
    }
}

// A barrier that waits for no memory by itself.
__device__ __forceinline__ void bare_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A lane's 4 values of each of two blocks side by side -> 8 consecutive values of its row, as words:
// a pair of 16-lane rows exchanges blocks (v_permlane16_swap), so that lanes of row g = lane / 16 hold
// the columns 8 ((g & 1) 2 + (g >> 1)) .. + 7 of the 32. Words: 8 of fp32, 4 of two 16-bit values.
template <class O>
__device__ __forceinline__ void eight_of_row(const float (&v)[2][4], unsigned (&out)[2 * sizeof(O)])
{
    constexpr int W = sizeof(O);  // words of 4 values
    unsigned w[2][W];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (W == 4) {
                w[j][i] = __builtin_bit_cast(unsigned, v[j][i]);
            } else {
                typedef O Pair __attribute__((ext_vector_type(2)));
                w[j][i] = __builtin_bit_cast(unsigned, Pair{(O)v[j][2 * i], (O)v[j][2 * i + 1]});
            }
        }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const auto s = __builtin_amdgcn_permlane16_swap(w[0][i], w[1][i], false, false);
        out[i] = s[0];
        out[W + i] = s[1];
    }
}

// Values first .. last - 1 of the 8 to C + at.
template <class O>
__device__ __forceinline__ void store_eight(void *C, int64_t at, const float (&v)[2][4], int first, int last)
{
    unsigned w[2 * sizeof(O)];
    eight_of_row<O>(v, w);  // every lane takes part
    O *c = static_cast<O *>(C) + at;
    if (first == 0 && last == 8) {
        struct __attribute__((packed)) Words {
            unsigned w[2 * sizeof(O)];
        } x;
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(O); ++i) x.w[i] = w[i];
        *reinterpret_cast<Words *>(c) = x;
    } else if (first < last) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < first || e >= last) continue;
            if constexpr (sizeof(O) == 4) c[e] = __builtin_bit_cast(O, w[e]);
            else c[e] = __builtin_bit_cast(O, (unsigned short)(w[e / 2] >> (16 * (e & 1))));
        }
    }
}

// Rows m0 .. m_end of C (of D_g), columns n0 .. N, the sum over k_lo .. k_end. LO: the rows end in
// the tile's first half. The workgroup holds KG groups of T::WAVES waves, each with a KG-th of the
// K-steps and LDS of its own; the first adds the sums in order and stores them.
template <class T, bool GRAD, bool LO, int KG>
__device__ __forceinline__ void tile_body(const GroupArgs &p, char *lds, int g, int m0, int m_end, int n0, int k_lo,
                                          int k_end)
{
    typedef typename T::E E;
    typedef typename E::T Elem;
    // origin of the panels: a T operand's columns start early enough to end inside the matrix
    constexpr int m_need = LO ? T::RH : T::BM;
    const int mb0 = T::AT ? (m_end >= m_need ? min(m0, m_end - m_need) : 0) : m0;
    const int nb0 = T::BT ? (p.N >= T::BN ? min(n0, p.N - T::BN) : 0) : n0;

    const int lane = threadIdx.x & 63;
    const int w_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = KG == 1 ? 0 : w_all / T::WAVES, w = w_all - kg * T::WAVES;
    const int wm = w / T::GN, wn = w % T::GN;

    // barriers that a group of waves passes for a sum of `len` elements, below
    auto barriers = [](int len) {
        return len == 0 ? 0 : (LO ? 2 : 4) * ((len + T::BK - 1) / T::BK) + 2 + (len % T::BK != 0);
    };
    int idle = 0;  // barriers that this group passes less than the other
    if constexpr (KG > 1) {
        const int steps = (k_end - k_lo + T::BK - 1) / T::BK;
        auto first_step = [&](int group) { return (group * steps) / KG; };  // so the last group has the most
        idle = barriers(k_end - k_lo - first_step(KG - 1) * T::BK);
        const int lo = k_lo + first_step(kg) * T::BK;
        if (kg < KG - 1) k_end = k_lo + first_step(kg + 1) * T::BK;
        k_lo = lo;
        idle -= barriers(k_end - k_lo);
        lds += kg * T::GROUP_LDS;
    }
    const int len = k_end - k_lo;
    const int ov = (T::BK - len % T::BK) % T::BK;
    const int nk = (len + T::BK - 1) / T::BK;
    const int halves = (LO ? 3 : 4) * nk;
    // where the partial K-step starts (a saturating subtraction is a vector instruction)
    const int k_partial = __builtin_amdgcn_readfirstlane(max(k_end - T::BK, 0));

    const Elem *A = static_cast<const Elem *>(p.A);
    const Elem *B = static_cast<const Elem *>(p.B) + (GRAD ? 0 : (int64_t)g * p.stride_b);

    // ---- DMA. This lane's byte offsets from the panel's corner at a K-step; the host keeps them
    // below 2^32.
    unsigned a_voff[2][T::A_LD], b_voff[2][T::B_LD];
    // first k of the partial step that is below row 0 of the matrix (groups near its start, whose only
    // step it is): those lanes read row 0
    // Mx4, whose scales take registers, keeps less: load l of half h is of rows h RH + 8 WAVES l + this
    // wave's and lane's, its offset that row's, at most the last row's (offsets grow with rows).
    unsigned a_row = 0, b_row = 0, mx_chunk = 0;
    // Mx4: 64 rows' scales for each wave (some twice): of B, then of A
    const int sc_row = 64 * (w % T::SC_SEGMENTS);
    const bool sc_of_b = sc_row < T::BN;
    const unsigned char *sc_base = nullptr;
    unsigned sc_voff = 0;
    if constexpr (T::MX) {
        const int row = sc_row + lane - (sc_of_b ? 0 : T::BN), last = sc_of_b ? p.N - 1 - nb0 : m_end - 1 - mb0;
        sc_base = sc_of_b ? p.mxb + g * p.stride_mxb + (int64_t)nb0 * p.ld_mxb : p.mxa + (int64_t)mb0 * p.ld_mxa;
        sc_voff = (unsigned)(min(row, last) * (sc_of_b ? p.ld_mxb : p.ld_mxa));
    }
    // the last row's offset, or the tile's where the matrix has more (whose offsets may pass 32 bits)
    const unsigned a_last = (unsigned)(min(m_end - 1 - mb0, T::BM - 1) * p.lda);
    const unsigned b_last = (unsigned)(min(p.N - 1 - nb0, T::BN - 1) * p.ldb);
    auto offsets_of = [&](int k_first) {
        if constexpr (T::MX) {
            const int r8 = 8 * w + lane / 8;
            a_row = (unsigned)(r8 * p.lda);
            b_row = (unsigned)(r8 * p.ldb);
            mx_chunk = min(16u * ((lane % 8) ^ swz_d(r8)), (unsigned)(min(p.K, T::BK) - 16));  // chunks past K: cleared
            static_assert(8 * T::WAVES % 16 == 0, "a wave's loads share their rows' swizzle");
            return;
        }
        const int below = k_first < 0 ? -k_first : 0;
        const int last16 = min(p.K, T::BK) * T::ES - 16;  // the last chunk of a row shorter than a K-step
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < T::A_LD; ++i) {
                if constexpr (T::AT) {
                    constexpr int CPR = T::RH / 8;  // chunks per row
                    const int krow = (64 / CPR) * (T::A_LD * w + i) + lane / CPR;
                    int col = mb0 + h * T::RH + 8 * ((lane % CPR) ^ swz_t<T::RH>(krow));
                    if (m_end < T::BM) col = min(col, m_end - 8);
                    a_voff[h][i] = (unsigned)((max(krow - below, 0) * p.lda + (col - mb0)) * 2);
                } else {
                    const int row = 8 * (T::A_LD * w + i) + lane / 8;
                    const int chunk = (lane % 8) ^ swz_d(row);
                    a_voff[h][i] = (unsigned)(min(h * T::RH + row, m_end - 1 - mb0) * p.lda * T::ES + min(16 * chunk, last16));
                }
            }
#pragma unroll
            for (int i = 0; i < T::B_LD; ++i) {
                if constexpr (T::BT) {
                    constexpr int CPR = T::CH / 8;
                    const int krow = (64 / CPR) * (T::B_LD * w + i) + lane / CPR;
                    int col = nb0 + h * T::CH + 8 * ((lane % CPR) ^ swz_t<T::CH>(krow));
                    if (p.N < T::BN) col = min(col, p.N - 8);
                    const int k = GRAD ? max(krow - below, 0) : min(krow, p.K - 8 + krow % 8);
                    b_voff[h][i] = (unsigned)((k * p.ldb + (col - nb0)) * 2);
                } else {
                    const int row = 8 * (T::B_LD * w + i) + lane / 8;
                    const int chunk = (lane % 8) ^ swz_d(row);
                    b_voff[h][i] = (unsigned)(min(h * T::CH + row, p.N - 1 - nb0) * p.ldb * T::ES + min(16 * chunk, last16));
                }
            }
        }
    };
    const unsigned lds0 = (unsigned)(uintptr_t)(lds_char *)lds;
    auto first_k = [&](int kt) { return ov ? (kt == 0 ? k_partial : k_lo + (kt - 1) * T::BK) : k_lo + kt * T::BK; };
    // Mx4: the scales of K-steps kt and kt + 1, kt even and not 0: a K-step's 8 follow each other. Of a
    // last K-step alone those of the one before it come too, and its own are the second 8.
    auto issue_scales = [&](int kt) {
        const int at = first_k(kt) / 16 - (kt + 1 < nk ? 0 : 8);
        dma16(lds0 + 2 * T::STAGE + (kt / 2 & 1) * T::SC_PAIR + 16 * sc_row, sc_base + at, sc_voff);
    };
    // half panel number 4 kt + i of the reading order (0: A lo, 1: B lo, 2: B hi, 3: A hi)
    auto issue_one = [&](int kt, int i, int l) {  // load l of it
        const int k0 = first_k(kt);
        const unsigned st = lds0 + (kt & 1) * T::STAGE;
        if constexpr (T::MX) {
            const unsigned at = (w + T::WAVES * l) * 1024;
            if (i == 0 || i == 3) {
                const unsigned down = (unsigned)(((i == 3) * T::RH + 8 * T::WAVES * l) * p.lda);
                dma16(st + T::A_OFF[i == 3] + at, A + (int64_t)mb0 * p.lda + k0, min(a_row + down, a_last) + mx_chunk);
            } else {
                const unsigned down = (unsigned)(((i - 1) * T::CH + 8 * T::WAVES * l) * p.ldb);
                dma16(st + T::B_OFF[i - 1] + at, B + (int64_t)nb0 * p.ldb + k0, min(b_row + down, b_last) + mx_chunk);
            }
            return;
        }
        if (i == 0 || i == 3) {
            const int h = i == 3;
            const Elem *base = T::AT ? A + (int64_t)k0 * p.lda + mb0 : A + (int64_t)mb0 * p.lda + k0;
            dma16(st + T::A_OFF[h] + (T::A_LD * w + l) * 1024, base, a_voff[h][l]);
        } else {
            const int h = i - 1;
            const Elem *base = T::BT ? B + (int64_t)k0 * p.ldb + nb0 : B + (int64_t)nb0 * p.ldb + k0;
            dma16(st + T::B_OFF[h] + (T::B_LD * w + l) * 1024, base, b_voff[h][l]);
        }
    };
    auto issue = [&](int kt, int i) {
#pragma unroll
        for (int l = 0; l < (i == 0 || i == 3 ? T::A_LD : T::B_LD); ++l) issue_one(kt, i, l);
    };

    // ---- operand reads: 64 bytes of k (MFMA step ks) of the 16-wide block blk of a half panel
    int d_off[T::KS];
#pragma unroll
    for (int ks = 0; ks < T::KS; ++ks)
        d_off[ks] = (lane % T::MB) * 128 + 16 * ((8 / T::KS * ks + lane / T::MB) ^ swz_d(lane % T::MB));
    const int t_g = lane >> 4, t_j = lane & 15;
    auto t_offset = [&](int blk, auto width) {
        constexpr int W = decltype(width)::value;
        const int krow = 8 * t_g + (t_j >> 2), col = T::MB * blk + 4 * (t_j & 3);
        return krow * 2 * W + 16 * ((col >> 3) ^ swz_t<W>(krow)) + 8 * ((col >> 2) & 1);
    };
    int a_toff[T::FM], b_toff[T::FN];
#pragma unroll
    for (int i = 0; i < T::FM; ++i) a_toff[i] = t_offset(wm * T::FM + i, std::integral_constant<int, T::RH>());
#pragma unroll
    for (int j = 0; j < T::FN; ++j) b_toff[j] = t_offset(wn * T::FN + j, std::integral_constant<int, T::CH>());
    auto read_d = [&](const lds_char *half, int blk, int ks) {
        return *(const lds_u32x4 *)(half + blk * T::MB * 128 + d_off[ks]);
    };
    auto read_t = [&](const lds_char *half, int toff, int ks, int row_bytes) {
        constexpr int rows = T::BK / T::KS;
        const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4i16 *)(half + toff + rows * ks * row_bytes));
        const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4i16 *)(half + toff + (rows * ks + 4) * row_bytes));
        const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
        return u32x4{l2[0], l2[1], h2[0], h2[1]};
    };
    // operands: a[0], a[1]: A lo, A hi; b[s], b[s ^ 1]: B lo, B hi in a K-step of parity s
    u32x4 a[2][T::KS][T::FM], b[2][T::KS][T::FN];
    // operand number r (of KS FM, KS FN) of a half panel
    auto read_a = [&](const lds_char *half, int r, u32x4 (&dst)[T::KS][T::FM]) {
        const int ks = r / T::FM, i = r % T::FM;
        if constexpr (T::AT) dst[ks][i] = read_t(half, a_toff[i], ks, 2 * T::RH);
        else dst[ks][i] = read_d(half, wm * T::FM + i, ks);
    };
    auto read_b = [&](const lds_char *half, int r, u32x4 (&dst)[T::KS][T::FN]) {
        const int ks = r / T::FN, j = r % T::FN;
        if constexpr (T::BT) dst[ks][j] = read_t(half, b_toff[j], ks, 2 * T::CH);
        else dst[ks][j] = read_d(half, wn * T::FN + j, ks);
    };

    // Mx4: a half panel's scales as read, and as the MFMAs take them (like a and b)
    u32x2 raw_a[T::DIRECT ? T::FM : 1] = {}, raw_b[T::SBW] = {};
    unsigned sa[2][T::SAW] = {}, sb4[2][T::SBW] = {};
    typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
    auto read_scales = [&](int kt, bool of_b, int half, auto &raw) {
        const lds_char *sc = (const lds_char *)lds + 2 * T::STAGE + (kt / 2 & 1) * T::SC_PAIR;
        const int second = (kt & 1) != 0 || (kt == nk - 1 && kt > 0) ? 8 : 0;
        // B's, of at most two blocks, come from the first 32 lanes; the rows that the others read lie in A's
        const int row0 = of_b ? half * T::CH + wn * T::QN : T::BN + half * T::RH + wm * T::QM;
        if constexpr (T::DIRECT) {
            constexpr int blocks = sizeof raw / sizeof raw[0];
#pragma unroll
            for (int i = 0; i < blocks; ++i) raw[i] = *(const lds_u32x2 *)(sc + second + 16 * (row0 + 16 * i + lane % 16));
        } else {
            raw[0] = *(const lds_u32x2 *)(sc + second + 16 * (row0 + (of_b ? lane : lane % T::QM)));
        }
    };
    auto spread = [&](auto &raw, auto &words) {
        if constexpr (T::DIRECT) {  // chunks g and 4 + g to bytes 0 and 1
            constexpr int blocks = sizeof raw / sizeof raw[0];
#pragma unroll
            for (int i = 0; i < blocks; ++i)
                words[i] = __builtin_amdgcn_perm(raw[i][1], raw[i][0], (unsigned)(lane >> 4) * 0x0101u | 0x0c0c0400u);
        } else {
            scales_of_lane(raw[0], words);
        }
    };
    // of the first two K-steps, through registers
    auto first_scales = [&] {
        struct __attribute__((packed)) Eight {
            u32x2 v;
        };
        const unsigned char *q = sc_base + sc_voff;
        u32x4 v = {0x7f7f7f7fu, 0x7f7f7f7fu};
        if (p.K >= T::BK) {
            const u32x2 x = reinterpret_cast<const Eight *>(q + first_k(0) / 16)->v;
            v[0] = x[0];
            v[1] = x[1];
        } else {  // a row of fewer, the chunks past them zeros of scale 1
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (16 * i < p.K) v[i / 4] = (v[i / 4] & ~(0xffu << (8 * (i % 4)))) | (unsigned)q[i] << (8 * (i % 4));
        }
        if (nk > 1) {
            const u32x2 y = reinterpret_cast<const Eight *>(q + first_k(1) / 16)->v;
            v[2] = y[0];
            v[3] = y[1];
        }
        *(lds_u32x4 *)((lds_char *)lds + 2 * T::STAGE + 16 * (sc_row + lane)) = v;
    };

    constexpr int HA = LO ? 1 : 2;  // halves of rows
    // blocks of C transposed (the MFMA's operands exchanged): lane l holds row l % 16 of C and the
    // columns 4 (l / 16) + r, r < 4
    typename E::template Acc<T::MB> acc[HA][2][T::FM][T::FN];
#pragma unroll
    for (int qa = 0; qa < HA; ++qa)
#pragma unroll
        for (int qb = 0; qb < 2; ++qb)
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int j = 0; j < T::FN; ++j)
#pragma unroll
                    for (int r = 0; r < T::ACC; ++r) acc[qa][qb][i][j][r] = 0;

    auto wait_reads = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };

    // One phase: I of a K-step of parity S. FULL: every half panel that the phase issues and waits
    // for exists.
    auto phase = [&](int kt, auto I_, auto S_, auto FULL_) {
        constexpr int I = decltype(I_)::value, S = decltype(S_)::value;
        constexpr bool FULL = decltype(FULL_)::value;
        constexpr int qa = I >= 2, qb = I == 1 || I == 2;
        constexpr bool reads_a = I == 1 || I == 2;
        constexpr int NM = T::KS * T::FM * T::FN, NR = T::KS * (reads_a ? T::FM : T::FN);
        constexpr int issues = (I + 1) % 4;  // the half panel issued: A lo in phase 3, B lo, B hi, A hi
        constexpr int NL = issues == 0 || issues == 3 ? T::A_LD : T::B_LD;
        constexpr int pre = NM / 8;          // MFMAs before the barrier
        // the reads and loads, mixed evenly, spread evenly over the MFMAs after the barrier
        constexpr int items = NR + NL, slots = NM - pre;
        const int stage = ((kt + (I >= 2)) & 1) * T::STAGE;
        const lds_char *half = (const lds_char *)lds + stage +
                               (reads_a ? T::A_OFF[I == 1] : T::B_OFF[I == 0]);
        auto mfma = [&](int m) {
            const int ks = m / (T::FM * T::FN), i = m / T::FN % T::FM, j = m % T::FN;
            if constexpr (!T::MX)  // phase_mx
                acc[qa][qb][i][j] = E::template mma<T::MB>(b[S ^ qb][ks][j], a[qa][ks][i], acc[qa][qb][i][j]);
        };
        auto read = [&](int r) {
            if constexpr (reads_a) read_a(half, r, a[I == 1]);
            else read_b(half, r, b[S ^ 1]);
        };
#pragma unroll
        for (int m = 0; m < pre; ++m) mfma(m);
        const int n = 4 * kt + 2 + I, issued = 4 * kt + 9 + I;
        if (FULL) wait_vm<loads_after<T, (2 + I) % 4, 6>()>();
        else if (n < halves) wait_halves<T, (2 + I) % 4, 6>(min(issued, halves) - 1 - n);
        wait_reads();
        bare_barrier();
#pragma unroll
        for (int m = pre; m < NM; ++m) {
#pragma unroll
            for (int t = (m - pre) * items / slots; t < (m - pre + 1) * items / slots; ++t) {
                const int l = t * NL / items;  // loads among the items before t
                if ((t + 1) * NL / items == l) read(t - l);
                else if (FULL || issued < halves) issue_one(kt + 2 + (I == 3), issues, l);
            }
            mfma(m);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // The same for Mx4, whose scales' registers leave none for both halves of A: a half replaces the
    // other operand by operand, each read behind the last MFMA of the one before it, B lo of the next
    // K-step likewise B hi. Phase 0: A lo x B lo, reads B hi; 1: A lo x B hi, reads A hi; 2: A hi x
    // B hi, reads B lo of the next K-step; 3: A hi x B lo, reads A lo of the next. So half panels are
    // numbered 4 kt + (0: B lo, 1: A lo, 2: B hi, 3: A hi), and the DMA goes out a phase later, so that a
    // phase waits for the reads of the phase before the last one only. Five half panels are on their way.
    // LEFT: K-steps that follow, 2 if there are more. (One body for all but the last two and no branches
    // in them: with bodies for even and odd K-steps, or branches around the loads, some of the sums went
    // through memory on the way.) B lo is in b[0], B hi in b[1], and so B lo of the next K-step, until its
    // first phase moves it.
    auto phase_mx = [&](int kt, auto I_, auto LEFT_) {
        constexpr int I = decltype(I_)::value, LEFT = decltype(LEFT_)::value;
        constexpr int qa = I >= 2, qb = I == 1 || I == 2;
        constexpr bool reads_a = I == 1 || I == 3;
        constexpr int NM = T::KS * T::FM * T::FN, NR = T::KS * (reads_a ? T::FM : T::FN), each = NM / NR;
        constexpr int issues = I == 0 ? 1 : I == 1 ? 0 : I;  // as issue_one counts
        constexpr int NL = issues == 0 || issues == 3 ? T::A_LD : T::B_LD;
        constexpr int pre = NM / 8;
        const lds_char *half = (const lds_char *)lds + ((kt + (I >= 2)) & 1) * T::STAGE +
                               (reads_a ? T::A_OFF[I == 1] : T::B_OFF[I == 0]);
        auto mfma = [&](int m) {  // operands in the order in which the next half replaces them
            const int ks = m / (T::FM * T::FN);
            const int i = I == 2 ? m % T::FM : m / T::FN % T::FM, j = I == 2 ? m / T::FM % T::FN : m % T::FN;
            acc[qa][qb][i][j] = mma_scaled<T>(b[qb][ks][j], sb4[qb], j, a[0][ks][i], sa[0], i, ks, acc[qa][qb][i][j]);
        };
        // the offsets of the loads and reads anew for each K-step: kept, they would take some 20 registers
        if constexpr (I == 0) asm volatile("" : "+v"(a_row), "+v"(b_row), "+v"(d_off[0]), "+v"(d_off[1]));
        // the scales that the phase before read
        if constexpr (reads_a) spread(raw_b, sb4[1]);
        else spread(raw_a, sa[0]);
#pragma unroll
        for (int m = 0; m < pre; ++m) mfma(m);
        // half panels issued after number 4 kt + 2 + I, which is read next
        constexpr int later = LEFT == 2 ? 5 : 4 * LEFT + 1 - I;
        if constexpr (later >= 0) wait_vm<later * T::A_LD>();  // scales among them: one more than need be
        // at most the reads of the phase before are left: those before it are done
        asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(T::KS * (reads_a ? T::FN : T::FM)) : "memory");
        bare_barrier();
        if constexpr (later < 0) {
        } else if constexpr (reads_a) {
            read_scales(kt + (I >= 2), false, I < 2, raw_a);
        } else {
            read_scales(kt + (I >= 2), true, I < 2, raw_b);
        }
        auto read = [&](int r) {
            if constexpr (later < 0) return;
            else if constexpr (reads_a) read_a(half, r, a[0]);
            else read_b(half, r, b[1]);
        };
#pragma unroll
        for (int m = pre; m < NM; ++m) {
            if (m > 0 && m % each == 0) read(m / each - 1);
#pragma unroll
            for (int l = 0; l < NL; ++l)
                if (LEFT == 2 && m == pre + (l + 1) * (NM - pre) / (NL + 1)) issue_one(kt + 2, issues, l);
            mfma(m);
            __builtin_amdgcn_sched_barrier(0);
        }
        read(NR - 1);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto k_step_mx = [&](int kt, auto LEFT) {
        static_assert(!T::MX || T::A_LD == T::B_LD, "half panels of as many loads");
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks)
#pragma unroll
            for (int j = 0; j < T::FN; ++j) b[0][ks][j] = b[1][ks][j];
#pragma unroll
        for (int j = 0; j < T::SBW; ++j) sb4[0][j] = sb4[1][j];
        phase_mx(kt, std::integral_constant<int, 0>(), LEFT);
        phase_mx(kt, std::integral_constant<int, 1>(), LEFT);
        phase_mx(kt, std::integral_constant<int, 2>(), LEFT);
        phase_mx(kt, std::integral_constant<int, 3>(), LEFT);
    };
    auto k_step = [&](int kt, auto S, auto FULL) {
        phase(kt, std::integral_constant<int, 0>(), S, FULL);
        phase(kt, std::integral_constant<int, 1>(), S, FULL);
        phase(kt, std::integral_constant<int, 2>(), S, FULL);
        phase(kt, std::integral_constant<int, 3>(), S, FULL);
    };

    // The same without A hi; half panels are numbered 3 kt + (0: A lo, 1: B lo, 2: B hi), S is the
    // parity of the K-step: A lo is in a[S], B lo in b[0], B hi in b[1].
    auto phase_lo = [&](int kt, auto I_, auto S_, auto FULL_) {
        constexpr int I = decltype(I_)::value, S = decltype(S_)::value;
        constexpr bool FULL = decltype(FULL_)::value;
        constexpr int NM = T::KS * T::FM * T::FN, NA = I == 1 ? T::KS * T::FM : 0, NR = NA + T::KS * T::FN;
        constexpr int NL = I == 0 ? T::A_LD + T::B_LD : T::B_LD;  // phase 0 issues A lo, B lo, phase 1 B hi
        constexpr int pre = NM / 8, items = NR + NL, slots = NM - pre;
        const lds_char *stage = (const lds_char *)lds + ((kt + I) & 1) * T::STAGE;
        auto mfma = [&](int m) {
            const int ks = m / (T::FM * T::FN), i = m / T::FN % T::FM, j = m % T::FN;
            if constexpr (T::MX)
                acc[0][I][i][j] = mma_scaled<T>(b[I][ks][j], sb4[I], j, a[S][ks][i], sa[S], i, ks, acc[0][I][i][j]);
            else acc[0][I][i][j] = E::template mma<T::MB>(b[I][ks][j], a[S][ks][i], acc[0][I][i][j]);
        };
        if constexpr (T::MX) {
            spread(raw_b, sb4[I]);
            if constexpr (I == 0) spread(raw_a, sa[S]);
        }
#pragma unroll
        for (int m = 0; m < pre; ++m) mfma(m);
        const int n = 3 * kt + (I == 0 ? 2 : 4), issued = 3 * kt + (I == 0 ? 6 : 8);
        if (FULL) wait_vm<loads_after<T, (3 * S + (I == 0 ? 2 : 4)) % 6, 3, 3>()>();
        else if (n < halves) wait_halves<T, (3 * S + (I == 0 ? 2 : 4)) % 6, 3, 3>(min(issued, halves) - 1 - n);
        wait_reads();
        bare_barrier();
        if constexpr (T::MX) {
            read_scales(kt + I, true, I == 0, raw_b);
            if constexpr (I == 1) read_scales(kt + 1, false, 0, raw_a);
            if constexpr (I == 0 && S == 0)
                if (FULL || kt + 2 < nk) issue_scales(kt + 2);
        }
#pragma unroll
        for (int m = pre; m < NM; ++m) {
#pragma unroll
            for (int t = (m - pre) * items / slots; t < (m - pre + 1) * items / slots; ++t) {
                const int l = t * NL / items, r = t - l;  // loads and reads among the items before t
                if ((t + 1) * NL / items == l) {
                    if (r < NA) read_a(stage + T::A_OFF[0], r, a[S ^ 1]);
                    else read_b(stage + T::B_OFF[I == 0], r - NA, b[I == 0]);
                } else if (FULL || kt + 2 < nk) {
                    if (I == 1) issue_one(kt + 2, 2, l);
                    else if (l < T::A_LD) issue_one(kt + 2, 0, l);
                    else issue_one(kt + 2, 1, l - T::A_LD);
                }
            }
            mfma(m);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto k_step_lo = [&](int kt, auto S, auto FULL) {
        phase_lo(kt, std::integral_constant<int, 0>(), S, FULL);
        phase_lo(kt, std::integral_constant<int, 1>(), S, FULL);
    };

    if (nk > 0) {
        constexpr int panels = LO ? 3 : 4;  // half panels per K-step
        offsets_of(ov ? k_end - T::BK : 0);
        if constexpr (T::MX) first_scales();
        constexpr int swapped = T::MX && !LO;  // B lo first, as it is read
        for (int i = 0; i < panels; ++i) issue(0, i < 2 ? i ^ swapped : i);
        if (nk > 1)
            for (int i = 0; i < panels; ++i) issue(1, i < 2 ? i ^ swapped : i);
        if (ov) {
            // zeros over the first ov k of both panels, once the whole step has landed everywhere
            if (nk > 1) wait_vm<(LO ? 1 : 2) * T::A_LD + 2 * T::B_LD>();
            else wait_vm<0>();
            bare_barrier();
            lds_char *st = (lds_char *)lds;
            // leading bytes of chunk c of the K-step to clear (all from 16 on, none below 1)
            auto clear_of = [&](int c) {
                if (GRAD || k_end >= T::BK) return ov * T::ES - 16 * c;
                return 16 * (c + 1) - k_end * T::ES;  // what the chunk repeats, or more than all of it
            };
            auto zero = [&](int off, int rows, bool t) {
                for (int e = 64 * w + lane; e < rows * 8; e += 64 * T::WAVES) {
                    lds_u32x4 *q = (lds_u32x4 *)(st + off + 16 * e);
                    if (t) {  // rows of k, rows / 8 chunks each
                        const int krow = e / (rows / 8);
                        if (krow % 8 * T::ES < clear_of(krow / 8)) *q = u32x4{0u, 0u, 0u, 0u};
                    } else {
                        const int row = e / 8, c = (e % 8) ^ swz_d(row);
                        const int bytes = clear_of(c);
                        if (bytes >= 16) {
                            *q = u32x4{0u, 0u, 0u, 0u};
                        } else if (bytes > 0) {
                            u32x4 v = *q;
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                const int z = bytes - 4 * d;  // leading bytes of word d to clear
                                v[d] = z >= 4 ? 0u : z > 0 ? v[d] & (0xffffffffu << (8 * z)) : v[d];
                            }
                            *q = v;
                        }
                    }
                }
            };
            for (int h = 0; h < 2; ++h) {
                if (h == 0 || !LO) zero(T::A_OFF[h], T::RH, T::AT);
                zero(T::B_OFF[h], T::CH, T::BT);
            }
            wait_reads();
        } else {
            wait_halves<T, 1, 6, panels>(min(halves, 2 * panels) - 2);
            if constexpr (T::MX) wait_reads();  // the first scales' write
        }
        bare_barrier();
#pragma unroll
        for (int r = 0; r < T::KS * T::FM; ++r) read_a((const lds_char *)lds + T::A_OFF[0], r, a[0]);
#pragma unroll
        for (int r = 0; r < T::KS * T::FN; ++r) read_b((const lds_char *)lds + T::B_OFF[0], r, b[T::MX && !LO]);
        if constexpr (T::MX) {
            read_scales(0, false, 0, raw_a);
            read_scales(0, true, 0, raw_b);
            if constexpr (!LO) spread(raw_b, sb4[1]);
        }
        wait_reads();
        bare_barrier();
        using S0 = std::integral_constant<int, 0>;
        using S1 = std::integral_constant<int, 1>;
        int kt = 0;
        if constexpr (LO) {
            for (; kt + 3 < nk; kt += 2) {
                k_step_lo(kt, S0(), std::true_type());
                k_step_lo(kt + 1, S1(), std::true_type());
            }
            for (; kt < nk; kt += 2) {
                k_step_lo(kt, S0(), std::false_type());
                if (kt + 1 < nk) k_step_lo(kt + 1, S1(), std::false_type());
            }
        } else if constexpr (T::MX) {
            for (; kt + 2 < nk; ++kt) {
                if (!(kt & 1)) issue_scales(kt + 2);
                k_step_mx(kt, std::integral_constant<int, 2>());
            }
            if (kt + 1 < nk) k_step_mx(kt++, std::integral_constant<int, 1>());
            k_step_mx(kt, std::integral_constant<int, 0>());
        } else {
            if (nk > 2) issue(2, 0);
            for (; kt + 4 < nk; kt += 2) {
                k_step(kt, S0(), std::true_type());
                k_step(kt + 1, S1(), std::true_type());
            }
            for (; kt < nk; kt += 2) {
                k_step(kt, S0(), std::false_type());
                if (kt + 1 < nk) k_step(kt + 1, S1(), std::false_type());
            }
        }
    }

    if constexpr (KG > 1) {
        for (int i = 0; i < idle; ++i) bare_barrier();
        // once every wave has read what it needs, the other groups' sums go through their panels' LDS
        typedef __attribute__((address_space(3))) typename E::template Acc<T::MB> lds_acc;
        static_assert(T::BM * T::BN * 4 <= T::GROUP_LDS, "a group's sums fit its LDS");
        bare_barrier();
        auto each = [&](const char *group, auto &&f) {
            lds_acc *part = (lds_acc *)(lds_char *)group + 64 * w + lane;
            int at = 0;
#pragma unroll
            for (int qa = 0; qa < HA; ++qa)
#pragma unroll
                for (int qb = 0; qb < 2; ++qb)
#pragma unroll
                    for (int i = 0; i < T::FM; ++i)
#pragma unroll
                        for (int j = 0; j < T::FN; ++j) f(acc[qa][qb][i][j], part + 64 * T::WAVES * at++);
        };
        if (kg > 0) {
            each(lds, [](auto &mine, lds_acc *at) { *at = mine; });
            wait_reads();
            bare_barrier();
            return;
        }
        bare_barrier();
#pragma unroll
        for (int group = 1; group < KG; ++group)
            each(lds + group * T::GROUP_LDS, [](auto &mine, lds_acc *at) { mine += *at; });
    }

    // ---- epilogue: 16 bytes (32 of fp32) of a row per lane, 16 rows of 32 columns per instruction,
    // straight from the registers. (Staging the tile in LDS to store whole rows took 4 us of a tile,
    // single elements from the untransposed blocks 7.)
    const int lane_row = lane & 15, lane_g = lane >> 4;
    const int n_lane = nb0 + wn * T::QN + 8 * ((lane_g & 1) * 2 + (lane_g >> 1));
    float sb[2][2][4];
    if constexpr (E::INT8) {
#pragma unroll
        for (int qb = 0; qb < 2; ++qb)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sb[qb][j][r] = p.sb[(int64_t)g * p.stride_sb +
                                        min(nb0 + qb * T::CH + wn * T::QN + 16 * j + 4 * lane_g + r, p.N - 1)];
    }
    auto store = [&](auto out) {
        typedef typename decltype(out)::T O;
#pragma unroll
        for (int qa = 0; qa < HA; ++qa)
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                const int block = mb0 + qa * T::RH + wm * T::QM + 16 * i;
                int m = block + lane_row;
                if (block >= m_end) break;
                bool live = m < m_end && (!T::AT || m >= m0);
                if (T::AT && m_end < m_need && m >= m_end / 8 * 8) {  // the last chunk, moved back
                    m -= -m_end & 7;
                    live = m < m_end && m >= m_end / 8 * 8;
                }
                float sa = 1.f;
                if constexpr (E::INT8) sa = p.sa[min(m, m_end - 1)];
                const int64_t row = (GRAD ? (int64_t)g * p.stride_c : 0) + (int64_t)m * p.ldc;
#pragma unroll
                for (int qb = 0; qb < 2; ++qb) {
                    float v[2][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            v[j][r] = (float)acc[qa][qb][i][j][r];
                            if constexpr (E::INT8) v[j][r] = v[j][r] * sa * sb[qb][j][r];
                        }
                    int n = n_lane + qb * T::CH;
                    int first = T::BT && n < n0 ? n0 - n : 0, last = live ? min(8, p.N - n) : 0;
                    if (T::BT && p.N < T::BN && n > p.N - 8 && n < p.N) {  // the last chunk, moved back
                        first = n + 8 - p.N;
                        last = live ? 8 : 0;
                        n = p.N - 8;
                    }
                    store_eight<O>(p.C, row + n, v, first, last);
                }
            }
    };
    if (p.c_type == 0) store(OutType<0>());
    else if (p.c_type == 1) store(OutType<1>());
    else store(OutType<2>());
}

// With one workgroup per CU, where the last round has tiles for at most half of the CUs, each of them
// is two workgroups' work, its first and second half of rows (bf16 4096 x 6144 x 4096, 1.5 rounds: 165
// -> 149 us; 2.25 rounds of 32 K-steps 141 -> 129). Workgroup bid of `tiles` tiles: its tile, and the
// half (-1: the whole tile); false: none.
constexpr int kCUs = 256;
template <bool SPLIT>
__device__ __forceinline__ bool tile_part(int64_t bid, int64_t tiles, unsigned &tile, int &half)
{
    const unsigned rest = (unsigned)(tiles % kCUs);
    half = -1;
    tile = (unsigned)bid;
    if (!SPLIT || rest == 0 || rest > kCUs / 2 || bid < tiles - rest) return bid < tiles;
    const unsigned in = (unsigned)(bid - (tiles - rest));
    half = (int)(in / rest);
    tile = (unsigned)(tiles - rest) + in % rest;
    return half < 2;
}

template <class T, bool GRAD, int KG>
__global__ __launch_bounds__(T::NT * KG) void group_tile_kernel(GroupArgs p)
{
    __shared__ __attribute__((aligned(1024))) char lds[KG * T::GROUP_LDS];

    const unsigned tiles_n = (unsigned)((p.N + T::BN - 1) / T::BN);
    const int64_t bid = linear_block();
    int g, m0, m_end, n0, k_lo, k_end, half;
    unsigned tile;
    if constexpr (GRAD) {
        const unsigned tiles_m = (unsigned)((p.K + T::BM - 1) / T::BM);
        const unsigned per = tiles_m * tiles_n;
        if (!tile_part<T::SPLIT>(bid, (int64_t)per * p.groups, tile, half)) return;
        // each group's tiles over all XCDs: the groups' sums differ in length
        unsigned tm, tn;
        g = (int)(tile / per);
        tile_of_group_block(tile - g * per, per, tiles_m, tiles_n, tm, tn);
        m0 = (int)tm * T::BM;
        n0 = (int)tn * T::BN;
        m_end = p.K;
        group_range(p.offsets, g, p.M, k_lo, k_end);
    } else {
        RowTile t;
        unsigned tm, tn;
        const RowTiles<T::BM> tiles(p);
        if (!tile_part<T::SPLIT>(bid, (int64_t)tiles.total * tiles_n, tile, half)) return;
        tile_of_group_block(tile, tiles.total * tiles_n, tiles.total, tiles_n, tm, tn);
        if (tn >= tiles_n || !tiles.find(p, tm, t)) return;  // (tn: where the count overflowed)
        g = t.g;
        m0 = t.row0;
        m_end = t.hi;
        n0 = (int)tn * T::BN;
        k_lo = 0;
        k_end = p.K;
    }
    if (T::SPLIT && half >= 0) {
        m0 += half * T::RH;
        if (m0 >= m_end) return;
        m_end = min(m_end, m0 + T::RH);
    }
    g = __builtin_amdgcn_readfirstlane(g);
    m0 = __builtin_amdgcn_readfirstlane(m0);
    m_end = __builtin_amdgcn_readfirstlane(m_end);
    k_lo = __builtin_amdgcn_readfirstlane(k_lo);
    k_end = __builtin_amdgcn_readfirstlane(k_end);
    if (m_end - m0 <= T::RH) tile_body<T, GRAD, true, KG>(p, lds, g, m0, m_end, n0, k_lo, k_end);
    else tile_body<T, GRAD, false, KG>(p, lds, g, m0, m_end, n0, k_lo, k_end);
}

// The tile takes the shape: rows of a D operand and of a T operand hold a chunk, and lane offsets fit
// 32 bits.
template <class T, bool GRAD>
bool tile_ok(const GroupArgs &a)
{
    constexpr int64_t limit = int64_t(1) << 32;
    constexpr int largest = 0x7fffffff - 1024;  // a tile's row and column numbers fit an int
    if (a.M > largest || a.N > largest || a.K > largest) return false;
    if (!GRAD && a.K * T::ES < 16) return false;  // a chunk
    if (T::MX && ((T::BM - 1) * a.ld_mxa >= limit || (T::BN - 1) * a.ld_mxb >= limit)) return false;
    if ((T::AT && a.K < 8) || (T::BT && a.N < 8)) return false;  // a chunk of a T operand's columns
    const int64_t a_rows = T::AT ? T::BK : T::BM, b_rows = T::BT ? T::BK : T::BN;
    return ((a_rows - 1) * a.lda + T::BM) * T::ES + 128 < limit && ((b_rows - 1) * a.ldb + T::BN) * T::ES + 128 < limit;
}

template <class T, bool GRAD, int KG>
hipError_t launch_tile(const GroupArgs &a, hipStream_t stream)
{
    const int64_t tiles_n = ((int64_t)a.N + T::BN - 1) / T::BN;
    const int64_t tiles_m = GRAD ? ((int64_t)a.K + T::BM - 1) / T::BM * a.groups : max_row_tiles(a, T::BM);
    if (tiles_m > 0x7fffffff / tiles_n) return hipErrorInvalidConfiguration;
    unsigned gx, gy;
    if (!grid_for(tiles_m * tiles_n + (T::SPLIT ? kCUs / 2 : 0), gx, gy)) return hipErrorInvalidConfiguration;
    GroupArgs arg = a;
    void *args[] = {&arg};
    return hipLaunchKernel(reinterpret_cast<const void *>(&group_tile_kernel<T, GRAD, KG>), dim3(gx, gy), dim3(T::NT * KG), args,
                           0, stream);
}

// The tiles of an element type and layouts.
template <class E, bool AT, bool BT>
struct Tiles {
    using Large = GroupTile<E, AT, BT, 128, 128, 2, 4>;
    using Mid = GroupTile<E, AT, BT, 64, 64, 4, 2>;
    using Small = GroupTile<E, AT, BT, 32, 32, 2, 1>;
    static bool ok(const GroupArgs &a, GroupTileKind kind)
    {
        return kind == GroupTileKind::Large ? tile_ok<Large, AT>(a)
               : kind == GroupTileKind::Mid ? tile_ok<Mid, AT>(a)
                                            : tile_ok<Small, AT>(a);
    }
    static hipError_t launch(const GroupArgs &a, GroupTileKind kind, hipStream_t stream)
    {
        return kind == GroupTileKind::Large ? launch_tile<Large, AT, 1>(a, stream)
               : kind == GroupTileKind::Mid  ? launch_tile<Mid, AT, 1>(a, stream)
               : kind == GroupTileKind::Small ? launch_tile<Small, AT, 2>(a, stream)
                                              : launch_tile<Small, AT, 4>(a, stream);
    }
};

// f(Tiles<...>()) for the call's element type and layouts.
template <class F>
auto with_tiles(const GroupArgs &a, F &&f)
{
    if (a.elem == GroupElem::I8) return f(Tiles<ElemI8, false, false>());
    if (a.elem == GroupElem::Mx4) return f(Tiles<ElemMx4, false, false>());
    const bool f16 = a.elem == GroupElem::F16;
    if (a.grad) return f16 ? f(Tiles<ElemF16, true, true>()) : f(Tiles<ElemBf16, true, true>());
    if (a.trans_b) return f16 ? f(Tiles<ElemF16, false, false>()) : f(Tiles<ElemBf16, false, false>());
    return f16 ? f(Tiles<ElemF16, false, true>()) : f(Tiles<ElemBf16, false, true>());
}

}  // namespace

// Fitted to some 300 shapes of all operators (the chosen kernel's time over the best one's: 1.03-1.04
// in the mean, up to 1.4 for single shapes; neither the stored bytes nor the wait of a partial K-step
// are terms of it). 256 x 256: 5.5 us per round for a tile's first loads and its stores, 1.35 per K-step of
// all CUs, 0.45-0.75 per K-step of a last round in halves. 128 x 128: 0.28 us per K-step, and 0.75 times
// the share of 512 tiles. 64 x 64 in four parts: 0.13-0.19 us per K-step and round of 256 tiles, in two
// 0.19-0.36 for up to 512, more with operands across k (64-byte rows). So many tiles go to 256 x 256
// (bf16 4608 x 8192 x 2048: 129 us, 145 in 128 x 128), fewer to 128 x 128 (1024 x 4096 x 4096: 36 us, 41
// in 256 x 256), few to 64 x 64 (256 x 4096 x 4096: 18 us, 27 in 128 x 128). Rows that start off 4-byte
// boundaries weigh the more the less a tile reuses them.
double group_tile_time(const GroupArgs &a, GroupTileKind kind)
{
    const bool large = kind == GroupTileKind::Large, small = kind <= GroupTileKind::Small;
    const double sum = a.grad ? (double)a.M / a.groups : (double)a.K;  // length of a tile's sums
    const double steps = ceil(sum * group_elem_size(a) / 128) * (aligned_words(a) ? 1.0 : large ? 1.25 : small && a.trans_b ? 2.3 : 1.5);
    const int t = large ? 256 : kind == GroupTileKind::Mid ? 128 : 64;
    const double tiles = (double)(((int64_t)a.N + t - 1) / t) *
                         (a.grad ? (double)(((int64_t)a.K + t - 1) / t) * a.groups : expected_row_tiles(a, t));
    // the groups' sizes are not known here, so neither is the number of rounds: between whole ones
    const bool known = a.grad || !a.offsets || a.groups == 1;
    double time;
    if (large) {
        const double round = 5.5 + 1.35 * steps, rest = known || tiles <= kCUs / 2 ? fmod(tiles, kCUs) : 0;
        const double full = known ? floor(tiles / kCUs) : fmax(1.0, tiles / kCUs + 0.1);
        if (rest == 0) time = full * round;
        else if (rest > kCUs / 2) time = (full + 1) * round;
        else time = (tiles <= kCUs / 2 ? 0 : full * round) + 5.5 + (0.45 + 0.3 * rest / (kCUs / 2)) * steps;
    } else if (kind == GroupTileKind::Small4) {
        const double rounds = known ? ceil(tiles / kCUs) : fmax(1.0, tiles / kCUs + 0.1);
        const bool halves = !a.grad && a.M <= 32 * expected_groups(a);  // tiles without a second half of rows
        const double step = (0.13 + 0.06 * fmin(1.0, tiles / kCUs)) * (a.trans_b ? 1 : 1.35) * (halves ? 0.75 : 1);
        time = rounds * (3 + step * steps);
    } else if (kind == GroupTileKind::Small) {
        const double full = floor(tiles / 512), rest = tiles / 512 - full, across = a.trans_b ? 1 : a.grad ? 1.35 : 1.15;
        time = full * (3 + 0.36 * across * steps);
        if (rest > 0) time += 2.7 + (0.185 + 0.35 * fmax(0.0, rest - 0.5)) * across * steps;
    } else {
        const double full = floor(tiles / 512), rest = tiles / 512 - full;
        time = full * (3 + 1.03 * steps) + (rest > 0 ? 2.5 + (0.28 + 0.75 * rest) * steps : 0);
    }
    // the weights' stream overlaps the products, not wholly
    const double stream = a.grad ? 0.0 : expected_weight_bytes(a) / 4.8e6;
    return 3 + fmax(time, stream) + 0.1 * fmin(time, stream);
}

bool group_tile_ok(const GroupArgs &a, GroupTileKind kind)
{
    return with_tiles(a, [&](auto t) { return decltype(t)::ok(a, kind); });
}

hipError_t group_tile_launch(const GroupArgs &a, GroupTileKind kind, hipStream_t stream)
{
    return with_tiles(a, [&](auto t) { return decltype(t)::launch(a, kind, stream); });
}

}  // namespace mm
