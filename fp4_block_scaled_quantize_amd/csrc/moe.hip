// moe.hip -- the router's choice among experts, and a whole mixture-of-experts
// layer over quantized weights for at most 16 tokens (quant_prune_distill/574
// "Эксперименты": weight-only NVFP4 with a memory-bound kernel for small-batch
// generation; here with the experts' matrices in the place of one).
//
//   y_i = res_i + sum_k w_ik D_e (act(G_e x_i) * (U_e x_i)),  e = ids_ik
//
// Two launches.  k_moe_up: a workgroup for 16 columns of one expert's gate and
// up matrices, the tokens that chose it as the rows of the product; it writes
// h = act(gate) up as two bf16 terms (17 bits of h: one bf16 would round what
// the down projection sums).  k_moe_down: a workgroup for 16 outputs, all
// experts one after another: a wave folds each expert's sums into its tokens'
// outputs with the router's weight in binary32, and the waves' sums join in
// LDS in a fixed order, so that no atomics and no partial sums in memory are
// needed and the same inputs give the same bits.
//
// Both read every byte of the chosen experts' weights once and nothing else
// of weight, so they are bound by memory (up + down: 4096 x 1536, NVFP4, 37
// experts met by 16 tokens, 262 + 131 MB in 62 + 47 us, 4.2 and 2.8 TB/s; 4096 x
// 11008, MXFP4, 5 met by 3 tokens, 240 + 120 MB in 44 + 29 us, 5.4 and 4.1; one
// token's 8 experts of 2048 x 768, 14 + 7 MB, 9.0 + 7.6 us, of which the
// latencies of a launch, the ids and the first chunk are most).  What keeps the
// down projection of many tokens from the copy's rate is the LDS: a slot holds the
// rows of h of its expert's tokens beside the weights, each wave its own, so that
// fewer bytes of weights are under way the more tokens an expert has (E2M1, block
// 16: 64 KiB a CU at 2, 40, 24 and 12 at 4, 8 and 16).  16 tokens, the whole layer,
// 4096 x 11008, NVFP4: top 2 of 8 experts 609 MB in 157 us (3.9 TB/s), of 4 304 MB
// in 105 (2.9), of 2, all tokens on both, 152 MB in 76 (2.0).  Nor do hidden / 16
// workgroups fit the CUs but at multiples of 4096: top 6 of 64, 47 met, 4096 x 1536
// 4.3 TB/s, 7168 x 2048 4.5, 5120 x 1536 3.6, 2048 x 1408 2.6.
//
// As in the weight-only product a wave
// streams 128-element chunks with loads straight into its own LDS ring, where
// their order keeps four lanes on one 64-byte run, and takes the fragments
// from there.  A wave's chunks are a contiguous part of the workgroup's
// (expert, chunk) list, which is the same length for every wave whatever the
// number of experts, and crosses few expert borders.
//
// A workgroup sorts the (token, choice) pairs by expert itself, from the ids:
// at most 256, one a thread.  Rows of the product are the tokens of one expert,
// a row of a matrix instruction's result depends on its own row of them alone,
// and the rows past the tokens, which repeat the last, are never folded: nothing
// of one token reaches another's outputs (NaN included).
#include "epilogue_device.hpp"
#include "fp4_device.hpp"
#include "fp4_internal.h"
#include "gemm_device.hpp"

namespace fp4 {

constexpr int kMoePairs = kMoeMaxTokens * kMoeMaxTop;      // 256: a pair's index is a byte
constexpr int kNoExpert = 0x7FFFFFFF;

// One side's weights as a wave streams them: RG groups of 16 rows of an
// expert's matrix, K elements each.
struct MoeSide {
    const uint8_t* q; const uint8_t* s;   // of expert 0
    int64_t expert_q, expert_s;           // bytes from an expert to the next
    uint32_t row0, row1;                  // the groups' first rows in an expert
    int32_t k;
    const uint16_t* x;                    // rows of the other operand, K elements
    int64_t ldx, plane;                   // plane: from its first bf16 term to its second
};

// A slot of a wave's ring: a chunk of SUB runs of 128 elements of K for 16 RG
// rows of W (as in the weight-only product's slot), their scales, and XR rows of
// XP terms of x, whose pieces of 256 bytes lie term by term, row by row, run by
// run, four to a load.
template <int RG, int XR, int XP, int ELEM, int BLOCK, int SUB>
struct MoeSlot {
    static constexpr int K = 128 * SUB;
    static constexpr int WP = WoRow<ELEM, SUB>::WP, WB = WoRow<ELEM, SUB>::WB, WD = WP / 64;
    static constexpr int SCB = K / BLOCK, SDW = SCB / 4;
    static constexpr int NSC = (RG * 16 * SDW + 63) / 64;
    static constexpr int W = 0, SC = RG * 16 * WP;
    static constexpr int X = SC + RG * 16 * SCB;
    static constexpr int Pieces = XR * XP * SUB, XL = (Pieces + 3) / 4;
    static constexpr int Bytes = X + 256 * Pieces;
    static constexpr int Loads = RG * WD + NSC + XL;
};

// Slots of a wave and waves that stream, within `budget` bytes of LDS for NW
// waves: up to eight slots each, and where two do not fit, fewer waves.
template <typename S, int NW, int BUDGET>
struct MoeShape {
    static constexpr int Fit = BUDGET / (NW * S::Bytes);
    static constexpr int slots()
    {
        int d = Fit > 8 ? 8 : Fit < 2 ? 2 : Fit;
        while ((d - 1) * S::Loads >= 64) --d;
        return d;
    }
    static constexpr int D = slots();
    static constexpr int Waves = Fit >= 2 ? NW : BUDGET / (2 * S::Bytes);
    static constexpr int Bytes = Waves * D * S::Bytes;
};

// `behind` whole slots of LOADS loads each may still be under way.
template <int LOADS, int MOST>
__device__ __forceinline__ void wait_slots(int behind)
{
    if constexpr (MOST == 0) {
        wait_vmcnt<0>();
    } else {
        if (behind >= MOST) wait_vmcnt<MOST * LOADS>();
        else wait_slots<LOADS, MOST - 1>(behind);
    }
}

// Streams items first .. first + mine - 1 of a list of (expert, chunk) pairs,
// K / (128 SUB) chunks to an expert.  expert(a) says who the a-th is:
// {id, tokens, their rows of x}.  fold(a, acc) takes the sums over this call's
// chunks of it: acc[g][r] is row 4 (lane / 16) + r of the expert's tokens, column
// lane % 16 of group g.
struct MoeExpert { int id, tokens; const uint8_t* rows; };

template <int D, int RG, int XR, int XP, int ELEM, int BLOCK, int SUB, bool SPLIT, bool POW2, typename E, typename F>
__device__ __forceinline__ void moe_stream(uint8_t* ring, const MoeSide& s, const float* sdec, int first, int mine, int lane,
                                           E expert, F fold)
{
    constexpr bool WIDE = ELEM >= 2;
    using S = MoeSlot<RG, XR, XP, ELEM, BLOCK, SUB>;
    static_assert(SUB == 1 || !WIDE, "two runs a chunk for the 4-bit grids");
    static_assert(D >= 2 && (D - 1) * S::Loads < 64, "ring");
    if (mine <= 0) return;
    const int r16 = lane & 15, grp = lane >> 4;
    const int nch = s.k / S::K;
    const uint32_t rowb = (uint32_t)((int64_t)s.k * (ELEM <= 1 ? 4 : ELEM <= 3 ? 8 : 6) / 8);
    const uint32_t srow = (uint32_t)(s.k / BLOCK);

    // byte offsets of this lane's loads in an expert's codes and scales
    uint32_t wsrc[RG][S::WD];
    bool wact[S::WD];
#pragma unroll
    for (int k = 0; k < S::WD; ++k) {
        const int r = S::WP == 128 ? 8 * k + (lane >> 3) : lane >> 2;
        const int pc = S::WP == 128 ? (lane & 7) ^ wo_swz8(r) : (lane & 3) ^ wo_swz(r);
        wact[k] = 16 * pc < S::WB;
#pragma unroll
        for (int g = 0; g < RG; ++g) wsrc[g][k] = ((g ? s.row1 : s.row0) + (uint32_t)r) * rowb + 16u * (uint32_t)pc;
    }
    uint32_t ssrc[S::NSC];
    bool sact[S::NSC];
#pragma unroll
    for (int j = 0; j < S::NSC; ++j) {
        const int f = 64 * j + lane, rr = f / S::SDW;
        sact[j] = rr < 16 * RG;
        const int r = sact[j] ? rr : 16 * RG - 1;
        ssrc[j] = ((r < 16 ? s.row0 : s.row1) + (uint32_t)(r & 15)) * srow + 4u * (uint32_t)(f % S::SDW);
    }
    // x: load q, lane l takes 16 bytes of piece 4 q + l / 16: run piece % SUB of
    // row piece / SUB, which is token row % XR (past the expert's last: the last
    // again), term row / XR
    const uint16_t* xsrc[S::XL];
    const uint8_t* qe = nullptr;
    const uint8_t* se = nullptr;
    int ia = first / nch, ik = first - ia * nch;           // the next chunk to load
    auto enter = [&](int a) {
        const MoeExpert w = expert(a);
        const int e = __builtin_amdgcn_readfirstlane(w.id), n = __builtin_amdgcn_readfirstlane(w.tokens);
        qe = s.q + (int64_t)e * s.expert_q;
        se = s.s + (int64_t)e * s.expert_s;
#pragma unroll
        for (int q = 0; q < S::XL; ++q) {
            const int piece = 4 * q + grp, row = piece / SUB, m = row % XR, h = row / XR;
            xsrc[q] = s.x + (int64_t)w.rows[m < n ? m : n - 1] * s.ldx + (XP > 1 && h == 1 ? s.plane : 0) +
                      128 * (piece % SUB) + 8 * (r16 ^ (m & 7));
        }
    };
    enter(ia);
    auto issue = [&](int d) {
        uint8_t* const sl = ring + d * S::Bytes;
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int k = 0; k < S::WD; ++k) {
                const uint8_t* const from = qe + wsrc[g][k] + (uint32_t)ik * (uint32_t)S::WB;
                uint8_t* const to = sl + S::W + 16 * S::WP * g + 1024 * k;
                // whole lines: 4096 x 1536, 37 experts met, 67 + 49 us -> 66 + 48; 4096 x 11008, 5 met, 48 + 31 -> 45 + 29
                if (S::WB == 128) dma16_once(from, to);
                else if (ELEM < 4 || wact[k]) dma16(from, to);
            }
#pragma unroll
        for (int j = 0; j < S::NSC; ++j)
            if (sact[j]) dma4(se + ssrc[j] + (uint32_t)ik * (uint32_t)S::SCB, sl + S::SC + 256 * j);
#pragma unroll
        for (int q = 0; q < S::XL; ++q)
            if (S::Pieces % 4 == 0 || 4 * q + grp < S::Pieces) dma16(xsrc[q] + (int64_t)ik * S::K, sl + S::X + 1024 * q);
    };
    // a chain of sums for each term: a matrix instruction waits for the one before it
    v4f acc[RG][XP];
    auto clear = [&] {
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int h = 0; h < XP; ++h) acc[g][h] = v4f{0.f, 0.f, 0.f, 0.f};
    };
    clear();
    const int mr = r16 < XR ? r16 : XR - 1;
    auto xoff = [&](int h, int u, int tt) {
        return S::X + 256 * ((h * XR + mr) * SUB + u) + 16 * ((4 * grp + tt) ^ (mr & 7));
    };
    auto woff = [&](int u, int j) {
        if (S::WP == 64) return S::W + 64 * r16 + 16 * (grp ^ wo_swz(r16));
        const int byte = ELEM >= 4 ? 24 * grp + 8 * j : ELEM >= 2 ? 32 * grp + 16 * j : 64 * u + 16 * grp;
        return S::W + S::WP * r16 + 16 * ((byte >> 4) ^ wo_swz8(r16)) + (byte & 15);
    };
    auto soff = [&](int u) { return S::SC + S::SCB * r16 + (BLOCK == 16 ? 8 * u + 2 * grp : 4 * u + grp); };
    auto consume = [&](int d) {
        const uint8_t* const sl = ring + d * S::Bytes;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            v4i xf[XP][4];
#pragma unroll
            for (int h = 0; h < XP; ++h)
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) xf[h][tt] = *reinterpret_cast<const v4i*>(sl + xoff(h, u, tt));
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                v4i wv;
                uint32_t dw[8];
                if constexpr (!WIDE) {
                    wv = *reinterpret_cast<const v4i*>(sl + woff(u, 0) + 16 * S::WP * g);
                } else if constexpr (ELEM <= 3) {
                    const v4i w0 = *reinterpret_cast<const v4i*>(sl + woff(u, 0) + 16 * S::WP * g);
                    const v4i w1 = *reinterpret_cast<const v4i*>(sl + woff(u, 1) + 16 * S::WP * g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) { dw[i] = (uint32_t)w0[i]; dw[4 + i] = (uint32_t)w1[i]; }
                } else {
#pragma unroll
                    for (int j = 0; j < 3; ++j) {
                        const uint64_t v = *reinterpret_cast<const uint64_t*>(sl + woff(u, j) + 16 * S::WP * g);
                        dw[2 * j] = (uint32_t)v;
                        dw[2 * j + 1] = (uint32_t)(v >> 32);
                    }
                    dw[6] = dw[7] = 0u;
                }
                const uint32_t sc = BLOCK == 16 ? (uint32_t)*reinterpret_cast<const uint16_t*>(sl + soff(u) + 16 * S::SCB * g)
                                                : (uint32_t)sl[soff(u) + 16 * S::SCB * g];
                const float s0 = sdec[sc & 0xFFu], s1 = BLOCK == 16 ? sdec[(sc >> 8) & 0xFFu] : s0;
#pragma unroll
                for (int tt = 0; tt < 4; ++tt) {
                    const float st = tt < 2 ? s0 : s1;                  // elements 0..15: the first block
                    v4i hi, lo;
                    if constexpr (WIDE) dq8_any<ELEM, SPLIT, true>(dw, tt, st, hi, lo);
                    else if constexpr (SPLIT) dq8_bf16_split<ELEM == 1, true>((uint32_t)wv[tt], st, hi, lo);
                    else hi = dq8_bf16<POW2, ELEM == 1>((uint32_t)wv[tt], st);
#pragma unroll
                    for (int h = 0; h < XP; ++h) {
                        acc[g][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xf[h][tt]),
                                                                            __builtin_bit_cast(v8bf, hi), acc[g][h], 0, 0, 0);
                        if (SPLIT)
                            acc[g][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xf[h][tt]),
                                                                                __builtin_bit_cast(v8bf, lo), acc[g][h], 0, 0, 0);
                    }
                }
            }
        }
        // the slot's reads have returned before a load may overwrite it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };

    int issued = 0, to = 0;               // to: the slot of the next load
    auto advance = [&] {
        issue(to);
        to = to + 1 == D ? 0 : to + 1;
        ++issued;
        if (++ik == nch) {
            ik = 0;
            ++ia;
            if (issued < mine) enter(ia);
        }
    };
    while (issued < D && issued < mine) advance();
    int at = 0, ca = first / nch, ck = first - ca * nch;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        wait_slots<S::Loads, D - 1>(mine - 1 - i);         // loads of later chunks that are still under way
        consume(at);
        at = at + 1 == D ? 0 : at + 1;
        if (issued < mine) advance();
        if (++ck == nch || i + 1 == mine) {
            v4f sum[RG];
#pragma unroll
            for (int g = 0; g < RG; ++g) sum[g] = XP == 1 ? acc[g][0] : acc[g][0] + acc[g][XP - 1];
            fold(ca, sum);
            clear();
            ck = 0;
            ++ca;
        }
    }
}

__device__ __forceinline__ ScaleFmt device_fmt(const ScaleFmtHost& f)
{
    return ScaleFmt{f.ebits, f.mbits, f.bias, f.maxcode, f.smax, f.is_e8m0};
}

// f(std::integral_constant<int, XR>) for an expert's number of tokens, XR at
// most the launch's MAXR
template <int MAXR, typename F>
__device__ __forceinline__ void moe_rows(int tokens, F f)
{
    if (MAXR == 1 || tokens <= 1) f(std::integral_constant<int, 1>{});
    else if (tokens <= 2) f(std::integral_constant<int, MAXR >= 2 ? 2 : 1>{});
    else if (MAXR == 4 || tokens <= 4) f(std::integral_constant<int, MAXR >= 4 ? 4 : 1>{});
    else if (tokens <= 8) f(std::integral_constant<int, MAXR >= 8 ? 8 : 1>{});
    else f(std::integral_constant<int, MAXR >= 16 ? 16 : 1>{});
}

// Bits from .. to - 1 of 256.
__device__ __forceinline__ bool any_bit(const uint64_t (&m)[kMoePairs / 64], int from, int to)
{
    uint64_t got = 0;
#pragma unroll
    for (int w = 0; w < kMoePairs / 64; ++w) {
        const int lo = from - 64 * w, hi = to - 64 * w;
        const uint64_t above = lo <= 0 ? ~0ull : lo >= 64 ? 0ull : ~0ull << lo;
        const uint64_t below = hi <= 0 ? 0ull : hi >= 64 ? ~0ull : ~(~0ull << hi);
        got |= m[w] & above & below;
    }
    return got != 0;
}

// Rings of 51 KiB, the most that lets three workgroups share a CU (two of them
// with larger rings: 4096 x 11008, 5 experts met, 55 us against 48, when the
// weights still went through the caches; now 44); 40 KiB
// leave fewer waves two slots (4096 x 1536, 37 met, 65.6 us against 62.4).  For
// one token, whose few workgroups do not fill the CUs so often, deeper rings
// and two.
constexpr int kMoeUpWaves = 4;
template <int MAXR>
constexpr int kMoeUpBudget = (MAXR == 1 ? 68 : 51) * 1024;
constexpr int kMoeDownWaves = 16;

// ---------------------------------------------------------------------------
// The gate and up projections: a workgroup for 16 columns of one expert, its
// four waves sharing K.  blockIdx.y is a (token, choice) pair, of which the
// first that names its expert does the work, or an expert where those are
// fewer; the others leave.  (A wave for each 16 columns with all of K, whose
// gate and up meet in registers, is slower: 4096 x 11008, 5 experts met 75 us
// against 61, 4096 x 1536, 37 met 83 against 79: fewer, longer workgroups end
// less evenly.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ void put_hidden(const MoeLaunch& p, float gate, float up, float f, int pair, int64_t n)
{
    float h = gate * f;
    with_act(p.act, [&](auto act) { h = act_value<decltype(act)::value>(h); });
    h *= up * f;
    // h as the sum of two bf16, both to nearest, 17 bits (a third term would cost
    // the down projection's rings half as much again).  A finite h past bf16's
    // largest value is cut instead: it must not become an infinity.
    uint32_t hi = (uint32_t)f32_to_bf16_rne(h) << 16;
    if ((hi & 0x7FFFFFFFu) == 0x7F800000u) hi = f_bits(h) & 0xFFFF0000u;
    const float left = h - bits_f(hi);
    const int64_t to = (int64_t)pair * p.ffn + n;
    p.h[to] = (uint16_t)(hi >> 16);
    p.h[to + (int64_t)p.m * p.top * p.ffn] = left == left ? (uint16_t)f32_to_bf16_rne(left) : (uint16_t)0;
}

template <int ELEM, int BLOCK, int SUB, bool SPLIT, bool POW2, int MAXR>
__global__ __launch_bounds__(64 * kMoeUpWaves) void k_moe_up(MoeLaunch p)
{
    constexpr int NW = kMoeUpWaves;
    static_assert(64 * NW >= kMoePairs, "a thread for each pair");
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ float sdec[256];
    __shared__ uint64_t found[2][kMoePairs / 64];
    __shared__ uint8_t pair[kMoeMaxTokens], token[kMoeMaxTokens];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = p.m * p.top, y = blockIdx.y;
    const bool by_pair = pairs <= p.experts;
    const int e = by_pair ? p.ids[y] : y;
    if (e < 0 || e >= p.experts) return;                   // the whole workgroup, here and below
    const bool match = tid < pairs && p.ids[tid] == e;
    const float g = p.up.g[0], pw = split_pow2(g), gres = g / pw;
    const float f = gres * (p.up.scale ? p.up.scale[e] : 1.0f);
    const ScaleFmt fw = device_fmt(p.up.fmt);
    for (int c = tid; c < 256; c += 64 * NW) sdec[c] = scale_decode_any((uint32_t)c, fw) * pw;
    const uint64_t here = __builtin_amdgcn_ballot_w64(match);
    if (lane == 0) found[0][wave] = here;
    __syncthreads();
    uint64_t all[kMoePairs / 64];
#pragma unroll
    for (int w = 0; w < kMoePairs / 64; ++w) all[w] = found[0][w];
    if (by_pair ? any_bit(all, 0, y) : !any_bit(all, 0, kMoePairs)) return;
    // a token that names the expert again has it once
    const int tok = tid / p.top;
    const bool keep = match && !any_bit(all, tok * p.top, tid);
    const uint64_t kept = __builtin_amdgcn_ballot_w64(keep);
    if (lane == 0) found[1][wave] = kept;
    __syncthreads();
    int before = __builtin_popcountll(kept & ((1ull << lane) - 1)), cnt = 0;
#pragma unroll
    for (int w = 0; w < kMoePairs / 64; ++w) {
        const int n = __builtin_popcountll(found[1][w]);
        before += w < wave ? n : 0;
        cnt += n;
    }
    if (keep) {
        pair[before] = (uint8_t)tid;
        token[before] = (uint8_t)tok;
    }
    cnt = __builtin_amdgcn_readfirstlane(cnt);
    __syncthreads();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    MoeSide s;
    s.q = p.up.q; s.s = p.up.s;
    s.expert_q = p.up.expert_q; s.expert_s = p.up.expert_s;
    s.row0 = (uint32_t)n0; s.row1 = (uint32_t)(p.ffn + n0);
    s.k = (int32_t)p.hidden;
    s.x = p.x; s.ldx = p.ldx; s.plane = 0;
    // a wave's sums: 256 of the gate, 256 of the up matrix, where its ring was
    int stream = 0, ring = 0;
    moe_rows<MAXR>(cnt, [&](auto rows) {
        constexpr int XR = decltype(rows)::value;
        using S = MoeSlot<2, XR, 1, ELEM, BLOCK, SUB>;
        using Shape = MoeShape<S, NW, kMoeUpBudget<MAXR>>;
        constexpr int NA = Shape::Waves;
        static_assert(Shape::D * S::Bytes >= 2048, "a wave's sums");
        stream = NA;
        ring = Shape::D * S::Bytes;
        const int nch = s.k / S::K, first = nch * wave / NA, mine = nch * (wave + 1) / NA - first;
        if (wave >= NA) return;
        v4f* const sums = reinterpret_cast<v4f*>(lds + wave * ring);
        auto put = [&](int, const v4f (&acc)[2]) {
            sums[lane] = acc[0];
            sums[64 + lane] = acc[1];
        };
        // its chunks end with the wave's last, when all that it loaded has been read
        if (mine > 0)
            moe_stream<Shape::D, 2, XR, 1, ELEM, BLOCK, SUB, SPLIT, POW2>(lds + wave * ring, s, sdec, first, mine, lane,
                                                                          [&](int) { return MoeExpert{e, cnt, token}; }, put);
        else put(0, {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}});
    });
    __syncthreads();
    const int j = tid >> 4, n = tid & 15;
    if (j >= cnt) return;
    const int at = 4 * (16 * (j >> 2) + n) + (j & 3);
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w >= stream) break;
        const float* const sums = reinterpret_cast<const float*>(lds + w * ring);
        gate += sums[at];
        up += sums[256 + at];
    }
    put_hidden(p, gate, up, f, pair[j], n0 + n);
}

// ---------------------------------------------------------------------------
// The down projection.  The table of all pairs by expert, built by each
// workgroup: the active experts in order of their number of tokens' class (at
// most 2, 4, 8, 16: each class has rings of its own depth, since a slot holds the
// rows of its tokens), in a class by their first pair.
// ---------------------------------------------------------------------------
constexpr int kMoeClasses = 4;
struct MoeTable {
    int32_t count[kMoeClasses];           // active experts of a class
    int32_t expert[kMoePairs];
    uint8_t tokens[kMoePairs];
    uint8_t pair[kMoePairs][kMoeMaxTokens];
    uint8_t tok[kMoePairs];               // of a pair
    float w[kMoePairs];                   // of a pair: the router's weight times the expert's scale
};
struct MoeScratch {
    int32_t id[kMoePairs];
    int32_t place[kMoePairs];             // of the active expert that a first pair stands for
    int32_t waves[kMoePairs / 64][kMoeClasses];
};

// Called by all threads (at least 256); scratch may be the ring.  An id that a
// token names again adds its weight to the first; one outside the experts is
// dropped.
__device__ __forceinline__ void moe_table(const MoeLaunch& p, MoeTable& t, MoeScratch& s, int tid, float gres)
{
    const int pairs = p.m * p.top;
    const bool in = tid < pairs;
    const int tok = in ? tid / p.top : 0, k = tid - tok * p.top;
    float w = in ? p.weights[tid] : 0.0f;
    int id = in ? p.ids[tid] : -1;
    if (tid < kMoePairs) s.id[tid] = id;
    __syncthreads();
    bool again = false;
    if (in) {
        for (int j = 0; j < k; ++j) again |= s.id[tok * p.top + j] == id;
        if (!again)
            for (int j = k + 1; j < p.top; ++j)
                if (s.id[tok * p.top + j] == id) w += p.weights[tok * p.top + j];
    }
    __syncthreads();
    if (again || id < 0 || id >= p.experts) id = kNoExpert;
    if (in) {
        s.id[tid] = id;
        t.w[tid] = w * (p.down.scale && id != kNoExpert ? gres * p.down.scale[id] : gres);
        t.tok[tid] = (uint8_t)tok;
    } else if (tid < kMoePairs) {
        s.id[tid] = -1;
    }
    __syncthreads();
    // of the same expert: all, those before this pair, the first
    int n = 0, before = 0, first = kMoePairs;
    if (in && id != kNoExpert) {
        for (int q = 0; q < pairs; q += 4) {               // past the pairs: -1
            const int4 o = *reinterpret_cast<const int4*>(&s.id[q]);
            const int v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool same = v[i] == id;
                n += same;
                before += same && q + i < tid;
                first = same && q + i < first ? q + i : first;
            }
        }
    }
    const bool lead = n > 0 && before == 0;
    const int cls = n <= 2 ? 0 : n <= 4 ? 1 : n <= 8 ? 2 : 3;
    int rank = 0;
#pragma unroll
    for (int c = 0; c < kMoeClasses; ++c) {
        const uint64_t b = __builtin_amdgcn_ballot_w64(lead && cls == c);
        if (cls == c) rank = __builtin_popcountll(b & ((1ull << (tid & 63)) - 1));
        if ((tid & 63) == 0 && tid < kMoePairs) s.waves[tid >> 6][c] = __builtin_popcountll(b);
    }
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int c = 0; c < kMoeClasses; ++c) {
        int all = 0;
#pragma unroll
        for (int u = 0; u < kMoePairs / 64; ++u) {
            const int v = s.waves[u][c];
            if (c == cls && u < (tid >> 6)) rank += v;
            all += v;
        }
        if (c < cls) base += all;
        if (tid == 0) t.count[c] = all;
    }
    if (lead) {
        s.place[tid] = base + rank;
        t.expert[base + rank] = id;
        t.tokens[base + rank] = (uint8_t)n;
    }
    __syncthreads();
    if (n > 0) t.pair[s.place[first]][before] = (uint8_t)tid;
    __syncthreads();
}

// One token's pairs, by the first wave: every expert that it names has one.
__device__ __forceinline__ void moe_table_one(const MoeLaunch& p, MoeTable& t, int tid, float gres)
{
    if (tid < 64) {
        const bool in = tid < p.top;
        const int id = in ? p.ids[tid] : -1;
        float w = in ? p.weights[tid] : 0.0f;
        bool again = false;
        float more = 0.0f;
#pragma unroll
        for (int j = 0; j < kMoeMaxTop; ++j) {             // lanes past the choices: -1
            const bool same = __builtin_amdgcn_readlane(id, j) == id;
            const float wj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(w), j));
            again |= same && j < tid;
            if (same && j > tid) more += wj;
        }
        w += more;
        const bool lead = in && !again && id >= 0 && id < p.experts;
        const uint64_t all = __builtin_amdgcn_ballot_w64(lead);
        if (lead) {
            const int a = __builtin_popcountll(all & ((1ull << tid) - 1));
            t.expert[a] = id;
            t.tokens[a] = 1;
            t.pair[a][0] = (uint8_t)tid;
            t.tok[tid] = 0;
            t.w[tid] = w * (p.down.scale ? gres * p.down.scale[id] : gres);
        }
        if (tid < kMoeClasses) t.count[tid] = tid == 0 ? __builtin_popcountll(all) : 0;
    }
    __syncthreads();
}

// What the LDS has left for the rings beside the table, the scales and the sums.
template <int MAXR>
constexpr int kMoeDownBudget = 160 * 1024 - (int)sizeof(MoeTable) - 4 * 256 - 4 * 16 * MAXR * kMoeDownWaves - 64;

template <int ELEM, int BLOCK, int SUB, bool SPLIT, bool POW2, int MAXR>
__global__ __launch_bounds__(64 * kMoeDownWaves) void k_moe_down(MoeLaunch p)
{
    constexpr int NW = kMoeDownWaves;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ MoeTable t;
    __shared__ float sdec[256];
    __shared__ float tot[NW][MAXR][16];   // a wave's sums: token, column
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float g = p.down.g[0], pw = split_pow2(g), gres = g / pw;
    const ScaleFmt fw = device_fmt(p.down.fmt);
    if (MAXR == 1) moe_table_one(p, t, tid, gres);
    else moe_table(p, t, *reinterpret_cast<MoeScratch*>(lds), tid, gres);
    for (int c = tid; c < 256; c += 64 * NW) sdec[c] = scale_decode_any((uint32_t)c, fw) * pw;
    for (int i = lane; i < 16 * MAXR; i += 64) (&tot[wave][0][0])[i] = 0.0f;
    __syncthreads();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    MoeSide s;
    s.q = p.down.q; s.s = p.down.s;
    s.expert_q = p.down.expert_q; s.expert_s = p.down.expert_s;
    s.row0 = s.row1 = (uint32_t)n0;
    s.k = (int32_t)p.ffn;
    s.x = p.h; s.ldx = p.ffn; s.plane = (int64_t)p.m * p.top * p.ffn;
    const int nch = s.k / (128 * SUB);
    int base = 0;
    auto run = [&](auto rows, int count) {
        constexpr int XR = decltype(rows)::value;
        using S = MoeSlot<1, XR, 2, ELEM, BLOCK, SUB>;
        using Shape = MoeShape<S, NW, kMoeDownBudget<MAXR>>;
        constexpr int NA = Shape::Waves;
        const int a0 = base;
        base += count;
        if (count == 0 || wave >= NA) return;
        // this wave's part of the class's (expert, chunk) list
        const int items = count * nch, first = (int)((int64_t)items * wave / NA);
        moe_stream<Shape::D, 1, XR, 2, ELEM, BLOCK, SUB, SPLIT, POW2>(
            lds + wave * (Shape::D * S::Bytes), s, sdec, first, (int)((int64_t)items * (wave + 1) / NA) - first, lane,
            [&](int a) { return MoeExpert{t.expert[a0 + a], t.tokens[a0 + a], t.pair[a0 + a]}; },
            [&](int a, const v4f (&acc)[1]) {
                const int n = t.tokens[a0 + a];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 4 * (lane >> 4) + r;
                    if (j < n) {
                        const int q = t.pair[a0 + a][j];
                        float& to = tot[wave][t.tok[q]][lane & 15];
                        to = __builtin_fmaf(t.w[q], acc[0][r], to);
                    }
                }
            });
    };
    // a class's rings lie where another's did: a wave's own loads have landed and
    // been read by then, but the classes cut the LDS differently
    run(std::integral_constant<int, MAXR == 1 ? 1 : 2>{}, t.count[0]);
    if constexpr (MAXR >= 4) {
        if (t.count[1]) {
            __syncthreads();
            run(std::integral_constant<int, 4>{}, t.count[1]);
        }
    }
    if constexpr (MAXR >= 16) {
        if (t.count[2]) {
            __syncthreads();
            run(std::integral_constant<int, 8>{}, t.count[2]);
        }
        if (t.count[3]) {
            __syncthreads();
            run(std::integral_constant<int, 16>{}, t.count[3]);
        }
    }
    __syncthreads();
    if (tid >= 256) return;
    const int m = tid >> 4;
    if (m >= p.m) return;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) y += tot[w][m][tid & 15];
    const int64_t n = n0 + (tid & 15);
    if (p.res) y += bf16_lo(p.res[m * p.ldres + n]);
    p.y[m * p.ldy + n] = (uint16_t)f32_to_bf16_rne(y);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// the largest of the rings that a launch may take
template <int NW, int BUDGET, int RG, int XP, int ELEM, int BLOCK, int SUB, int MAXR>
constexpr size_t ring_bytes()
{
    constexpr int b[5] = {MoeShape<MoeSlot<RG, 1, XP, ELEM, BLOCK, SUB>, NW, BUDGET>::Bytes,
                          MoeShape<MoeSlot<RG, 2, XP, ELEM, BLOCK, SUB>, NW, BUDGET>::Bytes,
                          MoeShape<MoeSlot<RG, 4, XP, ELEM, BLOCK, SUB>, NW, BUDGET>::Bytes,
                          MoeShape<MoeSlot<RG, 8, XP, ELEM, BLOCK, SUB>, NW, BUDGET>::Bytes,
                          MoeShape<MoeSlot<RG, 16, XP, ELEM, BLOCK, SUB>, NW, BUDGET>::Bytes};
    size_t most = sizeof(MoeScratch);
    for (int i = 0, r = 1; i < 5 && r <= MAXR; ++i, r *= 2) most = (size_t)b[i] > most ? (size_t)b[i] : most;
    return most;
}

template <int ELEM, int BLOCK, int SUB, bool SPLIT, bool POW2, int MAXR>
static hipError_t run_moe(const MoeLaunch& p, bool up, hipStream_t s)
{
    if (up) {
        constexpr size_t sh = ring_bytes<kMoeUpWaves, kMoeUpBudget<MAXR>, 2, 1, ELEM, BLOCK, SUB, MAXR>();
        static_assert(sh <= kMoeUpBudget<MAXR>, "LDS");
        const int most = p.m * p.top < p.experts ? p.m * p.top : p.experts;
        if (sh + 2 * 1024 > 64 * 1024) {                   // with the scales and the tokens
            const hipError_t e = allow_lds(k_moe_up<ELEM, BLOCK, SUB, SPLIT, POW2, MAXR>, sh);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((k_moe_up<ELEM, BLOCK, SUB, SPLIT, POW2, MAXR>), dim3((unsigned)(p.ffn / 16), (unsigned)most),
                           dim3(64 * kMoeUpWaves), sh, s, p);
    } else {
        constexpr size_t sh = ring_bytes<kMoeDownWaves, kMoeDownBudget<MAXR>, 1, 2, ELEM, BLOCK, SUB, MAXR>();
        static_assert(sh <= kMoeDownBudget<MAXR>, "LDS");
        const hipError_t e = allow_lds(k_moe_down<ELEM, BLOCK, SUB, SPLIT, POW2, MAXR>, sh);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((k_moe_down<ELEM, BLOCK, SUB, SPLIT, POW2, MAXR>), dim3((unsigned)(p.hidden / 16)),
                           dim3(64 * kMoeDownWaves), sh, s, p);
    }
    return hipGetLastError();
}

template <int ELEM, int BLOCK, int SUB, bool SPLIT, bool POW2>
static hipError_t run_moe_tokens(const MoeLaunch& p, bool up, hipStream_t s)
{
    if (p.m == 1) return run_moe<ELEM, BLOCK, SUB, SPLIT, POW2, 1>(p, up, s);
    if (p.m <= 4) return run_moe<ELEM, BLOCK, SUB, SPLIT, POW2, 4>(p, up, s);
    return run_moe<ELEM, BLOCK, SUB, SPLIT, POW2, 16>(p, up, s);
}

// Chunks of two runs for the 4-bit grids: a load's rows are whole 128-byte
// lines then (streaming alone, 37 experts of 4096 x 1536: 64 -> 54 us for gate
// and up, 38 -> 32 for down; K that is an odd multiple of 128 takes one run.
template <int ELEM, int BLOCK, bool SPLIT, bool POW2>
static hipError_t run_moe_chunk(const MoeLaunch& p, bool up, hipStream_t s)
{
    if constexpr (ELEM <= 1)
        if ((up ? p.hidden : p.ffn) % 256 == 0) return run_moe_tokens<ELEM, BLOCK, 2, SPLIT, POW2>(p, up, s);
    return run_moe_tokens<ELEM, BLOCK, 1, SPLIT, POW2>(p, up, s);
}

template <int ELEM, int BLOCK>
static hipError_t run_moe_scales(const MoeLaunch& p, bool up, hipStream_t s)
{
    const MoeWeights& w = up ? p.up : p.down;
    if (!wo_exact_in_bf16(ELEM, w.fmt)) return run_moe_chunk<ELEM, BLOCK, true, false>(p, up, s);
    if constexpr (ELEM == 0)
        if (w.fmt.is_e8m0) return run_moe_chunk<ELEM, BLOCK, false, true>(p, up, s);
    return run_moe_chunk<ELEM, BLOCK, false, false>(p, up, s);
}

template <int ELEM>
static hipError_t run_moe_block(const MoeLaunch& p, bool up, hipStream_t s)
{
    return (up ? p.up : p.down).block == 16 ? run_moe_scales<ELEM, 16>(p, up, s) : run_moe_scales<ELEM, 32>(p, up, s);
}

static hipError_t run_moe_side(const MoeLaunch& p, bool up, hipStream_t s)
{
    switch ((up ? p.up : p.down).elem) {
    case 1: return run_moe_block<1>(p, up, s);
    case 2: return run_moe_block<2>(p, up, s);
    case 3: return run_moe_block<3>(p, up, s);
    case 4: return run_moe_block<4>(p, up, s);
    case 5: return run_moe_block<5>(p, up, s);
    case 6: return run_moe_block<6>(p, up, s);
    default: return run_moe_block<0>(p, up, s);
    }
}

hipError_t launch_moe(const MoeLaunch& p, hipStream_t s)
{
    const hipError_t e = run_moe_side(p, true, s);
    return e != hipSuccess ? e : run_moe_side(p, false, s);
}

// ---------------------------------------------------------------------------
// The router's choice: a workgroup for each row, whose four waves all hold its
// experts' scores, NL a lane.  Up to 256 experts each wave counts, for every key,
// how many of a quarter of the keys are above it, from readlanes, and the counts
// add up to the keys' ranks (128 experts, top 8: 4.3 us; one wave with all keys
// 6.0; rounds of the wave's largest, six cross-lane steps of three values each,
// 7.4).  More experts take the rounds, by the first wave.  Scores are compared
// and divided in binary64: the order of two near scores plus their biases is the
// binary64 formula's, where binary32's exponential would turn neighbours round.
// ---------------------------------------------------------------------------
constexpr int kRouteWaves = 4;

__device__ __forceinline__ uint64_t order_key(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    if ((u & 0x7FFFFFFFFFFFFFFFull) > 0x7FF0000000000000ull) return ~0ull;     // NaN above everything
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

template <int NL>
__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_route(RouteLaunch p)
{
    constexpr bool RANK = NL <= 4;
    __shared__ int32_t part[RANK ? kRouteWaves : 1][RANK ? 64 * NL : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    if (!RANK && wave) return;
    const int E = p.experts;
    float z[NL];
    double score[NL];
    uint64_t key[NL];                     // 0: no candidate
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = 64 * i + lane;
        z[i] = -INFINITY;
        if (e < E) z[i] = p.bf16 ? bf16_lo(((const uint16_t*)p.logits)[row * p.ld + e]) : ((const float*)p.logits)[row * p.ld + e];
        top = fmaxf(top, z[i]);
    }
    double sum = 0.0;
    if (!p.sigmoid) {
#pragma unroll
        for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const double v = z[i];
        // a masked expert is never chosen; the largest logit's own score is 1 (also where it is infinite)
        score[i] = z[i] == -INFINITY ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-v)) : z[i] == top ? 1.0 : exp(v - (double)top);
        sum += score[i];
    }
    if (!p.sigmoid && (p.bias || !p.renormalize)) {        // else it cancels
#pragma unroll
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
#pragma unroll
        for (int i = 0; i < NL; ++i) score[i] /= sum;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = 64 * i + lane;
        key[i] = 0;
        // without a bias the scores' order is the logits', ties and underflow aside
        if (z[i] != -INFINITY) key[i] = order_key(p.bias ? score[i] + (double)p.bias[e < E ? e : 0] : (double)z[i]);
    }
    int32_t* const ids = p.ids + row * p.top;
    float* const weights = p.weights + row * p.top;
    double total = 0.0;
    int rank[NL], found = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        rank[i] = kNoExpert;
        found += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] != 0));
    }
    found = found < p.top ? found : p.top;
    if constexpr (RANK) {
#pragma unroll
        for (int i = 0; i < NL; ++i) rank[i] = 0;
        // the wave's quarter of every lane's keys; lanes past the experts hold none
        auto count = [&](auto above) {
#pragma unroll
            for (int o = 0; o < NL; ++o) {
                const uint32_t hi = (uint32_t)(key[o] >> 32), lo = (uint32_t)key[o];
#pragma unroll
                for (int u = 0; u < 64 / kRouteWaves; ++u) {
                    const int j = 64 / kRouteWaves * wave + u;
                    const uint64_t k = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, j) << 32) |
                                       (uint32_t)__builtin_amdgcn_readlane((int)lo, j);
#pragma unroll
                    for (int i = 0; i < NL; ++i) rank[i] += above(k, i, 64 * o + j);
                }
            }
        };
        auto join = [&] {
#pragma unroll
            for (int i = 0; i < NL; ++i) part[wave][64 * i + lane] = rank[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                rank[i] = 0;
#pragma unroll
                for (int w = 0; w < kRouteWaves; ++w) rank[i] += part[w][64 * i + lane];
            }
        };
        count([&](uint64_t k, int i, int) { return k > key[i]; });
        join();
        // without equal keys the ranks of n are 0 .. n - 1
        int all = 0, sum_of = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            all += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[i] != 0));
            sum_of += key[i] != 0 ? rank[i] : 0;
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) sum_of += __shfl_xor(sum_of, o);
        if (sum_of != all * (all - 1) / 2) {               // equal ones: the lower expert first; the same in every wave
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NL; ++i) rank[i] = 0;
            count([&](uint64_t k, int i, int e) { return k > key[i] || (k == key[i] && e < 64 * i + lane); });
            join();
        }
        if (wave) return;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            if (key[i] == 0) rank[i] = kNoExpert;
            if (rank[i] < p.top) total += score[i];
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) total += __shfl_xor(total, o);
    } else {
        for (int k = 0; k < found; ++k) {
            uint64_t best = 0;
            int e = kNoExpert;
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (key[i] > best) { best = key[i]; e = 64 * i + lane; s = score[i]; }
#pragma unroll
            for (int o = 32; o; o >>= 1) {
                const uint64_t b = ((uint64_t)(uint32_t)__shfl_xor((int)(best >> 32), o) << 32) | (uint32_t)__shfl_xor((int)best, o);
                const int oe = __shfl_xor(e, o);
                const double os = __shfl_xor(s, o);
                if (b > best || (b == best && oe < e)) { best = b; e = oe; s = os; }
            }
            total += s;
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (64 * i + lane == e) { rank[i] = k; key[i] = 0; }
        }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        if (rank[i] >= p.top) continue;
        const double w = !p.renormalize ? score[i] : total == 0.0 ? 0.0 : score[i] / total;
        ids[rank[i]] = 64 * i + lane;
        weights[rank[i]] = (float)(w * (double)p.scale);
    }
    if (lane >= found && lane < p.top) {
        ids[lane] = -1;
        weights[lane] = 0.0f;
    }
}

hipError_t launch_moe_route(const RouteLaunch& p, hipStream_t s)
{
    const dim3 grid((unsigned)p.rows), threads(64 * kRouteWaves);
    if (p.experts <= 64) hipLaunchKernelGGL((k_moe_route<1>), grid, threads, 0, s, p);
    else if (p.experts <= 128) hipLaunchKernelGGL((k_moe_route<2>), grid, threads, 0, s, p);
    else if (p.experts <= 256) hipLaunchKernelGGL((k_moe_route<4>), grid, threads, 0, s, p);
    else hipLaunchKernelGGL((k_moe_route<kMoeMaxRouted / 64>), grid, threads, 0, s, p);
    return hipGetLastError();
}

}  // namespace fp4
