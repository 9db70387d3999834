// moe.hip -- the router's choice among experts, and a whole mixture-of-experts
// layer over quantized weights for at most 16 tokens (quant_prune_distill/574
// "Эксперименты": weight-only NVFP4 with a memory-bound kernel for small-batch
// generation; here with the experts' matrices in the place of one).
//
//   y_i = res_i + sum_k w_ik D_e (act(G_e x_i) * (U_e x_i)),  e = ids_ik
//
// Two launches.  k_moe_up: a workgroup for 16 columns of one expert's gate and
// up matrices, the tokens that chose it as the rows of the product; it writes
// h = act(gate) up as two bf16 terms (16 bits of h: one bf16 would round what
// the down projection sums).  k_moe_down: a workgroup for 16 outputs, all
// experts one after another: a wave folds each expert's sums into its tokens'
// outputs with the router's weight in binary32, and the waves' sums join in
// LDS in a fixed order, so that no atomics and no partial sums in memory are
// needed and the same inputs give the same bits.
//
// Both read every byte of the chosen experts' weights once and nothing else
// of weight, so they are bound by memory; as in the weight-only product a wave
// streams 128-element chunks with loads straight into its own LDS ring, where
// their order keeps four lanes on one 64-byte run, and takes the fragments
// from there.  A wave's chunks are a contiguous part of the workgroup's
// (expert, chunk) list, which is the same length for every wave whatever the
// number of experts, and crosses few expert borders.
//
// A workgroup sorts the (token, choice) pairs by expert itself, from the ids:
// at most 256, one a thread.  Columns of the product are the tokens of one
// expert, so nothing of one token reaches another's outputs (NaN included).
#include "epilogue_device.hpp"
#include "fp4_device.hpp"
#include "fp4_internal.h"
#include "gemm_device.hpp"

namespace fp4 {

constexpr int kMoePairs = kMoeMaxTokens * kMoeMaxTop;      // 256
constexpr int kNoExpert = 0x7FFFFFFF;

// The pairs sorted by expert; experts without a token have no entry.
struct MoeTable {
    int32_t active;                       // experts with tokens
    int32_t expert[kMoePairs];
    uint16_t start[kMoePairs + 1];        // of the active expert's pairs
    uint16_t row[kMoePairs];              // token * top + choice
    uint8_t tok[kMoePairs];
    float w[kMoePairs];
};
struct MoeScratch {
    int32_t raw[kMoePairs], key[kMoePairs], sorted[kMoePairs];
    int32_t waves[kMoePairs / 64];
};

// Called by all threads (at least 256); scratch may be the ring.  An id that a
// token names again adds its weight to the first; one outside the experts is
// dropped.
__device__ __forceinline__ void moe_table(const MoeLaunch& p, MoeTable& t, MoeScratch& s, int tid)
{
    const int pairs = p.m * p.top;
    const bool in = tid < pairs;
    const int tok = in ? tid / p.top : 0, k = tid - tok * p.top;
    float w = 0.0f;
    if (in) {
        s.raw[tid] = p.ids[tid];
        w = p.weights[tid];
    }
    __syncthreads();
    int key = kNoExpert;
    if (in) {
        const int id = s.raw[tid];
        bool again = false;
        for (int j = 0; j < k; ++j) again |= s.raw[tok * p.top + j] == id;
        if (id >= 0 && id < p.experts && !again) {
            key = id;
            for (int j = k + 1; j < p.top; ++j)
                if (s.raw[tok * p.top + j] == id) w += p.weights[tok * p.top + j];
        }
        s.key[tid] = key;
    }
    __syncthreads();
    if (in && key != kNoExpert) {
        int at = 0;
        for (int q = 0; q < pairs; ++q) {
            const int o = s.key[q];
            at += o < key || (o == key && q < tid);
        }
        s.sorted[at] = key;
        t.tok[at] = (uint8_t)tok;
        t.row[at] = (uint16_t)tid;
        t.w[at] = w;
    }
    // pairs that have an expert
    const int mine = __builtin_popcountll(__builtin_amdgcn_ballot_w64(in && key != kNoExpert));
    if ((tid & 63) == 0 && tid < kMoePairs) s.waves[tid >> 6] = mine;
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int i = 0; i < kMoePairs / 64; ++i) n += s.waves[i];
    const bool first = tid < n && (tid == 0 || s.sorted[tid] != s.sorted[tid - 1]);
    const uint64_t lanes = __builtin_amdgcn_ballot_w64(first);
    __syncthreads();
    if ((tid & 63) == 0 && tid < kMoePairs) s.waves[tid >> 6] = __builtin_popcountll(lanes);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kMoePairs / 64; ++i) {
        before += i < (tid >> 6) ? s.waves[i] : 0;
        all += s.waves[i];
    }
    if (first) {
        const int a = before + __builtin_popcountll(lanes & ((1ull << (tid & 63)) - 1));
        t.expert[a] = s.sorted[tid];
        t.start[a] = (uint16_t)tid;
    }
    if (tid == 0) {
        t.active = all;
        t.start[all] = (uint16_t)n;
    }
    __syncthreads();
}

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

// The ring of one wave for XQ (0: one token, else up to 4 XQ), XP terms of x.
template <int RG, int XQ, int XP, int ELEM, int BLOCK>
struct MoeRing {
    static constexpr int WP = WoRow<ELEM, 1>::WP, SCB = 128 / BLOCK;
    using S = WoSlot<RG, XQ, WP, 1, SCB>;
    static constexpr int XBytes = 256 * S::XRows;
    static constexpr int Bytes = S::X + XP * XBytes;
    static constexpr int Loads = RG * S::WD + S::NSC + XP * (XQ == 0 ? 1 : XQ);
};

// Slots of a wave and waves that stream, within `budget` bytes of LDS for NW
// waves: up to four slots each, and where two do not fit, fewer waves.
template <typename R, int NW>
struct MoeShape {
    static constexpr int fit(int budget) { return budget / (NW * R::Bytes); }
    static constexpr int slots(int budget)
    {
        int d = fit(budget) > 4 ? 4 : fit(budget) < 2 ? 2 : fit(budget);
        while ((d - 1) * R::Loads >= 64) --d;
        return d;
    }
    static constexpr int waves(int budget) { return fit(budget) >= 2 ? NW : budget / (2 * R::Bytes); }
};

// fold(a, acc): the sums of active expert a over this wave's chunks of it;
// acc[g][r] is row 4 (lane / 16) + r of the expert's tokens, column lane % 16 of group g.
template <int NW, int BUDGET, int RG, int XQ, int XP, int ELEM, int BLOCK, bool SPLIT, bool POW2, typename F>
__device__ __forceinline__ void moe_stream(uint8_t* lds, const MoeSide& s, const MoeTable& t, const uint16_t* xrow_of_pair,
                                           const float* sdec, int a0, int experts, int wave, int lane, F fold)
{
    constexpr bool WIDE = ELEM >= 2;
    using R = MoeRing<RG, XQ, XP, ELEM, BLOCK>;
    using S = typename R::S;
    using Shape = MoeShape<R, NW>;
    constexpr int D = Shape::slots(BUDGET), NA = Shape::waves(BUDGET);
    constexpr int WP = R::WP, WB = WoRow<ELEM, 1>::WB, SCB = R::SCB, SDW = SCB / 4;
    static_assert(D >= 2 && NA >= 1 && (D - 1) * R::Loads < 64, "ring");
    static_assert(NA * D * R::Bytes <= BUDGET, "LDS");
    const int r16 = lane & 15, grp = lane >> 4;
    const int nch = s.k / 128;
    // this wave's part of the (expert, chunk) list
    const int items = experts * nch;
    if (wave >= NA) return;
    const int first = (int)((int64_t)items * wave / NA), mine = (int)((int64_t)items * (wave + 1) / NA) - first;
    if (mine <= 0) return;
    uint8_t* const ring = lds + wave * (D * R::Bytes);
    const uint32_t rowb = (uint32_t)((int64_t)s.k * (ELEM <= 1 ? 4 : ELEM <= 3 ? 8 : 6) / 8);
    const uint32_t srow = (uint32_t)(s.k / BLOCK);

    // byte offsets of this lane's loads in an expert's codes and scales
    uint32_t wsrc[RG][S::WD];
    bool wact[S::WD];
#pragma unroll
    for (int k = 0; k < S::WD; ++k) {
        const int r = WP == 128 ? 8 * k + (lane >> 3) : lane >> 2;
        const int pc = WP == 128 ? (lane & 7) ^ wo_swz8(r) : (lane & 3) ^ wo_swz(r);
        wact[k] = 16 * pc < WB;
#pragma unroll
        for (int g = 0; g < RG; ++g) wsrc[g][k] = ((g ? s.row1 : s.row0) + (uint32_t)r) * rowb + 16u * (uint32_t)pc;
    }
    uint32_t ssrc[S::NSC];
    bool sact[S::NSC];
#pragma unroll
    for (int j = 0; j < S::NSC; ++j) {
        const int f = 64 * j + lane, rr = f / SDW;
        sact[j] = rr < 16 * RG;
        const int r = sact[j] ? rr : 16 * RG - 1;
        ssrc[j] = ((r < 16 ? s.row0 : s.row1) + (uint32_t)(r & 15)) * srow + 4u * (uint32_t)(f % SDW);
    }
    constexpr int XL = XQ == 0 ? 1 : XQ;
    const uint16_t* xsrc[XL];
    const uint8_t* qe = nullptr;
    const uint8_t* se = nullptr;
    // the next chunk to load
    int ia = first / nch, ik = first - ia * nch;
    auto enter = [&](int a) {
        const int e = __builtin_amdgcn_readfirstlane(t.expert[a0 + a]);
        qe = s.q + (int64_t)e * s.expert_q;
        se = s.s + (int64_t)e * s.expert_s;
        const int b = __builtin_amdgcn_readfirstlane((int)t.start[a0 + a]);
        const int n = __builtin_amdgcn_readfirstlane((int)t.start[a0 + a + 1]) - b;
#pragma unroll
        for (int q = 0; q < XL; ++q) {
            if (XQ == 0) {
                xsrc[0] = s.x + (int64_t)xrow_of_pair[b] * s.ldx + 2 * lane;
            } else {
                const int m = 4 * q + grp;
                xsrc[q] = s.x + (int64_t)xrow_of_pair[b + (m < n ? m : n - 1)] * s.ldx + 8 * (r16 ^ (m & 7));
            }
        }
    };
    enter(ia);
    auto issue = [&](int d) {
        uint8_t* const sl = ring + d * R::Bytes;
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int k = 0; k < S::WD; ++k)
                if (ELEM < 4 || wact[k]) dma16(qe + wsrc[g][k] + (uint32_t)ik * (uint32_t)WB, sl + S::W + 16 * WP * g + 1024 * k);
#pragma unroll
        for (int j = 0; j < S::NSC; ++j)
            if (sact[j]) dma4(se + ssrc[j] + (uint32_t)ik * (uint32_t)SCB, sl + S::SC + 256 * j);
#pragma unroll
        for (int h = 0; h < XP; ++h) {
            const int64_t off = h * s.plane + (int64_t)ik * 128;
            if (XQ == 0) {
                dma4(xsrc[0] + off, sl + S::X + h * R::XBytes);
            } else {
#pragma unroll
                for (int q = 0; q < XL; ++q) dma16(xsrc[q] + off, sl + S::X + h * R::XBytes + 1024 * q);
            }
        }
        if (++ik == nch) ik = 0, ++ia;
    };
    v4f acc[RG];
    auto clear = [&] {
#pragma unroll
        for (int g = 0; g < RG; ++g) acc[g] = v4f{0.f, 0.f, 0.f, 0.f};
    };
    clear();
    const int mr = r16 < S::XRows ? r16 : S::XRows - 1;
    auto xoff = [&](int h, int tt) {
        return S::X + h * R::XBytes + (XQ == 0 ? 16 * (4 * grp + tt)
                                               : 1024 * (mr >> 2) + 256 * (mr & 3) + 16 * ((4 * grp + tt) ^ (mr & 7)));
    };
    auto woff = [&](int j) {
        if (WP == 64) return S::W + 64 * r16 + 16 * (grp ^ wo_swz(r16));
        const int byte = ELEM >= 4 ? 24 * grp + 8 * j : ELEM >= 2 ? 32 * grp + 16 * j : 16 * grp;
        return S::W + WP * r16 + 16 * ((byte >> 4) ^ wo_swz8(r16)) + (byte & 15);
    };
    const int soff = S::SC + SCB * r16 + (BLOCK == 16 ? 2 * grp : grp);
    auto consume = [&](int d) {
        const uint8_t* const sl = ring + d * R::Bytes;
        v4i xf[XP][4];
#pragma unroll
        for (int h = 0; h < XP; ++h)
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) xf[h][tt] = *reinterpret_cast<const v4i*>(sl + xoff(h, tt));
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            v4i wv;
            uint32_t dw[8];
            if constexpr (!WIDE) {
                wv = *reinterpret_cast<const v4i*>(sl + woff(0) + 16 * WP * g);
            } else if constexpr (ELEM <= 3) {
                const v4i w0 = *reinterpret_cast<const v4i*>(sl + woff(0) + 16 * WP * g);
                const v4i w1 = *reinterpret_cast<const v4i*>(sl + woff(1) + 16 * WP * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) { dw[i] = (uint32_t)w0[i]; dw[4 + i] = (uint32_t)w1[i]; }
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const uint64_t v = *reinterpret_cast<const uint64_t*>(sl + woff(j) + 16 * WP * g);
                    dw[2 * j] = (uint32_t)v;
                    dw[2 * j + 1] = (uint32_t)(v >> 32);
                }
                dw[6] = dw[7] = 0u;
            }
            const uint32_t sc = BLOCK == 16 ? (uint32_t)*reinterpret_cast<const uint16_t*>(sl + soff + 16 * SCB * g)
                                            : (uint32_t)sl[soff + 16 * SCB * g];
            const float s0 = sdec[sc & 0xFFu], s1 = BLOCK == 16 ? sdec[(sc >> 8) & 0xFFu] : s0;
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                const float st = tt < 2 ? s0 : s1;                  // elements 0..15: the first block
                v4i hi, lo;
                if constexpr (WIDE) dq8_any<ELEM, SPLIT>(dw, tt, st, hi, lo);
                else if constexpr (SPLIT) dq8_bf16_split<ELEM == 1>((uint32_t)wv[tt], st, hi, lo);
                else hi = dq8_bf16<POW2, ELEM == 1>((uint32_t)wv[tt], st);
#pragma unroll
                for (int h = 0; h < XP; ++h) {
                    acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xf[h][tt]),
                                                                     __builtin_bit_cast(v8bf, hi), acc[g], 0, 0, 0);
                    if (SPLIT)
                        acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xf[h][tt]),
                                                                         __builtin_bit_cast(v8bf, lo), acc[g], 0, 0, 0);
                }
            }
        }
        // the slot's reads have returned before a load may overwrite it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };

    int issued = 0, at = 0;               // at: the slot of chunk i; chunk i + D takes it next
    auto advance = [&] {
        const int was = ia;
        issue(issued % D);
        ++issued;
        if (ia != was && issued < mine) enter(ia);
    };
    while (issued < D && issued < mine) advance();
    int ca = first / nch, ck = first - ca * nch;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        // loads of later chunks that are still under way
        const int behind = mine - 1 - i < D - 1 ? mine - 1 - i : D - 1;
        if (behind >= 3) wait_vmcnt<(D > 3 ? 3 * R::Loads : 0)>();
        else if (behind == 2) wait_vmcnt<(D > 2 ? 2 * R::Loads : 0)>();
        else if (behind == 1) wait_vmcnt<R::Loads>();
        else wait_vmcnt<0>();
        consume(at);
        at = at + 1 == D ? 0 : at + 1;
        if (issued < mine) advance();
        if (++ck == nch || i + 1 == mine) {
            fold(ca, acc);
            clear();
            ck = 0;
            ++ca;
        }
    }
    wait_vmcnt<0>();
}

__device__ __forceinline__ ScaleFmt device_fmt(const ScaleFmtHost& f)
{
    return ScaleFmt{f.ebits, f.mbits, f.bias, f.maxcode, f.smax, f.is_e8m0};
}

// f(std::integral_constant<int, XQ>) for an expert's number of tokens, at most
// the launch's
template <int MAXQ, typename F>
__device__ __forceinline__ void moe_class(int tokens, F f)
{
    if (MAXQ == 0 || tokens <= 1) f(std::integral_constant<int, 0>{});
    else if (MAXQ == 1 || tokens <= 4) f(std::integral_constant<int, MAXQ >= 1 ? 1 : 0>{});
    else if (MAXQ == 2 || tokens <= 8) f(std::integral_constant<int, MAXQ >= 2 ? 2 : 0>{});
    else f(std::integral_constant<int, MAXQ >= 4 ? 4 : 0>{});
}

constexpr int kMoeUpWaves = 4, kMoeUpBudget = 60 * 1024;
constexpr int kMoeDownWaves = 8, kMoeDownBudget = 144 * 1024;

template <int ELEM, int BLOCK, bool SPLIT, bool POW2, int MAXQ>
__global__ __launch_bounds__(64 * kMoeUpWaves) void k_moe_up(MoeLaunch p)
{
    constexpr int NW = kMoeUpWaves;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ MoeTable t;
    __shared__ float sdec[256];
    __shared__ uint16_t xrow[kMoePairs];
    __shared__ float part[NW][2][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float g = p.up.g[0], pw = split_pow2(g), gres = g / pw;
    const ScaleFmt fw = device_fmt(p.up.fmt);
    moe_table(p, t, *reinterpret_cast<MoeScratch*>(lds), tid);
    const int a = blockIdx.y;
    if (a >= t.active) return;            // the whole workgroup
    for (int c = tid; c < 256; c += 64 * NW) sdec[c] = scale_decode_any((uint32_t)c, fw) * pw;
    if (tid < kMoePairs) xrow[tid] = t.tok[tid];
    const int e = t.expert[a], b = t.start[a], cnt = t.start[a + 1] - b;
    __syncthreads();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    MoeSide s;
    s.q = p.up.q; s.s = p.up.s;
    s.expert_q = p.up.expert_q; s.expert_s = p.up.expert_s;
    s.row0 = (uint32_t)n0; s.row1 = (uint32_t)(p.ffn + n0);
    s.k = (int32_t)p.hidden;
    s.x = p.x; s.ldx = p.ldx; s.plane = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave][i >> 2][4 * lane + (i & 3)] = 0.0f;
    moe_class<MAXQ>(cnt, [&](auto q) {
        moe_stream<NW, kMoeUpBudget, 2, decltype(q)::value, 1, ELEM, BLOCK, SPLIT, POW2>(
            lds, s, t, xrow, sdec, a, 1, wave, lane, [&](int, const v4f (&acc)[2]) {
#pragma unroll
                for (int r = 0; r < 4; ++r) { part[wave][0][4 * lane + r] = acc[0][r]; part[wave][1][4 * lane + r] = acc[1][r]; }
            });
    });
    __syncthreads();
    const float f = gres * (p.up.scale ? p.up.scale[e] : 1.0f);
    const int j = tid >> 4, n = tid & 15;
    if (j >= cnt) return;
    const int at = 4 * (16 * (j >> 2) + n) + (j & 3);
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) { gate += part[w][0][at]; up += part[w][1][at]; }
    float h = gate * f;
    with_act(p.act, [&](auto act) { h = act_value<decltype(act)::value>(h); });
    h *= up * f;
    // h as the sum of two bf16: its first eight bits, and what they leave, rounded
    const uint32_t hi = f_bits(h) & 0xFFFF0000u;
    const float left = h - bits_f(hi);
    const int64_t to = (int64_t)t.row[b + j] * p.ffn + n0 + n;
    p.h[to] = (uint16_t)(hi >> 16) | (h != h ? 0x40u : 0u);
    p.h[to + (int64_t)p.m * p.top * p.ffn] = left == left ? (uint16_t)f32_to_bf16_rne(left) : (uint16_t)0;
}

template <int ELEM, int BLOCK, bool SPLIT, bool POW2, int MAXQ>
__global__ __launch_bounds__(64 * kMoeDownWaves) void k_moe_down(MoeLaunch p)
{
    constexpr int NW = kMoeDownWaves;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ MoeTable t;
    __shared__ float sdec[256];
    __shared__ float tot[NW][16][16];     // a wave's sums: token, column
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const float g = p.down.g[0], pw = split_pow2(g), gres = g / pw;
    const ScaleFmt fw = device_fmt(p.down.fmt);
    moe_table(p, t, *reinterpret_cast<MoeScratch*>(lds), tid);
    for (int c = tid; c < 256; c += 64 * NW) sdec[c] = scale_decode_any((uint32_t)c, fw) * pw;
#pragma unroll
    for (int i = 0; i < 4; ++i) (&tot[wave][0][0])[64 * i + lane] = 0.0f;
    int most = 0;
    for (int a = 0; a < t.active; ++a) {
        const int n = t.start[a + 1] - t.start[a];
        most = n > most ? n : most;
    }
    most = __builtin_amdgcn_readfirstlane(most);
    __syncthreads();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    MoeSide s;
    s.q = p.down.q; s.s = p.down.s;
    s.expert_q = p.down.expert_q; s.expert_s = p.down.expert_s;
    s.row0 = s.row1 = (uint32_t)n0;
    s.k = (int32_t)p.ffn;
    s.x = p.h; s.ldx = p.ffn; s.plane = (int64_t)p.m * p.top * p.ffn;
    moe_class<MAXQ>(most, [&](auto q) {
        moe_stream<NW, kMoeDownBudget, 1, decltype(q)::value, 2, ELEM, BLOCK, SPLIT, POW2>(
            lds, s, t, t.row, sdec, 0, t.active, wave, lane, [&](int a, const v4f (&acc)[1]) {
                const int b = t.start[a], n = t.start[a + 1] - b;
                const float f = gres * (p.down.scale ? p.down.scale[t.expert[a]] : 1.0f);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 4 * (lane >> 4) + r;
                    if (j < n) {
                        float& to = tot[wave][t.tok[b + j]][lane & 15];
                        to = __builtin_fmaf(t.w[b + j] * f, acc[0][r], to);
                    }
                }
            });
    });
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
template <int NW, int BUDGET, int RG, int XP, int ELEM, int BLOCK, int XQ>
constexpr size_t ring_bytes()
{
    using R = MoeRing<RG, XQ, XP, ELEM, BLOCK>;
    using Shape = MoeShape<R, NW>;
    return (size_t)Shape::waves(BUDGET) * Shape::slots(BUDGET) * R::Bytes;
}
// the largest ring that an expert of the launch may take, and the sort before it
template <int NW, int BUDGET, int RG, int XP, int ELEM, int BLOCK, int MAXQ>
constexpr size_t lds_bytes()
{
    size_t b = sizeof(MoeScratch);
    const size_t r0 = ring_bytes<NW, BUDGET, RG, XP, ELEM, BLOCK, 0>(), r1 = ring_bytes<NW, BUDGET, RG, XP, ELEM, BLOCK, 1>();
    const size_t r2 = ring_bytes<NW, BUDGET, RG, XP, ELEM, BLOCK, 2>(), r4 = ring_bytes<NW, BUDGET, RG, XP, ELEM, BLOCK, 4>();
    b = r0 > b ? r0 : b;
    if (MAXQ >= 1) b = r1 > b ? r1 : b;
    if (MAXQ >= 2) b = r2 > b ? r2 : b;
    if (MAXQ >= 4) b = r4 > b ? r4 : b;
    return b;
}

template <int ELEM, int BLOCK, bool SPLIT, bool POW2, int MAXQ>
static hipError_t run_moe(const MoeLaunch& p, bool up, hipStream_t s)
{
    if (up) {
        constexpr size_t sh = lds_bytes<kMoeUpWaves, kMoeUpBudget, 2, 1, ELEM, BLOCK, MAXQ>();
        static_assert(sh <= 64 * 1024, "LDS");
        const int most = p.m * p.top < p.experts ? p.m * p.top : p.experts;
        hipLaunchKernelGGL((k_moe_up<ELEM, BLOCK, SPLIT, POW2, MAXQ>), dim3((unsigned)(p.ffn / 16), (unsigned)most),
                           dim3(64 * kMoeUpWaves), sh, s, p);
    } else {
        constexpr size_t sh = lds_bytes<kMoeDownWaves, kMoeDownBudget, 1, 2, ELEM, BLOCK, MAXQ>();
        static_assert(sh + sizeof(MoeTable) + 4 * (256 + 256 * kMoeDownWaves) <= 160 * 1024, "LDS");
        const hipError_t e = allow_lds(k_moe_down<ELEM, BLOCK, SPLIT, POW2, MAXQ>, sh);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((k_moe_down<ELEM, BLOCK, SPLIT, POW2, MAXQ>), dim3((unsigned)(p.hidden / 16)),
                           dim3(64 * kMoeDownWaves), sh, s, p);
    }
    return hipGetLastError();
}

template <int ELEM, int BLOCK, bool SPLIT, bool POW2>
static hipError_t run_moe_tokens(const MoeLaunch& p, bool up, hipStream_t s)
{
    if (p.m == 1) return run_moe<ELEM, BLOCK, SPLIT, POW2, 0>(p, up, s);
    if (p.m <= 4) return run_moe<ELEM, BLOCK, SPLIT, POW2, 1>(p, up, s);
    if (p.m <= 8) return run_moe<ELEM, BLOCK, SPLIT, POW2, 2>(p, up, s);
    return run_moe<ELEM, BLOCK, SPLIT, POW2, 4>(p, up, s);
}

template <int ELEM, int BLOCK>
static hipError_t run_moe_scales(const MoeLaunch& p, bool up, hipStream_t s)
{
    const MoeWeights& w = up ? p.up : p.down;
    if (!wo_exact_in_bf16(ELEM, w.fmt)) return run_moe_tokens<ELEM, BLOCK, true, false>(p, up, s);
    if constexpr (ELEM == 0)
        if (w.fmt.is_e8m0) return run_moe_tokens<ELEM, BLOCK, false, true>(p, up, s);
    return run_moe_tokens<ELEM, BLOCK, false, false>(p, up, s);
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
// The router's choice: a wave for each row, its experts' scores spread over
// the lanes (at most 16 each), `top` rounds of the wave's largest.  Scores
// are compared and divided in binary64: the order of two near scores plus
// their biases is the binary64 formula's, where binary32's exponential would
// turn neighbours round.
// ---------------------------------------------------------------------------
constexpr int kRouteLane = kMoeMaxRouted / 64;
constexpr int kRouteWaves = 4;

__device__ __forceinline__ uint64_t order_key(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    if ((u & 0x7FFFFFFFFFFFFFFFull) > 0x7FF0000000000000ull) return ~0ull;     // NaN above everything
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

__global__ __launch_bounds__(64 * kRouteWaves) void k_moe_route(RouteLaunch p)
{
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
    if (row >= p.rows) return;
    const int E = p.experts;
    double score[kRouteLane];
    uint64_t key[kRouteLane];             // 0: no candidate
    double top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kRouteLane; ++i) {
        const int e = 64 * i + lane;
        score[i] = -INFINITY;
        if (64 * i < E && e < E) {
            const float z = p.bf16 ? bf16_lo(((const uint16_t*)p.logits)[row * p.ld + e]) : ((const float*)p.logits)[row * p.ld + e];
            score[i] = z;
            top = fmax(top, (double)z);
        }
    }
    if (!p.sigmoid) {
#pragma unroll
        for (int o = 32; o; o >>= 1) top = fmax(top, __shfl_xor(top, o));
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kRouteLane; ++i) {
        key[i] = 0;
        if (64 * i >= E) continue;
        const int e = 64 * i + lane;
        const double z = score[i];
        const bool in = e < E && z != -INFINITY;             // a masked expert is never chosen
        // the largest logit's own score is 1 (also where it is infinite)
        score[i] = !in ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-z)) : z == top ? 1.0 : exp(z - top);
        sum += score[i];
    }
    if (!p.sigmoid) {
#pragma unroll
        for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    }
#pragma unroll
    for (int i = 0; i < kRouteLane; ++i) {
        if (64 * i >= E) continue;
        const int e = 64 * i + lane;
        if (e >= E) continue;
        const float z = p.bf16 ? bf16_lo(((const uint16_t*)p.logits)[row * p.ld + e]) : ((const float*)p.logits)[row * p.ld + e];
        if (!p.sigmoid) score[i] /= sum;
        if (z == -INFINITY) continue;
        // without a bias the scores' order is the logits', ties and underflow aside
        key[i] = order_key(p.bias ? score[i] + (double)p.bias[e] : (double)z);
    }
    // `top` rounds: the wave's largest key, of equal ones the lower expert
    double mine = 0.0, total = 0.0;
    int id = -1;
    for (int k = 0; k < p.top; ++k) {
        uint64_t best = 0;
        int at = 0;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < kRouteLane; ++i)
            if (key[i] > best) { best = key[i]; at = i; s = score[i]; }
        int e = best ? 64 * at + lane : kNoExpert;
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const uint64_t b = ((uint64_t)(uint32_t)__shfl_xor((int)(best >> 32), o) << 32) | (uint32_t)__shfl_xor((int)best, o);
            const int oe = __shfl_xor(e, o);
            const double os = __shfl_xor(s, o);
            if (b > best || (b == best && oe < e)) { best = b; e = oe; s = os; }
        }
        if (best == 0) break;                                  // nothing left to choose
        total += s;
        if (lane == k) { id = e; mine = s; }
#pragma unroll
        for (int i = 0; i < kRouteLane; ++i)
            if (64 * i + lane == e) key[i] = 0;
    }
    if (lane >= p.top) return;
    double w = mine;
    if (p.renormalize) w = total == 0.0 ? 0.0 : mine / total;
    p.ids[row * p.top + lane] = id;
    p.weights[row * p.top + lane] = id < 0 ? 0.0f : (float)(w * (double)p.scale);
}

hipError_t launch_moe_route(const RouteLaunch& p, hipStream_t s)
{
    hipLaunchKernelGGL(k_moe_route, dim3((unsigned)((p.rows + kRouteWaves - 1) / kRouteWaves)), dim3(64 * kRouteWaves), 0, s, p);
    return hipGetLastError();
}

}  // namespace fp4
