// distill.hip -- the loss of a student's logits against a teacher's top log
// probabilities, and the logits' gradient (quant_prune_distill/574 and
// ue5m3-fp4-pretraining: a model whose linear layers run in FP4, here trained
// towards a full-precision one).
//
// With c = 1 / temperature, q = softmax(c z) and the listed tokens v_j with
// p_j = exp(t_j), P = sum p_j, R = the student's probability of all others:
//   bucket       L = sum p_j (t_j - log q_vj) + (1 - P) (log(1 - P) - log R)
//                dL/dz = c (q_v - p_v) listed, c q_v (1 - (1 - P) / R) others
//   renormalize  p_j / P in the place of p_j:  L = sum p_j (log p_j - log q_vj)
//                dL/dz = c (q_v - p_v)
// L is a small difference of large terms.  R is summed without the listed
// tokens, about a maximum of its own -- a bitmap of the row's piece in LDS
// names them, a byte for every eight logits (1 - sum of theirs would keep
// nothing of a confident row's R) --, and what follows from the sums, a few
// numbers a row, is computed in binary64.  The sums use k = c log2 e rounded to binary32 and the listed
// terms the same k, so its rounding is a temperature 2^-24 off in both and
// cancels.
//
// Both passes are bound by memory: 8192 x 32000 bf16, 32 listed, 118 us for the
// sums (4.4 TB/s) and 200 for the gradient (5.2, read and written); 61 x 50257
// binary32, 8 listed, 12 and 8.
#include <type_traits>

#include "fp4_device.hpp"
#include "fp4_internal.h"
#include "logits_device.hpp"

namespace fp4 {

constexpr double kLn2d = 0.693147180559945309417;
constexpr int kDsThreads = 256;

// Tokens of the list inside the vocabulary; a token listed again keeps both
// probabilities and counts once among the student's.
__device__ __forceinline__ bool is_token(int32_t id, int64_t vocab) { return id >= 0 && id < vocab; }

template <typename T>
__device__ __forceinline__ T wave_sum(T v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// A row's list over the 64 lanes of a wave, two entries each, with the
// student's logits: fetched ahead of the sums.
constexpr int kDsLane = kDistillMaxTop / 64;
struct List { int32_t id[kDsLane]; float t[kDsLane], z[kDsLane]; };

template <bool BF16>
__device__ __forceinline__ List fetch_list(const DistillLaunch& p, int64_t row, int lane)
{
    using T = typename Logit<BF16>::Raw;
    List l;
#pragma unroll
    for (int i = 0; i < kDsLane; ++i) {
        const int j = 64 * i + lane;
        l.id[i] = j < p.top ? p.ids[row * p.top + j] : -1;
        if (!is_token(l.id[i], p.vocab)) l.id[i] = -1;
        l.t[i] = l.id[i] >= 0 ? p.logprobs[row * p.top + j] : -INFINITY;
        l.z[i] = l.id[i] >= 0 ? Logit<BF16>::one((const T*)p.logits + row * p.ld + l.id[i]) : -INFINITY;
    }
    return l;
}

// The loss and the row's statistics from its sums: mr the largest logit that
// is not listed, rest the sum of 2^((z - mr) k) over those.  By the 64 lanes of
// one wave.
__device__ __forceinline__ void finish_distill(const DistillLaunch& p, int64_t row, float mr, float rest, const List& l, int lane)
{
    const double k = (double)(p.inv_temperature * kLog2e);
    float m = mr;
#pragma unroll
    for (int i = 0; i < kDsLane; ++i) m = fmaxf(m, l.z[i]);
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    double mass = 0.0, plain = 0.0, cross = 0.0, own = 0.0;
#pragma unroll
    for (int i = 0; i < kDsLane; ++i) {
        if (64 * i >= p.top) continue;
        bool again = false;
#pragma unroll
        for (int o = 0; o <= i; ++o) {
            const int n = p.top - 64 * o < 64 ? p.top - 64 * o : 64;
            for (int j = 0; j < n; ++j)
                again |= __builtin_amdgcn_readlane(l.id[o], j) == l.id[i] && (o < i || j < lane);
        }
        if (l.id[i] < 0) continue;
        const double t = l.t[i], pj = exp(t);
        const double d = l.z[i] == -INFINITY ? -INFINITY : ((double)l.z[i] - (double)m) * k;   // log2 of its term
        mass += pj;
        if (!(pj == 0.0)) {                                // 0 log 0 = 0
            plain += pj * t;
            cross += pj * d;
        }
        if (!again) own += exp2(d);
    }
    mass = wave_sum(mass);
    plain = wave_sum(plain);
    cross = wave_sum(cross);
    own = wave_sum(own);
    if (lane) return;
    // a student's row of masks; own is NaN where a listed logit is, which no maximum shows
    const bool empty = m == -INFINITY && rest == 0.0f && own == 0.0;
    // the others' sum against the whole row's maximum, and its share R of the total
    const double below = mr == -INFINITY ? 0.0 : ((double)mr - (double)m) * k;
    const double total = own + (double)rest * exp2(below), logs = log(total);
    const bool others = !(rest == 0.0f);
    const double share = others ? (double)rest * exp2(below) / total : 0.0;
    double loss = 0.0, cl = 0.0, cu = 0.0, logmass = 0.0;
    if (!(mass == 0.0)) {
        if (p.renormalize) {
            logmass = log(mass);
            // sum p (t - log P - log q) over P
            loss = (plain - cross * kLn2d) / mass - logmass + logs;
            cl = 1.0;
            cu = share;
        } else {
            const double left = mass > 1.0 ? 0.0 : 1.0 - mass;
            loss = plain - cross * kLn2d + mass * logs;
            cl = mass;
            cu = mass * share;
            // a student that has nothing outside the list has no such term
            if (others && !(left == 0.0)) {
                loss += left * (log(left) - (log((double)rest) + below * kLn2d - logs));
                cl = 1.0;
                cu = share - left;
            }
        }
        if (empty) {                                       // no probability anywhere: no gradient
            loss = INFINITY;
            cl = cu = 0.0;
        }
    }
    p.loss[row] = (float)loss;
    float* const st = p.stats + row * kDistillStats;
    st[0] = empty ? 0.0f : m;
    st[1] = empty ? 0.0f : (float)(1.0 / total);
    st[2] = others ? mr : 0.0f;
    st[3] = others ? 1.0f / rest : 0.0f;
    st[4] = (float)cl;
    st[5] = (float)cu;
    st[6] = (float)logmass;
}

// Bit i of a piece's bitmap: element vb + i is listed.
__device__ __forceinline__ void mark_listed(uint32_t* bits, int words, const int32_t* ids, int top, int64_t from, int64_t to, int tid,
                                            int threads)
{
    for (int i = tid; i < words; i += threads) bits[i] = 0u;
    __syncthreads();
    for (int j = tid; j < top; j += threads) {
        const int64_t id = ids[j];
        if (id >= from && id < to) atomicOr(&bits[(id - from) >> 5], 1u << ((id - from) & 31));
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// One workgroup per row (gridDim.y = 1), or per piece of a row, whose sums
// k_distill_join joins.  Rows may start at any element.
// ---------------------------------------------------------------------------
template <bool BF16, int THREADS>
__global__ __launch_bounds__(THREADS) void k_distill_rows(DistillLaunch p)
{
    using L = Logit<BF16>;
    using T = typename L::Raw;
    constexpr int NW = THREADS / 64, VN = L::N;
    constexpr int64_t kRound = (int64_t)THREADS * kLpVec;
    extern __shared__ uint32_t bits[];
    __shared__ float sm[NW][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    const T* const z = (const T*)p.logits + row * p.ld;
    const int32_t* const ids = p.ids + row * p.top;
    const int64_t b = (int64_t)blockIdx.y * p.piece, e = b + p.piece < p.vocab ? b + p.piece : p.vocab;
    const float k = p.inv_temperature * kLog2e;
    const int64_t head = (int64_t)((16 - ((uintptr_t)(z + b) & 15)) & 15) / (int64_t)sizeof(T);
    const int64_t vb = b + head < e ? b + head : e;
    const int64_t nvec = (e - vb) / VN;
    const int64_t ve = vb + nvec * VN;
    const v4i* const zv = reinterpret_cast<const v4i*>(z + vb);
    v4i next[kLpVec];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + (int64_t)u * THREADS + tid;
            if (i < nvec) next[u] = zv[i];
        }
    };
    fetch(0);
    List list{};
    if (wave == 0 && gridDim.y == 1) list = fetch_list<BF16>(p, row, lane);
    mark_listed(bits, (int)((e - vb + 31) / 32), ids, p.top, vb, e, tid, THREADS);
    const uint8_t* const marks = reinterpret_cast<const uint8_t*>(bits);
    Running a{-INFINITY, 0.0f, 0.0f, 0.0f};
    auto round = [&](int64_t r0, auto whole) {             // whole: every thread has all of its vectors
        float f[kLpVec * VN], best = -INFINITY;
        uint32_t out[kLpVec];
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + (int64_t)u * THREADS + tid;
            const bool in = whole || i < nvec;
            float v[VN];
            L::unpack(next[u], v);
            out[u] = !in ? 0u : VN == 8 ? marks[i] : (uint32_t)marks[i >> 1] >> (4 * (int)(i & 1)) & 15u;
#pragma unroll
            for (int j = 0; j < VN; ++j) f[u * VN + j] = in ? v[j] : -INFINITY;
        }
        fetch(r0 + kRound);
        uint32_t some = 0;
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) some |= out[u];
        if (__builtin_amdgcn_ballot_w64(some != 0)) {
#pragma unroll
            for (int j = 0; j < kLpVec * VN; ++j)
                if (out[j / VN] >> (j % VN) & 1u) f[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kLpVec * VN; ++j) best = fmaxf(best, f[j]);
        a.raise(best, k);
        // a round's terms add up on their own before they join the row's
        const float s = a.s;
        a.s = 0.0f;
        if (__builtin_amdgcn_ballot_w64(a.far(k))) {
#pragma unroll
            for (int j = 0; j < kLpVec * VN; ++j) {
                if (a.far(k)) a.template add<true>(f[j], k);
                else a.template add<false>(f[j], k);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kLpVec * VN; ++j) a.template add<false>(f[j], k);
        }
        a.s += s;
    };
    int64_t r0 = 0;
    for (; r0 + kRound <= nvec; r0 += kRound) round(r0, std::true_type{});
    if (r0 < nvec) round(r0, std::false_type{});
    // at most VN - 1 elements on either side
    if (wave == 0) {
        const int64_t nh = vb - b, nt = e - ve;
        const int64_t i = tid < nh ? b + tid : ve + (tid - nh);
        if (tid < nh + nt) {
            const float v = L::one(z + i);
            bool listed = false;
            if (i >= vb) listed = bits[(i - vb) >> 5] >> ((i - vb) & 31) & 1u;
            else for (int j = 0; j < p.top; ++j) listed |= ids[j] == i;
            if (!listed) {
                a.raise(v, k);
                if (a.far(k)) a.template add<true>(v, k);
                else a.template add<false>(v, k);
            }
        }
    }
    Sums r = a.about_max(k);
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float m = __shfl_xor(r.m, o), s = __shfl_xor(r.s, o);
        sums_merge(r, m, s, 0.0f, k);
    }
    if (NW > 1) {
        if (lane == 0) { sm[wave][0] = r.m; sm[wave][1] = r.s; }
        __syncthreads();
        r = Sums{-INFINITY, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; ++w) sums_merge(r, sm[w][0], sm[w][1], 0.0f, k);
    }
    if (wave != 0) return;
    if (gridDim.y == 1) {
        finish_distill(p, row, r.m, r.s, list, lane);
    } else if (lane == 0) {
        float* const o = p.part + 2 * (row * gridDim.y + blockIdx.y);
        o[0] = r.m; o[1] = r.s;
    }
}

template <bool BF16>
__global__ __launch_bounds__(64) void k_distill_join(DistillLaunch p, int pieces)
{
    const int lane = threadIdx.x;
    const int64_t row = blockIdx.x;
    const float k = p.inv_temperature * kLog2e;
    const List list = fetch_list<BF16>(p, row, lane);
    Sums r{-INFINITY, 0.0f, 0.0f};
    if (lane < pieces) {
        const float* const o = p.part + 2 * (row * pieces + lane);
        r = Sums{o[0], o[1], 0.0f};
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float m = __shfl_xor(r.m, o), s = __shfl_xor(r.s, o);
        sums_merge(r, m, s, 0.0f, k);
    }
    finish_distill(p, row, r.m, r.s, list, lane);
}

// ---------------------------------------------------------------------------
// dz: one workgroup per row and piece.  A row whose gradient is zero, or
// whose list holds nothing, is written as zeros without reading its logits.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(kDsThreads) void k_distill_backward(DistillGradLaunch p)
{
    using L = Logit<BF16>;
    using T = typename L::Raw;
    constexpr int VN = L::N;
    __shared__ int32_t ids[kDistillMaxTop];
    __shared__ float prob[kDistillMaxTop], share[kDistillMaxTop];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const T* const z = (const T*)p.logits + row * p.ld;
    T* const dz = (T*)p.dlogits + row * p.ldd;
    const int64_t b = (int64_t)blockIdx.y * p.piece, e = b + p.piece < p.vocab ? b + p.piece : p.vocab;
    const float* const st = p.stats + row * kDistillStats;
    const float c = p.inv_temperature, g = p.g_loss[row], cl = st[4], cu = st[5], logmass = st[6];
    const bool none = g == 0.0f || (cl == 0.0f && cu == 0.0f);
    // a listed token's q against the row's maximum and total, another's share
    // of the others against theirs: R, however small, is in cu.  Powers are
    // taken as squares: the instruction flushes those below 2^-126, which a
    // large coefficient would make visible.
    const float k = 0.5f * c * kLog2e;
    const float ml = st[0], mu = st[2], gl = g * cl * st[1], gu = g * cu * st[3];
    auto other = [&](float x) {
        const float h = __builtin_amdgcn_exp2f((x - mu) * k);
        return c * (h * (h * gu));                        // c last: it must not overflow against q = 0
    };
    // elements that are vectors of both rows
    const int64_t head = (int64_t)((16 - ((uintptr_t)(z + b) & 15)) & 15) / (int64_t)sizeof(T);
    const bool same = (((uintptr_t)(z + b) ^ (uintptr_t)(dz + b)) & 15) == 0;
    const int64_t vb = !same ? e : b + head < e ? b + head : e;
    const int64_t nvec = (e - vb) / VN, ve = vb + nvec * VN;
    const v4i* const zv = reinterpret_cast<const v4i*>(z + vb);
    v4i* const dv = reinterpret_cast<v4i*>(dz + vb);
    v4i raw[kLpVec];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + kDsThreads * u + tid;
            if (i < nvec && !none) raw[u] = zv[i];
        }
    };
    fetch(0);
    // The listed tokens of this piece, whose logits are read before anything
    // is written: every element is first written as one of the others, and
    // theirs once more at the end, a token a thread.  (Looking for them among
    // the elements instead cost a third of the kernel's time: with 32 of 32000
    // listed every other wave's vectors hold one.)
    int32_t mine = -1;
    if (!none && tid < p.top) {
        const int32_t id = p.ids[row * p.top + tid];
        const bool in = id >= b && id < e;
        mine = in ? id : -1;
        ids[tid] = mine;
        if (in) {
            const float h = __builtin_amdgcn_exp2f((L::one(z + id) - ml) * k);
            share[tid] = h * (h * gl);
            prob[tid] = g * (float)exp((double)p.logprobs[row * p.top + tid] - (double)logmass);
        }
    }
    __syncthreads();
    auto put = [&](int64_t i) {
        const float d = none ? 0.0f : other(L::one(z + i));
        if constexpr (BF16) dz[i] = (uint16_t)f32_to_bf16_rne(d);
        else dz[i] = d;
    };
    for (int64_t r0 = 0; r0 < nvec; r0 += kDsThreads * kLpVec) {
        v4i out[kLpVec];
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            if (none) {
                out[u] = v4i{0, 0, 0, 0};
                continue;
            }
            float f[VN];
            L::unpack(raw[u], f);
#pragma unroll
            for (int j = 0; j < VN; ++j) f[j] = other(f[j]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (BF16) out[u][q] = (int)pack_bf16(f[2 * q], f[2 * q + 1]);
                else out[u][q] = (int)f_bits(f[q]);
            }
        }
        fetch(r0 + kDsThreads * kLpVec);
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + kDsThreads * u + tid;
            if (i < nvec) __builtin_nontemporal_store(out[u], dv + i);   // read next long after it has left the caches
        }
    }
    for (int64_t i = b + tid; i < vb; i += kDsThreads) put(i);
    for (int64_t i = ve + tid; i < e; i += kDsThreads) put(i);
    // every thread's stores have arrived before one of them is written again
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (mine < 0) return;
    float pm = 0.0f;                                       // a token may be listed twice
    for (int i = 0; i < p.top; ++i) pm += ids[i] == mine ? prob[i] : 0.0f;
    const float d = c * (share[tid] - pm);
    if constexpr (BF16) dz[mine] = (uint16_t)f32_to_bf16_rne(d);
    else dz[mine] = d;
}

// ---------------------------------------------------------------------------
// launch shapes
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A row is one workgroup's where the rows alone fill the device, and also where
// it is at most 512 KiB, in 16 waves.  For rows by the tens that is about what
// pieces and the launch that joins them take, for a few long ones more (one
// workgroup a row against pieces, us a call in a graph):
//             32000 f32    50257 f32    128256 f32   128256 bf16
//   1 row     9.4   8.6    10.8   8.6   15.2   8.8   13.9   8.8
//   8         9.6   8.9    11.3   9.7   15.5   8.9   14.2   8.9
//   61        10.3  10.6   12.1  12.6   16.2  14.9   15.1  13.3
//   256       12.9  14.6   17.2  19.1   29.8  31.2   18.7  19.7
// Longer rows are cut as the token log probabilities' are, and a piece has at
// most kDsMost elements, whose bitmap must fit the LDS.
int64_t distill_pieces(int64_t rows, int64_t vocab, int64_t esize)
{
    const int64_t n = vocab * esize <= 512 * 1024 ? 1 : logprob_pieces(rows, vocab), least = cdiv(vocab, kDsMost);
    return n > least ? n : least;
}

template <bool BF16>
static hipError_t run_distill(DistillLaunch p, int64_t pieces, hipStream_t s)
{
    p.piece = cdiv(cdiv(p.vocab, pieces), 64) * 64;
    pieces = cdiv(p.vocab, p.piece);
    const dim3 grid((unsigned)p.rows, (unsigned)pieces);
    const size_t sh = (size_t)cdiv(p.piece < p.vocab ? p.piece : p.vocab, 32) * 4;
    // a short row of many is one wave's, as in the token log probabilities
    if (pieces == 1 && p.rows < 512) hipLaunchKernelGGL((k_distill_rows<BF16, 1024>), grid, dim3(1024), sh, s, p);
    else if (pieces == 1 && p.vocab <= 16384) hipLaunchKernelGGL((k_distill_rows<BF16, 64>), grid, dim3(64), sh, s, p);
    else hipLaunchKernelGGL((k_distill_rows<BF16, 256>), grid, dim3(256), sh, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || pieces == 1) return e;
    hipLaunchKernelGGL((k_distill_join<BF16>), dim3((unsigned)p.rows), dim3(64), 0, s, p, (int)pieces);
    return hipGetLastError();
}

hipError_t launch_distill(const DistillLaunch& p, int64_t pieces, hipStream_t s)
{
    return p.bf16 ? run_distill<true>(p, pieces, s) : run_distill<false>(p, pieces, s);
}

hipError_t launch_distill_backward(const DistillGradLaunch& in, hipStream_t s)
{
    DistillGradLaunch p = in;
    // two rounds of a workgroup's threads: 16384 bf16 or 8192 binary32 elements
    p.piece = 2 * kDsThreads * kLpVec * (p.bf16 ? 8 : 4);
    static_assert(kDistillMaxTop <= kDsThreads, "a thread for each listed token");
    const dim3 grid((unsigned)p.rows, (unsigned)cdiv(p.vocab, p.piece));
    if (p.bf16) hipLaunchKernelGGL((k_distill_backward<true>), grid, dim3(kDsThreads), 0, s, p);
    else hipLaunchKernelGGL((k_distill_backward<false>), grid, dim3(kDsThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace fp4
