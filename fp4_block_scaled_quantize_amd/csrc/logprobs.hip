// logprobs.hip -- log probabilities of given tokens, entropy and the top
// alternatives of each row of logits, and the gradient of both sums
// (quant_prune_distill/574: reinforcement learning over FP4 weights, whose
// policy loss reads the chosen tokens' log probabilities and the entropy).
//
// With c = 1 / temperature, m = max_v z_v, d_v = (z_v - m) c:
//   s = sum exp(d_v),  w = sum exp(d_v) d_v
//   logprob(t) = d_t - log s,  entropy = log s - w / s
//   dz_v = c (gl ([v = t] - p_v) - ge p_v (log p_v + entropy))
// One pass over a row keeps the running (m, s, w) of every thread in
// binary32: a larger maximum m' = m + D rescales s by f = exp(-c D) and w to
// f (w - c D s).  The kernels work in powers of two (k = c log2 e), where w
// carries log2 units.
#include "fp4_device.hpp"
#include "fp4_internal.h"

namespace fp4 {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kLpMaxTop = 32;
constexpr int kLpBuf = 256;            // candidate keys of a wave
constexpr int kLpVec = 4;              // 16-byte vectors a thread reads per round

template <bool BF16>
struct Logit;
template <>
struct Logit<true> {
    using Raw = uint16_t;
    static constexpr int N = 8;        // elements of a 16-byte vector
    static __device__ __forceinline__ float one(const uint16_t* p) { return bits_f((uint32_t)*p << 16); }
    static __device__ __forceinline__ void unpack(v4i v, float* o)
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) { o[2 * q] = bf16_lo((uint32_t)v[q]); o[2 * q + 1] = bf16_hi((uint32_t)v[q]); }
    }
};
template <>
struct Logit<false> {
    using Raw = float;
    static constexpr int N = 4;
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ void unpack(v4i v, float* o)
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = bits_f((uint32_t)v[q]);
    }
};

// Running sums in log2 units.  m is a value of the row (or -inf).
struct Sums { float m, s, w; };

// (z - m) k, where a maximum of -inf (nothing finite so far) counts as 0.
__device__ __forceinline__ float shift2(float z, float m, float k)
{
    return (z - (m == -INFINITY ? 0.0f : m)) * k;
}
__device__ __forceinline__ void sums_add(Sums& a, float z, float k)
{
    const float d = shift2(z, a.m, k);
    const float e = __builtin_amdgcn_exp2f(d);        // NaN stays NaN
    a.s += e;
    a.w = __builtin_fmaf(e, fmaxf(d, -1000.0f), a.w);   // 0 * -inf must not meet the sum
}
// raise the maximum to m
__device__ __forceinline__ void sums_raise(Sums& a, float m, float k)
{
    if (!(m > a.m)) return;
    if (a.m == -INFINITY) {                            // nothing summed yet
        a.m = m;
        return;
    }
    const float d = fmaxf((a.m - m) * k, -1000.0f), f = __builtin_amdgcn_exp2f(d);
    a.w = f * __builtin_fmaf(d, a.s, a.w);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void sums_merge(Sums& a, float m, float s, float w, float k)
{
    sums_raise(a, m, k);
    if (m == -INFINITY) {
        a.s += s;                                      // zero, or NaN
        return;
    }
    const float d = fmaxf((m - a.m) * k, -1000.0f), f = __builtin_amdgcn_exp2f(d);
    a.w += f * __builtin_fmaf(d, s, w);
    a.s += f * s;
}

// Sort key of a logit: larger value first, then lower index; NaN above
// everything, the two zeros equal.
__device__ __forceinline__ uint64_t sort_key(float z, uint32_t idx)
{
    uint32_t u = f_bits(z + 0.0f);
    u = (u & 0x7FFFFFFFu) > 0x7F800000u ? 0xFFFFFFFFu : (u >> 31) ? ~u : u | 0x80000000u;
    return ((uint64_t)u << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(uint64_t key)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return u == 0xFFFFFFFFu ? __builtin_nanf("") : bits_f((u >> 31) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// ---------------------------------------------------------------------------
// The wave's running top list: keys above `thr` are collected in its LDS
// buffer, and a full buffer is reduced to the best `top`, whose last is the
// new threshold.  The first round's threshold comes from the lanes' own
// maxima (the top-th largest of 64 elements is below the top-th of all), so
// a row in no particular order sends few elements to the buffer.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct TopList {
    uint64_t* buf;
    uint64_t thr;              // keys above it are candidates
    int cnt, top;

    __device__ __forceinline__ void reduce(int lane)
    {
        uint64_t mine[kLpBuf / 64];
        int rank[kLpBuf / 64];
        wave_sync();
#pragma unroll
        for (int i = 0; i < kLpBuf / 64; ++i) { mine[i] = 64 * i + lane < cnt ? buf[64 * i + lane] : 0; rank[i] = 0; }
        for (int j = 0; j < cnt; ++j) {
            const uint64_t o = buf[j];
#pragma unroll
            for (int i = 0; i < kLpBuf / 64; ++i) rank[i] += o > mine[i];
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < kLpBuf / 64; ++i)
            if (64 * i + lane < cnt && rank[i] < top) buf[rank[i]] = mine[i];
        wave_sync();
        if (cnt > top) cnt = top;
        if (cnt == top) {
            const uint64_t last = buf[top - 1];
            if (last > thr) thr = last;
        }
    }
    // every lane offers one key
    __device__ __forceinline__ void offer(uint64_t key, int lane)
    {
        uint64_t want = __builtin_amdgcn_ballot_w64(key > thr);
        if (!want) return;
        if (cnt + __builtin_popcountll(want) > kLpBuf) {
            reduce(lane);
            want = __builtin_amdgcn_ballot_w64(key > thr);
            if (!want) return;
        }
        if (key > thr) buf[cnt + __builtin_popcountll(want & ((1ull << lane) - 1))] = key;
        cnt += __builtin_popcountll(want);
    }
    // a first threshold from one key a lane (0: none)
    __device__ __forceinline__ void start(uint64_t key)
    {
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < 64; ++j) {
            const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), j) << 32) |
                               (uint32_t)__builtin_amdgcn_readlane((int)key, j);
            rank += o > key;
        }
        const uint64_t at = __builtin_amdgcn_ballot_w64(key != 0 && rank == top - 1);
        if (at) {
            const int j = __builtin_ctzll(at);
            thr = (((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), j) << 32) |
                   (uint32_t)__builtin_amdgcn_readlane((int)key, j)) - 1;
        }
    }
};

// The best `top` of `n` distinct keys in LDS, sorted, by counting larger ones.
template <typename F>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int top, int tid, int threads, F put)
{
    for (int i = tid; i < n; i += threads) {
        const uint64_t mine = keys[i];
        if (mine == 0) continue;
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += keys[j] > mine;
        if (rank < top) put(rank, mine);
    }
}

// Results of a row from its sums; the token's logit is read again (one
// element).  A row with no finite logit and no NaN holds no probability:
// its entropy is 0 and every log probability -inf.
template <bool BF16>
__device__ __forceinline__ void finish_row(const LogprobLaunch& p, int64_t row, const Sums& r, const uint64_t* keys,
                                           int nkeys, int tid, int threads)
{
    using T = typename Logit<BF16>::Raw;
    const float c = p.inv_temperature;
    const bool empty = r.m == -INFINITY && r.s == 0.0f;
    const float m0 = r.m == -INFINITY ? 0.0f : r.m, logs = empty ? 0.0f : logf(r.s);
    if (tid == 0) {
        const int64_t t = p.tokens ? p.tokens[row] : -1;
        float lp = 0.0f;
        if (t >= 0 && t < p.vocab)
            lp = empty ? -INFINITY : (Logit<BF16>::one((const T*)p.logits + row * p.ld + t) - m0) * c - logs;
        if (p.logprob) p.logprob[row] = lp;
        p.entropy[row] = empty ? 0.0f : logs - r.w * kLn2 / r.s;
        p.stats[2 * row] = r.m;
        p.stats[2 * row + 1] = empty ? -INFINITY : logs;
    }
    if (p.top > 0)
        rank_keys(keys, nkeys, p.top, tid, threads, [&](int rank, uint64_t key) {
            p.top_ids[row * p.top + rank] = (int32_t)key_index(key);
            p.top_logprobs[row * p.top + rank] = empty ? -INFINITY : (key_value(key) - m0) * c - logs;
        });
}

// ---------------------------------------------------------------------------
// One workgroup per row (gridDim.y = 1), or per piece of a row, whose sums
// and top keys k_lp_join joins.  Rows may start at any element: the elements
// before the first 16-byte boundary and after the last whole vector are taken
// one a thread.
// ---------------------------------------------------------------------------
template <bool BF16, bool TOP, int THREADS>
__global__ __launch_bounds__(THREADS) void k_lp_rows(LogprobLaunch p)
{
    using L = Logit<BF16>;
    using T = typename L::Raw;
    constexpr int NW = THREADS / 64, VN = L::N;
    __shared__ uint64_t cand[TOP ? NW * kLpBuf : 1];
    __shared__ float sm[NW][3];
    __shared__ int counts[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    const T* const z = (const T*)p.logits + row * p.ld;
    const int64_t b = (int64_t)blockIdx.y * p.piece, e = b + p.piece < p.vocab ? b + p.piece : p.vocab;
    const float k = p.inv_temperature * kLog2e;

    Sums a{-INFINITY, 0.0f, 0.0f};
    TopList list{cand + (TOP ? wave * kLpBuf : 0), 0, 0, p.top};
    // elements before the first boundary, and after the last whole vector
    const int64_t head = (int64_t)((16 - ((uintptr_t)(z + b) & 15)) & 15) / (int64_t)sizeof(T);
    const int64_t vb = b + head < e ? b + head : e;
    const int64_t nvec = (e - vb) / VN;
    const int64_t ve = vb + nvec * VN;
    const v4i* const zv = reinterpret_cast<const v4i*>(z + vb);
    bool first = true;
    for (int64_t r0 = 0; r0 < nvec; r0 += (int64_t)THREADS * kLpVec) {
        v4i raw[kLpVec];
        bool in[kLpVec];
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + (int64_t)u * THREADS + tid;
            in[u] = i < nvec;
            if (in[u]) raw[u] = zv[i];
        }
        float f[kLpVec][VN], best = -INFINITY;
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            if (in[u]) {
                L::unpack(raw[u], f[u]);
            } else {
#pragma unroll
                for (int j = 0; j < VN; ++j) f[u][j] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < VN; ++j) best = fmaxf(best, f[u][j]);
        }
        sums_raise(a, best, k);
#pragma unroll
        for (int u = 0; u < kLpVec; ++u)
#pragma unroll
            for (int j = 0; j < VN; ++j) sums_add(a, f[u][j], k);
        if (TOP) {
            // a NaN is above everything and `best` drops it: look at the sum
            const bool odd = a.s != a.s;
            if (first) {
                uint64_t mk = 0;
#pragma unroll
                for (int u = 0; u < kLpVec; ++u)
#pragma unroll
                    for (int j = 0; j < VN; ++j)
                        if (in[u]) {
                            const uint64_t key = sort_key(f[u][j], (uint32_t)(vb + (r0 + (int64_t)u * THREADS + tid) * VN + j));
                            mk = key > mk ? key : mk;
                        }
                list.start(mk);
                first = false;
            }
            const uint64_t bk = sort_key(best, 0u);
            if (__builtin_amdgcn_ballot_w64(bk > list.thr || odd)) {
#pragma unroll
                for (int u = 0; u < kLpVec; ++u)
#pragma unroll
                    for (int j = 0; j < VN; ++j)
                        list.offer(in[u] ? sort_key(f[u][j], (uint32_t)(vb + (r0 + (int64_t)u * THREADS + tid) * VN + j)) : 0,
                                   lane);
            }
        }
    }
    // at most VN - 1 elements on either side
    {
        const int64_t nh = vb - b, nt = e - ve;
        const int64_t i = tid < nh ? b + tid : ve + (tid - nh);
        const bool in = tid < nh + nt;
        const float v = in ? L::one(z + i) : -INFINITY;
        sums_raise(a, v, k);
        sums_add(a, v, k);
        if (TOP && wave == 0) list.offer(in ? sort_key(v, (uint32_t)i) : 0, lane);
    }
    if (TOP) {
        list.reduce(lane);
        if (lane == 0) counts[wave] = list.cnt;
    }
    // threads of the wave, then the waves
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float m = __shfl_xor(a.m, o), s = __shfl_xor(a.s, o), w = __shfl_xor(a.w, o);
        sums_merge(a, m, s, w, k);
    }
    if (lane == 0) { sm[wave][0] = a.m; sm[wave][1] = a.s; sm[wave][2] = a.w; }
    __syncthreads();
    Sums r{-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; ++w) sums_merge(r, sm[w][0], sm[w][1], sm[w][2], k);
    int n = 0;
    if (TOP) {                                        // the waves' lists side by side
        uint64_t mine = 0;
        int at = 0;
        for (int w = 0; w < wave; ++w) at += counts[w];
        for (int w = 0; w < NW; ++w) n += counts[w];
        if (lane < counts[wave]) mine = list.buf[lane];
        __syncthreads();
        if (lane < counts[wave]) cand[at + lane] = mine;
        __syncthreads();
    }
    if (gridDim.y == 1) {
        finish_row<BF16>(p, row, r, cand, n, tid, THREADS);
        return;
    }
    const int64_t part = row * gridDim.y + blockIdx.y;
    if (tid == 0) {
        float* const o = p.part_sums + 4 * part;
        o[0] = r.m; o[1] = r.s; o[2] = r.w;
    }
    if (TOP) {
        uint64_t* const o = p.part_keys + part * p.top;
        for (int i = n + tid; i < p.top; i += THREADS) o[i] = 0;      // fewer elements than the list is long
        rank_keys(cand, n, p.top, tid, THREADS, [&](int rank, uint64_t key) { o[rank] = key; });
    }
}

template <bool BF16, bool TOP>
__global__ __launch_bounds__(256) void k_lp_join(LogprobLaunch p, int pieces)
{
    __shared__ uint64_t cand[TOP ? kLpMaxTop * kLpMaxPieces : 1];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const float k = p.inv_temperature * kLog2e;
    Sums r{-INFINITY, 0.0f, 0.0f};
    for (int i = 0; i < pieces; ++i) {
        const float* const o = p.part_sums + 4 * (row * pieces + i);
        sums_merge(r, o[0], o[1], o[2], k);
    }
    if (TOP) {
        for (int i = tid; i < pieces * p.top; i += 256) cand[i] = p.part_keys[row * pieces * p.top + i];
        __syncthreads();
    }
    finish_row<BF16>(p, row, r, cand, pieces * p.top, tid, 256);
}

// ---------------------------------------------------------------------------
// dz: one workgroup per row and piece.  A row whose two coefficients are both
// zero (padding) is written as zeros without reading its logits.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(256) void k_lp_backward(LogprobGradLaunch p)
{
    using L = Logit<BF16>;
    using T = typename L::Raw;
    constexpr int VN = L::N;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const T* const z = (const T*)p.logits + row * p.ld;
    T* const dz = (T*)p.dlogits + row * p.ldd;
    const int64_t b = (int64_t)blockIdx.y * p.piece, e = b + p.piece < p.vocab ? b + p.piece : p.vocab;
    const float c = p.inv_temperature;
    const float m = p.stats[2 * row], logs = p.stats[2 * row + 1], ent = p.entropy[row];
    const int64_t t = p.tokens ? p.tokens[row] : -1;
    const bool empty = logs == -INFINITY;                 // no probability anywhere: no gradient
    const float gl = p.g_logprob && t >= 0 && t < p.vocab && !empty ? p.g_logprob[row] : 0.0f;
    const float ge = p.g_entropy && !empty ? p.g_entropy[row] : 0.0f;
    const bool none = gl == 0.0f && ge == 0.0f;
    const float k = c * kLog2e, logs2 = logs * kLog2e;
    const float m0 = m == -INFINITY ? 0.0f : m;
    // -c (gl + ge (log p + H)) as u + v log2 p
    const float cu = -c * __builtin_fmaf(ge, ent, gl), cv = -c * ge * kLn2;
    auto grad = [&](float x) {
        const float l2 = (x - m0) * k - logs2;
        return __builtin_amdgcn_exp2f(l2) * __builtin_fmaf(cv, fmaxf(l2, -1000.0f), cu);
    };
    auto put = [&](int64_t i) {
        float g = 0.0f;
        if (!none) g = grad(L::one(z + i)) + (i == t ? c * gl : 0.0f);
        if constexpr (BF16) dz[i] = (uint16_t)f32_to_bf16_rne(g);
        else dz[i] = g;
    };
    const int64_t head = (int64_t)((16 - ((uintptr_t)(z + b) & 15)) & 15) / (int64_t)sizeof(T);
    // vectors where both rows reach a 16-byte boundary at the same element
    const bool same = (((uintptr_t)(z + b) ^ (uintptr_t)(dz + b)) & 15) == 0;
    const int64_t vb = !same ? e : b + head < e ? b + head : e;
    const int64_t nvec = (e - vb) / VN, ve = vb + nvec * VN;
    const v4i* const zv = reinterpret_cast<const v4i*>(z + vb);
    v4i* const dv = reinterpret_cast<v4i*>(dz + vb);
    for (int64_t r0 = 0; r0 < nvec; r0 += 256 * kLpVec) {
        v4i raw[kLpVec];
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + 256 * u + tid;
            if (i < nvec && !none) raw[u] = zv[i];
        }
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + 256 * u + tid;
            if (i >= nvec) continue;
            v4i out{0, 0, 0, 0};
            if (!none) {
                float f[VN];
                L::unpack(raw[u], f);
                const int64_t at = t - (vb + i * VN);
#pragma unroll
                for (int j = 0; j < VN; ++j) f[j] = grad(f[j]) + (at == j ? c * gl : 0.0f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (BF16) out[q] = (int)(f32_to_bf16_rne(f[2 * q]) | (f32_to_bf16_rne(f[2 * q + 1]) << 16));
                    else out[q] = (int)f_bits(f[q]);
                }
            }
            dv[i] = out;
        }
    }
    for (int64_t i = b + tid; i < vb; i += 256) put(i);
    for (int64_t i = ve + tid; i < e; i += 256) put(i);
}

// ---------------------------------------------------------------------------
// launch shapes
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A row stays whole when the rows alone fill the device; else it is cut so
// that about 512 workgroups run, none with less than one round of its
// threads (8192 elements).
int64_t logprob_pieces(int64_t rows, int64_t vocab)
{
    if (rows < 1 || rows >= 512) return 1;
    int64_t n = cdiv(512, rows), most = cdiv(vocab, 8192);
    n = n < most ? n : most;
    n = n < kLpMaxPieces ? n : kLpMaxPieces;
    return n < 1 ? 1 : n;
}

template <bool BF16, bool TOP>
static hipError_t run_logprobs(LogprobLaunch p, int64_t pieces, hipStream_t s)
{
    p.piece = cdiv(cdiv(p.vocab, pieces), 64) * 64;
    pieces = cdiv(p.vocab, p.piece);
    const dim3 grid((unsigned)p.rows, (unsigned)pieces);
    hipLaunchKernelGGL((k_lp_rows<BF16, TOP, 256>), grid, dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || pieces == 1) return e;
    hipLaunchKernelGGL((k_lp_join<BF16, TOP>), dim3((unsigned)p.rows), dim3(256), 0, s, p, (int)pieces);
    return hipGetLastError();
}

hipError_t launch_logprobs(const LogprobLaunch& p, int64_t pieces, hipStream_t s)
{
    if (p.bf16) return p.top ? run_logprobs<true, true>(p, pieces, s) : run_logprobs<true, false>(p, pieces, s);
    return p.top ? run_logprobs<false, true>(p, pieces, s) : run_logprobs<false, false>(p, pieces, s);
}

hipError_t launch_logprobs_backward(const LogprobGradLaunch& in, hipStream_t s)
{
    LogprobGradLaunch p = in;
    // two rounds of a workgroup's threads: 16384 bf16 or 8192 binary32 elements
    p.piece = 2 * 256 * kLpVec * (p.bf16 ? 8 : 4);
    const dim3 grid((unsigned)p.rows, (unsigned)cdiv(p.vocab, p.piece));
    if (p.bf16) hipLaunchKernelGGL((k_lp_backward<true>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_lp_backward<false>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace fp4
