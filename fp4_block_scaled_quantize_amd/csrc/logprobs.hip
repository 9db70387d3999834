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
// f (w - c D s).  A round of loads is summed on its own first, so that a
// thread's sum of thousands of terms takes few roundings.  The kernels work in
// powers of two (k = c log2 e), where w carries log2 units.
#include <type_traits>

#include "fp4_device.hpp"
#include "fp4_internal.h"
#include "logits_device.hpp"

namespace fp4 {

constexpr int kLpMaxTop = 32;
constexpr int kLpBuf = 256;            // candidate keys of a wave

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
    float value;               // its logit: a smaller one cannot be a candidate
    int cnt, top;

    __device__ __forceinline__ void raise(uint64_t key)
    {
        if (key <= thr) return;
        thr = key;
        value = key_value(key);
    }
    // rank the lane's N keys against the whole buffer and keep the best, sorted
    template <int N>
    __device__ __forceinline__ void rank(int lane)
    {
        uint64_t mine[N];
        int at[N];
#pragma unroll
        for (int i = 0; i < N; ++i) { mine[i] = 64 * i + lane < cnt ? buf[64 * i + lane] : 0; at[i] = 0; }
        for (int j = 0; j < cnt; j += 8) {             // eight reads in flight
            uint64_t o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] = buf[j + u];
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int i = 0; i < N; ++i) at[i] += o[u] > mine[i];
        }
        wave_sync();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (64 * i + lane < cnt && at[i] < top) buf[at[i]] = mine[i];
    }
    __device__ __forceinline__ void reduce(int lane)
    {
        if (lane < 8 && cnt + lane < kLpBuf) buf[cnt + lane] = 0;       // whole groups of eight
        wave_sync();
        if (cnt <= 64) rank<1>(lane);
        else rank<kLpBuf / 64>(lane);
        wave_sync();
        if (cnt > top) cnt = top;
        if (cnt == top) raise(buf[top - 1]);
    }
    // Every lane offers those of its N elements that may be above the
    // threshold (a NaN passes), one a turn: few lanes have more than a couple,
    // where visiting the N places for the wave would find one in nearly each.
    // index(e): the place of element e; have: bit e set where there is one.
    // A list well past its length is cut at the end: the sooner the threshold
    // rises, the fewer elements reach the buffer.
    template <int N, typename F>
    __device__ __forceinline__ void offer(const float (&f)[N], uint32_t have, int lane, F index)
    {
        static_assert(N <= 32, "a bit for each element");
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint32_t up = !(f[e] < value);
            mine |= up << e;
        }
        mine &= have;
        for (;;) {
            const bool more = __builtin_amdgcn_ballot_w64(mine != 0) != 0;
            if (cnt > (more ? kLpBuf - 64 : top + 32)) reduce(lane);
            if (!more) break;
            const int e = mine ? __builtin_ctz(mine) : 0;
            float v = f[0];
#pragma unroll
            for (int i = 1; i < N; ++i) v = e == i ? f[i] : v;
            const uint64_t key = mine ? sort_key(v, index(e)) : 0;
            const uint64_t want = __builtin_amdgcn_ballot_w64(key > thr);
            if (key > thr) buf[cnt + __builtin_popcountll(want & ((1ull << lane) - 1))] = key;
            cnt += __builtin_popcountll(want);
            mine &= mine - 1;
        }
    }
    // a first threshold from the lanes' largest logits: below the smallest of
    // those that fewer than `top` lanes exceed
    __device__ __forceinline__ void start(bool in, float z)
    {
        const uint32_t v = in ? (uint32_t)(sort_key(z, 0) >> 32) : 0;
        int at = 0;
#pragma unroll
        for (int j = 0; j < 64; ++j) at += (uint32_t)__builtin_amdgcn_readlane((int)v, j) > v;
        const uint64_t best = __builtin_amdgcn_ballot_w64(v != 0 && at < top);
        if (__builtin_popcountll(best) < top) return;
        // the last of them: the lane with the largest count
        uint32_t low = (best >> (threadIdx.x & 63)) & 1 ? v : 0xFFFFFFFFu;
#pragma unroll
        for (int o = 32; o; o >>= 1) { const uint32_t x = __shfl_xor((int)low, o); low = x < low ? x : low; }
        thr = (uint64_t)low << 32;                     // an index never makes all ones: every key of that value is above
        value = key_value(thr);
    }
};

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int j)
{
    return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), j) << 32) |
           (uint32_t)__builtin_amdgcn_readlane((int)v, j);
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int o)
{
    return ((uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), o) << 32) | (uint32_t)__shfl_xor((int)v, o);
}

// The best `top` keys, sorted, of `lists` sorted lists of at most `top` keys
// each (at most 64) side by side (zeros, which are no keys, fill a short one).  The last
// key of a whole list bounds the result from below; the few above the largest
// such bound are ranked by counting the larger ones.  `few` holds at most
// lists * top + 8 keys; all `threads` of the workgroup call.
template <typename F>
__device__ __forceinline__ void best_of_lists(const uint64_t* keys, int lists, int top, uint64_t* few, int* count, int tid,
                                              int threads, F put)
{
    uint64_t low = 0;
    const int lane = tid & 63;
    if (lane < lists) low = keys[(lane + 1) * top - 1];
#pragma unroll
    for (int o = 32; o; o >>= 1) { const uint64_t x = shfl_xor64(low, o); low = x > low ? x : low; }
    if (lists >= top) {                                // many short lists: the top-th of their first keys bounds it closer
        const uint64_t mine = lane < lists ? keys[lane * top] : 0;
        int at = 0;
#pragma unroll 8
        for (int j = 0; j < 64; ++j) at += readlane64(mine, j) > mine;
        const uint64_t last = __builtin_amdgcn_ballot_w64(mine != 0 && at == top - 1);
        if (last) {
            const uint64_t x = readlane64(mine, __builtin_ctzll(last));
            low = x > low ? x : low;
        }
    }
    if (tid == 0) *count = 0;
    __syncthreads();
    for (int i = tid; i < lists * top; i += threads) {
        const uint64_t o = keys[i];
        // an LDS counter: the places they get differ from run to run, the ranks below do not
        if (o != 0 && o >= low) few[atomicAdd(count, 1)] = o;
    }
    __syncthreads();
    const int n = *count;
    if (tid < 8) few[n + tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += threads) {
        const uint64_t mine = few[i];
        int rank = 0;
        for (int j = 0; j < n; j += 8) {               // eight reads in flight
            uint64_t o[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) o[u] = few[j + u];
#pragma unroll
            for (int u = 0; u < 8; ++u) rank += o[u] > mine;
        }
        if (rank < top) put(rank, mine);
    }
}

// The row's token and its logit, fetched ahead of the sums by one thread.
struct Given { bool is; float z; };

template <bool BF16>
__device__ __forceinline__ Given given_token(const LogprobLaunch& p, int64_t row)
{
    using T = typename Logit<BF16>::Raw;
    const int64_t t = p.tokens ? p.tokens[row] : -1;
    const bool is = t >= 0 && t < p.vocab;
    return Given{is, is ? Logit<BF16>::one((const T*)p.logits + row * p.ld + t) : 0.0f};
}

// Results of a row from its sums.  A row with no finite logit and no NaN holds
// no probability: its entropy is 0 and every log probability -inf.
__device__ __forceinline__ void finish_row(const LogprobLaunch& p, int64_t row, const Sums& r, const Given& g)
{
    const float c = p.inv_temperature;
    const bool empty = r.m == -INFINITY && r.s == 0.0f;
    const float m0 = r.m == -INFINITY ? 0.0f : r.m, logs = empty ? 0.0f : logf(r.s);
    if (p.logprob) p.logprob[row] = !g.is ? 0.0f : empty ? -INFINITY : (g.z - m0) * c - logs;
    p.entropy[row] = empty ? 0.0f : logs - r.w * kLn2 / r.s;
    p.stats[2 * row] = r.m;
    p.stats[2 * row + 1] = empty ? -INFINITY : logs;
}

__device__ __forceinline__ void put_top(const LogprobLaunch& p, int64_t row, const Sums& r, int rank, uint64_t key)
{
    const bool empty = r.m == -INFINITY && r.s == 0.0f;
    const float m0 = r.m == -INFINITY ? 0.0f : r.m;
    p.top_ids[row * p.top + rank] = (int32_t)key_index(key);
    p.top_logprobs[row * p.top + rank] = empty ? -INFINITY : (key_value(key) - m0) * p.inv_temperature - logf(r.s);
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
    constexpr int64_t kRound = (int64_t)THREADS * kLpVec;
    __shared__ uint64_t cand[TOP ? NW * kLpBuf : 1];
    __shared__ uint64_t lists[TOP ? NW * kLpMaxTop : 1];
    __shared__ int count;
    __shared__ float sm[NW][3];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    const T* const z = (const T*)p.logits + row * p.ld;
    const int64_t b = (int64_t)blockIdx.y * p.piece, e = b + p.piece < p.vocab ? b + p.piece : p.vocab;
    const float k = p.inv_temperature * kLog2e;

    Given given{false, 0.0f};
    if (tid == 0 && gridDim.y == 1) given = given_token<BF16>(p, row);
    Running a{-INFINITY, 0.0f, 0.0f, 0.0f};
    TopList list{cand + (TOP ? wave * kLpBuf : 0), 0, -INFINITY, 0, p.top};
    // elements before the first boundary, and after the last whole vector
    const int64_t head = (int64_t)((16 - ((uintptr_t)(z + b) & 15)) & 15) / (int64_t)sizeof(T);
    const int64_t vb = b + head < e ? b + head : e;
    const int64_t nvec = (e - vb) / VN;
    const int64_t ve = vb + nvec * VN;
    const v4i* const zv = reinterpret_cast<const v4i*>(z + vb);
    // the next round's vectors are on their way while this one's are summed
    v4i next[kLpVec];
    auto fetch = [&](int64_t r0) {
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            const int64_t i = r0 + (int64_t)u * THREADS + tid;
            if (i < nvec) next[u] = zv[i];
        }
    };
    fetch(0);
    bool first = true;
    auto round = [&](int64_t r0, auto whole) {             // whole: every thread has all of its vectors
        bool in[kLpVec];
        float f[kLpVec * VN], best = -INFINITY;
        uint32_t have = 0;
#pragma unroll
        for (int u = 0; u < kLpVec; ++u) {
            in[u] = whole || r0 + (int64_t)u * THREADS + tid < nvec;
            float v[VN];
            L::unpack(next[u], v);
#pragma unroll
            for (int j = 0; j < VN; ++j) f[u * VN + j] = in[u] ? v[j] : -INFINITY;
            have |= in[u] ? ((1u << VN) - 1) << (u * VN) : 0u;
        }
        fetch(r0 + kRound);
#pragma unroll
        for (int j = 0; j < kLpVec * VN; ++j) best = fmaxf(best, f[j]);
        a.raise(best, k);
        // the round's terms add up on their own before they join the row's: a
        // thread's sum takes roundings for the terms of one round and for the
        // rounds, not for thousands of terms
        const float s = a.s, w = a.w;
        a.s = a.w = 0.0f;
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
        a.w += w;
        if (TOP) {
            if (first) list.start(in[0], best);
            first = false;
            // a NaN is above everything and `best` drops it: look at the sum
            if (__builtin_amdgcn_ballot_w64(!(best < list.value) || a.s != a.s))
                list.offer(f, have, lane, [&](int j) {
                    return (uint32_t)(vb + (r0 + (int64_t)(j / VN) * THREADS + tid) * VN + j % VN);
                });
        }
    };
    int64_t r0 = 0;
    for (; r0 + kRound <= nvec; r0 += kRound) round(r0, std::true_type{});
    if (r0 < nvec) round(r0, std::false_type{});
    // at most VN - 1 elements on either side
    if (wave == 0) {
        const int64_t nh = vb - b, nt = e - ve;
        const int64_t i = tid < nh ? b + tid : ve + (tid - nh);
        const bool in = tid < nh + nt;
        const float v = in ? L::one(z + i) : -INFINITY;
        a.raise(v, k);
        if (a.far(k)) a.template add<true>(v, k);
        else a.template add<false>(v, k);
        if (TOP) {
            const float one[1]{v};
            list.offer(one, in, lane, [&](int) { return (uint32_t)i; });
        }
    }
    // threads of the wave, then the waves
    Sums r = a.about_max(k);
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float m = __shfl_xor(r.m, o), s = __shfl_xor(r.s, o), w = __shfl_xor(r.w, o);
        sums_merge(r, m, s, w, k);
    }
    if (lane == 0) { sm[wave][0] = r.m; sm[wave][1] = r.s; sm[wave][2] = r.w; }
    if (TOP) {
        list.reduce(lane);
        if (lane < p.top) lists[wave * p.top + lane] = lane < list.cnt ? list.buf[lane] : 0;
    }
    __syncthreads();
    r = Sums{-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; ++w) sums_merge(r, sm[w][0], sm[w][1], sm[w][2], k);
    if (gridDim.y == 1) {
        if (tid == 0) finish_row(p, row, r, given);
        if (TOP && NW == 1) {                              // the wave's list is the row's
            if (lane < p.top) put_top(p, row, r, lane, lists[lane]);
        } else if (TOP)
            best_of_lists(lists, NW, p.top, cand, &count, tid, THREADS,
                          [&](int rank, uint64_t key) { put_top(p, row, r, rank, key); });
        return;
    }
    const int64_t part = row * gridDim.y + blockIdx.y;
    if (tid == 0) {
        float* const o = p.part_sums + 4 * part;
        o[0] = r.m; o[1] = r.s; o[2] = r.w;
    }
    if (TOP) {
        uint64_t* const o = p.part_keys + part * p.top;
        if (e - b < p.top)                                 // fewer elements than the list is long
            for (int i = tid; i < p.top; i += THREADS)
                if (i >= e - b) o[i] = 0;
        best_of_lists(lists, NW, p.top, cand, &count, tid, THREADS, [&](int rank, uint64_t key) { o[rank] = key; });
    }
}

constexpr int kLpJoin = 256;           // threads

template <bool BF16, bool TOP>
__global__ __launch_bounds__(kLpJoin) void k_lp_join(LogprobLaunch p, int pieces)
{
    __shared__ uint64_t cand[TOP ? kLpMaxTop * kLpMaxPieces : 1];
    __shared__ uint64_t few[TOP ? kLpMaxTop * kLpMaxPieces + 8 : 1];
    __shared__ int count;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const float k = p.inv_temperature * kLog2e;
    Sums r{-INFINITY, 0.0f, 0.0f};
    Given given{false, 0.0f};
    if (tid == 0) given = given_token<BF16>(p, row);
    if (TOP)
#pragma unroll 4
        for (int i = tid; i < pieces * p.top; i += kLpJoin) cand[i] = p.part_keys[row * pieces * p.top + i];
    // a piece for each lane of every wave, joined as the lanes of k_lp_rows are
    if ((tid & 63) < pieces) {
        const float* const o = p.part_sums + 4 * (row * pieces + (tid & 63));
        r = Sums{o[0], o[1], o[2]};
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        const float m = __shfl_xor(r.m, o), s = __shfl_xor(r.s, o), w = __shfl_xor(r.w, o);
        sums_merge(r, m, s, w, k);
    }
    if (tid == 0) finish_row(p, row, r, given);
    if (TOP) {
        __syncthreads();
        best_of_lists(cand, pieces, p.top, few, &count, tid, kLpJoin,
                      [&](int rank, uint64_t key) { put_top(p, row, r, rank, key); });
    }
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
    // p is taken as the square of h = 2^(log2 p / 2): the instruction flushes
    // powers below 2^-126, which a large coefficient would make visible.  (A
    // power of p times 2^16 needs log2 p + 16, which in a confident row rounds
    // log p and the entropy away.)
    const float k = 0.5f * c * kLog2e, hlogs = 0.5f * logs * kLog2e;
    const float m0 = m == -INFINITY ? 0.0f : m;
    // -(gl + ge (log p + H)) as gu + gv (log2 p / 2); c comes last: where it is large (a
    // temperature near zero) it must not overflow against p = 0
    const float gv = -2.0f * kLn2 * ge, gu = -__builtin_fmaf(ge, ent, gl);
    auto grad = [&](float x, bool hit) {
        const float l = (x - m0) * k - hlogs, h = __builtin_amdgcn_exp2f(l);
        return c * __builtin_fmaf(h, h * __builtin_fmaf(gv, fmaxf(l, -1000.0f), gu), hit ? gl : 0.0f);
    };
    auto put = [&](int64_t i) {
        float g = 0.0f;
        if (!none) g = grad(L::one(z + i), i == t);
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
                for (int j = 0; j < VN; ++j) f[j] = grad(f[j], at == j);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (BF16) out[q] = (int)pack_bf16(f[2 * q], f[2 * q + 1]);
                    else out[q] = (int)f_bits(f[q]);
                }
            }
            __builtin_nontemporal_store(out, dv + i);     // read next long after it has left the caches
        }
    }
    for (int64_t i = b + tid; i < vb; i += 256) put(i);
    for (int64_t i = ve + tid; i < e; i += 256) put(i);
}

// ---------------------------------------------------------------------------
// launch shapes
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether a whole row is one wave's instead of four's: without top alternatives
// where it is short (8192 rows of 9000, bf16: 36 us against 49; of 32000 107
// against 100).  With them four waves keep four lists, each of which takes in
// its first few hundred logits, and wait to join them, so one is better
// wherever the rows alone fill the device (top 1: 4235 rows of 142 14 us
// against 52, 1500 of 9000 17 against 27, 5030 of 21562 65 against 101, 8192 of
// 32000 121 against 177; but 600 of 12000, top 20, 22 against 17, 600 of 30000 38
// against 27, 1061 of 115285 120 against 95).  All with logits that come from
// memory.
static bool row_is_a_wave(int64_t rows, int64_t vocab, bool top)
{
    if (!top) return vocab <= 16384;
    return vocab <= 4096 || rows >= (vocab <= 16384 ? 1024 : 2000);
}

// A row stays whole when the rows alone fill the device; else it is cut so
// that about 512 workgroups run, none with less than 4096 elements (two bf16
// vectors a thread).
int64_t logprob_pieces(int64_t rows, int64_t vocab)
{
    if (rows < 1 || rows >= 512) return 1;
    int64_t n = cdiv(512, rows), most = cdiv(vocab, 4096);
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
    const bool wave = pieces == 1 && row_is_a_wave(p.rows, p.vocab, TOP);
    if (wave) hipLaunchKernelGGL((k_lp_rows<BF16, TOP, 64>), grid, dim3(64), 0, s, p);
    else hipLaunchKernelGGL((k_lp_rows<BF16, TOP, 256>), grid, dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || pieces == 1) return e;
    hipLaunchKernelGGL((k_lp_join<BF16, TOP>), dim3((unsigned)p.rows), dim3(TOP ? kLpJoin : 64), 0, s, p, (int)pieces);
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
