// lora.hip -- low-rank adapters of many requests beside a shared projection
// (quant_prune_distill/574 "Метод": a trained low-rank adapter runs in
// parallel with the FP4 weight).
//
// Row i of a batch uses adapter l = slots[i] (none when l is outside the
// bank).  With A [L, R, K], B [L, N, R] in bf16 and a scale s_l:
//   forward   T = x A_l^T,  y = base + s_l T B_l^T
//   backward  dT = s_l dy B_l,  dx = base + dT A_l,
//             dA_l = sum_i dT_i^T x_i,  dB_l = s_l sum_i dy_i^T T_i
// T and dT stay in binary32.  Where one enters a bf16 matrix instruction it
// goes in as the sum of three bf16 terms, which hold its 24 bits, so the
// results are rounded once, at the end.  (Two terms, 16 bits, rounded about one
// output in a thousand the other way and saved nothing that showed.)
#include "fp4_device.hpp"
#include "fp4_internal.h"

namespace fp4 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// The adapter of a row: slots[row] when it names one of the bank, else -1.
__device__ __forceinline__ int row_slot(const int32_t* slots, int64_t row, int64_t m, int64_t adapters)
{
    if (row >= m) return -1;
    const int s = slots[row];
    return s >= 0 && s < adapters ? s : -1;
}

// Two values as three bf16 terms each, packed (a in the low half): each term
// the rounding of what the ones before leave.  A value that rounds to infinity
// leaves nothing, so that it stays one.
constexpr int kTerms = 3;
__device__ __forceinline__ void bf16_terms(float a, float b, uint32_t (&out)[kTerms])
{
    constexpr float kTop = 3.3961775e38f;               // the midpoint above the largest bf16
    const bool fa = !(fabsf(a) >= kTop), fb = !(fabsf(b) >= kTop);
    out[0] = pack_bf16(a, b);
#pragma unroll
    for (int i = 1; i < kTerms; ++i) {
        a = fa ? a - bf16_lo(out[i - 1]) : 0.0f;
        b = fb ? b - bf16_hi(out[i - 1]) : 0.0f;
        out[i] = pack_bf16(a, b);
    }
}

// Eight elements `stride` apart as a fragment: an operand whose contraction
// runs across its rows (TR below).  A small backward call takes B and A
// that way; for a larger one they are transposed once (k_lora_transpose).
__device__ __forceinline__ v4i gather8(const uint16_t* p, int64_t stride)
{
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = p[i * stride];
    v4i v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = (int)(e[2 * q] | ((uint32_t)e[2 * q + 1] << 16));
    return v;
}

// ---------------------------------------------------------------------------
// T = x A_l^T for at most 16 rows: one workgroup per K range, its eight waves
// on every eighth batch of 128 elements, joined through LDS in a fixed order.
// Both operands run along K, so each lane's 16 bytes are a matrix-instruction
// fragment as they come from memory; nothing is staged, and a batch's loads
// leave together: latency is what such a call waits for.  Rows of several
// adapters run the K range once for each (gridDim.z of them side by side) and
// keep each row's own.  With gridDim.x > 1 the K ranges' partial sums are left
// for the reader of T to join.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

template <int RT, bool TR>
__global__ __launch_bounds__(64 * kFewWaves) void k_lora_down_few(LoraDown p)
{
    constexpr int NW = kFewWaves;
    __shared__ v4f red[NW][RT * 64];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t M = p.m, K = p.k;
    const int R = p.rank;
    float* const t = p.t + (int64_t)blockIdx.x * M * R;
    const int slot = lane < 16 ? row_slot(p.slots, lane, M, p.adapters) : -1;

    if (blockIdx.z == 0) {                    // rows without an adapter
        for (int i = wave; i < (int)M; i += NW)
            if (__builtin_amdgcn_readlane(slot, i) < 0)
                for (int r = lane; r < R; r += 64) t[i * R + r] = 0.0f;
    }

    const int64_t kb = (int64_t)blockIdx.x * p.kstep, ke = kb + p.kstep < K ? kb + p.kstep : K;
    const uint16_t* const xr = p.x + (r16 < M ? r16 : M - 1) * p.ldx;
    int64_t ar[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) ar[j] = (int64_t)(16 * j + r16 < R ? 16 * j + r16 : R - 1) * (TR ? 1 : K);

    uint64_t todo = __builtin_amdgcn_ballot_w64(slot >= 0);
    for (unsigned nth = 0; todo; ++nth) {
        const int cur = __builtin_amdgcn_readlane(slot, __builtin_ctzll(todo));
        const uint64_t match = __builtin_amdgcn_ballot_w64(slot == cur);
        todo &= ~match;
        if (nth % gridDim.z != blockIdx.z) continue;
        const uint16_t* const a = p.a + (int64_t)cur * R * K;
        v4f acc[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int64_t k = kb + 128 * wave; k < ke; k += 128 * NW) {
            const v4i zero{0, 0, 0, 0};
            constexpr int U = TR ? (RT > 2 ? 1 : 2) : 4;       // steps whose loads leave together
#pragma unroll 1
            for (int u0 = 0; u0 < 4; u0 += U) {
                v4i xf[U], af[U][RT];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = k + 32 * (u0 + u) + 8 * grp;
                    const bool in = c < ke;                    // 8 elements, all in or all out
                    xf[u] = in ? *reinterpret_cast<const v4i*>(xr + c) : zero;
#pragma unroll
                    for (int j = 0; j < RT; ++j)
                        af[u][j] = !in  ? zero
                                   : TR ? gather8(a + c * R + ar[j], R)
                                        : *reinterpret_cast<const v4i*>(a + ar[j] + c);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[j] = mfma16(af[u][j], xf[u], acc[j]);
            }
        }
        // acc[j][e] = T[m = r16][r = 16 j + 4 grp + e]
#pragma unroll
        for (int j = 0; j < RT; ++j) red[wave][j * 64 + lane] = acc[j];
        __syncthreads();
        const float s = p.scale ? p.scale[cur] : 1.0f;
        for (int e = tid; e < RT * 64; e += 64 * NW) {
            const int l = e & 63, m = l & 15, r = 16 * (e >> 6) + 4 * (l >> 4);
            if (((match >> m) & 1) && r < R) {
                v4f v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < NW; ++w) v += red[w][e];
                *reinterpret_cast<v4f*>(t + m * R + r) = v * s;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// T = x A_l^T for more rows: one workgroup per 32 rows and K range, its four
// waves on every fourth chunk of 128 elements.  Bound by reading x, which
// wants whole lines: fragments taken straight from memory touch 64 bytes of
// 16 rows at a time (8192 rows of 11008, rank 16: 71 us that way, 42 so, 4.3
// TB/s).  So a wave brings its next chunk (32 rows x 256 bytes) into LDS with direct loads of four rows
// each while it multiplies the one before; A's fragments, shared by all row
// tiles, come from the cache.  A 16-byte piece c of row r lies at c ^ (r % 16),
// so that the 16 rows of a fragment read fall on distinct banks (the lanes
// pick their global pieces accordingly).  Adapters and K ranges as above; a
// tile's K ranges are neighbours in the grid, so that what is read at one time
// are longer pieces of fewer rows (47 us with the tiles first).
// ---------------------------------------------------------------------------
constexpr int kDownWaves = 4, kDownRows = 32;
constexpr int kDownSlot = kDownRows * 256;              // bytes of a chunk

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// At most N of the wave's loads still in flight.  The builtin, not inline
// assembly: the compiler then knows that older loads into registers have
// landed and adds no wait for everything before their use.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    static_assert(N < 16, "the low bits of the counter's field");
    __builtin_amdgcn_s_waitcnt(N | 0x0F70);
    asm volatile("" ::: "memory");
}

template <int RT, bool TR>
__global__ __launch_bounds__(64 * kDownWaves) void k_lora_down(LoraDown p)
{
    constexpr int NW = kDownWaves, MI = kDownRows / 16, ND = kDownSlot / 1024;
    // two chunks a wave, later the waves' partial tiles
    __shared__ __align__(16) uint8_t lds[NW * 2 * kDownSlot];
    static_assert(NW * MI * RT * 1024 <= NW * 2 * kDownSlot, "partial tiles fit");
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)blockIdx.y * kDownRows;
    const int64_t M = p.m, K = p.k;
    const int R = p.rank;
    float* const t = p.t + (int64_t)blockIdx.x * M * R;
    const int slot = lane < kDownRows ? row_slot(p.slots, m0 + lane, M, p.adapters) : -1;

    if (blockIdx.z == 0) {                    // rows without an adapter
        for (int i = wave; i < kDownRows; i += NW)
            if (__builtin_amdgcn_readlane(slot, i) < 0 && m0 + i < M)
                for (int r = lane; r < R; r += 64) t[(m0 + i) * R + r] = 0.0f;
    }

    const int64_t kb = (int64_t)blockIdx.x * p.kstep, ke = kb + p.kstep < K ? kb + p.kstep : K;
    uint8_t* const ring = lds + wave * 2 * kDownSlot;
    // direct load q of a chunk: lane l brings piece (l % 16) ^ (row % 16) of row 4 q + l / 16
    const uint16_t* xr[ND];
    int xp[ND];
#pragma unroll
    for (int q = 0; q < ND; ++q) {
        const int r = 4 * q + (lane >> 4);
        xr[q] = p.x + (m0 + r < M ? m0 + r : M - 1) * p.ldx;
        xp[q] = 8 * ((lane & 15) ^ (r & 15));
    }
    auto bring = [&](int64_t k, int s) {
#pragma unroll
        for (int q = 0; q < ND; ++q) {
            const int64_t at = k + xp[q] < ke ? k + xp[q] : ke - 8;       // past the end: any element, zeroed below
            __builtin_amdgcn_global_load_lds(xr[q] + at, (lds_ptr_t)(ring + s * kDownSlot + 1024 * q), 16, 0, 0);
        }
    };
    int64_t ar[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) ar[j] = (int64_t)(16 * j + r16 < R ? 16 * j + r16 : R - 1) * (TR ? 1 : K);

    uint64_t todo = __builtin_amdgcn_ballot_w64(slot >= 0);
    for (unsigned nth = 0; todo; ++nth) {
        const int cur = __builtin_amdgcn_readlane(slot, __builtin_ctzll(todo));
        const uint64_t match = __builtin_amdgcn_ballot_w64(slot == cur);
        todo &= ~match;
        if (nth % gridDim.z != blockIdx.z) continue;
        const uint16_t* const a = p.a + (int64_t)cur * R * K;
        v4f acc[MI][RT];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        const int64_t k0 = kb + 128 * wave;
        if (k0 < ke) bring(k0, 0);
        int s = 0;
        for (int64_t k = k0; k < ke; k += 128 * NW, s ^= 1) {
            const v4i zero{0, 0, 0, 0};
            v4i af[4][RT];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t c = k + 32 * u + 8 * grp < ke ? k + 32 * u + 8 * grp : ke - 8;
#pragma unroll
                for (int j = 0; j < RT; ++j)
                    af[u][j] = TR ? gather8(a + c * R + ar[j], R) : *reinterpret_cast<const v4i*>(a + ar[j] + c);
            }
            // Every load is issued unconditionally (the last chunk is brought
            // again instead of one past the end), so that the number in flight
            // is known: this chunk, and A's fragments, are older than the ND
            // loads of the next one.
            bring(k + 128 * NW < ke ? k + 128 * NW : k, s ^ 1);
            wait_loads<ND>();
            const uint8_t* const at = ring + s * kDownSlot;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool in = k + 32 * u + 8 * grp < ke;     // 8 elements, all in or all out
                v4i xf[MI];
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    xf[i] = *reinterpret_cast<const v4i*>(at + 256 * (16 * i + r16) + 16 * ((4 * u + grp) ^ r16));
                    xf[i] = in ? xf[i] : zero;
                }
#pragma unroll
                for (int j = 0; j < RT; ++j) af[u][j] = in ? af[u][j] : zero;
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[i][j] = mfma16(af[u][j], xf[i], acc[i][j]);
            }
            // every read of this chunk has returned before its place is filled again
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        wait_loads<0>();
        __syncthreads();
        // acc[i][j][e] = T[m = 16 i + r16][r = 16 j + 4 grp + e]
        v4f* const red = reinterpret_cast<v4f*>(lds);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < RT; ++j) red[((wave * MI + i) * RT + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        const float sc = p.scale ? p.scale[cur] : 1.0f;
        for (int e = tid; e < MI * RT * 64; e += 64 * NW) {
            const int tile = e >> 6, l = e & 63, i = tile / RT, j = tile % RT;
            const int m = 16 * i + (l & 15), r = 16 * j + 4 * (l >> 4);
            if (((match >> m) & 1) && r < R) {
                const v4f v = (red[e] + red[MI * RT * 64 + e]) + (red[2 * MI * RT * 64 + e] + red[3 * MI * RT * 64 + e]);
                *reinterpret_cast<v4f*>(t + (m0 + m) * R + r) = v * sc;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// y = base + s_l T B_l^T: a wave owns 16 rows, holds their T as fragments of
// its terms and walks the columns 64 at a time.  Bound by memory, so the wave
// is kept small (many in flight) and base and y move in whole 128-byte lines:
// the products, which leave the matrix instructions as 4 columns of a row a
// lane, pass through the wave's own 4 KB of LDS and come back as 8 columns a
// lane, 8 lanes a row.  8192 x 4096, rank 16, 134 MB: 27 to 29 us, 4.6 to 5.0 TB/s,
// what the same loads and stores take without the products.
// The WM waves of a workgroup on neighbouring rows read the same part of B:
// from the cache up to rank 32; above, a step's columns of B outweigh those of
// y and come through LDS once for all four (SH; 1111 rows of nine requests,
// rank 64, 11008 columns: 20 to 22 us against 25).  Rows of another adapter than the
// one whose B is multiplied drop the result (a select, so that nothing of one
// adapter reaches another's rows).
// ---------------------------------------------------------------------------
// Four waves a SIMD up to rank 32, which the compiler would pass by four
// registers.
template <int WM, int RC, bool TR, bool SH>
__global__ __launch_bounds__(256, RC == 1 && !TR ? 4 : 1) void k_lora_up(LoraUp p)
{
    constexpr int WN = 4 / WM;                          // waves side by side along the columns
    constexpr int Pitch = 68;                           // floats: 17 times 16 bytes
    __shared__ __align__(16) float tile[4][16 * Pitch];
    static_assert(!SH || (WM == 4 && !TR && RC > 1), "neighbouring rows share B's fragments");
    __shared__ __align__(16) uint8_t bsh[SH ? 2 * 64 * 64 * RC : 16];
    const int lane = threadIdx.x & 63, r16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t M = p.m, N = p.n;
    const int R = p.rank;
    const int64_t m0 = ((int64_t)blockIdx.y * WM + wave % WM) * 16, m = m0 + r16;
    // SH: the adapters of the workgroup's 64 rows, the j-th in lane j, if they
    // are at most four (0 in `kinds`: more, or none)
    int kinds = 0, kind = -1;
    if constexpr (SH) {
        const int ws = row_slot(p.slots, (int64_t)blockIdx.y * 64 + lane, M, p.adapters);
        uint64_t todo = __builtin_amdgcn_ballot_w64(ws >= 0);
        for (; todo && kinds < 4; ++kinds) {
            const int cur = __builtin_amdgcn_readlane(ws, __builtin_ctzll(todo));
            kind = lane == kinds ? cur : kind;
            todo &= ~__builtin_amdgcn_ballot_w64(ws == cur);
        }
        if (todo) kinds = 0;
    }
    if (m0 >= M && kinds == 0) return;                  // no barrier below: waves are on their own
    const int64_t nb = (int64_t)blockIdx.x * p.ncols, ne = nb + p.ncols < N ? nb + p.ncols : N;
    const int slot = row_slot(p.slots, m, M, p.adapters);   // the same in the four lanes of a row
    float* const out = tile[wave];

    v4i tf[RC][kTerms];
    {
        v4f v[RC][2];
#pragma unroll
        for (int c = 0; c < RC; ++c) v[c][0] = v[c][1] = v4f{0.f, 0.f, 0.f, 0.f};
        if (m < M) {
            const float* t = p.t + m * R + 8 * grp;
#pragma unroll 4
            for (int s = 0; s < p.splits; ++s, t += M * R) {
#pragma unroll
                for (int c = 0; c < RC; ++c)
                    if (32 * c + 8 * grp < R) {
                        v[c][0] += *reinterpret_cast<const v4f*>(t + 32 * c);
                        v[c][1] += *reinterpret_cast<const v4f*>(t + 32 * c + 4);
                    }
            }
        }
#pragma unroll
        for (int c = 0; c < RC; ++c) {
            if (p.t_out && blockIdx.x == 0 && wave / WM == 0 && m < M && 32 * c + 8 * grp < R) {
                *reinterpret_cast<v4f*>(p.t_out + m * R + 32 * c + 8 * grp) = v[c][0];
                *reinterpret_cast<v4f*>(p.t_out + m * R + 32 * c + 8 * grp + 4) = v[c][1];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t x[kTerms];
                bf16_terms(v[c][q >> 1][2 * (q & 1)], v[c][q >> 1][2 * (q & 1) + 1], x);
#pragma unroll
                for (int i = 0; i < kTerms; ++i) tf[c][i][q] = (int)x[i];
            }
        }
    }
    const uint64_t used = __builtin_amdgcn_ballot_w64(slot >= 0);
    // this lane's part of y: rows i and i + 8, 8 columns; a row without an
    // adapter keeps base's bits (and is left alone in place)
    const int yr = lane >> 3, yc = 8 * (lane & 7);
    int has[2];
    bool live[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        has[u] = __shfl(slot, yr + 8 * u) >= 0;
        live[u] = m0 + yr + 8 * u < M && (has[u] || p.base != p.y);
    }
    const uint16_t* const base = p.base ? p.base + (m0 + yr) * p.ldbase + yc : nullptr;
    uint16_t* const y = p.y + (m0 + yr) * p.ldy + yc;
    v4i next[2];
    auto fetch = [&](int64_t n0) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            next[u] = base && live[u] && n0 + yc < ne ? *reinterpret_cast<const v4i*>(base + 8 * u * p.ldbase + n0)
                                                      : v4i{0, 0, 0, 0};
    };
    // B's fragments: tile (u, h) holds columns n0 + 32 u + 16 h + r16
    v4i bf[2][2][RC];
    auto load_b = [&](int cur, int64_t n0) {
        const uint16_t* const b = p.b + (int64_t)cur * N * R;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = n0 + 32 * u + 16 * h + r16, n = at < N ? at : N - 1;
#pragma unroll
                for (int c = 0; c < RC; ++c) {
                    const int r = 32 * c + 8 * grp;
                    bf[u][h][c] = r >= R ? v4i{0, 0, 0, 0}
                                  : TR   ? gather8(b + r * N + n, N)
                                         : *reinterpret_cast<const v4i*>(b + n * R + r);
                }
            }
    };
    auto multiply = [&](int cur, float s, v4f (&o)[2][2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4f acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < RC; ++c)
#pragma unroll
                    for (int i = kTerms - 1; i >= 0; --i) acc = mfma16(bf[u][h][c], tf[c][i], acc);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[u][h][e] = slot == cur ? acc[e] * s : o[u][h][e];
            }
    };
    auto finish = [&](int64_t n0, const v4i (&old)[2], const v4f (&o)[2][2]) {
        // o[u][h][e]: row r16, column 32 u + 16 h + 4 grp + e
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<v4f*>(out + Pitch * r16 + 32 * u + 16 * h + 4 * grp) = o[u][h];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const v4f d0 = *reinterpret_cast<const v4f*>(out + Pitch * (yr + 8 * u) + yc);
            const v4f d1 = *reinterpret_cast<const v4f*>(out + Pitch * (yr + 8 * u) + yc + 4);
            v4i v = old[u];
            if (has[u]) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t w = (uint32_t)old[u][q];
                    const v4f& d = q < 2 ? d0 : d1;
                    v[q] = (int)pack_bf16(bf16_lo(w) + d[2 * (q & 1)], bf16_hi(w) + d[2 * (q & 1) + 1]);
                }
            }
            if (live[u] && n0 + yc < ne) *reinterpret_cast<v4i*>(y + 8 * u * p.ldy + n0) = v;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    if constexpr (SH) {
        // An adapter's 64 columns of B lie in LDS once for the four waves,
        // brought ahead by direct loads (16-byte piece c of column n at c ^ (n
        // % pieces), the fragment reads' banks apart); two barriers each.
        if (kinds) {
            constexpr int P = 4 * RC, Buf = 64 * 64 * RC;
            auto bring = [&](int cur, int64_t n0, int k) {
                const uint16_t* const b = p.b + (int64_t)cur * N * R;
#pragma unroll
                for (int q = 0; q < RC; ++q) {
                    const int at = 64 * (wave * RC + q) + lane, row = at / P, piece = (at & (P - 1)) ^ (row & (P - 1));
                    const int64_t n = n0 + row < N ? n0 + row : N - 1;
                    __builtin_amdgcn_global_load_lds(b + n * R + (8 * piece < R ? 8 * piece : 0),
                                                     (lds_ptr_t)(bsh + k * Buf + 1024 * (wave * RC + q)), 16, 0, 0);
                }
            };
            auto meet = [] {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
            };
            bring(__builtin_amdgcn_readlane(kind, 0), nb, 0);
            fetch(nb);
            int k = 0;
            for (int64_t n0 = nb; n0 < ne; n0 += 64) {
                const v4i old[2]{next[0], next[1]};
                v4f o[2][2];
#pragma unroll
                for (int u = 0; u < 2; ++u) o[u][0] = o[u][1] = v4f{0.f, 0.f, 0.f, 0.f};
                for (int j = 0; j < kinds; ++j, k ^= 1) {
                    const int cur = __builtin_amdgcn_readlane(kind, j);
                    meet();                             // the other buffer has been read
                    if (j + 1 < kinds) bring(__builtin_amdgcn_readlane(kind, j + 1), n0, k ^ 1);
                    else bring(__builtin_amdgcn_readlane(kind, 0), n0 + 64 < ne ? n0 + 64 : n0, k ^ 1);
                    wait_loads<RC>();                   // this wave's part of B
                    meet();
                    if (!__builtin_amdgcn_ballot_w64(slot == cur)) continue;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int row = 32 * u + 16 * h + r16;
#pragma unroll
                            for (int c = 0; c < RC; ++c) {
                                bf[u][h][c] = *reinterpret_cast<const v4i*>(bsh + k * Buf + 64 * RC * row +
                                                                            16 * ((4 * c + grp) ^ (row & (P - 1))));
                                if (32 * c + 8 * grp >= R) bf[u][h][c] = v4i{0, 0, 0, 0};
                            }
                        }
                    multiply(cur, p.scale ? p.scale[cur] : 1.0f, o);
                }
                fetch(n0 + 64);
                finish(n0, old, o);
            }
            wait_loads<0>();                            // the last bring, before the LDS is given up
            return;
        }
    }
    // the tile's only adapter (-1: several, or none): its next columns of B
    // are loaded while these are written (larger ranks' fragments would cost
    // a wave of the SIMD's four: rank 64, 1111 rows, 32 us against 26)
    int one = used ? __builtin_amdgcn_readlane(slot, __builtin_ctzll(used)) : -1;
    if (RC > 1 || (used & ~__builtin_amdgcn_ballot_w64(slot == one))) one = -1;
    const float scale1 = one >= 0 && p.scale ? p.scale[one] : 1.0f;
    if (one >= 0) load_b(one, nb + 64 * (wave / WM));
    fetch(nb + 64 * (wave / WM));
    for (int64_t n0 = nb + 64 * (wave / WM); n0 < ne; n0 += 64 * WN) {
        v4i old[2]{next[0], next[1]};
        v4f o[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) o[u][0] = o[u][1] = v4f{0.f, 0.f, 0.f, 0.f};
        if (one >= 0) {
            multiply(one, scale1, o);
            load_b(one, n0 + 64 * WN);
        } else {
            for (uint64_t todo = used; todo;) {
                const int cur = __builtin_amdgcn_readlane(slot, __builtin_ctzll(todo));
                todo &= ~__builtin_amdgcn_ballot_w64(slot == cur);
                load_b(cur, n0);
                multiply(cur, p.scale ? p.scale[cur] : 1.0f, o);
            }
        }
        fetch(n0 + 64 * WN);
        finish(n0, old, o);
    }
}

// T as the sum of its K ranges' partial sums.
__global__ __launch_bounds__(256) void k_lora_sum(const float* parts, int splits, int64_t n, float* t)
{
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= n) return;
    v4f v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const v4f*>(parts + s * n + e);
    *reinterpret_cast<v4f*>(t + e) = v;
}

// ---------------------------------------------------------------------------
// A_l [R, K] -> [K, R] and B_l [N, R] -> [R, N], 64 x 64 tiles through LDS:
// the backward products contract over the other index of each.  gridDim.x are
// one adapter's tiles, gridDim.y the adapters: the tiles of a whole bank may
// pass the 2^32 threads that one dimension takes.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_lora_transpose(LoraTranspose p)
{
    __shared__ uint16_t tile[64][66];
    int64_t b = blockIdx.x;
    const int which = b >= p.blocks[0];
    if (which) b -= p.blocks[0];
    const int64_t rows = p.rows[which], cols = p.cols[which];
    const int64_t tc = (cols + 63) / 64, l = blockIdx.y;
    const int64_t r0 = b / tc * 64, c0 = b % tc * 64;
    const uint16_t* const src = p.src[which] + l * rows * cols;
    uint16_t* const dst = p.dst[which] + l * rows * cols;
    for (int e = threadIdx.x; e < 64 * 8; e += 256) {
        const int r = e >> 3, c = 8 * (e & 7);
        if (r0 + r < rows && c0 + c < cols) {          // cols % 8 == 0
            const v4i v = *reinterpret_cast<const v4i*>(src + (r0 + r) * cols + c0 + c);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                tile[r][c + 2 * q] = (uint16_t)v[q];
                tile[r][c + 2 * q + 1] = (uint16_t)((uint32_t)v[q] >> 16);
            }
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * 8; e += 256) {
        const int c = e >> 3, r = 8 * (e & 7);
        if (c0 + c < cols && r0 + r < rows) {          // rows % 8 == 0
            v4i v;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = (int)(tile[r + 2 * q][c] | ((uint32_t)tile[r + 2 * q + 1][c] << 16));
            *reinterpret_cast<v4i*>(dst + (c0 + c) * rows + r0 + r) = v;
        }
    }
}

// ---------------------------------------------------------------------------
// G_l[c, r] = sum over the rows of adapter l of D[row, c] P[row, r]: dA (D =
// x, P = dT) and dB (D = dy, P = s_l T) in one launch.  The sum runs down the
// rows, so a fragment is a column's 8 values: each lane reads 16 bytes of 8
// rows and transposes its own 8 x 8 block with byte permutes; matrix
// instruction ci then covers columns {8 i + ci}, and a lane ends with 32
// consecutive columns of one r.  Each wave takes every fourth chunk of 32
// rows, skips the chunks without a row of l and zeroes other adapters' rows
// in both operands (an infinity there must not meet a zero).  Row ranges
// (gridDim.z) leave partial sums, joined in a fixed order by k_lora_join.
// Bound by reading D (once, past the caches): 8192 x (4096 + 11008), rank 16,
// 247 MB: 48 us, 5.1 TB/s; 63 us through the caches and with a chunk's loads
// waiting for its rows' adapters.
// ---------------------------------------------------------------------------
template <int RT>
__global__ __launch_bounds__(256, RT == 1 ? 3 : RT == 2 ? 2 : 1) void k_lora_outer(LoraOuter p)
{
    __shared__ v4f red[8 * RT * 64];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, grp = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int which = (int)blockIdx.x >= p.tiles[0];
    const LoraOuterJob& job = p.job[which];
    const int R = p.rank, rgroups = (R + 16 * RT - 1) / (16 * RT);
    const int l = (int)blockIdx.y / rgroups, rg = (int)blockIdx.y % rgroups;
    const int64_t M = p.m, C = job.c;
    const int64_t c0 = (int64_t)(blockIdx.x - (which ? p.tiles[0] : 0)) * 128;
    const int64_t cl = c0 + 8 * r16 < C ? c0 + 8 * r16 : C - 8;       // this lane's 8 columns (C % 8 == 0)
    const int64_t mb = (int64_t)blockIdx.z * p.mstep, me = mb + p.mstep < M ? mb + p.mstep : M;

    v4f acc[8][RT];
#pragma unroll
    for (int ci = 0; ci < 8; ++ci)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[ci][j] = v4f{0.f, 0.f, 0.f, 0.f};
    // A chunk is loaded while the one before is multiplied, and its rows'
    // adapters while that one is loaded.
    v4i d[8];
    float pv[RT][8];
    int pcol[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int r = 16 * (rg * RT + t) + r16;
        pcol[t] = r < R ? r : R - 1;
    }
    auto load = [&](int64_t mc) {
        if (mc + 32 <= M) {
            const uint16_t* const row = job.d + (mc + 8 * grp) * job.ldd + cl;
            const float* const pr = job.p + (mc + 8 * grp) * R;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(row + j * job.ldd));
#pragma unroll
                for (int t = 0; t < RT; ++t) pv[t][j] = pr[j * R + pcol[t]];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t m = mc + 8 * grp + j < M ? mc + 8 * grp + j : M - 1;
                d[j] = *reinterpret_cast<const v4i*>(job.d + m * job.ldd + cl);
#pragma unroll
                for (int t = 0; t < RT; ++t) pv[t][j] = job.p[m * R + pcol[t]];
            }
        }
    };
    // a chunk's adapters, one row a lane, read here and looked at a chunk
    // later: waiting for them at once would wait for the rows as well
    auto slots_of = [&](int64_t mc) { return p.slots[mc + (lane & 31) < M ? mc + (lane & 31) : M - 1]; };
    auto rows_of = [&](int s, int64_t mc) {
        return (uint32_t)__builtin_amdgcn_ballot_w64(lane < 32 && s == l && mc + lane < me);
    };
    int any = 0;
    int64_t mc = mb + 32 * wave;
    uint32_t rows = 0;
    int ahead = -1;
    if (mc < me) {
        rows = rows_of(slots_of(mc), mc);
        if (rows) load(mc);
        ahead = slots_of(mc + 128);
    }
    for (; mc < me; mc += 128) {
        const uint32_t now = rows;
        v4i f[8];
        v4i pf[RT][kTerms];
        if (now) {
            any = 1;
            const uint32_t keep = (now >> (8 * grp)) & 0xFFu;
            if (now != 0xFFFFFFFFu) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool in = (keep >> j) & 1;
                    d[j] = in ? d[j] : v4i{0, 0, 0, 0};
#pragma unroll
                    for (int t = 0; t < RT; ++t) pv[t][j] = in ? pv[t][j] : 0.0f;
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t x[kTerms];
                    bf16_terms(pv[t][2 * q], pv[t][2 * q + 1], x);
#pragma unroll
                    for (int i = 0; i < kTerms; ++i) pf[t][i][q] = (int)x[i];
                }
#pragma unroll
            for (int ci = 0; ci < 8; ++ci)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    f[ci][q] = (int)__builtin_amdgcn_perm((uint32_t)d[2 * q + 1][ci >> 1], (uint32_t)d[2 * q][ci >> 1],
                                                          (ci & 1) ? 0x07060302u : 0x05040100u);
        }
        rows = rows_of(ahead, mc + 128);
        ahead = slots_of(mc + 256);
        if (rows) load(mc + 128);
        if (now) {
#pragma unroll
            for (int ci = 0; ci < 8; ++ci)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int i = kTerms - 1; i >= 0; --i) acc[ci][t] = mfma16(f[ci], pf[t][i], acc[ci][t]);
        }
    }
    any = __syncthreads_or(any);
    if (gridDim.z > 1) {
        if (blockIdx.x == 0 && rg == 0 && tid == 0) p.flags[(int64_t)blockIdx.z * p.adapters + l] = (uint32_t)any;
        if (!any) return;
    }
    // Each wave joins a quarter of the tiles (the 2 RT from 2 RT wave on, by t
    // first): in three turns every wave passes the quarter of the wave s
    // places on, and the sums are its own + 1, 2, 3 places before, in order.
    constexpr int Q = 2 * RT;
    v4f sum[Q];
#pragma unroll
    for (int w = 0; w < 4; ++w)
        if (wave == w) {
#pragma unroll
            for (int i = 0; i < Q; ++i) sum[i] = acc[(Q * w + i) % 8][(Q * w + i) / 8];
        }
#pragma unroll
    for (int s = 1; s < 4; ++s) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (wave == w) {
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int at = Q * ((w + s) & 3) + i;
                    red[(Q * w + i) * 64 + lane] = acc[at % 8][at / 8];
                }
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < Q; ++i) sum[i] += red[(Q * ((wave - s) & 3) + i) * 64 + lane];
        __syncthreads();
    }
    // tile at = 8 t + ci: sum[at][e] = G[c = c0 + 32 grp + 8 e + ci][r = 16 (rg RT + t) + r16]
    const float s = job.scale ? job.scale[l] : 1.0f;
    float* const part = gridDim.z > 1 ? job.part + (int64_t)blockIdx.z * p.adapters * R * C : nullptr;
    const int t0 = Q * wave / 8, ci0 = Q * wave % 8;       // a quarter is Q consecutive columns of one t (all 8 from rank 64 on)
    const int r = 16 * (rg * RT + t0) + r16;
    if (r >= R) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t c = c0 + 32 * grp + 8 * e + ci0;
        if (c >= C) continue;
        // dA [R, C]: consecutive elements; dB [C, R]: one of each row, 16 lanes side by side
        const int64_t at = (int64_t)l * R * C + (job.by_col ? c * R + r : (int64_t)r * C + c);
        const int64_t step = job.by_col ? R : 1;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const float v = sum[i][e] * s;
            if (part) part[at + i * step] = v;
            else if (p.out_bf16) reinterpret_cast<uint16_t*>(job.out)[at + i * step] = (uint16_t)f32_to_bf16_rne(v);
            else reinterpret_cast<float*>(job.out)[at + i * step] = v;
        }
    }
}

// Sum of the row ranges' partial gradients that hold anything, in order.
__global__ __launch_bounds__(256) void k_lora_join(LoraOuter p, int splits)
{
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const LoraOuterJob& job = p.job[which];
        const int64_t per = (int64_t)p.rank * job.c, total = per * p.adapters;
        for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < total; e += (int64_t)gridDim.x * 1024) {
            const int64_t l = e / per;
            v4f v{0.f, 0.f, 0.f, 0.f};
            for (int s = 0; s < splits; ++s)
                if (p.flags[(int64_t)s * p.adapters + l]) v += *reinterpret_cast<const v4f*>(job.part + s * total + e);
            if (p.out_bf16) {
                uint2 w;
                w.x = f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16);
                w.y = f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16);
                *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(job.out) + e) = w;
            } else {
                *reinterpret_cast<v4f*>(reinterpret_cast<float*>(job.out) + e) = v;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// launch shapes
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
static int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// K ranges: about two workgroups of four waves for a CU (or many small ones
// for a few rows), none with less than one chunk a wave, at most 32 partial
// sums for the reader to join; four for a CU where each still has four chunks
// a wave or more (8192 rows of 11008: 42 us against 48; of 4096, where it would
// not: 20 against 18).  Then the adapters of a tile side by side while that
// leaves the device unfilled.
LoraDownShape lora_down_shape(int64_t m, int64_t k, int rank, int64_t adapters)
{
    LoraDownShape s;
    s.few = m <= 16;
    const int64_t rows = s.few ? 16 : kDownRows, waves = s.few ? kFewWaves : kDownWaves;
    const int64_t tiles = cdiv(m, rows);
    s.splits = clamp64(512 / tiles, 1, clamp64(cdiv(k, 128 * waves), 1, 32));
    const int64_t deep = clamp64(1024 / tiles, 1, k / (4 * 128 * waves));
    if (!s.few && deep > s.splits) s.splits = deep < 32 ? deep : 32;
    s.kstep = cdiv(cdiv(k, s.splits), 128) * 128;
    s.splits = cdiv(k, s.kstep);
    int64_t most = m < rows ? m : rows;
    if (adapters < most) most = adapters;
    s.z = clamp64(1024 / (tiles * s.splits), 1, most);
    return s;
}

static int outer_rt(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }

// The row ranges of the gradient sums, at least 256 rows each (two chunks a
// wave).  A range's rows are mostly one adapter's, so about column tiles x
// ranges workgroups have work whatever the number of adapters: as many as run
// at once (three, two or one on a CU, by their registers), since a second,
// half-empty round costs as much as the first.  A range also costs a partial sum of
// every adapter's gradient: 256 MB of them at most.
int64_t lora_outer_splits(int64_t m, int64_t n, int64_t k, int rank, int64_t adapters)
{
    const int rt = outer_rt(rank);
    const int64_t tiles = (cdiv(n, 128) + cdiv(k, 128)) * cdiv(rank, 16 * rt);
    const int64_t fit = 256 * (rt == 1 ? 3 : rt == 2 ? 2 : 1) / tiles;
    const int64_t part = 4 * adapters * rank * (n + k);
    return clamp64(fit, 1, clamp64(m / 256, 1, clamp64((int64_t(256) << 20) / part, 1, 16)));
}

template <int RT, bool TR>
static hipError_t run_down(const LoraDown& p, const LoraDownShape& sh, hipStream_t s)
{
    const dim3 grid((unsigned)sh.splits, (unsigned)(sh.few ? 1 : cdiv(p.m, kDownRows)), (unsigned)sh.z);
    if constexpr (!TR || RT <= 4)             // the rule of lora_across
        if (sh.few) {
            hipLaunchKernelGGL((k_lora_down_few<RT, TR>), grid, dim3(64 * kFewWaves), 0, s, p);
            return hipGetLastError();
        }
    hipLaunchKernelGGL((k_lora_down<RT, TR>), grid, dim3(64 * kDownWaves), 0, s, p);
    return hipGetLastError();
}

template <bool TR>
static hipError_t down_by_rank(const LoraDown& p, const LoraDownShape& sh, hipStream_t s)
{
    if (p.rank <= 16) return run_down<1, TR>(p, sh, s);
    if (p.rank <= 32) return run_down<2, TR>(p, sh, s);
    if (p.rank <= 64) return run_down<4, TR>(p, sh, s);
    return run_down<8, TR>(p, sh, s);
}

hipError_t launch_lora_down(const LoraDown& in, const LoraDownShape& sh, hipStream_t s)
{
    LoraDown p = in;
    p.kstep = sh.kstep;
    return p.across ? down_by_rank<true>(p, sh, s) : down_by_rank<false>(p, sh, s);
}

// Columns of a workgroup: 512 when the row tiles alone fill the device (the
// rows' T is then read once for eight steps of a wave), fewer where they do
// not, but at least four for every element of a row of T.
template <int WM, int RC, bool TR, bool SH = false>
static hipError_t run_up(const LoraUp& in, hipStream_t s)
{
    LoraUp p = in;
    const int64_t step = 64 * (4 / WM), rows = cdiv(p.m, 16 * WM);
    const int64_t least = step > 4 * p.rank ? step : 4 * p.rank;
    int64_t blocks = clamp64(1024 / rows, cdiv(p.n, 512), cdiv(p.n, least));
    // two workgroups a CU come before that
    if (blocks * rows < 512) blocks = clamp64(cdiv(512, rows), blocks, cdiv(p.n, step));
    p.ncols = cdiv(cdiv(p.n, blocks), step) * step;
    // every column block reads its rows' T: past 16 MB of partial sums (from
    // the caches) a launch that joins them once costs less than the difference
    if (p.splits > 1 && 4 * p.m * p.rank * p.splits * cdiv(p.n, p.ncols) > (int64_t(16) << 20)) {
        const int64_t n = p.m * p.rank;
        hipLaunchKernelGGL(k_lora_sum, dim3((unsigned)cdiv(n, 1024)), dim3(256), 0, s, p.t, p.splits, n, p.t_out);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.t = p.t_out;
        p.splits = 1;
        p.t_out = nullptr;
    }
    const dim3 grid((unsigned)cdiv(p.n, p.ncols), (unsigned)rows);
    hipLaunchKernelGGL((k_lora_up<WM, RC, TR, SH>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int WM, bool TR>
static hipError_t up_by_rank(const LoraUp& p, hipStream_t s)
{
    constexpr bool SH = WM == 4 && !TR;
    if (p.rank <= 32) return run_up<WM, 1, TR>(p, s);
    if (p.rank <= 64) return run_up<WM, 2, TR, SH>(p, s);
    if constexpr (WM == 1 && TR) return hipErrorInvalidValue;     // not by lora_across
    else return run_up<WM, 4, TR, SH>(p, s);
}

hipError_t launch_lora_up(const LoraUp& p, hipStream_t s)
{
    if (p.m <= 16) return p.across ? up_by_rank<1, true>(p, s) : up_by_rank<1, false>(p, s);
    return p.across ? up_by_rank<4, true>(p, s) : up_by_rank<4, false>(p, s);
}

// A backward call reads B and A across their rows (eight loads for a fragment)
// instead of transposing them first, which saves a launch, while that work
// (rows times columns of dx) is small: 200 rows, 11008 x 4096: rank 16 28.4 us
// against 31.2, rank 128 72.6 against 78.0; 2048 rows, 1024 x 1024, rank 16:
// 25.8 against 30.2; but 1024 rows, 4096 x 11008, rank 16: 50.0 against 47.3, and
// 8192 rows, 1024 x 1024: 43.4 against 41.9.  Up to 16 rows, whose T is one
// launch of little work, ranks above 64 gather too much (16 rows, 520 x 1000,
// rank 80: 33.2 against 29.0).
bool lora_across(int64_t m, int64_t k, int64_t rank)
{
    return m * k <= (int64_t(1) << 22) && (m > 16 || rank <= 64);
}

hipError_t launch_lora_transpose(const uint16_t* a, uint16_t* at, const uint16_t* b, uint16_t* bt, int64_t adapters,
                                 int64_t rank, int64_t k, int64_t n, hipStream_t s)
{
    LoraTranspose p;
    p.src[0] = a; p.dst[0] = at; p.rows[0] = rank; p.cols[0] = k;
    p.src[1] = b; p.dst[1] = bt; p.rows[1] = n; p.cols[1] = rank;
    for (int i = 0; i < 2; ++i) p.blocks[i] = cdiv(p.rows[i], 64) * cdiv(p.cols[i], 64);
    const dim3 grid((unsigned)(p.blocks[0] + p.blocks[1]), (unsigned)adapters);
    hipLaunchKernelGGL(k_lora_transpose, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int RT>
static hipError_t run_outer(const LoraOuter& p, int64_t splits, hipStream_t s)
{
    const dim3 grid((unsigned)(p.tiles[0] + p.tiles[1]), (unsigned)(p.adapters * cdiv(p.rank, 16 * RT)), (unsigned)splits);
    hipLaunchKernelGGL((k_lora_outer<RT>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_lora_outer(const LoraOuter& in, int64_t splits, hipStream_t s)
{
    LoraOuter p = in;
    p.tiles[0] = (int32_t)cdiv(p.job[0].c, 128);
    p.tiles[1] = (int32_t)cdiv(p.job[1].c, 128);
    p.mstep = cdiv(cdiv(p.m, splits), 128) * 128;
    hipError_t e;
    const int rt = outer_rt(p.rank);
    if (rt == 1) e = run_outer<1>(p, splits, s);
    else if (rt == 2) e = run_outer<2>(p, splits, s);
    else e = run_outer<4>(p, splits, s);
    if (e != hipSuccess || splits == 1) return e;
    const int64_t most = p.adapters * p.rank * (p.job[0].c > p.job[1].c ? p.job[0].c : p.job[1].c);
    hipLaunchKernelGGL(k_lora_join, dim3((unsigned)clamp64(cdiv(most, 1024), 1, 2048)), dim3(256), 0, s, p, (int)splits);
    return hipGetLastError();
}

}  // namespace fp4
