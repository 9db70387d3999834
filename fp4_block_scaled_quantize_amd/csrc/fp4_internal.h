// fp4_internal.h -- host-side launcher interface between the C ABI (api.cpp)
// and the kernel translation units.  Launchers assume validated arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4 {

struct ScaleFmtHost {
    int32_t ebits, mbits, bias, maxcode;
    float smax;
    int32_t is_e8m0;
};

// Fill the parameters of a block-scale format (fp4_scale_fmt value).
bool scale_fmt_params(int32_t fmt, ScaleFmtHost* out);

// Device workspace of an amax state.
//  - partial/stored: the two-kernel refresh (tensors larger than the fused
//    path holds in registers) writes one partial maximum per workgroup of
//    the amax kernel; the quantize kernel of the same call reduces them and
//    stores the result in `stored`, which calls between refreshes read.
//  - slot: the single-pass refresh exchanges per-workgroup maxima through
//    `slot` (64-bit {epoch, max bits} words, one per 64-byte segment so that
//    stores of different workgroups never share a line) within one launch.
//    Every single-pass launch that exchanges runs the same grid and
//    publishes every slot (a grid of one writes none), so a workgroup's own
//    slot holds the previous exchanging launch's epoch, and that + 1 is
//    this launch's.
//  - fallbacks: number of workgroups that did not see every other
//    workgroup's maximum within the wait bound and read the whole tensor
//    themselves instead (the result is the same either way).
constexpr int kAmaxParts = 256;
constexpr int kXchgSlots = 256;
constexpr int kXchgStride = 8;          // 64-bit words between slots (64 bytes)
struct AmaxDev {
    float partial[kAmaxParts];
    float stored;
    uint32_t reserved;
    uint32_t fallbacks;
    uint32_t reserved2;
    uint32_t pad[60];
    uint64_t slot[kXchgSlots * kXchgStride];
};
static_assert(sizeof(AmaxDev) == 17664, "amax state layout");

struct QuantLaunch {
    const void* x;
    int32_t x_bf16;
    int64_t rows, cols, ld;
    uint8_t* q;
    uint8_t* scales;
    float* tensor_scale;       // out: {g, amax}
    AmaxDev* amax_src;         // null: no tensor scale (g = 1)
    int32_t refresh;           // compute this call's maximum (else read amax_src->stored)
    int32_t block;
    int32_t stochastic;
    uint64_t seed, offset;
    ScaleFmtHost fmt;
    int32_t rht;               // blockwise randomized Hadamard transform first
    uint32_t rht_signs;
    int32_t elem;              // element grid (fp4_element)
};

// Bound on a single-pass refresh's wait for the other workgroups' maxima, in
// ticks of the 100 MHz real-time counter (process-wide; 0.2 s by default).
extern uint64_t g_exchange_wait_ticks;

struct DequantLaunch {
    const uint8_t* q;
    const uint8_t* scales;
    const float* tensor_scale;
    int64_t rows, cols;
    int32_t block;
    ScaleFmtHost fmt;
    void* y;
    int32_t y_bf16;
    int64_t ld;
    int32_t rht;               // inverse blockwise Hadamard transform last
    uint32_t rht_signs;
    int32_t elem;              // element grid (fp4_element)
};

hipError_t launch_quantize(const QuantLaunch& p, hipStream_t s);
// The row-wise output of a two-orientation call.
struct RowOut {
    uint8_t* q;
    uint8_t* scales;
    float* tensor_scale;
};
// Column-wise: rows/cols describe the output (x^T); x is [cols, rows].  With
// `rows`, the row-wise quantization of x is written there too (one read).
hipError_t launch_quantize_t(const QuantLaunch& p, hipStream_t s, const RowOut* rows = nullptr);
hipError_t launch_dequantize(const DequantLaunch& p, hipStream_t s);

struct GemmLaunch {
    const uint8_t* qa; const uint8_t* sa; const float* ga;   // A [M, K]
    const uint8_t* qb; const uint8_t* sb; const float* gb;   // W [N, K]
    int64_t m, n, k;
    int32_t block;
    ScaleFmtHost fa, fb;
    uint16_t* c;
    int64_t ldc;
    int32_t elem;              // element grid of both operands (fp4_element)
};

// The exact dequantize path needs one 16-bit type (f16 or bf16) that holds
// every element * scale product of both operands exactly.
bool gemm_dq_supported(const ScaleFmtHost& fa, const ScaleFmtHost& fb, int elem);
hipError_t launch_gemm_mx(const GemmLaunch& p, hipStream_t s);
// E2M1 with E8M0 scales at block 16 on the scaled FP4 matrix instruction,
// when the stage shape fits.
bool gemm_mx16_supported(const GemmLaunch& p);
hipError_t launch_gemm_mx16(const GemmLaunch& p, hipStream_t s);
hipError_t launch_gemm_dq(const GemmLaunch& p, hipStream_t s);
// Small products on one wave per 32 x 32 output tile (no LDS): E2M1 with
// E8M0 or f16- / bf16-exact ExMy scales on both operands, MXFP8, INT8 with
// E4M3 scales; M * N at most g_gemm_small_outputs (E2M1 with E8M0: an
// eighth of it, the bf16 forms 1.5 times it; process-wide).
extern int64_t g_gemm_small_outputs;
bool gemm_small_supported(const GemmLaunch& p);
hipError_t launch_gemm_small(const GemmLaunch& p, hipStream_t s);

// T = x A^T of the rows' adapters as `splits` partial sums [M, rank], and the
// up projections B [adapters, N, rank].
struct WoAdapters {
    const float* t; int32_t splits; int32_t rank;
    const uint16_t* b; const float* scale; const int32_t* slots; int64_t adapters;
};

struct WoGemmLaunch {
    const uint16_t* x; int64_t ldx; int64_t m;
    const uint8_t* qw; const uint8_t* sw; const float* gw;
    int64_t n, k;
    int32_t block;
    ScaleFmtHost fw;
    uint16_t* y; int64_t ldy;
    int32_t elem;              // element grid of the weights (fp4_element)
    WoAdapters ad{};           // low-rank adapters added in the epilogue (none: t null)
};

hipError_t launch_wo_gemm(const WoGemmLaunch& p, hipStream_t s);
// C[rows, cols] (bf16, row stride ld) = 0: the product over an empty K.
hipError_t launch_fill_zero_bf16(uint16_t* c, int64_t ld, int64_t rows, int64_t cols, hipStream_t s);


// ---------------------------------------------------------------------------
// low-rank adapters (lora.hip)
// ---------------------------------------------------------------------------
struct LoraDown {
    const uint16_t* x; int64_t ldx; int64_t m, k;
    const uint16_t* a; int64_t adapters; int32_t rank;    // [adapters, rank, k]
    const int32_t* slots;
    const float* scale;        // null: 1
    float* t;                  // [splits, m, rank]
    int64_t kstep;
    int32_t across;            // a is [adapters, k, rank] instead
};
// At most 16 rows or tiles of more, K ranges of kstep, z adapters of a tile at once.
struct LoraDownShape { bool few; int64_t splits, kstep, z; };
LoraDownShape lora_down_shape(int64_t m, int64_t k, int rank, int64_t adapters);
hipError_t launch_lora_down(const LoraDown& p, const LoraDownShape& sh, hipStream_t s);

struct LoraUp {
    const float* t; int32_t splits; int64_t m, n;
    const uint16_t* b; int64_t adapters; int32_t rank;    // [adapters, n, rank]
    const int32_t* slots;
    const float* scale;        // null: 1
    const uint16_t* base; int64_t ldbase;                 // null: zero
    uint16_t* y; int64_t ldy;
    float* t_out;              // the joined T [m, rank], if not null
    int64_t ncols;             // columns of a workgroup
    int32_t across;            // b is [adapters, rank, n] instead
};
hipError_t launch_lora_up(const LoraUp& p, hipStream_t s);
bool lora_across(int64_t m, int64_t k, int64_t rank);

struct LoraTranspose {
    const uint16_t* src[2]; uint16_t* dst[2];
    int64_t rows[2], cols[2], blocks[2];                  // blocks: tiles of one adapter
};
hipError_t launch_lora_transpose(const uint16_t* a, uint16_t* at, const uint16_t* b, uint16_t* bt, int64_t adapters,
                                 int64_t rank, int64_t k, int64_t n, hipStream_t s);

struct LoraOuterJob {
    const uint16_t* d; int64_t ldd; int64_t c;            // [m, c]
    const float* p; const float* scale;                   // [m, rank]; scale null: 1
    void* out; int32_t by_col;                            // [adapters, rank, c], or by_col [adapters, c, rank]
    float* part;               // [splits] of out in binary32
};
struct LoraOuter {
    LoraOuterJob job[2];
    int32_t tiles[2];
    int64_t m, mstep;
    int32_t rank; int64_t adapters;
    const int32_t* slots;
    int32_t out_bf16;
    uint32_t* flags;           // [splits, adapters]: the partial sum exists
};
int64_t lora_outer_splits(int64_t m, int64_t n, int64_t k, int rank, int64_t adapters);
hipError_t launch_lora_outer(const LoraOuter& p, int64_t splits, hipStream_t s);

// ---------------------------------------------------------------------------
// token log probabilities (logprobs.hip)
// ---------------------------------------------------------------------------
constexpr int kLpMaxPieces = 32;      // at most a lane of the join for each
struct LogprobLaunch {
    const void* logits; int32_t bf16; int64_t ld, rows, vocab;
    const int64_t* tokens;     // null: no token given
    float inv_temperature; int32_t top;
    float* logprob; float* entropy; float* stats;         // stats [rows, 2] = {maximum, log of the sum}
    int32_t* top_ids; float* top_logprobs;                // [rows, top]
    uint64_t* part_keys;       // [rows, pieces, top]
    float* part_sums;          // [rows, pieces, 4]
    int64_t piece;
};
int64_t logprob_pieces(int64_t rows, int64_t vocab);
hipError_t launch_logprobs(const LogprobLaunch& p, int64_t pieces, hipStream_t s);

struct LogprobGradLaunch {
    const void* logits; int32_t bf16; int64_t ld, rows, vocab;
    const int64_t* tokens;
    float inv_temperature;
    const float* entropy; const float* stats;
    const float* g_logprob; const float* g_entropy;       // null: zero
    void* dlogits; int64_t ldd;
    int64_t piece;
};
hipError_t launch_logprobs_backward(const LogprobGradLaunch& p, hipStream_t s);

// ---------------------------------------------------------------------------
// residual norms (norm.hip)
// ---------------------------------------------------------------------------
struct NormLaunch {
    const void* x; int64_t ldx; const void* res; int64_t ldres;
    int32_t x_bf16, res_bf16, w_bf16;
    int64_t rows, cols;
    const void* w_pre; const void* w_post;                // w_post null: no post norm
    const float* gate;                                    // [rows], null: 1
    float alpha, eps;
    void* h; int64_t ldh; void* n; int64_t ldn;
    float* stats;                                         // [rows, 2] = {rho(x), rho(h)}
};
struct NormGradLaunch {
    NormLaunch f;
    const void* dn; int64_t lddn; const void* dh; int64_t lddh;   // null: zero
    void* dx; int64_t lddx; void* dres; int64_t lddres;
    float* dw_pre; float* dw_post; float* dgate;
    float* part; int64_t part_rows, groups;               // [groups, part_rows, cols]
    int32_t sums;              // 1: w_pre's sums and every other output, 2: w_post's sums, 3: all
};
int64_t norm_groups(int64_t rows, int64_t cols);
hipError_t launch_norm(const NormLaunch& p, bool vec, hipStream_t s);
hipError_t launch_norm_backward(const NormGradLaunch& p, bool vec, hipStream_t s);

}  // namespace fp4
