/*
 * fp4.h -- C ABI of the MI355X (gfx950) block-scaled FP4 library.
 *
 * The method (page citations; the pages print no formula, the reading taken
 * where they are silent is stated at each call):
 *   quant_prune_distill/486 "Метод": NVFP4 = E2M1 elements in groups of 16
 *     with an E4M3 scale (4.5 bit/param); MXFP = groups of 32 with an E8M0
 *     (power-of-two) scale (4.25 bit/param); small groups need efficient
 *     kernels for the scale handling.
 *   gonzo_ML/3986 "Форматы FP4": group 16; scale encodings swept from E1M6
 *     to E8M0.  "Стохастическая квантизация": round to nearest, or up/down
 *     with probability set by the distance; nearest for forward weights and
 *     activations, stochastic for backward gradients.
 *   ue5m3-fp4-pretraining "Что сделали": unsigned UE5M3 block scales; the
 *     tensor maximum is refreshed every 50 steps, stored in between; all
 *     suitable linear layers run in FP4.
 *   quant_prune_distill/574 "Эксперименты": weight-only NVFP4 with a
 *     memory-bound small-batch kernel for rollouts.
 *
 * Conventions for every call:
 *   - Data pointers are DEVICE pointers owned by the caller (e.g. torch
 *     tensors).  The library never allocates or frees caller memory and
 *     allocates nothing per call; an fp4_amax_state owns 17664 bytes of
 *     device memory allocated at creation.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Every launch is asynchronous on it; no call synchronizes the host
 *     except fp4_amax_state_get / fp4_amax_state_set.
 *   - Arguments are validated before any launch.  A negative status means
 *     nothing was launched and nothing was written.  FP4_ERR_HIP means a
 *     launch was attempted and the runtime reported an error.
 *   - No exceptions cross the ABI.
 *   - Element codes: row-major [rows, cols/2] bytes, the even-index element
 *     in the low nibble; nibble = sign << 3 | E2M1 magnitude code.  Scales:
 *     row-major [rows, cols/block] bytes.  (Reading: the pages fix the
 *     storage cost, not the layout.)
 */
#ifndef FP4_H
#define FP4_H

#include <stdint.h>

#if defined(__GNUC__)
#define FP4_API __attribute__((visibility("default")))
#else
#define FP4_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fp4_status {
    FP4_OK = 0,
    FP4_ERR_INVALID_ARG = -1, /* null pointer, bad enum, bad block size     */
    FP4_ERR_UNSUPPORTED = -2, /* valid but unsupported combination          */
    FP4_ERR_SHAPE = -3,       /* cols % block != 0, K mismatch, ld < cols   */
    FP4_ERR_ALIGN = -4,       /* pointer or leading dimension misaligned    */
    FP4_ERR_HIP = -5          /* the HIP runtime reported an error          */
} fp4_status;

/* Block-scale encodings.  ExMy (sign + x exponent + y mantissa bits, x+y=7)
 * and UE5M3 (no sign bit): bias 2^(x-1)-1, exponent field 0 is subnormal,
 * no infinity, the code with every exponent and mantissa bit set is NaN
 * (reading; the pages name the formats only).  E8M0: value 2^(code-127). */
typedef enum fp4_scale_fmt {
    FP4_SCALE_E4M3 = 0,
    FP4_SCALE_UE5M3 = 1,
    FP4_SCALE_E3M4 = 2,
    FP4_SCALE_E1M6 = 3,
    FP4_SCALE_E8M0 = 4,
    FP4_SCALE_E2M5 = 5,
    FP4_SCALE_E5M2 = 6,
    FP4_SCALE_E6M1 = 7,
    FP4_SCALE_E7M0 = 8
} fp4_scale_fmt;

typedef enum fp4_rounding {
    FP4_ROUND_NEAREST_EVEN = 0, /* ties to the even code, saturate at 6      */
    FP4_ROUND_STOCHASTIC = 1    /* Philox4x32-10, 16 random bits per element */
} fp4_rounding;

typedef enum fp4_amax_policy {
    FP4_AMAX_NONE = 0,    /* no tensor scale (g = 1); required for E8M0      */
    FP4_AMAX_CURRENT = 1, /* g from max|x| of this call's tensor             */
    FP4_AMAX_DELAYED = 2  /* g from the stored max, refreshed every interval */
} fp4_amax_policy;

typedef enum fp4_dtype { FP4_DTYPE_F32 = 0, FP4_DTYPE_BF16 = 1 } fp4_dtype;

/* Transform applied to every block before quantization
 * (ue5m3-fp4-pretraining "Что сделали": a randomized Hadamard transform
 * spreads outliers over the block before quantization, and that scheme
 * leaves it out; quant_prune_distill/574 "Метод": Hadamard rotations bring
 * weights and activations closer to Gaussian).  The pages give no formula;
 * reading, for every block v of `block` consecutive elements along the
 * blocked dimension:
 *   y = c * H * D * v,  D = diag(-1 where bit j of transform_signs is set,
 *   else +1),  H the Sylvester Hadamard matrix ((H)_ij = (-1)^popcount(i&j)),
 *   c = 1/sqrt(block) rounded to binary32 (exactly 1/4 for block 16),
 * in binary32: H by butterfly stages h = 1, 2, 4, ... (each pair (i, i+h)
 * becomes (a + b, a - b)), then the product by c.  Block maxima, the tensor
 * maximum and the codes all see y.  Dequantization applies the inverse
 * v = D * (c * (H * y)) to the binary32 dequantized values.  H D / sqrt(B) is
 * orthogonal, so fp4_gemm of two operands transformed with the same
 * block and signs along K computes the same product. */
typedef enum fp4_transform {
    FP4_TRANSFORM_NONE = 0,
    FP4_TRANSFORM_RHT = 1      /* blockwise randomized Hadamard transform     */
} fp4_transform;

/* Element grid (quant_prune_distill/574 "Метод": the NV and MX block/scale
 * schemes paired with an FP or an INT element grid).  Reading for INT4: the
 * symmetric grid -7..7 as a two's-complement nibble (zero has no sign; the
 * code 0x8 is never produced); every rule that maps a maximum to the E2M1
 * maximum 6 maps it to 7 instead (g = amax_t / (7 Smax), u = amax_b /
 * RN(7 g)); the E8M0 exponent rule is unchanged (amax_b / s in [4, 8), the
 * MX convention for a sign + 3-bit fixed-point element); nearest rounding
 * ties to the even integer and saturates at 7; stochastic rounding as for
 * E2M1 with grid spacing 1.
 * The 8-bit grids (the same page's MXFP8 / MXINT8) store one byte per
 * element, codes [rows, cols] (reading): FP8 E4M3 elements, nearest-even
 * and saturating at 448, the sign bit kept (also for zero); INT8 on the
 * symmetric grid -127..127 (two's complement, zero unsigned).  448 or 127
 * takes the place of 6 in the tensor and block scales; the E8M0 rule uses
 * floor(log2 amax_b) - 8 (FP8) or - 6 (INT8) + 127, the OCP MX offsets.
 * Every call takes them.
 * The 6-bit grids (the same page's MXFP6 / MXINT6; reading: the OCP FP6
 * element formats E2M3 and E3M2, and INT6 on -31..31) pack six bits per
 * element as a little-endian bit stream: element c of a row at bits
 * 6c .. 6c + 5 of the row's cols*3/4 bytes.  FP6 E2M3: bias 1, largest 7.5;
 * E3M2: bias 3, largest 28; sign bit 5, subnormals, no reserved codes;
 * nearest-even, saturating.  INT6: six-bit two's complement, zero unsigned.
 * 7.5, 28 or 31 takes the place of 6; the E8M0 offsets are 2, 4 and 4.
 * Every call takes them (the column-wise and two-orientation calls with
 * R % 64 == 0, SHAPE otherwise). */
typedef enum fp4_element {
    FP4_ELEM_E2M1 = 0,
    FP4_ELEM_INT4 = 1,
    FP4_ELEM_FP8_E4M3 = 2,    /* MXFP8-style, one byte per element           */
    FP4_ELEM_INT8 = 3,        /* MXINT8-style, one byte per element          */
    FP4_ELEM_FP6_E2M3 = 4,    /* MXFP6-style, six bits per element           */
    FP4_ELEM_FP6_E3M2 = 5,    /* MXFP6-style, six bits per element           */
    FP4_ELEM_INT6 = 6         /* MXINT6-style, six bits per element          */
} fp4_element;

typedef struct fp4_format {
    int32_t block;            /* 16 or 32 elements per scale                  */
    int32_t scale;            /* fp4_scale_fmt                                */
    int32_t rounding;         /* fp4_rounding                                 */
    int32_t amax;             /* fp4_amax_policy                              */
    int32_t transform;        /* fp4_transform                                */
    uint32_t transform_signs; /* RHT: bit j negates element j of each block   */
    int32_t element;          /* fp4_element                                  */
} fp4_format;

/* A quantized tensor.  q: rows*cols/2 bytes (4-bit grids), rows*cols
 * bytes (8-bit grids) or rows*cols*3/4 bytes (6-bit grids); scales:
 * rows*cols/block bytes; tensor_scale: 2 floats {g, amax used} (g = 1 and
 * amax = 0 under NONE).  All three are device pointers; q must be 4-byte
 * aligned (8-byte for the 8- and 6-bit grids). */
typedef struct fp4_tensor {
    uint8_t* q;
    uint8_t* scales;
    float* tensor_scale;
    int64_t rows;
    int64_t cols;
    fp4_format fmt;
} fp4_tensor;

/* Per-tensor amax state (ue5m3-fp4-pretraining "Что сделали": the maximum
 * is refreshed every `interval` steps and the stored value used between).
 * Required by CURRENT (which refreshes on every call) and DELAYED.  Owns 17664
 * bytes of device memory on the device current at creation: the stored
 * amax, the per-workgroup partial maxima of the refresh and the exchange
 * words of the single-pass refresh.  Not thread-safe; calls that use one
 * state must be ordered (one stream, or synchronized). */
typedef struct fp4_amax_state fp4_amax_state;

/* interval >= 1.  Allocates the device workspace (zeroed, synchronously). */
FP4_API fp4_status fp4_amax_state_create(uint32_t interval, fp4_amax_state** out);
FP4_API fp4_status fp4_amax_state_destroy(fp4_amax_state* state);
/* Checkpoint: number of quantize calls seen and the stored amax.  Waits for
 * the device to finish outstanding work. */
FP4_API fp4_status fp4_amax_state_get(const fp4_amax_state* state, uint64_t* calls, float* amax);
/* Resume: overwrite the call count and stored amax (synchronous copy; also
 * clears the exchange words and the fallback count). */
FP4_API fp4_status fp4_amax_state_set(fp4_amax_state* state, uint64_t calls, float amax);

/* Single-pass refresh diagnostics.  In a single-pass refresh (see
 * fp4_quantize) the workgroups exchange their maxima through the state and
 * each waits a bounded time for all the others; a workgroup that gives up
 * (other work on the device kept some from being scheduled) reads the whole
 * tensor to take its maximum itself.  That maximum is the same value, so
 * codes, scales and tensor scale never depend on it; only the time does.
 * fp4_amax_state_fallbacks: the number of workgroups that took this path on
 * this state since its creation or last fp4_amax_state_set (waits for the
 * device).  fp4_set_exchange_wait: the process-wide wait bound in ticks of
 * the device's 100 MHz real-time counter (default 20000000, 0.2 s; 0 gives
 * up after one look at the other workgroups' words), for tests of the
 * fallback; the previous bound is returned in *previous if not null. */
FP4_API fp4_status fp4_amax_state_fallbacks(const fp4_amax_state* state, uint32_t* n);
FP4_API fp4_status fp4_set_exchange_wait(uint64_t ticks, uint64_t* previous);

/*
 * fp4_quantize -- quantize x[rows, cols] (row stride ld_x elements, f32 or
 * bf16) into out->q / out->scales / out->tensor_scale with out->fmt.
 * Pages: gonzo_ML/3986 "Форматы FP4" (E2M1 values, groups of 16, the swept
 * scale encodings) and "Стохастическая квантизация" (nearest rounding,
 * stochastic rounding for gradients); quant_prune_distill/486 "Метод" (NVFP4:
 * group 16 with an E4M3 scale under a tensor scale; MXFP4: group 32 with an
 * E8M0 scale); ue5m3-fp4-pretraining "Что сделали" (UE5M3 scales, the tensor
 * maximum refreshed every 50 steps).
 *
 * Per block of B elements (reading of the pages' "shared scale per small
 * group"; every step binary32 round-to-nearest-even):
 *   ExMy: g = amax_t / (6 * Smax) (g = 1 under NONE, or if the quotient is
 *         0 or not finite); u = RN(amax_b / RN(6 g)); code = nearest-even
 *         saturating ExMy encode of u; s = decode(code).
 *   E8M0: code = clamp(floor(log2 amax_b) - 2 + 127, 0, 254) (0 for an
 *         all-zero block); s = 2^(code-127); g = 1.
 *   S = RN(s g); inv = RN(1/S) clamped to FLT_MAX (inv = 0 when S = 0);
 *   v = RN(x inv); magnitude = nearest-even E2M1 code of |v| saturated at 6,
 *   or, for FP4_ROUND_STOCHASTIC, lo + [r16 / 2^16 < (|v|-lo)/(hi-lo)] with
 *   r16 the 16-bit half (i & 1) of word (i >> 1) & 3 of
 *   Philox4x32-10(key = seed, counter = {i >> 3 as 64 bits, offset as 64
 *   bits}), i = row * cols + col the logical element index.
 *
 * x: device, 16-byte aligned; ld_x * sizeof(elem) a multiple of 16; ld_x >=
 * cols.  cols % block == 0; block in {16, 32}; rows * cols / 8 < 2^31.  For an
 * empty tensor (rows or cols 0) x, q and scales may be null; tensor_scale
 * is still written ({1, 0} under CURRENT).
 * state: required for CURRENT and DELAYED (ignored for NONE).  CURRENT
 * recomputes amax_t on every call; DELAYED recomputes it when
 * state->calls % interval == 0 and otherwise reuses the stored value (a
 * tensor that outgrew it saturates at +-6).  Each call increments the
 * state's call count on the host (no device synchronization).  A refresh
 * reads x once when the tensor fits one workgroup per compute unit at 8192
 * units of 8 elements each (4096 x 4096 on a 256-CU device; the
 * workgroups agree on amax_t through the state), else twice (an amax pass,
 * then the quantize pass).
 * seed, offset: used only for FP4_ROUND_STOCHASTIC.
 * out->fmt.transform = FP4_TRANSFORM_RHT transforms every block first (see
 * fp4_transform); the tensor maximum is then that of the transformed tensor.
 * Errors: INVALID_ARG (null pointers, bad enums, missing state), SHAPE,
 * ALIGN, UNSUPPORTED (E8M0 with a tensor-scale policy).
 */
FP4_API fp4_status fp4_quantize(const void* x, int32_t x_dtype, int64_t ld_x, fp4_tensor* out,
                        fp4_amax_state* state, uint64_t seed, uint64_t offset, void* stream);

/*
 * fp4_quantize_noalloc -- for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): fp4_quantize with the policies NONE and CURRENT, the same
 * result bit for bit, but the current-amax workspace (17664 bytes) comes
 * from a static device array of the library, one per device, held until
 * the process ends, instead of an fp4_amax_state.  The workspace does not
 * grow with the tensor, so no size is refused on its account (fp4_quantize's
 * own limits apply).  The caller passes x and out as for fp4_quantize;
 * nothing is allocated or freed, on any call.  The first call on a device
 * looks up that device's array address (with the device current).
 * Every call on a device shares that one array: calls that overlap on one
 * device (different streams, or threads without ordering) race and must be
 * ordered by the caller.  Errors as fp4_quantize; UNSUPPORTED for DELAYED
 * (the stored maximum belongs to one tensor and needs an fp4_amax_state).
 */
FP4_API fp4_status fp4_quantize_noalloc(const void* x, int32_t x_dtype, int64_t ld_x, fp4_tensor* out,
                                        uint64_t seed, uint64_t offset, void* stream);

/*
 * fp4_quantize_transposed -- column-wise quantization for the backward
 * pass: out describes x^T, where x is [out->cols, out->rows] (row stride
 * ld_x elements, f32 or bf16), so each block holds `block` consecutive rows
 * of one column of x.  The result is, bit for bit, fp4_quantize applied to
 * the materialized transpose of x: same scale, rounding and amax rules,
 * and the stochastic-rounding index is that of x^T (i = c * out->cols + r
 * for element x[r, c]).  (gonzo_ML/3986 "Стохастическая квантизация":
 * stochastic rounding for the backward gradients; ue5m3-fp4-pretraining
 * "Что сделали": every suitable linear layer in FP4, which needs the
 * weight-gradient operands blocked along the token dimension.  Reading:
 * the pages give no layout for them; the transpose's row-major layout is
 * the [N, K] operand fp4_gemm consumes.)
 * x: device, 16-byte aligned, ld_x * sizeof(elem) a multiple of 16, ld_x >=
 * out->rows; out->rows % 8 == 0; out->cols % block == 0; out->q 16-byte
 * aligned.  A refresh of the tensor maximum reads x twice (an amax pass,
 * then the quantize pass).  With out->fmt.transform = FP4_TRANSFORM_RHT the
 * transform runs down the columns of x (over each block of x^T), and a
 * refresh takes the maximum of the transformed tensor.  Errors as
 * fp4_quantize.
 */
FP4_API fp4_status fp4_quantize_transposed(const void* x, int32_t x_dtype, int64_t ld_x, fp4_tensor* out,
                                   fp4_amax_state* state, uint64_t seed, uint64_t offset, void* stream);

/*
 * fp4_quantize_both -- both orientations of x [R, C] from one read: rowwise
 * [R, C] receives exactly what fp4_quantize(x) writes, colwise [C, R]
 * exactly what fp4_quantize_transposed(x) writes, and both get the same
 * tensor scale (gonzo_ML/3986 "Стохастическая квантизация" and
 * ue5m3-fp4-pretraining "Что сделали": the backward pass quantizes the
 * same gradient and activation tensors along both dimensions, one for each
 * of its two products).  Both tensors must carry the same block size, scale
 * encoding, rounding, amax policy and element grid, and no transform
 * (UNSUPPORTED otherwise: a transform along each axis would give the two
 * outputs different maxima).  The amax state counts the pair as one call.
 * Requirements as for the two calls together: R % block == 0, C % block ==
 * 0 (R % 64 == 0 for the 6-bit grids), x 16-byte aligned with ld_x *
 * sizeof(elem) a multiple of 16, colwise->q 16-byte aligned.  A refresh of the tensor maximum reads x twice (an amax
 * pass, then this one); otherwise x is read once.
 */
FP4_API fp4_status fp4_quantize_both(const void* x, int32_t x_dtype, int64_t ld_x, fp4_tensor* rowwise,
                                     fp4_tensor* colwise, fp4_amax_state* state, uint64_t seed, uint64_t offset,
                                     void* stream);

/*
 * fp4_dequantize -- y[rows, cols] (row stride ld_y, f32 or bf16) =
 * RN(RN(e2m1(code) * s) * g), rounded once more to bf16 (RNE) for bf16
 * output (quant_prune_distill/486 "Метод": the element times its group's
 * scale).  With in->fmt.transform = FP4_TRANSFORM_RHT the inverse transform
 * is applied to the binary32 values before any bf16 rounding.
 * in->tensor_scale[0] is read on the device.  y: 16-byte aligned,
 * ld_y * sizeof(elem) a multiple of 16.
 */
FP4_API fp4_status fp4_dequantize(const fp4_tensor* in, void* y, int32_t y_dtype, int64_t ld_y, void* stream);

/*
 * fp4_gemm -- C[M, N] (bf16, row stride ldc) = bf16_RNE(ga * gb *
 * sum_k (e2m1(a_mk) s_a)(e2m1(b_nk) s_b)) with fp32 accumulation, for
 * A = a [M, K] and W = b [N, K] both blocked along K (C = A W^T)
 * (ue5m3-fp4-pretraining "Что сделали": the linear layers run in FP4;
 * quant_prune_distill/574 "Выводы": weight + activation FP4 for the
 * compute-bound regime).  Both operands must use the same block size, the
 * same element grid and the same transform (kind and signs; UNSUPPORTED
 * otherwise).  Every element times its block scale enters a matrix
 * instruction exactly, in a 16-bit type chosen per pairing: INT4 in bf16
 * when int * s fits it exactly for both scale formats, else f16; FP8 E4M3
 * elements in bf16 for scale formats with at most 3 mantissa bits (E8M0,
 * E7M0, E6M1, E5M2, E4M3, UE5M3); INT8 in bf16 for power-of-two scales
 * (E8M0, E7M0) and in f16 for E4M3 scales; FP6 E2M3 as FP8, FP6 E3M2 in
 * bf16 for scales with at most 4 mantissa bits, INT6 in bf16 for at most 2
 * (E8M0, E7M0, E6M1, E5M2) and in f16 for E4M3 / E3M4 / E2M5; other 8- and
 * 6-bit pairings return UNSUPPORTED.
 * Paths: E2M1 with E8M0 scales on both operands runs on the gfx950
 * block-scaled FP4 matrix instruction (at block 16 when K % 256 == 0 and
 * each operand's codes are below 4 GiB; else in LDS); E2M1 with the formats
 * exact in f16 (E4M3, E3M4, E2M5, E1M6) or in bf16 (UE5M3, E5M2, E6M1,
 * E7M0), MXFP8 (FP8 with E8M0 on both) and INT8 with E4M3 on both are
 * converted to f16 / bf16 in registers; every other pairing is dequantized
 * to bf16 / f16 in LDS.  Small products of E2M1 with f16-exact ExMy scales
 * on both operands, of MXFP8 and of INT8 with E4M3 scales (M * N at most
 * the bound of fp4_set_gemm_small_outputs, 2^21 by default), of E2M1 with
 * bf16-exact ExMy scales (1.5 times the bound) or with E8M0 scales (an
 * eighth of it) run one wave per 32 x 32 output tile with the same
 * conversions and instructions and no LDS.  Result within 1e-5 * sum_k
 * |a||b| of the exact product before the bf16 rounding.
 * K % 128 == 0 (K = 0 writes C = 0 and reads no operand), M and N
 * arbitrary; ldc >= N; c 2-byte aligned (rows that
 * are 8-byte aligned are written with vector stores); operand codes 16-byte
 * and scales 4-byte aligned.
 */
FP4_API fp4_status fp4_gemm(const fp4_tensor* a, const fp4_tensor* b, uint16_t* c, int64_t ldc, void* stream);

/*
 * fp4_set_gemm_small_outputs -- the process-wide bound on M * N (output
 * elements) up to which fp4_gemm takes the small-product path for the
 * pairings it covers (above; E2M1 with E8M0 an eighth of it, E2M1 with the
 * bf16-exact ExMy pairings 1.5 times it).  0 turns the
 * path off, so that tests can run the tiled kernels on small shapes.
 * Results on either path meet the same error bound.  The previous value is
 * returned in *previous if not null; a negative bound is
 * FP4_ERR_INVALID_ARG.
 */
FP4_API fp4_status fp4_set_gemm_small_outputs(int64_t outputs, int64_t* previous);

/*
 * fp4_wo_gemm -- Y[M, N] (bf16, row stride ldy) = bf16_RNE(gw *
 * sum_k x[m, k] (e2m1(w_nk) s_w)), fp32 accumulation, weights dequantized
 * in registers (quant_prune_distill/574 "Метод"/"Эксперименты":
 * weight-only NVFP4, memory-bound small-batch generation).
 * x: bf16 [M, K] (row stride ldx), w: [N, K] quantized along K.
 * 1 <= M <= 16; K % 256 == 0 (K = 0 writes Y = 0 and reads neither x nor w);
 * x 16-byte aligned, ldx % 8 == 0, ldy >= N;
 * w's codes 16-byte and scales 4-byte aligned; w's codes < 4 GiB and no
 * transform on w (UNSUPPORTED otherwise).  Every element grid: E2M1, INT4
 * and the 8- and 6-bit ones (quant_prune_distill/486 "Метод": the MX
 * family's 8- and 6-bit members); each product e(w_nk) s_w enters the bf16
 * matrix instruction exactly, as one bf16 value or as the sum of two (an
 * infinity in x meets both, and where the second is zero that leaves NaN).
 */
FP4_API fp4_status fp4_wo_gemm(const uint16_t* x, int64_t ldx, int64_t m, const fp4_tensor* w, uint16_t* y,
                       int64_t ldy, void* stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection
 * (quant_prune_distill/574 "Метод": a trained low-rank adapter in parallel
 * with the NVFP4 weight; the page gives no formula).  Row i of a batch uses
 * adapter l = slots[i]; a value outside 0 .. adapters - 1 (-1 by convention)
 * gives the row none.  Reading:
 *   T = x A_l^T,  y = base + s_l T B_l^T
 * with T, and every sum, in binary32.  Rows of one adapter need not be
 * adjacent; a batch that keeps each request's rows together is read fewest
 * times.  Nothing of one adapter or row reaches another row's results
 * (infinities and NaN included).  Rows without an adapter keep base.  An
 * infinity in dy, x, A or B makes what it enters infinite or NaN: T and dT meet
 * it as a sum of three terms, which may leave NaN where their sum would leave
 * an infinity.
 *
 * A bank: a [adapters, rank, k] and b [adapters, n, rank] in bf16, dense and
 * 16-byte aligned; scale [adapters] in binary32.  rank % 8 == 0 and at most
 * 128 (a smaller rank is padded with zeros), k % 8 == 0, n % 8 == 0 (any n
 * for fp4_wo_gemm_lora), at most 16384 adapters.
 *
 * `workspace`: device memory, 16-byte aligned, of at least
 * fp4_lora_workspace bytes (it may be null when that is 0), in use until the
 * call's work on the stream has finished.  At most 2^20 rows a call. */
typedef struct fp4_lora_bank {
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    int64_t adapters, rank, k, n;
} fp4_lora_bank;

typedef enum fp4_lora_call {
    FP4_LORA_APPLY = 0,
    FP4_LORA_BACKWARD = 1,
    FP4_LORA_WO_GEMM = 2
} fp4_lora_call;

/* Bytes of workspace that a call on m rows needs (negative: a status). */
FP4_API int64_t fp4_lora_workspace(int32_t call, int64_t m, int64_t n, int64_t k, int64_t rank, int64_t adapters);

/*
 * fp4_lora_apply -- y[m, n] (bf16) = bf16_RNE(base + s_l T B_l^T) and T
 * [m, rank] (binary32, zero for rows without an adapter), which the backward
 * call reads.  base: bf16 [m, n], the shared projection's output; null for
 * zero; it may be y itself (same row stride).  x: bf16 [m, k].  Rows 16-byte
 * aligned (row strides % 8 == 0).
 */
FP4_API fp4_status fp4_lora_apply(const uint16_t* x, int64_t ldx, int64_t m, const fp4_lora_bank* bank,
                                  const int32_t* slots, const uint16_t* base, int64_t ld_base, uint16_t* y, int64_t ldy,
                                  float* t, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * fp4_lora_backward -- the gradients of fp4_lora_apply for dy [m, n]:
 *   dT = s_l dy B_l,  dx = bf16_RNE(dx_base + dT A_l),
 *   da[l] = sum_i dT_i^T x_i,  db[l] = s_l sum_i dy_i^T T_i
 * over the rows i of adapter l (zero for an adapter without rows).  t is
 * fp4_lora_apply's T; dx_base is the gradient that arrives at x through the
 * shared projection (null for zero; it may be dx; dx may be neither x nor
 * dy).  da, db have the bank's shapes in grad_dtype, are written whole and
 * 16-byte aligned.  The sums are
 * taken in a fixed order: the same inputs give the same bits.
 */
FP4_API fp4_status fp4_lora_backward(const uint16_t* dy, int64_t ld_dy, const uint16_t* x, int64_t ldx, int64_t m,
                                     const float* t, const fp4_lora_bank* bank, const int32_t* slots,
                                     const uint16_t* dx_base, int64_t ld_dx_base, uint16_t* dx, int64_t ld_dx, void* da,
                                     void* db, int32_t grad_dtype, void* workspace, int64_t workspace_bytes,
                                     void* stream);

/*
 * fp4_wo_gemm_lora -- fp4_wo_gemm with the rows' adapters in its epilogue:
 * Y = bf16_RNE(gw sum_k x (e(w) s_w) + s_l T B_l^T), rounded once.
 * Requirements and errors as fp4_wo_gemm (neither N nor K may be 0 here),
 * bank->k = K and bank->n = N.
 */
FP4_API fp4_status fp4_wo_gemm_lora(const uint16_t* x, int64_t ldx, int64_t m, const fp4_tensor* w,
                                    const fp4_lora_bank* bank, const int32_t* slots, uint16_t* y, int64_t ldy,
                                    void* workspace, int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * fp4_token_logprobs -- for every row z of logits [rows, vocab] (f32 or bf16,
 * any row stride ld >= vocab, element aligned), with p = softmax(z /
 * temperature) (quant_prune_distill/574: the rollouts' policy loss reads the
 * chosen tokens' log probabilities and the policy's entropy):
 *   logprob[row] = log p[tokens[row]] (0 when the token is outside 0 ..
 *     vocab - 1, by convention -100: no token); tokens may be null
 *   entropy[row] = -sum p log p
 *   top_ids / top_logprobs [rows, top]: the `top` (0 .. 32) largest, largest
 *     first, equal logits by the lower index; NaN sorts above everything
 *   stats [rows, 2]: {largest logit, log sum exp((z - largest) / temperature)},
 *     which the backward call reads
 * A logit of -inf has probability 0 and adds nothing.  A row of only -inf
 * has no probability: entropy 0, log probabilities -inf.  A NaN or +inf
 * makes its own row's results NaN.  Sums in binary32.  temperature > 0, and
 * 2 / temperature is finite.
 * Fewer than 2^22 rows and 2^27 tokens.  workspace: as above,
 * fp4_token_logprobs_workspace bytes.
 */
FP4_API int64_t fp4_token_logprobs_workspace(int64_t rows, int64_t vocab, int32_t top);
FP4_API fp4_status fp4_token_logprobs(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                                      const int64_t* tokens, float temperature, int32_t top, float* logprob,
                                      float* entropy, float* stats, int32_t* top_ids, float* top_logprobs,
                                      void* workspace, int64_t workspace_bytes, void* stream);

/*
 * fp4_token_logprobs_backward -- dlogits [rows, vocab] (the logits' type, row
 * stride ld_d; it may be the logits themselves) for the gradients
 * grad_logprob and grad_entropy [rows] (either null for zero):
 *   dz_v = (grad_logprob ([v = token] - p_v)
 *           - grad_entropy p_v (log p_v + entropy)) / temperature
 * entropy and stats are the forward call's.  A row whose two gradients are
 * zero, or whose token is none and whose grad_entropy is zero, gets zeros
 * whatever its logits hold; so does a row of only -inf.  The top
 * alternatives carry no gradient.
 */
FP4_API fp4_status fp4_token_logprobs_backward(const void* logits, int32_t dtype, int64_t ld, int64_t rows,
                                               int64_t vocab, const int64_t* tokens, float temperature,
                                               const float* entropy, const float* stats, const float* grad_logprob,
                                               const float* grad_entropy, void* dlogits, int64_t ld_d, void* stream);

/* ---------------------------------------------------------------------------
 * fp4_residual_norm -- the norms after and before a block, fused with its
 * gate and residual scale (quant_prune_distill/574 "Метод": the RMSNorms
 * around the FP4 products; reading):
 *   u = RMSNorm(x) w_post  (u = x when w_post is null)
 *   h = alpha res + gate u  (gate [rows], binary32; null for 1)
 *   n = RMSNorm(h) w_pre,  RMSNorm(v) = v / sqrt(mean v^2 + eps)
 * x and n in x_dtype, res and h in res_dtype, the weights in weight_dtype
 * (each f32 or bf16); n comes from the unrounded h.  The squares are summed in
 * binary32, so a row's norm must stay below 2^64.  Fewer than 2^22 rows;
 * cols at most 32768, any value and alignment of elements (rows of whole
 * 16-byte vectors, cols % 8 == 0, are read as vectors, others one element at a
 * time).  stats [rows, 2] = {1 / sqrt(mean x^2 + eps)
 * (1 without w_post), 1 / sqrt(mean h^2 + eps)} for the backward call.  h may
 * be res and n may be x (same row strides). */
typedef struct fp4_norm {
    const void* x; int64_t ld_x;
    const void* res; int64_t ld_res;
    int64_t rows, cols;
    const void* w_pre;
    const void* w_post;
    const float* gate;
    float alpha, eps;
    int32_t x_dtype, res_dtype, weight_dtype;
} fp4_norm;

FP4_API fp4_status fp4_residual_norm(const fp4_norm* args, void* h, int64_t ld_h, void* n, int64_t ld_n, float* stats,
                                     void* stream);

/*
 * fp4_residual_norm_backward -- gradients for dn (of n, x_dtype) and dh (of
 * h, res_dtype; either null for zero): dx, dres in the types of x and res,
 * dw_pre and dw_post [cols] and dgate [rows] in binary32 (dw_post, dgate only
 * where the forward call had w_post, gate).  dx may be x or dn, dres may be
 * res or dh.  The weights' sums over the rows are taken in a fixed order.
 * workspace: as above, fp4_residual_norm_workspace bytes (post: w_post given).
 */
FP4_API int64_t fp4_residual_norm_workspace(int64_t rows, int64_t cols, int32_t post);
FP4_API fp4_status fp4_residual_norm_backward(const fp4_norm* args, const float* stats, const void* dn, int64_t ld_dn,
                                              const void* dh, int64_t ld_dh, void* dx, int64_t ld_dx, void* dres,
                                              int64_t ld_dres, float* dw_pre, float* dw_post, float* dgate,
                                              void* workspace, int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Products with an epilogue (ue5m3-fp4-pretraining "Что сделали": all suitable
 * linear layers run in FP4; the pages give no formula for what follows a
 * product, reading):
 *   v = A W^T + bias,  y = bf16_RNE(residual + mul act(v)),  pre = bf16_RNE(v)
 * everything between the product's sums and the roundings in binary32.  With
 * s(x) = 1 / (1 + e^-x) and Phi the normal distribution, act(v) is
 *   none v; relu max(v, 0); silu v s(v); gelu v Phi(v);
 *   gelu_tanh v s(2 u), u = sqrt(2 / pi) (v + 0.044715 v^3)
 * (an exponential below 2^-126 counts as zero, which an act of about -1e-36 and
 * smaller then is) so that a gated layer is two products: the up projection's output is the
 * gate projection's mul.  bias: [n] in bias_dtype (f32 or bf16); mul, residual
 * and pre: bf16 [m, n], element aligned, row strides >= n; each may be null.
 * y may be mul or residual (same row stride), pre none of them. */
typedef enum fp4_act {
    FP4_ACT_NONE = 0,
    FP4_ACT_RELU = 1,
    FP4_ACT_SILU = 2,
    FP4_ACT_GELU = 3,
    FP4_ACT_GELU_TANH = 4
} fp4_act;

typedef struct fp4_epilogue {
    const void* bias;
    int32_t bias_dtype;
    int32_t act;
    const uint16_t* mul; int64_t ld_mul;
    const uint16_t* residual; int64_t ld_residual;
    uint16_t* pre; int64_t ld_pre;
} fp4_epilogue;

/*
 * fp4_gemm_epilogue -- fp4_gemm followed by the epilogue.  Requirements,
 * paths and errors as fp4_gemm (K may not be 0 here); the product's error
 * bound is that of fp4_gemm before any rounding.  A product of few tiles is
 * taken in ranges of K, whose sums are joined in a fixed order.  workspace: as
 * above, fp4_gemm_epilogue_workspace bytes for these operands (it depends on
 * their shapes and formats, and on fp4_set_gemm_small_outputs).
 */
FP4_API int64_t fp4_gemm_epilogue_workspace(const fp4_tensor* a, const fp4_tensor* b);
FP4_API fp4_status fp4_gemm_epilogue(const fp4_tensor* a, const fp4_tensor* b, const fp4_epilogue* e, uint16_t* y,
                                     int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * fp4_wo_gemm_epilogue -- fp4_wo_gemm followed by the epilogue, for serving
 * (pre is UNSUPPORTED).  Requirements and errors as fp4_wo_gemm (neither N nor
 * K may be 0 here).  y may not be x (INVALID_ARG), also where x is the
 * residual too.
 */
FP4_API fp4_status fp4_wo_gemm_epilogue(const uint16_t* x, int64_t ldx, int64_t m, const fp4_tensor* w,
                                        const fp4_epilogue* e, uint16_t* y, int64_t ldy, void* stream);

/*
 * fp4_epilogue_backward -- the epilogue's gradients for dy [rows, cols], at
 * the saved pre (bf16):
 *   dpre = bf16_RNE(dy mul act'(pre)),  dmul = bf16_RNE(dy act(pre)),
 *   dbias = sum over the rows of dy mul act'(pre), binary32, unrounded terms
 * (relu'(0) = 0; the residual's gradient is dy).  All bf16 with row strides
 * >= cols, element aligned.  mul null: 1, and no dmul.  dbias null: not
 * computed.  With act none and mul null dpre is dy itself: pre is not read
 * and dpre may be null.  dpre and dmul may be dy, pre or mul (same row
 * stride), but not each other.  The sums over the rows are taken in a fixed
 * order: the same inputs give the same bits.  cols at most 2^24.  workspace
 * (only with dbias): as above, fp4_epilogue_workspace bytes.
 */
FP4_API int64_t fp4_epilogue_workspace(int64_t rows, int64_t cols);
FP4_API fp4_status fp4_epilogue_backward(const uint16_t* dy, int64_t ld_dy, const uint16_t* pre, int64_t ld_pre,
                                         const uint16_t* mul, int64_t ld_mul, int64_t rows, int64_t cols, int32_t act,
                                         uint16_t* dpre, int64_t ld_dpre, uint16_t* dmul, int64_t ld_dmul, float* dbias,
                                         void* workspace, int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * fp4_moe_route -- a router's choice: for every row of logits [rows, experts]
 * (f32 or bf16, any row stride ld >= experts, element aligned)
 *   s = softmax(logits) or, each alone, 1 / (1 + e^-logits)
 *   ids [rows, top] = the `top` largest of s + bias (bias [experts] binary32,
 *     null for none: it takes part in the choice alone), largest first, equal
 *     ones by the lower index; without a bias by the logits themselves
 *   weights [rows, top] = scale s[ids], with renormalize divided by the chosen
 *     ones' sum (0 where that is 0)
 * in binary64, rounded once.  An expert whose logit is -inf is never chosen:
 * a row with fewer than `top` others ends in id -1 and weight 0.  NaN sorts
 * above everything.  top 1 .. 16 and at most experts, which are at most 1024;
 * fewer than 2^22 rows.
 */
typedef enum fp4_route_score {
    FP4_ROUTE_SOFTMAX = 0,
    FP4_ROUTE_SIGMOID = 1
} fp4_route_score;

FP4_API fp4_status fp4_moe_route(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t experts, int32_t top,
                                 int32_t score, const float* bias, int32_t renormalize, float scale, int32_t* ids,
                                 float* weights, void* stream);

/* The experts of a layer: gate_up [experts * 2 ffn, hidden], each expert's ffn
 * gate rows before its ffn up rows, and down [experts * hidden, ffn], quantized
 * along their columns on any element grid (they may differ); up_scale and
 * down_scale [experts] in binary32 (null: 1) multiply an expert's products, for
 * experts that were quantized each with a tensor scale of its own. */
typedef struct fp4_moe_bank {
    fp4_tensor gate_up, down;
    const float* up_scale;
    const float* down_scale;
    int64_t experts;
} fp4_moe_bank;

/*
 * fp4_moe -- a whole mixture-of-experts layer for 1 .. 16 tokens (the
 * weight-only product's rows; quant_prune_distill/574 "Эксперименты"):
 *   y_i = bf16_RNE(residual_i + sum_k w_ik D_e (act(G_e x_i) (U_e x_i))),
 *   e = ids_ik
 * with bf16 x, ids (int32) and weights (binary32) [m, top] dense, top 1 .. 16.
 * Weights enter the matrix instruction exactly, as in fp4_wo_gemm but so that
 * an infinity times a weight other than zero is one on every grid; sums are
 * binary32, and what act gives reaches the down projection with 17 bits (an
 * infinity there stays one).  An id outside 0 .. experts - 1 (-1 by
 * convention) is no expert; an id that a token names twice has both weights.
 * A token without experts gets residual (null: zero).  Nothing of one token
 * or expert reaches the results of a token that did not choose it.  The sums
 * are taken in a fixed order.
 * hidden % 128 == 0, ffn % 128 == 0; x 16-byte aligned with ldx % 8 == 0;
 * codes 16-byte and scales 4-byte aligned, no transform, one expert's codes
 * below 4 GiB, at most 65535 experts; y and residual element aligned, y may be
 * residual (same row stride) or x.  workspace: as above, fp4_moe_workspace
 * bytes.
 */
FP4_API int64_t fp4_moe_workspace(int64_t m, int32_t top, int64_t ffn);
FP4_API fp4_status fp4_moe(const uint16_t* x, int64_t ldx, int64_t m, const fp4_moe_bank* bank, const int32_t* ids,
                           const float* weights, int32_t top, int32_t act, const uint16_t* residual, int64_t ld_residual,
                           uint16_t* y, int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * fp4_distill_loss -- the loss of a student's logits z [rows, vocab] (f32 or
 * bf16, any row stride ld >= vocab, element aligned) against a teacher's top
 * log probabilities, for instance those of fp4_token_logprobs (the pages
 * train models with FP4 linear layers; the loss is a reading).  With q =
 * softmax(z / temperature), p_j = exp(top_logprobs_j), P = sum p_j and R the
 * student's probability of the tokens that are not listed:
 *   bucket       loss = sum p_j (log p_j - log q_j)
 *                       + (1 - P) (log(1 - P) - log R)
 *   renormalize  loss = the first sum with p_j / P in the place of p_j
 * top_ids (int32) and top_logprobs [rows, top] dense, top 1 .. 128.  An id
 * outside the vocabulary (-1 by convention) is no entry; a row without
 * entries, or whose entries have no probability, has loss 0 and no gradient.
 * A token that is listed twice has the sum of both probabilities, and both
 * terms.  In the bucket's form a P of 1 or more, by rounding, leaves nothing
 * for the other tokens, and a student that gives them nothing (all listed, or
 * -inf) has no such term.  A student's -inf at a token with p > 0 makes the
 * loss inf (its gradient stays finite); a row of only -inf has loss inf and
 * gradient 0; a NaN or +inf logit makes the loss of its row NaN (a row of loss
 * 0 by its list alone, above, keeps that).
 * stats [rows, 7]: for the backward call.  temperature > 0, and 2 /
 * temperature is finite.  Fewer than 2^22 rows, at most 2^24 tokens.
 * workspace: as above, fp4_distill_workspace bytes.
 */
typedef enum fp4_distill_rest {
    FP4_DISTILL_BUCKET = 0,
    FP4_DISTILL_RENORMALIZE = 1
} fp4_distill_rest;

FP4_API int64_t fp4_distill_workspace(int64_t rows, int64_t vocab, int32_t dtype);
FP4_API fp4_status fp4_distill_loss(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                                    const int32_t* top_ids, const float* top_logprobs, int32_t top, float temperature,
                                    int32_t rest, float* loss, float* stats, void* workspace, int64_t workspace_bytes,
                                    void* stream);

/*
 * fp4_distill_loss_backward -- dlogits [rows, vocab] (the logits' type, row
 * stride ld_d; it may be the logits themselves) for grad_loss [rows]:
 *   dz_v = grad_loss (q_v - p_v) / temperature           (bucket: listed v)
 *   dz_v = grad_loss q_v (1 - (1 - P) / R) / temperature (bucket: others)
 * with p_v / P, and 0 for the others, in the renormalized form.  Without the
 * bucket's second term (above) q_v comes with the factor P.  The arguments are
 * the forward call's; the teacher has no gradient.  A row whose grad_loss is 0
 * gets zeros whatever its logits hold.
 */
FP4_API fp4_status fp4_distill_loss_backward(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                                             const int32_t* top_ids, const float* top_logprobs, int32_t top,
                                             float temperature, int32_t rest, const float* stats, const float* grad_loss,
                                             void* dlogits, int64_t ld_d, void* stream);

/* Static description of a status code. */
FP4_API const char* fp4_status_string(fp4_status status);

/* Library ABI version (major * 100 + minor). */
FP4_API int32_t fp4_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP4_H */
