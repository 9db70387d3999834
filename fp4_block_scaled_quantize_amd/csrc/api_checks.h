// api_checks.h -- argument checks shared by the translation units of the C
// ABI (api.cpp, api_train.cpp, api_layer.cpp): what a quantized tensor and the
// products' operands must satisfy before any launch.
#pragma once

#include <math.h>
#include <stdint.h>

#include "fp4.h"
#include "fp4_internal.h"

namespace fp4 {

constexpr int64_t kMaxElems = int64_t(1) << 40;       // elements of one tensor: byte offsets stay far from 63 bits
constexpr int64_t kMaxLineRows = int64_t(1) << 22;    // rows with a workgroup each: below 2^32 threads at 1024

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int64_t up16(int64_t b) { return (b + 15) / 16 * 16; }
inline bool dtype_ok(int32_t d) { return d == FP4_DTYPE_F32 || d == FP4_DTYPE_BF16; }
inline int64_t esize(int32_t d) { return d == FP4_DTYPE_BF16 ? 2 : 4; }
inline fp4_status check_space(const void* ws, int64_t have, int64_t need)
{
    if (need == 0) return FP4_OK;
    if (!ws || have < need) return FP4_ERR_INVALID_ARG;
    return aligned(ws, 16) ? FP4_OK : FP4_ERR_ALIGN;
}
// Rows of logits and the temperature that a call takes them at.
inline fp4_status check_logits(const void* z, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab, float temperature)
{
    if (!dtype_ok(dtype)) return FP4_ERR_INVALID_ARG;
    // the kernels work with log2(e) / temperature
    if (!(temperature > 0.0f) || !isfinite(temperature) || !isfinite(2.0f / temperature)) return FP4_ERR_INVALID_ARG;
    if (rows < 0 || vocab < 1 || ld < vocab) return FP4_ERR_SHAPE;
    if (rows >= kMaxLineRows || vocab >= (int64_t(1) << 27) || ld > kMaxElems / (rows ? rows : 1))
        return FP4_ERR_UNSUPPORTED;
    if (!z && rows) return FP4_ERR_INVALID_ARG;
    if (!aligned(z, (uintptr_t)esize(dtype))) return FP4_ERR_ALIGN;
    return FP4_OK;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool elem_is_8bit(int32_t e) { return e == FP4_ELEM_FP8_E4M3 || e == FP4_ELEM_INT8; }
inline bool elem_is_6bit(int32_t e) { return e >= FP4_ELEM_FP6_E2M3 && e <= FP4_ELEM_INT6; }
// the 8- and 6-bit grids: their codes leave in wider pieces
inline bool elem_is_wide(int32_t e) { return elem_is_8bit(e) || elem_is_6bit(e); }

inline fp4_status check_tensor(const fp4_tensor* t, ScaleFmtHost* f)
{
    if (!t || !t->tensor_scale) return FP4_ERR_INVALID_ARG;
    const bool empty = t->rows == 0 || t->cols == 0;
    if (!empty && (!t->q || !t->scales)) return FP4_ERR_INVALID_ARG;
    if (t->fmt.block != 16 && t->fmt.block != 32) return FP4_ERR_INVALID_ARG;
    if (t->fmt.rounding != FP4_ROUND_NEAREST_EVEN && t->fmt.rounding != FP4_ROUND_STOCHASTIC)
        return FP4_ERR_INVALID_ARG;
    if (t->fmt.amax != FP4_AMAX_NONE && t->fmt.amax != FP4_AMAX_CURRENT && t->fmt.amax != FP4_AMAX_DELAYED)
        return FP4_ERR_INVALID_ARG;
    if (!scale_fmt_params(t->fmt.scale, f)) return FP4_ERR_INVALID_ARG;
    if (t->fmt.transform != FP4_TRANSFORM_NONE && t->fmt.transform != FP4_TRANSFORM_RHT) return FP4_ERR_INVALID_ARG;
    if (t->fmt.element < FP4_ELEM_E2M1 || t->fmt.element > FP4_ELEM_INT6) return FP4_ERR_INVALID_ARG;
    if (t->rows < 0 || t->cols < 0) return FP4_ERR_SHAPE;
    if (t->cols % t->fmt.block) return FP4_ERR_SHAPE;
    // codes leave as 4-byte pieces (4-bit grids), 8-byte pieces (8-bit
    // grids) or 2-byte pieces at 6-byte steps (6-bit grids; 8-byte alignment
    // asked for as for 8 bits)
    if (((uintptr_t)t->q & (elem_is_wide(t->fmt.element) ? 7u : 3u)) != 0) return FP4_ERR_ALIGN;
    if ((t->rows * (t->cols / 8)) >= (int64_t(1) << 31)) return FP4_ERR_SHAPE;
    return FP4_OK;
}

inline fp4_status hip_status(hipError_t e) { return e == hipSuccess ? FP4_OK : FP4_ERR_HIP; }

// fp4_gemm's arguments, in the order its errors are documented; on FP4_OK with
// a non-empty product *p describes the launch.
inline fp4_status check_gemm(const fp4_tensor* a, const fp4_tensor* b, uint16_t* c, int64_t ldc, GemmLaunch* p)
{
    ScaleFmtHost fa, fb;
    fp4_status st = check_tensor(a, &fa);
    if (st != FP4_OK) return st;
    st = check_tensor(b, &fb);
    if (st != FP4_OK) return st;
    if (!c) return FP4_ERR_INVALID_ARG;
    if (a->cols != b->cols) return FP4_ERR_SHAPE;
    if (a->fmt.block != b->fmt.block) return FP4_ERR_UNSUPPORTED;
    // transformed operands multiply to the same product only when both carry
    // the same transform along K
    if (a->fmt.element != b->fmt.element) return FP4_ERR_UNSUPPORTED;
    if (a->fmt.transform != b->fmt.transform) return FP4_ERR_UNSUPPORTED;
    if (a->fmt.transform != FP4_TRANSFORM_NONE && a->fmt.transform_signs != b->fmt.transform_signs)
        return FP4_ERR_UNSUPPORTED;
    if (a->cols % 128) return FP4_ERR_SHAPE;
    if (ldc < b->rows) return FP4_ERR_SHAPE;
    if (((uintptr_t)c & 1u) != 0) return FP4_ERR_ALIGN;
    if (a->rows == 0 || b->rows == 0 || a->cols == 0) return FP4_OK;
    if (!aligned16(a->q) || !aligned16(b->q) || ((uintptr_t)a->scales & 3u) || ((uintptr_t)b->scales & 3u))
        return FP4_ERR_ALIGN;
    p->qa = a->q; p->sa = a->scales; p->ga = a->tensor_scale;
    p->qb = b->q; p->sb = b->scales; p->gb = b->tensor_scale;
    p->m = a->rows; p->n = b->rows; p->k = a->cols;
    p->block = a->fmt.block;
    p->fa = fa; p->fb = fb;
    p->c = c; p->ldc = ldc;
    p->elem = a->fmt.element;
    return FP4_OK;
}
// Both operands E2M1 with E8M0 scales at block 32: the block-scaled instruction.
inline bool gemm_is_mx(const GemmLaunch& p)
{
    return p.elem == FP4_ELEM_E2M1 && p.fa.is_e8m0 && p.fb.is_e8m0 && p.block == 32;
}

// fp4_wo_gemm's arguments, in the order its errors are documented; on FP4_OK
// with a non-empty product *p describes the launch.
inline fp4_status check_wo_gemm(const uint16_t* x, int64_t ldx, int64_t m, const fp4_tensor* w, uint16_t* y,
                                int64_t ldy, WoGemmLaunch* p)
{
    ScaleFmtHost fw;
    fp4_status st = check_tensor(w, &fw);
    if (st != FP4_OK) return st;
    if (!y || (!x && w->cols != 0)) return FP4_ERR_INVALID_ARG;
    if (m < 1 || m > 16) return FP4_ERR_UNSUPPORTED;
    if (w->fmt.transform != FP4_TRANSFORM_NONE) return FP4_ERR_UNSUPPORTED;   // x would need the same transform
    if (w->cols % 256) return FP4_ERR_SHAPE;
    if (ldx < w->cols || ldy < w->rows) return FP4_ERR_SHAPE;
    if (w->rows == 0 || w->cols == 0) return FP4_OK;
    // the kernel addresses W and x with 32-bit byte/element offsets
    const int64_t wbits = elem_is_8bit(w->fmt.element) ? 8 : elem_is_6bit(w->fmt.element) ? 6 : 4;
    if (w->rows * (w->cols * wbits / 8) >= (int64_t(1) << 32) || ldx * m >= (int64_t(1) << 31))
        return FP4_ERR_UNSUPPORTED;
    if (!aligned16(x) || ldx % 8) return FP4_ERR_ALIGN;
    if (!aligned16(w->q) || ((uintptr_t)w->scales & 3u)) return FP4_ERR_ALIGN;
    p->x = x; p->ldx = ldx; p->m = m;
    p->qw = w->q; p->sw = w->scales; p->gw = w->tensor_scale;
    p->n = w->rows; p->k = w->cols;
    p->elem = w->fmt.element;
    p->block = w->fmt.block;
    p->fw = fw;
    p->y = y; p->ldy = ldy;
    return FP4_OK;
}

}  // namespace fp4
