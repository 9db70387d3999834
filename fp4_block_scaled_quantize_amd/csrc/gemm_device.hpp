// gemm_device.hpp -- pieces that the products share (gemm.hip, moe.hip): loads
// straight into LDS, exact conversions of the element grids to bf16, and the
// weight-only products' ring slots.
#pragma once

#include <type_traits>

#include "fp4_device.hpp"
#include "fp4_internal.h"

namespace fp4 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ void dma16(const void* g, uint8_t* lds)
{
    __builtin_amdgcn_global_load_lds(g, (lds_ptr_t)lds, 16, 0, 0);
}
// Past the caches (the instruction's non-temporal bit): for whole lines that
// are read once.
__device__ __forceinline__ void dma16_once(const void* g, uint8_t* lds)
{
    __builtin_amdgcn_global_load_lds(g, (lds_ptr_t)lds, 16, 0, 2);
}
__device__ __forceinline__ void dma4(const void* g, uint8_t* lds)
{
    __builtin_amdgcn_global_load_lds(g, (lds_ptr_t)lds, 4, 0, 0);
}

// Largest power of two not above a positive normal g (1 for anything else):
// g / split_pow2(g) lies in [1, 2) and the division is exact.
__device__ __forceinline__ float split_pow2(float g)
{
    const uint32_t e = __float_as_uint(g) & 0x7F800000u;
    return (e == 0u || e == 0x7F800000u || g < 0.0f) ? 1.0f : __uint_as_float(e);
}

typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Exact bf16 dequantization of one dword of 8 E2M1 codes with scale s.  The
// gfx950 converts apply only the exponent of their scale operand, so:
//  POW2 (E8M0 scales): v_cvt_scalef32_pk_bf16_fp4 with s does everything;
//  otherwise: convert with scale 1 to fp32, multiply by s (exact: at most
//  9 significant bits), keep the top half (exact when the value fits bf16).
// Elements 2b and 2b + 1 of a dword of codes as binary32: the hardware
// E2M1 conversion (scale 1), or for INT4 the sign-extended nibbles.
template <bool INT>
__device__ __forceinline__ v2f elem_pair_f32(uint32_t w, int b)
{
    if (INT)
        return v2f{(float)((int32_t)(w << (28 - 8 * b)) >> 28), (float)((int32_t)(w << (24 - 8 * b)) >> 28)};
    return b == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0)
         : b == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1)
         : b == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2)
                  : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
}

// Elements k and k + 1 (k even) of the codes dw of one chunk row piece (the
// grid's packing: 4-bit nibbles, bytes, or the six-bit stream) as binary32:
// E2M1 and FP8 E4M3 by the hardware conversions (scale 1, exact), INT4 /
// INT8 / INT6 sign-extended, FP6 E2M3 / E3M2 through the FP8 E4M3 / E5M2
// byte of the value times 2^-6 / 2^-12 (exact) and one multiply back.  k is
// a compile-time constant after unrolling.
template <int ELEM>
__device__ __forceinline__ v2f elem_pair_any(const uint32_t* dw, int k)
{
    if constexpr (ELEM <= 1) {
        return elem_pair_f32<ELEM == 1>(dw[k >> 3], (k & 7) >> 1);
    } else if constexpr (ELEM == 2) {
        return (k & 3) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)dw[k >> 2], true)
                       : __builtin_amdgcn_cvt_pk_f32_fp8((int)dw[k >> 2], false);
    } else if constexpr (ELEM == 3) {
        const uint32_t w = dw[k >> 2] >> (8 * (k & 3));
        return v2f{int8_value(w), int8_value(w >> 8)};
    } else {
        const int bit = 6 * k, i = bit >> 5, sh = bit & 31;
        const uint32_t x = sh + 12 <= 32 ? dw[i] >> sh : __builtin_amdgcn_alignbit(dw[i + 1], dw[i], sh);
        if constexpr (ELEM == 6) {
            return v2f{(float)((int32_t)(x << 26) >> 26), (float)((int32_t)(x << 20) >> 26)};
        } else {
            // the two codes to one byte each, sign bit 5 -> 7: the FP8 byte
            const uint32_t y = (x & 0x3Fu) | ((x << 2) & 0x3F00u);
            const uint32_t w = (y & 0x1F1Fu) | ((y & 0x2020u) << 2);
            const v2f e = ELEM == 4 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false)
                                    : __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
            constexpr float kFold = ELEM == 4 ? 64.0f : 4096.0f;
            return v2f{e[0] * kFold, e[1] * kFold};
        }
    }
}

// The two bf16 terms of products v = f s of up to 16 significant bits, as
// pairs: the first is the truncation, so that the second is the exact
// remainder.  With BOTH it is the truncation of the next value towards zero:
// then the remainder of a product other than zero is not zero either, has its
// sign, and an infinity times the two is an infinity and not a NaN.  (f s + 0
// is no negative zero, at which the step would wrap.  An instruction more an
// element: INT8 experts of 4096 x 1536 with E4M3 scales, 37 met by 16 tokens,
// 218 -> 223 us, with permutes in the place of shifts and masks (with those 210
// -> 225).)
template <bool BOTH>
__device__ __forceinline__ void split_pair(v2f f, float s, int& hi, int& lo)
{
    if constexpr (BOTH) {
        const float v0 = __builtin_fmaf(f[0], s, 0.0f), v1 = __builtin_fmaf(f[1], s, 0.0f);
        const uint32_t u0 = __builtin_elementwise_sub_sat(__float_as_uint(v0), 1u);
        const uint32_t u1 = __builtin_elementwise_sub_sat(__float_as_uint(v1), 1u);
        const float l0 = v0 - __uint_as_float(u0 & 0xFFFF0000u), l1 = v1 - __uint_as_float(u1 & 0xFFFF0000u);
        hi = (int)__builtin_amdgcn_perm(u1, u0, 0x07060302u);
        lo = (int)__builtin_amdgcn_perm(__float_as_uint(l1), __float_as_uint(l0), 0x07060302u);
    } else {
        const float v0 = f[0] * s, v1 = f[1] * s;
        const uint32_t h0 = __float_as_uint(v0) & 0xFFFF0000u, h1 = __float_as_uint(v1) & 0xFFFF0000u;
        const float l0 = v0 - __uint_as_float(h0), l1 = v1 - __uint_as_float(h1);
        hi = (int)((h0 >> 16) | h1);
        lo = (int)((__float_as_uint(l0) >> 16) | (__float_as_uint(l1) & 0xFFFF0000u));
    }
}

// Elements 8t .. 8t + 7 of dw times s as bf16 pairs: hi the truncation of
// each binary32 product (exact when it fits bf16), with SPLIT two terms.
template <int ELEM, bool SPLIT, bool BOTH = false>
__device__ __forceinline__ void dq8_any(const uint32_t* dw, int t, float s, v4i& hi, v4i& lo)
{
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const v2f f = elem_pair_any<ELEM>(dw, 8 * t + 2 * b);
        if constexpr (SPLIT) {
            int h, l;
            split_pair<BOTH>(f, s, h, l);
            hi[b] = h;
            lo[b] = l;
        } else {
            const float v0 = f[0] * s, v1 = f[1] * s;
            hi[b] = (int)__builtin_amdgcn_perm(__float_as_uint(v1), __float_as_uint(v0), 0x07060302u);
        }
    }
}

// INT: INT4 elements (never POW2: the multiply by s is exact for E8M0 too).
template <bool POW2, bool INT = false>
__device__ __forceinline__ v4i dq8_bf16(uint32_t w, float s)
{
    v4i r;
    if (POW2 && !INT) {
        r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    } else {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const v2f f = elem_pair_f32<INT>(w, b);
            const uint32_t lo = __float_as_uint(f[0] * s), hi = __float_as_uint(f[1] * s);
            r[b] = (int)__builtin_amdgcn_perm(hi, lo, 0x07060302u);     // {hi[31:16], lo[31:16]}
        }
    }
    return r;
}

// Products wider than bf16 (E1M6 with E2M1: 9 significant bits; INT4 with
// 5- or 6-bit mantissas: up to 10): split v = hi + lo, both exact bf16.
template <bool INT = false, bool BOTH = false>
__device__ __forceinline__ void dq8_bf16_split(uint32_t w, float s, v4i& hi, v4i& lo)
{
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const v2f f = elem_pair_f32<INT>(w, b);
        int h, l;
        split_pair<BOTH>(f, s, h, l);
        hi[b] = h;
        lo[b] = l;
    }
}

// One ring slot of the weight-only GEMM (byte offsets).  A chunk is SUB
// runs of 128 K-elements.  XQ = 0: M == 1, the single X row arrives by
// 4-byte loads (SUB of them); else XQ * SUB loads of four 256-byte X row
// pieces each.  WP: LDS pitch of a W chunk row (64 bytes, or 128 for the
// wider rows); SCB: scale bytes of a row per chunk.
template <int RG, int XQ, int WP, int SUB, int SCB>
struct WoSlot {
    static constexpr int WD = WP / 64;                 // W loads per 16-row group
    static constexpr int W = 0;                        // row r of group g at 16 WP g + WP r
    static constexpr int SC = RG * 16 * WP;            // row r of the slot's 16 RG rows at SC + SCB r
    static constexpr int SCBytes = (RG * 16 * SCB + 255) / 256 * 256;
    static constexpr int NSC = (RG * 16 * SCB / 4 + 63) / 64;      // 4-byte scale loads (64 lanes each)
    static constexpr int X = SC + SCBytes;             // piece h of row m at X + 1024 (SUB (m / 4) + h) + 256 (m % 4)
    static constexpr int XRows = XQ == 0 ? 1 : 4 * XQ;
    static constexpr int Bytes = X + 256 * SUB * XRows;
    static constexpr int Loads = RG * WD + NSC + SUB * (XQ == 0 ? 1 : XQ);   // direct-to-LDS loads per chunk
};

// 16-byte piece c of row r sits at c ^ swz(r): 64-byte rows (r >> 1) & 3,
// 128-byte rows (r >> 1) & 7 (16 consecutive rows, one piece each, on
// distinct banks)
__device__ __forceinline__ int wo_swz(int r) { return (r >> 1) & 3; }
__device__ __forceinline__ int wo_swz8(int r) { return (r >> 1) & 7; }

template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Code bytes of a W row per 128 K-elements and the LDS pitch of a chunk row.
template <int ELEM, int SUB>
struct WoRow {
    static constexpr int Bytes128 = ELEM <= 1 ? 64 : ELEM <= 3 ? 128 : 96;
    static constexpr int WB = SUB * Bytes128;
    static constexpr int WP = WB <= 64 ? 64 : 128;
};

// Kernels with more than 64 KiB of dynamic LDS must opt in once per device.
template <typename K>
inline hipError_t allow_lds(K kernel, size_t bytes)
{
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                               (int)bytes);
}

// Formats whose e2m1 * s products are exact in f16 (normal range) and those
// exact in bf16 (at most 8 significant bits).
inline bool exact_in_f16(const ScaleFmtHost& f) { return !f.is_e8m0 && f.ebits <= 4 && (f.ebits + f.mbits == 7); }
inline bool exact_in_bf16(const ScaleFmtHost& f) { return f.is_e8m0 || f.mbits <= 5; }


// Significant bits of the largest element of each grid (E2M1 2, INT4 3,
// FP8 E4M3 4, INT8 7, FP6 E2M3 4, FP6 E3M2 3, INT6 5) plus those of the
// scale: products with at most 8 are exact in bf16, the others (at most 14)
// take the hi + lo split.
inline bool wo_exact_in_bf16(int elem, const ScaleFmtHost& f)
{
    static const int ebits[7] = {2, 3, 4, 7, 4, 3, 5};
    const int sbits = f.is_e8m0 ? 1 : f.mbits + 1;
    return ebits[elem] + sbits <= 8;
}

}  // namespace fp4
