// epilogue_device.hpp -- what follows a product's sums in registers: bias,
// activation, multiplier and residual (gemm.hip's epilogue forms, epilogue.hip,
// moe.hip).
//
//   v = sum + bias,  y = res + mul act(v)
//
// in binary32, each output rounded once.  The activations, with s(x) = 1 /
// (1 + e^-x) and Phi the normal distribution:
//   relu max(v, 0); silu v s(v); gelu v Phi(v);
//   gelu_tanh v (1 + tanh u) / 2 = v s(2 u), u = sqrt(2 / pi) (v + 0.044715 v^3)
// The last two are taken in the forms that keep their small values' bits at
// far negative v, where 1 + erf and 1 + tanh cancel: Phi there is its tail
//   Phi(-a) = exp(-a^2 / 2) R(a),  R(a) = exp(a^2 / 2) Phi(-a), a >= 0,
// and R a polynomial in t = 1 / (1 + 0.35 a) times t, whose coefficients were
// fitted to R over 0 <= a <= 14.5 for the least relative error (3.9e-8 with the
// constants as binary32 has them).  On the device, over every binary32 a up to 13,
// the tail is within 4.2e-7 of itself and exp(-a^2 / 2) within 1.4e-7.
// Exponentials below 2^-126 come as zero, as the instruction gives them: silu is
// zero below -87.3 (where it is -1e-36), gelu_tanh below -10.1 (-1e-37), gelu below
// -13.2 (-6e-39).  The library's erfc takes
// about five times the instructions (a gelu over 8192 x 11008 products of 4096,
// MXFP4, 362 us; silu 262).
#pragma once

#include <type_traits>

#include "fp4_device.hpp"
#include "fp4_internal.h"

namespace fp4 {

constexpr float kEpiLog2e = 1.44269504088896340736f;
constexpr float kTanhOuter = 1.59576912160573071176f;      // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// {s(x), s(-x)}, neither by a subtraction
struct Logistic { float up, down; };
__device__ __forceinline__ Logistic logistic(float x)
{
    const float t = __builtin_amdgcn_exp2f(-fabsf(x) * kEpiLog2e), r = __builtin_amdgcn_rcpf(1.0f + t), l = t * r;
    return x >= 0.0f || x != x ? Logistic{r, l} : Logistic{l, r};
}

// {Phi(-|v|), exp(-v^2 / 2)}; nothing of either is left in binary32 past 16
struct Tail { float phi, e; };
__device__ __forceinline__ Tail normal_tail(float v)
{
    const float a = fminf(fabsf(v), 16.0f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, a, 1.0f));
    float r = -0.029157895594835f;
    r = __builtin_fmaf(r, t, 0.144030973315239f);
    r = __builtin_fmaf(r, t, -0.255839109420776f);
    r = __builtin_fmaf(r, t, 0.159319803118706f);
    r = __builtin_fmaf(r, t, -0.023212423548102f);
    r = __builtin_fmaf(r, t, 0.105552531778812f);
    r = __builtin_fmaf(r, t, 0.119821280241013f);
    r = __builtin_fmaf(r, t, 0.139863520860672f);
    r = __builtin_fmaf(r, t, 0.139621302485466f);
    // exp(-a^2 / 2): the square's and the product's roundings put back
    constexpr float k = -0.72134752044448170368f, klo = (float)(-0.72134752044448170368 - (double)k);
    const float s = a * a, lo = __builtin_fmaf(a, a, -s), x = s * k;
    const float left = __builtin_fmaf(s, k, -x) + __builtin_fmaf(lo, k, s * klo);
    float e = __builtin_amdgcn_exp2f(x);
    e = __builtin_fmaf(e, left * 0.69314718055994530942f, e);
    return Tail{e * (t * r), e};
}
__device__ __forceinline__ float normal_cdf(float v, const Tail& t) { return v >= 0.0f ? 1.0f - t.phi : t.phi; }

template <int ACT>
__device__ __forceinline__ float act_value(float v)
{
    if (ACT == kActRelu) return v < 0.0f ? 0.0f : v;         // NaN stays NaN
    if (ACT == kActSilu) return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kEpiLog2e));
    if (ACT == kActGelu) return v * normal_cdf(v, normal_tail(v));
    if (ACT == kActGeluTanh) {
        const float u = kTanhOuter * __builtin_fmaf(kTanhCubic * v * v, v, v);
        return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u * kEpiLog2e));
    }
    return v;
}

// The derivative.  gelu_tanh's is 0 or 1 in every bit of binary32 past |v| =
// 30, where its polynomials would overflow against a zero.
template <int ACT>
__device__ __forceinline__ float act_slope(float v)
{
    if (ACT == kActRelu) return v <= 0.0f ? 0.0f : 1.0f;
    if (ACT == kActSilu) {
        const Logistic s = logistic(v);
        return __builtin_fmaf(v * s.up, s.down, s.up);
    }
    if (ACT == kActGelu) {
        const Tail t = normal_tail(v);
        return __builtin_fmaf(v * 0.39894228040143267794f, t.e, normal_cdf(v, t));
    }
    if (ACT == kActGeluTanh) {
        const float x = v > 30.0f ? 30.0f : v < -30.0f ? -30.0f : v;
        const float q = kTanhCubic * x * x;
        const Logistic s = logistic(kTanhOuter * __builtin_fmaf(q, x, x));
        return __builtin_fmaf(x * s.up * s.down, kTanhOuter * __builtin_fmaf(3.0f, q, 1.0f), s.up);
    }
    return 1.0f;
}

// f(std::integral_constant<int, ACT>) for a run-time activation: the choice is
// the same for every lane.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
    }
}

// W (1, 4 or 8) neighbouring bf16 elements: all of them in one load or store
// at whatever element they start (global memory takes wide accesses at any
// alignment here, at no cost to aligned ones), or the first n.
typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(2)));
template <int W>
using epi_vec = typename std::conditional<W == 8, u4_any, u2_any>::type;

template <int W, bool PAST = false>
__device__ __forceinline__ void bf16_load(const uint16_t* p, int n, float (&o)[W])
{
    if (W > 1 && n >= W) {
        const epi_vec<W>* const q = reinterpret_cast<const epi_vec<W>*>(p);
        const epi_vec<W> v = PAST ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
        for (int i = 0; i < W / 2; ++i) { o[2 * i] = bf16_lo(v[i]); o[2 * i + 1] = bf16_hi(v[i]); }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) o[i] = i < n ? bf16_lo(p[i]) : 0.0f;
    }
}
template <int W, bool PAST = false>
__device__ __forceinline__ void bf16_store(uint16_t* p, int n, const float (&v)[W])
{
    if (W > 1 && n >= W) {
        epi_vec<W> o;
#pragma unroll
        for (int i = 0; i < W / 2; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        epi_vec<W>* const q = reinterpret_cast<epi_vec<W>*>(p);
        if (PAST) __builtin_nontemporal_store(o, q);
        else *q = o;
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (i < n) p[i] = (uint16_t)f32_to_bf16_rne(v[i]);
    }
}

__device__ __forceinline__ float epi_bias(const Epilogue& e, int64_t n)
{
    return e.bias_bf16 ? bf16_lo(((const uint16_t*)e.bias)[n]) : ((const float*)e.bias)[n];
}

// W outputs of row m from column n on, of N: `sum` the product, `bias` theirs
// (zeros without one).  PAST: rows that are read or written
// once, past the caches.
template <int W, bool PAST = false>
__device__ __forceinline__ void epi_put(const Epilogue& e, uint16_t* c, int64_t ldc, int64_t m, int64_t n, int64_t N,
                                        const float (&sum)[W], const float (&bias)[W])
{
    const int have = N - n < W ? (int)(N - n) : W;
    float v[W], mul[W], res[W];
    if (e.mul) bf16_load<W, PAST>(e.mul + m * e.ld_mul + n, have, mul);
    if (e.res) bf16_load<W, PAST>(e.res + m * e.ld_res + n, have, res);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = sum[i] + bias[i];
    if (e.pre) bf16_store<W, PAST>(e.pre + m * e.ld_pre + n, have, v);
    with_act(e.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = act_value<decltype(act)::value>(v[i]);
    });
    if (e.mul)
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] *= mul[i];
    if (e.res)
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] += res[i];
    bf16_store<W, PAST>(c + m * ldc + n, have, v);
}

}  // namespace fp4
