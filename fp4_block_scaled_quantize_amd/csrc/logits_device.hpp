// logits_device.hpp -- a row's running softmax sums in powers of two, shared by
// the kernels that read logits (logprobs.hip, distill.hip).
#pragma once

#include "fp4_device.hpp"
#include "fp4_internal.h"

namespace fp4 {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
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

// Running sums in log2 units, about the maximum m (or -inf).
struct Sums { float m, s, w; };

constexpr float kLpFar = 1e8f;         // beyond it RN(m k) is more than 4 from m k, far beyond it infinite

// A thread's sums while it reads: about h = RN(m k) instead of m k, so that
// an element costs one fused product and no subtraction (h only has to be
// near the maximum); where m k is beyond kLpFar (a row of masks, a
// temperature near zero) the maximum is subtracted first instead.
struct Running {
    float m, h, s, w;
    __device__ __forceinline__ bool far(float k) const { return fabsf(m) * k > kLpFar && m != -INFINITY; }
    // raise the maximum to `to`
    __device__ __forceinline__ void raise(float to, float k)
    {
        if (!(to > m)) return;
        const bool was = far(k), first = m == -INFINITY;
        const float m1 = m, h1 = h;
        m = to;
        const bool now = far(k);
        h = now ? 0.0f : to * k;
        if (first) return;                             // nothing but zeros (or NaN) summed yet
        float d = h1 - h;
        if (was || now) d = was && now ? (m1 - to) * k : was ? __builtin_fmaf(m1, k, -h) : __builtin_fmaf(-to, k, h1);
        d = fmaxf(d, -1000.0f);
        const float f = __builtin_amdgcn_exp2f(d);
        w = f * __builtin_fmaf(d, s, w);
        s *= f;
    }
    template <bool FAR>
    __device__ __forceinline__ void add(float z, float k)
    {
        const float d = FAR ? (z - (m == -INFINITY ? 0.0f : m)) * k : __builtin_fmaf(z, k, -h);
        const float e = __builtin_amdgcn_exp2f(d);     // NaN stays NaN
        s += e;
        w = __builtin_fmaf(e, fmaxf(d, -1000.0f), w);  // 0 * -inf must not meet the sum
    }
    // the sums about m k itself
    __device__ __forceinline__ Sums about_max(float k) const
    {
        if (far(k) || m == -INFINITY) return Sums{m, s, w};
        const float d = __builtin_fmaf(m, k, -h), f = __builtin_amdgcn_exp2f(-d);
        return Sums{m, s * f, f * __builtin_fmaf(-d, s, w)};
    }
};

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

}  // namespace fp4
