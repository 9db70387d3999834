// norm.hip -- the norms before and after a block, fused with its gate and
// its residual scale (quant_prune_distill/574 "Метод": the RMSNorms around
// the FP4 products carry the exploration noise in their weights, so a model
// trained that way calls them with fresh weights every step).
//
//   u = RMSNorm(x) w_post     (u = x without a post norm)
//   h = alpha r + gate u      (one gate per row, 1 without)
//   n = RMSNorm(h) w_pre
// with RMSNorm(v) = v rho(v), rho(v) = 1 / sqrt(mean v^2 + eps).  n comes
// from the unrounded h.  Backward, with rho1 = rho(x), rho2 = rho(h) kept
// from the forward call and C columns:
//   t  = dh + rho2 (dn w_pre) - h rho2^3 / C sum(dn w_pre h)
//   dr = alpha t,  dgate = q = sum(t u),  dw_pre = sum_rows dn h rho2
//   dx = rho1 w_post gate t - x rho1^2 gate q / C,  dw_post = sum_rows gate t x rho1
//
// Memory bound: a row stays with its workgroup between its loads and its
// stores, so that every tensor crosses memory once (the backward pass of rows
// above 16384 columns reads twice).  8192 x 4096, bf16 over a binary32 stream:
// forward 403 MB in 73 us, 5.5 TB/s, where a large copy reaches 5.2.  It stays in
// registers up to 32768 columns forward (16384 where rows are not whole aligned
// vectors), 8192 (2048) backward; past them a part of it lies in scratch.
#include "fp4_device.hpp"
#include "fp4_internal.h"

namespace fp4 {

typedef int v4i __attribute__((ext_vector_type(4)));

// Eight elements of a row at `i` (VEC), or elements i + j * stride below n.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* row, int64_t i, int stride, int64_t n, float (&o)[8])
{
    if (VEC) {
        if (i >= n) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0.0f;
        } else if (BF16) {
            const v4i v = *reinterpret_cast<const v4i*>((const uint16_t*)row + i);
#pragma unroll
            for (int q = 0; q < 4; ++q) { o[2 * q] = bf16_lo((uint32_t)v[q]); o[2 * q + 1] = bf16_hi((uint32_t)v[q]); }
        } else {
            const v4i* const p = reinterpret_cast<const v4i*>((const float*)row + i);
            const v4i a = p[0], b = p[1];
#pragma unroll
            for (int q = 0; q < 4; ++q) { o[q] = bits_f((uint32_t)a[q]); o[4 + q] = bits_f((uint32_t)b[q]); }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t at = i + (int64_t)j * stride;
            o[j] = at >= n ? 0.0f : BF16 ? bits_f((uint32_t)((const uint16_t*)row)[at] << 16) : ((const float*)row)[at];
        }
    }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void* row, int64_t i, int stride, int64_t n, const float (&o)[8])
{
    if (VEC) {
        if (i >= n) return;
        if (BF16) {
            v4i v;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = (int)pack_bf16(o[2 * q], o[2 * q + 1]);
            *reinterpret_cast<v4i*>((uint16_t*)row + i) = v;
        } else {
            v4i* const p = reinterpret_cast<v4i*>((float*)row + i);
            p[0] = v4i{(int)f_bits(o[0]), (int)f_bits(o[1]), (int)f_bits(o[2]), (int)f_bits(o[3])};
            p[1] = v4i{(int)f_bits(o[4]), (int)f_bits(o[5]), (int)f_bits(o[6]), (int)f_bits(o[7])};
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t at = i + (int64_t)j * stride;
            if (at >= n) continue;
            if (BF16) ((uint16_t*)row)[at] = (uint16_t)f32_to_bf16_rne(o[j]);
            else ((float*)row)[at] = o[j];
        }
    }
}

// The weights' type is one of the call's, uniform over the launch.
template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int bf16, int64_t i, int stride, int64_t n, float (&o)[8])
{
    if (bf16) load8<true, VEC>(w, i, stride, n, o);
    else load8<false, VEC>(w, i, stride, n, o);
}

// Sum over the T threads of a row, the same on all; `buf` alternates between
// the calls so that one barrier each is enough.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* buf)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if (T == 64) return v;
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) v += buf[w];
    return v;
}

template <bool XB>
__device__ __forceinline__ const void* row_at(const void* p, int64_t off)
{
    return (const uint8_t*)p + off * (XB ? 2 : 4);
}

template <bool XB, bool RB, bool VEC, int T, int NV>
__global__ __launch_bounds__(T) void k_norm(NormLaunch p)
{
    __shared__ float red[2][T / 64];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x, C = p.cols;
    const int st = VEC ? 1 : T;
    float x[NV][8], h[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t i = VEC ? ((int64_t)v * T + tid) * 8 : (int64_t)v * 8 * T + tid;
        load8<XB, VEC>(row_at<XB>(p.x, row * p.ldx), i, st, C, x[v]);
        load8<RB, VEC>(row_at<RB>(p.res, row * p.ldres), i, st, C, h[v]);
    }
    const float gate = p.gate ? p.gate[row] : 1.0f;
    float r1 = 1.0f;
    if (p.w_post) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(x[v][j], x[v][j], ss);
        r1 = 1.0f / sqrtf(row_sum<T>(ss, red[0]) / (float)C + p.eps);
    }
    ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t i = VEC ? ((int64_t)v * T + tid) * 8 : (int64_t)v * 8 * T + tid;
        float w[8];
        if (p.w_post) load_weight<VEC>(p.w_post, p.w_bf16, i, st, C, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = p.w_post ? x[v][j] * r1 * w[j] : x[v][j];
            h[v][j] = __builtin_fmaf(gate, u, p.alpha * h[v][j]);
            ss = __builtin_fmaf(h[v][j], h[v][j], ss);
        }
        store8<RB, VEC>((void*)row_at<RB>(p.h, row * p.ldh), i, st, C, h[v]);
    }
    const float r2 = 1.0f / sqrtf(row_sum<T>(ss, red[1]) / (float)C + p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int64_t i = VEC ? ((int64_t)v * T + tid) * 8 : (int64_t)v * 8 * T + tid;
        float w[8];
        load_weight<VEC>(p.w_pre, p.w_bf16, i, st, C, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= h[v][j] * r2;
        store8<XB, VEC>((void*)row_at<XB>(p.n, row * p.ldn), i, st, C, w);
    }
    if (tid == 0) {
        p.stats[2 * row] = r1;
        p.stats[2 * row + 1] = r2;
    }
}

// Rows blockIdx.x, + gridDim.x, ...  The weights' gradients of a workgroup's
// rows collect in LDS (each thread its own columns) and leave as one partial
// row each: in registers they would halve the rows in flight, and the two row
// sums' barriers would leave memory idle.  8192 x 4096, bf16 over a binary32
// stream (604 MB): 131 us, 4.6 TB/s; 157 us with the sums in registers and
// two waves a SIMD.
template <bool XB, bool RB, bool VEC, int T, int NV>
__global__ __launch_bounds__(T, 4) void k_norm_backward(NormGradLaunch p)
{
    __shared__ float red[2][T / 64];
    extern __shared__ __align__(16) float sums[];         // [1 or 2][NV][8][T]: conflict-free across a wave
    const NormLaunch& f = p.f;
    const int tid = threadIdx.x;
    const int64_t C = f.cols;
    const int st = VEC ? 1 : T;
    const bool pre = p.sums & 1, post = p.sums & 2;       // which weights' sums this launch takes
    float* const a2 = sums + tid;
    float* const a1 = sums + (pre ? NV * 8 * T : 0) + tid;
    auto col = [&](int v) { return VEC ? ((int64_t)v * T + tid) * 8 : (int64_t)v * 8 * T + tid; };
#pragma unroll
    for (int e = 0; e < 8 * NV; ++e) {
        if (pre) a2[e * T] = 0.0f;
        if (post) a1[e * T] = 0.0f;
    }
    const float inv_c = 1.0f / (float)C;
    for (int64_t row = blockIdx.x; row < f.rows; row += gridDim.x) {
        const float r1 = f.stats[2 * row], r2 = f.stats[2 * row + 1];
        const float gate = f.gate ? f.gate[row] : 1.0f;
        float x[NV][8], h[NV][8], t[NV][8], q[NV][8];      // x becomes x rho1, q = dn w_pre
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            load8<XB, VEC>(row_at<XB>(f.x, row * f.ldx), col(v), st, C, x[v]);
            load8<RB, VEC>(row_at<RB>(f.res, row * f.ldres), col(v), st, C, h[v]);
            if (p.dn) load8<XB, VEC>(row_at<XB>(p.dn, row * p.lddn), col(v), st, C, q[v]);
            if (p.dh) load8<RB, VEC>(row_at<RB>(p.dh, row * p.lddh), col(v), st, C, t[v]);
            if (!p.dn || !p.dh) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (!p.dn) q[v][j] = 0.0f;
                    if (!p.dh) t[v][j] = 0.0f;
                }
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w1[8], w2[8];
            if (f.w_post) load_weight<VEC>(f.w_post, f.w_bf16, col(v), st, C, w1);
            load_weight<VEC>(f.w_pre, f.w_bf16, col(v), st, C, w2);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[v][j] *= r1;                             // rho1 is 1 without a post norm
                const float u = f.w_post ? x[v][j] * w1[j] : x[v][j];
                h[v][j] = __builtin_fmaf(gate, u, f.alpha * h[v][j]);
                if (pre) a2[(8 * v + j) * T] += q[v][j] * (h[v][j] * r2);
                q[v][j] *= w2[j];
                s = __builtin_fmaf(q[v][j], h[v][j], s);
            }
        }
        const float k2 = row_sum<T>(s, red[0]) * r2 * r2 * r2 * inv_c;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w1[8], d[8];
            if (f.w_post) load_weight<VEC>(f.w_post, f.w_bf16, col(v), st, C, w1);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                t[v][j] = __builtin_fmaf(-k2, h[v][j], __builtin_fmaf(r2, q[v][j], t[v][j]));
                s = __builtin_fmaf(t[v][j], f.w_post ? x[v][j] * w1[j] : x[v][j], s);
                d[j] = f.alpha * t[v][j];
                t[v][j] *= gate;
                if (post) a1[(8 * v + j) * T] += t[v][j] * x[v][j];
            }
            if (pre) store8<RB, VEC>((void*)row_at<RB>(p.dres, row * p.lddres), col(v), st, C, d);
        }
        const float dg = row_sum<T>(s, red[1]);
        const float k1 = gate * dg * inv_c;
        if (!pre) continue;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float w1[8];
            if (f.w_post) {
                load_weight<VEC>(f.w_post, f.w_bf16, col(v), st, C, w1);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[v][j] = r1 * __builtin_fmaf(-k1, x[v][j], w1[j] * t[v][j]);
            }
            store8<XB, VEC>((void*)row_at<XB>(p.dx, row * p.lddx), col(v), st, C, t[v]);
        }
        if (tid == 0 && p.dgate) p.dgate[row] = dg;
    }
    float* const o2 = p.part + (int64_t)blockIdx.x * p.part_rows * C;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float d[8];
        if (pre) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = a2[(8 * v + j) * T];
            store8<false, VEC>(o2, col(v), st, C, d);
        }
        if (post) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = a1[(8 * v + j) * T];
            store8<false, VEC>(o2 + C, col(v), st, C, d);
        }
    }
}

// Column sums of the partial rows in a fixed order: 32 columns a workgroup,
// 32 threads down each, joined through LDS.
__global__ __launch_bounds__(1024) void k_norm_join(const float* part, int64_t groups, int64_t width, float* out0,
                                                    float* out1, int64_t cols)
{
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, down = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < width) {
#pragma unroll 4
        for (int64_t g = down; g < groups; g += 32) s += part[g * width + c];
    }
    red[down][lane] = s;
    __syncthreads();
    if (down == 0 && c < width) {
        s = 0.0f;
#pragma unroll
        for (int d = 0; d < 32; ++d) s += red[d][lane];
        if (c < cols) out0[c] = s;
        else out1[c - cols] = s;
    }
}

// ---------------------------------------------------------------------------
// launch shapes
// ---------------------------------------------------------------------------
template <bool XB, bool RB, bool VEC, int T, int NV>
static hipError_t run_norm(const NormLaunch& p, hipStream_t s)
{
    hipLaunchKernelGGL((k_norm<XB, RB, VEC, T, NV>), dim3((unsigned)p.rows), dim3(T), 0, s, p);
    return hipGetLastError();
}

template <bool XB, bool RB, bool VEC, int T, int NV>
static hipError_t run_norm_rows(const NormGradLaunch& p, size_t lds, hipStream_t s)
{
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_norm_backward<XB, RB, VEC, T, NV>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_norm_backward<XB, RB, VEC, T, NV>), dim3((unsigned)p.groups), dim3(T), lds, s, p);
    return hipGetLastError();
}

template <bool XB, bool RB, bool VEC, int T, int NV>
static hipError_t run_norm(const NormGradLaunch& in, hipStream_t s)
{
    NormGradLaunch p = in;
    constexpr size_t one = sizeof(float) * 8 * NV * T;
    // the widest rows' two sums do not fit the LDS together: a first launch
    // takes w_post's and writes nothing else (so that the outputs may still
    // lie on the inputs), the second everything else
    if (2 * one > 144 * 1024 && p.f.w_post) {
        p.sums = 2;
        const hipError_t e = run_norm_rows<XB, RB, VEC, T, NV>(p, one, s);
        if (e != hipSuccess) return e;
        p.sums = 1;
    } else {
        p.sums = p.f.w_post ? 3 : 1;
    }
    const hipError_t e = run_norm_rows<XB, RB, VEC, T, NV>(p, p.sums == 3 ? 2 * one : one, s);
    if (e != hipSuccess) return e;
    const int64_t width = p.part_rows * p.f.cols;
    hipLaunchKernelGGL(k_norm_join, dim3((unsigned)((width + 31) / 32)), dim3(1024), 0, s, p.part, p.groups, width,
                       p.dw_pre, p.dw_post, p.f.cols);
    return hipGetLastError();
}

// Threads for a row.  Forward: sixteen elements a thread from 2048 columns on
// (fewer waves to join for each sum).
template <bool XB, bool RB, bool VEC>
static hipError_t norm_by_cols(const NormLaunch& p, int64_t cols, hipStream_t s)
{
    if (cols <= 512) return run_norm<XB, RB, VEC, 64, 1>(p, s);
    if (cols <= 2048) return run_norm<XB, RB, VEC, 256, 1>(p, s);
    if (cols <= 4096) return run_norm<XB, RB, VEC, 256, 2>(p, s);
    if (cols <= 8192) return run_norm<XB, RB, VEC, 512, 2>(p, s);
    if (cols <= 16384) return run_norm<XB, RB, VEC, 1024, 2>(p, s);
    return run_norm<XB, RB, VEC, 1024, 4>(p, s);
}

// Backward: eight elements a thread as far as that goes: four operands of
// sixteen do not fit four waves on a SIMD, and spill.  8192 rows, bf16 over
// binary32: 5120 columns 191 us (4.0 TB/s), 8192 256 (4.7), 12288 517 (3.5); 4096 rows
// of 18432 2562 (0.5).  Rows that are not whole aligned vectors: 8192 x 4095
// 289 us (2.1 TB/s), 8191 558 (2.2), 12287 1408 (1.3).
template <bool XB, bool RB, bool VEC>
static hipError_t norm_by_cols(const NormGradLaunch& p, int64_t cols, hipStream_t s)
{
    if (cols <= 512) return run_norm<XB, RB, VEC, 64, 1>(p, s);
    if (cols <= 2048) return run_norm<XB, RB, VEC, 256, 1>(p, s);
    if (cols <= 4096) return run_norm<XB, RB, VEC, 512, 1>(p, s);
    if (cols <= 8192) return run_norm<XB, RB, VEC, 1024, 1>(p, s);
    if (cols <= 16384) return run_norm<XB, RB, VEC, 1024, 2>(p, s);
    return run_norm<XB, RB, VEC, 1024, 4>(p, s);
}

template <typename P>
static hipError_t norm_by_type(const P& p, const NormLaunch& f, bool vec, hipStream_t s)
{
    if (f.x_bf16) {
        if (f.res_bf16) return vec ? norm_by_cols<true, true, true>(p, f.cols, s) : norm_by_cols<true, true, false>(p, f.cols, s);
        return vec ? norm_by_cols<true, false, true>(p, f.cols, s) : norm_by_cols<true, false, false>(p, f.cols, s);
    }
    if (f.res_bf16) return vec ? norm_by_cols<false, true, true>(p, f.cols, s) : norm_by_cols<false, true, false>(p, f.cols, s);
    return vec ? norm_by_cols<false, false, true>(p, f.cols, s) : norm_by_cols<false, false, false>(p, f.cols, s);
}

// Workgroups of a backward call, each with one partial row of the weights'
// gradients: as many as run at once (four waves on each SIMD).
int64_t norm_groups(int64_t rows, int64_t cols)
{
    const int64_t most = cols <= 2048 ? 1024 : cols <= 4096 ? 512 : 256;
    return rows < 1 ? 1 : rows < most ? rows : most;
}

// vec: every row of every tensor starts on a 16-byte boundary and holds
// whole vectors of eight elements.
hipError_t launch_norm(const NormLaunch& p, bool vec, hipStream_t s) { return norm_by_type(p, p, vec, s); }
hipError_t launch_norm_backward(const NormGradLaunch& p, bool vec, hipStream_t s) { return norm_by_type(p, p.f, vec, s); }

}  // namespace fp4
