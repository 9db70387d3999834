// epilogue.hip -- the gradients of a product's epilogue y = res + mul act(v),
// v = product + bias, from the saved v (quant_prune_distill/574 and
// ue5m3-fp4-pretraining: the linear layers run in FP4; their layers' bias,
// activation and gate are the steps between two products).
//
//   dv = dy mul act'(v),  dmul = dy act(v),  dbias = sum over the rows of dv
//
// One pass: each element is read once and written once, in binary32 between.
// A workgroup owns a block of columns and a range of rows; its threads keep
// the columns' sums in registers over their rows, which join in LDS and then,
// one partial sum a workgroup, in a second launch, always in the same order.
#include <type_traits>

#include "epilogue_device.hpp"
#include "fp4_device.hpp"
#include "fp4_internal.h"

namespace fp4 {

// COLS columns of a workgroup, eight a thread.
template <int ACT, int COLS, int THREADS>
__global__ __launch_bounds__(THREADS) void k_epilogue_backward(EpiGradLaunch p, int64_t step)
{
    constexpr int CB = COLS / 8, ROWS = THREADS / CB;
    __shared__ float sums[ROWS][COLS + 1];
    const int tid = threadIdx.x, cb = tid % CB, r0 = tid / CB;
    const int64_t n = (int64_t)blockIdx.x * COLS + 8 * cb;
    const int64_t b = (int64_t)blockIdx.y * step, e = b + step < p.rows ? b + step : p.rows;
    const int have = n >= p.cols ? 0 : p.cols - n < 8 ? (int)(p.cols - n) : 8;
    float total[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) total[i] = 0.0f;
    if (have) {
#pragma unroll 2
        for (int64_t m = b + r0; m < e; m += ROWS) {
            float dy[8], v[8], mul[8], d[8];
            bf16_load<8>(p.dy + m * p.lddy + n, have, dy);
            if (ACT != kActNone || p.mul) bf16_load<8>(p.pre + m * p.ldpre + n, have, v);
            if (p.mul) bf16_load<8>(p.mul + m * p.ldmul + n, have, mul);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = dy[i];
                if (p.mul) d[i] *= mul[i];
                if (ACT != kActNone) d[i] *= act_slope<ACT>(v[i]);
                total[i] += d[i];                          // elements past the last are zeros
            }
            if (p.mul) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = dy[i] * act_value<ACT>(v[i]);
                bf16_store<8>(p.dmul + m * p.lddmul + n, have, v);
            }
            if (p.dpre) bf16_store<8>(p.dpre + m * p.lddpre + n, have, d);
        }
    }
    if (!p.dbias) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[r0][8 * cb + i] = total[i];
    __syncthreads();
    // rows in halves: always the same order
#pragma unroll
    for (int h = ROWS / 2; h >= 4; h /= 2) {
        for (int i = tid; i < h * COLS; i += THREADS) sums[i / COLS][i % COLS] += sums[i / COLS + h][i % COLS];
        __syncthreads();
    }
    const int64_t col = (int64_t)blockIdx.x * COLS + tid;
    if (tid >= COLS || col >= p.cols) return;
    const float s = (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
    (gridDim.y == 1 ? p.dbias : p.part + (int64_t)blockIdx.y * p.cols)[col] = s;
}

// 32 columns of a workgroup (one line of a partial sum's row), 32 threads a
// column: a narrow tensor has up to 1400 partial sums to join, and a thread a
// column would wait for them one after another.
__global__ __launch_bounds__(1024) void k_epilogue_join(const float* __restrict__ part, int64_t groups, int64_t cols,
                                                        float* __restrict__ out)
{
    __shared__ float sums[32][33];
    const int c = threadIdx.x % 32, r = threadIdx.x / 32;
    const int64_t col = (int64_t)blockIdx.x * 32 + c;
    float s = 0.0f;
    if (col < cols) {
#pragma unroll 8
        for (int64_t g = r; g < groups; g += 32) s += part[g * cols + col];
    }
    sums[r][c] = s;
    __syncthreads();
    if (r || col >= cols) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) s += sums[i][c];
    out[col] = s;
}

// The K ranges' partial sums of a product, joined in order, then its epilogue.
// Bound by memory: what the ranges' workgroups wrote is mostly still in the
// memory-side cache (1111 x 4096 in three ranges with a residual, 12.5 us).  Through the caches, unlike whole tiles: these products are
// small, and the next call reads their outputs there.
__global__ __launch_bounds__(256) void k_epilogue_product(GemmEpiLaunch p)
{
    const int64_t eights = p.ldp / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= p.m * eights) return;
    const int64_t m = i / eights, n = 8 * (i % eights);
    const int64_t from = m * p.ldp + n, step = p.m * p.ldp;
    float sum[8], bias[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        sum[j] = 0.0f;
        bias[j] = p.ep.bias && n + j < p.n ? epi_bias(p.ep, n + j) : 0.0f;
    }
#pragma unroll 4
    for (int64_t s = 0; s < p.splits; ++s) {
        const float4* const q = reinterpret_cast<const float4*>(p.part + s * step + from);
        const float4 a = q[0], b = q[1];
        sum[0] += a.x; sum[1] += a.y; sum[2] += a.z; sum[3] += a.w;
        sum[4] += b.x; sum[5] += b.y; sum[6] += b.z; sum[7] += b.w;
    }
    epi_put<8>(p.ep, p.c, p.ldc, m, n, p.n, sum, bias);
}

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

hipError_t launch_epilogue_join(const GemmEpiLaunch& p, hipStream_t s)
{
    hipLaunchKernelGGL(k_epilogue_product, dim3((unsigned)cdiv(p.m * (p.ldp / 8), 256)), dim3(256), 0, s, p);
    return hipGetLastError();
}

// Few rows take one launch, with workgroups of 64 columns over all of them;
// more are cut into ranges, about 1400 workgroups of 512 columns, whose sums a
// second launch joins. A row's piece of 512 columns is 1 KiB of each tensor in
// order, and a workgroup has eight such rows in flight: 8192 x 11008 with a
// multiplier 191 us (4.7 TB/s), 8192 x 11008 without one 116, 8000 x 5003 118,
// 4096 x 4096 39, against 215, 131, 135 and 41 with 2048 workgroups of 256
// columns and 256 threads (1024 of 1024 columns: 210, 127, 131, 41; stores
// past the caches changed none by more than 2 us).  One launch against ranges
// and their join, silu with a multiplier and sums, us a call in a graph:
//              x 256        x 1027       x 4096       x 11008
//   130 rows   5.4   7.8    8.0  13.5    5.8   8.3    8.2  11.4
//   256        6.5   8.7    8.3  16.0    7.0   9.4    9.2  12.7
//   512        9.8   8.9    14.2 16.1    12.5 12.6    14.5 17.0
//   1024       17.1  9.1    27.2 16.3    20.7 13.9    29.6 27.9
// so that the bound is late for the last of these.
constexpr int64_t kEgFewRows = 1024, kEgGroups = 1400;
constexpr int kEgCols = 512, kEgFewCols = 64;
int64_t epilogue_groups(int64_t rows, int64_t cols)
{
    if (rows <= kEgFewRows) return 1;
    const int64_t g = cdiv(kEgGroups, cdiv(cols, kEgCols)), most = cdiv(rows, 32);
    return g < most ? g : most;
}

template <int ACT>
static void run(const EpiGradLaunch& p, int64_t step, hipStream_t s)
{
    if (p.rows <= kEgFewRows)
        hipLaunchKernelGGL((k_epilogue_backward<ACT, kEgFewCols, 1024>), dim3((unsigned)cdiv(p.cols, kEgFewCols)), dim3(1024), 0, s,
                           p, step);
    else
        hipLaunchKernelGGL((k_epilogue_backward<ACT, kEgCols, kEgCols>), dim3((unsigned)cdiv(p.cols, kEgCols), (unsigned)p.groups),
                           dim3(kEgCols), 0, s, p, step);
}

hipError_t launch_epilogue_backward(const EpiGradLaunch& in, hipStream_t s)
{
    EpiGradLaunch p = in;
    const int64_t step = cdiv(p.rows, p.groups) > 0 ? cdiv(p.rows, p.groups) : 1;
    p.groups = p.rows ? cdiv(p.rows, step) : 1;
    switch (p.act) {
    case kActRelu: run<kActRelu>(p, step, s); break;
    case kActSilu: run<kActSilu>(p, step, s); break;
    case kActGelu: run<kActGelu>(p, step, s); break;
    case kActGeluTanh: run<kActGeluTanh>(p, step, s); break;
    default: run<kActNone>(p, step, s); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.dbias || p.groups == 1) return e;
    hipLaunchKernelGGL(k_epilogue_join, dim3((unsigned)cdiv(p.cols, 32)), dim3(1024), 0, s, p.part, p.groups, p.cols, p.dbias);
    return hipGetLastError();
}

}  // namespace fp4
