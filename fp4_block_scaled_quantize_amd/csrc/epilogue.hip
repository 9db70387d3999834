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

constexpr int kEgThreads = 256;
constexpr int kEgCols = 256;           // columns of a workgroup: 32 threads of eight
constexpr int kEgRows = kEgThreads / (kEgCols / 8);

template <int ACT>
__global__ __launch_bounds__(kEgThreads) void k_epilogue_backward(EpiGradLaunch p, int64_t step)
{
    __shared__ float sums[kEgRows][kEgCols];
    const int tid = threadIdx.x, cb = tid % (kEgCols / 8), r0 = tid / (kEgCols / 8);
    const int64_t n = (int64_t)blockIdx.x * kEgCols + 8 * cb;
    const int64_t b = (int64_t)blockIdx.y * step, e = b + step < p.rows ? b + step : p.rows;
    const bool full = p.vec && n + 8 <= p.cols;
    const int have = n >= p.cols ? 0 : p.cols - n < 8 ? (int)(p.cols - n) : 8;
    float total[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) total[i] = 0.0f;
    if (have) {
#pragma unroll 2
        for (int64_t m = b + r0; m < e; m += kEgRows) {
            float dy[8], v[8], mul[8], d[8];
            bf16_load<8>(p.dy + m * p.lddy + n, full, have, dy);
            if (ACT != kActNone || p.mul) bf16_load<8>(p.pre + m * p.ldpre + n, full, have, v);
            if (p.mul) bf16_load<8>(p.mul + m * p.ldmul + n, full, have, mul);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = dy[i];
                if (p.mul) d[i] *= mul[i];
                if (ACT != kActNone) d[i] *= act_slope<ACT>(v[i]);
                if (i < have) total[i] += d[i];
            }
            if (p.mul) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = dy[i] * act_value<ACT>(v[i]);
                bf16_store<8>(p.dmul + m * p.lddmul + n, full, have, v);
            }
            if (p.dpre) bf16_store<8>(p.dpre + m * p.lddpre + n, full, have, d);
        }
    }
    if (!p.dbias) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[r0][8 * cb + i] = total[i];
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * kEgCols + tid;
    if (col >= p.cols) return;
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kEgRows; ++r) s += sums[r][tid];
    (gridDim.y == 1 ? p.dbias : p.part + (int64_t)blockIdx.y * p.cols)[col] = s;
}

__global__ __launch_bounds__(256) void k_epilogue_join(const float* __restrict__ part, int64_t groups, int64_t cols,
                                                       float* __restrict__ out)
{
    const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (col >= cols) return;
    float s = 0.0f;
#pragma unroll 8
    for (int64_t g = 0; g < groups; ++g) s += part[g * cols + col];
    out[col] = s;
}

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row ranges: about 2048 workgroups, none with fewer than 32 rows.
int64_t epilogue_groups(int64_t rows, int64_t cols)
{
    const int64_t blocks = cdiv(cols, kEgCols);
    int64_t g = cdiv(2048, blocks), most = cdiv(rows, 32);
    g = g < most ? g : most;
    return g < 1 ? 1 : g;
}

template <int ACT>
static void run(const EpiGradLaunch& p, int64_t step, hipStream_t s)
{
    const dim3 grid((unsigned)cdiv(p.cols, kEgCols), (unsigned)p.groups);
    hipLaunchKernelGGL((k_epilogue_backward<ACT>), grid, dim3(kEgThreads), 0, s, p, step);
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
    hipLaunchKernelGGL(k_epilogue_join, dim3((unsigned)cdiv(p.cols, 256)), dim3(256), 0, s, p.part, p.groups, p.cols, p.dbias);
    return hipGetLastError();
}

}  // namespace fp4
