// api_layer.cpp -- the C ABI's products with an epilogue, mixture-of-experts
// and distillation calls: argument validation, workspace layout and kernel
// launches on the caller's stream.
#include "fp4.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_checks.h"
#include "fp4_internal.h"

using namespace fp4;

namespace {

// Rows [m, cols] of bf16 at any element.
fp4_status check_plain_rows(const void* p, int64_t ld, int64_t m, int64_t cols)
{
    if (!p) return m && cols ? FP4_ERR_INVALID_ARG : FP4_OK;
    if (ld < cols) return FP4_ERR_SHAPE;
    if (ld > kMaxElems / (m ? m : 1)) return FP4_ERR_UNSUPPORTED;
    return aligned(p, 2) ? FP4_OK : FP4_ERR_ALIGN;
}

bool act_ok(int32_t a) { return a >= FP4_ACT_NONE && a <= FP4_ACT_GELU_TANH; }

fp4_status check_epilogue(const fp4_epilogue* e, const uint16_t* y, int64_t ldy, int64_t m, int64_t n, Epilogue* out)
{
    if (!e || !act_ok(e->act)) return FP4_ERR_INVALID_ARG;
    if (e->bias && !dtype_ok(e->bias_dtype)) return FP4_ERR_INVALID_ARG;
    if (e->pre && (e->pre == y || e->pre == e->mul || e->pre == e->residual)) return FP4_ERR_INVALID_ARG;
    fp4_status st = check_plain_rows(y, ldy, m, n);
    if (st != FP4_OK) return st;
    if (e->mul && (st = check_plain_rows(e->mul, e->ld_mul, m, n)) != FP4_OK) return st;
    if (e->residual && (st = check_plain_rows(e->residual, e->ld_residual, m, n)) != FP4_OK) return st;
    if (e->pre && (st = check_plain_rows(e->pre, e->ld_pre, m, n)) != FP4_OK) return st;
    // in place means the same rows: another stride would let one row's output
    // overwrite another's input
    if ((e->mul == y && e->ld_mul != ldy) || (e->residual == y && e->ld_residual != ldy)) return FP4_ERR_SHAPE;
    if (e->bias && !aligned(e->bias, (uintptr_t)esize(e->bias_dtype))) return FP4_ERR_ALIGN;
    *out = Epilogue{};
    out->bias = e->bias; out->bias_bf16 = e->bias_dtype == FP4_DTYPE_BF16;
    out->act = e->act;
    out->mul = e->mul; out->ld_mul = e->ld_mul;
    out->res = e->residual; out->ld_res = e->ld_residual;
    out->pre = e->pre; out->ld_pre = e->ld_pre;
    return FP4_OK;
}

constexpr int64_t kMaxGradCols = int64_t(1) << 24;

// One side of the experts: `rows` of each expert's matrix.
fp4_status check_experts(const fp4_tensor* t, const float* scale, int64_t experts, int64_t rows, MoeWeights* w)
{
    if (t->rows != experts * rows || t->cols % 128) return FP4_ERR_SHAPE;
    if (t->fmt.transform != FP4_TRANSFORM_NONE) return FP4_ERR_UNSUPPORTED;   // x would need the same transform
    const int64_t bits = elem_is_8bit(t->fmt.element) ? 8 : elem_is_6bit(t->fmt.element) ? 6 : 4;
    w->expert_q = rows * (t->cols * bits / 8);
    w->expert_s = rows * (t->cols / t->fmt.block);
    // the kernels address an expert's matrix with 32-bit byte offsets
    if (w->expert_q >= (int64_t(1) << 32)) return FP4_ERR_UNSUPPORTED;
    if (!aligned16(t->q) || ((uintptr_t)t->scales & 3u) || !aligned(scale, 4)) return FP4_ERR_ALIGN;
    w->q = t->q; w->s = t->scales; w->g = t->tensor_scale;
    w->scale = scale;
    w->block = t->fmt.block; w->elem = t->fmt.element;
    return FP4_OK;
}

constexpr int64_t kMaxExperts = 65535;
constexpr int64_t kMaxDistillVocab = int64_t(1) << 24;    // 64 pieces of kDsMost: a lane of the join for each

fp4_status check_distill(const void* z, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab, const int32_t* ids,
                         const float* logprobs, int32_t top, float temperature, int32_t rest)
{
    const fp4_status st = check_logits(z, dtype, ld, rows, vocab, temperature);
    if (st != FP4_OK) return st;
    if (rest != FP4_DISTILL_BUCKET && rest != FP4_DISTILL_RENORMALIZE) return FP4_ERR_INVALID_ARG;
    if (top < 1) return FP4_ERR_SHAPE;
    if (top > kDistillMaxTop || vocab > kMaxDistillVocab) return FP4_ERR_UNSUPPORTED;
    if (rows && (!ids || !logprobs)) return FP4_ERR_INVALID_ARG;
    return aligned(ids, 4) && aligned(logprobs, 4) ? FP4_OK : FP4_ERR_ALIGN;
}

}  // namespace

extern "C" {

int64_t fp4_gemm_epilogue_workspace(const fp4_tensor* a, const fp4_tensor* b)
{
    GemmEpiLaunch p{};
    uint16_t* const any = reinterpret_cast<uint16_t*>(uintptr_t(16));     // y takes no part in it
    const fp4_status st = check_gemm(a, b, any, b ? b->rows : 0, &p);
    if (st != FP4_OK) return st;
    if (a->rows == 0 || b->rows == 0 || a->cols == 0) return 0;
    return epi::gemm_split(&p);
}

fp4_status fp4_gemm_epilogue(const fp4_tensor* a, const fp4_tensor* b, const fp4_epilogue* e, uint16_t* y, int64_t ldy,
                             void* workspace, int64_t workspace_bytes, void* stream)
{
    GemmEpiLaunch p{};
    fp4_status st = check_gemm(a, b, y, ldy, &p);
    if (st != FP4_OK) return st;
    if (a->cols == 0) return FP4_ERR_SHAPE;
    if ((st = check_epilogue(e, y, ldy, a->rows, b->rows, &p.ep)) != FP4_OK) return st;
    if (a->rows == 0 || b->rows == 0) return FP4_OK;
    const bool mx = gemm_is_mx(p), mx16 = !mx && gemm_mx16_supported(p);
    if (!mx && !mx16 && !gemm_dq_supported(p.fa, p.fb, p.elem)) return FP4_ERR_UNSUPPORTED;
    if ((st = check_space(workspace, workspace_bytes, epi::gemm_split(&p))) != FP4_OK) return st;
    p.part = (float*)workspace;
    hipStream_t s = (hipStream_t)stream;
    if (gemm_small_supported(p)) return hip_status(epi::launch_gemm_small(p, s));
    st = hip_status(mx ? epi::launch_gemm_mx(p, s) : mx16 ? epi::launch_gemm_mx16(p, s) : epi::launch_gemm_dq(p, s));
    if (st != FP4_OK || p.splits == 1) return st;
    return hip_status(launch_epilogue_join(p, s));
}

fp4_status fp4_wo_gemm_epilogue(const uint16_t* x, int64_t ldx, int64_t m, const fp4_tensor* w, const fp4_epilogue* e,
                                uint16_t* y, int64_t ldy, void* stream)
{
    WoEpiLaunch p{};
    fp4_status st = check_wo_gemm(x, ldx, m, w, y, ldy, &p);
    if (st != FP4_OK) return st;
    if (w->rows == 0 || w->cols == 0) return FP4_ERR_SHAPE;
    if ((st = check_epilogue(e, y, ldy, m, w->rows, &p.ep)) != FP4_OK) return st;
    if (e->pre) return FP4_ERR_UNSUPPORTED;              // a serving call: nothing is kept for a backward pass
    if (y == x) return FP4_ERR_INVALID_ARG;              // every workgroup reads all of x (y may be a residual, x is none here)
    return hip_status(epi::launch_wo_gemm(p, (hipStream_t)stream));
}

int64_t fp4_epilogue_workspace(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1) return FP4_ERR_SHAPE;
    if (cols > kMaxGradCols || rows > kMaxElems / cols) return FP4_ERR_UNSUPPORTED;
    const int64_t groups = epilogue_groups(rows, cols);
    return groups == 1 ? 0 : up16(4 * groups * cols);
}

fp4_status fp4_epilogue_backward(const uint16_t* dy, int64_t ld_dy, const uint16_t* pre, int64_t ld_pre,
                                 const uint16_t* mul, int64_t ld_mul, int64_t rows, int64_t cols, int32_t act,
                                 uint16_t* dpre, int64_t ld_dpre, uint16_t* dmul, int64_t ld_dmul, float* dbias,
                                 void* workspace, int64_t workspace_bytes, void* stream)
{
    if (!act_ok(act)) return FP4_ERR_INVALID_ARG;
    const int64_t need = fp4_epilogue_workspace(rows, cols);
    if (need < 0) return (fp4_status)need;
    fp4_status st = check_plain_rows(dy, ld_dy, rows, cols);
    if (st != FP4_OK) return st;
    const bool reads = act != FP4_ACT_NONE || mul;
    // without either the gradient of v is dy itself, and only the bias's sum is left to do
    if (rows && reads && (!dpre || !pre)) return FP4_ERR_INVALID_ARG;
    if (rows && mul && !dmul) return FP4_ERR_INVALID_ARG;
    if (reads && (st = check_plain_rows(pre, ld_pre, rows, cols)) != FP4_OK) return st;
    if (mul && (st = check_plain_rows(mul, ld_mul, rows, cols)) != FP4_OK) return st;
    if (dpre && (st = check_plain_rows(dpre, ld_dpre, rows, cols)) != FP4_OK) return st;
    if (mul && (st = check_plain_rows(dmul, ld_dmul, rows, cols)) != FP4_OK) return st;
    if (rows && mul && dpre == dmul) return FP4_ERR_INVALID_ARG;
    const struct { const uint16_t* p; int64_t ld; } in[3] = {{dy, ld_dy}, {reads ? pre : nullptr, ld_pre}, {mul, ld_mul}};
    for (const auto& i : in)
        if (i.p && ((dpre == i.p && ld_dpre != i.ld) || (mul && dmul == i.p && ld_dmul != i.ld))) return FP4_ERR_SHAPE;
    if (!aligned(dbias, 4)) return FP4_ERR_ALIGN;
    if (dbias && (st = check_space(workspace, workspace_bytes, need)) != FP4_OK) return st;
    if (!dbias && (rows == 0 || (!dpre && !mul))) return FP4_OK;
    EpiGradLaunch p{};
    p.dy = dy; p.lddy = ld_dy; p.pre = pre; p.ldpre = ld_pre; p.mul = mul; p.ldmul = ld_mul;
    p.rows = rows; p.cols = cols; p.act = act;
    p.dpre = dpre; p.lddpre = ld_dpre; p.dmul = mul ? dmul : nullptr; p.lddmul = ld_dmul;
    p.dbias = dbias;
    p.part = (float*)workspace;
    p.groups = epilogue_groups(rows, cols);
    return hip_status(launch_epilogue_backward(p, (hipStream_t)stream));
}

// ---------------------------------------------------------------------------
fp4_status fp4_moe_route(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t experts, int32_t top,
                         int32_t score, const float* bias, int32_t renormalize, float scale, int32_t* ids, float* weights,
                         void* stream)
{
    if (!dtype_ok(dtype) || (score != FP4_ROUTE_SOFTMAX && score != FP4_ROUTE_SIGMOID) || !isfinite(scale))
        return FP4_ERR_INVALID_ARG;
    if (rows < 0 || experts < 1 || ld < experts || top < 1 || top > experts) return FP4_ERR_SHAPE;
    if (rows >= kMaxLineRows || experts > kMoeMaxRouted || top > kMoeMaxTop || ld > kMaxElems / (rows ? rows : 1))
        return FP4_ERR_UNSUPPORTED;
    if (rows && (!logits || !ids || !weights)) return FP4_ERR_INVALID_ARG;
    if (!aligned(logits, (uintptr_t)esize(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return FP4_ERR_ALIGN;
    if (rows == 0) return FP4_OK;
    RouteLaunch p{};
    p.logits = logits; p.bf16 = dtype == FP4_DTYPE_BF16; p.ld = ld; p.rows = rows;
    p.experts = (int32_t)experts; p.top = top;
    p.sigmoid = score == FP4_ROUTE_SIGMOID; p.renormalize = renormalize != 0;
    p.bias = bias; p.scale = scale;
    p.ids = ids; p.weights = weights;
    return hip_status(launch_moe_route(p, (hipStream_t)stream));
}

int64_t fp4_moe_workspace(int64_t m, int32_t top, int64_t ffn)
{
    if (m < 0 || top < 1 || ffn < 1) return FP4_ERR_SHAPE;
    if (m > kMoeMaxTokens || top > kMoeMaxTop || ffn > kMaxElems) return FP4_ERR_UNSUPPORTED;
    return up16(4 * m * top * ffn);
}

fp4_status fp4_moe(const uint16_t* x, int64_t ldx, int64_t m, const fp4_moe_bank* bank, const int32_t* ids,
                   const float* weights, int32_t top, int32_t act, const uint16_t* residual, int64_t ld_residual,
                   uint16_t* y, int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream)
{
    MoeLaunch p{};
    if (!bank) return FP4_ERR_INVALID_ARG;
    fp4_status st = check_tensor(&bank->gate_up, &p.up.fmt);
    if (st != FP4_OK) return st;
    if ((st = check_tensor(&bank->down, &p.down.fmt)) != FP4_OK) return st;
    if (!act_ok(act) || !x || !y || !ids || !weights) return FP4_ERR_INVALID_ARG;
    if (m < 1 || m > kMoeMaxTokens || top > kMoeMaxTop || bank->experts > kMaxExperts) return FP4_ERR_UNSUPPORTED;
    const int64_t hidden = bank->gate_up.cols, ffn = bank->down.cols, experts = bank->experts;
    if (top < 1 || experts < 1 || hidden < 1 || ffn < 1) return FP4_ERR_SHAPE;
    if (hidden > kMaxElems || ffn > kMaxElems) return FP4_ERR_UNSUPPORTED;     // the products below stay far from 63 bits
    if ((st = check_experts(&bank->gate_up, bank->up_scale, experts, 2 * ffn, &p.up)) != FP4_OK) return st;
    if ((st = check_experts(&bank->down, bank->down_scale, experts, hidden, &p.down)) != FP4_OK) return st;
    if (ldx < hidden || ldy < hidden || (residual && ld_residual < hidden)) return FP4_ERR_SHAPE;
    if (ldx > kMaxElems / m || ldy > kMaxElems / m || (residual && ld_residual > kMaxElems / m)) return FP4_ERR_UNSUPPORTED;
    if (residual == y && ld_residual != ldy) return FP4_ERR_SHAPE;
    if (!aligned16(x) || (m > 1 && ldx % 8) || !aligned(y, 2) || !aligned(residual, 2) || !aligned(ids, 4) || !aligned(weights, 4))
        return FP4_ERR_ALIGN;
    const int64_t need = fp4_moe_workspace(m, top, ffn);
    if (need < 0) return (fp4_status)need;
    if ((st = check_space(workspace, workspace_bytes, need)) != FP4_OK) return st;
    p.x = x; p.ldx = ldx; p.m = (int32_t)m; p.top = top; p.experts = (int32_t)experts;
    p.ids = ids; p.weights = weights;
    p.hidden = hidden; p.ffn = ffn;
    p.act = act;
    p.h = (uint16_t*)workspace;
    p.res = residual; p.ldres = ld_residual; p.y = y; p.ldy = ldy;
    return hip_status(launch_moe(p, (hipStream_t)stream));
}

// ---------------------------------------------------------------------------
int64_t fp4_distill_workspace(int64_t rows, int64_t vocab, int32_t dtype)
{
    if (!dtype_ok(dtype)) return FP4_ERR_INVALID_ARG;
    if (rows < 0 || vocab < 1) return FP4_ERR_SHAPE;
    if (rows >= kMaxLineRows || vocab > kMaxDistillVocab) return FP4_ERR_UNSUPPORTED;
    const int64_t pieces = distill_pieces(rows, vocab, esize(dtype));
    return pieces == 1 ? 0 : up16(8 * rows * pieces);
}

fp4_status fp4_distill_loss(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                            const int32_t* top_ids, const float* top_logprobs, int32_t top, float temperature, int32_t rest,
                            float* loss, float* stats, void* workspace, int64_t workspace_bytes, void* stream)
{
    fp4_status st = check_distill(logits, dtype, ld, rows, vocab, top_ids, top_logprobs, top, temperature, rest);
    if (st != FP4_OK) return st;
    if (rows && (!loss || !stats)) return FP4_ERR_INVALID_ARG;
    if (!aligned(loss, 4) || !aligned(stats, 4)) return FP4_ERR_ALIGN;
    if ((st = check_space(workspace, workspace_bytes, fp4_distill_workspace(rows, vocab, dtype))) != FP4_OK) return st;
    if (rows == 0) return FP4_OK;
    DistillLaunch p{};
    p.logits = logits; p.bf16 = dtype == FP4_DTYPE_BF16; p.ld = ld; p.rows = rows; p.vocab = vocab;
    p.ids = top_ids; p.logprobs = top_logprobs; p.top = top;
    p.inv_temperature = 1.0f / temperature; p.renormalize = rest == FP4_DISTILL_RENORMALIZE;
    p.loss = loss; p.stats = stats;
    p.part = (float*)workspace;
    return hip_status(launch_distill(p, distill_pieces(rows, vocab, esize(dtype)), (hipStream_t)stream));
}

fp4_status fp4_distill_loss_backward(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                                     const int32_t* top_ids, const float* top_logprobs, int32_t top, float temperature,
                                     int32_t rest, const float* stats, const float* grad_loss, void* dlogits, int64_t ld_d,
                                     void* stream)
{
    const fp4_status st = check_distill(logits, dtype, ld, rows, vocab, top_ids, top_logprobs, top, temperature, rest);
    if (st != FP4_OK) return st;
    if (rows && (!stats || !grad_loss || !dlogits)) return FP4_ERR_INVALID_ARG;
    if (ld_d < vocab || (rows && dlogits == logits && ld_d != ld)) return FP4_ERR_SHAPE;
    if (ld_d > kMaxElems / (rows ? rows : 1)) return FP4_ERR_UNSUPPORTED;
    if (!aligned(dlogits, (uintptr_t)esize(dtype)) || !aligned(stats, 4) || !aligned(grad_loss, 4)) return FP4_ERR_ALIGN;
    if (rows == 0) return FP4_OK;
    DistillGradLaunch p{};
    p.logits = logits; p.bf16 = dtype == FP4_DTYPE_BF16; p.ld = ld; p.rows = rows; p.vocab = vocab;
    p.ids = top_ids; p.logprobs = top_logprobs; p.top = top;
    p.inv_temperature = 1.0f / temperature;
    p.stats = stats; p.g_loss = grad_loss;
    p.dlogits = dlogits; p.ldd = ld_d;
    return hip_status(launch_distill_backward(p, (hipStream_t)stream));
}

}  // extern "C"
