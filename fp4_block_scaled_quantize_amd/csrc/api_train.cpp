// api_train.cpp -- the C ABI's adapter, token-probability and residual-norm
// calls: argument validation, workspace layout and kernel launches on the
// caller's stream.
#include "fp4.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_checks.h"
#include "fp4_internal.h"

using namespace fp4;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 20;        // rows of an adapter call (grid dimensions)
constexpr int64_t kMaxAdapters = 16384;
constexpr int64_t kMaxDim = int64_t(1) << 24;         // k and n of a bank
constexpr int32_t kMaxRank = 128, kMaxTop = 32;
constexpr int64_t kMaxNormCols = 32768;


// The bank itself; n % 8 only where rows of n elements are read as vectors.
fp4_status check_bank(const fp4_lora_bank* b, bool vector_n)
{
    if (!b || !b->a || !b->b || !b->scale) return FP4_ERR_INVALID_ARG;
    if (b->adapters < 1 || b->rank < 1 || b->k < 1 || b->n < 1) return FP4_ERR_SHAPE;
    if (b->rank % 8 || b->k % 8 || (vector_n && b->n % 8)) return FP4_ERR_SHAPE;
    if (b->rank > kMaxRank || b->adapters > kMaxAdapters || b->k > kMaxDim || b->n > kMaxDim)
        return FP4_ERR_UNSUPPORTED;
    if (!aligned(b->a, 16) || !aligned(b->b, 16) || !aligned(b->scale, 4)) return FP4_ERR_ALIGN;
    return FP4_OK;
}

// Rows [m, cols] of bf16 read or written as 16-byte vectors.
fp4_status check_rows(const void* p, int64_t ld, int64_t m, int64_t cols)
{
    if (!p && m) return FP4_ERR_INVALID_ARG;
    if (ld < cols) return FP4_ERR_SHAPE;
    if (!aligned(p, 16) || ld % 8) return FP4_ERR_ALIGN;
    if (ld > kMaxElems / (m ? m : 1)) return FP4_ERR_UNSUPPORTED;
    return FP4_OK;
}

// Byte offsets of an adapter call's workspace.
struct LoraSpace {
    LoraDownShape down;
    int64_t outer_splits = 1;
    int64_t t = -1;                      // partial sums of T (apply, weight-only) or dT
    int64_t dt = -1, at = -1, bt = -1, part0 = -1, part1 = -1, flags = -1;   // backward
    int64_t bytes = 0;
    int64_t take(int64_t b)
    {
        const int64_t at_ = bytes;
        bytes += up16(b);
        return at_;
    }
};

LoraSpace lora_space(int32_t call, int64_t m, int64_t n, int64_t k, int64_t rank, int64_t adapters)
{
    LoraSpace w;
    const bool back = call == FP4_LORA_BACKWARD;
    const int64_t rows = m > 0 ? m : 1;
    w.down = lora_down_shape(rows, back ? n : k, (int)rank, adapters);
    if (w.down.splits > 1 || call == FP4_LORA_WO_GEMM) w.t = w.take(4 * w.down.splits * m * rank);
    if (back) {
        w.dt = w.take(4 * m * rank);
        if (!lora_across(m, k, rank)) {
            w.at = w.take(2 * adapters * rank * k);
            w.bt = w.take(2 * adapters * rank * n);
        }
        w.outer_splits = lora_outer_splits(m, n, k, (int)rank, adapters);
        if (w.outer_splits > 1) {
            w.part0 = w.take(4 * w.outer_splits * adapters * rank * k);
            w.part1 = w.take(4 * w.outer_splits * adapters * rank * n);
            w.flags = w.take(4 * w.outer_splits * adapters);
        }
    }
    return w;
}

template <typename T>
T* at(void* ws, int64_t off) { return off < 0 ? nullptr : reinterpret_cast<T*>((uint8_t*)ws + off); }

LoraDown down_of(const uint16_t* x, int64_t ldx, int64_t m, int64_t k, const uint16_t* a, const fp4_lora_bank* b,
                 const int32_t* slots, const float* scale, float* t)
{
    LoraDown d{};
    d.x = x; d.ldx = ldx; d.m = m; d.k = k;
    d.a = a; d.adapters = b->adapters; d.rank = (int32_t)b->rank;
    d.slots = slots; d.scale = scale; d.t = t;
    return d;
}

fp4_status check_slots(const int32_t* slots, int64_t m)
{
    if (!slots && m) return FP4_ERR_INVALID_ARG;
    return aligned(slots, 4) ? FP4_OK : FP4_ERR_ALIGN;
}

}  // namespace

extern "C" {

int64_t fp4_lora_workspace(int32_t call, int64_t m, int64_t n, int64_t k, int64_t rank, int64_t adapters)
{
    if (call < FP4_LORA_APPLY || call > FP4_LORA_WO_GEMM) return FP4_ERR_INVALID_ARG;
    if (m < 0 || n < 1 || k < 1 || rank < 1 || adapters < 1) return FP4_ERR_SHAPE;
    if (m > kMaxRows || n > kMaxDim || k > kMaxDim || rank > kMaxRank || adapters > kMaxAdapters)
        return FP4_ERR_UNSUPPORTED;
    return lora_space(call, m, n, k, rank, adapters).bytes;
}

fp4_status fp4_lora_apply(const uint16_t* x, int64_t ldx, int64_t m, const fp4_lora_bank* bank, const int32_t* slots,
                          const uint16_t* base, int64_t ld_base, uint16_t* y, int64_t ldy, float* t, void* workspace,
                          int64_t workspace_bytes, void* stream)
{
    fp4_status st = check_bank(bank, true);
    if (st != FP4_OK) return st;
    if (m < 0) return FP4_ERR_SHAPE;
    if (m > kMaxRows) return FP4_ERR_UNSUPPORTED;
    if ((st = check_slots(slots, m)) != FP4_OK) return st;
    if ((st = check_rows(x, ldx, m, bank->k)) != FP4_OK) return st;
    if ((st = check_rows(y, ldy, m, bank->n)) != FP4_OK) return st;
    if (base && (st = check_rows(base, ld_base, m, bank->n)) != FP4_OK) return st;
    // in place means the same rows: another stride would let one row's
    // output overwrite another's base
    if (base && base == y && ld_base != ldy) return FP4_ERR_SHAPE;
    if (!t && m) return FP4_ERR_INVALID_ARG;
    if (!aligned(t, 16)) return FP4_ERR_ALIGN;
    const LoraSpace w = lora_space(FP4_LORA_APPLY, m, bank->n, bank->k, bank->rank, bank->adapters);
    if ((st = check_space(workspace, workspace_bytes, w.bytes)) != FP4_OK) return st;
    if (m == 0) return FP4_OK;
    hipStream_t s = (hipStream_t)stream;
    float* const parts = w.down.splits > 1 ? at<float>(workspace, w.t) : t;
    st = hip_status(launch_lora_down(down_of(x, ldx, m, bank->k, bank->a, bank, slots, nullptr, parts), w.down, s));
    if (st != FP4_OK) return st;
    LoraUp u{};
    u.t = parts; u.splits = (int32_t)w.down.splits; u.m = m; u.n = bank->n;
    u.b = bank->b; u.adapters = bank->adapters; u.rank = (int32_t)bank->rank;
    u.slots = slots; u.scale = bank->scale;
    u.base = base; u.ldbase = ld_base; u.y = y; u.ldy = ldy;
    u.t_out = w.down.splits > 1 ? t : nullptr;
    return hip_status(launch_lora_up(u, s));
}

fp4_status fp4_lora_backward(const uint16_t* dy, int64_t ld_dy, const uint16_t* x, int64_t ldx, int64_t m,
                             const float* t, const fp4_lora_bank* bank, const int32_t* slots, const uint16_t* dx_base,
                             int64_t ld_dx_base, uint16_t* dx, int64_t ld_dx, void* da, void* db, int32_t grad_dtype,
                             void* workspace, int64_t workspace_bytes, void* stream)
{
    fp4_status st = check_bank(bank, true);
    if (st != FP4_OK) return st;
    if (!dtype_ok(grad_dtype)) return FP4_ERR_INVALID_ARG;
    if (m < 0) return FP4_ERR_SHAPE;
    if (m > kMaxRows) return FP4_ERR_UNSUPPORTED;
    if ((st = check_slots(slots, m)) != FP4_OK) return st;
    if ((st = check_rows(dy, ld_dy, m, bank->n)) != FP4_OK) return st;
    if ((st = check_rows(x, ldx, m, bank->k)) != FP4_OK) return st;
    if ((st = check_rows(dx, ld_dx, m, bank->k)) != FP4_OK) return st;
    if (dx_base && (st = check_rows(dx_base, ld_dx_base, m, bank->k)) != FP4_OK) return st;
    if (dx_base && dx_base == dx && ld_dx_base != ld_dx) return FP4_ERR_SHAPE;
    // the gradient sums read x and dy after dx is written
    if (m && (dx == x || dx == dy)) return FP4_ERR_INVALID_ARG;
    if ((!t && m) || !da || !db) return FP4_ERR_INVALID_ARG;
    if (!aligned(t, 16) || !aligned(da, 16) || !aligned(db, 16)) return FP4_ERR_ALIGN;
    const LoraSpace w = lora_space(FP4_LORA_BACKWARD, m, bank->n, bank->k, bank->rank, bank->adapters);
    if ((st = check_space(workspace, workspace_bytes, w.bytes)) != FP4_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    float* const dt = at<float>(workspace, w.dt);
    if (m > 0) {
        const bool across = lora_across(m, bank->k, bank->rank);
        uint16_t* const a_t = at<uint16_t>(workspace, w.at);
        uint16_t* const b_t = at<uint16_t>(workspace, w.bt);
        if (!across) {
            st = hip_status(launch_lora_transpose(bank->a, a_t, bank->b, b_t, bank->adapters, bank->rank, bank->k, bank->n, s));
            if (st != FP4_OK) return st;
        }
        // dT = s dy B
        float* const parts = w.down.splits > 1 ? at<float>(workspace, w.t) : dt;
        LoraDown d = down_of(dy, ld_dy, m, bank->n, across ? bank->b : b_t, bank, slots, bank->scale, parts);
        d.across = across;
        st = hip_status(launch_lora_down(d, w.down, s));
        if (st != FP4_OK) return st;
        // dx = base + dT A
        LoraUp u{};
        u.t = parts; u.splits = (int32_t)w.down.splits; u.m = m; u.n = bank->k;
        u.b = across ? bank->a : a_t; u.across = across; u.adapters = bank->adapters; u.rank = (int32_t)bank->rank;
        u.slots = slots;
        u.base = dx_base; u.ldbase = ld_dx_base; u.y = dx; u.ldy = ld_dx;
        u.t_out = w.down.splits > 1 ? dt : nullptr;
        st = hip_status(launch_lora_up(u, s));
        if (st != FP4_OK) return st;
    }
    LoraOuter o{};
    o.job[0] = {x, ldx, bank->k, dt, nullptr, da, 0, at<float>(workspace, w.part0)};
    o.job[1] = {dy, ld_dy, bank->n, t, bank->scale, db, 1, at<float>(workspace, w.part1)};
    o.m = m; o.rank = (int32_t)bank->rank; o.adapters = bank->adapters;
    o.slots = slots;
    o.out_bf16 = grad_dtype == FP4_DTYPE_BF16;
    o.flags = at<uint32_t>(workspace, w.flags);
    return hip_status(launch_lora_outer(o, w.outer_splits, s));
}

fp4_status fp4_wo_gemm_lora(const uint16_t* x, int64_t ldx, int64_t m, const fp4_tensor* w, const fp4_lora_bank* bank,
                            const int32_t* slots, uint16_t* y, int64_t ldy, void* workspace, int64_t workspace_bytes,
                            void* stream)
{
    WoGemmLaunch p;
    fp4_status st = check_wo_gemm(x, ldx, m, w, y, ldy, &p);
    if (st != FP4_OK) return st;
    // an empty product has no adapter to add to it
    if (w->rows == 0 || w->cols == 0) return FP4_ERR_SHAPE;
    if ((st = check_bank(bank, false)) != FP4_OK) return st;
    if (bank->k != w->cols || bank->n != w->rows) return FP4_ERR_SHAPE;
    if ((st = check_slots(slots, m)) != FP4_OK) return st;
    const LoraSpace sp = lora_space(FP4_LORA_WO_GEMM, m, bank->n, bank->k, bank->rank, bank->adapters);
    if ((st = check_space(workspace, workspace_bytes, sp.bytes)) != FP4_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    float* const t = at<float>(workspace, sp.t);
    st = hip_status(launch_lora_down(down_of(x, ldx, m, bank->k, bank->a, bank, slots, nullptr, t), sp.down, s));
    if (st != FP4_OK) return st;
    p.ad = {t, (int32_t)sp.down.splits, (int32_t)bank->rank, bank->b, bank->scale, slots, bank->adapters};
    return hip_status(launch_wo_gemm(p, s));
}

// ---------------------------------------------------------------------------
int64_t fp4_token_logprobs_workspace(int64_t rows, int64_t vocab, int32_t top)
{
    if (rows < 0 || vocab < 1) return FP4_ERR_SHAPE;
    if (top < 0 || top > kMaxTop || rows >= kMaxLineRows || vocab >= (int64_t(1) << 27)) return FP4_ERR_UNSUPPORTED;
    const int64_t pieces = logprob_pieces(rows, vocab);
    return pieces == 1 ? 0 : rows * pieces * (16 + 8 * (int64_t)top);
}

fp4_status fp4_token_logprobs(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                              const int64_t* tokens, float temperature, int32_t top, float* logprob, float* entropy,
                              float* stats, int32_t* top_ids, float* top_logprobs, void* workspace,
                              int64_t workspace_bytes, void* stream)
{
    fp4_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (st != FP4_OK) return st;
    if (top < 0 || top > kMaxTop) return FP4_ERR_UNSUPPORTED;
    if (top > vocab) return FP4_ERR_SHAPE;
    if (rows && (!entropy || !stats || (tokens && !logprob) || (top && (!top_ids || !top_logprobs))))
        return FP4_ERR_INVALID_ARG;
    if (!aligned(tokens, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(stats, 4) ||
        !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
        return FP4_ERR_ALIGN;
    const int64_t pieces = logprob_pieces(rows, vocab);
    if ((st = check_space(workspace, workspace_bytes, fp4_token_logprobs_workspace(rows, vocab, top))) != FP4_OK)
        return st;
    if (rows == 0) return FP4_OK;
    LogprobLaunch p{};
    p.logits = logits; p.bf16 = dtype == FP4_DTYPE_BF16; p.ld = ld; p.rows = rows; p.vocab = vocab;
    p.tokens = tokens;
    p.inv_temperature = 1.0f / temperature;
    p.top = top;
    p.logprob = logprob; p.entropy = entropy; p.stats = stats;
    p.top_ids = top_ids; p.top_logprobs = top_logprobs;
    p.part_sums = (float*)workspace;
    p.part_keys = pieces > 1 ? (uint64_t*)((uint8_t*)workspace + 16 * rows * pieces) : nullptr;
    return hip_status(launch_logprobs(p, pieces, (hipStream_t)stream));
}

fp4_status fp4_token_logprobs_backward(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                                       const int64_t* tokens, float temperature, const float* entropy,
                                       const float* stats, const float* grad_logprob, const float* grad_entropy,
                                       void* dlogits, int64_t ld_d, void* stream)
{
    fp4_status st = check_logits(logits, dtype, ld, rows, vocab, temperature);
    if (st != FP4_OK) return st;
    if (rows && (!entropy || !stats || !dlogits)) return FP4_ERR_INVALID_ARG;
    if (grad_logprob && !tokens && rows) return FP4_ERR_INVALID_ARG;
    if (ld_d < vocab || (rows && dlogits == logits && ld_d != ld)) return FP4_ERR_SHAPE;
    if (ld_d > kMaxElems / (rows ? rows : 1)) return FP4_ERR_UNSUPPORTED;
    if (!aligned(dlogits, (uintptr_t)esize(dtype)) || !aligned(tokens, 8) || !aligned(entropy, 4) ||
        !aligned(stats, 4) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4))
        return FP4_ERR_ALIGN;
    if (rows == 0) return FP4_OK;
    LogprobGradLaunch p{};
    p.logits = logits; p.bf16 = dtype == FP4_DTYPE_BF16; p.ld = ld; p.rows = rows; p.vocab = vocab;
    p.tokens = tokens;
    p.inv_temperature = 1.0f / temperature;
    p.entropy = entropy; p.stats = stats;
    p.g_logprob = grad_logprob; p.g_entropy = grad_entropy;
    p.dlogits = dlogits; p.ldd = ld_d;
    return hip_status(launch_logprobs_backward(p, (hipStream_t)stream));
}

// ---------------------------------------------------------------------------
// The tensor's rows, and whether they can be read as 16-byte vectors.
static fp4_status check_norm_rows(const void* p, int32_t dtype, int64_t ld, int64_t rows, int64_t cols, bool* vec)
{
    if (ld < cols) return FP4_ERR_SHAPE;
    if (ld > kMaxElems / (rows ? rows : 1)) return FP4_ERR_UNSUPPORTED;
    if (!aligned(p, (uintptr_t)esize(dtype))) return FP4_ERR_ALIGN;
    if (!aligned(p, 16) || (rows > 1 && ld * esize(dtype) % 16)) *vec = false;
    return FP4_OK;
}

static fp4_status check_norm(const fp4_norm* a, NormLaunch* p, bool* vec)
{
    if (!a) return FP4_ERR_INVALID_ARG;
    if (!dtype_ok(a->x_dtype) || !dtype_ok(a->res_dtype) || !dtype_ok(a->weight_dtype)) return FP4_ERR_INVALID_ARG;
    if (!isfinite(a->alpha) || !isfinite(a->eps) || a->eps < 0.0f) return FP4_ERR_INVALID_ARG;
    if (a->rows < 0 || a->cols < 1) return FP4_ERR_SHAPE;
    if (a->cols > kMaxNormCols || a->rows >= kMaxLineRows) return FP4_ERR_UNSUPPORTED;
    if (!a->w_pre || (a->rows && (!a->x || !a->res))) return FP4_ERR_INVALID_ARG;
    *vec = a->cols % 8 == 0;
    fp4_status st = check_norm_rows(a->x, a->x_dtype, a->ld_x, a->rows, a->cols, vec);
    if (st != FP4_OK) return st;
    if ((st = check_norm_rows(a->res, a->res_dtype, a->ld_res, a->rows, a->cols, vec)) != FP4_OK) return st;
    if ((st = check_norm_rows(a->w_pre, a->weight_dtype, a->cols, 1, a->cols, vec)) != FP4_OK) return st;
    if ((st = check_norm_rows(a->w_post, a->weight_dtype, a->cols, 1, a->cols, vec)) != FP4_OK) return st;
    if (!aligned(a->gate, 4)) return FP4_ERR_ALIGN;
    *p = NormLaunch{};
    p->x = a->x; p->ldx = a->ld_x; p->res = a->res; p->ldres = a->ld_res;
    p->x_bf16 = a->x_dtype == FP4_DTYPE_BF16;
    p->res_bf16 = a->res_dtype == FP4_DTYPE_BF16;
    p->w_bf16 = a->weight_dtype == FP4_DTYPE_BF16;
    p->rows = a->rows; p->cols = a->cols;
    p->w_pre = a->w_pre; p->w_post = a->w_post; p->gate = a->gate;
    p->alpha = a->alpha; p->eps = a->eps;
    return FP4_OK;
}

fp4_status fp4_residual_norm(const fp4_norm* args, void* h, int64_t ld_h, void* n, int64_t ld_n, float* stats,
                             void* stream)
{
    NormLaunch p;
    bool vec;
    fp4_status st = check_norm(args, &p, &vec);
    if (st != FP4_OK) return st;
    if (args->rows && (!h || !n || !stats)) return FP4_ERR_INVALID_ARG;
    if ((st = check_norm_rows(h, args->res_dtype, ld_h, args->rows, args->cols, &vec)) != FP4_OK) return st;
    if ((st = check_norm_rows(n, args->x_dtype, ld_n, args->rows, args->cols, &vec)) != FP4_OK) return st;
    if (!aligned(stats, 4)) return FP4_ERR_ALIGN;
    if (args->rows == 0) return FP4_OK;
    if ((h == args->res && ld_h != args->ld_res) || (n == args->x && ld_n != args->ld_x)) return FP4_ERR_SHAPE;
    p.h = h; p.ldh = ld_h; p.n = n; p.ldn = ld_n;
    p.stats = stats;
    return hip_status(launch_norm(p, vec, (hipStream_t)stream));
}

int64_t fp4_residual_norm_workspace(int64_t rows, int64_t cols, int32_t post)
{
    if (rows < 0 || cols < 1) return FP4_ERR_SHAPE;
    if (cols > kMaxNormCols || rows >= kMaxLineRows) return FP4_ERR_UNSUPPORTED;
    return up16(4 * norm_groups(rows, cols) * (post ? 2 : 1) * cols);
}

fp4_status fp4_residual_norm_backward(const fp4_norm* args, const float* stats, const void* dn, int64_t ld_dn,
                                      const void* dh, int64_t ld_dh, void* dx, int64_t ld_dx, void* dres,
                                      int64_t ld_dres, float* dw_pre, float* dw_post, float* dgate, void* workspace,
                                      int64_t workspace_bytes, void* stream)
{
    NormGradLaunch p{};
    bool vec;
    fp4_status st = check_norm(args, &p.f, &vec);
    if (st != FP4_OK) return st;
    const int64_t rows = args->rows, cols = args->cols;
    if (!dw_pre || (args->w_post && !dw_post) || (rows && (!stats || !dx || !dres || (args->gate && !dgate))))
        return FP4_ERR_INVALID_ARG;
    if (dn && (st = check_norm_rows(dn, args->x_dtype, ld_dn, rows, cols, &vec)) != FP4_OK) return st;
    if (dh && (st = check_norm_rows(dh, args->res_dtype, ld_dh, rows, cols, &vec)) != FP4_OK) return st;
    if ((st = check_norm_rows(dx, args->x_dtype, ld_dx, rows, cols, &vec)) != FP4_OK) return st;
    if ((st = check_norm_rows(dres, args->res_dtype, ld_dres, rows, cols, &vec)) != FP4_OK) return st;
    if (!aligned(stats, 4) || !aligned(dw_pre, 4) || !aligned(dw_post, 4) || !aligned(dgate, 4)) return FP4_ERR_ALIGN;
    if (rows && ((dx == args->x && ld_dx != args->ld_x) || (dx == dn && ld_dx != ld_dn) || (dres == dh && ld_dres != ld_dh) ||
        (dres == args->res && ld_dres != args->ld_res)))
        return FP4_ERR_SHAPE;
    if ((st = check_space(workspace, workspace_bytes, fp4_residual_norm_workspace(rows, cols, args->w_post != nullptr))) !=
        FP4_OK)
        return st;
    p.f.stats = const_cast<float*>(stats);
    p.dn = dn; p.lddn = ld_dn; p.dh = dh; p.lddh = ld_dh;
    p.dx = dx; p.lddx = ld_dx; p.dres = dres; p.lddres = ld_dres;
    p.dw_pre = dw_pre; p.dw_post = args->w_post ? dw_post : nullptr;
    p.dgate = args->gate ? dgate : nullptr;
    p.part = (float*)workspace;
    p.part_rows = args->w_post ? 2 : 1;
    p.groups = norm_groups(rows, cols);
    return hip_status(launch_norm_backward(p, vec, (hipStream_t)stream));
}

}  // extern "C"
