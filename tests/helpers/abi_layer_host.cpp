// Drives the host side of the epilogue, mixture-of-experts and distillation
// calls (api_layer.cpp and the launch code of gemm.hip, gemm_epilogue.hip,
// moe.hip, epilogue.hip and distill.hip, their host pass only) with a stand-in
// for the HIP runtime, for a build with AddressSanitizer and
// UndefinedBehaviorSanitizer and no GPU.  Nothing is launched: hipLaunchKernel
// below looks at each launch instead.  Its grid must be one that the runtime
// takes and cover the work, and what it reads or writes of the workspace must
// lie in the bytes that the call asked for.  The addresses are never
// dereferenced.  Exit status: 0 and "ok", or an abort at the first launch or
// status that is wrong.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>

#include <hip/hip_runtime.h>

#include "fp4.h"
#include "fp4_internal.h"

namespace {

using namespace fp4;

std::string now;                                       // the call being made
[[noreturn]] void fail(const char* what)
{
    std::fprintf(stderr, "%s: %s\n", now.c_str(), what);
    std::abort();
}

// fake device addresses, 2^44 apart
void* place(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 44); }
constexpr int kSpace = 20;
uintptr_t space_at = 0, space_end = 0;
int launches = 0;
// kernels register before main, in an order of their own
std::map<const void*, std::string>& names()
{
    static std::map<const void*, std::string> all;
    return all;
}

void uses(const void* ptr, int64_t bytes, const char* name)
{
    const uintptr_t p = (uintptr_t)ptr;
    if (p != space_at || bytes < 0 || p + (uintptr_t)bytes > space_end) fail(name);
}

template <typename T>
const T& arg(void** args, int i = 0) { return *static_cast<const T*>(args[i]); }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

void look(const std::string& name, dim3 g, dim3 b, void** args)
{
    auto is = [&](const char* s) { return name.find(s) != std::string::npos; };
    if (is("k_gemm_small")) {
        const GemmEpiLaunch& p = arg<GemmEpiLaunch>(args);
        if (g.z != 1 || (int64_t)g.y * 32 < p.m || (int64_t)g.x * 32 * 4 < p.n) fail("small tiles");
    } else if (is("k_gemm_")) {
        const GemmEpiLaunch& p = arg<GemmEpiLaunch>(args);
        if ((int64_t)g.x * g.y != cdiv(p.m, 256) * cdiv(p.n, 256)) fail("tiles");
        if ((int64_t)g.z != p.splits || p.kstep * (p.splits - 1) >= p.k || p.kstep * p.splits < p.k) fail("K ranges");
        if (p.splits > 1) {
            // whole stages and groups of scales from a range to the next, and at least a stage in the last
            const int64_t step = is("k_gemm_mxILi") || is("k_gemm_mx16") ? 1024 : 128;
            if (p.kstep % step || (p.k - p.kstep * (p.splits - 1)) % 128) fail("ends of K ranges");
            if (p.ldp < p.n || p.ldp % 8) fail("rows of the partial sums");
            uses(p.part, 4 * p.splits * p.m * p.ldp, "partial sums");
        }
    } else if (is("k_epilogue_product")) {
        const GemmEpiLaunch& p = arg<GemmEpiLaunch>(args);
        uses(p.part, 4 * p.splits * p.m * p.ldp, "partial sums, joined");
        if ((int64_t)g.x * 256 < p.m * (p.ldp / 8)) fail("pieces");
    } else if (is("k_epilogue_backward")) {
        const EpiGradLaunch& p = arg<EpiGradLaunch>(args);
        const int64_t step = arg<int64_t>(args, 1);
        if ((int64_t)g.x * (b.x == 1024 ? 64 : 512) < p.cols || (int64_t)g.y * step < p.rows) fail("rows and columns");
        if (g.y > 1 && p.dbias) uses(p.part, 4 * (int64_t)g.y * p.cols, "partial column sums");
    } else if (is("k_epilogue_join")) {
        uses(arg<const float*>(args, 0), 4 * arg<int64_t>(args, 1) * arg<int64_t>(args, 2), "partial column sums, joined");
    } else if (is("k_moe_up") || is("k_moe_down")) {
        const MoeLaunch& p = arg<MoeLaunch>(args);
        uses(p.h, 4 * (int64_t)p.m * p.top * p.ffn, "hidden values");
        if (is("k_moe_up")) {
            if ((int64_t)g.x * 16 != p.ffn || (int64_t)g.y < (p.m * p.top < p.experts ? p.m * p.top : p.experts)) fail("columns, experts");
        } else if ((int64_t)g.x * 16 != p.hidden) fail("columns");
        if (b.x < 256) fail("a thread for each pair");
    } else if (is("k_moe_route")) {
        if ((int64_t)g.x != arg<RouteLaunch>(args).rows) fail("rows");
    } else if (is("k_distill_rows")) {
        const DistillLaunch& p = arg<DistillLaunch>(args);
        if ((int64_t)g.y * p.piece < p.vocab || ((int64_t)g.y - 1) * p.piece >= p.vocab || g.y > 64) fail("pieces of a row");
        if ((p.piece < p.vocab ? p.piece : p.vocab) > kDsMost + 63) fail("a piece's bitmap");
        if (g.y > 1) uses(p.part, 8 * p.rows * g.y, "partial sums");
    } else if (is("k_distill_join")) {
        uses(arg<DistillLaunch>(args).part, 8 * arg<DistillLaunch>(args).rows * arg<int>(args, 1), "partial sums, joined");
    } else if (is("k_distill_backward")) {
        const DistillGradLaunch& p = arg<DistillGradLaunch>(args);
        if ((int64_t)g.y * p.piece < p.vocab) fail("pieces of a row");
    }
}

}  // namespace

// ---------------------------------------------------------------------------
// the HIP runtime's part
// ---------------------------------------------------------------------------
extern "C" {
static dim3 cfg_grid, cfg_block;
static size_t cfg_shared;
static hipStream_t cfg_stream;

void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* f, char*, const char* name, unsigned, void*, void*, void*, void*, int*)
{
    names()[f] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t sh, hipStream_t s)
{
    cfg_grid = g; cfg_block = b; cfg_shared = sh; cfg_stream = s;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* sh, hipStream_t* s)
{
    *g = cfg_grid; *b = cfg_block; *sh = cfg_shared; *s = cfg_stream;
    return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t shared, hipStream_t)
{
    ++launches;
    if (!names().count(f)) fail("an unknown kernel");
    if (g.x < 1 || g.y < 1 || g.z < 1 || g.y > 65535 || g.z > 65535) fail("a grid of no or too many work groups");
    if ((uint64_t)g.x * b.x >= (uint64_t)1 << 32) fail("2^32 threads or more in one dimension");
    if (b.x * b.y * b.z > 1024 || shared > 160 * 1024) fail("a work group beyond the device's");
    look(names()[f], g, b, args);
    return hipSuccess;
}
}

namespace fp4 {
// E8M0 as it is, every other encoding with E4M3's parameters
bool scale_fmt_params(int32_t fmt, ScaleFmtHost* f)
{
    *f = ScaleFmtHost{4, 3, 7, 126, 448.0f, fmt == FP4_SCALE_E8M0};
    return true;
}
int64_t logprob_pieces(int64_t rows, int64_t vocab)
{
    const int64_t n = rows < 1 || rows >= 512 ? 1 : cdiv(512, rows), most = cdiv(vocab, 4096);
    return n < most ? (n < kLpMaxPieces ? n : kLpMaxPieces) : (most < kLpMaxPieces ? most : kLpMaxPieces);
}
}  // namespace fp4

// ---------------------------------------------------------------------------
namespace {

void expect(fp4_status got, fp4_status want, int least = 0)
{
    if (got != want) {
        std::fprintf(stderr, "status %d, not %d\n", (int)got, (int)want);
        fail("status");
    }
    if (launches < least) fail("launched less than its work");
}

void begin(int64_t bytes)
{
    if (bytes < 0) fail("workspace refused");
    launches = 0;
    space_at = (uintptr_t)place(kSpace);
    space_end = space_at + (uintptr_t)bytes;
}
void* space(int64_t bytes) { return bytes ? place(kSpace) : nullptr; }

fp4_tensor tensor(int at, int64_t rows, int64_t cols, int32_t block, int32_t scale, int32_t element)
{
    fp4_tensor t;
    std::memset(&t, 0, sizeof t);
    t.q = (uint8_t*)place(at); t.scales = (uint8_t*)place(at + 1); t.tensor_scale = (float*)place(at + 2);
    t.rows = rows; t.cols = cols;
    t.fmt.block = block; t.fmt.scale = scale; t.fmt.element = element;
    return t;
}

void products(int64_t m, int64_t n, int64_t k, int32_t block, int32_t scale, int32_t element)
{
    char size[96];
    std::snprintf(size, sizeof size, "product %lld x %lld x %lld, block %d, scale %d, element %d", (long long)m, (long long)n,
                  (long long)k, block, scale, element);
    now = size;
    const fp4_tensor a = tensor(0, m, k, block, scale, element), b = tensor(3, n, k, block, scale, element);
    if (m * (k / 8) >= (int64_t)1 << 31 || n * (k / 8) >= (int64_t)1 << 31) return;
    fp4_epilogue e;
    std::memset(&e, 0, sizeof e);
    e.bias = place(6); e.act = FP4_ACT_SILU;
    e.mul = (uint16_t*)place(7); e.ld_mul = n; e.residual = (uint16_t*)place(8); e.ld_residual = n + 3;
    e.pre = (uint16_t*)place(9); e.ld_pre = n;
    uint16_t* y = (uint16_t*)place(10);
    const int64_t w = fp4_gemm_epilogue_workspace(&a, &b);
    begin(w);
    expect(fp4_gemm_epilogue(&a, &b, &e, y, n, space(w), w, nullptr), FP4_OK, w ? 2 : 1);
    if (w) expect(fp4_gemm_epilogue(&a, &b, &e, y, n, space(w), w - 1, nullptr), FP4_ERR_INVALID_ARG);
    if (m > 16 || k % 256 || n * k >= (int64_t)1 << 32) return;
    begin(0);
    e.pre = nullptr;
    expect(fp4_wo_gemm_epilogue((uint16_t*)place(11), k, m, &b, &e, y, n, nullptr), FP4_OK, 1);
}

void gradients(int64_t rows, int64_t cols, int32_t act, bool mul, bool bias)
{
    char size[64];
    std::snprintf(size, sizeof size, "epilogue gradients %lld x %lld", (long long)rows, (long long)cols);
    now = size;
    const int64_t w = fp4_epilogue_workspace(rows, cols);
    begin(w);
    uint16_t *x = (uint16_t*)place(0), *p = (uint16_t*)place(1), *u = mul ? (uint16_t*)place(2) : nullptr;
    uint16_t *dp = (uint16_t*)place(3), *du = (uint16_t*)place(4);
    float* db = bias ? (float*)place(5) : nullptr;
    expect(fp4_epilogue_backward(x, cols, p, cols, u, cols, rows, cols, act, dp, cols, du, cols, db, space(w), w, nullptr), FP4_OK,
           rows || bias ? 1 : 0);
    if (w && bias)
        expect(fp4_epilogue_backward(x, cols, p, cols, u, cols, rows, cols, act, dp, cols, du, cols, db, space(w), w - 1, nullptr),
               FP4_ERR_INVALID_ARG);
}

void experts(int64_t m, int32_t top, int64_t hidden, int64_t ffn, int64_t e, int32_t block, int32_t scale, int32_t element)
{
    char size[128];
    std::snprintf(size, sizeof size, "%lld tokens, top %d of %lld experts %lld x %lld, block %d, element %d", (long long)m, top,
                  (long long)e, (long long)hidden, (long long)ffn, block, element);
    now = size;
    const int64_t bits = element == FP4_ELEM_FP8_E4M3 || element == FP4_ELEM_INT8 ? 8 : element >= FP4_ELEM_FP6_E2M3 ? 6 : 4;
    // what a tensor, and an expert, may hold
    if (2.0 * (double)e * (double)ffn * (double)(hidden / 8) >= 2147483648.0 || 2 * ffn * (hidden * bits / 8) >= (int64_t)1 << 32) return;
    const fp4_moe_bank bank{tensor(0, e * 2 * ffn, hidden, block, scale, element), tensor(3, e * hidden, ffn, block, scale, element),
                            (float*)place(6), nullptr, e};
    const int64_t w = fp4_moe_workspace(m, top, ffn);
    begin(w);
    uint16_t *x = (uint16_t*)place(7), *y = (uint16_t*)place(8);
    const int32_t* ids = (int32_t*)place(9);
    const float* wt = (float*)place(10);
    expect(fp4_moe(x, hidden, m, &bank, ids, wt, top, FP4_ACT_SILU, y, hidden, y, hidden, space(w), w, nullptr), FP4_OK, 2);
    expect(fp4_moe(x, hidden, m, &bank, ids, wt, top, FP4_ACT_SILU, y, hidden, y, hidden, space(w), w - 1, nullptr),
           FP4_ERR_INVALID_ARG);
}

void distill(int64_t rows, int64_t vocab, int32_t top, int32_t dtype)
{
    char size[96];
    std::snprintf(size, sizeof size, "distillation %lld x %lld, top %d", (long long)rows, (long long)vocab, top);
    now = size;
    const int64_t w = fp4_distill_workspace(rows, vocab, dtype);
    begin(w);
    float* f = (float*)place(1);
    const int32_t* ids = (int32_t*)place(2);
    for (int32_t rest : {FP4_DISTILL_BUCKET, FP4_DISTILL_RENORMALIZE}) {
        expect(fp4_distill_loss(place(0), dtype, vocab, rows, vocab, ids, f, top, 0.5f, rest, f, f, space(w), w, nullptr), FP4_OK,
               rows ? 1 : 0);
        if (w)
            expect(fp4_distill_loss(place(0), dtype, vocab, rows, vocab, ids, f, top, 0.5f, rest, f, f, space(w), w - 1, nullptr),
                   FP4_ERR_INVALID_ARG);
        expect(fp4_distill_loss_backward(place(0), dtype, vocab, rows, vocab, ids, f, top, 0.5f, rest, f, f, place(3), vocab, nullptr),
               FP4_OK, rows ? 1 : 0);
    }
}

}  // namespace

int main()
{
    const struct { int32_t block, scale, element; } formats[] = {
        {32, FP4_SCALE_E8M0, FP4_ELEM_E2M1}, {16, FP4_SCALE_E8M0, FP4_ELEM_E2M1}, {16, FP4_SCALE_E4M3, FP4_ELEM_E2M1},
        {32, FP4_SCALE_E4M3, FP4_ELEM_E2M1}, {32, FP4_SCALE_E8M0, FP4_ELEM_FP8_E4M3}, {16, FP4_SCALE_E4M3, FP4_ELEM_INT8},
        {32, FP4_SCALE_E8M0, FP4_ELEM_INT4}, {32, FP4_SCALE_E8M0, FP4_ELEM_FP6_E2M3}, {32, FP4_SCALE_E8M0, FP4_ELEM_INT6}};
    for (const auto& f : formats) {
        for (int64_t small : {(int64_t)0, (int64_t)1 << 21}) {
            fp4::g_gemm_small_outputs = small;
            for (int64_t m : {1, 16, 31, 256, 257, 1111, 8192, 100000, 1 << 20})
                for (int64_t n : {1, 8, 264, 1027, 4096, 11008, 65536})
                    for (int64_t k : {128, 256, 384, 1024, 1152, 4096, 11008, 65536}) products(m, n, k, f.block, f.scale, f.element);
        }
        for (int64_t m : {1, 2, 4, 5, 8, 16})
            for (int32_t top : {1, 2, 8, 16})
                for (int64_t h : {128, 256, 384, 4096, 16384, 1 << 25})
                    for (int64_t n : {128, 640, 768, 11008, 1 << 18, 1 << 25})
                        for (int64_t e : {1, 8, 128, 65535}) experts(m, top, h, n, e, f.block, f.scale, f.element);
    }
    for (int64_t rows : {0, 1, 130, 1024, 1025, 8192, 1 << 22})
        for (int64_t cols : {1, 7, 64, 257, 11008, 1 << 17, 1 << 24})
            for (int32_t act : {FP4_ACT_NONE, FP4_ACT_RELU, FP4_ACT_GELU_TANH}) {
                if (rows > ((int64_t)1 << 40) / cols) continue;
                gradients(rows, cols, act, true, true);
                gradients(rows, cols, act, false, false);
                gradients(rows, cols, act, false, true);
            }
    for (int64_t rows : {(int64_t)0, (int64_t)1, (int64_t)3, (int64_t)61, (int64_t)511, (int64_t)512, (int64_t)2000, ((int64_t)1 << 22) - 1})
        for (int64_t vocab : {1, 33, 4097, 16385, 128000, 131072, 131073, 262145, 1 << 20, (1 << 24) - 1, 1 << 24})
            for (int32_t top : {1, 64, 65, 128}) {
                if (vocab > ((int64_t)1 << 40) / (rows ? rows : 1)) continue;
                for (int32_t dt : {FP4_DTYPE_F32, FP4_DTYPE_BF16}) distill(rows, vocab, top, dt);
            }
    now = "router";
    for (int64_t rows : {(int64_t)1, (int64_t)300, ((int64_t)1 << 22) - 1})
        for (int64_t e : {1, 64, 65, 128, 256, 257, 1024}) {
            launches = 0;
            expect(fp4_moe_route(place(0), FP4_DTYPE_F32, e, rows, e, 1, FP4_ROUTE_SIGMOID, (float*)place(1), 1, 1.0f, (int32_t*)place(2),
                                 (float*)place(3), nullptr), FP4_OK, 1);
        }
    std::puts("ok");
    return 0;
}
