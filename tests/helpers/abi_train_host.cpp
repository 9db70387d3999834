// Drives the host side of the adapter, token-probability and residual-norm
// calls (api_train.cpp and the launch code of lora.hip, logprobs.hip and
// norm.hip, their host pass only) with a stand-in for the HIP runtime, for a
// build with AddressSanitizer and UndefinedBehaviorSanitizer and no GPU.
// Nothing is launched: hipLaunchKernel below looks at each launch instead.  Its
// grid must be one that the runtime takes, and what it reads or writes of the
// workspace must lie in the bytes that the call asked for, apart from what
// other pieces of it hold.  The addresses are never dereferenced.  Exit status:
// 0 and "ok", or an abort at the first launch or status that is wrong.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

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

struct Piece { uintptr_t at, end; const char* name; };
uintptr_t space_at = 0, space_end = 0;
std::vector<Piece> pieces;
int launches = 0;
// kernels register before main, in an order of their own
std::map<const void*, std::string>& names()
{
    static std::map<const void*, std::string> all;
    return all;
}

// Bytes [p, p + bytes) are a part of the workspace, if p is in it at all; two
// uses of one place are one piece, and different pieces lie apart.
void uses(const void* ptr, int64_t bytes, const char* name)
{
    const uintptr_t p = (uintptr_t)ptr;
    if (!p || p < space_at || p - space_at >= ((uintptr_t)1 << 43)) return;
    if (bytes < 0 || p + (uintptr_t)bytes > space_end) fail(name);
    for (Piece& o : pieces)
        if (o.at == p) {
            if (p + (uintptr_t)bytes > o.end) o.end = p + (uintptr_t)bytes;
            return;
        }
    pieces.push_back({p, p + (uintptr_t)bytes, name});
}
void apart()
{
    for (size_t i = 0; i < pieces.size(); ++i)
        for (size_t j = 0; j < i; ++j)
            if (pieces[i].at < pieces[j].end && pieces[j].at < pieces[i].end) fail("pieces of the workspace overlap");
}

template <typename T>
const T& arg(void** args, int i = 0) { return *static_cast<const T*>(args[i]); }

void look(const std::string& name, dim3 g, void** args)
{
    auto is = [&](const char* s) { return name.find(s) != std::string::npos; };
    if (is("k_lora_down")) {
        const LoraDown& p = arg<LoraDown>(args);
        uses(p.t, 4 * (int64_t)g.x * p.m * p.rank, "partial sums of T");
        uses(p.a, 2 * p.adapters * p.rank * p.k, "B transposed");
        if ((int64_t)g.x * p.kstep < p.k || ((int64_t)g.x - 1) * p.kstep >= p.k) fail("K ranges");
        if (g.y * (p.m <= 16 ? 16 : 32) < p.m) fail("row tiles");
    } else if (is("k_lora_up")) {
        const LoraUp& p = arg<LoraUp>(args);
        uses(p.t, 4 * (int64_t)p.splits * p.m * p.rank, "partial sums of T, read");
        uses(p.t_out, 4 * p.m * p.rank, "T");
        uses(p.b, 2 * p.adapters * p.rank * p.n, "A transposed");
        if ((int64_t)g.x * p.ncols < p.n) fail("column blocks");
    } else if (is("k_lora_sum")) {
        const int64_t n = arg<int64_t>(args, 2);
        uses(arg<const float*>(args, 0), 4 * arg<int>(args, 1) * n, "partial sums of T, joined");
        uses(arg<float*>(args, 3), 4 * n, "T");
    } else if (is("k_lora_transpose")) {
        const LoraTranspose& p = arg<LoraTranspose>(args);
        for (int i = 0; i < 2; ++i) uses(p.dst[i], 2 * (int64_t)g.y * p.rows[i] * p.cols[i], "transposed bank");
        if ((int64_t)g.x != p.blocks[0] + p.blocks[1]) fail("tiles of the bank");
    } else if (is("k_lora_outer") || is("k_lora_join")) {
        const LoraOuter& p = arg<LoraOuter>(args);
        const int64_t splits = is("k_lora_join") ? arg<int>(args, 1) : g.z;
        for (const LoraOuterJob& j : p.job) {
            uses(j.p, 4 * p.m * p.rank, "T or dT");
            if (splits > 1) uses(j.part, 4 * splits * p.adapters * p.rank * j.c, "partial gradients");
        }
        if (splits > 1) uses(p.flags, 4 * splits * p.adapters, "flags");
        if (!is("k_lora_join") && (int64_t)g.z * p.mstep < p.m) fail("row ranges");
    } else if (is("k_lp_rows")) {
        const LogprobLaunch& p = arg<LogprobLaunch>(args);
        if ((int64_t)g.y * p.piece < p.vocab || ((int64_t)g.y - 1) * p.piece >= p.vocab || g.y > (unsigned)kLpMaxPieces)
            fail("pieces of a row");
        if (g.y > 1) {
            uses(p.part_sums, 16 * p.rows * g.y, "partial sums");
            if (p.top) uses(p.part_keys, 8 * p.rows * g.y * p.top, "keys");
        }
    } else if (is("k_norm_backward")) {
        const NormGradLaunch& p = arg<NormGradLaunch>(args);
        uses(p.part, 4 * p.groups * p.part_rows * p.f.cols, "partial rows");
        if ((int64_t)g.x != p.groups) fail("groups");
    } else if (is("k_norm_join")) {
        uses(arg<const float*>(args, 0), 4 * arg<int64_t>(args, 1) * arg<int64_t>(args, 2), "partial rows, joined");
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
    look(names()[f], g, args);
    return hipSuccess;
}
}

namespace fp4 {
hipError_t launch_wo_gemm(const WoGemmLaunch& p, hipStream_t)
{
    ++launches;
    uses(p.ad.t, 4 * (int64_t)p.ad.splits * p.m * p.ad.rank, "partial sums of T, read by the product");
    return hipSuccess;
}
bool scale_fmt_params(int32_t, ScaleFmtHost* f) { *f = ScaleFmtHost{}; return true; }
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
    apart();
}

void begin(int64_t bytes)
{
    if (bytes < 0) fail("workspace refused");
    launches = 0;
    pieces.clear();
    space_at = (uintptr_t)place(kSpace);
    space_end = space_at + (uintptr_t)bytes;
}
void* space(int64_t bytes) { return bytes ? place(kSpace) : nullptr; }

void adapters(int64_t m, int64_t n, int64_t k, int64_t rank, int64_t la)
{
    const fp4_lora_bank bank{(const uint16_t*)place(0), (const uint16_t*)place(1), (const float*)place(2), la, rank, k, n};
    const uint16_t* x = (const uint16_t*)place(3);
    const uint16_t* dy = (const uint16_t*)place(4);
    uint16_t* out = (uint16_t*)place(5);
    float* t = (float*)place(6);
    const int32_t* slots = (const int32_t*)place(7);
    char size[128];
    std::snprintf(size, sizeof size, "%lld x %lld x %lld, rank %lld, %lld adapters", (long long)m, (long long)n, (long long)k,
                  (long long)rank, (long long)la);
    now = std::string("apply ") + size;
    int64_t b = fp4_lora_workspace(FP4_LORA_APPLY, m, n, k, rank, la);
    begin(b);
    expect(fp4_lora_apply(x, k, m, &bank, slots, nullptr, 0, out, n, t, space(b), b, nullptr), FP4_OK, m ? 2 : 0);
    if (b) expect(fp4_lora_apply(x, k, m, &bank, slots, nullptr, 0, out, n, t, space(b), b - 1, nullptr), FP4_ERR_INVALID_ARG);
    now = std::string("backward ") + size;
    b = fp4_lora_workspace(FP4_LORA_BACKWARD, m, n, k, rank, la);
    for (int32_t gd : {FP4_DTYPE_F32, FP4_DTYPE_BF16}) {
        begin(b);
        expect(fp4_lora_backward(dy, n, x, k, m, t, &bank, slots, nullptr, 0, out, k, place(8), place(9), gd, space(b), b, nullptr),
               FP4_OK, m ? 3 : 1);
    }
    if (b)
        expect(fp4_lora_backward(dy, n, x, k, m, t, &bank, slots, nullptr, 0, out, k, place(8), place(9), 0, space(b), b - 1, nullptr),
               FP4_ERR_INVALID_ARG);
    if (m < 1 || m > 16 || k % 256 || n * k >= (int64_t)1 << 31) return;
    now = std::string("weight-only ") + size;
    fp4_tensor w;
    std::memset(&w, 0, sizeof w);
    w.q = (uint8_t*)place(10); w.scales = (uint8_t*)place(11); w.tensor_scale = (float*)place(12);
    w.rows = n; w.cols = k;
    w.fmt.block = 16; w.fmt.amax = FP4_AMAX_CURRENT;
    b = fp4_lora_workspace(FP4_LORA_WO_GEMM, m, n, k, rank, la);
    begin(b);
    expect(fp4_wo_gemm_lora(x, k, m, &w, &bank, slots, out, n, space(b), b, nullptr), FP4_OK, 2);
    expect(fp4_wo_gemm_lora(x, k, m, &w, &bank, slots, out, n, space(b), b - 1, nullptr), FP4_ERR_INVALID_ARG);
}

void logprobs(int64_t rows, int64_t vocab, int32_t top, int32_t dtype)
{
    char size[96];
    std::snprintf(size, sizeof size, "log probabilities %lld x %lld, top %d", (long long)rows, (long long)vocab, (int)top);
    now = size;
    const int64_t b = fp4_token_logprobs_workspace(rows, vocab, top);
    begin(b);
    float* f = (float*)place(1);
    expect(fp4_token_logprobs(place(0), dtype, vocab, rows, vocab, (const int64_t*)place(2), 0.5f, top, f, f, f,
                              (int32_t*)place(3), f, space(b), b, nullptr), FP4_OK, rows ? 1 : 0);
    if (b)
        expect(fp4_token_logprobs(place(0), dtype, vocab, rows, vocab, nullptr, 0.5f, top, f, f, f, (int32_t*)place(3), f,
                                  space(b), b - 1, nullptr), FP4_ERR_INVALID_ARG);
    launches = 0;
    expect(fp4_token_logprobs_backward(place(0), dtype, vocab, rows, vocab, (const int64_t*)place(2), 0.5f, f, f, f, f, place(4),
                                       vocab, nullptr), FP4_OK, rows ? 1 : 0);
}

void norms(int64_t rows, int64_t cols, bool post, int32_t xd, int32_t rd)
{
    char size[64];
    std::snprintf(size, sizeof size, "norm %lld x %lld", (long long)rows, (long long)cols);
    now = size;
    float* f = (float*)place(4);
    const fp4_norm a{place(0), cols, place(1), cols, rows, cols, place(2), post ? place(3) : nullptr, f, 0.5f, 1e-6f, xd, rd, 0};
    begin(0);
    expect(fp4_residual_norm(&a, place(5), cols, place(6), cols, f, nullptr), FP4_OK, rows ? 1 : 0);
    const int64_t b = fp4_residual_norm_workspace(rows, cols, post);
    begin(b);
    expect(fp4_residual_norm_backward(&a, f, place(5), cols, place(6), cols, place(7), cols, place(8), cols, f, f, f, space(b), b,
                                      nullptr), FP4_OK, 2);
    expect(fp4_residual_norm_backward(&a, f, place(5), cols, place(6), cols, place(7), cols, place(8), cols, f, f, f, space(b),
                                      b - 1, nullptr), FP4_ERR_INVALID_ARG);
}

}  // namespace

int main()
{
    const int64_t M[] = {0, 1, 7, 16, 17, 64, 130, 511, 2048, 8192, 100000, 1 << 20};
    const int64_t D[] = {8, 256, 264, 1000, 4096, 11008, 65536};
    for (int64_t m : M)
        for (int64_t n : D)
            for (int64_t k : D)
                for (int64_t rank : {8, 24, 40, 64, 72, 128})
                    for (int64_t la : {1, 3, 40}) adapters(m, n, k, rank, la);
    // the ends of what the calls take
    for (int64_t m : {0, 1, 16, 72, 1 << 16})
        for (int64_t la : {1, 16384})
            for (int64_t rank : {8, 128}) {
                adapters(m, 8, 1 << 24, rank, la);
                adapters(m, 1 << 24, 8, rank, la);
                adapters(m, 1 << 24, 1 << 24, rank, la);
                adapters(m, 8, 65536, rank, la);
            }
    for (int64_t rows : {(int64_t)0, (int64_t)1, (int64_t)3, (int64_t)61, (int64_t)511, (int64_t)512, (int64_t)2000, ((int64_t)1 << 22) - 1})
        for (int64_t vocab : {(int64_t)1, (int64_t)33, (int64_t)4095, (int64_t)4097, (int64_t)16385, (int64_t)128000, ((int64_t)1 << 27) - 1})
            for (int32_t top : {0, 1, 32}) {
                if (top > vocab || vocab > (((int64_t)1 << 40) / (rows ? rows : 1))) continue;
                for (int32_t dt : {FP4_DTYPE_F32, FP4_DTYPE_BF16}) logprobs(rows, vocab, top, dt);
            }
    for (int64_t rows : {(int64_t)0, (int64_t)1, (int64_t)300, (int64_t)1001, (int64_t)8192, ((int64_t)1 << 22) - 1})
        for (int64_t cols : {1, 7, 512, 513, 2048, 4095, 4096, 8192, 9001, 16384, 18944, 32767, 32768})
            for (int post = 0; post < 2; ++post)
                for (int t = 0; t < 4; ++t) norms(rows, cols, post, t & 1, t >> 1);
    std::puts("ok");
    return 0;
}
