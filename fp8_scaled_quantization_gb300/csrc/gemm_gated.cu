// gemm_gated.cu -- the gated feed-forward block's first half in block-scaled FP8:
// both projections, the activation, their product and its 1 x 128 quantization in
// one kernel.  The C entry points, their checks and the choice of kernel.
//
// "Megatron FP8" §6 (forward products over FP8 operands), §21 (experts); "Low
// Precision Training and Rollout" (128 x 128 weight blocks).
//
// Unfused, the projections come out as BF16 (4 bytes per element of h), the
// activation reads them and writes h, and the cast reads that and writes codes: 9
// bytes an element and two launches more, where 1 byte (with the checkpoint 3)
// leaves this kernel.
#include <cmath>

#include "fp8q_host.h"
#include "gemm_block.cuh"

namespace fp8q {
namespace {

fp8_status_t check(const char* fn, const GemmProblem& p) {
    const GatedOut& o = p.gated;
    if (!valid_fmt(p.fmt_a) || !valid_fmt(p.fmt_b)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format", fn);
    if (o.act != FP8_ACT_SILU && o.act != FP8_ACT_GELU_TANH)
        return fail(FP8_ERR_INVALID_ARG, "%s: unknown activation %d", fn, o.act);
    if (p.m < 0 || p.n < 0 || p.k < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size", fn);
    constexpr int64_t kMost = (1ll << 31) - 256, kMostTiles = 1ll << 30;
    if (p.m > kMost || p.n > kMost || p.k > kMost)
        return fail(FP8_ERR_UNSUPPORTED, "%s: sizes must be below 2^31 - 256", fn);
    // tiles are numbered with 32 bits: at least 16 x 128, one more along m for each group
    if (((p.m + 15) / 16 + p.groups) * ((p.n + 127) / 128) > kMostTiles)
        return fail(FP8_ERR_UNSUPPORTED, "%s: too many output tiles", fn);
    if ((o.gu == nullptr) != (o.sgu == nullptr))
        return fail(FP8_ERR_INVALID_ARG, "%s: the checkpoint needs both its codes and its scales", fn);
    if (p.m == 0 || p.n == 0) return FP8_OK;
    if (o.h == nullptr || o.sh == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: h or its scales are NULL", fn);
    if (p.k > 0 && (p.a == nullptr || p.b == nullptr || p.sa == nullptr || p.sb == nullptr))
        return fail(FP8_ERR_INVALID_ARG, "%s: an operand or its scales are NULL", fn);
    for (const float* s : {p.k > 0 ? p.sa : nullptr, p.k > 0 ? p.sb : nullptr, (const float*)o.sh, (const float*)o.sgu})
        if ((reinterpret_cast<uintptr_t>(s) & 3u) != 0)
            return fail(FP8_ERR_INVALID_ARG, "%s: scales are not 4-byte aligned", fn);
    return FP8_OK;
}

// Which kernel, by estimated times in microseconds from what they measured on GB300: the
// pair kernel (0), or the stream kernel by tiles of 16, 32 or 64 tokens.  [m, n, k] silu,
// without a checkpoint, in a CUDA graph, cold weights:
//   [3, 1024, 1024]    stream/16 5.4  /32 5.8  /64 6.1  pair 8.5    [1, 18432, 7168]  44  46  60  79
//   [16, 7168, 7168]   22  22  25  37      [32, 14336, 4096]  36  27  29  37    [48, 14336, 4096]  48  40  31  38
//   [64, 2048, 7168]   15  14  16  29      [4864, 6144, 128]  503  299  235  42
//   experts: 96 rows over 64 of 2048 x 7168  280  286  300  383;  512 over 32  143 to 158  161  176  203;
//   1024 over 16 of 2048 x 2048  78  55  45  44
// Over 73 random sizes of this range (1 to 8192 rows, up to 64 experts) the choices take
// 1.4% more than the fastest kernel does, 22% at worst.
int choose(const GemmProblem& p) {
    const int64_t kb = blocks_of(p.k), sms = sm_count();
    const double busy = (double)(p.groups < p.m ? p.groups : p.m), rows = (double)p.m / busy;  // groups with rows, and theirs
    const auto most = [](double a, double b) { return a > b ? a : b; };
    const auto tiles = [&](int high) {  // along m: one per group at least, the last one of longer ones half full on average
        return p.groups > 1 ? most(busy, (double)p.m / high + 0.5 * busy) : (double)((p.m + high - 1) / high);
    };
    const double memory = (2.0 * busy * (double)p.n * (double)p.k + (double)p.m * (double)(p.k + p.n)) / 6.5e6;
    const double columns = (double)((p.n + 127) / 128);
    const bool keep = p.gated.gu != nullptr;
    // the pair kernel: 0.46 per block, and the end of a tile
    const double pair = ceil(tiles(256) * columns / (double)(sms / 2)) * (0.46 * (double)kb + (keep ? 3.8 : 2.4));
    double best = 3.5 + most(pair, memory * 6.5 / 4.5);
    int choice = 0;
    // the stream kernel: per block, and the end of an item by the tokens that a CTA joins; the
    // next one starts 2.7 later
    constexpr double kBlock[3] = {0.40, 0.39, 0.66};
    for (int i = 0; i < 3; ++i) {
        const int tokens = 16 << i;
        const StreamPlan plan = stream_plan(p, tokens, (int)sms);
        const double rounds = ceil(tiles(tokens) * columns / plan.clusters);
        const double join = 0.6 + (keep ? 0.36 : 0.18) * (rows < tokens ? rows : tokens) / plan.split;
        const double compute = rounds * ceil((double)kb / (plan.split / 2)) * kBlock[i] + (rounds - 1.0) * (2.7 + join);
        const double us = 5.0 + 0.3 * i + join + most(compute, memory);
        if (us < best) best = us, choice = tokens;
    }
    return choice;
}

fp8_status_t run(const char* fn, const GemmProblem& p, cudaStream_t st) {
    const int tokens = p.k > 0 ? choose(p) : 0;
    return tokens > 0 ? run_gemm_stream(fn, p, tokens, st) : run_gemm_pair(fn, p, st);
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8_status_t fp8_gemm_block_gated(const uint8_t* a, fp8_format_t fmt_a, const float* scale_inv_a,
                                             const uint8_t* b, fp8_format_t fmt_b, const float* scale_inv_b,
                                             fp8_activation_t act, int64_t m, int64_t n, int64_t k, uint8_t* h,
                                             float* scale_inv_h, uint8_t* gu, float* scale_inv_gu, void* stream) {
    const char* fn = "fp8_gemm_block_gated";
    const GemmProblem p = {a, b, scale_inv_a, scale_inv_b, nullptr, nullptr, m, n, k, 1, (int)fmt_a, (int)fmt_b,
                           false, false, false, false, {h, scale_inv_h, gu, scale_inv_gu, (int)act}};
    const fp8_status_t s = check(fn, p);
    if (s != FP8_OK || m == 0 || n == 0) return s;
    return run(fn, p, static_cast<cudaStream_t>(stream));
}

extern "C" fp8_status_t fp8_gemm_block_gated_grouped(int groups, const int64_t* group_ends, const uint8_t* a,
                                                     fp8_format_t fmt_a, const float* scale_inv_a, const uint8_t* b,
                                                     fp8_format_t fmt_b, const float* scale_inv_b, fp8_activation_t act,
                                                     int64_t rows, int64_t n, int64_t k, uint8_t* h, float* scale_inv_h,
                                                     uint8_t* gu, float* scale_inv_gu, void* stream) {
    const char* fn = "fp8_gemm_block_gated_grouped";
    fp8_status_t s = check_groups(fn, groups, group_ends);
    if (s != FP8_OK) return s;
    const GemmProblem p = {a, b, scale_inv_a, scale_inv_b, nullptr, group_ends, rows, n, k, groups, (int)fmt_a, (int)fmt_b,
                           false, false, false, false, {h, scale_inv_h, gu, scale_inv_gu, (int)act}};
    s = check(fn, p);
    if (s != FP8_OK || rows == 0 || n == 0) return s;
    return run(fn, p, static_cast<cudaStream_t>(stream));
}
