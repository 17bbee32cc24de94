// gemm_block.cu -- block-scaled FP8 products: the C entry points, their checks,
// and the copy that aligns odd operands.
//
// "Megatron FP8" §6 (forward, dgrad and wgrad GEMMs over FP8 operands), "Low
// Precision Training and Rollout" (128x128 weight blocks), "[Pytorch][Common]
// Hybrid quantization #2817" (1x128 / 128x1 blockwise copies for the backward
// GEMMs), "Megatron FP8" §21 (experts).
#include <cmath>

#include "fp8q_host.h"
#include "gemm_block.cuh"

namespace fp8q {
namespace {

// Rows of `inner` bytes copied to rows of `stride` bytes (a multiple of 16, the
// rest zeros), one 16-byte piece per lane and step.  Sources start anywhere: a
// piece is cut out of the aligned 4-byte words around it, or put together from
// single bytes at the array's two ends, so that nothing outside is read.
constexpr int kPackThreads = 256;

__global__ void __launch_bounds__(kPackThreads)
align_rows_kernel(const uint8_t* __restrict__ src, int64_t rows, int64_t inner, uint8_t* __restrict__ dst, int64_t stride) {
    pdl_begin();
    const uint8_t* const end = src + rows * inner;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kPackThreads / 32);
    for (int64_t r = (int64_t)blockIdx.x * (kPackThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
#pragma unroll 4
        for (int64_t x = lane * 16; x < stride; x += 512) {
            const uint8_t* p = src + r * inner + x;
            const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 3u);
            const uint8_t* w = p - off;
            uint32_t v[5] = {0u, 0u, 0u, 0u, 0u};
            if (x + 16 <= inner && w >= src && w + 20 <= end) {
#pragma unroll
                for (int i = 0; i < 5; ++i) v[i] = __ldg(reinterpret_cast<const uint32_t*>(w) + i);
                const uint32_t sh = off * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], sh);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (x + i < inner) v[i >> 2] |= (uint32_t)__ldg(p + i) << (8 * (i & 3));
            }
            stg_stream(dst + r * stride + x, make_uint4(v[0], v[1], v[2], v[3]));
        }
    }
}

fp8_status_t check(const char* fn, const GemmProblem& p, int layout, int b_block_rows, int out_dtype) {
    if (!valid_fmt(p.fmt_a) || !valid_fmt(p.fmt_b)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format", fn);
    if (!valid_dtype(out_dtype)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown out_dtype %d", fn, out_dtype);
    if (layout != FP8_B_NK && layout != FP8_B_KN) return fail(FP8_ERR_INVALID_ARG, "%s: unknown layout %d", fn, layout);
    if (p.m < 0 || p.n < 0 || p.k < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size", fn);
    if (b_block_rows != 1 && b_block_rows != kBlk)
        return fail(FP8_ERR_UNSUPPORTED, "%s: b_block_rows must be 128 or 1", fn);
    if (b_block_rows == 1 && layout == FP8_B_KN)
        return fail(FP8_ERR_UNSUPPORTED, "%s: 1x128 tiles of B run along the contraction: B must be [n, k]", fn);
    if (p.accumulate && out_dtype != FP8_DT_FP32)
        return fail(FP8_ERR_UNSUPPORTED, "%s: accumulate needs an fp32 output", fn);
    constexpr int64_t kMost = (1ll << 31) - 256, kMostTiles = 1ll << 30;
    if (p.m > kMost || p.n > kMost || p.k > kMost)
        return fail(FP8_ERR_UNSUPPORTED, "%s: sizes must be below 2^31 - 256", fn);
    // Tiles are numbered with 32 bits: 256 x 256 outputs per group where the contraction
    // is ragged; else at least 16 x 128, and one more along m for each group (and for
    // the rows after the last one).
    const bool ragged_k = p.b_tiles && p.ends != nullptr;
    const int64_t tiles = ragged_k ? ((p.m + 255) / 256) * ((p.n + 255) / 256) * p.groups
                                   : ((p.m + 15) / 16 + p.groups) * ((p.n + 127) / 128);
    if (tiles > kMostTiles) return fail(FP8_ERR_UNSUPPORTED, "%s: too many output tiles", fn);
    if (p.m == 0 || p.n == 0) return FP8_OK;
    if (p.d == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: d is NULL", fn);
    if ((reinterpret_cast<uintptr_t>(p.d) & (uintptr_t)(dtype_size(out_dtype) - 1)) != 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: d is not element-aligned", fn);
    if (p.k > 0) {
        if (p.a == nullptr || p.b == nullptr || p.sa == nullptr || p.sb == nullptr)
            return fail(FP8_ERR_INVALID_ARG, "%s: an operand or its scales are NULL", fn);
        if ((reinterpret_cast<uintptr_t>(p.sa) & 3u) != 0 || (reinterpret_cast<uintptr_t>(p.sb) & 3u) != 0)
            return fail(FP8_ERR_INVALID_ARG, "%s: scales are not 4-byte aligned", fn);
    }
    return FP8_OK;
}

fp8_status_t check_groups(const char* fn, int groups, const int64_t* ends) {
    if (groups < 1 || groups > kMaxGroups)
        return fail(FP8_ERR_INVALID_ARG, "%s: groups must be in [1, %d]", fn, kMaxGroups);
    if (ends == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: group_ends is NULL", fn);
    if ((reinterpret_cast<uintptr_t>(ends) & 7u) != 0)
        return fail(FP8_ERR_INVALID_ARG, "%s: group_ends is not 8-byte aligned", fn);
    return FP8_OK;
}

}  // namespace

fp8_status_t operand_maps(const char* fn, const Operand& a, CUtensorMap* map_a, const Operand& b, CUtensorMap* map_b,
                          StreamUse& use, cudaStream_t st) {
    const Operand* const in[2] = {&a, &b};
    CUtensorMap* const map[2] = {map_a, map_b};
    size_t need[2];
    for (int i = 0; i < 2; ++i) {
        const bool fits = aligned16(in[i]->codes) && in[i]->inner % 16 == 0;
        need[i] = fits ? 0 : (size_t)((in[i]->inner + 15) / 16 * 16) * (size_t)(in[i]->rows * in[i]->groups);
    }
    fp8_status_t s = FP8_OK;
    uint8_t* scratch = nullptr;
    if (need[0] + need[1] > 0) {
        scratch = static_cast<uint8_t*>(use.scratch(need[0] + need[1], &s));
        if (scratch == nullptr) return s;
    }
    for (int i = 0; i < 2; ++i) {
        const Operand& o = *in[i];
        const int64_t stride = (o.inner + 15) / 16 * 16, rows = o.rows * o.groups;
        const uint8_t* base = o.codes;
        if (need[i] > 0) {
            const int64_t ctas = (rows + kPackThreads / 32 - 1) / (kPackThreads / 32), most = (int64_t)sm_count() * 16;
            s = launch(fn, align_rows_kernel, dim3((unsigned)(ctas < most ? ctas : most)), dim3(kPackThreads), st, o.codes,
                       rows, o.inner, scratch, stride);
            if (s != FP8_OK) return s;
            base = scratch;
            scratch += need[i];
        }
        s = encode_tile_map_u8(map[i], base, o.inner, stride, o.rows, o.groups, o.tile_rows);
        if (s != FP8_OK) return s;
    }
    return FP8_OK;
}

namespace {
// Which kernel, by estimated times in microseconds from what both measured on
// GB300 (one call, in a CUDA graph, cold weights; [m, n, k] bf16 out):
//   [8, 7168, 18432]   stream/16 25   pair 64      [48, 14336, 4096]  stream/32 17  stream/64 20  pair 20
//   [64, 7168, 7168]   stream/64 17   pair 29      [256, 4096, 4096]  stream/32 16  stream/128 20 pair 18
//   [256, 7168, 7168]  pair 30  stream/128 28      [512, 1024, 4096]  stream/64 12  pair 18
//   in 1 x 128 tiles: [256, 2048, 7168]  stream/128 16  pair 41    [768, 7168, 7168]  pair 79  stream/128 90
// A pair of CTAs takes 0.46 (1 x 128 tiles: 0.67) per 128-block of a 256 x 256
// tile, whatever part of the tile is used.  A CTA of the stream kernel takes
// kBlock per block with 16 / 32 / 64 / 128 tokens, with two CTAs per SM up to 64
// (1 x 128 tiles: 32).  Neither is faster than the operands come from memory,
// where the stream kernel reaches 6.5 TB/s and the pair kernel 4.5 (96 rows over
// 64 experts, 2048 x 7168 each: stream/16 99, stream/32 107, pair 137).  Over 405
// forms and sizes (8 to 4096 rows, weights of 512 x 2048 to 18432 x 7168) the
// choices take 0.3% more than the fastest do, 16% at worst.
struct Choice {
    int tokens;  // 0: the pair kernel
    double us;
};

Choice choose(const GemmProblem& p) {
    const int64_t kb = blocks_of(p.k), sms = sm_count();
    const double busy = (double)(p.groups < p.m ? p.groups : p.m);
    const auto tiles = [&](int rows) {  // along m: the groups' last tiles are half full on average
        return p.groups > 1 ? (double)p.m / rows + 0.5 * busy : (double)((p.m + rows - 1) / rows);
    };
    const auto most = [](double a, double b) { return a > b ? a : b; };
    const double memory = (busy * (double)p.n * (double)p.k + (double)p.m * (double)(p.k + 2 * p.n)) / 6.5e6;
    const double pair = ceil(tiles(256) * (double)((p.n + 255) / 256) / (double)(sms / 2)) * (double)kb * (p.b_tiles ? 0.67 : 0.46);
    Choice best = {0, 4.0 + most(pair, memory * 6.5 / 4.5)};
    constexpr double kBlock[2][4] = {{0.40, 0.39, 0.66, 0.53}, {0.43, 0.44, 0.39, 0.54}}, kJoin[4] = {1.0, 1.8, 2.2, 4.0};
    for (int i = 0; i < 4; ++i) {
        const int tokens = 16 << i;
        const StreamPlan plan = stream_plan(p, tokens, (int)sms);
        const double items = tiles(tokens) * (double)((p.n + 127) / 128);
        const double compute = ceil(items / plan.clusters) * ceil((double)kb / plan.split) * kBlock[p.b_tiles][i];
        const double us = 5.0 + (plan.split > 1 ? kJoin[i] : 0.0) + most(compute, memory);
        if (us < best.us) best = {tokens, us};
    }
    return best;
}

fp8_status_t run_gemm(const char* fn, const GemmProblem& p, cudaStream_t st) {
    if (p.k == 0 || (p.b_tiles && p.ends != nullptr)) return run_gemm_pair(fn, p, st);  // nothing to sum; ragged contraction
    const int tokens = choose(p).tokens;
    return tokens > 0 ? run_gemm_stream(fn, p, tokens, st) : run_gemm_pair(fn, p, st);
}
}  // namespace

}  // namespace fp8q

using namespace fp8q;

extern "C" fp8_status_t fp8_gemm_block(const uint8_t* a, fp8_format_t fmt_a, const float* scale_inv_a, const uint8_t* b,
                                       fp8_format_t fmt_b, const float* scale_inv_b, fp8_b_layout_t b_layout,
                                       int b_block_rows, int64_t m, int64_t n, int64_t k, void* d,
                                       fp8_dtype_t out_dtype, int accumulate, void* stream) {
    const char* fn = "fp8_gemm_block";
    const GemmProblem p = {a, b, scale_inv_a, scale_inv_b, d, nullptr, m, n, k, 1, (int)fmt_a, (int)fmt_b,
                           b_layout == FP8_B_KN, b_block_rows == 1, out_dtype == FP8_DT_FP32, accumulate != 0};
    const fp8_status_t s = check(fn, p, b_layout, b_block_rows, out_dtype);
    if (s != FP8_OK || m == 0 || n == 0 || (k == 0 && p.accumulate)) return s;
    return run_gemm(fn, p, static_cast<cudaStream_t>(stream));
}

extern "C" fp8_status_t fp8_gemm_block_grouped(int groups, const int64_t* group_ends, const uint8_t* a,
                                               fp8_format_t fmt_a, const float* scale_inv_a, const uint8_t* b,
                                               fp8_format_t fmt_b, const float* scale_inv_b, fp8_b_layout_t b_layout,
                                               int64_t rows, int64_t n, int64_t k, void* d, fp8_dtype_t out_dtype,
                                               void* stream) {
    const char* fn = "fp8_gemm_block_grouped";
    fp8_status_t s = check_groups(fn, groups, group_ends);
    if (s != FP8_OK) return s;
    const GemmProblem p = {a, b, scale_inv_a, scale_inv_b, d, group_ends, rows, n, k, groups, (int)fmt_a, (int)fmt_b,
                           b_layout == FP8_B_KN, false, out_dtype == FP8_DT_FP32, false};
    s = check(fn, p, b_layout, kBlk, out_dtype);
    if (s != FP8_OK || rows == 0 || n == 0) return s;
    return run_gemm(fn, p, static_cast<cudaStream_t>(stream));
}

extern "C" fp8_status_t fp8_gemm_block_grouped_wgrad(int groups, const int64_t* group_ends, const uint8_t* a,
                                                     fp8_format_t fmt_a, const float* scale_inv_a, const uint8_t* b,
                                                     fp8_format_t fmt_b, const float* scale_inv_b, int64_t m, int64_t n,
                                                     int64_t rows, void* d, fp8_dtype_t out_dtype, int accumulate,
                                                     void* stream) {
    const char* fn = "fp8_gemm_block_grouped_wgrad";
    fp8_status_t s = check_groups(fn, groups, group_ends);
    if (s != FP8_OK) return s;
    const GemmProblem p = {a, b, scale_inv_a, scale_inv_b, d, group_ends, m, n, rows, groups, (int)fmt_a, (int)fmt_b,
                           false, true, out_dtype == FP8_DT_FP32, accumulate != 0};
    s = check(fn, p, FP8_B_NK, 1, out_dtype);
    if (s != FP8_OK || m == 0 || n == 0 || (rows == 0 && p.accumulate)) return s;
    return run_gemm_pair(fn, p, static_cast<cudaStream_t>(stream));
}
