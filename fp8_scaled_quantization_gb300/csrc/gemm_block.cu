// gemm_block.cu -- block-scaled FP8 products: the C entry points, their checks,
// and the guarded kernel that takes every shape and alignment.
//
// "Megatron FP8" §6 (forward, dgrad and wgrad GEMMs over FP8 operands), "Low
// Precision Training and Rollout" (128x128 weight blocks), "[Pytorch][Common]
// Hybrid quantization #2817" (1x128 / 128x1 blockwise copies for the backward
// GEMMs), "Megatron FP8" §21 (experts).
#include "fp8q_host.h"
#include "gemm_block.cuh"

namespace fp8q {
namespace {

// ------------------------------------------------------------ guarded kernel
//
// One 64 x 64 tile of D per CTA and step; 256 threads of 4 x 4 outputs each,
// operands decoded to fp32 in shared memory 32 contraction steps at a time.
// Every 128 steps the block's partial sum is multiplied by the block's scales
// and added, so partial sums and totals are both fp32.  Loads are single bytes
// behind bounds checks: any size and alignment.
constexpr int kTile = 64, kStep = 32, kThreads = 256;

__device__ __forceinline__ float decode(int fmt, uint32_t code) {
    const uint32_t h = fmt == kE4M3 ? fp8x2_to_f16x2<kE4M3>(code) : fp8x2_to_f16x2<kE5M2>(code);
    return f16_lo_to_f32(h);
}

template <bool RAGGED_K>
__global__ void __launch_bounds__(kThreads) gemm_guarded_kernel(const __grid_constant__ GemmProblem p) {
    __shared__ GroupTable groups;
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    pdl_begin();
    const int tiles_m = (int)((p.m + kTile - 1) / kTile), tiles_n = (int)((p.n + kTile - 1) / kTile);
    const int count = RAGGED_K ? p.groups : p.groups + 1;
    const int total = build_groups(&groups, p.ends, p.groups, RAGGED_K ? p.k : p.m, kTile, RAGGED_K ? p.m : 0, tiles_n);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t kb_all = blocks_of(p.k), nb_all = blocks_of(p.n);
    (void)tiles_m;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const int e = find_group(&groups, count, t);
        const int local = t - groups.tile[e];
        const int begin = e > 0 ? groups.end[e - 1] : 0, end = groups.end[e];
        const int64_t row0 = (RAGGED_K ? 0 : begin) + (int64_t)(local / tiles_n) * kTile;
        const int64_t row_end = RAGGED_K ? p.m : end;
        const int64_t col0 = (int64_t)(local % tiles_n) * kTile;
        const int64_t k_lo = RAGGED_K ? begin : 0, k_hi = RAGGED_K ? end : (e < p.groups ? p.k : 0);
        const uint8_t* b = p.b + (RAGGED_K ? 0 : (int64_t)e * p.n * p.k);
        const float* sb = p.sb + (RAGGED_K ? 0 : (int64_t)e * (p.b_tiles ? p.n : nb_all) * kb_all);
        float acc[4][4] = {};
        for (int64_t blk = k_lo / kBlk; blk * kBlk < k_hi; ++blk) {
            float part[4][4] = {};
            for (int64_t k0 = blk * kBlk; k0 < (blk + 1) * kBlk && k0 < k_hi; k0 += kStep) {
                __syncthreads();
                for (int i = threadIdx.x; i < kStep * kTile; i += kThreads) {
                    {
                        const int kk = i % kStep, r = i / kStep;
                        const int64_t k = k0 + kk, row = row0 + r;
                        const bool in = row < row_end && k >= k_lo && k < k_hi;
                        as[kk][r] = in ? decode(p.fmt_a, p.a[row * p.k + k]) : 0.0f;
                    }
                    if (p.b_kn) {
                        const int kk = i / kTile, c = i % kTile;
                        const int64_t k = k0 + kk, col = col0 + c;
                        bs[kk][c] = col < p.n && k < k_hi ? decode(p.fmt_b, b[k * p.n + col]) : 0.0f;
                    } else {
                        const int kk = i % kStep, c = i / kStep;
                        const int64_t k = k0 + kk, col = col0 + c;
                        const bool in = col < p.n && k >= k_lo && k < k_hi;
                        bs[kk][c] = in ? decode(p.fmt_b, b[col * p.k + k]) : 0.0f;
                    }
                }
                __syncthreads();
#pragma unroll 8
                for (int kk = 0; kk < kStep; ++kk) {
                    float av[4], bv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) av[i] = as[kk][ty + 16 * i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) bv[j] = bs[kk][tx + 16 * j];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[i][j] = __fmaf_rn(av[i], bv[j], part[i][j]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = row0 + ty + 16 * i;
                const float sa = row < row_end ? p.sa[row * kb_all + blk] : 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t col = col0 + tx + 16 * j;
                    if (row >= row_end || col >= p.n) continue;
                    const float s = p.b_tiles ? sb[col * kb_all + blk]
                                    : p.b_kn  ? sb[blk * nb_all + col / kBlk]
                                              : sb[col / kBlk * kb_all + blk];
                    acc[i][j] = __fmaf_rn(part[i][j], __fmul_rn(sa, s), acc[i][j]);
                }
            }
        }
        const int64_t d0 = RAGGED_K ? (int64_t)e * p.m * p.n : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t row = row0 + ty + 16 * i, col = col0 + tx + 16 * j;
                if (row >= row_end || col >= p.n) continue;
                const int64_t at = d0 + row * p.n + col;
                if (p.out_f32) {
                    float* d = static_cast<float*>(p.d) + at;
                    *d = p.accumulate ? __fadd_rn(*d, acc[i][j]) : acc[i][j];
                } else {
                    static_cast<uint16_t*>(p.d)[at] = (uint16_t)f32x2_to_bf16x2(acc[i][j], 0.0f);
                }
            }
        }
    }
}

fp8_status_t run_guarded(const char* fn, const GemmProblem& p, bool ragged_k, cudaStream_t st) {
    const int64_t tiles_n = (p.n + kTile - 1) / kTile;
    const int64_t tiles_m = ragged_k ? (p.m + kTile - 1) / kTile * p.groups : (p.m + kTile - 1) / kTile + p.groups;
    const int64_t tiles = tiles_m * tiles_n, most = (int64_t)sm_count() * 6;
    const dim3 grid((unsigned)(tiles < most ? tiles : most)), block(kThreads);
    return ragged_k ? launch(fn, gemm_guarded_kernel<true>, grid, block, st, p)
                    : launch(fn, gemm_guarded_kernel<false>, grid, block, st, p);
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
    constexpr int64_t kMost = (1ll << 31) - 256;
    if (p.m > kMost || p.n > kMost || p.k > kMost)
        return fail(FP8_ERR_UNSUPPORTED, "%s: sizes must be below 2^31 - 256", fn);
    // tiles are numbered with 32 bits
    const int64_t tn = (p.n + kTile - 1) / kTile, tm = (p.m + kTile - 1) / kTile;
    if ((tm + p.groups) * tn > kMost || (p.groups > 1 && tm * tn * p.groups > kMost))
        return fail(FP8_ERR_UNSUPPORTED, "%s: too many output tiles", fn);
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
    return p.k > 0 ? run_gemm_pair(fn, p, static_cast<cudaStream_t>(stream)) : run_guarded(fn, p, false, static_cast<cudaStream_t>(stream));
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
    return p.k > 0 ? run_gemm_pair(fn, p, static_cast<cudaStream_t>(stream)) : run_guarded(fn, p, false, static_cast<cudaStream_t>(stream));
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
    return p.k > 0 ? run_gemm_pair(fn, p, static_cast<cudaStream_t>(stream)) : run_guarded(fn, p, true, static_cast<cudaStream_t>(stream));
}
