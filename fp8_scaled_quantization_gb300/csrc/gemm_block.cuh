// gemm_block.cuh -- what the kernels of the block-scaled FP8 products share:
// the problem, and the table of ragged groups that each CTA builds in shared
// memory from the device-side group ends.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fp8q_device.cuh"
#include "fp8q_host.h"

namespace fp8q {

constexpr int kBlk = 128;          // scale block along the contraction
constexpr int kMaxGroups = 1024;   // groups of one grouped call

// D[m, n] = sum over 128-blocks b of sa[m, b] * sb[n, b] * sum_k in b of
// dec(A[m, k]) * dec(B[n, k]).  `ends` (device, `groups` entries) cuts the rows
// of A (RAGGED_M) or the contraction (RAGGED_K) into groups; NULL: one group.
struct GemmProblem {
    const uint8_t* a;
    const uint8_t* b;
    const float* sa;
    const float* sb;
    void* d;
    const int64_t* ends;
    int64_t m;  // rows of A
    int64_t n;  // columns of D
    int64_t k;  // contraction length
    int groups;
    int fmt_a, fmt_b;
    bool b_kn;       // B stored [k, n] instead of [n, k]
    bool b_tiles;    // 1 x 128 scale tiles of B instead of 128 x 128 blocks
    bool out_f32;
    bool accumulate; // D += (fp32 only)
};

// One operand as stored: `groups` row-major [rows, inner] matrices of codes.
struct Operand {
    const uint8_t* codes;
    int64_t inner, rows, groups;
    int tile_rows;  // rows of one bulk copy
};

// Tensor maps of the operands of one product.  The bulk copies need 16-byte
// aligned rows: an operand whose base or row length is not is first copied
// into the stream's scratch with its rows a multiple of 16 apart; `use` lasts
// until the product that reads it is launched.
fp8_status_t operand_maps(const char* fn, const Operand& a, CUtensorMap* map_a, const Operand& b, CUtensorMap* map_b,
                          StreamUse& use, cudaStream_t st);

// gemm_block_pair.cu: 256 x 256 outputs per CTA pair.
fp8_status_t run_gemm_pair(const char* fn, const GemmProblem& p, cudaStream_t st);

// gemm_block_stream.cu: 128 columns of D per CTA and `tokens` (16, 32, 64 or 128)
// rows at a time, k > 0; the contraction is not ragged.
fp8_status_t run_gemm_stream(const char* fn, const GemmProblem& p, int tokens, cudaStream_t st);
// How it does so: items of `tokens` rows and 128 columns (with ragged rows, at
// most), CTAs that share an item's contraction, and clusters of them at one time.
struct StreamPlan {
    int64_t items;
    int split, clusters;
};
StreamPlan stream_plan(const GemmProblem& p, int tokens, int sms);

// The first `to` of four scales; one 16-byte load where they are aligned to it
// (and the row holds all four).
__device__ __forceinline__ float4 load_scales(const float* at, int to, bool wide) {
    if (wide) return __ldg(reinterpret_cast<const float4*>(at));
    float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (to > 0) r.x = __ldg(at);
    if (to > 1) r.y = __ldg(at + 1);
    if (to > 2) r.z = __ldg(at + 2);
    if (to > 3) r.w = __ldg(at + 3);
    return r;
}

__host__ __device__ inline int64_t blocks_of(int64_t n) { return (n + kBlk - 1) / kBlk; }

// Ragged groups: end[e] is the clamped, non-decreasing end of group e, end[-1]
// reads as 0; tile[e] the number of output tiles before group e.  With rows
// ragged, a last group (index `groups`, without a contraction) holds the rows
// after the last end, whose outputs are zeros.
struct GroupTable {
    int* end;   // groups + 1 entries
    int* tile;  // groups + 2 entries

    __device__ __forceinline__ GroupTable(int* words, int groups) : end(words), tile(words + groups + 1) {}
};
__host__ __device__ constexpr size_t group_table_bytes(int groups) { return (size_t)(2 * groups + 3) * sizeof(int); }

// Every thread of the CTA calls this (it synchronises the CTA).  Group ends
// come from device memory and are never trusted: each is clamped to [0, limit]
// and to the largest end before it, so no group reaches outside the arrays.
//   limit       rows of A (RAGGED_M) or contraction length (RAGGED_K)
//   tile_rows   rows of one tile; fixed_rows > 0: every group has that many
//               output rows instead (RAGGED_K)
//   tiles_n     tiles along n
// Returns the number of tiles in all.
__device__ __forceinline__ int build_groups(const GroupTable& t, const int64_t* ends, int groups, int64_t limit,
                                            int tile_rows, int64_t fixed_rows, int tiles_n) {
    const int total = fixed_rows > 0 ? groups : groups + 1;
    if (ends == nullptr) {  // one group, known on the host
        if (threadIdx.x == 0) {
            const int64_t rows = fixed_rows > 0 ? fixed_rows : limit;
            t.end[0] = t.end[1] = (int)limit;
            t.tile[0] = 0;
            t.tile[1] = t.tile[2] = (int)((rows + tile_rows - 1) / tile_rows) * tiles_n;
        }
        __syncthreads();
        return t.tile[1];
    }
    for (int e = threadIdx.x; e < total; e += blockDim.x) {
        int64_t v = e < groups ? ends[e] : limit;
        v = v < 0 ? 0 : (v > limit ? limit : v);
        t.end[e] = (int)v;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        // lane l owns entries [l * per, (l + 1) * per): running maxima, then tiles
        const int lane = threadIdx.x, per = (total + 31) / 32;
        const int lo = min(lane * per, total), hi = min(lo + per, total);
        int mx = 0;
        for (int e = lo; e < hi; ++e) mx = max(mx, t.end[e]);
        int before = mx;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
            if (lane >= o) before = max(before, v);
        }
        before = __shfl_up_sync(0xFFFFFFFFu, before, 1);
        if (lane == 0) before = 0;
        int run = before, sum = 0;
        for (int e = lo; e < hi; ++e) {
            const int end = max(run, t.end[e]);
            const int64_t rows = fixed_rows > 0 ? fixed_rows : end - run;
            t.end[e] = end;
            run = end;
            sum += (int)((rows + tile_rows - 1) / tile_rows) * tiles_n;
        }
        int pre = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, pre, o);
            if (lane >= o) pre += v;
        }
        pre -= sum;
        run = before;
        for (int e = lo; e < hi; ++e) {
            const int end = t.end[e];
            const int64_t rows = fixed_rows > 0 ? fixed_rows : end - run;
            run = end;
            t.tile[e] = pre;
            pre += (int)((rows + tile_rows - 1) / tile_rows) * tiles_n;
        }
        if (lane == 31) t.tile[total] = pre;
    }
    __syncthreads();
    return t.tile[total];
}

// Group of tile `i`: the last one that begins at or before it (groups without
// tiles share their begin with the next one).
__device__ __forceinline__ int find_group(const GroupTable& t, int total, int i) {
    int lo = 0, hi = total - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.tile[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace fp8q
