// gemm_block_pair.cu -- block-scaled FP8 products on the tensor cores, 256 x
// 256 outputs per pair of CTAs.
//
// The scales change every 128 contraction steps, and they are fp32 numbers, so
// they cannot ride in the tensor core: each block's product P_b is formed in
// TMEM from zero (four instructions of 32 steps), and eight warps per CTA read
// it back and add s * P_b to accumulators in registers (128 outputs per lane).
// Two TMEM buffers of 256 columns let the next block's product run meanwhile.
//
// Roles per CTA of 384 threads: warps 0-7 scale and add, then store; warp 8 of
// the pair's first CTA issues the products for both; warp 9 gathers the scales
// and says where each tile lies; warp 10 fills the ring of operand tiles by bulk
// copies; warp 11 zeroes the steps of other groups in blocks that a ragged
// group's end cuts.
//
// What bounds it, per block of 512 tensor-core cycles.  128 x 128 blocks, 800
// cycles: the way of a TMEM buffer around.  Sixteen warps read it (the reads run
// one piece ahead of the arithmetic, whose rate sets their time: 480 cycles), they
// arrive across the pair, the product is issued, takes its 512, and reports back
// to both CTAs; two buffers share that way, and TMEM has no room for a third
// (four of half the width run the tensor core at half its rate: 1000 cycles).
// 1 x 128 tiles, 1240 cycles: the scaling warps themselves, with two operations
// per element and 1020 cycles without any wait.  A spill in the loop costs more
// than any of this gains (a load from local memory takes 300 cycles with shared
// memory this full).  A tile costs another 2500 cycles (fp32 outputs: 4900),
// mostly to store it.
// Measured, a call after a pause and calls back to back, where the power limit holds
// the SM clock at 1730 to 1880 MHz instead of 2070: 4001 x 7168 x 18432 (rows, n, k)
// 389 and 429 us (2720 and 2460 TFLOP/s); 16384 x 18432 x 7168 against [k, n] 1.54 and
// 1.70 ms (2810, 2550); 4096 x 14336 x 8192 in 1 x 128 tiles 528 and 538 us (1820, 1790).
// Two figures beside one choice below were taken together, after pauses: compare
// them with one another only.
#include "fp8q_host.h"
#include "fp8q_tcgen05.cuh"
#include "gemm_block.cuh"

namespace fp8q {
namespace {

constexpr int kThreads = 384;
constexpr int kPairM = 256, kPairN = 256;  // outputs of a pair
constexpr int kScaleBlocks = 4;            // blocks of a tile whose scales are gathered together
constexpr int kScaleSlots = 3;             // such groups in the scale ring
// The scale warp is at most kScaleSlots groups ahead, so it writes a tile's place
// over that of a tile that every scaling warp has left.
constexpr int kPlaces = kScaleSlots + 1;
constexpr int kRaster = 8;                 // tiles along m that are walked before the next tile along n
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kOutBytes = 32 * 128;   // one staging buffer of a warp: 32 rows of 128 bytes

// Operand ring (A and B tile, 32 KB per CTA and stage) and staging buffers per
// warp: the second buffer gains 2%, a fifth stage in its place nothing.
constexpr int kStages = 4, kOuts = 2;

template <bool TILES>
struct Shared {
    union {
        float4 rows[kScaleSlots][2][128];  // 128 x 128 blocks: per column half and row, row scale x column block scale
        struct {
            float a[kScaleSlots][kScaleBlocks][128];    // 1 x 128 tiles: per block and row,
            alignas(8) float b[kScaleSlots][kScaleBlocks][kPairN];  // and per block and column
        } tile;
    } sc;
    int4 place[kPlaces];  // of the tiles under way: first row, end of rows, first column, blocks
    int matrix[kPlaces];  // and group
    uint64_t full[kStages], empty[kStages], landed[kStages];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
    uint32_t tmem, dead;
    int groups[2 * kMaxGroups + 3];
};
template <bool TILES>
constexpr size_t smem_bytes() {
    constexpr size_t bytes =
        1024 + (size_t)kStages * kStageBytes + 8 * kOuts * kOutBytes + sizeof(Shared<TILES>);
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    return bytes;
}

// Where a tile's operands and outputs lie.
struct Tile {
    int group;
    int row0, row_end;  // of A (and D)
    int col0;
    int k_lo, k_hi;     // contraction range
    int blk0, blks;     // its 128-blocks
};

template <bool RAGGED_K>
__device__ __forceinline__ Tile locate(const GemmProblem& p, const GroupTable& g, int count, int tiles_n, int t) {
    Tile r;
    const int e = find_group(g, count, t);
    const int local = t - g.tile[e], begin = e > 0 ? g.end[e - 1] : 0, end = g.end[e];
    const int m = (int)p.m, k = (int)p.k, rows = RAGGED_K ? m : end - begin;
    const int tiles_m = (rows + kPairM - 1) / kPairM;
    // columns of kRaster tiles along m: what runs at one time shares operands in L2
    const int strip = local / (kRaster * tiles_n), in_strip = local - strip * kRaster * tiles_n;
    const int high = min(kRaster, tiles_m - strip * kRaster);
    r.group = e;
    r.row0 = (RAGGED_K ? 0 : begin) + (strip * kRaster + in_strip % high) * kPairM;
    r.row_end = RAGGED_K ? m : end;
    r.col0 = in_strip / high * kPairN;
    r.k_lo = RAGGED_K ? begin : 0;
    r.k_hi = RAGGED_K ? end : (e < p.groups ? k : 0);
    // an empty contraction has no blocks, wherever it lies
    r.blk0 = r.k_hi > r.k_lo ? r.k_lo / kBlk : 0;
    r.blks = r.k_hi > r.k_lo ? (r.k_hi + kBlk - 1) / kBlk - r.blk0 : 0;
    return r;
}

// Whether the block at step x holds steps of other groups (beyond the last step
// the bulk copy fills with zeros itself).
__device__ __forceinline__ bool is_cut(const Tile& t, int x, int k) {
    return x < t.k_lo || (x + kBlk > t.k_hi && t.k_hi < k);
}

// Zeroes the bytes outside [lo, hi) of every row of the stage's two K-major tiles,
// by one warp: a 16-byte column of all rows at a time, and only a column that lo or
// hi divides is read (4 rows of each tile per lane at once, for one latency).
__device__ __forceinline__ void mask_stage(uint32_t stage, int lo, int hi, int lane) {
#pragma unroll 1
    for (int piece = 0; piece < 8; ++piece) {
        const int from = max(lo - piece * 16, 0), to = min(hi - piece * 16, 16);
        if (from <= 0 && to >= 16) continue;
        const uint32_t at = stage + lane * 128 + ((piece ^ (lane & 7)) << 4);
        uint32_t v[8][4] = {};
        if (from < to) {
            uint32_t keep[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                keep[w] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * w + i >= from && 4 * w + i < to) keep[w] |= 0xFFu << (8 * i);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                             : "r"(at + i * 32 * 128)
                             : "memory");
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) v[i][w] &= keep[w];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + i * 32 * 128), "r"(v[i][0]), "r"(v[i][1]),
                         "r"(v[i][2]), "r"(v[i][3])
                         : "memory");
    }
}

// A lane's 128 sums.  1 x 128 tiles, with two operations per element, keep them
// as 64 packed pairs (single numbers: 7% slower).  Else they are single numbers,
// although a packed operation does two: for packed pairs the compiler finds no
// registers to read the products one piece ahead, and 3 to 4% are lost.
template <bool TILES>
struct Sums {
    float v[128];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = 0.0f;
    }
    __device__ __forceinline__ float2 pair(int q) const { return make_float2(v[2 * q], v[2 * q + 1]); }
};
template <>
struct Sums<true> {
    uint64_t v[64];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = 0;
    }
    __device__ __forceinline__ float2 pair(int q) const { return unpack2(v[q]); }
};

// Which of a warp's 32 x 128 outputs the pair q of a lane's sums holds: columns
// col, col + 1 of row `row`.  TILES: the 16x256b order of TMEM, in which a lane
// has 4 rows and 32 columns; else lane = row and the 128 columns in order.
template <bool TILES>
__device__ __forceinline__ int row_of(int q, int lane) {
    return TILES ? (q >> 4 & 1) * 16 + (q & 1) * 8 + (lane >> 2) : lane;
}
template <bool TILES>
__device__ __forceinline__ int col_of(int q, int lane) {
    return TILES ? (q >> 5) * 64 + (q >> 1 & 7) * 8 + 2 * (lane & 3) : 2 * q;
}

// 128 bytes of each of a warp's rows, piece `part`, to shared memory.
template <bool TILES>
__device__ __forceinline__ void stage_out(bool f32, const Sums<TILES>& acc, int part, uint32_t stage, int lane) {
    if constexpr (TILES) {
        if (f32) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {  // 4 column blocks of 8, 4 rows
                const int q = (part >> 1) * 32 + (i >> 1 & 1) * 16 + ((part & 1) * 4 + (i >> 2)) * 2 + (i & 1);
                const int r = row_of<true>(q, lane), at = (col_of<true>(q, lane) & 31) * 4;
                const float2 v = acc.pair(q);
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(stage + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15)),
                             "f"(v.x), "f"(v.y)
                             : "memory");
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {  // 8 column blocks of 8, 4 rows
                const int q = (part & 1) * 32 + i;
                const int r = row_of<true>(q, lane), at = (col_of<true>(q, lane) & 63) * 2;
                const float2 v = acc.pair(q);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15)),
                             "r"(f32x2_to_bf16x2(v.x, v.y))
                             : "memory");
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t o[4];
            if (f32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 v = acc.pair(part * 16 + 2 * j + i);
                    o[2 * i] = __float_as_uint(v.x);
                    o[2 * i + 1] = __float_as_uint(v.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = acc.pair((part & 1) * 32 + 4 * j + i);
                    o[i] = f32x2_to_bf16x2(v.x, v.y);
                }
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((j ^ (lane & 7)) << 4)), "r"(o[0]),
                         "r"(o[1]), "r"(o[2]), "r"(o[3])
                         : "memory");
        }
    }
}

// Such a piece (outputs from column x on) from shared memory to D by plain stores
// and, when accumulating, loads: a row per step.
__device__ __forceinline__ void copy_out(const GemmProblem& p, uint32_t stage, int lane, int64_t base, int64_t row0,
                                         int64_t row_end, int64_t x) {
    const int rows = (int)(row_end - row0 < 32 ? row_end - row0 : 32), mine = p.out_f32 ? 1 : 2;
    const int64_t c = x + lane * mine;
    if (c >= p.n) return;
    const bool both = c + 1 < p.n, pair = (p.n & 1) == 0 && (reinterpret_cast<uintptr_t>(p.d) & 3u) == 0;
    uint8_t* d = static_cast<uint8_t*>(p.d) + (base + row0 * p.n + c) * (p.out_f32 ? 4 : 2);
    const int64_t pitch = p.n * (p.out_f32 ? 4 : 2);
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8, d += 8 * pitch) {
        const int to = min(rows - r0, 8);
        float old[8];
        if (p.accumulate) {
#pragma unroll
            for (int r = 0; r < 8; ++r) old[r] = r < to ? *reinterpret_cast<const float*>(d + r * pitch) : 0.0f;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r >= to) break;
            uint32_t v;
            asm volatile("ld.shared.u32 %0, [%1];"
                         : "=r"(v)
                         : "r"(stage + (r0 + r) * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4)
                         : "memory");
            if (p.out_f32) {
                const float f = __uint_as_float(v);
                *reinterpret_cast<float*>(d + r * pitch) = p.accumulate ? __fadd_rn(old[r], f) : f;
            } else if (pair) {
                *reinterpret_cast<uint32_t*>(d + r * pitch) = v;
            } else {
                uint16_t* const h = reinterpret_cast<uint16_t*>(d + r * pitch);
                h[0] = (uint16_t)v;
                if (both) h[1] = (uint16_t)(v >> 16);
            }
        }
    }
}

// The same where all rows of D are aligned to 16 bytes and nothing is added: 16
// bytes per lane, four rows per step (8191 rows over 16 experts, 7168 x 2048: 133
// us, a row per step 146; sums onto D gain nothing by it).
__device__ __forceinline__ void copy_out_wide(const GemmProblem& p, uint32_t stage, int lane, int matrix, int64_t row0,
                                              int64_t row_end, int64_t x) {
    const int r = lane >> 3, piece = lane & 7, size = p.out_f32 ? 4 : 2;
    const int rows = (int)(row_end - row0 < 32 ? row_end - row0 : 32) - r;
    const int64_t c = x + piece * (16 / size), pitch = p.n * size;
    if (c >= p.n) return;
    uint8_t* const d = static_cast<uint8_t*>(p.d) + ((int64_t)matrix * p.m + row0 + r) * pitch + c * size;
#pragma unroll
    for (int at = 0; at < 32; at += 8) {
        uint32_t v[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                         : "r"(stage + (r + at + 4 * i) * 128 + ((piece ^ ((r + 4 * i) & 7)) << 4))
                         : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at + 4 * i < rows)
                *reinterpret_cast<uint4*>(d + (at + 4 * i) * pitch) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
    }
}

// A warp's 32 x 128 outputs from (row0, c0) on: 128 bytes of each row at a time
// go through shared memory (16-byte pieces swizzled, so that the accesses spread
// over the banks).  Where all 32 rows are in the group the bulk-copy engine
// writes them and drops what lies outside D; rows that a group's end cuts,
// unaligned outputs and sums onto D take plain stores.
template <bool TILES>
__device__ __forceinline__ void store_tile(const GemmProblem& p, const CUtensorMap* map, bool bulk, const Sums<TILES>& acc,
                                           uint32_t stages, int lane, int64_t row0, int64_t row_end, int64_t c0, int matrix) {
#pragma unroll
    for (int part = 0; part < 4; ++part) {
        const uint32_t stage = stages + part % kOuts * kOutBytes;
        if (part >= 2 && !p.out_f32) break;
        const int64_t x = c0 + part * (p.out_f32 ? 32 : 64);
        if (x < p.n) {
            if (lane == 0)  // this buffer has been read: every piece commits a group, if an empty one
                asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kOuts - 1) : "memory");
            __syncwarp();
            stage_out<TILES>(p.out_f32, acc, part, stage, lane);
            if (bulk && row0 + 31 < row_end) {
                fence_to_async();
                __syncwarp();
                if (lane == 0)
                    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                                     reinterpret_cast<uint64_t>(map)),
                                 "r"((int)x), "r"((int)row0), "r"(matrix), "r"(stage)
                                 : "memory");
            } else if (bulk) {
                __syncwarp();
                copy_out_wide(p, stage, lane, matrix, row0, row_end, x);
                __syncwarp();
            } else {
                __syncwarp();
                copy_out(p, stage, lane, (int64_t)matrix * p.m * p.n, row0, row_end, x);
                __syncwarp();
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// FORM 0: B [n, k], 128 x 128 blocks; 1: B [k, n], 128 x 128 blocks; 2: both
// operands in 1 x 128 tiles, contraction ragged.
template <int FORM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_pair_kernel(const __grid_constant__ GemmProblem p, const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_d, bool bulk_store) {
    constexpr bool RAGGED_K = FORM == 2, B_KN = FORM == 1, B_TILES = FORM == 2;
    extern __shared__ uint8_t raw[];
    uint8_t* const tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* const out = tiles + kStages * kStageBytes;
    Shared<B_TILES>& sh = *reinterpret_cast<Shared<B_TILES>*>(out + 8 * kOuts * kOutBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        sh.dead = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);   // one arrival per CTA of the pair
            mbar_init(&sh.empty[i], 1);  // the products' commit
            mbar_init(&sh.landed[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.tmem_full[i], 1);
            mbar_init(&sh.tmem_empty[i], 16);  // eight warps of each CTA
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.sc_full[i], 1);
            mbar_init(&sh.sc_empty[i], 8);
        }
        mbar_init_fence();
    }
    if (warp == 8) tmem_alloc<2>(&sh.tmem, 512);
    if (threadIdx.x == 320) {
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    pdl_begin();
    const int tiles_n = (int)((p.n + kPairN - 1) / kPairN);
    const int count = RAGGED_K ? p.groups : p.groups + 1;
    const GroupTable groups(sh.groups, p.groups);
    const int total = build_groups(groups, p.ends, p.groups, RAGGED_K ? p.k : p.m, kPairM, RAGGED_K ? p.m : 0, tiles_n);
    tmem_fence_before();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    Waiter w;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 128;
        const uint32_t full0 = smem_addr(&sh.tmem_full[0]), empty0 = cluster_addr(smem_addr(&sh.tmem_empty[0]), 0);
        uint32_t it = 0, group = 0, at_place = 0;  // blocks and scale groups so far; this tile's place
        for (int t = first; t < total; t += step) {
            Sums<B_TILES> acc;
            acc.clear();
            float4 s4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), s4_next = s4;
            uint32_t slot = 0;
            // the next group of scales is there; 128 x 128 blocks: this row's four live in registers from here on
            const auto fetch = [&]() {
                slot = group % kScaleSlots;
                w.wait(smem_addr(&sh.sc_full[slot]), (group / kScaleSlots) & 1);
                __syncwarp();
                if constexpr (!B_TILES) {
                    s4_next = sh.sc.rows[slot][half][row];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.sc_empty[slot]);
                }
                ++group;
            };
            const auto release = [&]() {  // 1 x 128 tiles: every lane has read the group
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.sc_empty[slot]);
            };
            fetch();
            const int blks = sh.place[at_place].w;
            if (B_TILES && blks == 0) release();
            bool ready = false;  // (asking one block ahead pays with 1 x 128 tiles only)
            for (int b = 0; b < blks; ++b) {
                const uint32_t buf = it & 1, from = lanes + buf * kPairN;
                const int sub = b % kScaleBlocks;
                if (B_TILES && b > 0 && sub == 0) fetch();
                if (!B_TILES) s4 = sub == 0 ? s4_next : make_float4(s4.y, s4.z, s4.w, 0.0f);
                if (!B_TILES || !ready) w.wait(full0 + buf * 8, (it >> 1) & 1);
                __syncwarp();  // lanes may have left the wait apart
                tmem_fence_after();
                ++it;
                const auto read = [&]() {  // the buffer has been read
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) cluster_arrive<false>(empty0 + buf * 8);
                    if (B_TILES) ready = Waiter::test(full0 + (it & 1) * 8, (it >> 1) & 1);
                };
                if constexpr (B_TILES) {
                    uint64_t sr[4];  // this lane's four rows
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float f = sh.sc.tile.a[slot][sub][(warp & 3) * 32 + i * 8 + (lane >> 2)];
                        sr[i] = pack2(f, f);
                    }
                    const float2* const sb = reinterpret_cast<const float2*>(&sh.sc.tile.b[slot][sub][half * 128]) + (lane & 3);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint64_t sc[8];  // and eight of its column pairs
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 f = sb[h * 32 + i * 4];
                            sc[i] = pack2(f.x, f.y);
                        }
#pragma unroll
                        for (int rh = 0; rh < 2; ++rh) {
                            uint32_t v[32];
                            tmem_ld_16x64(from + ((uint32_t)(rh * 16) << 16) + h * 64, v);
                            tmem_wait_ld();
                            if (h + rh == 2) read();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                uint64_t* const at = acc.v + h * 32 + rh * 16 + i * 2;
                                at[0] = fma2(mul2(pack2(v[4 * i], v[4 * i + 1]), sc[i]), sr[rh * 2], at[0]);
                                at[1] = fma2(mul2(pack2(v[4 * i + 2], v[4 * i + 3]), sc[i]), sr[rh * 2 + 1], at[1]);
                            }
                        }
                    }
                    if (sub == kScaleBlocks - 1 || b == blks - 1) release();
                } else {
                    uint32_t v[2][16];
                    tmem_ld_32x16(from, v[0]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {  // reads run one piece ahead
                        tmem_wait_ld();
                        if (c < 7) tmem_ld_32x16(from + (c + 1) * 16, v[(c + 1) & 1]);
                        else read();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc.v[c * 16 + j] = __fmaf_rn(__uint_as_float(v[c & 1][j]), s4.x, acc.v[c * 16 + j]);
                        if (c == 1 && sub == 2 && b + 2 < blks) fetch();
                    }
                }
            }
            // store: this warp's 32 rows, 128 columns
            const int4 place = sh.place[at_place];
            const int matrix = RAGGED_K ? sh.matrix[at_place] : 0;
            at_place = (at_place + 1) % kPlaces;
            const int64_t r0 = place.x + (int)rank * 128 + (warp & 3) * 32, c0 = place.z + half * 128;
            store_tile<B_TILES>(p, &map_d, bulk_store, acc, smem_addr(out) + warp * kOuts * kOutBytes, lane, r0, place.y, c0,
                                matrix);
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) {
            // ---- products: the whole warp of the pair's first CTA walks, one thread issues
            if (rank == 0) {
                const uint32_t desc = mma_desc(p.fmt_a, p.fmt_b, false, B_KN, kPairM, kPairN);
                const uint64_t a0 = tile_desc(smem_addr(tiles)), b0 = tile_desc(smem_addr(tiles) + kTileBytes);
                uint32_t it = 0, stage = 0, phase = 0;
                for (int t = first; t < total; t += step) {
                    const int blks = locate<RAGGED_K>(p, groups, count, tiles_n, t).blks;
                    for (int b = 0; b < blks; ++b) {
                        const uint64_t at = a0 + stage * (kStageBytes >> 4), bt = b0 + stage * (kStageBytes >> 4);
                        const uint32_t buf = it & 1;
                        // (tiles that were masked with plain stores are released to the cluster)
                        w.template wait<RAGGED_K>(smem_addr(&sh.full[stage]), phase);
                        if (it >= 2) w.wait(smem_addr(&sh.tmem_empty[buf]), ((it >> 1) & 1) ^ 1);
                        ++it;
                        __syncwarp();
                        tmem_fence_after();
                        if (elect_one() && !w.dead) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_f8<2>(tmem + buf * kPairN, at + k * kStepKMajor, bt + k * (B_KN ? kStepMnMajor : kStepKMajor),
                                          desc, k > 0);
                            mma_commit<2>(smem_addr(&sh.tmem_full[buf]));
                            mma_commit<2>(smem_addr(&sh.empty[stage]));
                        }
                        __syncwarp();
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                // the other CTA's last arrivals on this one's barriers have come before it ends
                for (uint32_t i = it > 2 ? it - 2 : 0; i < it; ++i) w.wait(smem_addr(&sh.tmem_empty[i & 1]), (i >> 1) & 1);
            }
        } else if (warp == 9) {
            // ---- scales: this CTA's 128 rows and the pair's 256 columns (or their two 128-blocks)
            const int64_t kb = blocks_of(p.k), nb = blocks_of(p.n);
            const bool wide_a = kb % kScaleBlocks == 0 && (reinterpret_cast<uintptr_t>(p.sa) & 15u) == 0;
            const bool wide_b = kb % kScaleBlocks == 0 && (reinterpret_cast<uintptr_t>(p.sb) & 15u) == 0;
            uint32_t group = 0, at_place = 0;
            for (int t = first; t < total; t += step) {
                const Tile tile = locate<RAGGED_K>(p, groups, count, tiles_n, t);
                for (int done = 0; done == 0 || done < tile.blks; done += kScaleBlocks, ++group) {  // (once without blocks, too)
                    const int g0 = tile.blk0 + done, to = min(tile.blks - done, kScaleBlocks);
                    const bool whole = to > 0 && g0 % kScaleBlocks == 0;  // an aligned piece of a row of scales
                    const uint32_t slot = group % kScaleSlots;
                    float4 a[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // a row or column that is not there: any scale
                        const int64_t r = tile.row0 + (int)rank * 128 + i * 32 + lane;
                        a[i] = load_scales(p.sa + (r < p.m ? r : p.m - 1) * kb + g0, to, wide_a && whole);
                    }
                    if constexpr (B_TILES) {
                        if (group >= kScaleSlots) w.wait(smem_addr(&sh.sc_empty[slot]), (group / kScaleSlots - 1) & 1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float* dst = &sh.sc.tile.a[slot][0][i * 32 + lane];
                            dst[0] = a[i].x;
                            dst[128] = a[i].y;
                            dst[256] = a[i].z;
                            dst[384] = a[i].w;
                        }
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int64_t n = tile.col0 + h * 128 + i * 32 + lane;
                                a[i] = load_scales(p.sb + (n < p.n ? n : p.n - 1) * kb + g0, to, wide_b && whole);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float* dst = &sh.sc.tile.b[slot][0][h * 128 + i * 32 + lane];
                                dst[0] = a[i].x;
                                dst[kPairN] = a[i].y;
                                dst[2 * kPairN] = a[i].z;
                                dst[3 * kPairN] = a[i].w;
                            }
                        }
                    } else {
                        // lanes 4h + j load the scale of block g0 + j, column block h
                        const int64_t n = tile.col0 / kBlk + ((lane >> 2) & 1), cb = n < nb ? n : nb - 1;
                        const float* sb = p.sb + (int64_t)tile.group * kb * nb;
                        const int j = lane & 3;
                        float c = 0.0f;
                        if (j < to) c = __ldg(sb + (B_KN ? (int64_t)(g0 + j) * nb + cb : cb * kb + g0 + j));
                        if (group >= kScaleSlots) w.wait(smem_addr(&sh.sc_empty[slot]), (group / kScaleSlots - 1) & 1);
                        __syncwarp();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float c0 = __shfl_sync(0xFFFFFFFFu, c, 4 * h), c1 = __shfl_sync(0xFFFFFFFFu, c, 4 * h + 1);
                            const float c2 = __shfl_sync(0xFFFFFFFFu, c, 4 * h + 2), c3 = __shfl_sync(0xFFFFFFFFu, c, 4 * h + 3);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sh.sc.rows[slot][h][i * 32 + lane] = make_float4(__fmul_rn(a[i].x, c0), __fmul_rn(a[i].y, c1),
                                                                                 __fmul_rn(a[i].z, c2), __fmul_rn(a[i].w, c3));
                        }
                    }
                    if (done == 0 && lane == 0) {
                        sh.place[at_place] = make_int4(tile.row0, tile.row_end, tile.col0, tile.blks);
                        sh.matrix[at_place] = tile.group;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.sc_full[slot]);
                }
                at_place = (at_place + 1) % kPlaces;
            }
        } else if (warp == 10) {
            // ---- operand tiles: A rows [row0 + 128 rank, ..), B columns [col0 + 128 rank, ..)
            const uint32_t base = smem_addr(tiles), full0 = cluster_addr(smem_addr(&sh.full[0]), 0);
            uint32_t it = 0, stage = 0, phase = 0;
            for (int t = first; t < total; t += step) {
                const Tile tile = locate<RAGGED_K>(p, groups, count, tiles_n, t);
                const int row = tile.row0 + (int)rank * 128, col = tile.col0 + (int)rank * 128;
                for (int b = 0; b < tile.blks; ++b, ++it) {
                    const uint32_t a = base + stage * kStageBytes, bt = a + kTileBytes;
                    const int x = (tile.blk0 + b) * kBlk;
                    if (it >= kStages) w.wait(smem_addr(&sh.empty[stage]), phase ^ 1);
                    __syncwarp();
                    if (elect_one() && !w.dead) {
                        // a block that needs masking lands on this CTA's own barrier first
                        uint32_t bar = full0 + stage * 8;
                        if (RAGGED_K && is_cut(tile, x, (int)p.k)) bar = smem_addr(&sh.landed[stage]);
                        cluster_arrive_expect_tx(bar, kStageBytes);
                        tma_tile<true>(a, &map_a, x, row, 0, bar);
                        if constexpr (B_KN) tma_tile<true>(bt, &map_b, col, x, tile.group, bar);
                        else tma_tile<true>(bt, &map_b, x, col, RAGGED_K ? 0 : tile.group, bar);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // the last fills have been read before the CTA ends
            for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
                w.wait(smem_addr(&sh.empty[i % kStages]), (i / kStages) & 1);
        } else if (RAGGED_K) {
            // ---- masking: steps of other groups become zeros, in both operands (their codes may be NaN)
            const uint32_t base = smem_addr(tiles), full0 = cluster_addr(smem_addr(&sh.full[0]), 0);
            uint32_t stage = 0, phases = 0;  // bit s: the phase of landed[s]
            uint32_t passed = 0;             // blocks and tiles since this warp last waited
            for (int t = first; t < total; t += step, ++passed) {
                const Tile tile = locate<RAGGED_K>(p, groups, count, tiles_n, t);
                for (int b = 0; b < tile.blks; ++b, ++passed) {
                    const int x = (tile.blk0 + b) * kBlk;
                    if (is_cut(tile, x, (int)p.k)) {
                        // The other roles keep step with the ring; this one waits here while they go
                        // through all that it passed.  A contraction of 8e8 steps takes 4 s, so each
                        // 2^16 blocks (0.05 s, tiles of one block 0.2) add a limit's time.
                        const uint32_t bar = smem_addr(&sh.landed[stage]), parity = phases >> stage & 1;
                        for (uint32_t i = passed >> 16; i > 0 && !w.dead && !Waiter::within_limit(bar, parity); --i)
                            if (*(volatile uint32_t*)&sh.dead != 0) break;
                        passed = 0;
                        w.wait(bar, parity);
                        phases ^= 1u << stage;
                        __syncwarp();
                        mask_stage(base + stage * kStageBytes, tile.k_lo - x, tile.k_hi - x, lane);
                        fence_to_async();
                        __syncwarp();
                        if (lane == 0 && !w.dead) cluster_arrive<true>(full0 + stage * 8);
                    }
                    if (++stage == kStages) stage = 0;
                }
            }
        }
        __syncwarp();
    }
    if (w.dead) report_dead(smem_addr(&sh.dead), 2);
    tmem_fence_before();
    cluster_meet();
    if (sh.dead != 0) {
        linger();
        cluster_meet();
    }
    tmem_fence_after();
    if (warp == 8) tmem_free<2>(tmem, 512);
}

}  // namespace

fp8_status_t run_gemm_pair(const char* fn, const GemmProblem& p, cudaStream_t st) {
    const int64_t inner_b = p.b_kn ? p.n : p.k, rows_b = p.b_kn ? p.k : p.n;
    const bool bulk = aligned16(p.d) && p.n % (p.out_f32 ? 4 : 8) == 0 && !p.accumulate;
    const Operand oa = {p.a, p.k, p.m, 1, 128}, ob = {p.b, inner_b, rows_b, p.b_tiles ? 1 : p.groups, 128};
    CUtensorMap a = {}, b = {}, d = {};
    StreamUse use(st);
    fp8_status_t s = FP8_OK;
    if (p.k > 0) s = operand_maps(fn, oa, &a, ob, &b, use, st);
    if (bulk && s == FP8_OK) s = encode_out_map(&d, p.d, p.out_f32, p.n, p.m, p.b_tiles ? p.groups : 1);
    if (s != FP8_OK) return s;
    const int64_t tiles_n = (p.n + kPairN - 1) / kPairN, tiles_m = (p.m + kPairM - 1) / kPairM;
    const int64_t most = p.b_tiles ? tiles_m * tiles_n * p.groups : (tiles_m + p.groups - 1) * tiles_n;
    const int sms = sm_count() / 2, pairs = (int)(most < sms ? most : sms);
    const auto go = [&](auto kernel, size_t smem) {
        return launch_smem(fn, kernel, dim3(2 * pairs), dim3(kThreads), smem, st, p, a, b, d, bulk);
    };
    return p.b_tiles ? go(gemm_pair_kernel<2>, smem_bytes<true>())
           : p.b_kn  ? go(gemm_pair_kernel<1>, smem_bytes<false>())
                     : go(gemm_pair_kernel<0>, smem_bytes<false>());
}

fp8_status_t gemm_pair_wait_timeouts(unsigned long long* count) {
    return cuda_status(cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof *count), "fp8_wait_timeouts");
}

}  // namespace fp8q
