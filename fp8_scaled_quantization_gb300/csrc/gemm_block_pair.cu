// gemm_block_pair.cu -- block-scaled FP8 products on the tensor cores, 256 x
// 256 outputs per pair of CTAs.
//
// The scales change every 128 contraction steps, and they are fp32 numbers, so
// they cannot ride in the tensor core: each block's product P_b is formed in
// TMEM from zero (four instructions of 32 steps), and eight warps per CTA read
// it back and add s * P_b to accumulators in registers (one row per lane, 128
// columns per thread, packed two-lane fused multiply-adds).  Two TMEM buffers
// of 256 columns let the next block's product run meanwhile.
//
// Roles per CTA of 384 threads: warps 0-7 scale and add, then store; warp 8 of
// the pair's first CTA issues the products for both; warp 9 gathers the scales;
// warp 10 fills the ring of operand tiles by bulk copies; warp 11 zeroes the
// steps of other groups in blocks that a ragged group's end cuts.
//
// What bounds it: the scaling warps.  A block takes the tensor core 512 cycles
// and the warps about 890 (1 x 128 tiles: 1340): the arithmetic of a scheduler's
// two warps is 292, and the way of each warp through a block -- the barrier's
// answer 190 cycles, four reads of TMEM with their arithmetic 100 each, the
// arrival, the loop -- hides behind the other's in part only.  A third warp per
// scheduler or reads further ahead do not fit the registers: any spill costs
// more (a load from local memory takes 300 cycles with shared memory this full).
// Measured: 8192^3 418 us, 2630 TFLOP/s; 16384 x 18432 x 7168 in one call 1.6
// ms; products alone, without scaling, would take 266 us.  The SM clock falls
// from 2070 to about 1850 MHz meanwhile (power).
#include "fp8q_host.h"
#include "fp8q_tcgen05.cuh"
#include "gemm_block.cuh"

namespace fp8q {
namespace {

constexpr int kThreads = 384;
constexpr int kPairM = 256, kPairN = 256;  // outputs of a pair
constexpr int kScaleBlocks = 4;            // blocks of a tile whose scales are gathered together
constexpr int kScaleSlots = 3;             // such groups in the scale ring
constexpr int kRaster = 8;                 // tiles along m that are walked before the next tile along n
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t kOutBytes = 32 * 128;   // one staging buffer of a warp: 32 rows of 128 bytes

// Operand ring (A and B tile, 32 KB per CTA and stage) and staging buffers per
// warp.  With 128 x 128 blocks two buffers gain 2% and the fifth stage nothing;
// with ragged contractions, whose cut blocks stay longer in the ring, the fifth
// stage is worth 4%.
template <bool TILES>
struct Ring {
    static constexpr int kStages = TILES ? 5 : 4, kOuts = TILES ? 1 : 2;
};

template <bool TILES>
struct Shared {
    static constexpr int kStages = Ring<TILES>::kStages;
    union {
        float4 rows[kScaleSlots][2][128];  // 128 x 128 blocks: per column half and row, row scale x column block scale
        struct {
            float a[kScaleSlots][kScaleBlocks][128];    // 1 x 128 tiles: per block and row,
            alignas(8) float b[kScaleSlots][kScaleBlocks][kPairN];  // and per block and column
        } tile;
    } sc;
    uint64_t full[kStages], empty[kStages], landed[kStages];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
    uint32_t tmem, dead;
    int groups[2 * kMaxGroups + 3];
};
template <bool TILES>
constexpr size_t smem_bytes() {
    constexpr size_t bytes =
        1024 + (size_t)Ring<TILES>::kStages * kStageBytes + 8 * Ring<TILES>::kOuts * kOutBytes + sizeof(Shared<TILES>);
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

// Zeroes the bytes outside [lo, hi) of every row of a K-major tile, by one warp.
__device__ __forceinline__ void mask_tile(uint32_t tile, int lo, int hi, int lane) {
    const int piece = lane & 7, from = max(lo - piece * 16, 0), to = min(hi - piece * 16, 16);
    if (from <= 0 && to >= 16) return;
    uint32_t keep[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        keep[w] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * w + i >= from && 4 * w + i < to) keep[w] |= 0xFFu << (8 * i);
    }
    const bool some = (keep[0] | keep[1] | keep[2] | keep[3]) != 0;
#pragma unroll 4
    for (int r = lane >> 3; r < 128; r += 4) {
        const uint32_t at = tile + r * 128 + ((piece ^ (r & 7)) << 4);
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (some) {
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(at)
                         : "memory");
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] &= keep[w];
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                     : "memory");
    }
}

// Which of a warp's 32 x 128 outputs the pair acc[q] of a lane holds: columns
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

// A warp's 32 x 128 outputs from (row0, c0) on, by plain stores (and, when
// accumulating, loads): rows that a group's end cuts, unaligned outputs.
template <bool TILES>
__device__ __forceinline__ void store_direct(const GemmProblem& p, const uint64_t (&acc)[64], int lane, int64_t base,
                                             int64_t row0, int64_t row_end, int64_t c0) {
    const bool pairs = (p.n & 1) == 0 && (reinterpret_cast<uintptr_t>(p.d) & (p.out_f32 ? 7u : 3u)) == 0;
#pragma unroll
    for (int q = 0; q < 64; ++q) {
        const int64_t r = row0 + row_of<TILES>(q, lane), c = c0 + col_of<TILES>(q, lane);
        if (r >= row_end || c >= p.n) continue;
        const int64_t at = base + r * p.n + c;
        float2 v = unpack2(acc[q]);
        if (p.out_f32) {
            float* d = static_cast<float*>(p.d) + at;
            if (pairs) {
                if (p.accumulate) {
                    const float2 old = *reinterpret_cast<const float2*>(d);
                    v = make_float2(__fadd_rn(old.x, v.x), __fadd_rn(old.y, v.y));
                }
                *reinterpret_cast<float2*>(d) = v;
            } else {
                d[0] = p.accumulate ? __fadd_rn(d[0], v.x) : v.x;
                if (c + 1 < p.n) d[1] = p.accumulate ? __fadd_rn(d[1], v.y) : v.y;
            }
        } else {
            uint16_t* d = static_cast<uint16_t*>(p.d) + at;
            const uint32_t o = f32x2_to_bf16x2(v.x, v.y);
            if (pairs) {
                *reinterpret_cast<uint32_t*>(d) = o;
            } else {
                d[0] = (uint16_t)o;
                if (c + 1 < p.n) d[1] = (uint16_t)(o >> 16);
            }
        }
    }
}

// The same for a warp whose 32 rows are all in the group: staged in shared
// memory 128 bytes of each row at a time (16-byte pieces swizzled, so that the
// stores spread over the banks) and written by the bulk-copy engine, which
// drops what lies outside D.
template <bool TILES>
__device__ __forceinline__ void store_bulk(const GemmProblem& p, const CUtensorMap* map, const uint64_t (&acc)[64],
                                           uint32_t stages, int lane, int64_t row0, int64_t c0, int z) {
#pragma unroll
    for (int part = 0; part < 4; ++part) {
        const uint32_t stage = stages + part % Ring<TILES>::kOuts * kOutBytes;
        if (part >= 2 && !p.out_f32) break;
        const int64_t x = c0 + part * (p.out_f32 ? 32 : 64);
        if (x >= p.n) break;
        if (lane == 0)  // this buffer has been read
            asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(Ring<TILES>::kOuts - 1) : "memory");
        __syncwarp();
        if constexpr (TILES) {
            if (p.out_f32) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {  // 4 column blocks of 8, 4 rows
                    const int q = (part >> 1) * 32 + (i >> 1 & 1) * 16 + ((part & 1) * 4 + (i >> 2)) * 2 + (i & 1);
                    const int r = row_of<true>(q, lane), at = (col_of<true>(q, lane) & 31) * 4;
                    asm volatile("st.shared.b64 [%0], %1;" ::"r"(stage + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15)),
                                 "l"(acc[q])
                                 : "memory");
                }
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {  // 8 column blocks of 8, 4 rows
                    const int q = (part & 1) * 32 + i;
                    const int r = row_of<true>(q, lane), at = (col_of<true>(q, lane) & 63) * 2;
                    const float2 v = unpack2(acc[q]);
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15)),
                                 "r"(f32x2_to_bf16x2(v.x, v.y))
                                 : "memory");
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t o[4];
                if (p.out_f32) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 a = unpack2(acc[part * 16 + 2 * j + i]);
                        o[2 * i] = __float_as_uint(a.x);
                        o[2 * i + 1] = __float_as_uint(a.y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = unpack2(acc[(part & 1) * 32 + 4 * j + i]);
                        o[i] = f32x2_to_bf16x2(a.x, a.y);
                    }
                }
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((j ^ (lane & 7)) << 4)),
                             "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                             : "memory");
            }
        }
        fence_to_async();
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"((int)x), "r"((int)row0), "r"(z), "r"(stage)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
}

// FORM 0: B [n, k], 128 x 128 blocks; 1: B [k, n], 128 x 128 blocks; 2: both
// operands in 1 x 128 tiles, contraction ragged.
template <int FORM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_pair_kernel(const __grid_constant__ GemmProblem p, const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_d, bool bulk_store) {
    constexpr bool RAGGED_K = FORM == 2, B_KN = FORM == 1, B_TILES = FORM == 2;
    constexpr int kStages = Ring<B_TILES>::kStages, kOuts = Ring<B_TILES>::kOuts;
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
        uint32_t it = 0, group = 0;  // blocks and scale groups so far
        for (int t = first; t < total; t += step) {
            const Tile tile = locate<RAGGED_K>(p, groups, count, tiles_n, t);
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
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
            if (!B_TILES && tile.blks > 0) fetch();
            bool ready = false;  // (asking one block ahead pays with 1 x 128 tiles only)
            for (int b = 0; b < tile.blks; ++b) {
                const uint32_t buf = it & 1, from = lanes + buf * kPairN;
                const int sub = b % kScaleBlocks;
                if (B_TILES && sub == 0) fetch();
                if (!B_TILES) {
                    s4 = sub == 0 ? s4_next : make_float4(s4.y, s4.z, s4.w, 0.0f);
                }
                if (!B_TILES || !ready) w.wait(full0 + buf * 8, (it >> 1) & 1);
                __syncwarp();  // lanes may have left the wait apart
                tmem_fence_after();
                ++it;
                const auto read = [&]() {  // the buffer has been read
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) cluster_arrive<false>(empty0 + buf * 8);
                    if (B_TILES) ready = b + 1 < tile.blks && Waiter::test(full0 + (it & 1) * 8, (it >> 1) & 1);
                };
                uint32_t v[32];
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
                            tmem_ld_16x64(from + ((uint32_t)(rh * 16) << 16) + h * 64, v);
                            tmem_wait_ld();
                            if (h + rh == 2) read();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                uint64_t* const at = acc + h * 32 + rh * 16 + i * 2;
                                at[0] = fma2(mul2(pack2(v[4 * i], v[4 * i + 1]), sc[i]), sr[rh * 2], at[0]);
                                at[1] = fma2(mul2(pack2(v[4 * i + 2], v[4 * i + 3]), sc[i]), sr[rh * 2 + 1], at[1]);
                            }
                        }
                    }
                    if (sub == kScaleBlocks - 1 || b == tile.blks - 1) release();
                } else {
                    const uint64_t s2 = pack2(s4.x, s4.x);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld_32x32(from + c * 32, v);
                        tmem_wait_ld();
                        if (c == 3) read();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[c * 16 + j] = fma2(pack2(v[2 * j], v[2 * j + 1]), s2, acc[c * 16 + j]);
                        if (c == 1 && sub == 2 && b + 2 < tile.blks) fetch();
                    }
                }
            }
            // store: this warp's 32 rows, 128 columns
            const int64_t r0 = tile.row0 + (int)rank * 128 + (warp & 3) * 32, c0 = tile.col0 + half * 128;
            if (bulk_store && r0 + 31 < tile.row_end) {
                store_bulk<B_TILES>(p, &map_d, acc, smem_addr(out) + warp * kOuts * kOutBytes, lane, r0, c0, RAGGED_K ? tile.group : 0);
            } else {
                store_direct<B_TILES>(p, acc, lane, RAGGED_K ? (int64_t)tile.group * p.m * p.n : 0, r0, tile.row_end, c0);
            }
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
                    for (int b = 0; b < blks; ++b, ++it) {
                        const uint32_t buf = it & 1, free_bar = smem_addr(&sh.tmem_empty[buf]), free_phase = ((it >> 1) & 1) ^ 1;
                        const uint64_t at = a0 + stage * (kStageBytes >> 4), bt = b0 + stage * (kStageBytes >> 4);
                        const bool is_free = it < 2 || Waiter::test(free_bar, free_phase);
                        // (tiles that were masked with plain stores are released to the cluster)
                        w.template wait<RAGGED_K>(smem_addr(&sh.full[stage]), phase);
                        if (!is_free) w.wait(free_bar, free_phase);
                        __syncwarp();
                        tmem_fence_after();
                        if (elect_one() && !w.dead) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_f8<2>(tmem + buf * kPairN, at + k * kStepKMajor,
                                          bt + k * (B_KN ? kStepMnMajor : kStepKMajor), desc, k > 0);
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
            }
        } else if (warp == 9) {
            // ---- scales: this CTA's 128 rows and the pair's 256 columns (or their two 128-blocks)
            const int64_t kb = blocks_of(p.k), nb = blocks_of(p.n);
            const bool wide_a = kb % kScaleBlocks == 0 && (reinterpret_cast<uintptr_t>(p.sa) & 15u) == 0;
            const bool wide_b = kb % kScaleBlocks == 0 && (reinterpret_cast<uintptr_t>(p.sb) & 15u) == 0;
            uint32_t group = 0;
            for (int t = first; t < total; t += step) {
                const Tile tile = locate<RAGGED_K>(p, groups, count, tiles_n, t);
                for (int done = 0; done < tile.blks; done += kScaleBlocks, ++group) {
                    const int g0 = tile.blk0 + done, to = min(tile.blks - done, kScaleBlocks);
                    const bool whole = g0 % kScaleBlocks == 0;  // an aligned piece of a row of scales
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
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.sc_full[slot]);
                }
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
            for (int t = first; t < total; t += step) {
                const Tile tile = locate<RAGGED_K>(p, groups, count, tiles_n, t);
                for (int b = 0; b < tile.blks; ++b) {
                    const int x = (tile.blk0 + b) * kBlk;
                    if (is_cut(tile, x, (int)p.k)) {
                        w.wait(smem_addr(&sh.landed[stage]), phases >> stage & 1);
                        phases ^= 1u << stage;
                        __syncwarp();
                        mask_tile(base + stage * kStageBytes, tile.k_lo - x, tile.k_hi - x, lane);
                        mask_tile(base + stage * kStageBytes + kTileBytes, tile.k_lo - x, tile.k_hi - x, lane);
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
    fp8_status_t s = FP8_OK;
    if (p.k > 0) s = operand_maps(fn, oa, &a, ob, &b, st);
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
