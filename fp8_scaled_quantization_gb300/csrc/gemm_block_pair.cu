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
// Roles per CTA of 512 threads: warps 0-7 scale and add, then store; warps 8-11
// fill the ring of operand tiles (one thread issuing bulk copies, or all four
// warps with plain loads where sizes or addresses are not multiples of 16, or
// where a ragged group's end cuts a block); warp 12 of the pair's first CTA
// issues the products for both; warps 13 and 14 gather the scales.
#include "fp8q_host.h"
#include "fp8q_tcgen05.cuh"
#include "gemm_block.cuh"

namespace fp8q {
namespace {

constexpr int kThreads = 512;
constexpr int kPairM = 256, kPairN = 256;  // outputs of a pair
constexpr int kStages = 6;                 // operand ring: A and B tile, 32 KB per CTA and stage
constexpr int kScaleSlots = 8;             // scale ring, blocks ahead
constexpr int kRaster = 8;                 // tiles along m that are walked before the next tile along n
constexpr uint32_t kStageBytes = 2 * kTileBytes;

struct Shared {
    float sa[kScaleSlots][128];
    alignas(16) float sb[kScaleSlots][kPairN];  // 128 x 128 blocks use entries 0 and 128
    uint64_t full[kStages], empty[kStages];
    uint64_t tmem_full[2], tmem_empty[2];
    uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
    uint32_t tmem;
    GroupTable groups;
};
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

// Where a tile's operands and outputs lie.
struct Tile {
    int group;
    int64_t row0, row_end;   // of A (and D)
    int64_t col0;
    int64_t k_lo, k_hi;      // contraction range
    int blk0, blks;          // its 128-blocks
};

template <bool RAGGED_K>
__device__ __forceinline__ Tile locate(const GemmProblem& p, const GroupTable& g, int count, int tiles_n, int t) {
    Tile r;
    const int e = find_group(&g, count, t);
    const int local = t - g.tile[e], begin = e > 0 ? g.end[e - 1] : 0, end = g.end[e];
    const int64_t rows = RAGGED_K ? p.m : end - begin;
    const int tiles_m = (int)((rows + kPairM - 1) / kPairM);
    // columns of kRaster tiles along m: what runs at one time shares operands in L2
    const int strip = local / (kRaster * tiles_n), in_strip = local - strip * kRaster * tiles_n;
    const int high = min(kRaster, tiles_m - strip * kRaster);
    r.group = e;
    r.row0 = (RAGGED_K ? 0 : begin) + (int64_t)(strip * kRaster + in_strip % high) * kPairM;
    r.row_end = RAGGED_K ? p.m : end;
    r.col0 = (int64_t)(in_strip / high) * kPairN;
    r.k_lo = RAGGED_K ? begin : 0;
    r.k_hi = RAGGED_K ? end : (e < p.groups ? p.k : 0);
    r.blk0 = (int)(r.k_lo / kBlk);
    r.blks = r.k_hi > r.k_lo ? (int)((r.k_hi + kBlk - 1) / kBlk) - r.blk0 : 0;
    return r;
}

// FORM 0: B [n, k], 128 x 128 blocks; 1: B [k, n], 128 x 128 blocks; 2: both
// operands in 1 x 128 tiles, contraction ragged.  TMA: operand tiles by the
// bulk-copy engine (except blocks that a group end cuts).
template <int FORM, bool TMA>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_pair_kernel(const __grid_constant__ GemmProblem p, const __grid_constant__ CUtensorMap map_a,
                 const __grid_constant__ CUtensorMap map_b) {
    constexpr bool RAGGED_K = FORM == 2, B_KN = FORM == 1, B_TILES = FORM == 2;
    extern __shared__ uint8_t raw[];
    uint8_t* const tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Shared& sh = *reinterpret_cast<Shared*>(tiles + kStages * kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 2);   // one arrival per CTA of the pair
            mbar_init(&sh.empty[i], 1);  // the products' commit
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.tmem_full[i], 1);
            mbar_init(&sh.tmem_empty[i], 16);  // eight warps of each CTA
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.sc_full[i], 64);  // the lanes of two warps
            mbar_init(&sh.sc_empty[i], 8);
        }
        mbar_init_fence();
    }
    if (warp == 12) tmem_alloc<2>(&sh.tmem, 512);
    pdl_begin();
    const int tiles_n = (int)((p.n + kPairN - 1) / kPairN);
    const int count = RAGGED_K ? p.groups : p.groups + 1;
    const int total = build_groups(&sh.groups, p.ends, p.groups, RAGGED_K ? p.k : p.m, kPairM, RAGGED_K ? p.m : 0, tiles_n);
    tmem_fence_before();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    Waiter w;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 128;
        const uint32_t empty0 = cluster_addr(smem_addr(&sh.tmem_empty[0]), 0);
        uint32_t it = 0;
        for (int t = first; t < total; t += step) {
            const Tile tile = locate<RAGGED_K>(p, sh.groups, count, tiles_n, t);
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            for (int b = 0; b < tile.blks; ++b, ++it) {
                const uint32_t slot = it % kScaleSlots, buf = it & 1;
                w.wait(smem_addr(&sh.sc_full[slot]), (it / kScaleSlots) & 1);
                const float sa = sh.sa[slot][row];
                float s = sa;
                if constexpr (!B_TILES) s = __fmul_rn(sa, sh.sb[slot][half * 128]);
                const uint64_t s2 = pack2(s, s);
                w.wait(smem_addr(&sh.tmem_full[buf]), (it >> 1) & 1);
                tmem_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld32(lanes + buf * kPairN + c * 32, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if constexpr (B_TILES) {
                            if (j & 1) continue;
                            uint64_t s0, s1;  // scales of columns 2j .. 2j + 3
                            asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                                         : "=l"(s0), "=l"(s1)
                                         : "r"(smem_addr(&sh.sb[slot][half * 128 + c * 32 + 2 * j])));
                            acc[c * 16 + j] = fma2(mul2(pack2(v[2 * j], v[2 * j + 1]), s0), s2, acc[c * 16 + j]);
                            acc[c * 16 + j + 1] = fma2(mul2(pack2(v[2 * j + 2], v[2 * j + 3]), s1), s2, acc[c * 16 + j + 1]);
                        } else {
                            acc[c * 16 + j] = fma2(pack2(v[2 * j], v[2 * j + 1]), s2, acc[c * 16 + j]);
                        }
                    }
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    cluster_arrive(empty0 + buf * 8);
                    mbar_arrive(&sh.sc_empty[slot]);
                }
            }
            // store: this thread's row, 128 columns
            const int64_t r = tile.row0 + rank * 128 + row, c0 = tile.col0 + half * 128;
            if (r < tile.row_end && c0 < p.n) {
                const int64_t at = (RAGGED_K ? (int64_t)tile.group * p.m * p.n : 0) + r * p.n + c0;
                const int cols = (int)(p.n - c0 < 128 ? p.n - c0 : 128);
                if (p.out_f32) {
                    float* d = static_cast<float*>(p.d) + at;
                    if ((p.n & 3) == 0 && (reinterpret_cast<uintptr_t>(p.d) & 15u) == 0) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (j * 4 >= cols) continue;
                            const float2 a = unpack2(acc[2 * j]), b = unpack2(acc[2 * j + 1]);
                            float4 o = make_float4(a.x, a.y, b.x, b.y);
                            float4* q = reinterpret_cast<float4*>(d) + j;
                            if (p.accumulate) {
                                const float4 old = *q;
                                o = make_float4(__fadd_rn(old.x, o.x), __fadd_rn(old.y, o.y), __fadd_rn(old.z, o.z),
                                                __fadd_rn(old.w, o.w));
                            }
                            *q = o;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 128; ++j) {
                            if (j >= cols) continue;
                            const float2 a = unpack2(acc[j >> 1]);
                            const float o = j & 1 ? a.y : a.x;
                            d[j] = p.accumulate ? __fadd_rn(d[j], o) : o;
                        }
                    }
                } else {
                    uint16_t* d = static_cast<uint16_t*>(p.d) + at;
                    if ((p.n & 7) == 0 && (reinterpret_cast<uintptr_t>(p.d) & 15u) == 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (j * 8 >= cols) continue;
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 a = unpack2(acc[4 * j + i]);
                                o[i] = f32x2_to_bf16x2(a.x, a.y);
                            }
                            reinterpret_cast<uint4*>(d)[j] = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 128; ++j) {
                            if (j >= cols) continue;
                            const float2 a = unpack2(acc[j >> 1]);
                            d[j] = (uint16_t)f32x2_to_bf16x2(j & 1 ? a.y : a.x, 0.0f);
                        }
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp < 12) {
            // ---- operand tiles: A rows [row0 + 128 rank, ..), B columns [col0 + 128 rank, ..)
            const int tid = threadIdx.x - 256;
            const uint32_t base = smem_addr(tiles), full0 = cluster_addr(smem_addr(&sh.full[0]), 0);
            uint32_t it = 0;
            if (!TMA || RAGGED_K || tid == 0) {
                for (int t = first; t < total; t += step) {
                    const Tile tile = locate<RAGGED_K>(p, sh.groups, count, tiles_n, t);
                    const int64_t row = tile.row0 + rank * 128, col = tile.col0 + rank * 128;
                    for (int b = 0; b < tile.blks; ++b, ++it) {
                        const uint32_t stage = it % kStages, a = base + stage * kStageBytes, bt = a + kTileBytes;
                        const int64_t x = (int64_t)(tile.blk0 + b) * kBlk;
                        // a block that a group's end cuts holds other groups' codes too: masked loads
                        const bool cut = RAGGED_K && (x < tile.k_lo || (x + kBlk > tile.k_hi && tile.k_hi < p.k));
                        if (tid == 0 && it >= kStages) w.wait(smem_addr(&sh.empty[stage]), (it / kStages - 1) & 1);
                        if (TMA && !cut) {
                            if (tid != 0) continue;
                            cluster_arrive_expect_tx(full0 + stage * 8, kStageBytes);
                            tma_tile<true>(a, &map_a, (int)x, (int)row, 0, full0 + stage * 8);
                            if constexpr (B_KN) tma_tile<true>(bt, &map_b, (int)col, (int)x, tile.group, full0 + stage * 8);
                            else tma_tile<true>(bt, &map_b, (int)x, (int)col, RAGGED_K ? 0 : tile.group, full0 + stage * 8);
                            continue;
                        }
                        __syncwarp();
                        group_sync(1, 128);  // the stage is free
                        const TileSource as = {p.a, p.a + p.m * p.k, p.k};
                        load_tile(a, as, x, tile.k_lo, tile.k_hi, row, p.m, tid);
                        const int64_t weight = RAGGED_K ? 0 : (int64_t)tile.group * p.n * p.k;
                        const TileSource bs = {p.b + weight, p.b + weight + p.n * p.k, B_KN ? p.n : p.k};
                        if constexpr (B_KN) load_tile(bt, bs, col, 0, p.n, x, p.k, tid);
                        else load_tile(bt, bs, x, tile.k_lo, tile.k_hi, col, p.n, tid);
                        fence_to_async();
                        group_sync(1, 128);  // every warp's part is written
                        if (tid == 0) cluster_arrive(full0 + stage * 8);
                    }
                }
                // the last fills have been read before the CTA ends
                if (tid == 0)
                    for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
                        w.wait(smem_addr(&sh.empty[i % kStages]), (i / kStages) & 1);
            }
        } else if (warp == 12) {
            // ---- products, by one thread of the pair's first CTA
            if (rank == 0 && lane == 0) {
                const uint32_t desc = mma_desc(p.fmt_a, p.fmt_b, false, B_KN, kPairM, kPairN);
                const uint64_t a0 = tile_desc(smem_addr(tiles)), b0 = tile_desc(smem_addr(tiles) + kTileBytes);
                uint32_t it = 0;
                for (int t = first; t < total; t += step) {
                    const int blks = locate<RAGGED_K>(p, sh.groups, count, tiles_n, t).blks;
                    for (int b = 0; b < blks; ++b, ++it) {
                        const uint32_t stage = it % kStages, buf = it & 1;
                        if (it >= 2) w.wait(smem_addr(&sh.tmem_empty[buf]), ((it >> 1) - 1) & 1);
                        w.wait(smem_addr(&sh.full[stage]), (it / kStages) & 1);
                        tmem_fence_after();
                        const uint64_t at = a0 + stage * (kStageBytes >> 4), bt = b0 + stage * (kStageBytes >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8<2>(tmem + buf * kPairN, at + k * kStepKMajor, bt + k * (B_KN ? kStepMnMajor : kStepKMajor),
                                      desc, k > 0);
                        mma_commit<2>(smem_addr(&sh.empty[stage]));
                        mma_commit<2>(smem_addr(&sh.tmem_full[buf]));
                    }
                }
            }
        } else if (warp == 13) {
            // ---- row scales: this CTA's 128 rows
            const int64_t kb = blocks_of(p.k);
            uint32_t it = 0;
            for (int t = first; t < total; t += step) {
                const Tile tile = locate<RAGGED_K>(p, sh.groups, count, tiles_n, t);
                const float* sa[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t r = tile.row0 + rank * 128 + i * 32 + lane;
                    sa[i] = p.sa + (r < p.m ? r : p.m - 1) * kb + tile.blk0;  // a row that is not there: any scale
                }
                for (int b = 0; b < tile.blks; ++b, ++it) {
                    const uint32_t slot = it % kScaleSlots;
                    if (it >= kScaleSlots) w.wait(smem_addr(&sh.sc_empty[slot]), (it / kScaleSlots - 1) & 1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) copy4_async(smem_addr(&sh.sa[slot][i * 32 + lane]), sa[i] + b);
                    copies_arrive(smem_addr(&sh.sc_full[slot]));
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == 14) {
            // ---- column scales: the pair's 256 columns, or their two 128-blocks
            const int64_t kb = blocks_of(p.k), nb = blocks_of(p.n);
            uint32_t it = 0;
            for (int t = first; t < total; t += step) {
                const Tile tile = locate<RAGGED_K>(p, sh.groups, count, tiles_n, t);
                const float* sb[B_TILES ? 8 : 1];
                if constexpr (B_TILES) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t c = tile.col0 + i * 32 + lane;
                        sb[i] = p.sb + (c < p.n ? c : p.n - 1) * kb + tile.blk0;
                    }
                } else {
                    const int64_t c = tile.col0 / kBlk + (lane & 1), cb = c < nb ? c : nb - 1;
                    sb[0] = p.sb + (int64_t)tile.group * kb * nb + (B_KN ? cb : cb * kb);
                }
                const int64_t next_b = B_KN ? nb : 1;
                for (int b = 0; b < tile.blks; ++b, ++it) {
                    const uint32_t slot = it % kScaleSlots;
                    if (it >= kScaleSlots) w.wait(smem_addr(&sh.sc_empty[slot]), (it / kScaleSlots - 1) & 1);
                    if constexpr (B_TILES) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) copy4_async(smem_addr(&sh.sb[slot][i * 32 + lane]), sb[i] + b);
                    } else if (lane < 2) {
                        copy4_async(smem_addr(&sh.sb[slot][lane * 128]), sb[0] + b * next_b);
                    }
                    copies_arrive(smem_addr(&sh.sc_full[slot]));
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        __syncwarp();
    }
    tmem_fence_before();
    cluster_sync();
    tmem_fence_after();
    if (warp == 12) tmem_free<2>(tmem, 512);
}

template <int FORM, bool TMA>
fp8_status_t launch_pair(const char* fn, const GemmProblem& p, const CUtensorMap& a, const CUtensorMap& b, int pairs,
                         cudaStream_t st) {
    return launch_smem(fn, gemm_pair_kernel<FORM, TMA>, dim3(2 * pairs), dim3(kThreads), kSmemBytes, st, p, a, b);
}

}  // namespace

fp8_status_t run_gemm_pair(const char* fn, const GemmProblem& p, cudaStream_t st) {
    const int form = p.b_tiles ? 2 : p.b_kn ? 1 : 0;
    const int64_t inner_b = p.b_kn ? p.n : p.k, rows_b = p.b_kn ? p.k : p.n;
    // the bulk copies need 16-byte aligned bases and row strides
    const bool tma = aligned16(p.a) && aligned16(p.b) && p.k % 16 == 0 && inner_b % 16 == 0;
    CUtensorMap a = {}, b = {};
    if (tma) {
        fp8_status_t s = encode_tile_map_u8(&a, p.a, p.k, p.m, 1);
        if (s == FP8_OK) s = encode_tile_map_u8(&b, p.b, inner_b, rows_b, p.b_tiles ? 1 : p.groups);
        if (s != FP8_OK) return s;
    }
    const int64_t tiles_n = (p.n + kPairN - 1) / kPairN, tiles_m = (p.m + kPairM - 1) / kPairM;
    const int64_t most = p.b_tiles ? tiles_m * tiles_n * p.groups : (tiles_m + p.groups - 1) * tiles_n;
    const int sms = sm_count() / 2, pairs = (int)(most < sms ? most : sms);
    if (form == 0) return tma ? launch_pair<0, true>(fn, p, a, b, pairs, st) : launch_pair<0, false>(fn, p, a, b, pairs, st);
    if (form == 1) return tma ? launch_pair<1, true>(fn, p, a, b, pairs, st) : launch_pair<1, false>(fn, p, a, b, pairs, st);
    return tma ? launch_pair<2, true>(fn, p, a, b, pairs, st) : launch_pair<2, false>(fn, p, a, b, pairs, st);
}

fp8_status_t gemm_pair_wait_timeouts(unsigned long long* count) {
    return cuda_status(cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof *count), "fp8_wait_timeouts");
}

}  // namespace fp8q
