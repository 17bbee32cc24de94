// gemm_block_stream.cu -- block-scaled FP8 products with few rows of A (tokens):
// each CTA streams 128 rows of the weight past one tile of tokens.
//
// With few tokens the product is a read of the weight, so the roles of the
// operands are exchanged: the weight's 128 rows (columns of D) fill the tensor
// core's M = 128, the tokens its N = 16 .. 128, and a lane of the scaling warps
// holds one column of D.  The contraction is split over the CTAs of a cluster
// until there are enough of them to draw the memory's full rate; they add their
// partial sums through distributed shared memory, in the order of their ranks,
// so that results do not depend on timing and no workspace is needed.
//
// The gated form gives the gate's weight to the even CTAs of a cluster and the up
// projection's to the odd ones, each half of them sharing the contraction; both
// sums of a token meet where they are joined.  A CTA that streamed both, one after the
// other, needs twice the sums, and 64 tokens no longer fit an SM twice: 15% longer for 48
// x 14336 x 4096 (tokens, n, k), 5% for 16 x 7168 x 7168.  As the plain product with
// twice the columns takes, so does the gated one: 1 x 18432 x 7168 44 us (6.0 TB/s), 16 x
// 7168 x 7168 22, 48 x 14336 x 4096 30, 96 rows over 64 experts of 2048 x 7168 274 (6.9 TB/s).
//
// Roles per CTA: four warps (eight from 32 tokens on, each pair of them sharing
// the tokens of 32 columns) scale, add, join and store; then one warp fills the
// ring of operand tiles and gathers the scales, and one issues the products.
#include <atomic>

#include "fp8q_host.h"
#include "fp8q_tcgen05.cuh"
#include "gated.cuh"
#include "gemm_block.cuh"

namespace fp8q {
namespace {

constexpr int kRows = 128;        // rows of the weight per CTA
constexpr int kScaleBlocks = 4;   // blocks of an item whose scales are gathered together
constexpr int kScaleSlots = 3;
constexpr int kMostSplit = 8;     // CTAs of a cluster

// FORM 0: B [n, k], 128 x 128 blocks; 1: B [k, n], 128 x 128 blocks; 2: B [n,
// k], 1 x 128 tiles; 3: gated, two B [n, k] per group, 128 x 128 blocks.
constexpr int kTiles = 2, kGated = 3;

// Per number of tokens: ring depth and CTAs per SM.  Two CTAs per SM where their
// tiles fit, so that one's start and end overlap the other's stream.
template <int TOKENS, bool TILES>
struct Shape {
    static constexpr int kCtas = TOKENS <= 32 || (TOKENS == 64 && !TILES) ? 2 : 1;
    static constexpr int kStages = TOKENS == 16 ? 5 - TILES : TOKENS == 32 ? 4 - TILES : TOKENS == 64 && !TILES ? 3 : 4;
    static constexpr int kBufs = 4;                           // TMEM buffers (128 tokens with two: 2% slower)
    static constexpr uint32_t kColumns = TOKENS * kBufs;      // a power of two, 64 .. 512
    static constexpr uint32_t kStageBytes = kTileBytes + TOKENS * 128;
    static constexpr int kScalers = TOKENS == 16 ? 4 : 8;     // warps
    static constexpr int kMine = TOKENS * 4 / kScalers;       // tokens per scaling warp: 16, 16, 32, 64
    static constexpr int kThreads = (kScalers + 2) * 32;      // 10 warps leave 96 registers with two CTAs per SM
};

template <int TOKENS, int FORM>
struct Shared {
    static constexpr bool TILES = FORM == kTiles;
    using S = Shape<TOKENS, TILES>;
    alignas(16) float part[TOKENS][kRows];                           // this CTA's partial sums
    alignas(16) float token[kScaleSlots][kScaleBlocks][TOKENS];      // per block: token scale (x block scale)
    alignas(16) float weight[TILES ? kScaleSlots : 1][kScaleBlocks][TILES ? kRows : 1];  // 1 x 128 tiles: the weight rows' scales
    // gated: the largest |h|, |g| and |u| (bits) of each token that this CTA joins, in each warp's 32 columns
    alignas(16) uint32_t most[FORM == kGated ? 3 : 1][FORM == kGated ? TOKENS / 2 : 1][4];
    uint64_t full[S::kStages], empty[S::kStages];
    uint64_t tmem_full[S::kBufs], tmem_empty[S::kBufs];
    uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
    uint64_t part_full, part_empty;
    uint32_t tmem, dead;
    int groups[1];  // the group table: as long as the launch asks for
};

template <int TOKENS, int FORM>
constexpr size_t smem_bytes(int groups) {
    using S = Shape<TOKENS, FORM == kTiles>;
    constexpr size_t bytes = 1024 + (size_t)S::kStages * S::kStageBytes + sizeof(Shared<TOKENS, FORM>);
    static_assert(S::kCtas * (bytes + group_table_bytes(256) + 1024) <= 228 * 1024, "shared memory of an SM");
    static_assert(bytes + group_table_bytes(kMaxGroups) <= 227 * 1024, "shared memory of a CTA");
    return bytes + group_table_bytes(groups);
}

// One item: a tile of tokens, 128 rows of the weight, this CTA's share of the blocks.
struct Item {
    int group;
    int row0, row_end;  // tokens
    int col0;           // rows of the weight
    int blk0, blks;
};

template <int TOKENS>
__device__ __forceinline__ Item locate(const GemmProblem& p, const GroupTable& g, int tiles_n, int t, int share, int shares) {
    Item r;
    const int e = find_group(g, p.groups + 1, t);
    const int local = t - g.tile[e], begin = e > 0 ? g.end[e - 1] : 0, end = g.end[e];
    const int tiles_m = (end - begin + TOKENS - 1) / TOKENS;
    // tiles of tokens first: neighbours read the same rows of the weight
    r.group = e;
    r.row0 = begin + local % tiles_m * TOKENS;
    r.row_end = end;
    r.col0 = local / tiles_m * kRows;
    const int blks = e < p.groups ? (int)blocks_of(p.k) : 0;
    r.blk0 = (int)((int64_t)blks * share / shares);
    r.blks = (int)((int64_t)blks * (share + 1) / shares) - r.blk0;
    return r;
}

// acc += s_j * P_j over the warp's tokens, scales s at `token` (shared memory); with
// 1 x 128 tiles acc += s_j * (P_j * w), w the lane's own weight-row scale (w2: a pair of
// it).  That order is the pair kernel's: which one runs must not show in the result.
// TMEM is read one piece ahead of the arithmetic; the sums are single numbers, as
// packed pairs leave the compiler fewer registers (256 x 7168 x 7168 with 64
// tokens: 34.6 us, packed 35.5, without reading ahead 38.6).
template <int MINE, bool B_TILES>
__device__ __forceinline__ void scale_add(float (&acc)[MINE], uint32_t from, const float* token, uint64_t w2) {
    constexpr int kPieces = MINE / 16;
    uint32_t v[2][16];
    tmem_ld_32x16(from, v[0]);
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {  // reads run one piece ahead
        tmem_wait_ld();
        if (c + 1 < kPieces) tmem_ld_32x16(from + (c + 1) * 16, v[(c + 1) & 1]);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 s = *reinterpret_cast<const float4*>(token + c * 16 + j);
            float* const at = acc + c * 16 + j;
            uint32_t* const x = v[c & 1] + j;
            if constexpr (B_TILES) {
                const float2 x0 = unpack2(mul2(pack2(x[0], x[1]), w2)), x1 = unpack2(mul2(pack2(x[2], x[3]), w2));
                x[0] = __float_as_uint(x0.x), x[1] = __float_as_uint(x0.y);
                x[2] = __float_as_uint(x1.x), x[3] = __float_as_uint(x1.y);
            }
            at[0] = __fmaf_rn(__uint_as_float(x[0]), s.x, at[0]);
            at[1] = __fmaf_rn(__uint_as_float(x[1]), s.y, at[1]);
            at[2] = __fmaf_rn(__uint_as_float(x[2]), s.z, at[2]);
            at[3] = __fmaf_rn(__uint_as_float(x[3]), s.w, at[3]);
        }
    }
}

__device__ __forceinline__ void store_out(const GemmProblem& p, int64_t at, float v) {
    if (p.out_f32) {
        float* d = static_cast<float*>(p.d) + at;
        *d = p.accumulate ? __fadd_rn(*d, v) : v;
    } else {
        static_cast<uint16_t*>(p.d)[at] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
    }
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Both sums of token j and this lane's column over the cluster: the gate's in even ranks,
// the up projection's in odd ones, added in their order.
template <int TOKENS>
__device__ __forceinline__ float2 join_gated(const Shared<TOKENS, kGated>& sh, int j, int row, int split) {
    float x[kMostSplit];
#pragma unroll
    for (int r = 0; r < kMostSplit; ++r) x[r] = r < split ? ld_cluster(cluster_addr(smem_addr(&sh.part[j][row]), r)) : 0.0f;
    float2 v = make_float2(x[0], x[1]);
#pragma unroll
    for (int r = 2; r < kMostSplit; r += 2)
        if (r < split) v.x = __fadd_rn(v.x, x[r]), v.y = __fadd_rn(v.y, x[r + 1]);
    return v;
}

// The end of a gated item, of the tokens j0 .. j1 - 1 that this CTA joins: h of this lane's
// column, quantized in tiles of the CTA's 128 columns, by four warps, of which the CTA has
// one set or two that take the tokens in turn.  One pass for the maxima and one for the
// codes; in between a lane per token derives the scales.  (Four tokens at a time through
// both, a scale in every lane: 10% longer for 48 x 14336 x 4096.)
template <int ACT, int TOKENS>
__device__ __forceinline__ void finish_gated(const GemmProblem& p, Shared<TOKENS, kGated>& sh, const Item& item, int warp, int lane,
                                             int j0, int j1, int split) {
    constexpr int kSets = Shape<TOKENS, false>::kScalers / 4;
    static_assert(TOKENS / 2 / kSets <= 32, "a lane per token");
    const GatedOut& out = p.gated;
    const int quarter = warp & 3, row = quarter * 32 + lane, first = j0 + (warp >> 2);
    const int64_t col = item.col0 + row, nb = blocks_of(p.n);
    const bool keep = out.gu != nullptr, mine = col < p.n;
#pragma unroll 4
    for (int j = first; j < j1; j += kSets) {
        // A lane without a column reads nothing: what it read it would not wait for, and the
        // CTA that holds it may leave once this one's warps have met it.
        const float2 v = mine ? join_gated<TOKENS>(sh, j, row, split) : make_float2(0.0f, 0.0f);
        const float h = gated<ACT>(v.x, v.y);
        const uint32_t mh = warp_max_u32(abs_bits(h));
        if (lane == 0) sh.most[0][j - j0][quarter] = mh;
        if (keep) {
            const uint32_t mg = warp_max_u32(abs_bits(v.x)), mu = warp_max_u32(abs_bits(v.y));
            if (lane == 0) sh.most[1][j - j0][quarter] = mg, sh.most[2][j - j0][quarter] = mu;
        } else {
            sh.part[j][row] = h;  // in the place of this CTA's sum, which no other one reads
        }
    }
    group_sync(1 + (warp >> 2), 128);  // (the next item's maxima come after all warps have met over its sums)
    float scale[3] = {1.0f, 1.0f, 1.0f};  // of h, g and u of token first + lane * kSets
    const int own = first + lane * kSets;
    if (own < j1) {
        const int64_t token = item.row0 + own, block = item.col0 / kBlk;
#pragma unroll
        for (int kind = 0; kind < 3; ++kind) {
            if (kind > 0 && !keep) break;
            const uint4 m = *reinterpret_cast<const uint4*>(sh.most[kind][own - j0]);
            float factor;
            scale_from_amax<kE4M3>(__uint_as_float(umax(umax(m.x, m.y), umax(m.z, m.w))), 0, &scale[kind], &factor);
            if (quarter == 0) {
                if (kind == 0) out.sh[token * nb + block] = factor;
                else out.sgu[(2 * token + kind - 1) * nb + block] = factor;
            }
        }
    }
#pragma unroll 4
    for (int j = first; j < j1; j += kSets) {
        const int64_t token = item.row0 + j;
        const auto write = [&](float v, float s, uint8_t* at) {
            const uint8_t code = (uint8_t)cvt2<kE4M3>(__fmul_rn(v, s), 0.0f);
            if (mine) *at = code;
        };
        const int i = (j - first) / kSets;
        const float s = __shfl_sync(0xFFFFFFFFu, scale[0], i);
        if (!keep) {
            write(sh.part[j][row], s, out.h + token * p.n + col);
        } else {
            const float2 v = mine ? join_gated<TOKENS>(sh, j, row, split) : make_float2(0.0f, 0.0f);
            write(gated<ACT>(v.x, v.y), s, out.h + token * p.n + col);
            write(v.x, __shfl_sync(0xFFFFFFFFu, scale[1], i), out.gu + 2 * token * p.n + col);
            write(v.y, __shfl_sync(0xFFFFFFFFu, scale[2], i), out.gu + (2 * token + 1) * p.n + col);
        }
    }
}

// The cluster's size is the number of shares (gated: of both projections).
template <int FORM, int TOKENS>
__global__ void __launch_bounds__(Shape<TOKENS, FORM == kTiles>::kThreads, Shape<TOKENS, FORM == kTiles>::kCtas)
gemm_stream_kernel(const __grid_constant__ GemmProblem p, const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_b, int split) {
    constexpr bool B_KN = FORM == 1, B_TILES = FORM == kTiles, GATED = FORM == kGated;
    using S = Shape<TOKENS, B_TILES>;
    extern __shared__ uint8_t raw[];
    uint8_t* const tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Shared<TOKENS, FORM>& sh = *reinterpret_cast<Shared<TOKENS, FORM>*>(tiles + S::kStages * S::kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    // this CTA's share of the contraction, of how many, and (gated) its projection
    const int share = GATED ? rank >> 1 : rank, shares = GATED ? split >> 1 : split, half = GATED ? rank & 1 : 0;

    if (threadIdx.x == 0) {
        sh.dead = 0;
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&sh.tmem_full[i], 1);
            mbar_init(&sh.tmem_empty[i], S::kScalers);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh.sc_full[i], 1);
            mbar_init(&sh.sc_empty[i], S::kScalers);
        }
        mbar_init(&sh.part_full, S::kScalers * split);   // the scaling warps of every CTA
        mbar_init(&sh.part_empty, S::kScalers * split);
        mbar_init_fence();
    }
    constexpr int kLoad = S::kScalers, kProduct = kLoad + 1;  // warps
    if (threadIdx.x == kLoad * 32) {
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    if (warp == kProduct) {
        tmem_alloc<1>(&sh.tmem, S::kColumns);
        tmem_fence_before();
    }
    pdl_begin();
    const int tiles_n = (int)((p.n + kRows - 1) / kRows);
    const GroupTable groups(sh.groups, p.groups);
    const int total = build_groups(groups, p.ends, p.groups, p.m, TOKENS, 0, tiles_n);  // synchronises the CTA
    // Every CTA's barriers are ready before another one arrives on them; the tile
    // and scale warps, which do not, go ahead without waiting for that.
    if (split > 1) {
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        if (warp < S::kScalers) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    const int first = blockIdx.x / split, step = gridDim.x / split;
    Waiter w;

    if (warp < S::kScalers) {
        constexpr int kMine = S::kMine;
        const int row = (warp & 3) * 32 + lane, token0 = (warp >> 2) * kMine;  // this lane's column of D, this warp's first token
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + token0;
        uint32_t it = 0, group = 0, items = 0;
        for (int t = first; t < total; t += step, ++items) {
            const Item item = locate<TOKENS>(p, groups, tiles_n, t, share, shares);
            float acc[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) acc[i] = 0.0f;
            for (int b0 = 0; b0 < item.blks; b0 += kScaleBlocks, ++group) {
                const uint32_t slot = group % kScaleSlots;
                w.wait(smem_addr(&sh.sc_full[slot]), (group / kScaleSlots) & 1);
#pragma unroll 1
                for (int sub = 0; sub < min(item.blks - b0, kScaleBlocks); ++sub, ++it) {
                    const uint32_t buf = it % S::kBufs;
                    w.wait(smem_addr(&sh.tmem_full[buf]), (it / S::kBufs) & 1);
                    __syncwarp();  // lanes may have left the wait apart
                    tmem_fence_after();
                    uint64_t w2 = 0;
                    if constexpr (B_TILES) {
                        const float f = sh.weight[slot][sub][row];
                        w2 = pack2(f, f);
                    }
                    scale_add<kMine, B_TILES>(acc, lanes + buf * TOKENS, &sh.token[slot][sub][token0], w2);
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.tmem_empty[buf]);
                }
                if (lane == 0) mbar_arrive(&sh.sc_empty[slot]);
            }
            // The partial sums go to shared memory.  Without shares of the contraction every
            // lane takes its own back; else each CTA adds its part of the tokens over all
            // CTAs, the first warp of a column quarter the even ones, the second the odd.
            const int64_t col = item.col0 + row;
            const int tokens = min(TOKENS, item.row_end - item.row0);
            if (split > 1 && items > 0) {
                w.template wait<true>(smem_addr(&sh.part_empty), (items - 1) & 1);
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
                if (token0 + j < tokens) sh.part[token0 + j][row] = acc[j];
            }
            if (!GATED && split == 1) {
                if (col < p.n) {
#pragma unroll 4
                    for (int j = token0; j < min(token0 + kMine, tokens); ++j)
                        store_out(p, (int64_t)(item.row0 + j) * p.n + col, sh.part[j][row]);
                }
                continue;
            }
            __syncwarp();
            if (lane < split) cluster_arrive<true>(cluster_addr(smem_addr(&sh.part_full), lane));
            w.template wait<true>(smem_addr(&sh.part_full), items & 1);
            __syncwarp();
            const int first_token = tokens * rank / split, last_token = tokens * (rank + 1) / split;
            if constexpr (GATED) {
                if (p.gated.act == kSilu) finish_gated<kSilu, TOKENS>(p, sh, item, warp, lane, first_token, last_token, split);
                else finish_gated<kGeluTanh, TOKENS>(p, sh, item, warp, lane, first_token, last_token, split);
            } else {
                // A lane without a column reads nothing: what it read it would not wait for, and the
                // CTA that holds it may leave once this one's warps have met it.
                const int j0 = first_token, j1 = col < p.n ? last_token : j0;
                for (int j = j0 + (warp >> 2); j < j1; j += S::kScalers / 4) {
                    float v[kMostSplit];
#pragma unroll
                    for (int r = 0; r < kMostSplit; ++r)
                        v[r] = r < split ? ld_cluster(cluster_addr(smem_addr(&sh.part[j][row]), r)) : 0.0f;
                    float sum = v[0];
#pragma unroll
                    for (int r = 1; r < kMostSplit; ++r)
                        if (r < split) sum = __fadd_rn(sum, v[r]);
                    store_out(p, (int64_t)(item.row0 + j) * p.n + col, sum);
                }
            }
            __syncwarp();
            // (nothing overwrites the last item's sums)
            if (lane < split && t + step < total) cluster_arrive<true>(cluster_addr(smem_addr(&sh.part_empty), lane));
        }
    } else if (warp == kLoad) {
        // ---- operand tiles, and scales: those of the next group of blocks are loaded into
        // registers while the copies of this group's tiles are issued
        const int64_t kb = blocks_of(p.k), nb = blocks_of(p.n);
        const bool wide_a = kb % kScaleBlocks == 0 && (reinterpret_cast<uintptr_t>(p.sa) & 15u) == 0;
        const bool wide_b = kb % kScaleBlocks == 0 && (reinterpret_cast<uintptr_t>(p.sb) & 15u) == 0;
        constexpr int kTokens = (TOKENS + 31) / 32, kWeights = B_TILES ? 4 : 1;
        float4 ts[kTokens], ws[kWeights];  // this lane's tokens; its weight rows, or the weight's blocks
        const auto load_group = [&](const Item& item, int done) {
            const int g0 = item.blk0 + done, to = min(item.blks - done, kScaleBlocks);
            const bool whole = g0 % kScaleBlocks == 0;  // an aligned piece of a row of scales
            if constexpr (B_TILES) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // a token or row that is not there: any scale
                    const int64_t n = item.col0 + i * 32 + lane;
                    ws[i] = load_scales(p.sb + (n < p.n ? n : p.n - 1) * kb + g0, to, wide_b && whole);
                }
            } else {
                const int64_t cb = item.col0 / kBlk;
                const float* const sb = p.sb + (GATED ? 2 * (int64_t)item.group + half : (int64_t)item.group) * kb * nb;
                if constexpr (B_KN) {
                    const float* const at = sb + (int64_t)g0 * nb + cb;
                    ws[0] = make_float4(__ldg(at), to > 1 ? __ldg(at + nb) : 0.0f, to > 2 ? __ldg(at + 2 * nb) : 0.0f,
                                        to > 3 ? __ldg(at + 3 * nb) : 0.0f);
                } else {
                    ws[0] = load_scales(sb + cb * kb + g0, to, wide_b && whole);
                }
            }
#pragma unroll
            for (int i = 0; i < kTokens; ++i) {
                const int64_t r = item.row0 + min(i * 32 + lane, TOKENS - 1);
                ts[i] = load_scales(p.sa + (r < p.m ? r : p.m - 1) * kb + g0, to, wide_a && whole);
            }
        };
        uint32_t group = 0;
        const auto publish = [&]() {
            const uint32_t slot = group % kScaleSlots;
            if (group >= kScaleSlots) w.wait(smem_addr(&sh.sc_empty[slot]), (group / kScaleSlots - 1) & 1);
            __syncwarp();
            const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f), c = B_TILES ? one : ws[0];
#pragma unroll
            for (int i = 0; i < kTokens; ++i) {
                const int j = i * 32 + lane;
                if (TOKENS % 32 == 0 || j < TOKENS) {
                    sh.token[slot][0][j] = __fmul_rn(ts[i].x, c.x);
                    sh.token[slot][1][j] = __fmul_rn(ts[i].y, c.y);
                    sh.token[slot][2][j] = __fmul_rn(ts[i].z, c.z);
                    sh.token[slot][3][j] = __fmul_rn(ts[i].w, c.w);
                }
            }
            if constexpr (B_TILES) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sh.weight[slot][0][i * 32 + lane] = ws[i].x;
                    sh.weight[slot][1][i * 32 + lane] = ws[i].y;
                    sh.weight[slot][2][i * 32 + lane] = ws[i].z;
                    sh.weight[slot][3][i * 32 + lane] = ws[i].w;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.sc_full[slot]);
            ++group;
        };
        const uint32_t base = smem_addr(tiles);
        uint32_t it = 0, stage = 0, phase = 0;
        bool loaded = false;  // the next group's scales are in registers
        for (int t = first; t < total; t += step) {
            const Item item = locate<TOKENS>(p, groups, tiles_n, t, share, shares);
            if (!loaded && item.blks > 0) load_group(item, 0);
            for (int b = 0; b < item.blks; ++b, ++it) {
                const uint32_t wt = base + stage * S::kStageBytes, xt = wt + kTileBytes, bar = smem_addr(&sh.full[stage]);
                const int x = (item.blk0 + b) * kBlk;
                if (it >= S::kStages) w.wait(smem_addr(&sh.empty[stage]), phase ^ 1);
                __syncwarp();
                if (elect_one() && !w.dead) {
                    mbar_arrive_expect_tx(&sh.full[stage], S::kStageBytes);
                    const int matrix = B_TILES ? 0 : GATED ? 2 * item.group + half : item.group;
                    if constexpr (B_KN) tma_tile<false>(wt, &map_b, item.col0, x, matrix, bar);
                    else tma_tile<false>(wt, &map_b, x, item.col0, matrix, bar);
                    tma_tile<false>(xt, &map_a, x, item.row0, 0, bar);
                }
                __syncwarp();
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                // The products of this group's first blocks wait for sums of earlier groups
                // only, so its scales may follow the copies of its second block (or the last).
                if (b % kScaleBlocks == 1 || (b % kScaleBlocks == 0 && b == item.blks - 1)) {
                    publish();
                    const int next = (b / kScaleBlocks + 1) * kScaleBlocks;
                    if (next < item.blks) {
                        load_group(item, next);
                    } else if (t + step < total) {
                        const Item after = locate<TOKENS>(p, groups, tiles_n, t + step, share, shares);
                        loaded = after.blks > 0;
                        if (loaded) load_group(after, 0);
                    }
                }
            }
        }
        // the last fills have been read before the CTA ends
        for (uint32_t i = it > S::kStages ? it - S::kStages : 0; i < it; ++i)
            w.wait(smem_addr(&sh.empty[i % S::kStages]), (i / S::kStages) & 1);
    } else {
        // ---- products: weight rows are M, tokens N
        const uint32_t desc = mma_desc(p.fmt_b, p.fmt_a, B_KN, false, kRows, TOKENS);
        const uint64_t w0 = tile_desc(smem_addr(tiles)), x0 = tile_desc(smem_addr(tiles) + kTileBytes);
        uint32_t it = 0, stage = 0, phase = 0;
        bool ready = false;  // the next block's tiles and buffer, asked for while this block's products are issued
        for (int t = first; t < total; t += step) {
            const int blks = locate<TOKENS>(p, groups, tiles_n, t, share, shares).blks;
            for (int b = 0; b < blks; ++b, ++it) {
                const uint32_t buf = it % S::kBufs;
                if (!ready) {
                    if (it >= S::kBufs) w.wait(smem_addr(&sh.tmem_empty[buf]), (it / S::kBufs - 1) & 1);
                    w.wait(smem_addr(&sh.full[stage]), phase);
                }
                __syncwarp();
                const uint64_t wt = w0 + stage * (S::kStageBytes >> 4), xt = x0 + stage * (S::kStageBytes >> 4);
                const uint32_t now = stage;
                if (++stage == S::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                const uint32_t next = it + 1;
                const bool free = next < S::kBufs || Waiter::test(smem_addr(&sh.tmem_empty[next % S::kBufs]), (next / S::kBufs - 1) & 1);
                const bool filled = Waiter::test(smem_addr(&sh.full[stage]), phase);
                tmem_fence_after();
                if (elect_one() && !w.dead) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8<1>(tmem + buf * TOKENS, wt + k * (B_KN ? kStepMnMajor : kStepKMajor), xt + k * kStepKMajor, desc,
                                  k > 0);
                    mma_commit<1>(smem_addr(&sh.tmem_full[buf]));
                    mma_commit<1>(smem_addr(&sh.empty[now]));
                }
                ready = __all_sync(0xFFFFFFFFu, free && filled);
            }
        }
    }
    __syncwarp();
    if (w.dead) report_dead(smem_addr(&sh.dead), split);
    tmem_fence_before();
    if (split > 1) {  // no CTA leaves while another reads its partial sums
        if (warp >= S::kScalers) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        cluster_meet();
    } else {
        __syncthreads();
    }
    if (sh.dead != 0) {
        linger();
        if (split > 1) cluster_meet();
        else __syncthreads();
    }
    tmem_fence_after();
    if (warp == kProduct) tmem_free<1>(tmem, S::kColumns);
}

// How many clusters of `split` CTAs run at one time, one CTA per SM: a cluster
// lies within one group of SMs, so that these are fewer than the SMs divided (of
// 152: 23 clusters of 6, 15 of 8).  A grid beyond them runs in two turns: 96 x 2048
// x 7168 in 48 clusters of 6 on two CTAs per SM takes 17 us, in 32 of 3 11.
// Asked once, of the kernel of which one CTA fits an SM (of one that allocates
// TMEM the runtime counts no second CTA, although it runs).
int clusters_per_turn(int split, int sms) {
    static std::atomic<int> known[kMostSplit + 1];
    int n = known[split].load(std::memory_order_relaxed);
    if (n > 0) return n;
    using S = Shape<128, false>;
    const int most = sms / split;
    n = max_clusters(reinterpret_cast<const void*>(gemm_stream_kernel<0, 128>), S::kThreads, smem_bytes<128, 0>(1), split);
    n = n <= 0 || n > most ? most : n;
    known[split].store(n, std::memory_order_relaxed);
    return n;
}

template <int TOKENS>
StreamPlan plan(const GemmProblem& p, int sms) {
    const int ctas = p.b_tiles ? Shape<TOKENS, true>::kCtas : Shape<TOKENS, false>::kCtas;  // per SM
    const int64_t tiles_n = (p.n + kRows - 1) / kRows, tiles_m = (p.m + TOKENS - 1) / TOKENS, kb = blocks_of(p.k);
    const int64_t busy = p.groups < p.m ? p.groups : p.m;  // groups with rows, at most
    StreamPlan r = {(tiles_m + busy - 1) * tiles_n, 1, ctas * sms};
    // shares of the contraction: as many as run at one time, each at least two blocks
    // long; gated: CTAs for both projections of each
    const int each = p.gated.h != nullptr ? 2 : 1;
    if (each == 2) r = {r.items, 2, ctas * clusters_per_turn(2, sms)};
    for (int split = each * 2; split <= kMostSplit && kb >= 2 * (split / each); split += each) {
        const int clusters = ctas * clusters_per_turn(split, sms);
        if (r.items <= clusters) r = {r.items, split, clusters};
    }
    return r;
}

template <int TOKENS>
fp8_status_t run(const char* fn, const GemmProblem& p, const CUtensorMap& a, const CUtensorMap& b, cudaStream_t st) {
    const StreamPlan how = plan<TOKENS>(p, sm_count());
    const int64_t clusters = how.items + 1 < how.clusters ? how.items + 1 : how.clusters;
    const auto go = [&](auto kernel, size_t smem) {
        return launch_cluster(fn, kernel, dim3((unsigned)(clusters * how.split)), dim3(Shape<TOKENS, false>::kThreads), smem,
                              how.split, st, p, a, b, how.split);
    };
    if constexpr (TOKENS <= 64)
        if (p.gated.h != nullptr) return go(gemm_stream_kernel<kGated, TOKENS>, smem_bytes<TOKENS, kGated>(p.groups));
    return p.b_tiles ? go(gemm_stream_kernel<kTiles, TOKENS>, smem_bytes<TOKENS, kTiles>(p.groups))
           : p.b_kn  ? go(gemm_stream_kernel<1, TOKENS>, smem_bytes<TOKENS, 1>(p.groups))
                     : go(gemm_stream_kernel<0, TOKENS>, smem_bytes<TOKENS, 0>(p.groups));
}

}  // namespace

StreamPlan stream_plan(const GemmProblem& p, int tokens, int sms) {
    switch (tokens) {
        case 16: return plan<16>(p, sms);
        case 32: return plan<32>(p, sms);
        case 64: return plan<64>(p, sms);
        default: return plan<128>(p, sms);
    }
}

fp8_status_t run_gemm_stream(const char* fn, const GemmProblem& p, int tokens, cudaStream_t st) {
    const int matrices = p.groups * (p.gated.h != nullptr ? 2 : 1);
    const Operand oa = {p.a, p.k, p.m, 1, tokens}, ob = {p.b, p.b_kn ? p.n : p.k, p.b_kn ? p.k : p.n, matrices, 128};
    CUtensorMap a = {}, b = {};
    StreamUse use(st);
    const fp8_status_t s = operand_maps(fn, oa, &a, ob, &b, use, st);
    if (s != FP8_OK) return s;
    switch (tokens) {
        case 16: return run<16>(fn, p, a, b, st);
        case 32: return run<32>(fn, p, a, b, st);
        case 64: return run<64>(fn, p, a, b, st);
        default: return run<128>(fn, p, a, b, st);
    }
}

fp8_status_t gemm_stream_wait_timeouts(unsigned long long* count) {
    return cuda_status(cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof *count), "fp8_wait_timeouts");
}

}  // namespace fp8q
