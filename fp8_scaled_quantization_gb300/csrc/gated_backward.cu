// gated_backward.cu -- the backward pass of the gated activation from an 8-bit
// checkpoint: the gradient of h and the FP8 codes of both projections in, FP8
// codes for the two backward products of each weight out.
//
//   dg = dh u act'(g),   du = dh act(g),   h = act(g) u     (gated.cuh)
//
// dg and du are written along their rows (1 x 128 tiles, the input gradient's
// operand) and transposed (1 x 128 tiles along the rows of dh, the weight
// gradient's), h transposed only (the down projection's weight gradient): 9 bytes
// an element with a BF16 dh, each read or written once.
//
// One CTA of 16 warps per SM takes 128 x 128 tiles, one after another.  A warp has
// 8 whole rows and a lane 4 columns of them, so that a row's maximum is one warp
// reduction, a word of row codes is a lane's 4 columns, and a word of transposed
// codes a lane's 4 rows: no byte is moved between lanes to transpose.  All 96
// values of a lane stay in registers until both scales are known.  Column maxima
// go through shared memory, and so do the transposed codes, to be written 16 bytes
// per lane while the next tile is computed; that one's inputs are copied into
// shared memory a tile ahead.
//
// What bounds it: 4096 x 14336 takes 116 us, without any arithmetic 101, without the
// factors (single words a row of memory apart: a tenth of the requests) 88, which is
// nine tenths of the copy's rate.  96 values and four warps per scheduler fill the
// registers, and 37 instructions per element issue in half of the slots.
// Measured, one call after another on inputs larger than L2: 4096 x 14336 116 us,
// 16384 x 18432 574 (4.7 TB/s), 8192 x 2048 38; rows that are no multiple of 16 share
// cache lines between tiles of a column (16400 x 18432 617, 8195 x 2048 46, with fp32
// gradients 54, 1337 x 13841 102).
// Others of the same mathematics, 4096 x 14336: values computed twice, by warps that
// have whole rows and warps that have whole columns, no barrier, three CTAs per SM,
// 162 us when this form took 139; 32 warps of 64 registers 179 (spills); pairs of CTAs
// with half a tile's columns each, two per SM, that exchange the rows' maxima through
// distributed shared memory 131; tiles walked down strips of 2 to 32 rows of them 122.
#include <type_traits>

#include "fp8q_host.h"
#include "fp8q_tcgen05.cuh"
#include "gated.cuh"

namespace fp8q {
namespace {

constexpr int kTile = 128, kWarps = 16, kThreads = kWarps * 32;
constexpr int kRows = kTile / kWarps;  // of a warp
constexpr int kGroup = 4;              // tiles whose factors are read and written together

struct Backward {
    const void* dh;      // [rows, n]
    const uint8_t* gu;   // [rows, 2, n] E4M3, factors [rows, 2, blocks of n]
    const float* sgu;
    int rows, n;
    uint8_t* dgu;        // as gu; nullable
    float* sdgu;
    uint8_t* dgu_t;      // [2, n, rows], factors [2, n, blocks of rows]; nullable
    float* sdgu_t;
    uint8_t* h_t;        // [n, rows] E4M3, factors [n, blocks of rows]; nullable
    float* sh_t;
    int copy_in;         // columns of dh and gu that one asynchronous copy takes: 16, 4 (aligned to that) or 0
    int run;             // tiles along a row of tiles that a CTA takes one after another: 4 or 1
    bool factors_in, factors_out;  // four tiles' factors of a row lie in aligned pieces of 16 bytes
    bool words_out;      // 4 columns store to dgu as an aligned word
    bool pieces_t, words_t;  // transposed rows are multiples of 16 (4) bytes, and aligned to that
};

// A 64-bit product of two sizes or indexes, none of them negative.
__device__ __forceinline__ int64_t wide(uint32_t a, uint32_t b) { return (int64_t)((uint64_t)a * b); }

template <bool F32>
struct Stage {  // a tile's inputs; rows and columns that are not there are zeros
    using Grad = typename std::conditional<F32, float, uint16_t>::type;
    alignas(16) Grad dh[kTile][kTile];
    alignas(16) uint8_t gu[2][kTile][kTile];
};

template <bool F32>
struct Smem {
    static constexpr int kStages = F32 ? 1 : 2;  // (two of fp32 do not fit)
    Stage<F32> stage[kStages];
    alignas(16) float most[3][kWarps][kTile];     // column maxima of each warp's rows: dg, du, h
    alignas(16) float scale[3][kTile];
    alignas(16) uint8_t codes[3][kTile * kTile];  // transposed codes, 8-byte pieces swizzled
    alignas(16) float exchange[kWarps][2 * kRows];  // row maxima and scales within a warp
    // Factors of four tiles along a row of tiles, in and out, of row i / 2, gate or up projection
    // i % 2.  Words that lie a row apart in memory cost a request each, and as single words,
    // which go through L1, more: 139 us for 4096 x 14336, in pieces of four past L1 122.
    alignas(16) float factor_in[2][2 * kTile][kGroup], factor_out[2 * kTile][kGroup];
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool there) {
    const int size = there ? BYTES : 0;  // the rest is filled with zeros
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(size) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(dst)), "l"(src), "n"(BYTES), "r"(size)
                     : "memory");
}

// Copies of a tile's inputs, COLUMNS of them at a time, which lie inside or outside the
// array as a whole.
template <int COLUMNS, bool F32>
__device__ __forceinline__ void load_pieces(const Backward& p, Stage<F32>& s, int r0, int c0) {
    constexpr int kPieces = kTile / COLUMNS, kSize = F32 ? 4 : 2, kBytes = COLUMNS * kSize, kStep = kThreads / kPieces;
    constexpr int kOne = kBytes < 16 ? kBytes : 16;
    const int x = threadIdx.x % kPieces * COLUMNS, y0 = threadIdx.x / kPieces;
    const int64_t row = wide(r0 + y0, p.n), at = row + c0 + x;
    const char* d = static_cast<const char*>(p.dh) + at * kSize;
    const uint8_t *g = p.gu + at + row, *u = g + p.n;
    if (r0 + kTile <= p.rows && c0 + kTile <= p.n) {  // all are there
#pragma unroll
        for (int y = 0; y < kTile; y += kStep, d += wide(p.n, kStep * kSize), g += wide(p.n, 2 * kStep), u += wide(p.n, 2 * kStep)) {
#pragma unroll
            for (int b = 0; b < kBytes; b += 16)
                copy_async<kOne>(reinterpret_cast<char*>(&s.dh[y0 + y][x]) + b, d + b, true);
            copy_async<COLUMNS>(&s.gu[0][y0 + y][x], g, true);
            copy_async<COLUMNS>(&s.gu[1][y0 + y][x], u, true);
        }
    } else {
#pragma unroll 1
        for (int y = 0; y < kTile; y += kStep, d += wide(p.n, kStep * kSize), g += wide(p.n, 2 * kStep), u += wide(p.n, 2 * kStep)) {
            const bool there = r0 + y0 + y < p.rows && c0 + x < p.n;
#pragma unroll
            for (int b = 0; b < kBytes; b += 16)
                copy_async<kOne>(reinterpret_cast<char*>(&s.dh[y0 + y][x]) + b, there ? d + b : p.dh, there);
            copy_async<COLUMNS>(&s.gu[0][y0 + y][x], there ? g : p.gu, there);
            copy_async<COLUMNS>(&s.gu[1][y0 + y][x], there ? u : p.gu, there);
        }
    }
}

// Bytes 4 word .. 4 word + 3 of a line of len bytes, zeros from its end on.  Only aligned
// words are read that hold a byte of the line.
__device__ __forceinline__ uint32_t word_of_line(const uint8_t* line, int word, int len) {
    const int off = (int)(reinterpret_cast<uintptr_t>(line) & 3u), left = len - 4 * word;
    const uint32_t* const from = reinterpret_cast<const uint32_t*>(line - off) + word;
    const uint32_t lo = left + off > 0 && len > 0 ? __ldg(from) : 0u, hi = left + off > 4 && off > 0 ? __ldg(from + 1) : 0u;
    const uint32_t v = __funnelshift_r(lo, hi, 8 * off);
    return left >= 4 ? v : left <= 0 ? 0u : v & (0xFFFFFFFFu >> (32 - 8 * left));
}

// A line of `len` codes that starts anywhere, a word per lane, to q: aligned words, and the
// line's first and last bytes, which share words with other lines, one by one.
__device__ __forceinline__ void store_line(uint8_t* q, uint32_t w, int len, int lane) {
    const uint32_t before = __shfl_up_sync(0xFFFFFFFFu, w, 1);
    const int off = (int)(reinterpret_cast<uintptr_t>(q) & 3u), left = len - lane * 4;
    if ((lane > 0 || off == 0) && left >= 4 - off) *reinterpret_cast<uint32_t*>(q + lane * 4 - off) = __funnelshift_l(before, w, 8 * off);
    const int head = lane == 0 ? -off & 3 : 0, tail = left - ((len + off) & 3);
    if (head > 0 || tail < 4) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x < left && (x < head || x >= tail)) q[lane * 4 + x] = (uint8_t)(w >> (8 * x));
    }
}

template <bool F32>
__device__ __forceinline__ void load_tile(const Backward& p, Stage<F32>& s, int tr, int tc) {
    const int r0 = tr * kTile, c0 = tc * kTile;
    if (p.copy_in == 16) {
        load_pieces<16>(p, s, r0, c0);
    } else if (p.copy_in == 4) {
        load_pieces<4>(p, s, r0, c0);
    } else {
        // Rows that start anywhere, by the warp that uses them: each word put together from the two
        // aligned ones that hold it.
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cols = min(p.n - c0, kTile);
#pragma unroll 4
        for (int i = 0; i < kRows; ++i) {
            const int y = warp * kRows + i;
            const bool there = r0 + y < p.rows;
            const int64_t row = wide(r0 + y, p.n), at = row + c0;
            const int len = there ? cols : 0;
            *reinterpret_cast<uint32_t*>(&s.gu[0][y][lane * 4]) = word_of_line(p.gu + at + row, lane, len);
            *reinterpret_cast<uint32_t*>(&s.gu[1][y][lane * 4]) = word_of_line(p.gu + at + row + p.n, lane, len);
            if constexpr (F32) {
#pragma unroll
                for (int x = lane; x < kTile; x += 32) s.dh[y][x] = x < len ? __ldg(static_cast<const float*>(p.dh) + at + x) : 0.0f;
            } else {
                const uint8_t* const line = static_cast<const uint8_t*>(p.dh) + 2 * at;
#pragma unroll
                for (int w = lane; w < kTile / 2; w += 32)
                    *reinterpret_cast<uint32_t*>(&s.dh[y][2 * w]) = word_of_line(line, w, 2 * len);
            }
        }
    }
}

// The factors of a tile, or of the four tiles around it where they lie in aligned pieces.
__device__ __forceinline__ void load_factors(const Backward& p, float (&in)[2 * kTile][kGroup], int tr, int tc, int nb, bool whole) {
    if (threadIdx.x >= 2 * kTile) return;
    const uint32_t at = 2u * tr * kTile + threadIdx.x;
    const bool there = (int)(at >> 1) < p.rows;
    const float* const from = p.sgu + (there ? wide(at, nb) + tc : 0);
    if (whole) copy_async<16>(in[threadIdx.x], there ? from - tc % kGroup : from, there);
    else copy_async<4>(&in[threadIdx.x][tc % kGroup], from, there);
}

// The factors of dg and du of the tiles tc - tc % 4 + first .. tc.
__device__ __forceinline__ void store_factors(const Backward& p, const float (&out)[2 * kTile][kGroup], int tr, int tc, int nb, int first) {
    if (threadIdx.x >= 2 * kTile) return;
    const uint32_t at = 2u * tr * kTile + threadIdx.x;
    const int last = tc % kGroup;
    if ((int)(at >> 1) >= p.rows) return;
    float* const to = p.sdgu + wide(at, nb) + (tc - last);
    const float4 v = *reinterpret_cast<const float4*>(out[threadIdx.x]);
    if (p.factors_out && first == 0 && last == kGroup - 1) {
        *reinterpret_cast<float4*>(to) = v;
    } else {
        if (first == 0) to[0] = v.x;
        if (first <= 1 && last >= 1) to[1] = v.y;
        if (first <= 2 && last >= 2) to[2] = v.z;
        if (last == 3) to[3] = v.w;
    }
}

// Four codes of scaled values.  cvt.satfinite gives every code by the rule but that of
// an E5M2 infinity, which is the code of the largest value and one more; `special`:
// there may be some (a finite value times its tile's scale is finite).
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, bool special) {
    uint32_t r = cvt4<FMT>(a, b, c, d);
    if (FMT == kE5M2 && special)
        r += (isinf(a) ? 1u : 0u) + (isinf(b) ? 1u << 8 : 0u) + (isinf(c) ? 1u << 16 : 0u) + (isinf(d) ? 1u << 24 : 0u);
    return r;
}

// Where the 8 bytes of a warp's rows in column `col` lie: pieces move with the column's
// lane, so that a warp's stores (column 4 lane + j) and the copy's reads spread over the banks.
__device__ __forceinline__ uint32_t piece_at(int col, int piece) { return col * kTile + ((piece ^ (col >> 2 & 15)) << 3); }

// The transposed codes of a tile from shared memory to the outputs.
__device__ __forceinline__ void write_columns(const Backward& p, const uint8_t (&codes)[3][kTile * kTile], int tr, int tc,
                                              int warp, int lane) {
    const int rows = min(p.rows - tr * kTile, kTile), there = min(p.n - tc * kTile, kTile);
    const int64_t mine = wide(lane >> 3, p.rows) + (lane & 7) * 16;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint8_t* const out = k < 2 ? p.dgu_t : p.h_t;
        if (out == nullptr) continue;
        uint8_t* const base = out + wide((k == 1 ? (uint32_t)p.n : 0u) + tc * kTile, p.rows) + tr * kTile;
        if (p.pieces_t) {  // 4 columns of 8 times 16 bytes per warp and step
            const int col = warp * 4 + (lane >> 3), piece = lane & 7;
            uint8_t* q = base + wide(warp * 4, p.rows) + mine;
            const int left = piece * 16 < rows ? there - col : 0;
#pragma unroll
            for (int step = 0; step < 2; ++step, q += wide(64, p.rows)) {
                // two pieces of 8 bytes that the swizzle keeps together, the warp's all in one order
                const uint4 v = *reinterpret_cast<const uint4*>(&codes[k][piece_at(col + step * 64, 2 * piece) & ~15u]);
                if (step * 64 < left) stg_stream(q, warp & 1 ? make_uint4(v.z, v.w, v.x, v.y) : v);
            }
        } else {  // a column per warp, 4 bytes of it per lane, all columns at once
            constexpr int kEach = kTile / kWarps;
            uint32_t w[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                w[i] = *reinterpret_cast<const uint32_t*>(&codes[k][piece_at(i * kWarps + warp, lane >> 1) + (lane & 1) * 4]);
            uint8_t* q = base + wide(warp, p.rows) + lane * 4;
            if (p.words_t) {
#pragma unroll
                for (int i = 0; i < kEach; ++i, q += wide(kWarps, p.rows))
                    if (i * kWarps + warp < there && lane * 4 < rows) *reinterpret_cast<uint32_t*>(q) = w[i];
            } else {
#pragma unroll
                for (int i = 0; i < kEach; ++i, q += wide(kWarps, p.rows)) {
                    // the aligned word that starts `off` bytes before this lane's, where it lies in the column
                    const uint32_t before = __shfl_up_sync(0xFFFFFFFFu, w[i], 1);
                    const int off = (int)(reinterpret_cast<uintptr_t>(q) & 3u), left = rows - lane * 4;
                    if (i * kWarps + warp < there && (lane > 0 || off == 0) && left >= 4 - off)
                        *reinterpret_cast<uint32_t*>(q - off) = __funnelshift_l(before, w[i], 8 * off);
                }
                // What is left of a column shares words with others and goes byte by byte: its first
                // -off mod 4 bytes and its last (rows + off) mod 4, six at most.  A column's on 4 lanes.
                static_assert(kEach * 4 == 32, "a warp's columns, 4 lanes each");
                const int col = (lane >> 2) * kWarps + warp;
                uint8_t* const line = base + wide(col, p.rows);
                const int off = (int)(reinterpret_cast<uintptr_t>(line) & 3u), head = min(-off & 3, rows);
                const int tail = min((rows + off) & 3, rows - head);
#pragma unroll
                for (int turn = 0; turn < 2; ++turn) {
                    const int e = turn * 4 + (lane & 3), x = e < head ? e : rows - tail + e - head;
                    if (e < head + tail && col < there) line[x] = codes[k][piece_at(col, x >> 3) + (x & 7)];
                }
            }
        }
    }
}

// Two columns at once, as packed pairs (fma.rn.f32x2 and its like).
template <int ACT>
__device__ __forceinline__ void differentiate(uint64_t d, uint64_t g, uint64_t u, uint64_t* dg, uint64_t* du, uint64_t* h) {
    uint64_t dy = 0;
    const uint64_t s = gate2<ACT, true>(g, &dy), a = mul2(g, s), rest = fma2(s, pack2(-1.0f, -1.0f), pack2(1.0f, 1.0f));
    // y' with 1 - s first, which is 0 where g is large: a y' would be Inf for g beyond 1.5e36
    const uint64_t slope = fma2(a, ACT == kSilu ? rest : mul2(rest, dy), s);
    *dg = mul2(mul2(d, u), slope);
    *du = mul2(d, a);
    *h = mul2(a, u);
}

// Two E4M3 codes (the low half of c) times a factor, as a packed pair.
__device__ __forceinline__ uint64_t values2(uint32_t c, uint64_t factor) {
    const uint32_t v = fp8x2_to_f16x2<kE4M3>(c);
    return mul2(pack2(f16_lo_to_f32(v), f16_hi_to_f32(v)), factor);
}

// The scale of a tile by the rule of scale_from_amax, its format known at run time.
__device__ __forceinline__ void scale_of(float amax, bool e5m2, float* scale, float* factor) {
    const bool usual = amax > 0.0f && !isinf(amax);
    float s = __fdiv_rn(e5m2 ? Fmt<kE5M2>::kMax : Fmt<kE4M3>::kMax, usual ? amax : 1.0f);
    s = usual ? fminf(fmaxf(s, 1.175494351e-38f), 3.402823466e+38f) : 1.0f;
    *scale = s;
    *factor = __fdiv_rn(1.0f, s);
}

template <int FMT, int ACT, bool F32>
__global__ void __launch_bounds__(kThreads, 1) gated_backward_kernel(const __grid_constant__ Backward p) {
    extern __shared__ __align__(128) uint8_t raw[];
    Smem<F32>& sm = *reinterpret_cast<Smem<F32>*>(raw);
    constexpr int kStages = Smem<F32>::kStages;
    // (a shuffle tells the compiler that the number is the same in the whole warp)
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int nb = (p.n + kTile - 1) / kTile, rb = (p.rows + kTile - 1) / kTile;
    // Runs of p.run tiles along the columns, every gridDim.x-th of them: what the CTAs work on at
    // one time lies close together, and the pieces of a cache line that two tiles of a column
    // share meet in L2.  (One long run per CTA: 1.8 times as long for 16400 x 18432.)
    const int runs = (nb + p.run - 1) / p.run, step_r = gridDim.x / runs, step_c = gridDim.x % runs;
    int run_r = blockIdx.x / runs, run_c = blockIdx.x % runs, tr = run_r, tc = run_c * p.run;
    pdl_begin();
    const auto load = [&](int r, int c, int stage, bool there) {
        if (there) load_tile<F32>(p, sm.stage[stage], r, c);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load_factors(p, sm.factor_in[0], tr, tc, nb, p.factors_in);
    load(tr, tc, 0, true);
    const bool columns = p.dgu_t != nullptr || p.h_t != nullptr;
    int at = 0, last_r = -1, last_c = 0;    // the tile whose transposed codes wait in shared memory
    int group = 0, first = tc % kGroup;     // the place of this run's factors, its first tile of four
    for (int next_r, next_c, next_group; tr < rb; tr = next_r, tc = next_c, group = next_group) {
        next_r = tr, next_c = tc + 1, next_group = group;
        const bool last_of_run = next_c == nb || next_c % p.run == 0;
        if (last_of_run) {
            run_r += step_r, run_c += step_c;
            if (run_c >= runs) run_c -= runs, ++run_r;
            next_r = run_r, next_c = run_c * p.run, next_group = group ^ 1;
        }
        const bool more = next_r < rb;
        const int r0 = tr * kTile + warp * kRows, c0 = tc * kTile + lane * 4;
        const int rows = min(p.rows - r0, kRows);  // here
        const Stage<F32>& st = sm.stage[at];
        const float (&factors)[2 * kTile][kGroup] = sm.factor_in[group];
        if (kStages == 2) {  // the other stage was left by all before the last tile's maxima
            at ^= 1;
            load(next_r, next_c, at, more);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncthreads();  // this tile's inputs have landed, and the last one's codes are all there
        if (last_r >= 0) write_columns(p, sm.codes, last_r, last_c, warp, lane);

        float dg[kRows][4], du[kRows][4], h[kRows][4];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int y = warp * kRows + i;
            uint64_t d[2];
            if constexpr (F32) {
                const float4 v = *reinterpret_cast<const float4*>(&st.dh[y][lane * 4]);
                d[0] = pack2(v.x, v.y), d[1] = pack2(v.z, v.w);
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(&st.dh[y][lane * 4]);
                d[0] = pack2(bf16lo(v.x), bf16hi(v.x)), d[1] = pack2(bf16lo(v.y), bf16hi(v.y));
            }
            const uint32_t gq = *reinterpret_cast<const uint32_t*>(&st.gu[0][y][lane * 4]);
            const uint32_t uq = *reinterpret_cast<const uint32_t*>(&st.gu[1][y][lane * 4]);
            const float fg = factors[2 * y][tc % kGroup], fu = factors[2 * y + 1][tc % kGroup];
            const uint64_t sg = pack2(fg, fg), su = pack2(fu, fu);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint64_t g = values2(gq >> (16 * j), sg), u = values2(uq >> (16 * j), su);
                uint64_t vg, vu, vh;
                differentiate<ACT>(d[j], g, u, &vg, &vu, &vh);
                const float2 a = unpack2(vg), b = unpack2(vu), c = unpack2(vh);
                dg[i][2 * j] = a.x, dg[i][2 * j + 1] = a.y;
                du[i][2 * j] = b.x, du[i][2 * j + 1] = b.y;
                h[i][2 * j] = c.x, h[i][2 * j + 1] = c.y;
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {  // the largest of each column, of this warp's rows
            const float (&v)[kRows][4] = k == 0 ? dg : k == 1 ? du : h;
            float m[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[j] = max_abs3(fabsf(v[0][j]), v[1][j], v[2][j]);
#pragma unroll
                for (int i = 3; i < kRows; i += 2) m[j] = max_abs3(m[j], v[i][j], v[i + 1 < kRows ? i + 1 : i][j]);
            }
            *reinterpret_cast<float4*>(&sm.most[k][warp][lane * 4]) = make_float4(m[0], m[1], m[2], m[3]);
        }
        // A warp's row maxima are the same in all lanes, and go through shared memory four words
        // at a time (fewer instructions than selects and shuffles): 2 i + k of row i of dg (k 0) or du.
        float* const exchange = sm.exchange[warp];
        {
            uint32_t most[2 * kRows];
#pragma unroll
            for (int i = 0; i < 2 * kRows; ++i) {
                const float (&v)[4] = i & 1 ? du[i >> 1] : dg[i >> 1];
                most[i] = warp_max_u32(__float_as_uint(max_abs3(max_abs3(v[0], v[0], v[1]), v[2], v[3])));
            }
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < 2 * kRows; i += 4)
                    *reinterpret_cast<uint4*>(exchange + i) = make_uint4(most[i], most[i + 1], most[i + 2], most[i + 3]);
            }
        }
        __syncthreads();
        if (more && (last_of_run || !p.factors_in)) load_factors(p, sm.factor_in[next_group], next_r, next_c, nb, p.factors_in);
        load(next_r, next_c, 0, kStages == 1 && more);

        // ---- scales: a warp's 16 of its rows, and the tile's 384 of columns, a thread each, in one
        // chain of divisions.  The sign, which no scale has, marks a tile with Inf or NaN.
        {
            const int k = threadIdx.x / kTile, col = threadIdx.x % kTile;  // (k 3: no column)
            float most = 0.0f;
            if (k < 3) {
#pragma unroll
                for (int w = 0; w < kWarps; w += 2) most = max_abs3(most, sm.most[k][w][col], sm.most[k][w + 1][col]);
            }
            const float amax = exchange[lane % (2 * kRows)];
            float scale, factor, row_scale, row_factor;
            scale_of(most, FMT == kE5M2 && k < 2, &scale, &factor);
            scale_of(amax, FMT == kE5M2, &row_scale, &row_factor);
            __syncwarp();
            if (lane < 2 * kRows) {
                exchange[lane] = __float_as_uint(amax) >= 0x7F800000u ? -row_scale : row_scale;
                sm.factor_out[warp * 2 * kRows + lane][tc % kGroup] = row_factor;
            }
            if (k < 3) {
                sm.scale[k][col] = __float_as_uint(most) >= 0x7F800000u ? -scale : scale;
                const int c = tc * kTile + col;
                float* const out = k < 2 ? p.sdgu_t : p.sh_t;
                if (out != nullptr && c < p.n) out[wide((k == 1 ? (uint32_t)p.n : 0u) + c, rb) + tr] = factor;
            }
        }
        __syncthreads();

        if (last_of_run) {
            if (p.dgu != nullptr) store_factors(p, sm.factor_out, tr, tc, nb, first);
            first = next_c % kGroup;
        }

        // ---- codes along the rows
        if (p.dgu != nullptr) {
            uint8_t* q = p.dgu + wide(2u * r0, p.n) + c0;
            const auto codes = [&](auto store) {
#pragma unroll
                for (int i0 = 0; i0 < 2 * kRows; i0 += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(exchange + i0);
                    const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i, q += p.n) {
                        const float (&v)[4] = i & 1 ? du[(i0 + i) >> 1] : dg[(i0 + i) >> 1];
                        const float2 a = fmul2_rn(v[0], v[1], fabsf(s[i])), b = fmul2_rn(v[2], v[3], fabsf(s[i]));
                        store((i0 + i) >> 1, codes4<FMT>(a.x, a.y, b.x, b.y, s[i] < 0.0f));
                    }
                }
            };
            if (p.words_out && rows == kRows && (tc + 1) * kTile <= p.n)  // all are there
                codes([&](int, uint32_t c) { *reinterpret_cast<uint32_t*>(q) = c; });
            else
                codes([&](int i, uint32_t c) {
                    if (i < rows) store_line(q - lane * 4, c, min(p.n - tc * kTile, kTile), lane);
                });
        }
        if (!columns) continue;

        // ---- transposed codes: products of two columns at a time, codes of four rows
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float (&v)[kRows][4] = k == 0 ? dg : k == 1 ? du : h;
            const float4 s4 = *reinterpret_cast<const float4*>(&sm.scale[k][lane * 4]);
            const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const uint64_t s2 = pack2(fabsf(s[j]), fabsf(s[j + 1]));
                float2 x[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) x[i] = unpack2(mul2(pack2(v[i][j], v[i][j + 1]), s2));
                uint2 c[2];
                if (k < 2) {
                    c[0] = make_uint2(codes4<FMT>(x[0].x, x[1].x, x[2].x, x[3].x, s[j] < 0.0f),
                                      codes4<FMT>(x[4].x, x[5].x, x[6].x, x[7].x, s[j] < 0.0f));
                    c[1] = make_uint2(codes4<FMT>(x[0].y, x[1].y, x[2].y, x[3].y, s[j + 1] < 0.0f),
                                      codes4<FMT>(x[4].y, x[5].y, x[6].y, x[7].y, s[j + 1] < 0.0f));
                } else {
                    c[0] = make_uint2(cvt4<kE4M3>(x[0].x, x[1].x, x[2].x, x[3].x), cvt4<kE4M3>(x[4].x, x[5].x, x[6].x, x[7].x));
                    c[1] = make_uint2(cvt4<kE4M3>(x[0].y, x[1].y, x[2].y, x[3].y), cvt4<kE4M3>(x[4].y, x[5].y, x[6].y, x[7].y));
                }
                *reinterpret_cast<uint2*>(&sm.codes[k][piece_at(lane * 4 + j, warp)]) = c[0];
                *reinterpret_cast<uint2*>(&sm.codes[k][piece_at(lane * 4 + j + 1, warp)]) = c[1];
            }
        }
        last_r = tr, last_c = tc;
    }
    if (last_r >= 0) {
        __syncthreads();
        write_columns(p, sm.codes, last_r, last_c, warp, lane);
    }
}

fp8_status_t run(const char* fn, Backward p, bool f32, int fmt, int act, cudaStream_t st) {
    // Runs of four tiles share reads and writes of factors (single tiles: 3% longer for 4096 x 14336,
    // 1.5% for 16384 x 18432), but their last round may leave more CTAs idle (8192 x 2048: 10% longer).
    const int64_t nb = (p.n + kTile - 1) / kTile, rb = (p.rows + kTile - 1) / kTile;
    const int sms = sm_count();
    int64_t ctas = 0;
    double best = 0.0;
    for (int run : {4, 1}) {
        const int64_t runs = (nb + run - 1) / run * rb;
        const double cost = (double)((runs + sms - 1) / sms) * run * (run == 4 ? 1.0 : 1.02);
        if (ctas == 0 || cost < best) best = cost, p.run = run, ctas = runs < sms ? runs : sms;
    }
    const auto go = [&](auto kernel) {
        return launch_smem(fn, kernel, dim3((unsigned)ctas), dim3(kThreads), f32 ? sizeof(Smem<true>) : sizeof(Smem<false>), st, p);
    };
    const auto pick = [&](auto silu, auto gelu) { return act == kSilu ? go(silu) : go(gelu); };
    if (fmt == kE4M3)
        return f32 ? pick(gated_backward_kernel<kE4M3, kSilu, true>, gated_backward_kernel<kE4M3, kGeluTanh, true>)
                   : pick(gated_backward_kernel<kE4M3, kSilu, false>, gated_backward_kernel<kE4M3, kGeluTanh, false>);
    return f32 ? pick(gated_backward_kernel<kE5M2, kSilu, true>, gated_backward_kernel<kE5M2, kGeluTanh, true>)
               : pick(gated_backward_kernel<kE5M2, kSilu, false>, gated_backward_kernel<kE5M2, kGeluTanh, false>);
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8_status_t fp8_gated_block_backward(const void* dh, fp8_dtype_t dtype, const uint8_t* gu,
                                                 const float* scale_inv_gu, fp8_activation_t act, int64_t rows,
                                                 int64_t n, fp8_format_t fmt_grad, uint8_t* dgu, float* scale_inv_dgu,
                                                 uint8_t* dgu_t, float* scale_inv_dgu_t, uint8_t* h_t,
                                                 float* scale_inv_h_t, void* stream) {
    const char* fn = "fp8_gated_block_backward";
    if (!valid_dtype(dtype)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (!valid_fmt(fmt_grad)) return fail(FP8_ERR_INVALID_ARG, "%s: unknown format %d", fn, (int)fmt_grad);
    if (act != FP8_ACT_SILU && act != FP8_ACT_GELU_TANH)
        return fail(FP8_ERR_INVALID_ARG, "%s: unknown activation %d", fn, (int)act);
    if (rows < 0 || n < 0) return fail(FP8_ERR_INVALID_ARG, "%s: negative size", fn);
    constexpr int64_t kMost = (1ll << 31) - 256, kMostTiles = 1ll << 30;
    if (rows > kMost || n > kMost) return fail(FP8_ERR_UNSUPPORTED, "%s: sizes must be below 2^31 - 256", fn);
    if (((rows + kTile - 1) / kTile) * ((n + kTile - 1) / kTile) > kMostTiles)
        return fail(FP8_ERR_UNSUPPORTED, "%s: too many tiles", fn);
    if ((dgu == nullptr) != (scale_inv_dgu == nullptr) || (dgu_t == nullptr) != (scale_inv_dgu_t == nullptr) ||
        (h_t == nullptr) != (scale_inv_h_t == nullptr))
        return fail(FP8_ERR_INVALID_ARG, "%s: each output needs both its codes and its scales", fn);
    if (rows == 0 || n == 0) return FP8_OK;
    if (dgu == nullptr && dgu_t == nullptr && h_t == nullptr)
        return fail(FP8_ERR_INVALID_ARG, "%s: no output requested", fn);
    if (dh == nullptr || gu == nullptr || scale_inv_gu == nullptr)
        return fail(FP8_ERR_INVALID_ARG, "%s: an input is NULL", fn);
    if (reinterpret_cast<uintptr_t>(dh) % dtype_size(dtype))
        return fail(FP8_ERR_INVALID_ARG, "%s: dh is not element-aligned", fn);
    for (const float* s : {scale_inv_gu, (const float*)scale_inv_dgu, (const float*)scale_inv_dgu_t, (const float*)scale_inv_h_t})
        if ((reinterpret_cast<uintptr_t>(s) & 3u) != 0)
            return fail(FP8_ERR_INVALID_ARG, "%s: scales are not 4-byte aligned", fn);
    const auto aligned = [](const void* q, uintptr_t to) { return reinterpret_cast<uintptr_t>(q) % to == 0; };
    Backward p = {dh, gu, scale_inv_gu, (int)rows, (int)n, dgu, scale_inv_dgu, dgu_t, scale_inv_dgu_t, h_t, scale_inv_h_t};
    const auto copies = [&](int columns) {
        const int bytes = columns * dtype_size(dtype);
        return n % columns == 0 && aligned(gu, columns) && aligned(dh, bytes < 16 ? bytes : 16);
    };
    p.copy_in = copies(16) ? 16 : copies(4) ? 4 : 0;
    const bool pieces = (n + kTile - 1) / kTile % kGroup == 0;
    p.factors_in = pieces && aligned16(scale_inv_gu);
    p.factors_out = pieces && aligned16(scale_inv_dgu);
    p.words_out = n % 4 == 0 && aligned(dgu, 4);
    p.words_t = rows % 4 == 0 && aligned(dgu_t, 4) && aligned(h_t, 4);
    p.pieces_t = rows % 16 == 0 && aligned16(dgu_t) && aligned16(h_t);
    return run(fn, p, dtype == FP8_DT_FP32, (int)fmt_grad, (int)act, static_cast<cudaStream_t>(stream));
}
