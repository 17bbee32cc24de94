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
// One CTA of 16 warps per 128 x 128 tile at a time.  A warp has 8 whole rows and
// a lane 4 columns of them, so that a row's maximum is one warp reduction, a
// word of row codes is a lane's 4 columns, and a word of transposed codes a
// lane's 4 rows: no byte is moved between lanes to transpose.  Column maxima go
// through shared memory, and so do the transposed codes, to be written 16 bytes
// per lane.
#include "fp8q_host.h"
#include "fp8q_pipeline.cuh"
#include "gated.cuh"

namespace fp8q {
namespace {

constexpr int kTile = 128, kWarps = 16, kThreads = kWarps * 32;
constexpr int kRows = kTile / kWarps;  // of a warp

struct Backward {
    const void* dh;      // [rows, n]
    const uint8_t* gu;   // [rows, 2, n] E4M3, factors [rows, 2, blocks of n]
    const float* sgu;
    int64_t rows, n;
    uint8_t* dgu;        // as gu; nullable
    float* sdgu;
    uint8_t* dgu_t;      // [2, n, rows], factors [2, n, blocks of rows]; nullable
    float* sdgu_t;
    uint8_t* h_t;        // [n, rows] E4M3, factors [n, blocks of rows]; nullable
    float* sh_t;
    bool words_in;       // 4 columns of dh and gu load as aligned words
    bool words_out;      // and store to dgu
    bool pieces_t;       // transposed rows are multiples of 16 bytes, 16-byte aligned
};

struct Smem {
    uint32_t most[3][kWarps][kTile];       // column maxima of each warp's rows: dg, du, h
    float scale[3][kTile];
    alignas(16) uint8_t codes[3][kTile * kTile];  // transposed codes, 8-byte pieces swizzled
};

// Four codes of values whose tile holds Inf or NaN (scale 1), each by its own rule.
template <int FMT>
__device__ __noinline__ uint32_t cvt4_exact(float a, float b, float c, float d) {
    uint32_t sat;
    return quant_one<FMT>(a, 1.0f, &sat) | quant_one<FMT>(b, 1.0f, &sat) << 8 | quant_one<FMT>(c, 1.0f, &sat) << 16 |
           quant_one<FMT>(d, 1.0f, &sat) << 24;
}

// cvt.satfinite gives every code by the rule but that of an E5M2 infinity.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float scale, bool special) {
    if (FMT == kE5M2 && special) return cvt4_exact<FMT>(a, b, c, d);
    const float2 lo = fmul2_rn(a, b, scale), hi = fmul2_rn(c, d, scale);
    return cvt4<FMT>(lo.x, lo.y, hi.x, hi.y);
}

// Where the 8 bytes of a warp's rows in column `col` lie: pieces move with the column's
// lane, so that a warp's stores (column 4 lane + j) and the copy's reads spread over the banks.
__device__ __forceinline__ uint32_t piece_at(int col, int piece) { return col * kTile + ((piece ^ (col >> 2 & 15)) << 3); }

template <int FMT, int ACT, bool F32>
__global__ void __launch_bounds__(kThreads, 1) gated_backward_kernel(const __grid_constant__ Backward p) {
    extern __shared__ __align__(128) uint8_t raw[];
    Smem& sm = *reinterpret_cast<Smem*>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nb = (int)((p.n + kTile - 1) / kTile), rb = (int)((p.rows + kTile - 1) / kTile);
    pdl_begin();
    for (int64_t t = blockIdx.x; t < (int64_t)nb * rb; t += gridDim.x) {
        const int tr = (int)(t / nb), tc = (int)(t % nb);
        const int64_t r0 = (int64_t)tr * kTile + warp * kRows, c0 = (int64_t)tc * kTile + lane * 4;
        const int cols = (int)(p.n - c0 < 4 ? p.n - c0 : 4);  // of this lane
        float dg[kRows][4], du[kRows][4], h[kRows][4];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t r = r0 + i;
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t gq = 0, uq = 0;
            float sg = 0.0f, su = 0.0f;
            if (r < p.rows && cols > 0) {
                const uint8_t* const g = p.gu + 2 * r * p.n + c0;
                const int64_t at = r * p.n + c0;
                if (p.words_in) {
                    gq = __ldg(reinterpret_cast<const uint32_t*>(g));
                    uq = __ldg(reinterpret_cast<const uint32_t*>(g + p.n));
                    if constexpr (F32) {
                        const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.dh) + at));
                        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
                    } else {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.dh) + at));
                        d[0] = bf16lo(v.x), d[1] = bf16hi(v.x), d[2] = bf16lo(v.y), d[3] = bf16hi(v.y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j >= cols) break;
                        gq |= (uint32_t)__ldg(g + j) << (8 * j);
                        uq |= (uint32_t)__ldg(g + p.n + j) << (8 * j);
                        d[j] = F32 ? __ldg(static_cast<const float*>(p.dh) + at + j)
                                   : __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p.dh) + at + j) << 16);
                    }
                }
                sg = __ldg(p.sgu + 2 * r * nb + tc);
                su = __ldg(p.sgu + (2 * r + 1) * nb + tc);
            }
            const uint32_t gh[2] = {fp8x2_to_f16x2<kE4M3>(gq), fp8x2_to_f16x2<kE4M3>(gq >> 16)};
            const uint32_t uh[2] = {fp8x2_to_f16x2<kE4M3>(uq), fp8x2_to_f16x2<kE4M3>(uq >> 16)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float gv = (j & 1 ? f16_hi_to_f32(gh[j >> 1]) : f16_lo_to_f32(gh[j >> 1])) * sg;
                const float uv = (j & 1 ? f16_hi_to_f32(uh[j >> 1]) : f16_lo_to_f32(uh[j >> 1])) * su;
                float dy = 1.0f;
                const float s = gate<ACT, true>(gv, &dy), a = gv * s;
                const float slope = __fmaf_rn(ACT == kSilu ? a : a * dy, 1.0f - s, s);
                const bool there = j < cols && r < p.rows;  // (a factor that is NaN counts for no other row)
                dg[i][j] = there ? d[j] * uv * slope : 0.0f;
                du[i][j] = there ? d[j] * a : 0.0f;
                h[i][j] = there ? a * uv : 0.0f;
            }
        }

        // ---- along the rows: lane 8 k + i derives the scale of row i of dg (k 0) or du (k 1)
        if (p.dgu != nullptr) {
            uint32_t mine = 0;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                uint32_t a = 0, b = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) a = max_abs(a, dg[i][j]), b = max_abs(b, du[i][j]);
                a = warp_max_u32(a), b = warp_max_u32(b);
                if (lane == i) mine = a;
                if (lane == 8 + i) mine = b;
            }
            float scale, factor;
            scale_from_amax<FMT>(__uint_as_float(mine), 0, &scale, &factor);
            if (lane < 16 && r0 + (lane & 7) < p.rows)
                p.sdgu[(2 * (r0 + (lane & 7)) + (lane >> 3)) * nb + tc] = factor;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float (&v)[4] = k == 0 ? dg[i] : du[i];
                    const float s = __shfl_sync(0xFFFFFFFFu, scale, 8 * k + i);
                    const uint32_t top = FMT == kE5M2 ? __shfl_sync(0xFFFFFFFFu, mine, 8 * k + i) : 0u;
                    const uint32_t c = codes4<FMT>(v[0], v[1], v[2], v[3], s, top >= 0x7F800000u);
                    if (r0 + i >= p.rows || cols <= 0) continue;
                    uint8_t* const q = p.dgu + (2 * (r0 + i) + k) * p.n + c0;
                    if (p.words_out) {
                        *reinterpret_cast<uint32_t*>(q) = c;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < cols) q[j] = (uint8_t)(c >> (8 * j));
                    }
                }
            }
        }

        // ---- along the columns
        if (p.dgu_t == nullptr && p.h_t == nullptr) continue;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float (&v)[kRows][4] = k == 0 ? dg : k == 1 ? du : h;
            uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) m[j] = max_abs(m[j], v[i][j]);
            *reinterpret_cast<uint4*>(&sm.most[k][warp][lane * 4]) = make_uint4(m[0], m[1], m[2], m[3]);
        }
        __syncthreads();  // (and the codes of the last tile have been read)
        if (threadIdx.x < 3 * kTile) {
            const int k = threadIdx.x / kTile, col = threadIdx.x % kTile;
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = umax(m, sm.most[k][w][col]);
            float scale, factor;
            if (k < 2) scale_from_amax<FMT>(__uint_as_float(m), 0, &scale, &factor);
            else scale_from_amax<kE4M3>(__uint_as_float(m), 0, &scale, &factor);
            // the sign, which no scale has, marks a tile with Inf or NaN
            sm.scale[k][col] = m >= 0x7F800000u ? -scale : scale;
            const int64_t c = (int64_t)tc * kTile + col;
            float* const out = k < 2 ? p.sdgu_t : p.sh_t;
            if (out != nullptr && c < p.n) out[((k == 1 ? p.n : 0) + c) * rb + tr] = factor;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float (&v)[kRows][4] = k == 0 ? dg : k == 1 ? du : h;
            const float4 s4 = *reinterpret_cast<const float4*>(&sm.scale[k][lane * 4]);
            const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                constexpr int kGrad = FMT;
                uint2 c;
                if (k < 2) {
                    c.x = codes4<kGrad>(v[0][j], v[1][j], v[2][j], v[3][j], fabsf(s[j]), s[j] < 0.0f);
                    c.y = codes4<kGrad>(v[4][j], v[5][j], v[6][j], v[7][j], fabsf(s[j]), s[j] < 0.0f);
                } else {
                    c.x = codes4<kE4M3>(v[0][j], v[1][j], v[2][j], v[3][j], fabsf(s[j]), false);
                    c.y = codes4<kE4M3>(v[4][j], v[5][j], v[6][j], v[7][j], fabsf(s[j]), false);
                }
                *reinterpret_cast<uint2*>(&sm.codes[k][piece_at(lane * 4 + j, warp)]) = c;
            }
        }
        __syncthreads();
        const int rows = (int)(p.rows - (int64_t)tr * kTile < kTile ? p.rows - (int64_t)tr * kTile : kTile);
#pragma unroll 1
        for (int k = 0; k < 3; ++k) {
            uint8_t* const out = k < 2 ? p.dgu_t : p.h_t;
            if (out == nullptr) continue;
            const int64_t first = (k == 1 ? p.n : 0) + (int64_t)tc * kTile;
            uint8_t* const base = out + first * p.rows + (int64_t)tr * kTile;
            const int there = (int)(p.n - (int64_t)tc * kTile < kTile ? p.n - (int64_t)tc * kTile : kTile);
            if (p.pieces_t) {  // 4 columns of 8 pieces per warp and step
#pragma unroll
                for (int step = 0; step < 2; ++step) {
                    const int col = step * 64 + warp * 4 + (lane >> 3), piece = lane & 7;
                    const uint2 a = *reinterpret_cast<const uint2*>(&sm.codes[k][piece_at(col, 2 * piece)]);
                    const uint2 b = *reinterpret_cast<const uint2*>(&sm.codes[k][piece_at(col, 2 * piece + 1)]);
                    if (col < there && piece * 16 < rows)
                        stg_stream(base + col * p.rows + piece * 16, make_uint4(a.x, a.y, b.x, b.y));
                }
            } else {  // a column per warp and step, 4 bytes of it per lane
#pragma unroll 1
                for (int col = warp; col < there; col += kWarps) {
                    uint8_t* const q = base + col * p.rows;
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(&sm.codes[k][piece_at(col, lane >> 1) + (lane & 1) * 4]);
                    const uint32_t before = __shfl_up_sync(0xFFFFFFFFu, w, 1);
                    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(q) & 3u);
                    if (rows == kTile && off + lane > 0) {
                        // the aligned word that starts `off` bytes before this lane's
                        if (lane > 0) *reinterpret_cast<uint32_t*>(q + lane * 4 - off) = __funnelshift_l(before, w, 8 * off);
                        if (lane == 0 || lane == 31)
#pragma unroll
                            for (int i = 0; i < 4; ++i)  // the first one's last bytes, the last one's first
                                if (lane == 0 ? i < 4 - (int)off : i >= 4 - (int)off) q[lane * 4 + i] = (uint8_t)(w >> (8 * i));
                    } else if (rows == kTile) {
                        *reinterpret_cast<uint32_t*>(q) = w;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (lane * 4 + i < rows) q[lane * 4 + i] = (uint8_t)(w >> (8 * i));
                    }
                }
            }
        }
    }
}

fp8_status_t run(const char* fn, const Backward& p, bool f32, int fmt, int act, cudaStream_t st) {
    const int64_t tiles = ((p.n + kTile - 1) / kTile) * ((p.rows + kTile - 1) / kTile);
    const int sms = sm_count();
    const auto go = [&](auto kernel) {
        return launch_smem(fn, kernel, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(kThreads), sizeof(Smem), st, p);
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
    constexpr int64_t kMost = (1ll << 31) - 256;
    if (rows > kMost || n > kMost) return fail(FP8_ERR_UNSUPPORTED, "%s: sizes must be below 2^31 - 256", fn);
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
    Backward p = {dh, gu, scale_inv_gu, rows, n, dgu, scale_inv_dgu, dgu_t, scale_inv_dgu_t, h_t, scale_inv_h_t};
    p.words_in = n % 4 == 0 && aligned(gu, 4) && aligned(dh, 4 * dtype_size(dtype));
    p.words_out = n % 4 == 0 && aligned(dgu, 4);
    p.pieces_t = rows % 16 == 0 && aligned16(dgu_t) && aligned16(h_t);
    return run(fn, p, dtype == FP8_DT_FP32, (int)fmt_grad, (int)act, static_cast<cudaStream_t>(stream));
}
