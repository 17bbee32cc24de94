// grad_clip.cu -- the global gradient norm over many tensors, and clipping.
//
// "Megatron FP8" §24 (the overhead around the FP8 step should stay small): all
// tensors share the launches, as in the grouped amax.  norm = sqrt(sum of
// squares over every element of every tensor), factor = min(1, max_norm /
// (norm + eps)), y = x * factor.
//
// Pass 1 reads every gradient once and stores one partial sum of squares per
// CTA (64 bits) in the stream's workspace; pass 2 reads them again, scales and
// stores.  Both are bound by HBM; there is no way around the second read once
// the gradients exceed L2, because the factor needs all of them.
#include "fp8q_device.cuh"
#include "fp8q_host.h"

namespace fp8q {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 8;                              // 16-byte loads in flight per thread
constexpr int kChunkBytes = kThreads * kLoads * 16;    // bytes of x of one chunk
constexpr int kMaxTensors = 4096;
constexpr int kFewPartials = 512;                      // folded by the clip's own CTAs up to here

// A launch's tensors, by value in the kernel parameters (29 KB for N = 1024).
template <int N>
struct Table {
    const uint8_t* x[N];
    uint8_t* y[N];
    int64_t n[N];
    int begin[N + 1];   // prefix sums of per-tensor chunk counts
    uint8_t kind[N];    // bit 0: x is fp32, bit 1: y is fp32, bit 2: 16-byte aligned
    int count;
};

template <int N>
__device__ __forceinline__ int find_tensor(const Table<N>& t, int chunk) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.begin[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float element(const uint8_t* x, bool f32, int64_t i) {
    return f32 ? reinterpret_cast<const float*>(x)[i]
               : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(x)[i] << 16);
}

// Sum of (x * s)^2 over the elements of [lo, hi) that this thread owns:
// 16-byte pieces (or single elements when unaligned) at a stride of kThreads.
// `any` collects the magnitude bits, so that a sum of zeros is told from one
// whose squares fell below the fp32 range.
template <bool SCALED>
__device__ __forceinline__ float squares(const uint8_t* x, bool f32, bool vec, int64_t lo, int64_t hi, float s, uint32_t* any) {
    float total = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t bits = 0;
    const auto fold = [&]() {
        total = __fadd_rn(total, __fadd_rn(__fadd_rn(acc[0], acc[1]), __fadd_rn(acc[2], acc[3])));
        acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
    };
    const auto add = [&](float v, int j) {
        if constexpr (SCALED) v = __fmul_rn(v, s);
        acc[j] = __fmaf_rn(v, v, acc[j]);
    };
    const int per = f32 ? 4 : 8;
    const int64_t last = vec ? lo + (hi - lo) / per * per : lo;  // lo is a multiple of per: chunks are
    for (int64_t base = lo + (int64_t)threadIdx.x * per; base < last; base += (int64_t)kThreads * kLoads * per) {
        uint4 v[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int64_t i = base + (int64_t)k * kThreads * per;
            v[k] = i < last ? ldg_stream(x + i * (f32 ? 4 : 2)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            bits |= (v[k].x | v[k].y) | (v[k].z | v[k].w);
            if (f32) {
                add(__uint_as_float(v[k].x), 0);
                add(__uint_as_float(v[k].y), 1);
                add(__uint_as_float(v[k].z), 2);
                add(__uint_as_float(v[k].w), 3);
            } else {
                add(bf16lo(v[k].x), 0);
                add(bf16hi(v[k].x), 1);
                add(bf16lo(v[k].y), 2);
                add(bf16hi(v[k].y), 3);
                add(bf16lo(v[k].z), 0);
                add(bf16hi(v[k].z), 1);
                add(bf16lo(v[k].w), 2);
                add(bf16hi(v[k].w), 3);
            }
        }
        fold();
    }
    for (int64_t i = last + threadIdx.x, step = 1; i < hi; i += 4 * kThreads, ++step) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = i + j * kThreads < hi ? element(x, f32, i + j * kThreads) : 0.0f;
            bits |= __float_as_uint(v);
            add(v, j);
        }
        if (step % 16 == 0) fold();
    }
    *any = bits & (f32 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
    fold();
    return total;
}

__device__ __forceinline__ double block_sum_f64(double v, double* smem) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    __syncthreads();
    if (lane == 0) smem[warp] = v;
    __syncthreads();
    v = lane < nw ? smem[lane] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Pass 1: one CTA per `reps` chunks, one 64-bit partial per CTA.
//
// A thread adds its squares in fp32: four sums of at most 16 values, then those
// sums one after another, at most reps of them.
// Squares leave the fp32 range for |x| above 2^63 and below 2^-63: where the
// thread's sum is not below 2^120, or is below 2^-100 with some x nonzero, it
// reads its elements again scaled by 2^-96 or 2^96, and the power of two is
// taken back in 64 bits.  An Inf or NaN among them stays one either way.
template <int N>
__global__ void __launch_bounds__(kThreads)
square_sum_kernel(const __grid_constant__ Table<N> t, int reps, double* __restrict__ parts) {
    pdl_begin();
    const int i = find_tensor(t, blockIdx.x);
    const bool f32 = t.kind[i] & 1, vec = t.kind[i] & 4;
    const int64_t per_chunk = (int64_t)(kChunkBytes / (f32 ? 4 : 2)) * reps;
    const int64_t lo = (int64_t)(blockIdx.x - t.begin[i]) * per_chunk;
    const int64_t hi = lo + per_chunk < t.n[i] ? lo + per_chunk : t.n[i];
    uint32_t any;
    const float sum = squares<false>(t.x[i], f32, vec, lo, hi, 1.0f, &any);
    double total = sum;
    const bool big = !(sum < 0x1p120f), small = sum < 0x1p-100f && any != 0;
    if (big || small) {
        const float again = squares<true>(t.x[i], f32, vec, lo, hi, big ? 0x1p-96f : 0x1p96f, &any);
        total = (double)again * (big ? 0x1p192 : 0x1p-192);
    }
    __shared__ double red[32];
    total = block_sum_f64(total, red);
    if (threadIdx.x == 0) parts[blockIdx.x] = total;
}

struct Clip {
    const double* parts;
    int nparts;
    float max_norm, eps;
    float* norm_out;   // nullable
    float* coef_out;   // nullable
    float* coef;       // the workspace's copy, for the clip kernel
};

// Norm and factor from the partials, by one CTA; every thread returns the
// factor.  A norm that is NaN or Inf gives the factor 1: the gradients stay as
// they are and the caller sees the norm (as a NaN or Inf amax gives scale 1).
__device__ __forceinline__ float norm_and_factor(const Clip& c, double* smem, float* norm) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < c.nparts; i += blockDim.x) sum = __dadd_rn(sum, c.parts[i]);
    sum = block_sum_f64(sum, smem);
    *norm = (float)sqrt(sum);
    if (!(*norm < __uint_as_float(0x7F800000u))) return 1.0f;
    const float f = __fdiv_rn(c.max_norm, __fadd_rn(*norm, c.eps));
    return f < 1.0f ? f : 1.0f;
}

__global__ void __launch_bounds__(1024) norm_finalize_kernel(const __grid_constant__ Clip c) {
    pdl_begin();
    __shared__ double red[32];
    float norm;
    const float f = norm_and_factor(c, red, &norm);
    if (threadIdx.x != 0) return;
    if (c.norm_out) *c.norm_out = norm;
    if (c.coef_out) *c.coef_out = f;
    *c.coef = f;
}

// One chunk of y = x * f.  An item is what one 16-byte side holds: 8 elements
// for BF16 to BF16, else 4; a warp's loads and stores are contiguous.
template <bool XF, bool YF>
__device__ __forceinline__ void scale_chunk(const uint8_t* x, uint8_t* y, int64_t lo, int64_t hi, float f) {
    constexpr int kPer = !XF && !YF ? 8 : 4, kItems = kChunkBytes / (XF ? 4 : 2) / kThreads / kPer;
    const int64_t last = lo + (hi - lo) / kPer * kPer;
#pragma unroll
    for (int h = 0; h < kItems; h += 8) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t i = lo + ((int64_t)(h + k) * kThreads + threadIdx.x) * kPer;
            if (i >= last) continue;
            if constexpr (XF) {
                v[k] = *reinterpret_cast<const uint4*>(x + i * 4);
            } else if constexpr (YF) {
                const uint2 w = *reinterpret_cast<const uint2*>(x + i * 2);
                v[k] = make_uint4(w.x << 16, w.x & 0xFFFF0000u, w.y << 16, w.y & 0xFFFF0000u);
            } else {
                v[k] = *reinterpret_cast<const uint4*>(x + i * 2);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t i = lo + ((int64_t)(h + k) * kThreads + threadIdx.x) * kPer;
            if (i >= last) continue;
            if constexpr (XF || YF) {
                const float2 a = fmul2_rn(__uint_as_float(v[k].x), __uint_as_float(v[k].y), f);
                const float2 b = fmul2_rn(__uint_as_float(v[k].z), __uint_as_float(v[k].w), f);
                if constexpr (YF)
                    stg_evict_first(y + i * 4, make_uint4(__float_as_uint(a.x), __float_as_uint(a.y),
                                                          __float_as_uint(b.x), __float_as_uint(b.y)));
                else
                    stg_stream(y + i * 2, make_uint2(f32x2_to_bf16x2(a.x, a.y), f32x2_to_bf16x2(b.x, b.y)));
            } else {
                const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 p = fmul2_rn(bf16lo(w[j]), bf16hi(w[j]), f);
                    o[j] = f32x2_to_bf16x2(p.x, p.y);
                }
                stg_evict_first(y + i * 2, make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
    const int64_t i = last + threadIdx.x;  // the tensor's last elements, fewer than one item
    if (i < hi) {
        const float v = __fmul_rn(element(x, XF, i), f);
        if constexpr (YF) reinterpret_cast<float*>(y)[i] = v;
        else reinterpret_cast<uint16_t*>(y)[i] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
    }
}

// Elements one by one, where x and y are not both 16-byte aligned (1.5e9 BF16 into fp32:
// 10.2 ms with the norm, aligned 1.8).
__device__ __forceinline__ void scale_elements(const uint8_t* x, bool xf, uint8_t* y, bool yf, int64_t lo, int64_t hi, float f) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
        const float v = __fmul_rn(element(x, xf, i), f);
        if (yf) reinterpret_cast<float*>(y)[i] = v;
        else reinterpret_cast<uint16_t*>(y)[i] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
    }
}

// Pass 2: one chunk per CTA, last chunk first, so that it starts on the part
// of the gradients that pass 1 left in L2.  FOLD: the CTA reduces the partials
// itself (CTA 0 writes norm and factor); otherwise the finalize kernel did.
// In place with factor 1 there is nothing to do.
template <int N, bool FOLD>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Table<N> t, const __grid_constant__ Clip c) {
    pdl_begin();
    float f;
    if constexpr (FOLD) {
        __shared__ double red[32];
        float norm;
        f = norm_and_factor(c, red, &norm);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            if (c.norm_out) *c.norm_out = norm;
            if (c.coef_out) *c.coef_out = f;
        }
    } else {
        f = *c.coef;
    }
    const int chunk = (int)(gridDim.x - 1 - blockIdx.x);
    const int i = find_tensor(t, chunk);
    const bool xf = t.kind[i] & 1, yf = t.kind[i] & 2, vec = t.kind[i] & 4;
    const uint8_t* x = t.x[i];
    uint8_t* y = t.y[i];
    if (f == 1.0f && x == y) return;
    const int64_t per_chunk = kChunkBytes / (xf ? 4 : 2);
    const int64_t lo = (int64_t)(chunk - t.begin[i]) * per_chunk;
    const int64_t hi = lo + per_chunk < t.n[i] ? lo + per_chunk : t.n[i];
    if (!vec) scale_elements(x, xf, y, yf, lo, hi, f);
    else if (xf) yf ? scale_chunk<true, true>(x, y, lo, hi, f) : scale_chunk<true, false>(x, y, lo, hi, f);
    else yf ? scale_chunk<false, true>(x, y, lo, hi, f) : scale_chunk<false, false>(x, y, lo, hi, f);
}

struct Tensors {
    int count;
    const void* const* xs;
    const int64_t* ns;
    const int* dtypes;
    void* const* ys;     // NULL: in place
    const int* y_dtypes;
};

fp8_status_t check(const char* fn, const Tensors& g, bool clip) {
    if (g.count < 1 || g.count > kMaxTensors)
        return fail(FP8_ERR_INVALID_ARG, "%s: count must be in [1, %d]", fn, kMaxTensors);
    if (g.xs == nullptr || g.ns == nullptr || g.dtypes == nullptr)
        return fail(FP8_ERR_INVALID_ARG, "%s: xs / ns / dtypes is NULL", fn);
    if (clip && (g.ys == nullptr) != (g.y_dtypes == nullptr))
        return fail(FP8_ERR_INVALID_ARG, "%s: ys and y_dtypes must both be set or both NULL", fn);
    for (int i = 0; i < g.count; ++i) {
        if (g.ns[i] < 0) return fail(FP8_ERR_INVALID_ARG, "%s: tensor %d has n < 0", fn, i);
        if (!valid_dtype(g.dtypes[i])) return fail(FP8_ERR_INVALID_ARG, "%s: tensor %d has an unknown dtype", fn, i);
        if (g.ys && !valid_dtype(g.y_dtypes[i]))
            return fail(FP8_ERR_INVALID_ARG, "%s: output %d has an unknown dtype", fn, i);
        if (g.ns[i] == 0) continue;
        if (g.xs[i] == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: tensor %d is NULL", fn, i);
        if (reinterpret_cast<uintptr_t>(g.xs[i]) % dtype_size(g.dtypes[i]) != 0)
            return fail(FP8_ERR_INVALID_ARG, "%s: tensor %d is not element-aligned", fn, i);
        if (g.ys == nullptr) continue;
        if (g.ys[i] == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: output %d is NULL", fn, i);
        if (reinterpret_cast<uintptr_t>(g.ys[i]) % dtype_size(g.y_dtypes[i]) != 0)
            return fail(FP8_ERR_INVALID_ARG, "%s: output %d is not element-aligned", fn, i);
        if (g.ys[i] == g.xs[i] && g.dtypes[i] != g.y_dtypes[i])
            return fail(FP8_ERR_UNSUPPORTED, "%s: output %d overlays its tensor in another type", fn, i);
    }
    return FP8_OK;
}

// Chunks of tensor i when a chunk holds `reps` base chunks.
int64_t chunks_of(const Tensors& g, int i, int64_t reps) {
    const int64_t per = (int64_t)(kChunkBytes / dtype_size(g.dtypes[i])) * reps;
    return (g.ns[i] + per - 1) / per;
}

// Launch `go(table, chunks)` over the nonempty tensors, as many per launch as
// fit its table and a grid.
template <int N, typename Go>
fp8_status_t for_tables(const char* fn, const Tensors& g, int64_t reps, Go go) {
    static thread_local Table<N> t;  // 29 KB: not on the stack
    int i = 0;
    while (i < g.count) {
        t.count = 0;
        t.begin[0] = 0;
        for (; i < g.count && t.count < N; ++i) {
            if (g.ns[i] == 0) continue;
            const int64_t chunks = chunks_of(g, i, reps);
            if (chunks > 0x3FFFFFFF) return fail(FP8_ERR_UNSUPPORTED, "%s: tensor %d is too large", fn, i);
            if (t.begin[t.count] + chunks > 0x7FFFFFFFll) break;
            const int k = t.count++;
            const void* y = g.ys ? g.ys[i] : g.xs[i];
            t.x[k] = static_cast<const uint8_t*>(g.xs[i]);
            t.y[k] = static_cast<uint8_t*>(const_cast<void*>(y));
            t.n[k] = g.ns[i];
            t.begin[k + 1] = t.begin[k] + (int)chunks;
            const int yd = g.ys ? g.y_dtypes[i] : g.dtypes[i];
            t.kind[k] = (uint8_t)((g.dtypes[i] == FP8_DT_FP32 ? 1 : 0) | (yd == FP8_DT_FP32 ? 2 : 0) |
                                  (aligned16(g.xs[i]) && aligned16(y) ? 4 : 0));
        }
        if (t.count == 0) break;
        const fp8_status_t s = go(t, t.begin[t.count]);
        if (s != FP8_OK) return s;
    }
    return FP8_OK;
}

template <int N>
fp8_status_t run(const char* fn, const Tensors& g, bool clip, Clip c, cudaStream_t st) {
    fp8_status_t s = FP8_OK;
    StreamUse use(st);
    Workspace* ws = use.workspace(&s);
    if (!ws) return s;
    double* parts = reinterpret_cast<double*>(ws->sat);
    c.parts = parts;
    c.coef = ws->scratch;
    // About 16 CTAs per SM once there is work for more of them: the 64-bit block sum at
    // a CTA's end costs as much as a third of a chunk's reads (4 x 67 MB, one chunk per
    // CTA: 53 us, 5.1 TB/s).  Every tensor rounds its chunk count up, so that there are
    // at most total / reps + count partials.
    int64_t total = 0, reps = 1;
    for (int i = 0; i < g.count; ++i) total += chunks_of(g, i, 1);
    if (total > 16 * sm_count()) reps = total / (16 * sm_count());
    if (total / reps + g.count > kMaxPartials) reps = (total + (kMaxPartials - g.count) - 1) / (kMaxPartials - g.count);
    if (reps > 0x7FFFFFFF) return fail(FP8_ERR_UNSUPPORTED, "%s: too many elements", fn);
    int done = 0;
    s = for_tables<N>(fn, g, reps, [&](const Table<N>& t, int chunks) {
        const fp8_status_t r = launch(fn, square_sum_kernel<N>, dim3(chunks), dim3(kThreads), st, t, (int)reps, parts + done);
        done += chunks;
        return r;
    });
    if (s != FP8_OK) return s;
    c.nparts = done;
    const bool fold = clip && done > 0 && done <= kFewPartials && g.count <= N;
    if (!fold) {
        s = launch(fn, norm_finalize_kernel, dim3(1), dim3(1024), st, c);
        if (s != FP8_OK || !clip) return s;
    }
    return for_tables<N>(fn, g, 1, [&](const Table<N>& t, int chunks) {
        return fold ? launch(fn, clip_kernel<N, true>, dim3(chunks), dim3(kThreads), st, t, c)
                    : launch(fn, clip_kernel<N, false>, dim3(chunks), dim3(kThreads), st, t, c);
    });
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8_status_t fp8_grad_norm_grouped(int count, const void* const* xs, const int64_t* ns, const int* dtypes,
                                              float* norm_out, void* stream) {
    const char* fn = "fp8_grad_norm_grouped";
    const Tensors g = {count, xs, ns, dtypes, nullptr, nullptr};
    const fp8_status_t s = check(fn, g, false);
    if (s != FP8_OK) return s;
    if (norm_out == nullptr) return fail(FP8_ERR_INVALID_ARG, "%s: norm_out is NULL", fn);
    if (reinterpret_cast<uintptr_t>(norm_out) & 3u) return fail(FP8_ERR_INVALID_ARG, "%s: norm_out not 4-byte aligned", fn);
    Clip c = {};
    c.max_norm = 1.0f;
    c.norm_out = norm_out;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return count <= 128 ? run<128>(fn, g, false, c, st) : run<1024>(fn, g, false, c, st);
}

extern "C" fp8_status_t fp8_grad_clip_grouped(int count, const void* const* xs, const int64_t* ns, const int* dtypes,
                                              void* const* ys, const int* y_dtypes, float max_norm, float eps,
                                              float* norm_out, float* coef_out, void* stream) {
    const char* fn = "fp8_grad_clip_grouped";
    const Tensors g = {count, xs, ns, dtypes, ys, y_dtypes};
    const fp8_status_t s = check(fn, g, true);
    if (s != FP8_OK) return s;
    if (!(max_norm >= 0.0f) || !(max_norm <= 3.402823466e+38f))
        return fail(FP8_ERR_INVALID_ARG, "%s: max_norm must be finite and not negative", fn);
    if (!(eps >= 0.0f) || !(eps <= 3.402823466e+38f))
        return fail(FP8_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    if ((reinterpret_cast<uintptr_t>(norm_out) & 3u) || (reinterpret_cast<uintptr_t>(coef_out) & 3u))
        return fail(FP8_ERR_INVALID_ARG, "%s: norm_out / coef_out not 4-byte aligned", fn);
    Clip c = {};
    c.max_norm = max_norm;
    c.eps = eps;
    c.norm_out = norm_out;
    c.coef_out = coef_out;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return count <= 128 ? run<128>(fn, g, true, c, st) : run<1024>(fn, g, true, c, st);
}
