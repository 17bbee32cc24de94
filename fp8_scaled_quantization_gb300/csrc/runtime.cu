// runtime.cu -- status strings, per-thread error text, launch counting, SM
// count cache and the per-(device, stream) reduction workspace.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include <cudaTypedefs.h>

#include "fp8q_device.cuh"
#include "fp8q_host.h"

namespace fp8q {

namespace {
thread_local char g_last_error[512] = "";
std::atomic<unsigned long long> g_launches{0};

std::mutex g_mu;
std::map<int, int> g_sm_count;  // device -> SMs
}  // namespace

struct StreamMemory {
    std::recursive_mutex mu;
    Workspace* ws = nullptr;
    void* scratch = nullptr;        // in use
    size_t scratch_bytes = 0;
    bool scratch_captured = false;  // a graph may hold its address
    std::vector<void*> captured;    // outgrown, held by graphs
    std::vector<void*> outgrown;    // while the stream was being captured: freed by a later call
};

namespace {
std::map<std::pair<int, uintptr_t>, StreamMemory> g_streams;  // (device, stream); entries stay, for those who wait for one
}  // namespace

fp8_status_t fail(fp8_status_t st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return st;
}

fp8_status_t cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return FP8_OK;
    return fail(FP8_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

fp8_status_t after_launch(const char* kernel) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e, kernel);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return FP8_OK;
}

fp8_status_t allow_smem(const char* what, const void* kernel, size_t smem) {
    static std::map<std::pair<const void*, int>, size_t> allowed;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e, what);
    std::lock_guard<std::mutex> lk(g_mu);
    size_t& had = allowed[std::make_pair(kernel, dev)];
    if (had >= smem) return FP8_OK;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_status(e, what);
    had = smem;
    return FP8_OK;
}

int max_clusters(const void* kernel, int threads, size_t smem, int cluster) {
    if (smem > 48 * 1024 && allow_smem("max_clusters", kernel, smem) != FP8_OK) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
    (void)cudaGetLastError();
    return 0;
}

int sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = g_sm_count.find(dev);
    if (it != g_sm_count.end()) return it->second;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    g_sm_count[dev] = n;
    return n;
}

namespace {
// The driver's tensor-map encoder, reached through the runtime.
fp8_status_t tile_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* out) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    if (encode == nullptr) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || fn == nullptr)
            return fail(FP8_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    *out = encode;
    return FP8_OK;
}
}  // namespace

fp8_status_t encode_tile_map_u16(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows,
                                 int box_cols) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const fp8_status_t s = tile_map_encoder(&encode);
    if (s != FP8_OK) return s;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t elem_strides[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box,
                              elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FP8_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return FP8_OK;
}

fp8_status_t encode_tile_map_u8(CUtensorMap* map, const void* base, int64_t inner, int64_t stride, int64_t rows,
                                int64_t groups, int tile_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const fp8_status_t s = tile_map_encoder(&encode);
    if (s != FP8_OK) return s;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)groups};
    const cuuint64_t strides[2] = {(cuuint64_t)stride, (cuuint64_t)stride * (cuuint64_t)rows};
    const cuuint32_t box[3] = {128, (cuuint32_t)tile_rows, 1};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
                              elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FP8_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return FP8_OK;
}

fp8_status_t encode_out_map(CUtensorMap* map, void* base, bool f32, int64_t cols, int64_t rows, int64_t groups) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const fp8_status_t s = tile_map_encoder(&encode);
    if (s != FP8_OK) return s;
    const cuuint64_t row_bytes = (cuuint64_t)cols * (f32 ? 4 : 2);
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)groups};
    const cuuint64_t strides[2] = {row_bytes, row_bytes * (cuuint64_t)rows};
    const cuuint32_t box[3] = {f32 ? 32u : 64u, 32, 1};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    const CUresult r = encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
                              strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FP8_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return FP8_OK;
}

fp8_status_t encode_code_map(CUtensorMap* map, void* base, int64_t cols, int64_t groups, int64_t rows, int box_cols) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const fp8_status_t s = tile_map_encoder(&encode);
    if (s != FP8_OK) return s;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)groups, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)cols, (cuuint64_t)cols * (cuuint64_t)groups};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, 1, 32};
    const cuuint32_t elem_strides[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, elem_strides,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FP8_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return FP8_OK;
}

bool StreamUse::take(fp8_status_t* st) {
    *st = FP8_OK;
    if (held_ != nullptr) return true;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        *st = cuda_status(e, "cudaGetDevice");
        return false;
    }
    StreamMemory* m;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        m = &g_streams[std::make_pair(dev, reinterpret_cast<uintptr_t>(stream_))];
    }
    m->mu.lock();
    held_ = m;
    return true;
}

StreamUse::~StreamUse() {
    if (held_ != nullptr) held_->mu.unlock();
}

Workspace* StreamUse::workspace(fp8_status_t* st) {
    if (!take(st)) return nullptr;
    if (held_->ws != nullptr) return held_->ws;
    // First use on this stream.  Relax the thread's capture mode so that the
    // allocation is legal while a stream is being captured.  The partial slots
    // need no initial value: a launch writes every slot its finalize reads.
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    void* p = nullptr;
    const cudaError_t e = cudaMalloc(&p, sizeof(Workspace));
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) {
        *st = cuda_status(e, "cudaMalloc(workspace)");
        return nullptr;
    }
    held_->ws = static_cast<Workspace*>(p);
    return held_->ws;
}

void* StreamUse::scratch(size_t bytes, fp8_status_t* st) {
    if (!take(st)) return nullptr;
    StreamMemory& m = *held_;
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream_, &status);
    if (e != cudaSuccess) {
        cudaGetLastError();
        *st = cuda_status(e, "cudaStreamIsCapturing");
        return nullptr;
    }
    const bool capturing = status != cudaStreamCaptureStatusNone;
    if (m.scratch_bytes >= bytes) {
        m.scratch_captured |= capturing;
        return m.scratch;
    }
    // a quarter more than asked for, so that slowly growing requests do not allocate each time
    const size_t want = (bytes + bytes / 4 + 255) & ~(size_t)255;
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    // The smaller one goes first, in stream order (work that uses it is before it on the
    // stream), so that both need not fit at once.
    if (m.scratch != nullptr) {
        std::vector<void*>& to = m.scratch_captured ? m.captured : m.outgrown;
        to.push_back(m.scratch);
        m.scratch = nullptr;
        m.scratch_bytes = 0;
    }
    void* p = nullptr;
    if (capturing) {  // an allocation in stream order would become part of the graph
        e = cudaMalloc(&p, want);
    } else {
        for (; e == cudaSuccess && !m.outgrown.empty(); m.outgrown.pop_back()) e = cudaFreeAsync(m.outgrown.back(), stream_);
        if (e == cudaSuccess) e = cudaMallocAsync(&p, want, stream_);
    }
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) {
        cudaGetLastError();  // the failed allocation is reported here, not by a later launch
        *st = cuda_status(e, "allocation of scratch");
        return nullptr;
    }
    m.scratch = p;
    m.scratch_bytes = want;
    m.scratch_captured = capturing;
    return p;
}

}  // namespace fp8q

extern "C" {

const char* fp8_status_string(fp8_status_t status) {
    switch (status) {
        case FP8_OK: return "FP8_OK";
        case FP8_ERR_INVALID_ARG: return "FP8_ERR_INVALID_ARG";
        case FP8_ERR_UNSUPPORTED: return "FP8_ERR_UNSUPPORTED";
        case FP8_ERR_CUDA: return "FP8_ERR_CUDA";
    }
    return "FP8_ERR_UNKNOWN";
}

const char* fp8_last_error_message(void) { return fp8q::g_last_error; }

int fp8_version(void) { return (FP8Q_VERSION_MAJOR << 16) | FP8Q_VERSION_MINOR; }

unsigned long long fp8_launch_count(void) { return fp8q::g_launches.load(std::memory_order_relaxed); }

fp8_status_t fp8_wait_timeouts(unsigned long long* count) {
    using namespace fp8q;
    if (count == nullptr) return fail(FP8_ERR_INVALID_ARG, "fp8_wait_timeouts: count is NULL");
    fp8_status_t st = cuda_status(cudaDeviceSynchronize(), "fp8_wait_timeouts");
    unsigned long long pair = 0, stream = 0;
    if (st == FP8_OK) st = block_ct_wait_timeouts(count);
    if (st == FP8_OK) st = gemm_pair_wait_timeouts(&pair);
    if (st == FP8_OK) st = gemm_stream_wait_timeouts(&stream);
    if (st == FP8_OK) *count += pair + stream;
    return st;
}

fp8_status_t fp8_release_stream_workspace(void* stream) {
    using namespace fp8q;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_status(e, "fp8_release_stream_workspace: cudaGetDevice");
    StreamMemory* m = nullptr;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        const auto it = g_streams.find(std::make_pair(dev, reinterpret_cast<uintptr_t>(stream)));
        if (it != g_streams.end()) m = &it->second;
    }
    std::vector<void*> mine;
    bool graphs = false;
    if (m != nullptr) {
        std::lock_guard<std::recursive_mutex> lk(m->mu);  // after the calls that are being enqueued
        graphs = m->scratch_captured || !m->captured.empty();
        mine.swap(m->captured);
        mine.insert(mine.end(), m->outgrown.begin(), m->outgrown.end());
        m->outgrown.clear();
        if (m->scratch != nullptr) mine.push_back(m->scratch);
        m->scratch = nullptr;
        m->scratch_bytes = 0;
        m->scratch_captured = false;
        if (m->ws != nullptr) mine.push_back(m->ws);
        m->ws = nullptr;
    }
    if (mine.empty()) return FP8_OK;  // nothing was allocated for this stream
    // The stream's queued work may still use the memory, and graphs that run elsewhere.
    e = graphs ? cudaDeviceSynchronize() : cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    for (void* p : mine) {
        const cudaError_t f = cudaFree(p);
        if (e == cudaSuccess) e = f;
    }
    return cuda_status(e, "fp8_release_stream_workspace");
}

}  // extern "C"
