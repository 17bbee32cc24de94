// fp8q_tcgen05.cuh -- the fifth-generation tensor core of sm_103a as the FP8
// products use it: descriptors, tcgen05 instructions for one CTA or a pair,
// cluster barriers and the waits around them.
//
// Operand tiles are 128 rows of 128 bytes in shared memory with the 128-byte
// swizzle (16-byte piece p of row r sits at piece p ^ (r % 8)); a tile is 16 KB
// and starts at a multiple of 1024 bytes.  A tile whose rows run along the
// contraction is "K-major"; one whose rows are contraction steps and whose
// bytes run along m or n is "MN-major".
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8q_pipeline.cuh"

namespace fp8q {

constexpr int kTileBytes = 128 * 128;

// ------------------------------------------------------------- descriptors

// Shared-memory matrix descriptor of such a tile: start address, leading
// dimension offset (the next 128 bytes of m or n of an MN-major tile: tiles
// follow one another; not used by a K-major one), stride offset 1024 (the next
// 8 rows), descriptor version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(kTileBytes >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}
// Advance of the start address (in 16-byte units) by 32 contraction steps:
// 32 bytes along a K-major row, 32 rows of an MN-major tile.
constexpr uint64_t kStepKMajor = 32 >> 4, kStepMnMajor = (32 * 128) >> 4;

// Instruction descriptor of kind::f8f6f4 with fp32 accumulators: element types
// (0 E4M3, 1 E5M2), whether A / B are MN-major, tile shape m x n.
__host__ __device__ inline uint32_t mma_desc(int fmt_a, int fmt_b, bool a_mn, bool b_mn, int m, int n) {
    return 1u << 4 | (uint32_t)fmt_a << 7 | (uint32_t)fmt_b << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// ------------------------------------------------------ cluster and barriers

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The same where only the meeting counts: the last one before the CTAs end.
// (A release would wait for the outputs' stores, about a microsecond.)
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}
// Address in the cluster's shared window of the same variable in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrival in any CTA of the cluster.  RELEASE orders this thread's writes before
// it; without, it orders only what tcgen05.fence::before_thread_sync did (a
// release waits for the thread's copies in flight, far longer than a block).
template <bool RELEASE>
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    if constexpr (RELEASE)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The expectation of a bulk copy: relaxed, since the bytes that it announces are
// not this thread's writes.  (With release semantics the arrival waited for the
// thread's earlier bulk copies: the pair's ring ran at 20 bytes per cycle and SM
// instead of more than 40.)
__device__ __forceinline__ void cluster_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// Waits give up after about two seconds; a thread whose wait did so polls each
// later barrier once only, so that the kernel always ends (its outputs are then
// incomplete, which fp8_wait_timeouts reports).  It issues no further copy or
// product and arrives on no barrier that copies report to: such a barrier holds
// 2^20 - 1 bytes, and no arrivals beyond its count while bytes are in flight.
struct Waiter {
    bool dead = false;

    template <bool CLUSTER>
    static __device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
        uint32_t done;
        if constexpr (CLUSTER)
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done)
                : "r"(bar), "r"(parity)
                : "memory");
        else
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done)
                : "r"(bar), "r"(parity)
                : "memory");
        return done != 0;
    }

    // The same without waiting at all: asked for early, used later.
    static __device__ __forceinline__ bool test(uint32_t bar, uint32_t parity) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        return done != 0;
    }

    // Polls for one limit's time; whether the phase completed.
    // CLUSTER: acquire what the other CTA's threads wrote before they arrived.
    template <bool CLUSTER = false>
    static __device__ __forceinline__ bool within_limit(uint32_t bar, uint32_t parity) {
        // Reading the timer takes longer than most waits do: not before many polls.
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (poll<CLUSTER>(bar, parity)) return true;
        const uint64_t t0 = global_ns();
#pragma unroll 1
        for (uint32_t i = 0; i < kMbarWaitMaxPolls; ++i) {
            if (poll<CLUSTER>(bar, parity)) return true;
            if ((i & 15) == 15 && global_ns() - t0 > kMbarWaitLimitNs) break;
        }
        return false;
    }

    template <bool CLUSTER = false>
    __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity) {
        if (poll<CLUSTER>(bar, parity) || dead) return;
        if (within_limit<CLUSTER>(bar, parity)) return;
        dead = true;
        atomicAdd(&g_wait_timeouts, 1ull);
    }
};

// A role whose wait gave up says so in `flag` (shared memory) of every CTA of its
// cluster before the CTAs meet for the last time: copies and products may then
// still be in flight, and the CTAs stay for another millisecond.
__device__ __forceinline__ void report_dead(uint32_t flag, int ctas) {
    for (int r = 0; r < ctas; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(flag, r)), "r"(1) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}
__device__ __forceinline__ void linger() {
    const uint64_t t0 = global_ns();
#pragma unroll 1
    for (uint32_t i = 0; i < (1u << 20) && global_ns() - t0 < 1000000ull; ++i) {
    }
}

// One thread of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// ------------------------------------------------------------------- tcgen05

template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
    if constexpr (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A * B for 32 contraction steps, by one thread.
template <int CTAS>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
            : "memory");
}

// Arrive on `bar` (in both CTAs of the pair when CTAS == 2) once every product
// this thread has issued is done.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    if constexpr (CTAS == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 columns of this warp's 32 lanes: lane l gets row l, r[j] column j.
__device__ __forceinline__ void tmem_ld_32x16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

// 64 columns of 16 of this warp's lanes (the 16 from `addr`'s lane on): lane l
// gets row l / 4 in r[4i], r[4i + 1] and row l / 4 + 8 in r[4i + 2], r[4i + 3],
// columns 8i + 2 (l % 4) and the one after it.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

// ---------------------------------------------------------------- tile loads

// Fetches a tensor map ahead of its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// One 128 x 128-byte tile at byte x, row y of matrix z by the bulk-copy engine;
// x a multiple of 16; what lies outside reads as zero.  PAIR: `bar` may be the
// other CTA's (an address of the cluster's shared window).
template <bool PAIR>
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

// Shared-memory writes of this thread become visible to the tensor core.
__device__ __forceinline__ void fence_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ----------------------------------------------------------- packed fp32 math

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace fp8q
