// gated.cuh -- the gated activation h = act(g) * u of a feed-forward block, its
// derivative, and the E4M3 tiles that its kernels write.
//
//   act(g)  = g * s,  s = 1 / (1 + exp(-y))      SiLU: y = g
//   act'(g) = s + act(g) * (1 - s) * y'          GELU (tanh form, 0.5 g (1 + tanh z) with
//                                                z = c (g + 0.044715 g^3)): y = 2 z
// Both are one sigmoid, so one exponential and one reciprocal per element.
#pragma once

#include "fp8q_device.cuh"
#include "fp8q_tcgen05.cuh"

namespace fp8q {

constexpr int kSilu = FP8_ACT_SILU, kGeluTanh = FP8_ACT_GELU_TANH;

// The hardware's approximations, two units in the last place each.  Their
// argument is rounded up to four times (GELU's polynomial, the product with log2
// e), so that exp(-y) is off by up to (|y| + 1) * 2^-22 of its value: far below
// the FP8 step of what is written.
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Constants and their products are rounded once.
constexpr double kLog2E = 1.4426950408889634, kGeluTwoC = 1.5957691216057308 /* 2 sqrt(2 / pi) */, kGeluCube = 0.044715;
// Beyond it the sigmoid of GELU is 0 or 1, and g^2 stays finite (0 * Inf would make a NaN of 0).
constexpr float kGeluFar = 32.0f;

// s(g).
template <int ACT>
__device__ __forceinline__ float gate(float g) {
    float t;  // -y log2 e
    if constexpr (ACT == kSilu) {
        t = g * (float)-kLog2E;
    } else {
        const float c = fminf(fmaxf(g, -kGeluFar), kGeluFar), c2 = c * c;
        t = c * __fmaf_rn(c2, (float)(-kLog2E * kGeluTwoC * kGeluCube), (float)(-kLog2E * kGeluTwoC));
    }
    return rcp_approx(1.0f + exp2_approx(t));
}

// The same of two values as a packed pair, and y'(g) where DERIVATIVE (not set for SiLU, 1).
template <int ACT, bool DERIVATIVE>
__device__ __forceinline__ uint64_t gate2(uint64_t g, uint64_t* dy) {
    const auto both = [](double v) { return pack2((float)v, (float)v); };
    uint64_t t;
    if constexpr (ACT == kSilu) {
        t = mul2(g, both(-kLog2E));
    } else {
        const float2 v = unpack2(g);
        const uint64_t c = pack2(fminf(fmaxf(v.x, -kGeluFar), kGeluFar), fminf(fmaxf(v.y, -kGeluFar), kGeluFar)), c2 = mul2(c, c);
        t = mul2(c, fma2(c2, both(-kLog2E * kGeluTwoC * kGeluCube), both(-kLog2E * kGeluTwoC)));
        if constexpr (DERIVATIVE) *dy = fma2(c2, both(3.0 * kGeluTwoC * kGeluCube), both(kGeluTwoC));
    }
    const float2 x = unpack2(t), e = unpack2(add2(pack2(exp2_approx(x.x), exp2_approx(x.y)), both(1.0)));
    return pack2(rcp_approx(e.x), rcp_approx(e.y));
}

template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
    return g * gate<ACT>(g) * u;
}

// The same of two columns; the same values, and h the same bits, as gated().
template <int ACT>
__device__ __forceinline__ uint64_t gated2(uint64_t g, uint64_t u) {
    return mul2(mul2(g, gate2<ACT, false>(g, nullptr)), u);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// max(m, |a|, |b|), a NaN if any of them is one.
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

}  // namespace fp8q
