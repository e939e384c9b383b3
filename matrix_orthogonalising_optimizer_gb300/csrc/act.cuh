// Element formulas shared by the operators' kernels: the activations of the
// gated block and the exponential of the vocabulary loss.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "ops.h"

namespace dmuon {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// act(a) = a gate(a), act'(a) = gate + a gate'.  bf16 results take the
// approximate exponential and reciprocal (relative error about 2^-22, far
// below the storage rounding).
template <bool kF32>
__device__ __forceinline__ float act_gate(int act, float a) {
    if (act == OPS_SILU) {
        if (kF32) return 1.0f / (1.0f + expf(-a));
        return rcp_approx(1.0f + ex2(-a * kLog2e));
    }
    return 0.5f * erfcf(-a * 0.70710678118654752f);
}

template <bool kF32>
__device__ __forceinline__ float act_slope(int act, float a, float gate) {
    if (act == OPS_SILU) return gate * (1.0f + a * (1.0f - gate));
    const float pdf = 0.3989422804014327f * (kF32 ? expf(-0.5f * a * a) : ex2(-0.5f * kLog2e * a * a));
    return gate + a * pdf;
}

// What is subtracted from a block's logits before their exponentials are taken: the
// maximum m or, where there is no finite logit (m = -inf), 0, so that they are 0
// and not exp(-inf + inf).
__device__ __forceinline__ float exp_shift(float m) { return m == __int_as_float(0xff800000) ? 0.0f : m; }

// An exponential relative to its block's maximum, 0 <= e <= 1, in 16 bits: 5
// exponent and 11 mantissa bits of the fp32 value (relative error 2^-12), zero
// below 2^-31.  bf16 would round the probability once more, by 2^-8, before the
// gradient's own rounding.  (A NaN reaches the gradient through lse.)
constexpr uint32_t kE16Base = 96u << 11;  // exponent of 2^-31

__device__ __forceinline__ uint32_t e16_encode(float e) {
    const uint32_t b = (__float_as_uint(e) + 0x800u) >> 12;  // 8 + 11 bits, rounded half up
    return b <= kE16Base ? 0u : min(b - kE16Base, 0xffffu);
}

__device__ __forceinline__ float e16_decode(uint32_t c) {
    return c ? __uint_as_float((c + kE16Base) << 12) : 0.0f;
}

}  // namespace dmuon
