// sv_reference.cuh -- the references of the attention kernels' running softmax.
//
// A sum whose reference, a score, is r has weights 2^(s * scale + add) with add = lift - r * scale rounded once, while
// |add| is below FAR: one fused operation for an exponent, and the rounding is the same for all of a sum's weights.  From
// FAR on it would be whole exponents, and weights are 2^((s - r) * scale + lift), of the difference of two scores.  What
// takes a sum from one reference to another follows the same rule, so that it is never a difference of two products
// that have lost their digits (at a scale of 1, scores of 2^24 and 2^24 + 4 in two tiles had a ratio of 2^-4 instead of
// e^-4), nor of two that have passed fp32.
#pragma once

#include "sv_ops.cuh"

namespace sv {

constexpr float FAR = 0x1p24f;

// log2 of the reference's weight: fp16 keeps a long tail of small weights below 2^15 (sv_attention.cuh).
__host__ __device__ constexpr float lift(bool bf16) { return bf16 ? 0.f : 7.f; }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What is added to a score times the scale (log2(e) in it).
template <bool BF>
__device__ __forceinline__ float reference_add(float ref, float scale)
{
    return ref == -INFINITY ? 0.f : fmaf(-ref, scale, lift(BF));
}

// The factor that takes a sum from reference `old` to `now`, which is no lower (`was`, `is`: what they add).
template <bool BF>
__device__ __forceinline__ float reference_factor(float old, float was, float now, float is, float scale)
{
    if (old == now) return 1.f;
    if (old == -INFINITY) return 0.f;
    float x = is - was;
    const bool far0 = fabsf(was) >= FAR, far1 = fabsf(is) >= FAR;
    if (far0 || far1)
        x = far0 && far1 ? (old - now) * scale : far1 ? fmaf(-now, scale, -was) + lift(BF) : fmaf(old, scale, is) - lift(BF);
    return ex2(x);
}

template <bool BF>
__device__ __forceinline__ float reference_factor(float old, float now, float scale)
{
    return reference_factor<BF>(old, reference_add<BF>(old, scale), now, reference_add<BF>(now, scale), scale);
}

}  // namespace sv
