// sv_e4m3.cuh -- the cache's rows in 8 bits: e4m3 values with a power of two for each head.
//
// A slot's row is [Hkv][D] e4m3, then a byte for each head (the exponent e of its power of two, + 127), then zeros
// up to a multiple of 16 bytes; what a value stands for is e4m3 * 2^e.  e is the smallest exponent with which the
// head's largest value is within e4m3's 448.  A power of two does for a floating-point format what any other scale
// would (e4m3's four digits are the same all over its range), and the products are exact in 16 bits: four digits
// times a power.  So a row that is read back, by whichever kernel, has the same values, and moving a row's bytes
// (accepted-path compaction) moves its scales.
#pragma once

#include "sv_ops.cuh"

namespace sv {

// Exponents end at 7, whatever the type: 2^(120 + e), by which the attention kernels bring a value's bits to bf16,
// is then a number, and values saturate at 448 * 2^7 = 57344, which fp16 holds.  They begin where 2^e is a normal
// fp32; in fp16 at -15, below which nothing is gained: e4m3's smallest step is then 2^-24, fp16's own.
constexpr int E4M3_HI = 7;
__host__ __device__ constexpr int e4m3_lo(bool bf16) { return bf16 ? -126 : -15; }

__host__ __device__ constexpr int64_t e4m3_row_bytes(int64_t Hkv, int64_t D) { return (Hkv * (D + 1) + 15) / 16 * 16; }

// The exponent for a largest magnitude of m (an infinity's is the highest).
__device__ __forceinline__ int e4m3_exponent(float m, bool bf16)
{
    const uint32_t bits = __float_as_uint(m);
    // m = f * 2^x with f in [1, 2): 448 * 2^e holds it from e = x - 8 on while f <= 1.75.
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
    return e < e4m3_lo(bf16) ? e4m3_lo(bf16) : e > E4M3_HI ? E4M3_HI : e;
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two values rounded to nearest even; those beyond 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pack(float lo, float hi)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// The two values of 16 bits, exactly, as fp16.
__device__ __forceinline__ uint32_t e4m3_half2(uint32_t bits)
{
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)bits));
    return d;
}

__device__ __forceinline__ float2 e4m3_unpack(uint32_t bits) { return Half2<false>::unpack(e4m3_half2(bits)); }

// Pairs of values (the low 16 bits) in 16 bits, times their head's power of two, from its byte: exact.
template <bool BF>
struct E4m3Scale;

template <>
struct E4m3Scale<true> {
    uint64_t f;
    __device__ __forceinline__ explicit E4m3Scale(int byte)
    {
        const float x = __uint_as_float((uint32_t)byte << 23);
        f = f2(x, x);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t bits) const
    {
        const float2 x = e4m3_unpack(bits), y = f2_split(f2_mul(f2(x.x, x.y), f));
        return Half2<true>::pack(y.x, y.y);
    }
};

// (2^e in two factors that fp16 holds, the first of them exact on every value: rounded once, where 2^e is below -15.)
template <>
struct E4m3Scale<false> {
    __half2 f, g;
    __device__ __forceinline__ explicit E4m3Scale(int byte)
    {
        const int e = byte - 127, a = e < -14 ? -14 : e > 15 ? 15 : e, b = e - a < -24 ? -25 : e - a > 15 ? 15 : e - a;
        f = __float2half2_rn(exp2_int(a));
        g = __float2half2_rn(exp2_int(b));
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t bits) const
    {
        const uint32_t h = e4m3_half2(bits);
        const __half2 y = __hmul2(__hmul2(*reinterpret_cast<const __half2 *>(&h), f), g);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
};

}  // namespace sv
