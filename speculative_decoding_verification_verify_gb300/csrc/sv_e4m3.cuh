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

// Values in 16 bits, times their head's power of two: exact, NaN too.  `bits` of a head are the factor in the type.  (Shifting the bits to where bf16 has them and one product is as many instructions, but knows no NaN.)
template <bool BF>
struct E4m3Scale;

template <>
struct E4m3Scale<true> {
    uint64_t f;
    static __device__ __forceinline__ uint16_t bits(int byte) { return (uint16_t)(byte << 7); }
    __device__ __forceinline__ explicit E4m3Scale(uint16_t bits)
    {
        const float x = __uint_as_float((uint32_t)bits << 16);
        f = f2(x, x);
    }
    // Two values, of the low 16 bits.  (The product's low half is zeros: four digits.  bf16's subnormals lose some.)
    __device__ __forceinline__ uint32_t operator()(uint32_t two) const
    {
        const float2 x = e4m3_unpack(two), y = f2_split(f2_mul(f2(x.x, x.y), f));
        return __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
    }
};

// (2^e is a number of fp16, subnormal below -14, for all exponents that append writes from fp16.)
template <>
struct E4m3Scale<false> {
    __half2 f;
    static __device__ __forceinline__ uint16_t bits(int byte)
    {
        return __half_as_ushort(__float2half_rn(__uint_as_float((uint32_t)byte << 23)));
    }
    __device__ __forceinline__ explicit E4m3Scale(uint16_t bits) { f = __half2half2(__ushort_as_half(bits)); }
    __device__ __forceinline__ uint32_t operator()(uint32_t two) const
    {
        const uint32_t h = e4m3_half2(two);
        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), f);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
};

// What a lane reads where a row is not there: zeros, or NaN.
#define SV_NAN4 {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu}
static __device__ const uint4 g_e4m3_none[2][8] = {{}, {SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4}};
#undef SV_NAN4
__device__ __forceinline__ const unsigned char *e4m3_none(bool nan) { return reinterpret_cast<const unsigned char *>(g_e4m3_none[nan]); }

// A warpgroup's tiles of 128 rows from 8-bit rows to 16-bit units in shared memory (128-byte swizzle, halves of 64
// values), through registers.  A warp has 32 rows of a tile, in ITER loads of RPI rows; each row's address and power
// of two are worked out by one lane, and come to the lanes that read it through shared memory: a load is then two
// additions.  (With a shuffle and a test for each, a tile's widening took half as long again.)
template <bool BF, int DP>
struct E4m3Feed {
    static constexpr int CPR = DP / 16, RPI = 32 / CPR, ITER = CPR;
    struct __align__(16) Smem {
        const unsigned char *row[2][RPI][ITER];
        uint16_t scale[2][RPI][ITER];
    };
    Smem &sm;
    int own, sub, mine_sub, mine_i;  // the row whose slot the lane keeps, of a warp's tile; its place
    uint32_t to;
    int offset;  // of the lane's chunk in a row; below 0: beyond the head
    uint4 raw[ITER];

    // `warp` of the warpgroup.  Eight lanes that store together have chunks of two rows: no bank twice.
    __device__ __forceinline__ E4m3Feed(void *s, int warp, int lane, int D) : sm(*static_cast<Smem *>(s))
    {
        const int chunk = DP == 128 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
        sub = DP == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane >> 2;
        mine_sub = lane % RPI;
        mine_i = lane / RPI;
        own = warp * RPI + mine_sub + 4 * RPI * mine_i;
        const int first = warp * RPI + sub;
        to = (chunk >> 2) * 128 * 128 + first * 128 + (((2 * chunk & 7) ^ (first & 7)) << 4);
        offset = chunk * 16 < D ? chunk * 16 : -1;
    }
    // The address of the lane's own row of a tile in buffer b: a head's values; its power of two.
    __device__ __forceinline__ void put_row(int b, const unsigned char *at) { sm.row[b][mine_sub][mine_i] = at; }
    __device__ __forceinline__ void put_scale(int b, int byte) { sm.scale[b][mine_sub][mine_i] = E4m3Scale<BF>::bits(byte); }
    __device__ __forceinline__ void load(int b, int i)
    {
        const unsigned char *at = sm.row[b][sub][i];
        const unsigned char *const p = offset < 0 ? e4m3_none(false) : at + offset;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                     : "l"(p));
    }
    __device__ __forceinline__ void load_all(int b)
    {
#pragma unroll
        for (int i = 0; i < ITER; ++i) load(b, i);
    }
    // The loaded rows, with buffer b's powers of two, to a unit; where `more`, the rows of buffer `next` are asked for.
    __device__ __forceinline__ void widen(uint32_t unit, int b, bool more, int next)
    {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const uint4 w = raw[i];
            const E4m3Scale<BF> f(sm.scale[b][sub][i]);
            if (more) load(next, i);
            const uint32_t at = unit + to + i * 4 * RPI * 128;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(f(w.x)), "r"(f(w.x >> 16)), "r"(f(w.y)),
                         "r"(f(w.y >> 16))
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ 16), "r"(f(w.z)), "r"(f(w.z >> 16)), "r"(f(w.w)),
                         "r"(f(w.w >> 16))
                         : "memory");
        }
    }
};

// What a warp of it has in shared memory; nothing in a kernel of 16-bit rows.
template <bool BF, int DP, bool E4>
struct E4m3FeedSmem {
    using type = typename E4m3Feed<BF, DP>::Smem;
};
template <bool BF, int DP>
struct E4m3FeedSmem<BF, DP, false> {
    struct type {};
};

}  // namespace sv
