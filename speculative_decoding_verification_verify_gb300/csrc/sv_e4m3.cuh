// sv_e4m3.cuh -- the cache's rows in 8 bits: e4m3 values with a power of two for each head.
//
// A slot's row is [Hkv][D] e4m3, then a byte for each head (the exponent e of its power of two, + 127), then zeros
// up to a multiple of 16 bytes; what a value stands for is e4m3 * 2^e.  e is the smallest exponent with which the
// head's largest value is within e4m3's 448.  A power of two does for a floating-point format what any other scale
// would (e4m3's four digits are the same all over its range), and the products are exact in 16 bits: four digits
// times a power.  (But for bf16's subnormals, below 2^-126, of heads that are smaller than 2^-116 throughout: the digits
// that they lack are cut off.)  So a row that is read back, by whichever kernel, has the same values, and moving a row's
// bytes (accepted-path compaction) moves its scales.
#pragma once

#include "sv_ops.cuh"

namespace sv {

// Exponents end at 7, whatever the type: values saturate at 448 * 2^7 = 57344, the largest of them that fp16 holds, and
// one limit serves both types (bf16's larger values are lost by it).  They begin where 2^e is a normal fp32; in fp16
// at -15, below which nothing is gained: e4m3's smallest step is then 2^-24, fp16's own.
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

// Values in 16 bits, times their head's power of two: exact, NaN too.  128 values of a thread take 800 clocks of four
// warps in bf16, 380 in fp16, half of it the conversions at a quarter of the rate.  `bits` of a head are the factor in
// the type.  (Shifting the bits to where bf16 has them and one product is as many instructions, but knows no NaN.)
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

// NaN's bits, a row of them.
#define SV_NAN4 {0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu}
static __device__ const uint4 g_e4m3_nan[8] = {SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4, SV_NAN4};
#undef SV_NAN4

// A warpgroup's tiles of 128 rows, from the cache's 8-bit rows to 16-bit units in shared memory (128-byte swizzle,
// halves of 64 values).  Rows come by asynchronous copies into a ring of R tiles and are widened from there: a thread
// reads what it copied itself, so the ring needs no barriers, and R tiles are under way whatever the memory's latency.
// (Rows loaded to registers a tile ahead took 390 us where this takes 360, for one token of 64 requests over 8192
// positions.)  A warp has 32 rows of a tile, in ITER copies of RPI rows; a row's slot and power
// of two are one lane's.
template <bool BF, int DP, int R>
struct E4m3Feed {
    static constexpr int CPR = DP / 16, RPI = 32 / CPR, ITER = CPR;
    static constexpr int TILE_BYTES = 128 * DP + 128 * 4;  // a tile of the ring: rows, then a word with each row's power of two
    static constexpr int BYTES = R * TILE_BYTES;
    int own, sub, tid;  // the row whose slot the lane keeps, of a tile
    uint32_t to, ring;
    int offset;         // of the lane's chunk in a row; below 0: beyond the head
    bool full;          // no lane's is
    uint32_t shifts;    // where in their words the powers of two are, two bits for each tile under way, the oldest first

    // `warp` of the warpgroup, whose ring it is.  Eight lanes that store together have chunks of two rows: no bank twice.
    __device__ __forceinline__ E4m3Feed(uint32_t ring_at, int warp, int lane, int D) : tid(warp * 32 + lane), ring(ring_at), shifts(0)
    {
        const int chunk = DP == 128 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
        sub = DP == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane >> 2;
        own = warp * RPI + lane % RPI + 4 * RPI * (lane / RPI);
        const int first = warp * RPI + sub;
        to = (chunk >> 2) * 128 * 128 + first * 128 + (((2 * chunk & 7) ^ (first & 7)) << 4);
        offset = chunk * 16 < D ? chunk * 16 : -1;
        full = D == DP;
    }
    // The tile's row of the lane's i-th copy; where a list in the order of lanes' copies has a row, and the lane's first.
    __device__ __forceinline__ int row(int i) const { return (to >> 7 & 127) + 4 * RPI * i; }
    static __device__ __forceinline__ int place(int row) { return row % (4 * RPI) * ITER + row / (4 * RPI); }
    __device__ __forceinline__ int first() const { return (to >> 7 & 127) * ITER; }
    // The copies of a tile into place r, of rows whose slots are given: `whole` where all of the warp's 32 rows are
    // there, else below 0 where one is not (zeros; -2: NaN).  `cache` is where the head's values of slot 0 are.
    __device__ __forceinline__ void ask(int r, bool whole, const unsigned char *cache, uint32_t stride, const int (&slot)[ITER])
    {
        const uint32_t dst = ring + r * TILE_BYTES + tid * 16;
        if (whole && full) {
            const unsigned char *const at = cache + offset;
#pragma unroll
            for (int i = 0; i < ITER; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 2048), "l"(at + (uint64_t)(uint32_t)slot[i] * stride)
                             : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                const int s = slot[i];
                const unsigned char *at = s == -2 ? reinterpret_cast<const unsigned char *>(g_e4m3_nan)
                                                  : cache + (uint64_t)(uint32_t)(s < 0 ? 0 : s) * stride;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 2048), "l"(at + (offset < 0 ? 0 : offset)),
                             "r"(s != -1 && offset >= 0 ? 16 : 0)
                             : "memory");
            }
        }
    }
    // Its powers of two (`slot`: the lane's own row's, below 0 where it is not there), `at` bytes into a slot of `cache`, and
    // the end of its copies; `count`: tiles under way before it.
    __device__ __forceinline__ void asked(int r, int count, int slot, const unsigned char *cache, uint32_t stride, int at)
    {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ring + r * TILE_BYTES + 128 * DP + place(own) * 4),
                     "l"(cache + (at & ~3) + (uint64_t)(uint32_t)(slot < 0 ? 0 : slot) * stride), "r"(slot < 0 ? 0 : 4)
                     : "memory");
        shifts |= (uint32_t)(at & 3) << 2 * count;
        commit();
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // The oldest of the R tiles (or empty groups) is there.
    static __device__ __forceinline__ void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(R - 1) : "memory");
        __syncwarp();  // (the powers of two were copied by other lanes)
    }
    // A tile is read whole before it is stored: its place in the ring is free for the next copies meanwhile.
    struct Tile {
        uint4 w[ITER];
        uint32_t power[ITER];  // the words that have the rows' powers of two, at `shift`
        int shift;
    };
    // The tile in place r.  (Copies into it may follow once the warp's lanes are past this: a warp's accesses of shared
    // memory are carried out in their order, and a copy's write comes a trip to memory later.)
    __device__ __forceinline__ void read(int r, Tile &t)
    {
#pragma unroll
        for (int i = 0; i < ITER; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(t.power[i]), "=r"(t.power[i + 1]), "=r"(t.power[i + 2]), "=r"(t.power[i + 3])
                         : "r"(ring + r * TILE_BYTES + 128 * DP + (first() + i) * 4)
                         : "memory");
#pragma unroll
        for (int i = 0; i < ITER; ++i)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(t.w[i].x), "=r"(t.w[i].y), "=r"(t.w[i].z), "=r"(t.w[i].w)
                         : "r"(ring + r * TILE_BYTES + i * 2048 + tid * 16)
                         : "memory");
        t.shift = 8 * (shifts & 3);
        shifts >>= 2;
        __syncwarp();
    }
    __device__ __forceinline__ void write(uint32_t unit, const Tile &t)
    {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const E4m3Scale<BF> g(E4m3Scale<BF>::bits(t.power[i] >> t.shift & 0xff));
            const uint32_t at = unit + to + i * 4 * RPI * 128;
            const uint4 &w = t.w[i];
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(g(w.x)), "r"(g(w.x >> 16)), "r"(g(w.y)),
                         "r"(g(w.y >> 16))
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ 16), "r"(g(w.z)), "r"(g(w.z >> 16)), "r"(g(w.w)),
                         "r"(g(w.w >> 16))
                         : "memory");
        }
    }
};

}  // namespace sv
