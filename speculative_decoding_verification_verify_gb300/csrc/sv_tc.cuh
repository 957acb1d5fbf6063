// sv_tc.cuh -- the asynchronous machinery of the tensor-core attention kernel: mbarriers with bounded
// waits, tcgen05 matrix products and their operand descriptors.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ---------------------------------------------------------------------------------------------
// mbarriers.  Every wait ends: when a phase has not completed within WAIT_CLOCKS the waiting thread
// raises the CTA's abort word, on which all other waits of the CTA give up too.
// ---------------------------------------------------------------------------------------------
constexpr int64_t WAIT_CLOCKS = 1000000000;  // about half a second

// The limit of waits for other warps, copies and products; what a CTA waits for before it ends after that, its own
// copies and products in flight, has WAIT_CLOCKS always.  In debug builds a test can lower it
// (spec_verify_debug_wait_clocks); below 0 a wait that is not over at the first look runs out.
#ifdef SV_DEBUG
static __device__ long long g_wait_clocks = WAIT_CLOCKS;
__device__ __forceinline__ int64_t wait_clocks() { return *(volatile long long *)&g_wait_clocks; }
#else
__device__ __forceinline__ constexpr int64_t wait_clocks() { return WAIT_CLOCKS; }
#endif
static __device__ unsigned long long g_timeouts;  // CTAs in which a wait ran out (spec_verify_wait_timeouts)

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Whether the phase of this parity has completed, without waiting.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}

// True once the phase of this parity has completed; false when the wait, or another of the CTA,
// ran out of time.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *abort)
{
#ifdef SV_DEBUG
    if (wait_clocks() < 0) {
        if (bar_test(bar, parity)) return true;
        *abort = 1;
        return false;
    }
#endif
    if (bar_try(bar, parity)) return true;
    const int64_t t0 = clock64();
    while (!bar_try(bar, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > wait_clocks()) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------------------------------------
// tcgen05.
// ---------------------------------------------------------------------------------------------
// One lane of a whole warp.  The lane that issues products is chosen this way: under a test of its
// index instead the compiler does not know that it is alone, and eight products and two commits took
// 465 clocks instead of 335.
__device__ __forceinline__ bool elect()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p;
}

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Values loaded before this are not to be used above it, which the operands tell the compiler.
template <int C>
__device__ __forceinline__ void wait_ld(float (&v)[C])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < C; i += 8)
        asm volatile(""
                     : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]), "+f"(v[i + 6]),
                       "+f"(v[i + 7]));
}

__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The mbarrier arrives once when all the products this thread issued before have completed.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Operand in shared memory under the 128-byte swizzle.  Rows of 128 bytes, groups of eight rows
// `sbo` bytes apart; when the contiguous direction is M or N, blocks of 64 elements of it `lbo`
// bytes apart.  (Under the 64-byte swizzle rows of 64 bytes, blocks of 32 elements.)
//
// A product by its descriptors' low words; the high ones are constants of the layouts.  (Fewer registers to be moved for
// each product: the first eight and two commits take 416 clocks against 675.)
__host__ __device__ constexpr uint32_t desc_high(uint32_t sbo, bool swizzle64 = false) { return sbo >> 4 | 1u << 14 | (swizzle64 ? 4u : 2u) << 29; }
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return (addr & 0x3ffff) >> 4 | (lbo >> 4) << 16; }
template <uint32_t HIGH_A, uint32_t HIGH_B>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %6};\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(HIGH_A), "n"(HIGH_B)
        : "memory");
}

// fp32 accumulators, A and B of one 16-bit type; *_mn: contiguous along M / N instead of K.
__device__ __forceinline__ constexpr uint32_t instr_desc(bool bf16, bool a_mn, bool b_mn, int m, int n)
{
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// One lane's values of 8 or 16 consecutive accumulator columns.
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st(uint32_t addr, const float (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(addr));
}

// 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}

// The product with A in TMEM: a row per lane, two 16-bit values per column.
template <uint32_t HIGH_B>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(HIGH_B)
        : "memory");
}

// Host: this module's count of timeouts, read and cleared, and its limit of waits (debug builds).
[[maybe_unused]] static bool read_timeouts(unsigned long long &n)
{
    unsigned long long x = 0, z = 0;
    if (cudaMemcpyFromSymbol(&x, g_timeouts, sizeof x) != cudaSuccess || cudaMemcpyToSymbol(g_timeouts, &z, sizeof z) != cudaSuccess)
        return false;
    n += x;
    return true;
}

[[maybe_unused]] static bool set_wait_clocks([[maybe_unused]] long long clocks)
{
#ifdef SV_DEBUG
    return cudaMemcpyToSymbol(g_wait_clocks, &clocks, sizeof clocks) == cudaSuccess;
#else
    return false;
#endif
}

}  // namespace tc
