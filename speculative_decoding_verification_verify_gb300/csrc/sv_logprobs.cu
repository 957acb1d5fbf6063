// sv_logprobs.cu -- what is answered beside emitted tokens: the token's log probability, its rank,
// the distribution's entropy and its most likely alternatives, in one pass over the logits.
//
//   t = x c - m, c = log2(e) / T, Z = sum 2^t, S = sum t 2^t     (m: a reference near the maximum of x c)
//   logprob = ln 2 (t_tok - log2 Z), entropy = ln 2 (log2 Z - S / Z), rank = 1 + #{x > x_tok}
//
// Reading the rows once bounds it.  The rows that have a token are cut into tiles of NT * VPT 16-byte
// vectors and every CTA takes an equal run of tiles, so few rows are spread over the GPU and absent
// ones cost nothing; where a run cuts a row, the CTA that finishes last joins its parts in order.
// One thread of a CTA streams its tiles through shared memory with bulk copies, STAGES of them in
// flight across rows' ends; loads into registers, a tile ahead, gave half the bandwidth.
//
// Threads keep (m, Z, S) of their own; m moves only when a tile passes it by more than 8.  It is kept
// as the rounded product x c, so that t is one fused operation and parts join without another rounding.
//
// Alternatives cost the fold one store per thread and tile: its maximum there, the maximum of a cell of VPT
// vectors.  When a row is folded, the `top`-th best of the warps' best lane maxima bounds its `top`-th best from
// below; only the cells that reach it, a few more than `top`, are read again (from L2) by one of two more
// warps, while the others are at the next rows.  (Looking for candidates while folding, behind a bound shared
// by the warps, took twice the fold's own time, in every form tried; with one finishing warp a row's end
// waited for the one before: 48.6 us against 38.1 for the 512 rows below.)
//
// Measured (GB300, copy rate 6.68 TB/s): 512 rows of 128256 bf16 logits, 20 alternatives, 35 us for 131 MB,
// 3.7 TB/s; 216 rows of 151936, 5 alternatives, 22 us for 66 MB; 4 rows of 128256 or 16 of 32003 in fp32 10 us.
// The stream itself runs at 95% of the copy rate; before it lie 4 us (entries counted and placed, the
// first tiles' way), after it 5 to 7 us (the last row's cells, its alternatives, the join where it is cut).
#include "sv_ops.cuh"
#include "sv_tc.cuh"

#include <mutex>

namespace svlp {

constexpr int NT = 256, NW = NT / 32;  // folding threads; one more warp copies, and two finish rows in turn
constexpr int NT_ALL = NT + 96;
constexpr int MAX_TOP = 32;
constexpr int VPT = 4;               // 16-byte vectors per thread and tile
constexpr int TILE_VEC = NT * VPT;
constexpr int STAGES = 4;
constexpr int CAP = 256;             // candidates the list holds
constexpr int FLY = 4;               // vectors that a finishing lane asks for at once; a bit for each of their logits
constexpr int SLOTS = 16;            // cells per thread and row; longer rows have cells of several tiles
static_assert(SLOTS * NT / 128 <= 32, "a bit for each of a lane's cells");
// Lane maxima of each warp that the bound comes from: 2 * top in all, so that a warp with more than its share of the
// best costs a few candidates only.
__device__ __forceinline__ int sample_of(int top) { return (2 * top + NW - 1) / NW; }
constexpr int SAMPLES = 2 * MAX_TOP;
constexpr int CTAS_PER_SM = 2;
constexpr int MAX_CTAS = 1024;
constexpr int ROWS = 128;            // rows of its run that a CTA lists at a time
constexpr float SLACK = 8.f;         // log2 of the largest term
constexpr float LEAST = -0x1.92p99f;  // about -1e30, a bf16 value; logits below it count as it: 2^t is 0 and t stays finite
constexpr float MOST_C = 1e8f, LEAST_C = 1e-26f;  // of log2(e) / T: LEAST c lies between -1e38 and -1e4
constexpr float NEG_INF = -__builtin_huge_valf(), LOWEST = -0x1.fffffep127f;

struct Params {
    const void *logits;
    const int32_t *tokens, *row_index;
    const float *temperatures;
    float temperature;
    int B, rows, T, V, top;
    float *logprobs, *entropy;
    int32_t *ranks, *top_ids;
    float *top_logprobs;
    int32_t *dev_status;
    int mis;       // logits base address mod 16, in elements
    int tpr;       // tiles per row
    unsigned *counters;
    unsigned char *parts;
};

struct Cand {
    float v;
    int i;
};
__device__ __forceinline__ bool better(float v, int i, float ov, int oi) { return v > ov || (v == ov && i < oi); }

// A part of a row: reference, sums, larger logits than the token's; its best, sorted.
struct __align__(16) Part {
    float m, z, s;
    int count;
    Cand top[MAX_TOP];
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fmax_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------------------------------------
// The two logit types: a 16-byte vector's maximum (NaN if it holds one), its values as pairs, how
// many exceed the token's logit.
// ---------------------------------------------------------------------------------------------
template <typename T>
struct Elt;

template <>
struct Elt<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static constexpr uint32_t NEG = 0xff80ff80u;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float load(const void *row, int64_t c)
    {
        return __uint_as_float((uint32_t)__ldg((const unsigned short *)row + c) << 16);
    }
    static __device__ __forceinline__ float vmax(const uint4 &w)
    {
        const uint32_t m = max2(max2(w.x, w.y), max2(w.z, w.w));
        return fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    // A bit for each logit that reaches the bound.
    static __device__ __forceinline__ unsigned reach(const uint4 &w, float bound)
    {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
        unsigned mask = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (__uint_as_float(a[i] << 16) >= bound) mask |= 1u << 2 * i;
            if (__uint_as_float(a[i] & 0xffff0000u) >= bound) mask |= 2u << 2 * i;
        }
        return mask;
    }
    static __device__ __forceinline__ float at(const uint4 *w, int e)
    {
        return __uint_as_float((uint32_t)reinterpret_cast<const unsigned short *>(w)[e] << 16);
    }
    static __device__ __forceinline__ void set(uint4 &w, int e, const void *row, int64_t c)
    {
        const uint32_t bits = __ldg((const unsigned short *)row + c);
        uint32_t &x = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
        x = e & 1 ? (x & 0xffffu) | bits << 16 : (x & 0xffff0000u) | bits;
    }
    static __device__ __forceinline__ void pairs(const uint4 &w, uint64_t (&x)[4])
    {
        const uint32_t least = 0xf149f149u;  // LEAST in bf16
        const uint32_t a[4] = {max2(w.x, least), max2(w.y, least), max2(w.z, least), max2(w.w, least)};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = sv::f2(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u));
    }
    // Counts of a pair add up in bf16, exact to 256: `acc` takes 4 per vector and half.
    struct Count {
        uint32_t tok, acc;
        int n;
        __device__ __forceinline__ void start(float x)
        {
            const uint32_t b = __float_as_uint(x) >> 16;
            tok = b | b << 16;
            acc = 0;
            n = 0;
        }
        __device__ __forceinline__ void add(const uint4 &w)
        {
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t g;
                asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(g) : "r"(a[i]), "r"(tok));
                asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(acc) : "r"(acc), "r"(g));
            }
        }
        __device__ __forceinline__ void tile_done()
        {
            n += (int)__uint_as_float(acc << 16) + (int)__uint_as_float(acc & 0xffff0000u);
            acc = 0;
        }
    };
};

template <>
struct Elt<float> {
    static constexpr int VEC = 4;
    static constexpr uint32_t NEG = 0xff800000u;
    static __device__ __forceinline__ float load(const void *row, int64_t c) { return __ldg((const float *)row + c); }
    static __device__ __forceinline__ float vmax(const uint4 &w)
    {
        return fmax_nan(fmax_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                        fmax_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
    static __device__ __forceinline__ unsigned reach(const uint4 &w, float bound)
    {
        return (__uint_as_float(w.x) >= bound ? 1u : 0u) | (__uint_as_float(w.y) >= bound ? 2u : 0u) |
               (__uint_as_float(w.z) >= bound ? 4u : 0u) | (__uint_as_float(w.w) >= bound ? 8u : 0u);
    }
    static __device__ __forceinline__ float at(const uint4 *w, int e) { return reinterpret_cast<const float *>(w)[e]; }
    static __device__ __forceinline__ void set(uint4 &w, int e, const void *row, int64_t c)
    {
        (e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w) = __ldg((const unsigned *)row + c);
    }
    static __device__ __forceinline__ void pairs(const uint4 &w, uint64_t (&x)[2])
    {
        x[0] = sv::f2(fmax_nan(__uint_as_float(w.x), LEAST), fmax_nan(__uint_as_float(w.y), LEAST));
        x[1] = sv::f2(fmax_nan(__uint_as_float(w.z), LEAST), fmax_nan(__uint_as_float(w.w), LEAST));
    }
    struct Count {
        float tok;
        int n;
        __device__ __forceinline__ void start(float x)
        {
            tok = x;
            n = 0;
        }
        __device__ __forceinline__ void add(const uint4 &w)
        {
            n += (__uint_as_float(w.x) > tok) + (__uint_as_float(w.y) > tok) + (__uint_as_float(w.z) > tok) +
                 (__uint_as_float(w.w) > tok);
        }
        __device__ __forceinline__ void tile_done() {}
    };
};

// An entry with a row to read.
struct Row {
    int64_t first;  // the row's first logit
    int r, tok;
    float temp, x;  // x: the token's logit
};

// What a row's warps share; two of them, so that the next row may begin before the last one is done.
struct Shared {
    __align__(16) float cell[SLOTS][NT];
    __align__(16) float best[SAMPLES];  // each warp's best lane maxima
    float m[NW], z[NW], s[NW];
    int count[NW];
};

// A finishing warp's.
struct Finish {
    uint4 vec[FLY][32];  // each lane's vectors
    int col[FLY][32];    // and their first columns
    Cand list[CAP + 32], top[MAX_TOP];
    int hit[CAP];
};

struct Smem {
    uint4 ring[STAGES][TILE_VEC];
    uint64_t full[STAGES], empty[STAGES], folded[2], freed[2];
    Shared row[2];
    Row rows[ROWS];
    Finish fin[2];
    int scan[NW];
    int abort;
};

// The best `top` of fin.list[0 .. n), sorted, into fin.top, by a warp.  A candidate's place is the number
// of better ones; their order in the list does not matter.
__device__ __forceinline__ void rank(Finish &fin, int n, int top)
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    fin.top[lane] = {NEG_INF, -1};
    __syncwarp();
    for (int e = lane; e < n; e += 32) {
        const Cand x = fin.list[e];
        int place = 0;
        for (int o = 0; o < n; ++o) place += better(fin.list[o].v, fin.list[o].i, x.v, x.i);
        if (place < top) fin.top[place] = x;
    }
    __syncwarp();
}

// The `top`-th best of the warps' best lane maxima, the greatest that `top` of them reach: at least `top` of
// the row's logits reach it.
__device__ __forceinline__ float bound_of(const Shared &sh, int top)
{
    const int lane = threadIdx.x & 31;
    const int n = NW * sample_of(top);
    const float y0 = lane < n ? sh.best[lane] : NEG_INF, y1 = 32 + lane < n ? sh.best[32 + lane] : NEG_INF;
    int p0 = 0, p1 = 0;
#pragma unroll 2
    for (int a = 0; a < n; a += 4) {
        const float4 o = *reinterpret_cast<const float4 *>(&sh.best[a]);
        p0 += (o.x >= y0) + (o.y >= y0) + (o.z >= y0) + (o.w >= y0);
        p1 += (o.x >= y1) + (o.y >= y1) + (o.z >= y1) + (o.w >= y1);
    }
    return warp_max(fmaxf(p0 >= top ? y0 : NEG_INF, p1 >= top ? y1 : NEG_INF));
}

// The candidates of columns [from, to) of a row whose list overflowed, read again by a warp, with the
// exact bound whenever the list is full.  They go from lower to higher tokens: one that equals the
// `top`-th best is no candidate, and once that is the row's maximum the search is over.
template <typename T>
__device__ __noinline__ void list_again(const Params &P, Finish &fin, const Row &w, int64_t from, int64_t to, int top, float most)
{
    const int lane = threadIdx.x & 31;
    const T *row = static_cast<const T *>(P.logits) + w.first;
    if (from < 0) from = 0;
    if (to > P.V) to = P.V;
    int n = 0;
    float bound = NEG_INF;  // NEG_INF is never a candidate
    for (int64_t c0 = from; c0 < to && bound < most; c0 += 32) {
        const float y = c0 + lane < to ? Elt<T>::load(row, c0 + lane) : NEG_INF;
        const unsigned in = __ballot_sync(0xffffffffu, y > bound);
        if ((in >> lane) & 1) fin.list[n + __popc(in & ((1u << lane) - 1))] = {y, (int)(c0 + lane)};
        n += __popc(in);
        if (n < CAP && !(n >= top && bound == NEG_INF)) continue;
        rank(fin, n, top);
        fin.list[lane] = fin.top[lane];
        bound = fin.top[top - 1].v;
        n = top;
        __syncwarp();
    }
    rank(fin, n, top);
}

// Quotients of tile counts: in 32 bits wherever they fit, for 64-bit division is a hundred instructions.
__device__ __noinline__ int64_t quotient64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return (uint64_t)(a | b) >> 32 ? quotient64(a, b) : (int64_t)((unsigned)a / (unsigned)b);
}
__device__ __forceinline__ int64_t run_begin(int c, int64_t total, int G) { return quotient(total * c, G); }
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int G) { return (int)quotient((x + 1) * G - 1, total); }

// Whether entry r has a row to read (0), nothing (-1), or a fault (a device status code).
__device__ __forceinline__ int fault_of(const Params &P, int r)
{
    [[maybe_unused]] const int n = P.B * P.T;
    const int tok = SV_INB(r, n, 1201) ? P.tokens[r] : -1;
    const int idx = P.row_index ? (SV_INB(r, n, 1202) ? P.row_index[r] : -1) : 0;
    const int b = (int)((unsigned)r / (unsigned)P.T);
    const float temp = P.temperatures && SV_INB(b, P.B, 1203) ? P.temperatures[b] : 1.f;
    if (tok < -1 || tok >= P.V) return SPEC_VERIFY_DEV_BAD_TOKEN;
    if (idx < -1 || idx >= P.rows) return SPEC_VERIFY_DEV_BAD_ROW;
    if (tok < 0 || idx < 0) return -1;
    return temp >= 0.f && temp < 3.4e38f ? 0 : SPEC_VERIFY_DEV_BAD_ROW;
}

// The sums of a row for which the fold's fused product does not hold, by a warp, with differences before the
// scale: a reference of such size is too coarse for the product (a row of nothing but finite masks; a
// temperature close to 0), LEAST times c has left fp32, or comes so near to 0 that masks have weight.
// 4 rows of 128256 at T = 1e-6 take 177 us in bf16 and 121 in fp32, against 35 and 50 at T = 1.  (Not called but
// in place: what a call has to keep across it cost every row's end, 35.8 against 35.3 us for the 512 rows above.)
template <typename T>
__device__ __forceinline__ float2 sums_again(const T *row, int V, float top1, float temp)
{
    constexpr int FLY = 16;  // loads of a lane in flight
    // log2(e) / T in two factors, so that no temperature takes it out of fp32.
    const float a = temp < 1e-30f ? 0x1p64f : 1.f, b = 1.44269504f / (temp * a);
    // One warp adds thousands of terms in a row, and equal ones are rounded the same way every time: what a
    // sum loses is carried along.
    float z = 0.f, s = 0.f, z_lost = 0.f, s_lost = 0.f;
    auto add = [](float &sum, float &lost, float x) {
        const float y = x - lost, now = sum + y;
        lost = (now - sum) - y;
        sum = now;
    };
    for (int i0 = threadIdx.x & 31; i0 < V; i0 += 32 * FLY) {
        float x[FLY], zb = 0.f, sb = 0.f;
#pragma unroll
        for (int f = 0; f < FLY; ++f) x[f] = i0 + 32 * f < V ? Elt<T>::load(row, i0 + 32 * f) : NEG_INF;
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
            const float t = (x[f] - top1) * a * b, e = ex2(t);
            zb += e;
            if (e > 0.f) sb += e * t;
        }
        add(z, z_lost, zb);
        add(s, s_lost, sb);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    return make_float2(z, s);
}

// The answers for a row's entry, by a warp; fin.top: its alternatives.
template <typename T>
__device__ __forceinline__ void answer(const Params &P, const Finish &fin, const Row &w, float m, float z, float s, int count)
{
    const int lane = threadIdx.x & 31;
    const int64_t r = w.r;
    const float temp = w.temp;
    const T *row = static_cast<const T *>(P.logits) + w.first;
    const float top1 = fin.top[0].v;
    const float c = 1.44269504f / temp;
    const bool low = fin.top[0].i >= 0 && !(fabsf(top1) * c < 1e7f && c < MOST_C && c > LEAST_C);
    if (__builtin_expect(low, 0)) {
        const float2 sums = sums_again<T>(row, P.V, top1, temp);
        z = sums.x;
        s = sums.y;
    }
    const bool bad = fin.top[0].i < 0 || !(z < __builtin_huge_valf());
    const float log_z = log2f(z);
    auto said = [&](float x) {
        if (low || x < LEAST) return (x - (low ? top1 : 0.f)) / temp - log_z * 0.69314718f;
        return (fmaf(x, c, -m) - log_z) * 0.69314718f;
    };
    if (lane == 0) {
        P.logprobs[r] = bad ? NAN : said(w.x);
        if (P.entropy) P.entropy[r] = bad ? NAN : fmaxf((log_z - s / z) * 0.69314718f, 0.f);
        if (P.ranks) P.ranks[r] = bad ? -1 : count + 1;
        if (bad && P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_BAD_ROW);
    }
    if (lane < P.top) {
        const Cand y = fin.top[lane];
        if (SV_INB(r * P.top + lane, (int64_t)P.B * P.T * P.top, 1204)) {
            P.top_ids[r * P.top + lane] = bad ? -1 : y.i;
            P.top_logprobs[r * P.top + lane] = bad ? NAN : y.i < 0 ? NEG_INF : said(y.v);
        }
    }
}

// A row, or its part in this CTA's run (tiles [j0, j1)), is folded: by a finishing warp.  A part goes
// to the workspace, and the warp that brings a row's last part joins them, in order.  CTAs c0 to c1 have
// the row's parts; first0: c0's run begins with it.
template <typename T>
__device__ __forceinline__ void finish(const Params &P, Finish &fin, const Shared &sh, const Row &w, int j0, int j1, int c0,
                                    int c1, bool first0, int top)
{
    const int lane = threadIdx.x & 31, cta = blockIdx.x;
    float M = lane < NW ? sh.m[lane] : NEG_INF;
    M = warp_max(M);
    float z = lane < NW ? sh.z[lane] : 0.f, s = 0.f;
    int n = lane < NW ? sh.count[lane] : 0;
    auto sum = [&] {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            s += __shfl_xor_sync(0xffffffffu, s, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
    };
    if (lane < NW && z != 0.f) {
        const float d = M - sh.m[lane], f = ex2(-d);
        s = f * fmaf(-d, z, sh.s[lane]);
        z *= f;
    }
    sum();
    // The logits that reach the bound, in the cells whose maxima do; then the best of them.
    using E = Elt<T>;
    const int head = (int)((unsigned)(w.first + P.mis) & (E::VEC - 1));
    const T *row = static_cast<const T *>(P.logits) + w.first;
    const float bound = fmaxf(bound_of(sh, top), LOWEST);  // -inf is no candidate
    const int step = (int)((unsigned)(j1 - j0 + SLOTS - 1) / SLOTS), slots = (int)((unsigned)(j1 - j0 + step - 1) / (unsigned)step);
    // A lane marks which of its fours of cells have one, then all list theirs in turn.
    unsigned mark = 0;
#pragma unroll 4
    for (int c = 0; c < slots * (NT / 128); ++c) {
        const float4 y = *reinterpret_cast<const float4 *>(&sh.cell[0][0] + c * 128 + lane * 4);
        if (fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w)) >= bound) mark |= 1u << c;
    }
    int hits = 0;
    for (; __any_sync(0xffffffffu, mark != 0); mark &= mark - 1) {
        const int four = (__ffs(mark) - 1) * 128 + lane * 4;
        float4 y = make_float4(NEG_INF, NEG_INF, NEG_INF, NEG_INF);
        if (mark) y = *reinterpret_cast<const float4 *>(&sh.cell[0][0] + four);
        const float a[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned in = __ballot_sync(0xffffffffu, a[i] >= bound);
            const int at = hits + __popc(in & ((1u << lane) - 1));
            if (a[i] >= bound && at < CAP) fin.hit[at] = four + i;
            hits += __popc(in);
        }
    }
    __syncwarp();
    // Their vectors, FLY per lane in flight: under the folding warps' streams a read takes a microsecond.
    // (What runs once per row is written to be short: its first run is bound by the fetching of its
    // instructions, at some ten clocks each.)
    int listed = hits > CAP ? CAP + 1 : 0;
    const int vecs = hits > CAP ? 0 : hits * step * VPT;
#pragma unroll 1
    for (int e0 = 0; e0 < vecs; e0 += 32 * FLY) {
#pragma unroll 1
        for (int f = 0; f < FLY && e0 + f * 32 + lane < vecs; ++f) {
            const unsigned e = e0 + f * 32 + lane, h = e / VPT, cell = fin.hit[step == 1 ? h : h / step];
            const int j = j0 + (int)(cell / NT) * step + (step == 1 ? 0 : (int)(h % step));
            const int64_t at = (int64_t)((((unsigned)j * VPT + e % VPT) * NT + cell % NT) * E::VEC) - head;
            fin.col[f][lane] = (int)at;
            if (j < j1 && at >= 0 && at + E::VEC <= P.V) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(&fin.vec[f][lane])), "l"(row + at)
                             : "memory");
            } else {
                uint4 x = make_uint4(E::NEG, E::NEG, E::NEG, E::NEG);
                for (int i = 0; i < E::VEC; ++i)
                    if (j < j1 && at + i >= 0 && at + i < P.V) E::set(x, i, row, at + i);
                fin.vec[f][lane] = x;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        unsigned mask = 0;
#pragma unroll 1
        for (int f = 0; f < FLY && e0 + f * 32 + lane < vecs; ++f) mask |= E::reach(fin.vec[f][lane], bound) << f * E::VEC;
        __syncwarp();
        // Each lane's next one, until no lane has any.
        for (unsigned in; (in = __ballot_sync(0xffffffffu, mask != 0)) != 0; mask &= mask - 1) {
            const int i = __ffs(mask) - 1, f = i / E::VEC, at = listed + __popc(in & ((1u << lane) - 1));
            if (mask && at < CAP) fin.list[at] = {E::at(&fin.vec[f][lane], i % E::VEC), fin.col[f][lane] + i % E::VEC};
            listed += __popc(in);
        }
    }
    __syncwarp();
    if (listed > CAP)
        list_again<T>(P, fin, w, (int64_t)j0 * TILE_VEC * E::VEC - head, (int64_t)j1 * TILE_VEC * E::VEC - head, top,
                      warp_max(lane < NW ? sh.best[lane * sample_of(top)] : NEG_INF));
    else
        rank(fin, listed, top);
    if (c0 == c1) {
        answer<T>(P, fin, w, M, z, s, n);
        return;
    }
    auto part_of = [&](int x) { return reinterpret_cast<Part *>(P.parts) + 2 * x + (x == c0 && !first0); };
    Part *part = part_of(cta);
    if (lane == 0) part->m = M, part->z = z, part->s = s, part->count = n;
    if (lane < top) part->top[lane] = fin.top[lane];
    __syncwarp();
    unsigned came = 0;
    if (lane == 0)
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(came) : "l"(&P.counters[c0]) : "memory");
    came = __shfl_sync(0xffffffffu, came, 0);
    __syncwarp();
    if (came != (unsigned)(c1 - c0)) return;
    if (lane == 0) P.counters[c0] = 0;
    // All of a round's reads are in flight together.
    constexpr int FLYP = 8;
    auto best_of = [&](int x) {
        return x <= c1 && lane < top ? __ldcg(reinterpret_cast<const int2 *>(&part_of(x)->top[lane])) : make_int2(0, -1);
    };
    int2 y[FLYP];
#pragma unroll
    for (int a = 0; a < FLYP; ++a) y[a] = best_of(c0 + a);
    M = NEG_INF;
    z = s = 0.f;
    n = 0;
    float floor_ = NEG_INF;  // `top` logits reach the largest of the parts' `top`-th best
    for (int x = c0 + lane; x <= c1; x += 32) {  // (a lane's parts in turn, if there are more than 32)
        const float4 p = __ldcg(reinterpret_cast<const float4 *>(part_of(x)));
        floor_ = fmaxf(floor_, __ldcg(&part_of(x)->top[top - 1].v));
        n += __float_as_int(p.w);
        if (p.y != 0.f) {
            const float now = fmaxf(M, p.x), f0 = ex2(M - now), f1 = ex2(p.x - now);
            s = (z == 0.f ? 0.f : f0 * fmaf(M - now, z, s)) + f1 * fmaf(p.x - now, p.y, p.z);
            z = (z == 0.f ? 0.f : f0 * z) + f1 * p.y;
            M = now;
        }
    }
    floor_ = warp_max(floor_);
    {
        const float own = M;
        M = warp_max(M);
        if (z != 0.f) {
            const float d = M - own, f = ex2(-d);
            s = f * fmaf(-d, z, s);
            z *= f;
        }
    }
    sum();
    int have = 0;
    for (int x0 = c0; x0 <= c1; x0 += FLYP) {
        if (x0 > c0)
#pragma unroll
            for (int a = 0; a < FLYP; ++a) y[a] = best_of(x0 + a);
#pragma unroll
        for (int a = 0; a < FLYP; ++a) {
            const unsigned in = __ballot_sync(0xffffffffu, y[a].y >= 0 && __int_as_float(y[a].x) >= floor_);
            if (!in) continue;
            if ((in >> lane) & 1) fin.list[have + __popc(in & ((1u << lane) - 1))] = {__int_as_float(y[a].x), y[a].y};
            have += __popc(in);
            if (have > CAP) {  // many equal logits
                rank(fin, have, top);
                if (lane < top) fin.list[lane] = fin.top[lane];
                have = top;
                __syncwarp();
            }
        }
    }
    rank(fin, have, top);
    answer<T>(P, fin, w, M, z, s, n);
}

template <typename T>
__global__ void __launch_bounds__(NT_ALL, CTAS_PER_SM) logprobs_kernel(const Params P)
{
    using E = Elt<T>;
    constexpr int VEC = E::VEC;
    extern __shared__ __align__(16) unsigned char smem[];
    Smem &sm = *reinterpret_cast<Smem *>(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const int top = P.top > 0 ? P.top : 1;  // the best one is the row's maximum
    volatile int *abort = &sm.abort;
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            tc::bar_init(tc::smem_u32(&sm.full[i]), 1);
            tc::bar_init(tc::smem_u32(&sm.empty[i]), NW);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_u32(&sm.folded[i]), NW);
            tc::bar_init(tc::smem_u32(&sm.freed[i]), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.abort = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The entries that have a row; what the others answer is written here, each by one CTA.
    const int R = P.B * P.T, per = (int)((unsigned)(R + NT - 1) / NT);
    const int r0 = tid * per, r1 = tid < NT ? min(r0 + per, R) : 0;  // the thread's
    int mine = 0;
    unsigned which = 0;  // of its first 32
    {
#pragma unroll 2
        for (int r = r0; r < r1; ++r) {
            const int code = fault_of(P, r);
            if (code == 0) {
                ++mine;
                if (r - r0 < 32) which |= 1u << (r - r0);
            } else if ((unsigned)r % gridDim.x == (unsigned)cta) {
                P.logprobs[r] = code > 0 ? NAN : 0.f;
                if (P.entropy) P.entropy[r] = code > 0 ? NAN : 0.f;
                if (P.ranks) P.ranks[r] = code > 0 ? -1 : 0;
#pragma unroll 1
                for (int k = 0; k < P.top; ++k) {
                    P.top_ids[(int64_t)r * P.top + k] = -1;
                    P.top_logprobs[(int64_t)r * P.top + k] = code > 0 ? NAN : NEG_INF;
                }
                if (code > 0 && P.dev_status) atomicMax(P.dev_status, code);
            }
        }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31 && warp < NW) sm.scan[warp] = incl;
    __syncthreads();
    const int in = lane < NW ? sm.scan[lane] : 0;
    const int before = incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? in : 0), nrows = __reduce_add_sync(0xffffffffu, in);
    const int64_t total = (int64_t)nrows * P.tpr;
    const int G = total < (int64_t)gridDim.x ? (int)total : (int)gridDim.x;
    if (cta >= G) return;
    // Odd lanes work on the run's end, even ones on its beginning.
    const int64_t edge = run_begin(cta + (lane & 1), total, G) - (lane & 1), edge_row = quotient(edge, P.tpr);
    const int64_t t0 = __shfl_sync(0xffffffffu, edge, 0), t1 = __shfl_sync(0xffffffffu, edge, 1) + 1;
    const int row_first = __shfl_sync(0xffffffffu, (int)edge_row, 0), row_last = __shfl_sync(0xffffffffu, (int)edge_row, 1);
    const int begin = (int)(t0 - (int64_t)row_first * P.tpr), end = (int)(t1 - (int64_t)row_last * P.tpr);  // the run's tiles of these
    const uintptr_t base_addr = reinterpret_cast<uintptr_t>(P.logits);
    const uintptr_t end_addr = base_addr + (uintptr_t)P.B * P.rows * P.V * sizeof(T);
    const uintptr_t copy_from = (base_addr + 15) & ~(uintptr_t)15, copy_to = end_addr & ~(uintptr_t)15;

    int k = 0, rr = 0;  // tiles copied or folded; rows folded
    for (int base = row_first; base <= row_last; base += ROWS) {
        // Entries of the run's next rows.
        if (base > row_first) __syncthreads();
        if (mine && before + mine > base && before < base + ROWS) {
            int at = before;
#pragma unroll 1
            for (int r = r0; r < r1 && at < base + ROWS; ++r) {
                if (r - r0 < 32 ? !((which >> (r - r0)) & 1) : fault_of(P, r) != 0) continue;
                if (at >= base) {
                    const int b = (int)((unsigned)r / (unsigned)P.T);
                    const int idx = P.row_index ? P.row_index[r] : r - b * P.T;
                    const float temp = P.temperatures ? P.temperatures[b] : P.temperature;
                    Row &w = sm.rows[at - base];
                    w.first = ((int64_t)b * P.rows + idx) * P.V;
                    w.r = r;
                    w.tok = P.tokens[r];
                    w.temp = temp == 0.f ? 1.f : temp;
                }
                ++at;
            }
        }
        __syncthreads();
        if (warp == NW) {
            // ---- copies ------------------------------------------------------------------------
            if (lane == 0)
                for (int q = base; q < base + ROWS && q <= row_last; ++q) {
                    bool ok = true;
                    const int64_t rowf = sm.rows[q - base].first;
                    const int head = (int)((unsigned)(rowf + P.mis) & (VEC - 1));
                    const int nvec = (int)(((unsigned)P.V + head + VEC - 1) / VEC);
                    const int j0 = q == row_first ? begin : 0, j1 = q == row_last ? end : P.tpr;
                    const uintptr_t first = base_addr + (uintptr_t)(rowf - head) * sizeof(T);  // may lie before the logits
                    for (int j = j0; j < j1; ++j, ++k) {
                        const int s = k % STAGES;
                        if (k >= STAGES)
                            ok = tc::bar_wait(tc::smem_u32(&sm.empty[s]), (k / STAGES + 1) & 1, abort);
                        // (Warps that gave up on a copy release its stage all the same.)
                        if (!ok || *abort) {
                            ok = false;
                            break;
                        }
                        const uintptr_t t = first + (uintptr_t)j * TILE_VEC * 16;
                        uintptr_t a = t, z = t + TILE_VEC * 16;
                        if (z > first + (uintptr_t)nvec * 16) z = first + (uintptr_t)nvec * 16;
                        if (a < copy_from) a = copy_from;  // vectors that the logits do not fill are not copied
                        if (z > copy_to) z = copy_to;
                        const uint32_t bytes = z > a ? (uint32_t)(z - a) : 0, bar = tc::smem_u32(&sm.full[s]);
                        tc::bar_expect(bar, bytes);
                        if (bytes)
                            asm volatile(
                                "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                    tc::smem_u32(sm.ring[s]) + (uint32_t)(a - t)),
                                "l"(a), "r"(bytes), "r"(bar)
                                : "memory");
                    }
                    if (!ok) break;
                }
            __syncwarp();
            continue;
        }
        if (warp > NW) {
            // ---- rows that are folded ----------------------------------------------------------
            for (int q = base; q < base + ROWS && q <= row_last; ++q, ++rr) {
                if ((rr & 1) != warp - NW - 1) continue;
                Row w = sm.rows[q - base];
                if (SV_INB(w.first + w.tok, (int64_t)P.B * P.rows * P.V, 1206))
                    w.x = E::load(static_cast<const T *>(P.logits) + w.first, w.tok);
                const int j0 = q == row_first ? begin : 0, j1 = q == row_last ? end : P.tpr;
                int c0 = cta, c1 = cta;
                bool first0 = true;
                if (j0 > 0 || j1 < P.tpr) {
                    const int64_t t = (int64_t)q * P.tpr;
                    c0 = cta_of(t, total, G);
                    c1 = cta_of(t + P.tpr - 1, total, G);
                    first0 = run_begin(c0, total, G) == t;
                }
                const bool ok = tc::bar_wait(tc::smem_u32(&sm.folded[rr & 1]), (rr / 2) & 1, abort);
                if (!__all_sync(0xffffffffu, ok)) break;
                finish<T>(P, sm.fin[rr & 1], sm.row[rr & 1], w, j0, j1, c0, c1, first0, top);
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem_u32(&sm.freed[rr & 1]));
            }
            continue;
        }
        // ---- folds -----------------------------------------------------------------------------
        for (int q = base; q < base + ROWS && q <= row_last; ++q, ++rr) {
            const int64_t rowf = sm.rows[q - base].first;
            const float temp = sm.rows[q - base].temp;
            const T *row = static_cast<const T *>(P.logits) + rowf;
            const int head = (int)((unsigned)(rowf + P.mis) & (VEC - 1));  // the row's first element in its first vector
            const int nvec = (int)(((unsigned)P.V + head + VEC - 1) / VEC);
            const int j0 = q == row_first ? begin : 0, j1 = q == row_last ? end : P.tpr;
            const int step = (int)((unsigned)(j1 - j0 + SLOTS - 1) / SLOTS);
            const float c = 1.44269504f / temp;
            const uint64_t c2 = sv::f2(c, c);
            Shared &sh = sm.row[rr & 1];
            const float tok_x = SV_INB(rowf + sm.rows[q - base].tok, (int64_t)P.B * P.rows * P.V, 1205)
                                    ? E::load(row, sm.rows[q - base].tok) : 0.f;
            if (rr >= 2) tc::bar_wait(tc::smem_u32(&sm.freed[rr & 1]), (rr / 2 + 1) & 1, abort);

            float m = NEG_INF, limit = 0.1f * LEAST;  // reference; the value that moves it
            uint64_t nmc2 = sv::f2(LEAST, LEAST), z2[2] = {0, 0}, s2[2] = {0, 0};
            float best = NEG_INF, cell = NEG_INF;  // the lane's maximum: of the row, of the cell
            int slot = 0, left = step;
            typename E::Count count;
            count.start(tok_x);
            for (int j = j0; j < j1; ++j, ++k) {
                const int st = k % STAGES;
                tc::bar_wait(tc::smem_u32(&sm.full[st]), (k / STAGES) & 1, abort);
                uint4 x4[VPT];
#pragma unroll
                for (int i = 0; i < VPT; ++i) x4[i] = sm.ring[st][i * NT + tid];
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem_u32(&sm.empty[st]));
                if (j == 0 || (j + 1) * TILE_VEC >= nvec) {
                    // The row's ends: what lies outside counts as -inf; a vector that the logits do not fill
                    // was not copied.
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
                        const int v = j * TILE_VEC + i * NT + tid;
                        const int64_t col = (int64_t)v * VEC - head;
                        if (col >= 0 && col + VEC <= P.V) continue;
                        x4[i] = make_uint4(E::NEG, E::NEG, E::NEG, E::NEG);
                        if (v < nvec)
                            for (int e = 0; e < VEC; ++e)
                                if (col + e >= 0 && col + e < P.V) E::set(x4[i], e, row, col + e);
                    }
                }
                float tm = NEG_INF;
#pragma unroll
                for (int i = 0; i < VPT; ++i) tm = fmaxf(tm, E::vmax(x4[i]));
                best = fmaxf(best, tm);
                cell = fmaxf(cell, tm);
                if (--left == 0 || j + 1 == j1) {
                    sh.cell[slot++][tid] = cell;
                    cell = NEG_INF;
                    left = step;
                }
                if (tm > limit) {
                    // A new reference: 2^-d of the sums, t of every term less by d.
                    const float now = tm * c, d = m == NEG_INF ? 0.f : now - m, f = ex2(-d);
                    float2 za = sv::f2_split(z2[0]), zb = sv::f2_split(z2[1]);
                    float2 sa = sv::f2_split(s2[0]), sb = sv::f2_split(s2[1]);
                    s2[0] = sv::f2(f * fmaf(-d, za.x, sa.x), f * fmaf(-d, za.y, sa.y));
                    s2[1] = sv::f2(f * fmaf(-d, zb.x, sb.x), f * fmaf(-d, zb.y, sb.y));
                    z2[0] = sv::f2(f * za.x, f * za.y);
                    z2[1] = sv::f2(f * zb.x, f * zb.y);
                    m = now;
                    limit = fmaf(SLACK * 0.69314718f, temp, tm);
                    nmc2 = sv::f2(-now, -now);
                }
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    uint64_t x[VEC / 2];
                    E::pairs(x4[i], x);
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        const uint64_t t = sv::f2_fma(x[e], c2, nmc2);
                        const float2 a = sv::f2_split(t);
                        const uint64_t p = sv::f2(ex2(a.x), ex2(a.y));
                        z2[e & 1] = sv::f2_add(z2[e & 1], p);
                        s2[e & 1] = sv::f2_fma(p, t, s2[e & 1]);
                    }
                    count.add(x4[i]);
                }
                count.tile_done();
            }

            // ---- the row's end, or the run's: this warp's share ----------------------------------
            const float2 za = sv::f2_split(sv::f2_add(z2[0], z2[1])), sa = sv::f2_split(sv::f2_add(s2[0], s2[1]));
            float z = za.x + za.y, s = sa.x + sa.y;
            int n = count.n;
            const float wm = warp_max(m);
            if (z != 0.f) {
                const float d = wm - m, f = ex2(-d);
                s = f * fmaf(-d, z, s);
                z *= f;
            } else {
                s = 0.f;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                z += __shfl_xor_sync(0xffffffffu, z, o);
                s += __shfl_xor_sync(0xffffffffu, s, o);
                n += __shfl_xor_sync(0xffffffffu, n, o);
            }
            const int sample = sample_of(top);
#pragma unroll 1
            for (int a = 0; a < sample; ++a) {
                const float y = warp_max(best);
                const unsigned who = __ballot_sync(0xffffffffu, best == y);
                if (lane == __ffs(who) - 1) best = NEG_INF;
                if (lane == 0) sh.best[warp * sample + a] = y;
            }
            if (lane == 0) {
                sh.m[warp] = wm;
                sh.z[warp] = z;
                sh.s[warp] = s;
                sh.count[warp] = n;
            }
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tc::smem_u32(&sm.folded[rr & 1]));
        }
    }
    __syncthreads();  // any warp's wait may have been the one that ran out
    if (*abort && lane == 0) {
        // Copies land before the CTA ends, folded or not.
        if (warp == NW) {
            atomicAdd(&tc::g_timeouts, 1ull);
            const int64_t begin = clock64();
            for (int i = k > STAGES ? k - STAGES : 0; i < k; ++i)
                while (!tc::bar_try(tc::smem_u32(&sm.full[i % STAGES]), (i / STAGES) & 1) &&
                       clock64() - begin < tc::WAIT_CLOCKS) {}
        } else if (P.dev_status) {
            atomicMax(P.dev_status, SPEC_VERIFY_DEV_TIMEOUT);
        }
    }
}

// -------------------------------------------------------------------------------------------------
// Host side.
// -------------------------------------------------------------------------------------------------
static std::mutex g_mu;
static int g_sms[64];

// Once per device: the SM count, the kernels' shared memory.
static int device_sms()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_sms[dev]) {
        int sms = 0;
        const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute((const void *)logprobs_kernel<__nv_bfloat16>, attr, (int)sizeof(Smem)) != cudaSuccess ||
            cudaFuncSetAttribute((const void *)logprobs_kernel<float>, attr, (int)sizeof(Smem)) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        g_sms[dev] = sms;
    }
    return g_sms[dev];
}

constexpr size_t COUNTER_BYTES = 65536 * 4;  // the workspace's fixed region of counters

template <typename T>
static cudaError_t launch(const Params &P, int grid, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(NT_ALL);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, P);
}

}  // namespace svlp

namespace sv {
bool logprobs_timeouts(unsigned long long &n) { return tc::read_timeouts(n); }
bool logprobs_wait_clocks(long long clocks) { return tc::set_wait_clocks(clocks); }

// This module's first range violation (debug builds; 0 otherwise), cleared when read.
unsigned long long logprobs_debug_fault()
{
#ifdef SV_DEBUG
    unsigned long long w = 0, z = 0;
    if (cudaMemcpyFromSymbol(&w, g_sv_debug_fault, sizeof w) != cudaSuccess ||
        cudaMemcpyToSymbol(g_sv_debug_fault, &z, sizeof z) != cudaSuccess)
        return ~0ull;
    return w;
#else
    return 0;
#endif
}
}  // namespace sv

extern "C" size_t spec_verify_logprobs_workspace_bytes(int B, int T, int V, int top_n)
{
    if (B < 1 || B > 65536 || T < 1 || T > sv::MAX_TREE || V < 1 || top_n < 0 || top_n > svlp::MAX_TOP) return 0;
    return svlp::COUNTER_BYTES + 2 * svlp::MAX_CTAS * sizeof(svlp::Part);
}

extern "C" int spec_verify_logprobs(const void *logits, int dtype, const int32_t *tokens, const int32_t *row_index, int B,
                                    int rows, int T, int V, const float *temperatures, float temperature, int top_n,
                                    float *logprobs, float *entropy, int32_t *ranks, int32_t *top_ids,
                                    float *top_logprobs, void *workspace, size_t ws_bytes, int32_t *dev_status,
                                    void *stream)
{
    using namespace svlp;
    if (!logits || !tokens || !logprobs || !workspace) return SPEC_VERIFY_EINVAL;
    if (dtype != SPEC_VERIFY_BF16 && dtype != SPEC_VERIFY_FP32) return SPEC_VERIFY_EINVAL;
    const size_t need = spec_verify_logprobs_workspace_bytes(B, T, V, top_n);
    if (!need || rows < 1 || rows > sv::MAX_TREE || (top_n && (!top_ids || !top_logprobs)) || (!row_index && T > rows))
        return SPEC_VERIFY_EINVAL;
    if (!temperatures && !(temperature >= 0.f && temperature < 3e38f)) return SPEC_VERIFY_EINVAL;
    const int size = dtype == SPEC_VERIFY_BF16 ? 2 : 4, vec = 16 / size;
    if ((uintptr_t)logits % size ||
        ((uintptr_t)tokens | (uintptr_t)row_index | (uintptr_t)temperatures | (uintptr_t)logprobs | (uintptr_t)entropy |
         (uintptr_t)ranks | (uintptr_t)top_ids | (uintptr_t)top_logprobs | (uintptr_t)dev_status) % 4)
        return SPEC_VERIFY_EINVAL;
    if (ws_bytes < need || (uintptr_t)workspace % 256) return SPEC_VERIFY_EWORKSPACE;
    const int sms = device_sms();
    if (!sms) return SPEC_VERIFY_ECUDA;
    Params P;
    P.logits = logits;
    P.tokens = tokens;
    P.row_index = row_index;
    P.temperatures = temperatures;
    P.temperature = temperature;
    P.B = B;
    P.rows = rows;
    P.T = T;
    P.V = V;
    P.top = top_n;
    P.logprobs = logprobs;
    P.entropy = entropy;
    P.ranks = ranks;
    P.top_ids = top_ids;
    P.top_logprobs = top_logprobs;
    P.dev_status = dev_status;
    P.mis = (int)((uintptr_t)logits % 16) / size;
    P.tpr = (int)((((int64_t)V + 2 * vec - 2) / vec + TILE_VEC - 1) / TILE_VEC);  // wherever the row begins
    P.counters = static_cast<unsigned *>(workspace);
    P.parts = static_cast<unsigned char *>(workspace) + COUNTER_BYTES;
    int grid = sms * CTAS_PER_SM < MAX_CTAS ? sms * CTAS_PER_SM : MAX_CTAS;
    if ((int64_t)B * T * P.tpr < grid) grid = (int)((int64_t)B * T * P.tpr);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SPEC_VERIFY_BF16 ? launch<__nv_bfloat16>(P, grid, s) : launch<float>(P, grid, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SPEC_VERIFY_ECUDA;
    }
    return SPEC_VERIFY_OK;
}
