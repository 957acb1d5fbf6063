// sv_logprobs.cu -- what is answered beside emitted tokens: the token's log probability, its rank,
// the distribution's entropy and its most likely alternatives, in one pass over the logits.
//
//   t = x c - m, c = log2(e) / T, Z = sum 2^t, S = sum t 2^t     (m: a reference near the maximum of x c)
//   logprob = ln 2 (t_tok - log2 Z), entropy = ln 2 (log2 Z - S / Z), rank = 1 + #{x > x_tok}
//
// Reading the rows once bounds it.  The rows that have a token are cut into tiles of NT * VPT 16-byte
// vectors and every CTA takes an equal run of tiles, so few rows are spread over the GPU and absent
// ones cost nothing; where a run cuts a row, the CTA that finishes last joins its parts in order.
//
// Threads keep (m, Z, S) of their own; m moves only when a vector passes it by more than 8.  It is kept
// as the rounded product x c, so that t is one fused operation and parts join without another rounding.
// Alternatives: every warp keeps its best `top` logits sorted across its lanes and a vector is
// looked at only when its maximum reaches a bound below which no alternative can lie: the least, over
// the warps, of each warp's ceil(top / NW)-th best (together these are `top` logits that reach it).
// A row's first tile gives the bound from the lanes' maxima, so that its logits do not all enter.
#include "sv_ops.cuh"

#include <mutex>

namespace svlp {

constexpr int NT = 256, NW = NT / 32;
constexpr int VPT = 4;               // 16-byte vectors per thread and tile
constexpr int CTAS_PER_SM = 3;
constexpr int MAX_CTAS = 1024;
constexpr int MAX_TOP = 32;
constexpr int ROWS = 256;            // rows of its run that a CTA lists at a time
constexpr int CAP = 512;             // candidates ranked at once
constexpr float SLACK = 8.f;         // log2 of the largest term
constexpr float LEAST = -0x1.92p99f;  // about -1e30, a bf16 value; logits below it count as it: 2^t is 0 and t stays finite
constexpr float NEG_INF = -__builtin_huge_valf();

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
    int64_t tpr;   // tiles per row
    unsigned *counters;
    unsigned char *parts;
};

struct Cand {
    float v;
    int i;
};
__device__ __forceinline__ bool better(float v, int i, float ov, int oi) { return v > ov || (v == ov && i < oi); }

// A part of a row: reference, sums, larger logits than the token's, whether a NaN or +inf was seen.
struct Part {
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

__device__ __forceinline__ float4 lds_volatile(const float *p)
{
    float4 r;
    asm volatile("ld.volatile.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)));
    return r;
}

__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 r;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
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
    static __device__ __forceinline__ float get(const uint4 &w, int e)
    {
        const uint32_t x = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
        return __uint_as_float(e & 1 ? x & 0xffff0000u : x << 16);
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
    static __device__ __forceinline__ float get(const uint4 &w, int e)
    {
        return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
    }
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

struct Smem {
    __align__(16) float bound[NW];  // each warp's ceil(top / NW)-th best so far
    float m[NW], z[NW], s[NW];
    int count[NW], scan[NW];
    Cand list[NW * MAX_TOP];  // the warps' lists, then the ranked candidates
    Cand cand[CAP];
    Cand best[MAX_TOP];
    int n, rows[ROWS], flag, join[2];
};

// The best `top` of total candidates get(0 .. total - 1), sorted, into sm.best; `bound`: at least `top` of
// them reach it (or it is -inf).  All threads of the CTA; sm.best is valid after the last barrier.
template <typename Get>
__device__ __forceinline__ void choose(Smem &sm, int total, int top, float bound, Get get)
{
    const int tid = threadIdx.x;
    if (tid == 0) sm.n = 0;
    if (tid < MAX_TOP) sm.best[tid] = {NEG_INF, -1};
    __syncthreads();
    for (int e = tid; e < total; e += NT) {
        const Cand x = get(e);
        if (x.v >= bound && x.i >= 0) {
            const int at = atomicAdd(&sm.n, 1);
            if (at < CAP) sm.cand[at] = x;
        }
    }
    __syncthreads();
    const int n = sm.n;
    if (n <= CAP) {
        // A candidate's place is the number of better ones; their order in the list does not matter.
        for (int e = tid; e < n; e += NT) {
            const Cand x = sm.cand[e];
            int place = 0;
            for (int o = 0; o < n; ++o) place += better(sm.cand[o].v, sm.cand[o].i, x.v, x.i);
            if (place < top) sm.best[place] = x;
        }
        __syncthreads();
        return;
    }
    // Many equal logits: the next best, one after the other.
    Cand last = {__builtin_huge_valf(), -1};
    for (int k = 0; k < top; ++k) {
        Cand b = {NEG_INF, 0x7fffffff};
        for (int e = tid; e < total; e += NT) {
            const Cand x = get(e);
            if (x.i >= 0 && better(last.v, last.i, x.v, x.i) && better(x.v, x.i, b.v, b.i)) b = x;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float v = __shfl_xor_sync(0xffffffffu, b.v, o);
            const int i = __shfl_xor_sync(0xffffffffu, b.i, o);
            if (better(v, i, b.v, b.i)) b = {v, i};
        }
        __syncthreads();
        if (tid % 32 == 0) sm.cand[tid / 32] = b;
        __syncthreads();
        for (int w = 0; w < NW; ++w)
            if (better(sm.cand[w].v, sm.cand[w].i, b.v, b.i)) b = sm.cand[w];
        last = b;
        if (tid == 0) sm.best[k] = b;
    }
    __syncthreads();
}

__device__ __forceinline__ int64_t run_begin(int c, int64_t total, int G) { return total * c / G; }
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int G) { return (int)(((x + 1) * G - 1) / total); }

// An entry's fault (a device status code), or whether it has a row to read.
__device__ __forceinline__ int fault_of(const Params &P, int64_t r, bool &present, int &tok, int &idx, float &temp)
{
    [[maybe_unused]] const int64_t n = (int64_t)P.B * P.T;
    const int b = (int)(r / P.T);
    tok = SV_INB(r, n, 1201) ? P.tokens[r] : -1;
    idx = P.row_index ? (SV_INB(r, n, 1202) ? P.row_index[r] : -1) : (int)(r - (int64_t)b * P.T);
    temp = P.temperatures ? (SV_INB(b, P.B, 1203) ? P.temperatures[b] : 1.f) : P.temperature;
    const int code = tok < -1 || tok >= P.V                                     ? SPEC_VERIFY_DEV_BAD_TOKEN
                     : idx < -1 || idx >= P.rows                                ? SPEC_VERIFY_DEV_BAD_ROW
                     : tok >= 0 && idx >= 0 && !(temp >= 0.f && temp < 3.4e38f) ? SPEC_VERIFY_DEV_BAD_ROW
                                                                                : 0;
    present = !code && tok >= 0 && idx >= 0;
    if (temp == 0.f) temp = 1.f;
    return code;
}

// The answers for entry r, by all threads; best: its alternatives.
template <typename T>
__device__ __noinline__ void answer(const Params &P, Smem &sm, int64_t r, const void *row, int tok, float temp, float m, float z, float s,
                       int count)
{
    const int tid = threadIdx.x;
    const float top1 = sm.best[0].v;
    const float c = 1.44269504f / temp;
    // A reference of such size is too coarse for the fused product (a row of nothing but finite masks):
    // differences are taken before the scale.
    const bool low = sm.best[0].i >= 0 && !(fabsf(top1) * c < 1e7f);
    if (low) {
        float zz = 0.f, ss = 0.f;
        for (int i = tid; i < P.V; i += NT) {
            const float t = (Elt<T>::load(row, i) - top1) * c, e = ex2(t);
            zz += e;
            if (e > 0.f) ss += e * t;
        }
        for (int o = 16; o; o >>= 1) {
            zz += __shfl_xor_sync(0xffffffffu, zz, o);
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        __syncthreads();
        if (tid % 32 == 0) sm.z[tid / 32] = zz, sm.s[tid / 32] = ss;
        __syncthreads();
        z = s = 0.f;
        for (int w = 0; w < NW; ++w) z += sm.z[w], s += sm.s[w];
    }
    const bool bad = sm.best[0].i < 0 || !(z < __builtin_huge_valf());
    const float log_z = log2f(z);
    auto said = [&](float x) {
        if (low || x < LEAST) return (x - (low ? top1 : 0.f)) / temp - log_z * 0.69314718f;
        return (fmaf(x, c, -m) - log_z) * 0.69314718f;
    };
    if (tid == 0) {
        P.logprobs[r] = bad ? NAN : said(Elt<T>::load(row, tok));
        if (P.entropy) P.entropy[r] = bad ? NAN : fmaxf((log_z - s / z) * 0.69314718f, 0.f);
        if (P.ranks) P.ranks[r] = bad ? -1 : count + 1;
        if (bad && P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_BAD_ROW);
    }
    if (tid < P.top) {
        const Cand y = sm.best[tid];
        if (SV_INB(r * P.top + tid, (int64_t)P.B * P.T * P.top, 1204)) {
            P.top_ids[r * P.top + tid] = bad ? -1 : y.i;
            P.top_logprobs[r * P.top + tid] = bad ? NAN : y.i < 0 ? NEG_INF : said(y.v);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(NT, CTAS_PER_SM) logprobs_kernel(const Params P)
{
    using E = Elt<T>;
    constexpr int VEC = E::VEC;
    __shared__ Smem sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const int top = P.top > 0 ? P.top : 1;  // the best one is the row's maximum
    const int quota = (top + NW - 1) / NW;
    if (tid < 2) sm.join[tid] = -1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The entries that have a row; what the others answer is written here, each by one CTA.
    const int64_t R = (int64_t)P.B * P.T;
    const int64_t per = (R + NT - 1) / NT;
    const int64_t w0 = run_begin(cta, R, gridDim.x), w1 = run_begin(cta + 1, R, gridDim.x);
    int mine = 0;
    for (int64_t r = tid * per; r < (tid + 1) * per && r < R; ++r) {
        bool present;
        int tok, idx;
        float temp;
        const int code = fault_of(P, r, present, tok, idx, temp);
        mine += present;
        if (!present && r >= w0 && r < w1) {
            P.logprobs[r] = code ? NAN : 0.f;
            if (P.entropy) P.entropy[r] = code ? NAN : 0.f;
            if (P.ranks) P.ranks[r] = code ? -1 : 0;
            for (int k = 0; k < P.top; ++k) {
                P.top_ids[r * P.top + k] = -1;
                P.top_logprobs[r * P.top + k] = code ? NAN : NEG_INF;
            }
            if (code && P.dev_status) atomicMax(P.dev_status, code);
        }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, nrows = 0;
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += sm.scan[w];
        nrows += sm.scan[w];
    }
    const int64_t total = nrows * P.tpr;
    const int G = total < (int64_t)gridDim.x ? (int)total : (int)gridDim.x;
    if (cta >= G) return;
    const int64_t t0 = run_begin(cta, total, G), t1 = run_begin(cta + 1, total, G);
    const int64_t row_first = t0 / P.tpr, row_last = (t1 - 1) / P.tpr;

    for (int64_t base = row_first; base <= row_last; base += ROWS) {
        // Entries of the run's next rows.
        __syncthreads();
        if (before + mine > base && before < base + ROWS) {
            int64_t at = before;
            for (int64_t r = tid * per; r < (tid + 1) * per && r < R && at < base + ROWS; ++r) {
                bool present;
                int tok, idx;
                float temp;
                fault_of(P, r, present, tok, idx, temp);
                if (!present) continue;
                if (at >= base) sm.rows[at - base] = (int)r;
                ++at;
            }
        }
        __syncthreads();
        for (int64_t q = base; q < base + ROWS && q <= row_last; ++q) {
            const int64_t r = sm.rows[q - base];
            bool present;
            int tok, idx;
            float temp;
            fault_of(P, r, present, tok, idx, temp);
            const int64_t rowf = ((r / P.T) * P.rows + idx) * P.V;
            const T *row = static_cast<const T *>(P.logits) + rowf;
            const int head = (int)((rowf + P.mis) % VEC);  // the row's first element in its first vector
            const int nvec = (int)(((int64_t)head + P.V + VEC - 1) / VEC);
            const int64_t j0 = q == row_first ? t0 - q * P.tpr : 0, j1 = q == row_last ? t1 - q * P.tpr : P.tpr;
            const float c = 1.44269504f / temp;
            const uint64_t c2 = sv::f2(c, c);

            auto load = [&](int64_t j, uint4 (&w)[VPT]) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int64_t v = (j * VPT + i) * NT + tid;
                    const int64_t col = v * VEC - head;
                    if (v < nvec && col >= 0 && col + VEC <= P.V) {
                        if (SV_INB(rowf + col + VEC - 1, (int64_t)P.B * P.rows * P.V, 1205)) w[i] = ldg_stream(row + col);
                    } else {  // the row's ends, element by element; past them -inf
                        w[i] = make_uint4(E::NEG, E::NEG, E::NEG, E::NEG);
                        if (v < nvec)
                            for (int e = 0; e < VEC; ++e)
                                if (col + e >= 0 && col + e < P.V) E::set(w[i], e, row, col + e);
                    }
                }
            };
            float m = NEG_INF, limit = 0.1f * LEAST;  // reference; the value that moves it
            uint64_t nmc2 = sv::f2(LEAST, LEAST), z2[2] = {0, 0}, s2[2] = {0, 0};
            float lv = NEG_INF;  // lane k: the warp's k-th best
            int li = 0x7fffffff;
            typename E::Count count;
            uint4 w[VPT], next[VPT];
            load(j0, w);
            count.start(E::load(row, tok));
            float bound = NEG_INF;
            {
                // The bound from the first tile's maxima.
                float x = NEG_INF;
#pragma unroll
                for (int i = 0; i < VPT; ++i) x = fmaxf(x, E::vmax(w[i]));
                float y = NEG_INF;
                for (int k = 0; k < quota; ++k) {
                    y = warp_max(x);
                    const unsigned who = __ballot_sync(0xffffffffu, x == y);
                    if (lane == __ffs(who) - 1) x = NEG_INF;
                }
                __syncthreads();  // the row before has been read to its end
                if (lane == 0) sm.bound[warp] = y;
                __syncthreads();
            }
            for (int64_t j = j0; j < j1; ++j) {
                if (j + 1 < j1) load(j + 1, next);
#pragma unroll
                for (int k = 0; k < NW; k += 4) {
                    const float4 y = lds_volatile(&sm.bound[k]);
                    const float l = fminf(fminf(y.x, y.y), fminf(y.z, y.w));
                    bound = k == 0 ? l : fminf(bound, l);
                }
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const float vm = E::vmax(w[i]);
                    if (vm > limit) {
                        // A new reference: 2^-d of the sums, t of every term less by d.
                        const float now = vm * c, d = m == NEG_INF ? 0.f : now - m, f = ex2(-d);
                        float2 z0 = sv::f2_split(z2[0]), z1 = sv::f2_split(z2[1]);
                        float2 s0 = sv::f2_split(s2[0]), s1 = sv::f2_split(s2[1]);
                        s2[0] = sv::f2(f * fmaf(-d, z0.x, s0.x), f * fmaf(-d, z0.y, s0.y));
                        s2[1] = sv::f2(f * fmaf(-d, z1.x, s1.x), f * fmaf(-d, z1.y, s1.y));
                        z2[0] = sv::f2(f * z0.x, f * z0.y);
                        z2[1] = sv::f2(f * z1.x, f * z1.y);
                        m = now;
                        limit = fmaf(SLACK * 0.69314718f, temp, vm);
                        nmc2 = sv::f2(-now, -now);
                    }
                    uint64_t x[VEC / 2];
                    E::pairs(w[i], x);
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        const uint64_t t = sv::f2_fma(x[e], c2, nmc2);
                        const float2 a = sv::f2_split(t);
                        const uint64_t p = sv::f2(ex2(a.x), ex2(a.y));
                        z2[e & 1] = sv::f2_add(z2[e & 1], p);
                        s2[e & 1] = sv::f2_fma(p, t, s2[e & 1]);
                    }
                    count.add(w[i]);
                    // Candidates of this warp's 32 vectors.
                    unsigned who = __ballot_sync(0xffffffffu, vm >= bound && vm > NEG_INF);
                    if (who) {
                        do {
                            const int src = __ffs(who) - 1;
                            who &= who - 1;
                            uint4 u;
                            u.x = __shfl_sync(0xffffffffu, w[i].x, src);
                            u.y = __shfl_sync(0xffffffffu, w[i].y, src);
                            u.z = __shfl_sync(0xffffffffu, w[i].z, src);
                            u.w = __shfl_sync(0xffffffffu, w[i].w, src);
                            const int col = (int)(((j * VPT + i) * NT + warp * 32 + src) * VEC) - head;
                            const float mv = E::get(u, lane & (VEC - 1));
                            const float last = __shfl_sync(0xffffffffu, lv, top - 1);
                            unsigned in = __ballot_sync(0xffffffffu, lane < VEC && mv >= bound && mv >= last && mv > NEG_INF);
                            while (in) {
                                const int e = __ffs(in) - 1;
                                in &= in - 1;
                                const float v = __shfl_sync(0xffffffffu, mv, e);
                                const int place = __popc(__ballot_sync(0xffffffffu, better(lv, li, v, col + e)));
                                const float uv = __shfl_up_sync(0xffffffffu, lv, 1);
                                const int ui = __shfl_up_sync(0xffffffffu, li, 1);
                                if (lane > place) lv = uv, li = ui;
                                if (lane == place) lv = v, li = col + e;
                            }
                        } while (who);
                        const float own = __shfl_sync(0xffffffffu, lv, quota - 1);
                        if (lane == 0 && own > sm.bound[warp]) *(volatile float *)&sm.bound[warp] = own;
                        bound = fmaxf(bound, __shfl_sync(0xffffffffu, lv, top - 1));
                    }
                }
                count.tile_done();
#pragma unroll
                for (int i = 0; i < VPT; ++i) w[i] = next[i];
            }

            // ---- the row's end, or the run's: join the threads ---------------------------------
            float2 za = sv::f2_split(sv::f2_add(z2[0], z2[1])), sa = sv::f2_split(sv::f2_add(s2[0], s2[1]));
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
            if (lane == 0) sm.m[warp] = wm, sm.z[warp] = z, sm.s[warp] = s, sm.count[warp] = n;
            if (lane < top) sm.list[warp * MAX_TOP + lane] = {lv, lv == NEG_INF ? -1 : li};
            __syncthreads();
            float M = NEG_INF;
            for (int k = 0; k < NW; ++k) M = fmaxf(M, sm.m[k]);
            z = s = 0.f;
            n = 0;
            float least = sm.bound[0];
            for (int k = 0; k < NW; ++k) {
                least = fminf(least, sm.bound[k]);
                n += sm.count[k];
                if (sm.z[k] != 0.f) {
                    const float d = M - sm.m[k], f = ex2(-d);
                    s += f * fmaf(-d, sm.z[k], sm.s[k]);
                    z += f * sm.z[k];
                }
            }
            choose(sm, NW * top, top, least, [&](int e) { return sm.list[(e / top) * MAX_TOP + e % top]; });
            if (j0 == 0 && j1 == P.tpr) {
                answer<T>(P, sm, r, row, tok, temp, M, z, s, n);
                continue;
            }
            // A part: this CTA's slot of the workspace.
            const int c0 = cta_of(q * P.tpr, total, G), c1 = cta_of((q + 1) * P.tpr - 1, total, G);
            const bool first0 = run_begin(c0, total, G) == q * P.tpr;
            auto part_of = [&](int x) {
                return reinterpret_cast<Part *>(P.parts) + 2 * x + (x == c0 && !first0);
            };
            Part *part = part_of(cta);
            if (tid == 0) part->m = M, part->z = z, part->s = s, part->count = n;
            if (tid < top) part->top[tid] = sm.best[tid];
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                sm.flag = atomicAdd(&P.counters[c0], 1u) == (unsigned)(c1 - c0);
                if (sm.flag) P.counters[c0] = 0;
            }
            __syncthreads();
            if (!sm.flag) continue;
            // The last part to be written: join them, in order.
            __threadfence();
            M = NEG_INF;
            float floor_ = NEG_INF;
            for (int x = c0 + lane; x <= c1; x += 32) {
                M = fmaxf(M, __ldcg(&part_of(x)->m));
                floor_ = fmaxf(floor_, __ldcg(&part_of(x)->top[top - 1].v));  // `top` logits reach the best of these
            }
            M = warp_max(M);
            floor_ = warp_max(floor_);
            z = s = 0.f;
            n = 0;
            for (int x = c0 + lane; x <= c1; x += 32) {
                const Part *p = part_of(x);
                const float pz = __ldcg(&p->z);
                n += __ldcg(&p->count);
                if (pz != 0.f) {
                    const float d = M - __ldcg(&p->m), f = ex2(-d);
                    s += f * fmaf(-d, pz, __ldcg(&p->s));
                    z += f * pz;
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                z += __shfl_xor_sync(0xffffffffu, z, o);
                s += __shfl_xor_sync(0xffffffffu, s, o);
                n += __shfl_xor_sync(0xffffffffu, n, o);
            }
            choose(sm, (c1 - c0 + 1) * top, top, floor_, [&](int e) {
                const int2 y = __ldcg(reinterpret_cast<const int2 *>(&part_of(c0 + e / top)->top[e % top]));
                return Cand{__int_as_float(y.x), y.y};
            });
            answer<T>(P, sm, r, row, tok, temp, M, z, s, n);
        }
    }
}

// -------------------------------------------------------------------------------------------------
// Host side.
// -------------------------------------------------------------------------------------------------
static std::mutex g_mu;
static int g_sms[64];

static int device_sms()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_sms[dev] && cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return g_sms[dev];
}

constexpr size_t COUNTER_BYTES = 65536 * 4;  // the workspace's fixed region of counters

template <typename T>
static cudaError_t launch(const Params &P, int grid, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(NT);
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
    P.tpr = (((int64_t)V + 2 * vec - 2) / vec + NT * VPT - 1) / (NT * VPT);  // wherever the row begins
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
