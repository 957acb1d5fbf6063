// sv_attention.cu -- attention of a verification step's nodes over the paged cache.
//
//   s_j = scale * q . k_j over the positions j that node n sees: j < committed, and the positions
//   committed + a of the nodes a on the path from the root to n (a chain: a <= n)
//   out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), lse = m + ln sum_j e^(s_j - m)
//
// Reading the cache bounds it: a key head's N * Hq/Hkv query rows are all the arithmetic that a
// position's 4 D bytes get, far below what the tensor cores do in the time.  So the products are
// turned round: positions, of which there are always plenty, fill the 128 rows of the matrix
// instruction and the query rows are its columns (16, 32 or 64, whatever the call has):
//
//   S^T [128 positions][rows] = K [128][D] . Q^T          both operands from shared memory
//   O^T [128 dims][rows]     += V^T [dims][128] . P^T     V as it lies in the cache, read transposed
//
// Each CTA takes an equal run of the batch's work, whatever the lengths: tiles (128 positions of one
// request and key head) at COST_TILE each and segments (a request and key head) at COST_SEGMENT for
// their beginning and end.  So one long request is split over all SMs and many short ones share them;
// where a run cuts a request, the parts are joined by the CTA that finishes last.
//
// Warps 0-3 copy tiles into a ring of K and V units, a row of 16-byte chunks per slot (gathers by
// TMA were tried first: four 128-byte rows took 61 clocks to issue, 8 bytes per clock, where an SM's
// share of HBM is 23).  Warp 4 issues the products, warp 5 lists the run's segments (a segment: the
// run's tiles of one request and key head) a few ahead of everybody, warps 6-7 stage the queries and
// the tree's mask.  The warpgroups from warp 8 on do the softmax, a position and a share of the columns
// per thread: scores come to them as columns, so the exponentials are spread evenly however few the
// query rows.
//
// The softmax's reference, a score, moves only when another passes it by more than a factor of 2^8 in
// weight (a vote of 128 threads per tile), so that the accumulators are left alone in nearly every tile.
// A weight keeps its digits at any size in bf16, whose exponents are fp32's.  In fp16 it does down to
// 2^-14, then loses them one by one, and below 2^-25 it is 0: there the reference has weight 2^7, so that
// weights reach from 2^15 (of 65504) down to 2^-32 of an ordinary largest one.  131072 positions at
// 2^-25.2 of one other, together 0.003 of the sum, were lost with a reference of weight 1.
// An exponent is one fused operation on the score and the reference's rounded product with the scale.  From
// FAR on that rounding is whole exponents, and the reference is taken from the scores before.  (Everywhere:
// 101.6 us against 100.7 for the tree of 16 below, 44.7 against 44.4 for the 96 requests.)
//
// Measured (GB300, copy rate 6.68 TB/s; 32 query and 8 key heads of 128 unless said): 64 chains of 8 over
// 509 to 8192 positions 122-125 us for 742 MB, 5.9-6.1 TB/s; one tree of 16 over 131000 positions 100 us
// for 537 MB, 5.3 TB/s (9 us until the first tile is there, 8 us for the joins); 96 requests of one token and 12
// heads of 64 over 1 to 4001 positions 44 us for 148 MB, 3.4 TB/s; 48 trees of 8 over up to 504 positions 19 us.
// One token of each of 64 requests over 8192 positions 320 us for 2.15 GB, 6.7 TB/s.  Heads of 80, 96 and 112 are padded
// to 128 by the copies' zero-filling form: the 64 chains 138, 138 and 164 us for 464, 557 and 649 MB.
// Long segments are bound by HBM; short ones by the chain through a segment, some 5000 clocks (its
// first scores 1000, references 600, weights and the last product 1300, what it writes 900), which is
// all the SM does unless two CTAs share it.
#include "sv_ops.cuh"
#include "sv_tc.cuh"

#include <mutex>

namespace svatt {

using sv::Half2;

constexpr int TILE = 128;     // positions per tile
constexpr int MAXD = 128;
constexpr int MAX_SMS = 192;  // the workspace has room for two parts per CTA
constexpr int COUNTERS = 2 * MAX_SMS;
constexpr int FLAGS = 16;     // bad-slot flags: more than the segments the ring can hold
constexpr int SEGS = 8;       // segments listed ahead
constexpr float SLACK = 8.f;  // log2 of how much a weight may pass the reference's
constexpr float FAR = 0x1p24f;  // of a reference times the scale
// log2 of the reference's weight.
__host__ __device__ constexpr float lift(bool bf16) { return bf16 ? 0.f : 7.f; }
// In half tiles.  A segment at 3 or 5: 45.9 or 46.8 us against 45.8 for the 96 short requests above, 20.7 or 21.2
// against 20.8 for the 48 trees; at 2 (with one CTA per SM) 63 against 56.
constexpr int COST_TILE = 2, COST_SEGMENT = 4;

// Warpgroups of the softmax: two hold 16 columns a thread at most, and so do four where there are 64 columns
// (with 32 a thread: one tree of 16 over 131000 positions 105.6 us against 102.7).
__host__ __device__ constexpr int groups(int nq) { return nq == 64 ? 4 : 2; }
__host__ __device__ constexpr int threads(int nq) { return 256 + 128 * groups(nq); }
// CTAs that an SM holds.  With at most 8 columns a thread, 64 registers nearly do (32 bytes spilled), and one CTA
// works while the other is between segments: 96 requests of 12 heads of 64 take 44.4 us against 52.4, 128
// requests of up to 504 positions (8 key heads of 128) 30.2 against 30.7.  Two units of 128 dimensions are then all
// that fit in a ring, and longer requests lose: 64 requests of 509 to 8192 positions 122.5 us against 118.6, of
// 8192 320 against 315, one of 131000 93.2 against 89.7.  At 32 columns 64 registers spill 260 bytes: 139 us
// against 125 for the 64 chains above.
__host__ __device__ constexpr int ctas_per_sm(int nq) { return nq == 16 ? 2 : 1; }

struct Params {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;
    int64_t q_row, k_slot, v_slot, num_slots;
    const int32_t *slot_table, *committed, *parents, *num_nodes;
    int max_pos, B, N, Hq, Hkv, D, G, QT;  // G query heads per key head, QT column blocks
    float scale_log2;
    int32_t *dev_status;
    unsigned *counters;  // arrivals at joins, COUNTERS each: of a segment's first group (by the CTA that began the segment),
                         // of its others (by the group's first CTA), of the groups (by the segment's CTA)
    float *parts;
};

// Shared memory: a ring of units (a K or V tile each; tile k's K is unit 2 k, its V unit 2 k + 1),
// two query buffers, the weights, then Misc.  All bases are multiples of 1024 bytes.
template <int NQ, int DP>
struct Layout {
    static constexpr int HALVES = DP / 64;
    static constexpr int UNIT = TILE * DP * 2;
    static constexpr int NU = ctas_per_sm(NQ) == 2 ? (DP == 64 ? 5 : 2) : 5 * 128 / DP;
    static constexpr int QBYTES = NQ * DP * 2;
    static constexpr int QSTEP = QBYTES < 1024 ? 1024 : QBYTES;
    static constexpr int PBYTES = TILE * 128;  // a row of 64 columns per position
    static constexpr int Q0 = NU * UNIT, P0 = Q0 + 2 * QSTEP, M0 = P0 + PBYTES;
    static constexpr int COLS = 3 * NQ <= 64 ? 64 : 3 * NQ <= 128 ? 128 : 256;  // TMEM columns
};

// A run's tiles [j0, j1) of one request, key head and column block.
struct __align__(16) Seg {
    int b, h, qt, kind;        // kind 0: to attend; 1: no nodes; 2: lengths are wrong; 3: no more segments
    int c, nn, j0, j1;
    int part, c0, c1, pad;     // part: the workspace part it writes (-1: it is the whole); the CTAs it spans
};

// Parts to be joined: of segment g, `n` from the `first` on, `step` apart.
struct Join {
    Seg g;
    int first, n, step;
};

// A segment's parts in groups: more than 8 are joined in two levels, for one CTA reads them at 50 bytes a clock
// (20 parts of 64 columns 116.5 us for the call against 118, 38 of 16 columns 111 against 117).
__device__ __forceinline__ int group_size(int parts)
{
    if (parts <= 8) return parts;
    int s = 3;
    while (s * s < parts) ++s;
    return s;
}

template <int NQ, int NU>
struct Misc {
    uint64_t full[NU], empty[NU];
    static constexpr int NT = threads(NQ), WG = groups(NQ);
    uint64_t sfull[2], sempty[2], qfull[2], qempty[2], segfull[SEGS], segempty[SEGS], pfull, pvdone, drain;
    Seg seg[SEGS];
    unsigned long long desc[2][sv::MAX_TREE];  // columns that see node a, of the staged queries
    float ref[NQ], off[NQ], nref[NQ];  // a column's reference; what scores lose before the scale, what is added after it
    float fac[NQ], red[4][NQ], red2[4][NQ];
    int code[2], poison[2];
    int bad[WG][FLAGS];
    int begin_b, abort;
    int64_t begin_base, scan[NT / 32];
    uint32_t tmem;
    Join join[2];
    int joins[2];
    int8_t par[sv::MAX_TREE];
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void group_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

__device__ __forceinline__ bool group_or(int id, int n, bool x)
{
    uint32_t y;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(y)
        : "r"(id), "r"(n), "r"((uint32_t)x)
        : "memory");
    return y;
}

// Sums over the warp's lanes of W values per lane, by exchanges that halve the columns a lane still
// holds (31 shuffles for 32 columns instead of 5 for each); lane c < W returns column c's.
template <int W>
__device__ __forceinline__ float column_sum(const float (&v)[W], int lane)
{
    float x[W];
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = v[i];
#pragma unroll
    for (int half = W / 2; half; half >>= 1) {
        const bool up = lane & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = up ? x[i + half] : x[i], give = up ? x[i] : x[i + half];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
        }
    }
#pragma unroll
    for (int o = W; o < 32; o <<= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    return x[0];
}

// Floats of one part: per column the weighted values, then references, sums, sums of the rounded
// weights.
template <int NQ>
__host__ __device__ constexpr int part_floats()
{
    return NQ * MAXD + 3 * NQ;
}

// Runs are cut at multiples of total / G on the axis of costs.  A cut x into a segment of n tiles leaves the
// tiles before `cut_tile` to the run before; cuts are at least COST_TILE apart, so no run between two
// cuts of a segment is empty.
// (Quotients in 32 bits wherever they fit: 64-bit division is a hundred instructions.)
__device__ __noinline__ int64_t quotient64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return (uint64_t)(a | b) >> 32 ? quotient64(a, b) : (int64_t)((unsigned)a / (unsigned)b);
}
__device__ __forceinline__ int64_t run_begin(int c, int64_t total, int G) { return quotient(total * c, G); }
__device__ __forceinline__ int cut_tile(int64_t x, int n)
{
    const int64_t t = (x - COST_SEGMENT + COST_TILE / 2) / COST_TILE;
    return t <= 0 ? 0 : t < n ? (int)t : n;
}
// The last run that begins before x.
__device__ __forceinline__ int run_before(int64_t x, int64_t total, int G) { return (int)quotient(x * G + total - 1, total) - 1; }

__device__ __forceinline__ int kind_of(const Params &P, int c, int nn)
{
    return nn < 0 || nn > P.N || c < 0 || (int64_t)c + nn > P.max_pos ? 2 : nn == 0 ? 1 : 0;
}
__device__ __forceinline__ int tiles_of(int kind, int c, int nn) { return kind ? 1 : (c + nn + TILE - 1) / TILE; }
__device__ __forceinline__ int64_t cost_of(int tiles) { return COST_SEGMENT + (int64_t)tiles * COST_TILE; }

__device__ __forceinline__ void lengths(const Params &P, int b, int &c, int &nn)
{
    c = SV_INB(b, P.B, 1101) ? P.committed[b] : 0;
    nn = P.num_nodes ? (SV_INB(b, P.B, 1102) ? P.num_nodes[b] : 0) : P.N;
}

template <bool BF, int NQ, int DP>
__global__ void __launch_bounds__(threads(NQ), ctas_per_sm(NQ)) attention_kernel(const Params P)
{
    using L = Layout<NQ, DP>;
    using M = Misc<NQ, L::NU>;
    constexpr int NU = L::NU, HALVES = L::HALVES, NT = threads(NQ), WG = groups(NQ);
    extern __shared__ __align__(1024) unsigned char smem[];
    M &ms = *reinterpret_cast<M *>(smem + L::M0);
    const uint32_t s0 = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    volatile int *abort = &ms.abort;

    if (tid == NT - 32) {  // a warp that has no request to look at in a batch of ordinary size
        for (int s = 0; s < NU; ++s) {
            tc::bar_init(tc::smem_u32(&ms.full[s]), 128);
            tc::bar_init(tc::smem_u32(&ms.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_u32(&ms.sfull[i]), 1);
            tc::bar_init(tc::smem_u32(&ms.sempty[i]), 128 * WG);
            tc::bar_init(tc::smem_u32(&ms.qfull[i]), 64);
            tc::bar_init(tc::smem_u32(&ms.qempty[i]), 1 + 4 * WG);  // the last scores' products, the softmax's warps
            ms.joins[i] = 0;
        }
        for (int i = 0; i < SEGS; ++i) {
            tc::bar_init(tc::smem_u32(&ms.segfull[i]), 1);
            tc::bar_init(tc::smem_u32(&ms.segempty[i]), NT / 32 - 1);  // warps but the one that lists
        }
        tc::bar_init(tc::smem_u32(&ms.pfull), 128 * WG);
        tc::bar_init(tc::smem_u32(&ms.pvdone), 1);
        tc::bar_init(tc::smem_u32(&ms.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ms.abort = 0;
    }
    if (tid < WG * FLAGS) (&ms.bad[0][0])[tid] = 0;
    if (warp == 4) tc::tmem_alloc(tc::smem_u32(&ms.tmem), L::COLS);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The batch's cost, and the request that this CTA's run begins in.
    const int HT = P.Hkv * P.QT;
    const int per = (P.B + NT - 1) / NT;
    int64_t mine = 0;
#pragma unroll 1
    for (int i = 0; i < per && tid * per + i < P.B; ++i) {
        int c, nn;
        lengths(P, tid * per + i, c, nn);
        mine += cost_of(tiles_of(kind_of(P, c, nn), c, nn)) * HT;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) ms.scan[warp] = incl;
    __syncthreads();
    // (Sums over the warps in two halves of 32 bits: costs are below 2^56.)
    const int64_t in = lane < NT / 32 ? ms.scan[lane] : 0;
    auto sum = [](int64_t x) {
        return ((int64_t)__reduce_add_sync(0xffffffffu, (unsigned)(x >> 24)) << 24) + __reduce_add_sync(0xffffffffu, (unsigned)x & 0xffffffu);
    };
    const int64_t before = incl - mine + sum(lane < warp ? in : 0), total = sum(in);
    // Small batches leave the last CTAs out: a run costs COST_TILE at least.
    const int G = total / COST_TILE < (int64_t)gridDim.x ? (int)(total / COST_TILE) : (int)gridDim.x;
    // Odd lanes work out the run's end, even ones its beginning.
    const int64_t edge = cta + (lane & 1) <= G ? run_begin(cta + (lane & 1), total, G) : total;
    const int64_t t0 = __shfl_sync(0xffffffffu, edge, 0), t1 = __shfl_sync(0xffffffffu, edge, 1);
    if (t0 >= before && t0 < before + mine) {
        int64_t at = before;
        int b = tid * per;
#pragma unroll 1
        for (; per > 1 && b < P.B; ++b) {
            int c, nn;
            lengths(P, b, c, nn);
            const int64_t n = cost_of(tiles_of(kind_of(P, c, nn), c, nn)) * HT;
            if (t0 < at + n) break;
            at += n;
        }
        ms.begin_b = b;
        ms.begin_base = at;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ms.tmem;

    // The next segment, for every warp but the one that lists them; kind 3 also when a wait failed.
    int si = 0;
    auto take = [&](Seg &g) {
        const bool ok = tc::bar_wait(tc::smem_u32(&ms.segfull[si % SEGS]), (si / SEGS) & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) return false;
        g = ms.seg[si % SEGS];
        __syncwarp();
        if (lane == 0) tc::bar_arrive(tc::smem_u32(&ms.segempty[si % SEGS]));
        ++si;
        return true;
    };

    if (t1 > t0) {
        if (warp < 4) {
            // ---- tiles into shared memory -------------------------------------------------
            // A row's CPR chunks go to CPR lanes, 32 / CPR rows to a warp's copy.  A lane keeps the
            // slot of one of its warp's 32 rows; they are read one tile ahead of the copies.
            constexpr int CPR = DP / 8, RPI = 32 / CPR, ITER = TILE / (4 * RPI);
            const int chunk = lane % CPR, sub = lane / CPR;
            const int own = warp * RPI + lane % RPI + 4 * RPI * (lane / RPI);  // the row whose slot it keeps
            const int first = warp * RPI + sub;                                // its row of the first copy
            const uint32_t to = (chunk >> 3) * TILE * 128 + first * 128 + (((chunk & 7) ^ (first & 7)) << 4);
            const bool wide = chunk * 8 < P.D;
            Seg g = {};
            int seg = -1, j = 0, slot = -1, u = 0;
            bool ok = true;
            // To the next tile, and its slot: 1, or 0 when there is none.  A segment that is not listed yet
            // may wait for the tile at hand: without `block` the answer is then 2.
            auto seek = [&](bool block) {
                if (seg >= 0 && !g.kind && j + 1 < g.j1) {
                    ++j;
                } else {
                    do {
                        if (!block &&
                            !__all_sync(0xffffffffu, tc::bar_test(tc::smem_u32(&ms.segfull[si % SEGS]), (si / SEGS) & 1)))
                            return 2;
                        if (!take(g) || g.kind == 3) return 0;
                    } while (g.kind);
                    ++seg;
                    j = g.j0;
                }
                const int pos = j * TILE + own;
                slot = -1;
                if (pos < g.c + g.nn) {
                    const int64_t at = (int64_t)g.b * P.max_pos + pos;
                    slot = SV_INB(at, (int64_t)P.B * P.max_pos, 1103) ? P.slot_table[at] : -1;
                }
                return 1;
            };
            // The slot read ahead, in the pool or -1 (past the end, or wrong: its segment is marked).
            auto check = [&](bool past) {
                if (!past && (slot < 0 || slot >= P.num_slots)) {
#pragma unroll
                    for (int i = 0; i < WG; ++i) *(volatile int *)&ms.bad[i][seg % FLAGS] = 1;
                    slot = -1;
                }
                return slot;
            };
            for (int found = seek(true); found == 1 && ok;) {
                const int slots = check(j * TILE + own >= g.c + g.nn);
                const int64_t at = (int64_t)g.h * P.D + (wide ? chunk * 8 : 0);
                const bool whole = __all_sync(0xffffffffu, slots >= 0 && wide);
                found = seek(false);
#pragma unroll 1
                for (int kv = 0; kv < 2 && ok; ++kv, ++u) {
                    if (u >= NU) {
                        const bool free = tc::bar_wait(tc::smem_u32(&ms.empty[u % NU]), (u / NU + 1) & 1, abort);
                        ok = __all_sync(0xffffffffu, free);
                        if (!ok) break;
                    }
                    const uint32_t dst = s0 + (u % NU) * L::UNIT + to;
                    const unsigned char *base = reinterpret_cast<const unsigned char *>((kv ? P.v : P.k) + at);
                    const uint32_t stride = (uint32_t)(kv ? P.v_slot : P.k_slot) * 2;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < ITER; ++i) {
                            const uint32_t s = __shfl_sync(0xffffffffu, slots, i * RPI + sub);
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 4 * RPI * 128),
                                         "l"(base + (uint64_t)s * stride)
                                         : "memory");
                        }
                    } else {
#pragma unroll 4
                        for (int i = 0; i < ITER; ++i) {  // zeros where there is nothing to copy
                            const int s = __shfl_sync(0xffffffffu, slots, i * RPI + sub);
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 4 * RPI * 128),
                                         "l"(base + (uint64_t)(uint32_t)(s < 0 ? 0 : s) * stride), "r"(s >= 0 && wide ? 16 : 0)
                                         : "memory");
                        }
                    }
                    // The unit's barrier hears of each thread's copies as they land; nobody waits for them here.
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(&ms.full[u % NU]))
                                 : "memory");
                }
                if (found == 2 && ok) found = seek(true);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == 4) {
            // ---- products ------------------------------------------------------------------
            constexpr uint32_t ID_S = tc::instr_desc(BF, false, false, 128, NQ);
            constexpr uint32_t ID_O = tc::instr_desc(BF, true, true, 128, NQ);
            const int dsteps = P.D / 16;
            const uint64_t kd = tc::smem_desc(s0, 0, 1024), qd = tc::smem_desc(s0 + L::Q0, 0, 1024);
            const uint64_t vd = tc::smem_desc(s0, HALVES > 1 ? TILE * 128 : 0, 1024), pd = tc::smem_desc(s0 + L::P0, 0, 1024);
            int k = 0, seg = -1;       // tiles whose scores are under way
            int wk = 0, wsteps = 0, wstart = 0;  // tiles weighed; the waiting one's
            bool ok = true;
            Seg g = {};
            auto ready_p = [&] {
                const int u = 2 * wk + 1;
                return tc::bar_test(tc::smem_u32(&ms.pfull), wk & 1) && tc::bar_test(tc::smem_u32(&ms.full[u % NU]), (u / NU) & 1);
            };
            auto weigh = [&] {  // O^T (+)= V^T P^T of tile wk
                const int u = 2 * wk + 1;
                tc::fence_after();
                tc::fence_async_smem();  // the copies are ordinary writes; this thread has seen them land
                const uint64_t a = vd + (uint64_t)((u % NU) * (L::UNIT >> 4));
                if (wsteps == 8) {  // straight-line code for whole tiles
                    tc::mma_f16(tmem + 2 * NQ, a, pd, ID_O, !wstart);
#pragma unroll
                    for (int i = 1; i < 8; ++i) tc::mma_f16(tmem + 2 * NQ, a + i * 128, pd + i * 128, ID_O, true);
                } else {
                    for (int i = 0; i < wsteps; ++i)
                        tc::mma_f16(tmem + 2 * NQ, a + i * 128, pd + i * 128, ID_O, !wstart || i > 0);
                }
                tc::commit(tc::smem_u32(&ms.empty[u % NU]));
                tc::commit(tc::smem_u32(&ms.pvdone));
                ++wk;
            };
            // One thread does it all, and waits for nothing without weighing what is ready meanwhile.
            int64_t begin = 0;
            auto late = [&] {
                if (!*abort && clock64() - begin <= tc::wait_clocks()) return false;
                *abort = 1;
                return true;
            };
            const bool me = tc::elect();
            while (me) {
                begin = clock64();
                while (ok && !tc::bar_test(tc::smem_u32(&ms.segfull[si % SEGS]), (si / SEGS) & 1)) {
                    if (wk < k && ready_p()) weigh();
                    ok = !late();
                }
                if (!ok) break;
                g = ms.seg[si % SEGS];
                tc::bar_arrive(tc::smem_u32(&ms.segempty[si % SEGS]));
                ++si;
                if (g.kind == 3) break;
                if (g.kind) continue;
                ++seg;
                for (int j = g.j0; j < g.j1 && ok; ++j) {
                    // Scores of this tile and weighing of the one before, whichever is ready first.
                    const int u = 2 * k, sb = k & 1;
                    bool scored = false;
                    begin = clock64();
                    while (!scored || wk < k) {
                        if (!scored && tc::bar_test(tc::smem_u32(&ms.full[u % NU]), (u / NU) & 1) &&
                            tc::bar_test(tc::smem_u32(&ms.qfull[seg & 1]), (seg >> 1) & 1) &&
                            (k < 2 || tc::bar_test(tc::smem_u32(&ms.sempty[sb]), ((k >> 1) & 1) ^ 1))) {
                            tc::fence_after();
                            tc::fence_async_smem();
                            const uint64_t a = kd + (uint64_t)((u % NU) * (L::UNIT >> 4));
                            const uint64_t b = qd + (uint64_t)((seg & 1) * (L::QSTEP >> 4));
                            if (dsteps == DP / 16) {
#pragma unroll
                                for (int d = 0; d < DP / 16; ++d)
                                    tc::mma_f16(tmem + sb * NQ, a + (d >> 2) * (TILE * 8) + (d & 3) * 2,
                                                b + (d >> 2) * (NQ * 8) + (d & 3) * 2, ID_S, d > 0);
                            } else {
                                for (int d = 0; d < dsteps; ++d)
                                    tc::mma_f16(tmem + sb * NQ, a + (d >> 2) * (TILE * 8) + (d & 3) * 2,
                                                b + (d >> 2) * (NQ * 8) + (d & 3) * 2, ID_S, d > 0);
                            }
                            tc::commit(tc::smem_u32(&ms.empty[u % NU]));
                            tc::commit(tc::smem_u32(&ms.sfull[sb]));
                            if (j + 1 == g.j1) tc::commit(tc::smem_u32(&ms.qempty[seg & 1]));
                            scored = true;
                        }
                        if (wk < k && ready_p()) weigh();
                        if (late()) {
                            ok = false;
                            break;
                        }
                    }
                    const int left = g.c + g.nn - j * TILE;
                    wsteps = left >= TILE ? TILE / 16 : (left + 15) / 16;
                    wstart = j == g.j0;
                    ++k;
                }
                if (!ok) break;
            }
            begin = clock64();
            while (me && ok && wk < k) {
                if (ready_p()) weigh();
                ok = !late();
            }
            __syncwarp();
        } else if (warp == 5) {
            // ---- the run's segments ----------------------------------------------------------
            // The lengths of 32 requests are read at a time.
            int b = ms.begin_b, base = b, c = 0, nn = 0, n = 0;
            if (b + lane < P.B) lengths(P, b + lane, c, nn);
            int64_t at = ms.begin_base;  // the cost before the item
            bool ok = true;
            auto put = [&](const Seg &g) {
                if (n >= SEGS) {
                    ok = tc::bar_wait(tc::smem_u32(&ms.segempty[n % SEGS]), (n / SEGS + 1) & 1, abort);
                    ok = __all_sync(0xffffffffu, ok);  // the lanes stay together
                    if (!ok) return;
                }
                if (lane == 0) {
                    ms.seg[n % SEGS] = g;
                    tc::bar_arrive(tc::smem_u32(&ms.segfull[n % SEGS]));
                }
                __syncwarp();
                ++n;
            };
            Seg g = {};
            bool first = true;
            while (at < t1 && ok) {
                if (b == base + 32) {
                    base = b;
                    if (b + lane < P.B) lengths(P, b + lane, c, nn);
                }
                g.b = b;
                g.c = __shfl_sync(0xffffffffu, c, b - base);
                g.nn = __shfl_sync(0xffffffffu, nn, b - base);
                g.kind = kind_of(P, g.c, g.nn);
                const int ntile = tiles_of(g.kind, g.c, g.nn);
                const int64_t cost = cost_of(ntile);
                int item = 0;
                if (first) {  // items before the one that the run begins in
                    item = (int)quotient(t0 - at, cost);
                    at += item * cost;
                    first = false;
                }
                for (; item < HT && at < t1 && ok; ++item, at += cost) {
                    g.h = P.QT == 1 ? item : item / P.QT;
                    g.qt = item - g.h * P.QT;
                    g.j0 = cut_tile(t0 - at, ntile);
                    g.j1 = cut_tile(t1 - at, ntile);
                    if (g.j0 >= g.j1) continue;
                    g.part = -1;
                    if (g.j0 > 0 || g.j1 < ntile) {
                        // The runs that hold its first and its last tile, and all between.
                        const int run = run_before(at + (lane & 1 ? cost - COST_TILE / 2 : COST_SEGMENT + COST_TILE / 2), total, G);
                        g.c0 = __shfl_sync(0xffffffffu, run, 0);
                        g.c1 = __shfl_sync(0xffffffffu, run, 1);
                        g.part = 2 * cta + (cta == g.c0);
                    }
                    put(g);
                }
                ++b;
            }
            g.kind = 3;
            if (ok) put(g);
        } else if (warp < 8) {
            // ---- queries and the tree's mask -----------------------------------------------
            const int t = tid - 192;
            constexpr int CH = DP / 8, RPI = 64 / CH;  // 16-byte chunks of a row; rows at a time
            const int step_n = (int)((unsigned)RPI / (unsigned)P.G), step_h = RPI - step_n * P.G;  // RPI rows in nodes and heads
            const int64_t src_step = step_n * P.q_row + step_h * P.D, src_wrap = P.q_row - (int64_t)P.G * P.D;
            int seg = -1;
            Seg g = {};
            for (;;) {
                const bool got = take(g);
                if (group_or(2, 64, !got) || g.kind == 3) break;
                if (g.kind) continue;
                ++seg;
                const int buf = seg & 1;
                // Which nodes see node a: every node's path to the root, then transposed.
                bool wrong = false;
                int p = t - 1;
                if (P.parents && t < g.nn) {
                    const int64_t at = (int64_t)g.b * P.N + t;
                    p = SV_INB(at, (int64_t)P.B * P.N, 1104) ? P.parents[at] : -1;
                    wrong = t == 0 ? p != -1 : (p < 0 || p >= t);
                    if (wrong) p = -1;
                }
                const int ch = t % CH, r0 = t / CH;
                const unsigned gr = g.qt * NQ + r0;
                int n = (int)(gr / (unsigned)P.G), h = (int)gr - n * P.G;
                const uint16_t *src = P.q + ((int64_t)g.b * P.N + n) * P.q_row + (int64_t)(g.h * P.G + h) * P.D + ch * 8;
                const bool wide = ch * 8 < P.D;
                bool ok = true;
                if (seg >= 2) ok = tc::bar_wait(tc::smem_u32(&ms.qempty[buf]), ((seg >> 1) & 1) ^ 1, abort);
                const uint32_t to = s0 + L::Q0 + buf * L::QSTEP + (ch >> 3) * NQ * 128;
#pragma unroll 2
                for (int r = r0; r < NQ; r += RPI) {
                    const bool in = n < g.nn && wide && SV_INB(src - P.q, (int64_t)P.B * P.N * P.q_row, 1105);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                                 "l"(in ? src : P.q), "r"(in ? 16 : 0)
                                 : "memory");
                    // RPI rows on
                    n += step_n;
                    h += step_h;
                    src += src_step;
                    if (h >= P.G) h -= P.G, ++n, src += src_wrap;
                }
                ms.par[t] = (int8_t)p;
                if (t == 0) ms.code[buf] = ms.poison[buf] = 0;
                if (group_or(2, 64, !ok)) break;
                if (wrong) ms.code[buf] = 1;
                unsigned long long path = 0;
                if (t < g.nn) {
                    if (P.parents)
                        for (int a = t; a >= 0; a = ms.par[a]) path |= 1ull << a;
                    else
                        path = ~0ull >> (63 - t);
                }
                ms.desc[buf][t] = path;
                group_sync(2, 64);
                // A thread takes a column; its node's path says which nodes it sees.
                const unsigned node = (g.qt * NQ + t) / (unsigned)P.G;
                path = t < NQ && (int)node < g.nn ? ms.desc[buf][node] : 0;
                group_sync(2, 64);
#pragma unroll 4
                for (int a = 0; a < g.nn; ++a) {
                    const unsigned see = __ballot_sync(0xffffffffu, (path >> a) & 1);
                    if (lane == (a & 31)) reinterpret_cast<uint32_t *>(&ms.desc[buf][a])[warp & 1] = see;
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                tc::fence_async_smem();
                tc::bar_arrive(tc::smem_u32(&ms.qfull[buf]));
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            // ---- softmax: one position of a tile and a share of its columns per thread -------
            constexpr int CW = NQ / WG;
            const int t = tid & 127, wq = warp & 3, wg = (warp - 8) >> 2, bar = 4 + wg;
            const int col0 = wg * CW;
            const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16) + col0;
            // A reference's exponent, negated: what is added to a score times the scale.
            auto minus = [&](float ref) { return ref == -INFINITY ? 0.f : fmaf(-ref, P.scale_log2, lift(BF)); };
            const uint64_t scale2 = sv::f2(P.scale_log2, P.scale_log2);
            uint64_t raw[CW / 2], rnd[CW / 2];  // this position's share of the columns' sums
            int k = 0, seg = -1;
            bool fail = false;
            Seg g = {};
            for (;;) {
                const bool got = take(g);
                if (group_or(bar, 128, !got || fail) || g.kind == 3) break;
                const int row0 = g.qt * NQ + col0, n0 = row0 / P.G, h0 = row0 - n0 * P.G;
                if (g.kind) {
                    // Nothing to read: zeros where the request has no nodes, NaN where its lengths are wrong.
                    const bool nan = g.kind == 2;
                    for (int c = 0, n = n0, h = h0; c < CW && n < P.N; ++c) {
                        const int64_t row = ((int64_t)g.b * P.N + n) * P.Hq + g.h * P.G + h;
                        if (t < P.D && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1106))
                            P.out[row * P.D + t] = nan ? (uint16_t)Half2<BF>::NAN2 : 0;
                        if (t == 0 && P.lse) P.lse[row] = nan ? NAN : -INFINITY;
                        if (++h == P.G) h = 0, ++n;
                    }
                    if (nan && t == 0 && P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_BAD_KV_POSITION);
                    continue;
                }
                ++seg;
                const int buf = seg & 1, len = g.c + g.nn;
                bool fresh = true;  // some column has no reference yet, or one from FAR on: they move in every tile
                fail |= !tc::bar_wait(tc::smem_u32(&ms.qfull[buf]), (seg >> 1) & 1, abort);  // the tree's mask
#pragma unroll
                for (int c = 0; c < CW / 2; ++c) raw[c] = rnd[c] = 0;
                for (int j = g.j0; j < g.j1; ++j, ++k) {
                    const int sb = k & 1, pos = j * TILE + t;
                    const bool special = (j + 1) * TILE > g.c;  // holds nodes, or ends inside
                    fail |= !tc::bar_wait(tc::smem_u32(&ms.sfull[sb]), (k >> 1) & 1, abort);
                    tc::fence_after();
                    float x[CW];
                    tc::tmem_ld(lanes + sb * NQ, x);
                    unsigned vis = 0xffffffffu;  // the columns that see this position
                    if (special) {
                        vis = 0;
                        if (pos < g.c) {
                            vis = 0xffffffffu;
                        } else if (pos < len) {
                            vis = (unsigned)(ms.desc[buf][pos - g.c] >> col0);
                        }
                    }
                    tc::wait_ld(x);
                    // What this position's columns do not see is -inf.
                    auto mask = [&] {
                        if (special) {
#pragma unroll
                            for (int c = 0; c < CW; ++c) x[c] = (vis >> c) & 1 ? x[c] : -INFINITY;
                        }
                    };
                    mask();
                    // Exponents against the references.
                    auto exponents = [&] {
#pragma unroll
                        for (int c = 0; c < CW; c += 2) {
                            const float2 d = sv::f2_split(sv::f2_fma(sv::f2(x[c], x[c + 1]), scale2,
                                                                     *reinterpret_cast<const uint64_t *>(&ms.nref[col0 + c])));
                            x[c] = d.x;
                            x[c + 1] = d.y;
                        }
                    };
                    bool move = j == g.j0;  // a segment's first tile needs no vote
                    if (!move) {
                        exponents();
                        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                        for (int c = 4; c < CW; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
                        move = group_or(bar, 128, fresh || fail ||
                                                      fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > SLACK + lift(BF));
                    }
                    if (move) {
                        if (j > g.j0) {
                            if (group_or(bar, 128, fail)) break;
                            tc::tmem_ld(lanes + sb * NQ, x);
                            tc::wait_ld(x);
                            mask();
                        }
                        // Move the references to the columns' maxima.
                        float m = 0.f;
#pragma unroll
                        for (int c = 0; c < CW; ++c) {
                            const float y = warp_max(x[c]);
                            if (lane == c) m = y;
                        }
                        if (lane < CW) ms.red[wq][col0 + lane] = m;
                        group_sync(bar, 128);
                        bool slow = false;
                        if (t < CW) {
                            const int c = col0 + t;
                            m = fmaxf(fmaxf(ms.red[0][c], ms.red[1][c]), fmaxf(ms.red[2][c], ms.red[3][c]));
                            const float old = j == g.j0 ? -INFINITY : ms.ref[c];
                            const float now = fmaxf(m, old), add = minus(now);
                            const bool far = fabsf(add) >= FAR;
                            ms.ref[c] = now;
                            ms.off[c] = far ? now : 0.f;
                            ms.nref[c] = far ? lift(BF) : add;
                            ms.fac[c] = old == -INFINITY ? 0.f : ex2(add - minus(old));
                            slow = far || now == -INFINITY;
                        }
                        fresh = group_or(bar, 128, slow);
                        if (j > g.j0) {
#pragma unroll
                            for (int c = 0; c < CW; c += 2) {
                                const uint64_t f = *reinterpret_cast<const uint64_t *>(&ms.fac[col0 + c]);
                                raw[c / 2] = sv::f2_mul(raw[c / 2], f);
                                rnd[c / 2] = sv::f2_mul(rnd[c / 2], f);
                            }
                            // The accumulators follow, once the products before have come to an end.
                            fail |= !tc::bar_wait(tc::smem_u32(&ms.pvdone), (k - 1) & 1, abort);
                            tc::fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < CW; c0 += 8) {
                                float o[8];
                                tc::tmem_ld(lanes + 2 * NQ + c0, o);
                                tc::wait_ld(o);
#pragma unroll
                                for (int c = 0; c < 8; ++c) o[c] *= ms.fac[col0 + c0 + c];
                                tc::tmem_st(lanes + 2 * NQ + c0, o);
                            }
                            tc::wait_st();
                        }
                        if (fresh) {
#pragma unroll
                            for (int c = 0; c < CW; ++c) x[c] -= ms.off[col0 + c];
                        }
                        exponents();
                    }
                    tc::fence_before();
                    tc::bar_arrive(tc::smem_u32(&ms.sempty[sb]));
                    // The weights, rounded to the values' type, go where the tile before's were read from; both
                    // sums go on.
                    if (k > 0) fail |= !tc::bar_wait(tc::smem_u32(&ms.pvdone), (k - 1) & 1, abort);
#pragma unroll
                    for (int ch = 0; ch < CW / 8; ++ch) {
                        uint32_t pk[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = ch * 8 + 2 * i;
                            const float a = ex2(x[c]), b = ex2(x[c + 1]);
                            pk[i] = Half2<BF>::pack(a, b);
                            const float2 r = Half2<BF>::unpack(pk[i]);
                            raw[c / 2] = sv::f2_add(raw[c / 2], sv::f2(a, b));
                            rnd[c / 2] = sv::f2_add(rnd[c / 2], sv::f2(r.x, r.y));
                        }
                        *reinterpret_cast<uint4 *>(smem + L::P0 + t * 128 + (((col0 / 8 + ch) ^ (t & 7)) << 4)) =
                            make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    if (wg < 2 && special && pos >= g.c && pos < len) {
                        // A weight of 0 does not undo an infinity or a NaN: what is not finite in a node's
                        // values is set aside, and its readers get it at the segment's end.
                        const int u = 2 * k + 1;
                        fail |= !tc::bar_wait(tc::smem_u32(&ms.full[u % NU]), (u / NU) & 1, abort);
                        // An exponent of all ones carries into the sign's place.
                        constexpr uint32_t EXP2 = Half2<BF>::EXP_MASK * 0x10001u;
                        constexpr uint32_t ONE2 = (0x8000u - Half2<BF>::EXP_MASK) * 0x10001u;
                        unsigned char *const at = smem + (u % NU) * L::UNIT + t * 128 +
                                                  (HALVES > 1 ? wg * TILE * 128 : wg * 64);
                        constexpr int CHS = DP / 16;
                        uint32_t carry = 0;
#pragma unroll
                        for (int ch = 0; ch < CHS; ++ch) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(at + ch * 16);
                            carry |= ((y.x & EXP2) + ONE2) | ((y.y & EXP2) + ONE2) | ((y.z & EXP2) + ONE2) | ((y.w & EXP2) + ONE2);
                        }
                        const bool odd = carry & 0x80008000u;
                        if (odd)
#pragma unroll 1
                            for (int e = 0; e < CHS * 4; ++e) {
                                uint32_t *w = reinterpret_cast<uint32_t *>(at) + e, y = *w;
                                if ((y & Half2<BF>::EXP_MASK) == Half2<BF>::EXP_MASK) y &= 0xffff0000u;
                                if (((y >> 16) & Half2<BF>::EXP_MASK) == Half2<BF>::EXP_MASK) y &= 0xffffu;
                                *w = y;
                            }
                        if (odd) *(volatile int *)&ms.poison[buf] = 1;
                    }
                    tc::fence_async_smem();
                    tc::fence_before();
                    tc::bar_arrive(tc::smem_u32(&ms.pfull));
                }

                // ---- the segment's end: join the columns' sums, write rows or a part -----------
                auto column_totals = [&](const uint64_t (&pairs)[CW / 2], float *to) {
                    float y[CW];
#pragma unroll
                    for (int c = 0; c < CW; c += 2) {
                        const float2 f = sv::f2_split(pairs[c / 2]);
                        y[c] = f.x;
                        y[c + 1] = f.y;
                    }
                    const float total = column_sum<CW>(y, lane);
                    if (lane < CW) to[lane] = total;
                };
                column_totals(raw, &ms.red[wq][col0]);
                column_totals(rnd, &ms.red2[wq][col0]);
                group_sync(bar, 128);
                // While the last products run, a thread t < CW says what there is to say of column t.
                const int raise = *(volatile int *)&ms.bad[wg][seg % FLAGS] ? SPEC_VERIFY_DEV_BAD_KV_SLOT
                                  : ms.code[buf]                            ? SPEC_VERIFY_DEV_BAD_TREE
                                                                            : 0;
                float *const part = P.parts + (int64_t)g.part * part_floats<NQ>();
                if (t < CW) {
                    float sum = 0.f, rsum = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        sum += ms.red[w][col0 + t];
                        rsum += ms.red2[w][col0 + t];
                    }
                    if (g.part < 0) {
                        ms.fac[col0 + t] = raise ? NAN : 1.f / rsum;
                        const int nt = (row0 + t) / P.G;
                        if (nt < P.N && P.lse) {
                            const int64_t row = ((int64_t)g.b * P.N + nt) * P.Hq + g.h * P.G + row0 + t - nt * P.G;
                            if (SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1109))
                                P.lse[row] = raise ? NAN : nt < g.nn ? (log2f(sum) - minus(ms.ref[col0 + t])) * 0.69314718f : -INFINITY;
                        }
                    } else {
                        float *r = part + NQ * MAXD + col0 + t;
                        r[0] = ms.ref[col0 + t] == -INFINITY ? -INFINITY : -minus(ms.ref[col0 + t]);
                        r[NQ] = raise ? NAN : sum;
                        r[2 * NQ] = raise ? NAN : rsum;
                    }
                }
                if (k > 0) fail |= !tc::bar_wait(tc::smem_u32(&ms.pvdone), (k - 1) & 1, abort);
                if (group_or(bar, 128, fail)) break;
                tc::fence_after();
                float o[CW];
                tc::tmem_ld(lanes + 2 * NQ, o);
                tc::wait_ld(o);
                if (*(volatile int *)&ms.poison[buf] && t < P.D) {
                    const int from = g.j0 * TILE, to = len < g.j1 * TILE ? len : g.j1 * TILE;
                    for (int y = from > g.c ? from : g.c; y < to; ++y) {
                        const int64_t st = (int64_t)g.b * P.max_pos + y;
                        const int slot = SV_INB(st, (int64_t)P.B * P.max_pos, 1107) ? P.slot_table[st] : -1;
                        if (slot < 0 || slot >= P.num_slots) continue;
                        const uint32_t bits = P.v[(int64_t)slot * P.v_slot + g.h * P.D + t];
                        if ((bits & Half2<BF>::EXP_MASK) != Half2<BF>::EXP_MASK) continue;
                        const float val = Half2<BF>::unpack(bits).x;
                        const unsigned see = (unsigned)(ms.desc[buf][y - g.c] >> col0);
#pragma unroll
                        for (int c = 0; c < CW; ++c)
                            if ((see >> c) & 1) o[c] += val;
                    }
                }
                __syncwarp();
                if (lane == 0) tc::bar_arrive(tc::smem_u32(&ms.qempty[buf]));
                if (t == 0) {
                    if (raise && P.dev_status) atomicMax(P.dev_status, raise);
                    *(volatile int *)&ms.bad[wg][seg % FLAGS] = 0;
                }
                if (g.part < 0) {
                    uint16_t *out = P.out + (((int64_t)g.b * P.N + n0) * P.Hq + g.h * P.G + h0) * P.D + t;
                    const int64_t wrap = (int64_t)(P.Hq - P.G + 1) * P.D;  // to the next node's first head
                    const int cols = P.N * P.G - row0, live = g.nn * P.G - row0;  // columns that are rows; that are nodes'
                    const float rest = raise ? NAN : 0.f;
                    int h = h0;
                    if (t < P.D) {
#pragma unroll
                        for (int c = 0; c < CW; ++c) {
                            const float y = c < live ? o[c] * ms.fac[col0 + c] : rest;
                            if (c < cols && SV_INB(out - P.out, (int64_t)P.B * P.N * P.Hq * P.D, 1108))
                                *out = (uint16_t)Half2<BF>::pack(y, y);
                            const bool next = ++h == P.G;
                            h = next ? 0 : h;
                            out += next ? wrap : (int64_t)P.D;
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < CW; ++c) part[(col0 + c) * MAXD + t] = o[c];
                    // Every warpgroup of every CTA comes to the segment's counter; the last one's CTA joins the parts.
                    // The part that a run begins with is there early, so that it seldom joins two at its end.
                    group_sync(bar, 128);
                    if (t == 0 && !fail) {
                        const int parts = g.c1 - g.c0 + 1, size = group_size(parts), first = (cta - g.c0) / size * size;
                        const int n = parts - first < size ? parts - first : size;
                        unsigned *count = &P.counters[first ? COUNTERS + g.c0 + first : g.c0];
                        __threadfence();
                        if (atomicAdd(count, 1u) == (unsigned)(WG * n - 1)) {
                            __threadfence();
                            *count = 0;
                            ms.join[cta == g.c0] = {g, first, n, 1};
                            ms.joins[cta == g.c0] = 1;
                        }
                    }
                }
                // The references and factors are read until here; the next segment writes them anew.
            }

            // ---- the parts of which this CTA brought the last --------------------------------------
            const bool off = group_or(3, 128 * WG, *abort != 0);
            for (int end = 0; end < 2; ++end)  // the run's beginning, its end
                while (ms.joins[end] && !off) {
                    // A thread takes four dimensions of IT columns, and one column's reference and sums; these
                    // go through the ring, which is done with.  The parts are added in their order, so the
                    // result does not depend on who joins.  A group's sum replaces its first part.
                    constexpr int WARPS = 4 * WG, IT = NQ / WARPS;
                    const Join &jn = ms.join[end];
                    g = jn.g;
                    const int parts = jn.n, t = tid - 256, d = (t & 31) * 4, c0 = t >> 5;  // columns c0, c0 + WARPS, ...
                    const bool all = g.c1 - g.c0 + 1 == parts || jn.step > 1;
                    float *const jm = reinterpret_cast<float *>(smem), *const jl = jm + parts * NQ, *const jr = jl + parts * NQ;
                    uint32_t *const jrow = reinterpret_cast<uint32_t *>(jr + parts * NQ);  // columns' rows of the output (2^32 would be 550 GB)
                    auto part_of = [&](int x) {
                        const int y = jn.first + x * jn.step;
                        return P.parts + (int64_t)(2 * (g.c0 + y) + (y == 0)) * part_floats<NQ>();
                    };
                    float4 y[2][IT], acc[IT];
                    auto load = [&](int x, float4 (&y)[IT]) {
                        if (x >= parts) return;
                        const float *part = part_of(x) + c0 * MAXD + d;
#pragma unroll
                        for (int i = 0; i < IT; ++i) y[i] = __ldcg(reinterpret_cast<const float4 *>(part + WARPS * i * MAXD));
                    };
                    auto add = [&](int x, const float4 (&y)[IT]) {
                        if (x >= parts) return;
#pragma unroll
                        for (int i = 0; i < IT; ++i) {
                            const float f = jm[x * NQ + c0 + WARPS * i];
                            if (f == 0.f) continue;
                            acc[i].x += f * y[i].x;
                            acc[i].y += f * y[i].y;
                            acc[i].z += f * y[i].z;
                            acc[i].w += f * y[i].w;
                        }
                    };
                    load(0, y[0]);
                    load(1, y[1]);
#pragma unroll 1
                    for (int e = t; e < parts * NQ; e += 128 * WG) {
                        const float *r = part_of(e / NQ) + NQ * MAXD + e % NQ;
                        jm[e] = __ldcg(r);
                        jl[e] = __ldcg(r + NQ);
                        jr[e] = __ldcg(r + 2 * NQ);
                    }
                    group_sync(3, 128 * WG);
                    if (t < NQ) {
                        float top = -INFINITY, sum = 0.f, rsum = 0.f;
#pragma unroll 1
                        for (int x = 0; x < parts; ++x) top = fmaxf(top, jm[x * NQ + t]);
#pragma unroll 1
                        for (int x = 0; x < parts; ++x) {
                            const float m = jm[x * NQ + t], l = jl[x * NQ + t];
                            // 0: the part's positions have no weight in this row
                            const float f = l == 0.f ? 0.f : ex2(m == -INFINITY ? 0.f : m - top);
                            if (l != 0.f) sum += f * l, rsum += f * jr[x * NQ + t];
                            jm[x * NQ + t] = f;
                        }
                        if (all) {
                            const int gr = g.qt * NQ + t, n = (int)((unsigned)gr / (unsigned)P.G);
                            const bool bad = sum != sum;
                            const int64_t row = ((int64_t)g.b * P.N + n) * P.Hq + g.h * P.G + gr - n * P.G;
                            ms.fac[t] = n < g.nn || bad ? 1.f / rsum : 0.f;
                            jrow[t] = n < P.N ? (uint32_t)row : ~0u;
                            if (n < P.N && P.lse && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1111))
                                P.lse[row] = n < g.nn || bad ? ((top == -INFINITY ? 0.f : top) + log2f(sum)) * 0.69314718f
                                                             : -INFINITY;
                        } else {
                            float *r = part_of(0) + NQ * MAXD + t;
                            r[0] = top;
                            r[NQ] = sum;
                            r[2 * NQ] = rsum;
                        }
                    }
                    group_sync(3, 128 * WG);
#pragma unroll
                    for (int i = 0; i < IT; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                    for (int x = 0; x < parts; x += 2) {
                        add(x, y[0]);
                        load(x + 2, y[0]);
                        add(x + 1, y[1]);
                        load(x + 3, y[1]);
                    }
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
                        const int c = c0 + WARPS * i;
                        if (!all) {
                            *reinterpret_cast<float4 *>(part_of(0) + c * MAXD + d) = acc[i];
                            continue;
                        }
                        const float inv = ms.fac[c];
                        uint2 y = make_uint2(0, 0);
                        if (inv != 0.f)
                            y = make_uint2(Half2<BF>::pack(acc[i].x * inv, acc[i].y * inv),
                                           Half2<BF>::pack(acc[i].z * inv, acc[i].w * inv));
                        const uint32_t row = jrow[c];
                        if (row != ~0u && d < P.D && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1110))
                            *reinterpret_cast<uint2 *>(P.out + (int64_t)row * P.D + d) = y;
                    }
                    group_sync(3, 128 * WG);
                    if (t == 0) {
                        // The last group's CTA goes on to join the groups.
                        ms.joins[end] = 0;
                        if (!all) {
                            const int size = group_size(g.c1 - g.c0 + 1), n = (g.c1 - g.c0) / size + 1;
                            unsigned *count = &P.counters[2 * COUNTERS + g.c0];
                            __threadfence();
                            if (atomicAdd(count, 1u) == (unsigned)(n - 1)) {
                                __threadfence();
                                *count = 0;
                                ms.join[end] = {g, 0, n, size};
                                ms.joins[end] = 1;
                            }
                        }
                    }
                    group_sync(3, 128 * WG);
                }
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (ms.abort) {
        // A bounded wait ran out: what is written is not an answer.  The products in flight end
        // (again with a limit) before their memory is given back; the copies were waited for.  A commit is
        // for the products of its own thread: the lane that issued them, which every election picks.
        if (warp == 4 && tc::elect()) {
            atomicAdd(&tc::g_timeouts, 1ull);
            const int64_t begin = clock64();
            tc::commit(tc::smem_u32(&ms.drain));
            while (!tc::bar_try(tc::smem_u32(&ms.drain), 0) && clock64() - begin < tc::WAIT_CLOCKS) {}
            if (P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_TIMEOUT);
        }
        __syncthreads();
    }
    if (warp == 4) tc::tmem_free(tmem, L::COLS);
}

// -------------------------------------------------------------------------------------------------
// Host side.
// -------------------------------------------------------------------------------------------------
struct DevInfo {
    int sms = 0;
};
static std::mutex g_mu;
static DevInfo g_dev[64];

template <bool BF, int NQ, int DP>
constexpr size_t smem_bytes()
{
    using L = Layout<NQ, DP>;
    return L::M0 + sizeof(Misc<NQ, L::NU>);
}

template <bool BF, int NQ, int DP>
static bool allow()
{
    static_assert(smem_bytes<BF, NQ, DP>() <= 232448, "shared memory of a CTA");
    return cudaFuncSetAttribute((const void *)attention_kernel<BF, NQ, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<BF, NQ, DP>()) == cudaSuccess;
}

// Once per device: the kernels' shared memory, the SM count.
static const DevInfo *device_info()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    DevInfo &d = g_dev[dev];
    if (d.sms == 0) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            !(allow<true, 16, 64>() && allow<true, 32, 64>() && allow<true, 64, 64>() && allow<true, 16, 128>() &&
              allow<true, 32, 128>() && allow<true, 64, 128>() && allow<false, 16, 64>() && allow<false, 32, 64>() &&
              allow<false, 64, 64>() && allow<false, 16, 128>() && allow<false, 32, 128>() && allow<false, 64, 128>())) {
            cudaGetLastError();
            return nullptr;
        }
        d.sms = sms;
    }
    return &d;
}

// Columns per CTA: the fewest of 16, 32, 64 that hold a key head's query rows, 64 at most (a
// wider call reads the cache once per 64 rows, the second time from L2).
static int columns(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

constexpr size_t COUNTER_BYTES = 65536 * 4;  // the workspace's fixed region of counters
constexpr float MAX_SCALE = 2.3e38f;         // times log2(e) it is still a number of fp32

template <bool BF, int NQ, int DP>
static cudaError_t launch(const Params &P, int grid, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads(NQ));
    cfg.dynamicSmemBytes = smem_bytes<BF, NQ, DP>();
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_kernel<BF, NQ, DP>, P);
}

template <bool BF>
static cudaError_t dispatch(int nq, int dp, const Params &P, int grid,
                            cudaStream_t s)
{
    if (dp == 64)
        return nq == 16 ? launch<BF, 16, 64>(P, grid, s)
               : nq == 32 ? launch<BF, 32, 64>(P, grid, s)
                          : launch<BF, 64, 64>(P, grid, s);
    return nq == 16 ? launch<BF, 16, 128>(P, grid, s)
           : nq == 32 ? launch<BF, 32, 128>(P, grid, s)
                      : launch<BF, 64, 128>(P, grid, s);
}

}  // namespace svatt

namespace sv {
bool attention_timeouts(unsigned long long &n) { return tc::read_timeouts(n); }
bool attention_wait_clocks(long long clocks) { return tc::set_wait_clocks(clocks); }

// This module's first range violation (debug builds; 0 otherwise), cleared when read.
unsigned long long attention_debug_fault()
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

extern "C" size_t spec_verify_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int max_pos)
{
    if (B < 1 || B > 65536 || N < 1 || N > sv::MAX_TREE || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq > (1 << 16) || D < 64 ||
        D > svatt::MAXD || D % 16 || max_pos < 1)
        return 0;
    const size_t nq = (size_t)svatt::columns(N * (Hq / Hkv));
    return svatt::COUNTER_BYTES + 2 * svatt::MAX_SMS * svatt::ctas_per_sm((int)nq) * (nq * svatt::MAXD + 3 * nq) * sizeof(float);
}

extern "C" int spec_verify_attention(const void *q, int dtype, int64_t q_stride, const void *k_cache,
                                     const void *v_cache, int64_t num_slots, int64_t k_slot_stride,
                                     int64_t v_slot_stride, const int32_t *slot_table, int max_pos,
                                     const int32_t *committed, const int32_t *parents, const int32_t *num_nodes, int B,
                                     int N, int Hq, int Hkv, int D, float scale, void *out, float *lse, void *workspace,
                                     size_t ws_bytes, int32_t *dev_status, void *stream)
{
    using namespace svatt;
    if (!q || !k_cache || !v_cache || !slot_table || !committed || !out || !workspace) return SPEC_VERIFY_EINVAL;
    if (dtype != SPEC_VERIFY_BF16 && dtype != SPEC_VERIFY_FP16) return SPEC_VERIFY_EINVAL;
    const size_t need = spec_verify_attention_workspace_bytes(B, N, Hq, Hkv, D, max_pos);
    if (!need || num_slots < 1 || num_slots > 0x7fffffff || !(scale > 0.f) || scale > MAX_SCALE) return SPEC_VERIFY_EINVAL;
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hkv * D;
    if (q_stride % 8 || k_slot_stride % 8 || v_slot_stride % 8 || q_stride < qw || k_slot_stride < kw || v_slot_stride < kw ||
        k_slot_stride >= (1ll << 31) || v_slot_stride >= (1ll << 31))
        return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) % 16) return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)slot_table | (uintptr_t)committed | (uintptr_t)parents | (uintptr_t)num_nodes | (uintptr_t)lse |
         (uintptr_t)dev_status) % 4)
        return SPEC_VERIFY_EINVAL;
    if (ws_bytes < need || (uintptr_t)workspace % 256) return SPEC_VERIFY_EWORKSPACE;
    const DevInfo *dev = device_info();
    if (!dev) return SPEC_VERIFY_ECUDA;
    const bool bf = dtype == SPEC_VERIFY_BF16;
    Params P;
    P.q = static_cast<const uint16_t *>(q);
    P.k = static_cast<const uint16_t *>(k_cache);
    P.v = static_cast<const uint16_t *>(v_cache);
    P.out = static_cast<uint16_t *>(out);
    P.lse = lse;
    P.q_row = q_stride;
    P.k_slot = k_slot_stride;
    P.v_slot = v_slot_stride;
    P.num_slots = num_slots;
    P.slot_table = slot_table;
    P.committed = committed;
    P.parents = parents;
    P.num_nodes = num_nodes;
    P.max_pos = max_pos;
    P.B = B;
    P.N = N;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.D = D;
    P.G = Hq / Hkv;
    const int nq = columns(N * P.G);
    P.QT = (N * P.G + nq - 1) / nq;
    P.scale_log2 = (float)((double)scale * 1.4426950408889634);
    P.dev_status = dev_status;
    P.counters = static_cast<unsigned *>(workspace);
    P.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + COUNTER_BYTES);
    int grid = (dev->sms < MAX_SMS ? dev->sms : MAX_SMS) * ctas_per_sm(nq);
    const int64_t most = (int64_t)B * Hkv * P.QT * ((max_pos + TILE - 1) / TILE);
    if (most < grid) grid = (int)most;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int dp = D <= 64 ? 64 : 128;
    const cudaError_t e = bf ? dispatch<true>(nq, dp, P, grid, s) : dispatch<false>(nq, dp, P, grid, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SPEC_VERIFY_ECUDA;
    }
    return SPEC_VERIFY_OK;
}
