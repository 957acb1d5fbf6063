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
// One CTA per SM takes an equal run of the batch's tiles (a tile: 128 positions of one request and
// key head), whatever the lengths, so one long request is split over all SMs and many short ones
// share them; where a run cuts a request, the parts are joined by the CTA that finishes last.
// Warp 0 gathers tiles by their slots with TMA (four rows per copy), warp 1 issues the products,
// warps 2-3 stage the queries and the tree's mask, warps 4-7 hold a position per thread: a tile's
// scores come to them as columns, so the exponentials are spread evenly however few the query rows.
//
// The softmax's reference moves only when a score passes it by more than 2^8 (a vote of the 128
// threads per tile): the weights are then at most 2^8, exact in fp32 as in 16 bits up to their
// rounding, and the accumulators are left alone in nearly every tile.
#include <cuda.h>

#include <mutex>

#include "sv_ops.cuh"
#include "sv_tc.cuh"

namespace svatt {

using sv::Half2;

constexpr int NT = 256;
constexpr int TILE = 128;     // positions per tile
constexpr int MAXD = 128;
constexpr int MAX_CTAS = 256; // parts the workspace has room for: two per CTA
constexpr int FLAGS = 16;     // segments whose bad-slot flags are in use at once (more than stages + 2)
constexpr float SLACK = 8.f;  // log2 of the largest weight

struct Params {
    const uint16_t *q, *v;
    uint16_t *out;
    float *lse;
    int64_t q_row, v_slot, num_slots;
    const int32_t *slot_table, *committed, *parents, *num_nodes;
    int max_pos, B, N, Hq, Hkv, D, G, QT;  // G query heads per key head, QT column blocks
    float scale_log2;
    int32_t *dev_status;
    unsigned *counters;  // [CTAs] arrivals at the join of the segment that CTA began
    float *parts;
};

// Shared memory after the tiles, whose bases are multiples of 1024 bytes.
template <int NQ, int DP>
struct Layout {
    static constexpr int HALVES = DP / 64;
    static constexpr int UNIT = TILE * DP * 2;                  // bytes of a K or V tile
    static constexpr int NS = (NQ <= 32 ? 3 : 2) * 128 / DP;    // stages
    static constexpr int QBYTES = NQ * DP * 2;
    static constexpr int QSTEP = QBYTES < 1024 ? 1024 : QBYTES;
    static constexpr int PBYTES = TILE * 128;                   // P: a row of 64 columns per position
    static constexpr int K0 = 0, V0 = NS * UNIT, Q0 = 2 * NS * UNIT, P0 = Q0 + 2 * QSTEP;
    static constexpr int M0 = P0 + PBYTES;                      // Misc
    static constexpr int COLS = 3 * NQ <= 64 ? 64 : 3 * NQ <= 128 ? 128 : 256;  // TMEM columns
};

template <int NQ, int NS>
struct Misc {
    uint64_t kfull[NS], kempty[NS], vfull[NS], vempty[NS];
    uint64_t sfull[2], sempty[2], qfull[2], qempty[2], pfull, pvdone, drain;
    unsigned long long desc[2][sv::MAX_TREE];  // nodes that see node a, of the staged queries' request
    float nref[NQ], fac[NQ], red[4][NQ], sum[2][NQ];
    int code[2];
    int bad[FLAGS];
    int8_t par[sv::MAX_TREE];
    int begin_b, abort, issued[2];  // tiles of K and V asked for
    int64_t begin_base, scan[NT / 32];
    uint32_t tmem;
    struct {
        int on, b, h, qt, c0, c1, first0;
    } join[2];
};

// A CTA's walk over its tiles.  Every role keeps one of its own.
struct Walk {
    int b, item, j, ntile, c, nn;
    int dummy;  // nothing to attend with: the request has no nodes here, or its lengths are wrong

    __device__ __forceinline__ void load(const Params &P)
    {
        c = SV_INB(b, P.B, 1101) ? P.committed[b] : 0;
        nn = P.num_nodes ? (SV_INB(b, P.B, 1102) ? P.num_nodes[b] : 0) : P.N;
        const bool fault = nn < 0 || nn > P.N || c < 0 || (int64_t)c + nn > P.max_pos;
        dummy = fault ? 2 : nn == 0 ? 1 : 0;
        ntile = dummy ? 1 : (c + nn + TILE - 1) / TILE;
    }
    __device__ __forceinline__ void start(const Params &P, int b0, int64_t skip)
    {
        b = b0;
        load(P);
        item = (int)(skip / ntile);
        j = (int)(skip - (int64_t)item * ntile);
    }
    __device__ __forceinline__ void next(const Params &P)
    {
        if (++j < ntile) return;
        j = 0;
        if (++item < P.Hkv * P.QT) return;
        item = 0;
        if (++b < P.B) load(P);
    }
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

// Sums over the warp's lanes of NQ values per lane: halving exchanges leave column sums in the
// lanes (31 shuffles for 32 columns instead of 5 for each).  sum[c] of columns c of v.
template <int NQ>
__device__ __forceinline__ void column_sums(float (&v)[NQ], float *sum, int lane)
{
    constexpr int W = NQ < 32 ? NQ : 32;
#pragma unroll
    for (int base = 0; base < NQ; base += W) {
        float x[W];
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = v[base + i];
#pragma unroll
        for (int half = W / 2; half; half >>= 1) {
            const bool up = lane & half;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float keep = up ? x[i + half] : x[i], give = up ? x[i] : x[i + half];
                x[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
            }
        }
        if (W < 32) x[0] += __shfl_xor_sync(0xffffffffu, x[0], 16);
        if (lane < W) sum[base + lane] = x[0];
    }
}

// Floats of one part: per column the weighted values, then references, sums, sums of the rounded
// weights.
template <int NQ>
__host__ __device__ constexpr int part_floats()
{
    return NQ * MAXD + 3 * NQ;
}

// The CTA whose run holds tile x, and a run's first tile.
__device__ __forceinline__ int cta_of(int64_t x, int64_t total, int G) { return (int)(((x + 1) * G - 1) / total); }
__device__ __forceinline__ int64_t run_begin(int c, int64_t total, int G) { return total * c / G; }

template <bool BF, int NQ, int DP>
__global__ void __launch_bounds__(NT, 1) attention_kernel(const __grid_constant__ CUtensorMap kmap,
                                                          const __grid_constant__ CUtensorMap vmap, const Params P)
{
    using L = Layout<NQ, DP>;
    using M = Misc<NQ, L::NS>;
    constexpr int NS = L::NS, HALVES = L::HALVES;
    extern __shared__ __align__(1024) unsigned char smem[];
    M &ms = *reinterpret_cast<M *>(smem + L::M0);
    const uint32_t s0 = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    volatile int *abort = &ms.abort;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            tc::bar_init(tc::smem_u32(&ms.kfull[s]), 1);
            tc::bar_init(tc::smem_u32(&ms.kempty[s]), 1);
            tc::bar_init(tc::smem_u32(&ms.vfull[s]), 1);
            tc::bar_init(tc::smem_u32(&ms.vempty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_u32(&ms.sfull[i]), 1);
            tc::bar_init(tc::smem_u32(&ms.sempty[i]), 128);
            tc::bar_init(tc::smem_u32(&ms.qfull[i]), 64);
            tc::bar_init(tc::smem_u32(&ms.qempty[i]), 2);
            ms.join[i].on = 0;
        }
        tc::bar_init(tc::smem_u32(&ms.pfull), 128);
        tc::bar_init(tc::smem_u32(&ms.pvdone), 1);
        tc::bar_init(tc::smem_u32(&ms.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ms.abort = ms.issued[0] = ms.issued[1] = 0;
        tc::tma_prefetch_map(&kmap);
        tc::tma_prefetch_map(&vmap);
    }
    if (tid < FLAGS) ms.bad[tid] = 0;
    if (warp == 1) tc::tmem_alloc(tc::smem_u32(&ms.tmem), L::COLS);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The batch's tiles, and the request that this CTA's run begins in.
    const int HT = P.Hkv * P.QT;
    const int per = (P.B + NT - 1) / NT;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i) {
        Walk w;
        w.b = tid * per + i;
        if (w.b >= P.B) break;
        w.load(P);
        mine += (int64_t)w.ntile * HT;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) ms.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += ms.scan[w];
        total += ms.scan[w];
    }
    // Every run holds a tile: a batch of fewer tiles than CTAs leaves the last CTAs out.
    const int G = total < (int64_t)gridDim.x ? (int)total : (int)gridDim.x;
    const int64_t t0 = cta < G ? run_begin(cta, total, G) : total, t1 = cta < G ? run_begin(cta + 1, total, G) : total;
    if (t0 >= before && t0 < before + mine) {
        Walk w;
        int64_t at = before;
        for (w.b = tid * per; w.b < P.B; ++w.b) {
            w.load(P);
            if (t0 < at + (int64_t)w.ntile * HT) break;
            at += (int64_t)w.ntile * HT;
        }
        ms.begin_b = w.b;
        ms.begin_base = at;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ms.tmem;
    const int64_t count = t1 - t0;

    if (count > 0) {
        Walk w;
        w.start(P, ms.begin_b, t0 - ms.begin_base);
        if (warp == 0) {
            // ---- tiles into shared memory -------------------------------------------------
            // A lane owns positions 4 lane .. 4 lane + 3 of every tile; their slots are read one
            // tile ahead, so the table's latency lies under the wait for a free stage.
            int slot[4], seg = -1;
            bool ok = true;
            auto slots_of = [&](const Walk &x) {
                const int len = x.c + x.nn;
                bool bad = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int pos = x.j * TILE + 4 * lane + i;
                    slot[i] = 0;
                    if (!x.dummy && pos < len) {
                        const int64_t at = (int64_t)x.b * P.max_pos + pos;
                        const int s = SV_INB(at, (int64_t)P.B * P.max_pos, 1103) ? P.slot_table[at] : -1;
                        bad |= s < 0 || s >= P.num_slots;
                        slot[i] = s < 0 || s >= P.num_slots ? 0 : s;
                    }
                }
                return bad;
            };
            bool bad = slots_of(w);
            int k = 0, kissued = 0;
            for (int64_t i = 0; i < count; ++i) {
                if (!w.dummy) {
                    if (seg < 0 || w.j == 0) ++seg;
                    const int s = k % NS, ph = (k / NS) & 1;
                    const int len = w.c + w.nn - w.j * TILE;
                    const int groups = len >= TILE ? TILE / 4 : (len + 3) / 4;
                    const uint32_t bytes = (uint32_t)groups * 4 * DP * 2;
                    const int x = (w.item / P.QT) * P.D;
                    const bool any = __any_sync(0xffffffffu, bad);
                    if (any && lane == 0) *(volatile int *)&ms.bad[seg % FLAGS] = 1;
                    if (lane == 0 && k >= NS) ok = tc::bar_wait(tc::smem_u32(&ms.kempty[s]), ph ^ 1, abort);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    const uint32_t kb = tc::smem_u32(&ms.kfull[s]), vb = tc::smem_u32(&ms.vfull[s]);
                    ++kissued;
                    if (lane == 0) tc::bar_expect(kb, bytes);
                    __syncwarp();
                    if (lane < groups)
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
                            tc::tma_gather4(s0 + L::K0 + s * L::UNIT + hf * TILE * 128 + lane * 512, &kmap, kb,
                                            x + hf * 64, slot);
                    if (lane == 0 && k >= NS) ok = tc::bar_wait(tc::smem_u32(&ms.vempty[s]), ph ^ 1, abort);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) tc::bar_expect(vb, bytes);
                    __syncwarp();
                    if (lane < groups)
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
                            tc::tma_gather4(s0 + L::V0 + s * L::UNIT + hf * TILE * 128 + lane * 512, &vmap, vb,
                                            x + hf * 64, slot);
                    ++k;
                }
                if (i + 1 < count) {
                    w.next(P);
                    bad = slots_of(w);
                }
            }
            if (lane == 0) ms.issued[0] = kissued, ms.issued[1] = k;
        } else if (warp == 1) {
            // ---- products ------------------------------------------------------------------
            if (lane == 0) {
                constexpr uint32_t ID_S = tc::instr_desc(BF, false, false, 128, NQ);
                constexpr uint32_t ID_O = tc::instr_desc(BF, true, true, 128, NQ);
                const int dsteps = P.D / 16;
                int k = 0, seg = -1, psteps = 0, pstart = 0;
                bool ok = true;
                auto weigh = [&](int t) {  // O^T (+)= V^T P^T of tile t
                    const int s = t % NS;
                    ok = tc::bar_wait(tc::smem_u32(&ms.pfull), t & 1, abort) &&
                         tc::bar_wait(tc::smem_u32(&ms.vfull[s]), (t / NS) & 1, abort);
                    if (!ok) return;
                    tc::fence_after();
                    for (int i = 0; i < psteps; ++i)
                        tc::mma_f16(tmem + 2 * NQ,
                                    tc::smem_desc(s0 + L::V0 + s * L::UNIT + i * 2048, HALVES > 1 ? TILE * 128 : 0, 1024),
                                    tc::smem_desc(s0 + L::P0 + i * 2048, 0, 1024), ID_O, !pstart || i > 0);
                    tc::commit(tc::smem_u32(&ms.vempty[s]));
                    tc::commit(tc::smem_u32(&ms.pvdone));
                };
                bool begun = false;
                for (int64_t i = 0; i < count && ok; ++i) {
                    if (!w.dummy) {
                        const bool start = !begun || w.j == 0;
                        if (start) {
                            ++seg;
                            begun = true;
                            if (!tc::bar_wait(tc::smem_u32(&ms.qfull[seg & 1]), (seg >> 1) & 1, abort)) break;
                        }
                        const int s = k % NS, sb = k & 1;
                        ok = tc::bar_wait(tc::smem_u32(&ms.kfull[s]), (k / NS) & 1, abort);
                        if (ok && k >= 2) ok = tc::bar_wait(tc::smem_u32(&ms.sempty[sb]), ((k >> 1) & 1) ^ 1, abort);
                        if (!ok) break;
                        tc::fence_after();
                        for (int d = 0; d < dsteps; ++d)
                            tc::mma_f16(tmem + sb * NQ,
                                        tc::smem_desc(s0 + L::K0 + s * L::UNIT + (d >> 2) * TILE * 128 + (d & 3) * 32, 0, 1024),
                                        tc::smem_desc(s0 + L::Q0 + (seg & 1) * L::QSTEP + (d >> 2) * NQ * 128 + (d & 3) * 32,
                                                      0, 1024),
                                        ID_S, d > 0);
                        tc::commit(tc::smem_u32(&ms.kempty[s]));
                        tc::commit(tc::smem_u32(&ms.sfull[sb]));
                        const bool end = i + 1 == count || w.j + 1 == w.ntile;
                        if (end) tc::commit(tc::smem_u32(&ms.qempty[seg & 1]));
                        if (k > 0) weigh(k - 1);
                        const int left = w.c + w.nn - w.j * TILE;
                        psteps = left >= TILE ? TILE / 16 : (left + 15) / 16;
                        pstart = start;
                        ++k;
                    }
                    w.next(P);
                }
                if (ok && k > 0 && !*abort) weigh(k - 1);
            }
            __syncwarp();
        } else if (warp < 4) {
            // ---- queries and the tree's mask -----------------------------------------------
            const int t = tid - 64;
            int seg = -1;
            bool ok = true;
            for (int64_t i = 0; i < count;) {
                if (!w.dummy) {
                    ++seg;
                    const int buf = seg & 1;
                    if (seg >= 2) ok = tc::bar_wait(tc::smem_u32(&ms.qempty[buf]), ((seg >> 1) & 1) ^ 1, abort);
                    if (group_or(2, 64, !ok)) break;
                    // Which nodes see node a: every node's path to the root, then transposed.
                    bool wrong = false;
                    int p = t - 1;
                    if (P.parents && t < w.nn) {
                        const int64_t at = (int64_t)w.b * P.N + t;
                        p = SV_INB(at, (int64_t)P.B * P.N, 1104) ? P.parents[at] : -1;
                        wrong = t == 0 ? p != -1 : (p < 0 || p >= t);
                        if (wrong) p = -1;
                    }
                    if (t == 0) ms.code[buf] = 0;
                    ms.par[t] = (int8_t)p;
                    const int h = w.item / P.QT, qt = w.item % P.QT;
                    constexpr int CH = DP / 8;  // 16-byte chunks of a row
                    for (int e = t; e < NQ * CH; e += 64) {
                        const int r = e / CH, ch = e - r * CH, g = qt * NQ + r, n = g / P.G;
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (n < w.nn && ch * 8 < P.D) {
                            const int64_t at = ((int64_t)w.b * P.N + n) * P.q_row + (int64_t)(h * P.G + g - n * P.G) * P.D +
                                               ch * 8;
                            if (SV_INB(at, (int64_t)P.B * P.N * P.q_row, 1105))
                                x = *reinterpret_cast<const uint4 *>(P.q + at);
                        }
                        *reinterpret_cast<uint4 *>(smem + L::Q0 + buf * L::QSTEP + (ch >> 3) * NQ * 128 + r * 128 +
                                                   (((ch & 7) ^ (r & 7)) << 4)) = x;
                    }
                    tc::fence_async_smem();
                    group_sync(2, 64);
                    if (wrong) ms.code[buf] = 1;
                    unsigned long long path = 0;
                    if (t < w.nn) {
                        if (P.parents)
                            for (int n = t; n >= 0; n = ms.par[n]) path |= 1ull << n;
                        else
                            path = ~0ull >> (63 - t);
                    }
                    ms.desc[buf][t] = path;
                    group_sync(2, 64);
                    unsigned long long see = 0;
                    for (int n = t; n < w.nn; ++n) see |= ((ms.desc[buf][n] >> t) & 1ull) << n;
                    group_sync(2, 64);
                    ms.desc[buf][t] = see;
                    tc::bar_arrive(tc::smem_u32(&ms.qfull[buf]));
                }
                // On to the next segment.
                const int64_t step = w.ntile - w.j;
                i += step;
                w.j = w.ntile - 1;
                if (i < count) w.next(P);
            }
        } else {
            // ---- softmax: one position of a tile per thread ---------------------------------
            const int t = tid - 128, wq = warp - 4;
            const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
            constexpr int NC = NQ / 16;
            float raw[NQ], rnd[NQ];  // this position's share of the columns' sums
            int k = 0, seg = -1, pv = 0;  // seg: segments with something to attend with
            bool begun = false, fail = false, fresh = true;
            int first_j = 0, poison = 0;
            for (int64_t i = 0; i < count; ++i) {
                const bool start = !begun || w.j == 0, end = i + 1 == count || w.j + 1 == w.ntile;
                begun = true;
                const int h = w.item / P.QT, qt = w.item % P.QT;
                if (w.dummy) {
                    // Nothing to read: zeros where the request has no nodes, NaN where its lengths are wrong.
                    const bool nan = w.dummy == 2;
                    for (int col = 0; col < NQ; ++col) {
                        const int g = qt * NQ + col, n = g / P.G;
                        if (n >= P.N) break;
                        const int64_t row = ((int64_t)w.b * P.N + n) * P.Hq + h * P.G + g - n * P.G;
                        if (t < P.D && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1106))
                            P.out[row * P.D + t] = nan ? (uint16_t)Half2<BF>::NAN2 : 0;
                        if (t == 0 && P.lse) P.lse[row] = nan ? NAN : -INFINITY;
                    }
                    if (nan && t == 0 && P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_BAD_KV_POSITION);
                    w.next(P);
                    continue;
                }
                if (start) {
                    ++seg;
                    first_j = w.j;
                    poison = 0;
                    fresh = true;
#pragma unroll
                    for (int c = 0; c < NQ; ++c) raw[c] = rnd[c] = 0.f;
                    fail |= !tc::bar_wait(tc::smem_u32(&ms.qfull[seg & 1]), (seg >> 1) & 1, abort);
                }
                const int sb = k & 1, s = k % NS;
                const int pos = w.j * TILE + t, len = w.c + w.nn;
                const bool special = (w.j + 1) * TILE > w.c;  // holds nodes, or ends inside
                unsigned long long vis = ~0ull;               // the columns that see this position
                if (special) {
                    if (pos >= len) {
                        vis = 0;
                    } else if (pos >= w.c) {
                        const unsigned long long see = ms.desc[seg & 1][pos - w.c];
                        vis = 0;
                        int n = qt * NQ / P.G, g = qt * NQ - n * P.G;
                        for (int c = 0; c < NQ; ++c) {
                            if (n < w.nn) vis |= ((see >> n) & 1ull) << c;
                            if (++g == P.G) g = 0, ++n;
                        }
                    }
                }
                fail |= !tc::bar_wait(tc::smem_u32(&ms.sfull[sb]), (k >> 1) & 1, abort);
                tc::fence_after();
                float x[NC][16];
#pragma unroll
                for (int c = 0; c < NC; ++c) tc::tmem_ld16(lanes + sb * NQ + c * 16, x[c]);
                tc::wait_ld(x);
                tc::fence_before();
                tc::bar_arrive(tc::smem_u32(&ms.sempty[sb]));
                bool over = fresh | fail;
#pragma unroll
                for (int c = 0; c < NQ; ++c) {
                    const float d = fmaf(x[c / 16][c % 16], P.scale_log2, ms.nref[c]);
                    over |= d > SLACK && ((vis >> c) & 1);
                }
                if (group_or(1, 128, over)) {
                    if (group_or(1, 128, fail)) break;
                    // Move the references to the columns' maxima.
#pragma unroll
                    for (int c = 0; c < NQ; ++c) {
                        const float y = (vis >> c) & 1 ? x[c / 16][c % 16] * P.scale_log2 : -INFINITY;
                        const float m = warp_max(y);
                        if (lane == 0) ms.red[wq][c] = m;
                    }
                    group_sync(1, 128);
                    bool none = false;
                    if (t < NQ) {
                        const float m = fmaxf(fmaxf(ms.red[0][t], ms.red[1][t]), fmaxf(ms.red[2][t], ms.red[3][t]));
                        const float old = start ? -INFINITY : ms.sum[0][t];  // the reference, -inf: none yet
                        const float to = fmaxf(m, old);
                        ms.sum[0][t] = to;
                        ms.nref[t] = to == -INFINITY ? 0.f : -to;
                        ms.fac[t] = old == -INFINITY ? 0.f : ex2(old - to);
                        none = to == -INFINITY;
                    }
                    fresh = group_or(1, 128, none);
                    if (!start) {
#pragma unroll
                        for (int c = 0; c < NQ; ++c) {
                            raw[c] *= ms.fac[c];
                            rnd[c] *= ms.fac[c];
                        }
                        // The accumulators follow, once the products before have come to an end.
                        if (pv < k) {
                            fail |= !tc::bar_wait(tc::smem_u32(&ms.pvdone), (k - 1) & 1, abort);
                            pv = k;
                        }
                        tc::fence_after();
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            float o[1][16];
                            tc::tmem_ld16(lanes + 2 * NQ + c * 16, o[0]);
                            tc::wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[0][e] *= ms.fac[c * 16 + e];
                            tc::tmem_st16(lanes + 2 * NQ + c * 16, o[0]);
                        }
                        tc::wait_st();
                    }
                }
                // The weights, rounded to the values' type; both sums go on.
                uint32_t pk[NQ / 2];
#pragma unroll
                for (int c = 0; c < NQ; c += 2) {
                    float a = ex2(fmaf(x[c / 16][c % 16], P.scale_log2, ms.nref[c]));
                    float b = ex2(fmaf(x[c / 16][c % 16 + 1], P.scale_log2, ms.nref[c + 1]));
                    if (special) {
                        if (!((vis >> c) & 1)) a = 0.f;
                        if (!((vis >> (c + 1)) & 1)) b = 0.f;
                    }
                    pk[c / 2] = Half2<BF>::pack(a, b);
                    const float2 r = Half2<BF>::unpack(pk[c / 2]);
                    raw[c] += a;
                    raw[c + 1] += b;
                    rnd[c] += r.x;
                    rnd[c + 1] += r.y;
                }
                if (special && pos >= w.c) {
                    // Values nobody may see with weight 0: rows past the end become zeros, and what is
                    // not finite in a node's row is set aside (its readers get it at the end).
                    fail |= !tc::bar_wait(tc::smem_u32(&ms.vfull[s]), (k / NS) & 1, abort);
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
                        for (int ch = 0; ch < 8; ++ch) {
                            uint4 *at = reinterpret_cast<uint4 *>(smem + L::V0 + s * L::UNIT + hf * TILE * 128 + t * 128 +
                                                                  ch * 16);
                            if (pos >= len) {
                                *at = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            uint4 y = *at;
                            uint32_t *wd = &y.x;
                            bool odd = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((wd[e] & Half2<BF>::EXP_MASK) == Half2<BF>::EXP_MASK) wd[e] &= 0xffff0000u, odd = true;
                                if (((wd[e] >> 16) & Half2<BF>::EXP_MASK) == Half2<BF>::EXP_MASK) wd[e] &= 0xffffu, odd = true;
                            }
                            if (odd) {
                                *at = y;
                                poison = 1;
                            }
                        }
                }
                if (pv < k) {
                    fail |= !tc::bar_wait(tc::smem_u32(&ms.pvdone), (k - 1) & 1, abort);
                    pv = k;
                }
#pragma unroll
                for (int ch = 0; ch < NQ / 8; ++ch)
                    *reinterpret_cast<uint4 *>(smem + L::P0 + t * 128 + ((ch ^ (t & 7)) << 4)) =
                        make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
                tc::fence_async_smem();
                tc::fence_before();
                tc::bar_arrive(tc::smem_u32(&ms.pfull));
                ++k;
                if (!end) {
                    w.next(P);
                    continue;
                }

                // ---- the segment's end: join the columns' sums, write rows or a part -----------
                fail |= !tc::bar_wait(tc::smem_u32(&ms.pvdone), (k - 1) & 1, abort);
                pv = k;
                if (group_or(1, 128, fail)) break;
                tc::fence_after();
                float o[NC][16];
#pragma unroll
                for (int c = 0; c < NC; ++c) tc::tmem_ld16(lanes + 2 * NQ + c * 16, o[c]);
                column_sums<NQ>(raw, ms.red[wq], lane);
                tc::wait_ld(o);
                group_sync(1, 128);
                if (t < NQ) ms.fac[t] = ms.red[0][t] + ms.red[1][t] + ms.red[2][t] + ms.red[3][t];
                group_sync(1, 128);
                column_sums<NQ>(rnd, ms.red[wq], lane);
                const bool any_poison = group_or(1, 128, poison);
                if (t < NQ) ms.sum[1][t] = ms.red[0][t] + ms.red[1][t] + ms.red[2][t] + ms.red[3][t];
                if (any_poison && t < P.D) {
                    const int from = first_j * TILE, to = len < (w.j + 1) * TILE ? len : (w.j + 1) * TILE;
                    for (int y = from > w.c ? from : w.c; y < to; ++y) {
                        const int64_t st = (int64_t)w.b * P.max_pos + y;
                        const int slot = SV_INB(st, (int64_t)P.B * P.max_pos, 1107) ? P.slot_table[st] : -1;
                        if (slot < 0 || slot >= P.num_slots) continue;
                        const uint32_t bits = P.v[(int64_t)slot * P.v_slot + h * P.D + t];
                        if ((bits & Half2<BF>::EXP_MASK) != Half2<BF>::EXP_MASK) continue;
                        const float val = Half2<BF>::unpack(bits).x;
                        const unsigned long long see = ms.desc[seg & 1][y - w.c];
#pragma unroll
                        for (int c = 0; c < NQ; ++c) {
                            const int n = (qt * NQ + c) / P.G;
                            if (n < w.nn && ((see >> n) & 1)) o[c / 16][c % 16] += val;
                        }
                    }
                }
                const int raise = *(volatile int *)&ms.bad[seg % FLAGS] ? SPEC_VERIFY_DEV_BAD_KV_SLOT
                                  : ms.code[seg & 1]                    ? SPEC_VERIFY_DEV_BAD_TREE
                                                                        : 0;
                group_sync(1, 128);
                if (t == 0) {
                    if (raise && P.dev_status) atomicMax(P.dev_status, raise);
                    *(volatile int *)&ms.bad[seg % FLAGS] = 0;
                    tc::bar_arrive(tc::smem_u32(&ms.qempty[seg & 1]));
                }
                if (first_j == 0 && w.j + 1 == w.ntile) {
                    int n = qt * NQ / P.G, g = qt * NQ - n * P.G;
#pragma unroll
                    for (int c = 0; c < NQ; ++c) {
                        if (n < P.N) {
                            const int64_t row = ((int64_t)w.b * P.N + n) * P.Hq + h * P.G + g;
                            float y = n < w.nn ? o[c / 16][c % 16] / ms.sum[1][c] : 0.f;
                            if (raise) y = NAN;
                            if (t < P.D && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1108))
                                P.out[row * P.D + t] = (uint16_t)Half2<BF>::pack(y, y);
                            if (t == c && P.lse && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1109))
                                P.lse[row] = raise ? NAN
                                             : n < w.nn ? (log2f(ms.fac[c]) - ms.nref[c]) * 0.69314718f
                                                        : -INFINITY;
                        }
                        if (++g == P.G) g = 0, ++n;
                    }
                    group_sync(1, 128);
                } else {
                    // A part of a request: its CTAs are those whose runs hold the segment's tiles.
                    const int64_t ib = t0 + i - w.j, total_ = total;
                    const int c0 = cta_of(ib, total_, G), c1 = cta_of(ib + w.ntile - 1, total_, G);
                    const int first0 = run_begin(c0, total_, G) == ib;
                    const int slot = 2 * cta + (cta == c0 && !first0);
                    float *part = P.parts + (int64_t)slot * part_floats<NQ>();
#pragma unroll
                    for (int c = 0; c < NQ; ++c) part[c * MAXD + t] = raise ? NAN : o[c / 16][c % 16];
                    if (t < NQ) {
                        float *r = part + NQ * MAXD;
                        r[t] = ms.sum[0][t];
                        r[NQ + t] = raise ? NAN : ms.fac[t];
                        r[2 * NQ + t] = raise ? NAN : ms.sum[1][t];
                    }
                    __threadfence();
                    group_sync(1, 128);
                    if (t == 0) {
                        const unsigned n = (unsigned)(c1 - c0);
                        const unsigned was = atomicAdd(&P.counters[c0], 1u);
                        if (was == n) {
                            P.counters[c0] = 0;
                            auto &jn = ms.join[cta == c0 ? 1 : 0];
                            jn.on = 1;
                            jn.b = w.b;
                            jn.h = h;
                            jn.qt = qt;
                            jn.c0 = c0;
                            jn.c1 = c1;
                            jn.first0 = first0;
                        }
                    }
                }
                w.next(P);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (ms.abort) {
        // A bounded wait ran out: what is written is not an answer.  The copies and products in
        // flight end (again with a limit) before their memory is given back.
        const uint64_t begin = tc::now_ns();
        if (tid == 0)
            for (int kv = 0; kv < 2; ++kv)
                for (int n = ms.issued[kv], i = n > NS ? n - NS : 0; i < n; ++i)
                    while (!tc::bar_try(tc::smem_u32(kv ? &ms.vfull[i % NS] : &ms.kfull[i % NS]), (i / NS) & 1) &&
                           tc::now_ns() - begin < tc::WAIT_NS) {}
        if (tid == 32) {
            tc::commit(tc::smem_u32(&ms.drain));
            while (!tc::bar_try(tc::smem_u32(&ms.drain), 0) && tc::now_ns() - begin < tc::WAIT_NS) {}
        }
        if (tid == 0 && P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_TIMEOUT);
        __syncthreads();
    }
    if (warp == 1) tc::tmem_free(tmem, L::COLS);
    if (ms.abort) return;

    // ---- joins left to this CTA, by all its threads -----------------------------------------
    for (int i = 0; i < 2; ++i) {
        if (!ms.join[i].on) continue;
        __threadfence();
        const auto jn = ms.join[i];
        const int b = jn.b, nn = P.num_nodes ? P.num_nodes[b] : P.N;
        auto part_of = [&](int c) {
            return P.parts + (int64_t)(2 * c + (c == jn.c0 && !jn.first0)) * part_floats<NQ>();
        };
        // A thread takes four dimensions of a column; the parts are read in their order, so the
        // result does not depend on who joins.
        for (int e = tid; e < NQ * (MAXD / 4); e += NT) {
            const int c = e / (MAXD / 4), d = (e - c * (MAXD / 4)) * 4;
            const int g = jn.qt * NQ + c, n = g / P.G;
            if (n >= P.N) break;
            float top = -INFINITY;
            for (int x = jn.c0; x <= jn.c1; ++x) top = fmaxf(top, __ldcg(part_of(x) + NQ * MAXD + c));
            float sum = 0.f, rsum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int x = jn.c0; x <= jn.c1; ++x) {
                const float *part = part_of(x);
                const float m = __ldcg(part + NQ * MAXD + c), l = __ldcg(part + NQ * MAXD + NQ + c);
                const float r = __ldcg(part + NQ * MAXD + 2 * NQ + c);
                const float4 y = __ldcg(reinterpret_cast<const float4 *>(part + c * MAXD + d));
                const float f = l == 0.f ? 0.f : ex2(m == -INFINITY ? 0.f : m - top);
                if (l != 0.f) {
                    sum += f * l;
                    rsum += f * r;
                    acc.x += f * y.x;
                    acc.y += f * y.y;
                    acc.z += f * y.z;
                    acc.w += f * y.w;
                }
            }
            const int64_t row = ((int64_t)b * P.N + n) * P.Hq + jn.h * P.G + g - n * P.G;
            if (d < P.D && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1110)) {
                uint2 y = make_uint2(0, 0);
                if (n < nn) {
                    const float inv = 1.f / rsum;
                    y = make_uint2(Half2<BF>::pack(acc.x * inv, acc.y * inv), Half2<BF>::pack(acc.z * inv, acc.w * inv));
                }
                *reinterpret_cast<uint2 *>(P.out + row * P.D + d) = y;
            }
            if (d == 0 && P.lse)
                P.lse[row] = n < nn ? ((top == -INFINITY ? 0.f : top) + log2f(sum)) * 0.69314718f : -INFINITY;
        }
    }
}

// -------------------------------------------------------------------------------------------------
// Host side.
// -------------------------------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct DevInfo {
    int sms = 0;
};
static std::mutex g_mu;
static DevInfo g_dev[64];
static EncodeFn g_encode;

template <bool BF, int NQ, int DP>
constexpr size_t smem_bytes()
{
    using L = Layout<NQ, DP>;
    return L::M0 + sizeof(Misc<NQ, L::NS>);
}

template <bool BF, int NQ, int DP>
static bool allow()
{
    static_assert(smem_bytes<BF, NQ, DP>() <= 232448, "shared memory of a CTA");
    return cudaFuncSetAttribute((const void *)attention_kernel<BF, NQ, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<BF, NQ, DP>()) == cudaSuccess;
}

// Once per device: the kernels' shared memory, the SM count, the driver's tensor-map encoder.
static const DevInfo *device_info()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lk(g_mu);
    DevInfo &d = g_dev[dev];
    if (d.sms == 0) {
        int sms = 0;
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult how;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess || !fn ||
            !(allow<true, 16, 64>() && allow<true, 32, 64>() && allow<true, 64, 64>() && allow<true, 16, 128>() &&
              allow<true, 32, 128>() && allow<true, 64, 128>() && allow<false, 16, 64>() && allow<false, 32, 64>() &&
              allow<false, 64, 64>() && allow<false, 16, 128>() && allow<false, 32, 128>() && allow<false, 64, 128>())) {
            cudaGetLastError();
            return nullptr;
        }
        g_encode = reinterpret_cast<EncodeFn>(fn);
        d.sms = sms;
    }
    return &d;
}

// The cache as a matrix: a row per slot, a gather's box 64 elements of a row.
static bool encode(CUtensorMap *map, bool bf16, const void *base, int64_t slots, int64_t stride, int64_t width)
{
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)slots};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, 1}, elem[2] = {1, 1};
    return g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                    const_cast<void *>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Columns per CTA: the fewest of 16, 32, 64 that hold a key head's query rows, 64 at most (a
// wider call reads the cache once per 64 rows, the second time from L2).
static int columns(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

constexpr size_t COUNTER_BYTES = 65536 * 4;  // the workspace's fixed region of counters

template <bool BF, int NQ, int DP>
static cudaError_t launch(const CUtensorMap &km, const CUtensorMap &vm, const Params &P, int grid, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem_bytes<BF, NQ, DP>();
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_kernel<BF, NQ, DP>, km, vm, P);
}

template <bool BF>
static cudaError_t dispatch(int nq, int dp, const CUtensorMap &km, const CUtensorMap &vm, const Params &P, int grid,
                            cudaStream_t s)
{
    if (dp == 64)
        return nq == 16 ? launch<BF, 16, 64>(km, vm, P, grid, s)
               : nq == 32 ? launch<BF, 32, 64>(km, vm, P, grid, s)
                          : launch<BF, 64, 64>(km, vm, P, grid, s);
    return nq == 16 ? launch<BF, 16, 128>(km, vm, P, grid, s)
           : nq == 32 ? launch<BF, 32, 128>(km, vm, P, grid, s)
                      : launch<BF, 64, 128>(km, vm, P, grid, s);
}

}  // namespace svatt

namespace sv {
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
    return svatt::COUNTER_BYTES + 2 * svatt::MAX_CTAS * (nq * svatt::MAXD + 3 * nq) * sizeof(float);
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
    if (!need || num_slots < 1 || num_slots > 0x7fffffff || !(scale > 0.f) || scale > 3e38f) return SPEC_VERIFY_EINVAL;
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hkv * D;
    if (q_stride % 8 || k_slot_stride % 8 || v_slot_stride % 8 || q_stride < qw || k_slot_stride < kw || v_slot_stride < kw)
        return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) % 16) return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)slot_table | (uintptr_t)committed | (uintptr_t)parents | (uintptr_t)num_nodes | (uintptr_t)lse |
         (uintptr_t)dev_status) % 4)
        return SPEC_VERIFY_EINVAL;
    if (ws_bytes < need || (uintptr_t)workspace % 256) return SPEC_VERIFY_EWORKSPACE;
    const DevInfo *dev = device_info();
    if (!dev) return SPEC_VERIFY_ECUDA;
    CUtensorMap km, vm;
    const bool bf = dtype == SPEC_VERIFY_BF16;
    if (!encode(&km, bf, k_cache, num_slots, k_slot_stride, kw) || !encode(&vm, bf, v_cache, num_slots, v_slot_stride, kw))
        return SPEC_VERIFY_EINVAL;
    Params P;
    P.q = static_cast<const uint16_t *>(q);
    P.v = static_cast<const uint16_t *>(v_cache);
    P.out = static_cast<uint16_t *>(out);
    P.lse = lse;
    P.q_row = q_stride;
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
    int grid = dev->sms < MAX_CTAS ? dev->sms : MAX_CTAS;
    const int64_t most = (int64_t)B * Hkv * P.QT * ((max_pos + TILE - 1) / TILE);
    if (most < grid) grid = (int)most;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int dp = D <= 64 ? 64 : 128;
    const cudaError_t e = bf ? dispatch<true>(nq, dp, km, vm, P, grid, s) : dispatch<false>(nq, dp, km, vm, P, grid, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SPEC_VERIFY_ECUDA;
    }
    return SPEC_VERIFY_OK;
}
