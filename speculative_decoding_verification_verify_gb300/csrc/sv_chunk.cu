// sv_chunk.cu -- attention of a chunk of a prompt over the paged cache, causal, with grouped heads and requests of
// different lengths.
//
//   node n of request b sees the positions j <= committed + n;  s_j = scale * q . k_j
//   out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), lse = m + ln sum_j e^(s_j - m)
//
// The products bound it: 4 D operations for each pair of a query row and a position it sees.  A key head's query rows
// (a token's G heads are neighbours) come in blocks of 256, two halves of 128 rows of the matrix instruction; a tile
// of 128 positions serves both:
//
//   S [128 rows][128 positions] = Q [128][D] . K^T     both from shared memory
//   O [128 rows][D]            += P . V                P from TMEM, where it takes the place of S; V as it lies in the cache
//
// While one half's softmax runs, the other's products do: the tensor cores are fed by the halves in turn.  A thread has
// a row, so maxima and sums are its own; the softmax's reference moves only when a score passes it by a factor of more
// than 2^8 in weight (a vote of 32 rows), and the accumulators are scaled then, by the same warps.  Maxima, sums and
// accumulators are fp32.  Weights are rounded to q's type for the product with v, as the matrix instruction has it; the sum
// that divides is of the unrounded ones, whose roundings are as often up as down.  (A second sum of the rounded ones, as the
// nodes' kernel has, would be an unpacking and an addition more for each weight of the part that bounds the kernel.)
//
// Each CTA takes an equal run of the batch's work: the blocks of all requests and key heads on one axis of costs
// (positions that a block sees, plus SEGMENT for its beginning and end), cut into equal pieces; where a cut falls
// inside a block, the parts go to the workspace and a second kernel joins them, with all SMs.  So one short chunk
// behind a long prefix is spread over all SMs, and a triangle of blocks leaves none waiting.
//
// Warps 0-3 copy queries and tiles (16-byte rows as they are, 8-bit rows widened in registers), warp 4 issues the
// products, warp 5 lists the run's segments (a segment: the run's tiles of one block), warps 8-11 and 12-15 are the
// halves' softmax.
//
// Measured (GB300, products at 1922 TFLOP/s; 32 query and 8 key heads of 128): 2048 tokens behind 14337 391-395 us, 1.31-1.32
// PFLOP/s; 4096 behind 28001 over 8-bit rows 1680 us, 1.2 PFLOP/s; 8 prompts of 512 to 4096 (heads of 64, fp16) 349
// us, 627 TFLOP/s; 3 x 67 tokens behind 901 to 9001 (14 and 2 heads of 80) 27-28 us.  A half's turn is some 3300
// clocks a tile: 1700 of softmax (scores and maximum 300, vote 300, weights 900), then the products of its own weights
// and next scores behind the other half's, 1024 of 2048 clocks of tensor work.  With heads of 64 the products
// are half of that and the softmax the same; scores issued before the weights' products (there are columns of TMEM
// for both) took 364 us against 350, for the halves' softmax then runs in step.
#include "sv_e4m3.cuh"
#include "sv_reference.cuh"
#include "sv_tc.cuh"

#include <mutex>

namespace svch {

using sv::ex2;
using sv::FAR;
using sv::Half2;
using sv::lift;

constexpr int TILE = 128, ROWS = 256, HALF = 128, MAXD = 128;
constexpr int MAX_SMS = 192;
constexpr int NT = 512;
constexpr int SEGS = 4;         // segments listed ahead
constexpr int SEGMENT = 384;    // the cost of a block's beginning and end, in positions
// Of a run.  (2: 16 tokens behind 30000, one key head, 53 us for a call waited for, against 45.5; 6: 3 x 67 tokens 50
// against 44.)
constexpr int MIN_TILES = 4;
constexpr float SLACK = 8.f;    // log2 of how much a weight may pass the reference's

// A block in parts: of CTA c0's run the second part, of c0 + 1 .. c1's the first.
struct __align__(16) Join {
    int b, h, qb, c0;  // (read as two vectors)
    int c1, nn, pad0, pad1;  // c1 = c0: nothing to join
};

struct Params {
    const uint16_t *q;
    const unsigned char *k, *v;
    uint16_t *out;
    float *lse;
    int64_t q_row, k_slot, v_slot, num_slots;  // the slots' strides in bytes
    const int32_t *slot_table, *committed, *num_nodes;
    int max_pos, B, N, Hq, Hkv, D, G;
    float scale_log2;
    int32_t *dev_status;
    Join *joins;   // one per CTA: the block that its run began and others ended
    float *parts;  // two per CTA
    int ctas;
};

// A run's tiles [j0, j1) of block qb of a request and key head; tiles that each half sees.
struct __align__(16) Seg {
    int b, h, qb, last;
    int c, nn, j0, j1;
    int nt[2], part, pad;
};

template <int DP, bool E4>
struct Layout {
    static constexpr int UNIT = TILE * DP * 2;      // a tile's keys or values
    static constexpr int QHALF = HALF * DP * 2;
    // Units in the ring; 8-bit rows have one of their own before it, of AHEAD tiles' keys or values in turn.
    static constexpr int NU = (E4 ? 3 : 5) * 128 / DP, AHEAD = 3 * 128 / DP;
    static constexpr int Q0 = NU * UNIT, R0 = Q0 + 2 * QHALF, M0 = R0 + (E4 ? AHEAD * (128 * DP + 512) : 0);
};

template <int NU>
struct Misc {
    uint64_t full[NU], empty[NU];
    uint64_t sfull[2], pfull[2][2], odone[2], qfull, qempty, segfull[SEGS], segempty[SEGS], drain;
    union {
        Seg seg[SEGS];
        int64_t scan[NT / 32];  // (before any segment is listed)
    };
    int64_t begin_base;
    int begin_b, abort;
    int poison[4];  // a segment's number: its values have some that are not finite behind the block's first row
    uint32_t tmem;
};

// Floats of a part: the weighted values [dimensions / 4][row][4], references and sums of the rows.
constexpr int PART = ROWS * MAXD + 2 * ROWS;

// The keys of a slot outside the pool: NaN of either type.
static __device__ const uint4 g_nan = {0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu};

// ---------------------------------------------------------------------------------------------
// The axis of costs.  A block sees c + 256 (i + 1) / G positions at most; times G that is a whole number, and so
// is the sum over the blocks before the i-th.
// ---------------------------------------------------------------------------------------------
struct Request {
    int c, nn, blocks;
    bool wrong;
    int64_t first, head;  // a block's fixed cost; a key head's blocks
};

__device__ __forceinline__ Request request(const Params &P, int b)
{
    Request r;
    r.c = SV_INB(b, P.B, 1301) ? P.committed[b] : 0;
    r.nn = P.num_nodes ? (SV_INB(b, P.B, 1302) ? P.num_nodes[b] : 0) : P.N;
    r.wrong = r.nn < 0 || r.nn > P.N || r.c < 0 || (int64_t)r.c + r.nn > P.max_pos;
    if (r.wrong) r.c = r.nn = 0;  // (the second kernel reports it)
    r.blocks = (int)(((int64_t)r.nn * P.G + ROWS - 1) / ROWS);
    r.first = (int64_t)P.G * (SEGMENT + r.c + TILE / 2);
    r.head = r.blocks * r.first + (int64_t)(ROWS / 2) * r.blocks * (r.blocks + 1);
    return r;
}
__device__ __forceinline__ int64_t block_at(const Request &r, int64_t i) { return i * r.first + (ROWS / 2) * i * (i + 1); }

// A cut x into a block leaves the tiles before it to the run before; a tile t belongs to the last run that begins
// before tile_key(t).
__device__ __forceinline__ int cut_tile(const Params &P, int64_t x, int tiles)
{
    const int64_t y = x - (int64_t)P.G * (SEGMENT - TILE / 2);
    if (y <= 0) return 0;
    const int64_t t = y / ((int64_t)P.G * TILE);
    return t < tiles ? (int)t : tiles;
}
__device__ __forceinline__ int64_t tile_key(const Params &P, int64_t t) { return (int64_t)P.G * (SEGMENT + TILE / 2 + TILE * t); }
__device__ __forceinline__ int64_t run_begin(int64_t r, int64_t total, int runs) { return total * r / runs; }
__device__ __forceinline__ int run_before(int64_t x, int64_t total, int runs) { return (int)((x * runs + total - 1) / total) - 1; }

template <bool BF, int DP, bool E4>
using MiscOf = Misc<Layout<DP, E4>::NU>;

template <bool BF, int DP, bool E4>
__global__ void __launch_bounds__(NT, 1) chunk_kernel(const __grid_constant__ Params P)
{
    using L = Layout<DP, E4>;
    constexpr int NU = L::NU;
    extern __shared__ __align__(1024) unsigned char smem[];
    auto &ms = *reinterpret_cast<MiscOf<BF, DP, E4> *>(smem + L::M0);
    const uint32_t s0 = tc::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    volatile int *abort = &ms.abort;

    if (tid == NT - 32) {
        for (int s = 0; s < NU; ++s) {
            tc::bar_init(tc::smem_u32(&ms.full[s]), 128);
            tc::bar_init(tc::smem_u32(&ms.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(tc::smem_u32(&ms.sfull[i]), 1);
            tc::bar_init(tc::smem_u32(&ms.pfull[i][0]), 128);
            tc::bar_init(tc::smem_u32(&ms.pfull[i][1]), 128);
            tc::bar_init(tc::smem_u32(&ms.odone[i]), 1);
        }
        tc::bar_init(tc::smem_u32(&ms.qfull), 128);
        tc::bar_init(tc::smem_u32(&ms.qempty), 1);
        tc::bar_init(tc::smem_u32(&ms.drain), 1);
        for (int i = 0; i < SEGS; ++i) {
            tc::bar_init(tc::smem_u32(&ms.segfull[i]), 1);
            tc::bar_init(tc::smem_u32(&ms.segempty[i]), 13);  // warps that take segments
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        ms.abort = 0;
        ms.begin_b = P.B;
        ms.begin_base = 0;
        for (int i = 0; i < 4; ++i) ms.poison[i] = 0;
    }
    if (warp == 4) tc::tmem_alloc(tc::smem_u32(&ms.tmem), 512);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The batch's cost, and the request that this CTA's run begins in.
    const int per = (P.B + NT - 1) / NT;
    int64_t mine = 0;
#pragma unroll 1
    for (int i = 0; i < per && tid * per + i < P.B; ++i) mine += request(P, tid * per + i).head * P.Hkv;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) ms.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll 1
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += ms.scan[w];
        total += ms.scan[w];
    }
    const int64_t most = total / ((int64_t)P.G * TILE * MIN_TILES);
    const int runs = most < 1 ? 1 : most < P.ctas ? (int)most : P.ctas;
    const int64_t t0 = cta < runs ? run_begin(cta, total, runs) : total, t1 = cta < runs ? run_begin(cta + 1, total, runs) : total;
    if (t0 >= before && t0 < before + mine) {
        int64_t at = before;
        int b = tid * per;
#pragma unroll 1
        for (; b < P.B; ++b) {
            const int64_t n = request(P, b).head * P.Hkv;
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

    int si = 0;
    // The next segment; false when there is none, or a wait failed.
    auto take = [&](Seg &g) {
        const bool ok = tc::bar_wait(tc::smem_u32(&ms.segfull[si % SEGS]), (si / SEGS) & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) return false;
        g = ms.seg[si % SEGS];
        __syncwarp();
        if (lane == 0) tc::bar_arrive(tc::smem_u32(&ms.segempty[si % SEGS]));
        ++si;
        return !g.last;
    };

    // (The registers of a launch, 128 a thread, go to those who hold a row of scores.)
    if (warp < 4) {
        if constexpr (E4) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ---- queries and tiles into shared memory ---------------------------------------------
        constexpr int QCPR = DP / 8, QRPI = 32 / QCPR;            // 16-byte chunks of a query row; rows of a warp's copy
        [[maybe_unused]] constexpr int CPR = DP / 8, RPI = 32 / CPR, ITER = TILE / (4 * RPI);
        constexpr int AHEAD = L::AHEAD;
        using Feed = sv::E4m3Feed<BF, DP, AHEAD>;
        Feed feed(s0 + L::R0, warp, lane, P.D);
        const int chunk = lane % CPR, sub = lane / CPR;
        const int own = E4 ? feed.own : warp * RPI + lane % RPI + 4 * RPI * (lane / RPI);  // the row whose slot the lane keeps
        const int first = warp * RPI + sub;                                                // its row of the first copy
        const bool wide = chunk * 8 < P.D;
        Seg g;
        int u = 0, seg = 0;
        bool ok = true;
        while (ok && take(g)) {
            // The block's queries, once the products of the segment before have read theirs.
            if (seg > 0) ok = __all_sync(0xffffffffu, tc::bar_wait(tc::smem_u32(&ms.qempty), (seg - 1) & 1, abort));
            if (!ok) break;
            ++seg;
            const int qc = lane % QCPR;
            const unsigned rows = (unsigned)g.nn * P.G;
#pragma unroll 4
            for (int r = warp * QRPI + lane / QCPR; r < ROWS; r += 4 * QRPI) {
                const unsigned gr = (unsigned)g.qb * ROWS + r, n = gr / (unsigned)P.G, h = gr - n * P.G;
                const int64_t at = ((int64_t)g.b * P.N + n) * P.q_row + (int64_t)(g.h * P.G + h) * P.D + qc * 8;
                const bool in = gr < rows && qc * 8 < P.D && SV_INB(at, (int64_t)P.B * P.N * P.q_row, 1303);
                const uint32_t dst = s0 + L::Q0 + (r >> 7) * L::QHALF + (qc >> 3) * HALF * 128 + (r & 127) * 128 +
                                     (((qc & 7) ^ (r & 7)) << 4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(in ? P.q + at : P.q), "r"(in ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(&ms.qfull)) : "memory");

            const int len = g.c + g.nn;
            const int64_t table = (int64_t)g.b * P.max_pos;
            // A row's slot: -1 past the end, -2 (reported) outside the pool; its keys are then NaN, its values 0.
            auto look = [&](int j) {
                const int pos = j * TILE + own;
                if (j >= g.j1 || pos >= len) return -1;
                return SV_INB(table + pos, (int64_t)P.B * P.max_pos, 1304) ? P.slot_table[table + pos] : -2;
            };
            auto check = [&](int j, int slot) {
                if (j * TILE + own >= len) return -1;
                if (slot >= 0 && slot < P.num_slots) return slot;
                if (P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_BAD_KV_SLOT);
                return -2;
            };
            auto room = [&] {
                if (u >= NU)
                    ok = __all_sync(0xffffffffu, tc::bar_wait(tc::smem_u32(&ms.empty[u % NU]), (u / NU + 1) & 1, abort));
                return ok;
            };
            int ahead = look(g.j0);
            if constexpr (!E4) {
                const uint32_t to = s0 + (chunk >> 3) * TILE * 128 + first * 128 + (((chunk & 7) ^ (first & 7)) << 4);
                for (int j = g.j0; j < g.j1 && ok; ++j) {
                    const int slots = check(j, ahead);
                    ahead = look(j + 1);
                    const bool whole = __all_sync(0xffffffffu, slots >= 0 && wide);
                    const int64_t at = 2 * ((int64_t)g.h * P.D + (wide ? chunk * 8 : 0));
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++u) {
                        if (!room()) break;
                        const uint32_t dst = to + (u % NU) * L::UNIT;
                        const unsigned char *base = (kv ? P.v : P.k) + at;
                        const uint64_t stride = kv ? P.v_slot : P.k_slot;
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < ITER; ++i) {
                                const uint32_t s = __shfl_sync(0xffffffffu, slots, i * RPI + sub);
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 4 * RPI * 128),
                                             "l"(base + s * stride)
                                             : "memory");
                            }
                        } else {
#pragma unroll 1
                            for (int i = 0; i < ITER; ++i) {  // zeros where there is nothing to copy
                                const int s = __shfl_sync(0xffffffffu, slots, i * RPI + sub);
                                const bool nan = s == -2 && kv == 0;
                                const void *src = nan ? (const void *)&g_nan : base + (uint64_t)(uint32_t)(s < 0 ? 0 : s) * stride;
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * 4 * RPI * 128),
                                             "l"(src), "r"(nan || (s >= 0 && wide) ? 16 : 0)
                                             : "memory");
                            }
                        }
                        // The unit's barrier hears of each thread's copies as they land; nobody waits for them here.
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(&ms.full[u % NU]))
                                     : "memory");
                    }
                }
            } else {
                // The segment's units (keys and values of a tile in turn): while one is widened its place in the ring is
                // filled with the one AHEAD units on.
                const int units = 2 * (g.j1 - g.j0);
                int slot = -1, x = 0;  // the slots of the unit to be asked for next, the x-th
                auto next = [&] {
                    if (x & 1) return;
                    slot = check(g.j0 + x / 2, ahead);
                    ahead = look(g.j0 + x / 2 + 1);
                };
                auto place = [&] {
                    const bool whole = __all_sync(0xffffffffu, slot >= 0);
                    int slots[Feed::ITER];
#pragma unroll
                    for (int i = 0; i < Feed::ITER; ++i) slots[i] = __shfl_sync(0xffffffffu, x & 1 && slot == -2 ? -1 : slot, i * Feed::RPI + feed.sub);
                    feed.ask(x % AHEAD, whole, (x & 1 ? P.v : P.k) + g.h * P.D, (uint32_t)(x & 1 ? P.v_slot : P.k_slot), slots);
                };
                auto placed = [&](int count) {
                    feed.asked(x % AHEAD, count, slot, x & 1 ? P.v : P.k, x & 1 ? P.v_slot : P.k_slot, P.Hkv * P.D + g.h);
                    ++x;
                };
                for (int a = 0; a < AHEAD; ++a) {
                    if (x >= units) {
                        feed.commit();
                        continue;
                    }
                    next();
                    place();
                    placed(a);
                }
                for (int y = 0; y < units; ++y, ++u) {
                    const bool more = x < units;
                    if (more) next();
                    feed.wait();
                    typename Feed::Tile tile;
                    feed.read(y % AHEAD, tile);
                    if (more) {
                        place();
                        placed(AHEAD - 1);
                    } else {
                        feed.commit();
                    }
                    if (!room()) break;
                    feed.write(s0 + (u % NU) * L::UNIT, tile);
                    tc::bar_arrive(tc::smem_u32(&ms.full[u % NU]));  // (the products' thread fences what it sees)
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < 8) {
        if constexpr (E4) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 4) {
            // ---- products ----------------------------------------------------------------------
            const uint32_t id_s = tc::instr_desc(BF, false, false, 128, TILE), id_o = tc::instr_desc(BF, false, true, 128, P.D);
            const int dsteps = P.D / 16;
            constexpr uint32_t HIGH = tc::desc_high(1024);
            const uint32_t kd = tc::desc_low(s0, 0), qd = tc::desc_low(s0 + L::Q0, 0);
            const uint32_t vd = tc::desc_low(s0, DP > 64 ? TILE * 128 : 0);
            Seg g;
            int u = 0, seg = 0, k[2] = {0, 0};  // units, segments and the halves' tiles so far
            bool ok = true;
            const bool me = tc::elect();
            auto wait = [&](uint64_t &bar, int n) { ok = ok && tc::bar_wait(tc::smem_u32(&bar), n & 1, abort); };
            auto score = [&](int h, int unit) {
                const uint32_t a = qd + h * (L::QHALF >> 4), b = kd + (unit % NU) * (L::UNIT >> 4);
#pragma unroll 4
                for (int d = 0; d < dsteps; ++d)
                    tc::mma_f16<HIGH, HIGH>(tmem + h * TILE, a + (d >> 2) * (HALF * 8) + (d & 3) * 2, b + (d >> 2) * (TILE * 8) + (d & 3) * 2, id_s,
                                d > 0);
                tc::commit(tc::smem_u32(&ms.sfull[h]));
            };
            while (take(g)) {
                if (me) {
                    const int e[2] = {g.nt[0] < g.j1 ? g.nt[0] : g.j1, g.nt[1] < g.j1 ? g.nt[1] : g.j1};
                    wait(ms.qfull, seg);
                    for (int j = g.j0 - 1; j < g.j1 && ok; ++j) {
                        // Of tile j the weighted values, of tile j + 1 the scores: half 0's, then half 1's.
                        const int uk = u + 2 * (j + 1 - g.j0), uv = uk - 1;
                        const bool more = j + 1 < g.j1;
#pragma unroll
                        for (int h = 0; h < 2 && ok; ++h) {
                            if (j >= g.j0 && j < e[h]) {
                                wait(ms.full[uv % NU], uv / NU);
                                wait(ms.pfull[h][0], k[h]);
                                if (!ok) break;
                                tc::fence_after();
                                tc::fence_async_smem();
                                const uint32_t b = vd + (uv % NU) * (L::UNIT >> 4);
                                const uint32_t a = tmem + h * TILE, d = tmem + 256 + h * MAXD;
#pragma unroll
                                for (int i = 0; i < 4; ++i) tc::mma_f16_ts<HIGH>(d, a + i * 8, b + i * 128, id_o, j > g.j0 || i > 0);
                                if constexpr (!E4) {
                                    wait(ms.pfull[h][1], k[h]);
                                    if (!ok) break;
                                    tc::fence_after();
                                }
#pragma unroll
                                for (int i = 4; i < 8; ++i) tc::mma_f16_ts<HIGH>(d, a + i * 8, b + i * 128, id_o, true);
                                if (j + 1 == e[h]) tc::commit(tc::smem_u32(&ms.odone[h]));
                                ++k[h];
                            }
                            if (h == 1 && j >= g.j0) tc::commit(tc::smem_u32(&ms.empty[uv % NU]));
                            if (more) {
                                wait(ms.full[uk % NU], uk / NU);
                                if (!ok) break;
                                tc::fence_after();
                                tc::fence_async_smem();  // the copies are ordinary writes; this thread has seen them land
                                if (j + 1 < e[h]) score(h, uk);
                                if (h == 1) {
                                    tc::commit(tc::smem_u32(&ms.empty[uk % NU]));
                                    if (j + 2 == g.j1) tc::commit(tc::smem_u32(&ms.qempty));
                                }
                            }
                        }
                    }
                    u += 2 * (g.j1 - g.j0);
                    ++seg;
                }
                if (__any_sync(0xffffffffu, me && !ok)) break;
            }
            __syncwarp();
        } else if (warp == 5) {
            // ---- the run's segments --------------------------------------------------------------
            int n = 0;
            bool ok = true;
            Join jn = {};
            auto put = [&](const Seg &g) {
                if (n >= SEGS) ok = __all_sync(0xffffffffu, tc::bar_wait(tc::smem_u32(&ms.segempty[n % SEGS]), (n / SEGS + 1) & 1, abort));
                if (!ok) return;
                if (lane == 0) {
                    ms.seg[n % SEGS] = g;
                    tc::bar_arrive(tc::smem_u32(&ms.segfull[n % SEGS]));
                }
                __syncwarp();
                ++n;
            };
            Seg g = {};
            int64_t base = ms.begin_base;  // the cost before the request
            bool begun = false;
            for (int b = ms.begin_b; b < P.B && base < t1 && ok; ++b) {
                const Request r = request(P, b);
                int h = 0, i = 0;
                if (!begun && r.blocks) {  // the block that the run begins in
                    const int64_t x = t0 - base;
                    h = (int)(x / r.head);
                    int hi = r.blocks - 1;
                    while (i < hi) {
                        const int mid = i + (hi - i + 1) / 2;
                        if (block_at(r, mid) <= x - h * r.head) i = mid;
                        else hi = mid - 1;
                    }
                    begun = true;
                }
                g.b = b, g.c = r.c, g.nn = r.nn;
                for (; h < P.Hkv && ok; ++h, i = 0) {
                    for (; i < r.blocks && ok; ++i) {
                        const int64_t at = base + h * r.head + block_at(r, i);
                        if (at >= t1) break;
                        const int64_t rows = (int64_t)r.nn * P.G;
                        int nt = 0;
                        for (int x = 0; x < 2; ++x) {
                            const int64_t r0 = (int64_t)i * ROWS + x * HALF, r1 = r0 + HALF < rows ? r0 + HALF : rows;
                            g.nt[x] = r1 > r0 ? (r.c + (int)((r1 - 1) / P.G)) / TILE + 1 : 0;
                            nt = g.nt[x] > nt ? g.nt[x] : nt;
                        }
                        g.h = h, g.qb = i;
                        g.j0 = cut_tile(P, t0 - at, nt);
                        g.j1 = cut_tile(P, t1 - at, nt);
                        if (g.j0 >= g.j1) continue;
                        g.part = -1;
                        if (g.j0 > 0 || g.j1 < nt) {
                            const int c0 = run_before(at + tile_key(P, 0), total, runs);
                            g.part = 2 * cta + (cta == c0);
                            if (cta == c0) jn = {b, h, i, c0, run_before(at + tile_key(P, nt - 1), total, runs), r.nn, 0, 0};
                        }
                        put(g);
                    }
                }
                base += r.head * P.Hkv;
            }
            g.last = 1;
            if (ok) put(g);
            if (lane == 0) P.joins[cta] = jn;
        }
    } else {
        if constexpr (E4) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        // ---- softmax: a row per thread ---------------------------------------------------------
        const int half = (warp - 8) >> 2, wq = warp & 3, t = tid & 127;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        const uint32_t st = tmem + lanes + half * TILE, ot = tmem + lanes + 256 + half * MAXD;
        const int dsteps = (P.D + 31) / 32;  // in blocks of 32 columns
        const uint64_t scale2 = sv::f2(P.scale_log2, P.scale_log2);
        int k = 0, seg = 0, ends = 0, units = 0;
        bool ok = true;
        Seg g;
        while (ok && take(g)) {
            ++seg;
            const unsigned gr = (unsigned)g.qb * ROWS + half * HALF + t;
            const int n = (int)(gr / (unsigned)P.G), h = (int)gr - n * P.G;
            const int edge = g.c + n;  // the last position that the row sees
            const int front = g.c + (int)((unsigned)g.qb * ROWS / (unsigned)P.G);                     // that the block's first row does
            const int wfront = g.c + (int)(((unsigned)g.qb * ROWS + half * HALF + wq * 32) / (unsigned)P.G);  // the warp's
            const int end = (half ? g.nt[1] : g.nt[0]) < g.j1 ? (half ? g.nt[1] : g.nt[0]) : g.j1;
            float ref = -INFINITY, add = 0.f, sum = 0.f;
            bool far = false;
            for (int j = g.j0; j < end; ++j, ++k) {
                float x[TILE];
                ok = __all_sync(0xffffffffu, tc::bar_wait(tc::smem_u32(&ms.sfull[half]), k & 1, abort));
                if (!ok) break;
                tc::fence_after();
#pragma unroll
                for (int i = 0; i < 4; ++i) tc::tmem_ld32(st + 32 * i, x + 32 * i);
                tc::wait_ld(x);
                if ((j + 1) * TILE - 1 > wfront) {
                    const int seen = edge - j * TILE;  // the last of the tile's columns that the row sees
#pragma unroll
                    for (int i = 0; i < TILE; ++i) x[i] = i <= seen ? x[i] : -INFINITY;
                }
                float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int i = 4; i < TILE; i += 4) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) top[y] = fmaxf(top[y], x[i + y]);
                }
                const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // Move the references of the warp's rows when one is passed by too much, or there is none.
                const bool move = far || ref == -INFINITY || fmaf(m, P.scale_log2, add) > SLACK + lift(BF);
                if (__any_sync(0xffffffffu, move)) {
                    const float now = fmaxf(m, ref), was = add;
                    add = sv::reference_add<BF>(now, P.scale_log2);
                    const float fac = sv::reference_factor<BF>(ref, was, now, add, P.scale_log2);
                    ref = now;
                    far = fabsf(add) >= FAR;
                    sum *= fac;
                    if (j > g.j0) {
                        // (The scores' barrier is behind the products of the tile before.)
#pragma unroll 1
                        for (int d = 0; d < dsteps; ++d) {
                            float o[32];
                            uint32_t w[32];
                            tc::tmem_ld32(ot + 32 * d, o);
                            tc::wait_ld(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * fac);
                            tc::tmem_st32(ot + 32 * d, w);
                        }
                        tc::wait_st();
                    }
                }
                float bias = add;
                if (__any_sync(0xffffffffu, far)) {
                    // The reference is taken from the scores before the scale.
                    const float off = far ? ref : 0.f;
                    bias = far ? lift(BF) : add;
#pragma unroll
                    for (int i = 0; i < TILE; ++i) x[i] -= off;
                }
                auto set_aside = [&] {
                    if ((j + 1) * TILE - 1 <= front) return;
                    const int pos = j * TILE + t;
                    // A weight of 0 does not undo an infinity or a NaN: what is not finite in values that the block's
                    // first row does not see is set aside, and the rows that do see it get it at the segment's end.
                    // (Both halves do so, each before its own products; what the other has set aside reads as 0.)
                    const int uv = units + 2 * (j - g.j0) + 1;
                    ok = __all_sync(0xffffffffu, tc::bar_wait(tc::smem_u32(&ms.full[uv % NU]), (uv / NU) & 1, abort));
                    if (pos > front && pos < g.c + g.nn) {
                        // An exponent of all ones carries into the sign's place.
                        constexpr uint32_t EXP2 = Half2<BF>::EXP_MASK * 0x10001u;
                        constexpr uint32_t ONE2 = (0x8000u - Half2<BF>::EXP_MASK) * 0x10001u;
                        unsigned char *const at = smem + (uv % NU) * L::UNIT + t * 128;
                        uint32_t carry = 0;
#pragma unroll 4
                        for (int ch = 0; ch < DP / 8; ++ch) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(at + (ch >> 3) * TILE * 128 + (ch & 7) * 16);
                            carry |= ((y.x & EXP2) + ONE2) | ((y.y & EXP2) + ONE2) | ((y.z & EXP2) + ONE2) | ((y.w & EXP2) + ONE2);
                        }
                        if (carry & 0x80008000u) {
                            *(volatile int *)&ms.poison[seg & 3] = seg;
                            __threadfence_block();
#pragma unroll 1
                            for (int e = 0; e < DP / 2; ++e) {
                                uint32_t *w = reinterpret_cast<uint32_t *>(at + (e >> 5) * TILE * 128) + (e & 31), y = *w;
                                if ((y & Half2<BF>::EXP_MASK) == Half2<BF>::EXP_MASK) y &= 0xffff0000u;
                                if (((y >> 16) & Half2<BF>::EXP_MASK) == Half2<BF>::EXP_MASK) y &= 0xffffu;
                                *w = y;
                            }
                        }
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                };
                if (!E4) set_aside();
                const uint64_t bias2 = sv::f2(bias, bias);
                uint64_t acc[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t p[32];
#pragma unroll
                    for (int y = 0; y < 32; ++y) {
                        const float2 e = sv::f2_split(sv::f2_fma(sv::f2(x[64 * i + 2 * y], x[64 * i + 2 * y + 1]), scale2, bias2));
                        const float a = ex2(e.x), b = ex2(e.y);
                        acc[y & 1] = sv::f2_add(acc[y & 1], sv::f2(a, b));
                        p[y] = Half2<BF>::pack(a, b);
                    }
                    tc::tmem_st32(st + 32 * i, p);
                    // The first half's products start while the second half's weights are made.  (Not with 8-bit rows: beside
                    // the widening a look at one more barrier costs more than that, 2180 us against 1690 below.)
                    if constexpr (!E4) {
                        tc::wait_st();
                        tc::fence_before();
                        tc::bar_arrive(tc::smem_u32(&ms.pfull[half][i]));
                    }
                }
                const float2 s = sv::f2_split(sv::f2_add(acc[0], acc[1]));
                sum += s.x + s.y;
                if constexpr (E4) {
                    set_aside();
                    tc::wait_st();
                    tc::fence_before();
                    tc::bar_arrive(tc::smem_u32(&ms.pfull[half][0]));
                }
            }
            units += 2 * (g.j1 - g.j0);
            if (!ok) break;

            // ---- the segment's end: rows, or a part ----------------------------------------------
            const bool any = end > g.j0;
            if (any) {
                ok = __all_sync(0xffffffffu, tc::bar_wait(tc::smem_u32(&ms.odone[half]), ends & 1, abort));
                ++ends;
                if (!ok) break;
                tc::fence_after();
            }
            __threadfence_block();
            const bool poisoned = *(volatile int *)&ms.poison[seg & 3] == seg;
            // What was set aside, to the rows that see it.
            auto mend = [&](float (&o)[32], int d) {
                const int from = front + 1 > g.j0 * TILE ? front + 1 : g.j0 * TILE, to = edge < end * TILE - 1 ? edge : end * TILE - 1;
                for (int y = from; y <= to; ++y) {
                    const int64_t at = (int64_t)g.b * P.max_pos + y;
                    const int slot = SV_INB(at, (int64_t)P.B * P.max_pos, 1307) ? P.slot_table[at] : -1;
                    if (slot < 0 || slot >= P.num_slots) continue;
                    const unsigned char *src = P.v + slot * P.v_slot;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (32 * d + i >= P.D) continue;
                        uint32_t bits;
                        if constexpr (E4) bits = sv::E4m3Scale<BF>(sv::E4m3Scale<BF>::bits(src[P.Hkv * P.D + g.h]))(src[g.h * P.D + 32 * d + i]) & 0xffffu;
                        else bits = reinterpret_cast<const uint16_t *>(src)[g.h * P.D + 32 * d + i];
                        if ((bits & Half2<BF>::EXP_MASK) == Half2<BF>::EXP_MASK) o[i] += Half2<BF>::unpack(bits).x;
                    }
                }
            };
            const bool mine = n < g.nn;
            const int64_t row = ((int64_t)g.b * P.N + n) * P.Hq + g.h * P.G + h;
            const float inv = 1.f / sum;
            float *const part = P.parts + (int64_t)g.part * PART;
            const int r = half * HALF + t;
            if (g.part >= 0) {
                part[ROWS * MAXD + r] = ref;
                part[ROWS * MAXD + ROWS + r] = sum;
            } else if (mine && P.lse && SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1305)) {
                P.lse[row] = (log2f(sum) - add) * 0.69314718f;
            }
            if (any) {
#pragma unroll 1
                for (int d = 0; d < dsteps; ++d) {
                    float o[32];
                    __syncwarp();
                    tc::tmem_ld32(ot + 32 * d, o);
                    tc::wait_ld(o);
                    if (!mine || !SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1306)) continue;
                    if (poisoned) mend(o, d);
                    if (g.part >= 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<float4 *>(part)[(8 * d + i) * ROWS + r] =
                                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    } else {
                        uint4 *const dst = reinterpret_cast<uint4 *>(P.out + row * P.D + 32 * d);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (32 * d + 8 * i < P.D)
                                dst[i] = make_uint4(Half2<BF>::pack(o[8 * i] * inv, o[8 * i + 1] * inv),
                                                    Half2<BF>::pack(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                                    Half2<BF>::pack(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                                    Half2<BF>::pack(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                    }
                }
            }
            tc::fence_before();
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (ms.abort) {
        // A bounded wait ran out: what is written is not an answer.  The products in flight end (again with a limit)
        // before their memory is given back; the copies were waited for.  A commit is for the products of its own
        // thread: the lane that issued them, which every election picks.
        if (warp == 4 && tc::elect()) {
            atomicAdd(&tc::g_timeouts, 1ull);
            const int64_t begin = clock64();
            tc::commit(tc::smem_u32(&ms.drain));
            while (!tc::bar_try(tc::smem_u32(&ms.drain), 0) && clock64() - begin < tc::WAIT_CLOCKS) {}
            if (P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_TIMEOUT);
        }
        __syncthreads();
    }
    if (warp == 4) tc::tmem_free(tmem, 512);
}

// The second kernel: rows of nodes that are not there, requests whose lengths are wrong, and the blocks in parts.  (The
// first has two warps with nothing to do, but no registers for them: 4096 tokens over 8-bit rows took 1990 us against
// 1690.)  A slice is 4 rows of a block; 4 groups of threads take every fourth part, a thread 4 dimensions of a row.
constexpr int JT = 512, SLICES = ROWS / 4;

template <bool BF>
__global__ void __launch_bounds__(JT) finish_kernel(const __grid_constant__ Params P)
{
    __shared__ int s_list[MAX_SMS], s_warp[JT / 32];
    __shared__ float s_part[3][6][128];
    const int tid = threadIdx.x;
    // Requests are shared by as many CTAs as there are to each.
    const int share = P.B >= (int)gridDim.x ? 1 : gridDim.x / P.B;
    for (int64_t w = blockIdx.x; w < (int64_t)P.B * share; w += gridDim.x) {
        const int b = (int)(w / share), s = (int)(w - (int64_t)b * share);
        const Request r = request(P, b);
        if (r.wrong && s == 0 && tid == 0 && P.dev_status) atomicMax(P.dev_status, SPEC_VERIFY_DEV_BAD_KV_POSITION);
        const uint32_t fill = r.wrong ? Half2<BF>::NAN2 : 0u;
        const int64_t from = ((int64_t)b * P.N + r.nn) * P.Hq, rows = (int64_t)(P.N - r.nn) * P.Hq;
        uint4 *const out = reinterpret_cast<uint4 *>(P.out + from * P.D);
        for (int64_t i = (int64_t)s * JT + tid; i < rows * P.D / 8; i += (int64_t)share * JT)
            out[i] = make_uint4(fill, fill, fill, fill);
        if (P.lse)
            for (int64_t i = (int64_t)s * JT + tid; i < rows; i += (int64_t)share * JT) P.lse[from + i] = r.wrong ? NAN : -INFINITY;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // The CTAs whose runs began a block that others ended.
    bool has = false;
    if (tid < P.ctas) {
        const int4 lo = __ldcg(reinterpret_cast<const int4 *>(P.joins + tid)), hi = __ldcg(reinterpret_cast<const int4 *>(P.joins + tid) + 1);
        has = hi.x > lo.w;  // c1 > c0
    }
    const unsigned all = __ballot_sync(0xffffffffu, has);
    if ((tid & 31) == 0) s_warp[tid >> 5] = __popc(all);
    __syncthreads();
    int before = 0, count = 0;
#pragma unroll
    for (int w = 0; w < (MAX_SMS + 31) / 32; ++w) {
        before += w < tid >> 5 ? s_warp[w] : 0;
        count += s_warp[w];
    }
    if (has) s_list[before + __popc(all & ((1u << (tid & 31)) - 1))] = tid;
    __syncthreads();
    const int group = tid >> 7, x = tid & 127, d = x >> 2;
#pragma unroll 1
    for (int w = blockIdx.x; w < count * SLICES; w += gridDim.x) {
        const Join jn = P.joins[s_list[w / SLICES]];
        const int r = (w % SLICES) * 4 + (x & 3);
        const unsigned gr = (unsigned)jn.qb * ROWS + r, n = gr / (unsigned)P.G, h = gr - n * P.G;
        const bool live = (int)n < jn.nn && 4 * d < P.D;
        const int parts = jn.c1 - jn.c0 + 1;
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // Sums join at the higher reference; a part without weight has none (NaN has).
        auto join = [&](float m, float l, const float4 &o) {
            if (l == 0.f) return;
            const float now = fmaxf(top, m);
            const float f0 = sv::reference_factor<BF>(top, now, P.scale_log2), f1 = sv::reference_factor<BF>(m, now, P.scale_log2);
            top = now;
            sum = sum * f0 + l * f1;
            // (A factor of 0 leaves what is not finite among values of next to no weight NaN.)
            acc.x = acc.x * f0 + o.x * f1;
            acc.y = acc.y * f0 + o.y * f1;
            acc.z = acc.z * f0 + o.z * f1;
            acc.w = acc.w * f0 + o.w * f1;
        };
        if (live) {
#pragma unroll 4
            for (int p = group; p < parts; p += 4) {
                const float *part = P.parts + (int64_t)(2 * (jn.c0 + p) + (p == 0)) * PART;
                const float m = __ldcg(part + ROWS * MAXD + r), l = __ldcg(part + ROWS * MAXD + ROWS + r);
                const float4 o = __ldcg(reinterpret_cast<const float4 *>(part) + d * ROWS + r);
                join(m, l, o);
            }
        }
        __syncthreads();
        if (group) {
            float *const y = &s_part[group - 1][0][x];
            y[0] = top, y[128] = sum, y[256] = acc.x, y[384] = acc.y, y[512] = acc.z, y[640] = acc.w;
        }
        __syncthreads();
        if (group == 0 && live) {
            for (int i = 0; i < 3; ++i) {
                const float *y = &s_part[i][0][x];
                join(y[0], y[128], make_float4(y[256], y[384], y[512], y[640]));
            }
            const int64_t row = ((int64_t)jn.b * P.N + n) * P.Hq + jn.h * P.G + h;
            if (SV_INB(row, (int64_t)P.B * P.N * P.Hq, 1308)) {
                const float inv = 1.f / sum;
                reinterpret_cast<uint2 *>(P.out + row * P.D)[d] =
                    make_uint2(Half2<BF>::pack(acc.x * inv, acc.y * inv), Half2<BF>::pack(acc.z * inv, acc.w * inv));
                if (d == 0 && P.lse) P.lse[row] = (log2f(sum) - sv::reference_add<BF>(top, P.scale_log2)) * 0.69314718f;
            }
        }
    }
}

// -------------------------------------------------------------------------------------------------
// Host side.
// -------------------------------------------------------------------------------------------------
static std::mutex g_mu;
static int g_sms[64];

template <bool BF, int DP, bool E4>
constexpr size_t smem_bytes()
{
    return Layout<DP, E4>::M0 + sizeof(MiscOf<BF, DP, E4>);
}

template <bool BF, int DP, bool E4>
static bool allow()
{
    static_assert(smem_bytes<BF, DP, E4>() <= 232448, "shared memory of a CTA");
    return cudaFuncSetAttribute((const void *)chunk_kernel<BF, DP, E4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)smem_bytes<BF, DP, E4>()) == cudaSuccess;
}

// Once per device: the kernels' shared memory; the SM count, 0 when it cannot be had.
static int sm_count()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_sms[dev] == 0) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            !(allow<true, 64, false>() && allow<true, 128, false>() && allow<false, 64, false>() && allow<false, 128, false>() &&
              allow<true, 64, true>() && allow<true, 128, true>() && allow<false, 64, true>() && allow<false, 128, true>())) {
            cudaGetLastError();
            return 0;
        }
        g_sms[dev] = sms < MAX_SMS ? sms : MAX_SMS;
    }
    return g_sms[dev];
}

constexpr size_t COUNTER_BYTES = 65536 * 4;  // the workspace's region of counters, which other calls keep at zero
constexpr size_t JOIN_BYTES = MAX_SMS * sizeof(Join);
constexpr float MAX_SCALE = 2.3e38f;         // times log2(e) it is still a number of fp32

static bool sizes_ok(int B, int N, int Hq, int Hkv, int D, int max_pos)
{
    if (B < 1 || B > 65536 || N < 1 || (int64_t)B * N > 0x7fffffff || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq > (1 << 16) ||
        D < 64 || D > MAXD || D % 16 || max_pos < 1 || max_pos > 0x7fffffff - 1024 || (int64_t)N * (Hq / Hkv) > 0x7fffffff - ROWS)
        return false;
    // The batch's cost times the runs is formed in 64 bits.
    const double G = Hq / Hkv, blocks = (double)N * G / ROWS + 1;
    return (double)B * Hkv * blocks * (G * ((double)max_pos + SEGMENT + TILE) + ROWS * blocks) * MAX_SMS < 4e18;
}

template <class F>
static cudaError_t launch(F *kernel, const Params &P, int grid, int threads, size_t smem, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

template <bool BF, bool E4>
static cudaError_t dispatch(const Params &P, int sms, cudaStream_t s)
{
    const cudaError_t e = P.D <= 64 ? launch(chunk_kernel<BF, 64, E4>, P, P.ctas, NT, smem_bytes<BF, 64, E4>(), s)
                                    : launch(chunk_kernel<BF, 128, E4>, P, P.ctas, NT, smem_bytes<BF, 128, E4>(), s);
    return e != cudaSuccess ? e : launch(finish_kernel<BF>, P, 4 * sms, JT, 0, s);
}

}  // namespace svch

namespace sv {
bool chunk_timeouts(unsigned long long &n) { return tc::read_timeouts(n); }
bool chunk_wait_clocks(long long clocks) { return tc::set_wait_clocks(clocks); }

// This module's first range violation (debug builds; 0 otherwise), cleared when read.
unsigned long long chunk_debug_fault()
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

extern "C" size_t spec_verify_attention_chunk_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int max_pos)
{
    using namespace svch;
    if (!sizes_ok(B, N, Hq, Hkv, D, max_pos)) return 0;
    return COUNTER_BYTES + JOIN_BYTES + 2 * (size_t)MAX_SMS * PART * sizeof(float);
}

extern "C" int spec_verify_attention_chunk(const void *q, int dtype, int64_t q_stride, const void *k_cache,
                                           const void *v_cache, int cache_dtype, int64_t num_slots, int64_t k_slot_stride,
                                           int64_t v_slot_stride, const int32_t *slot_table, int max_pos,
                                           const int32_t *committed, const int32_t *num_nodes, int B, int N, int Hq,
                                           int Hkv, int D, float scale, void *out, float *lse, void *workspace,
                                           size_t ws_bytes, int32_t *dev_status, void *stream)
{
    using namespace svch;
    if (!q || !k_cache || !v_cache || !slot_table || !committed || !out || !workspace) return SPEC_VERIFY_EINVAL;
    if (dtype != SPEC_VERIFY_BF16 && dtype != SPEC_VERIFY_FP16) return SPEC_VERIFY_EINVAL;
    if (cache_dtype != dtype && cache_dtype != SPEC_VERIFY_E4M3) return SPEC_VERIFY_EINVAL;
    if (!sizes_ok(B, N, Hq, Hkv, D, max_pos) || num_slots < 1 || num_slots > 0x7fffffff || !(scale > 0.f) || scale > MAX_SCALE)
        return SPEC_VERIFY_EINVAL;
    const bool e4 = cache_dtype == SPEC_VERIFY_E4M3;
    const int64_t need = e4 ? sv::e4m3_row_bytes(Hkv, D) : (int64_t)Hkv * D, step = e4 ? 16 : 8;
    if (q_stride % 8 || q_stride < (int64_t)Hq * D || k_slot_stride % step || v_slot_stride % step || k_slot_stride < need ||
        v_slot_stride < need || k_slot_stride >= (1ll << 31) || v_slot_stride >= (1ll << 31))
        return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) % 16) return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)slot_table | (uintptr_t)committed | (uintptr_t)num_nodes | (uintptr_t)lse | (uintptr_t)dev_status) % 4)
        return SPEC_VERIFY_EINVAL;
    if (ws_bytes < spec_verify_attention_chunk_workspace_bytes(B, N, Hq, Hkv, D, max_pos) || (uintptr_t)workspace % 256)
        return SPEC_VERIFY_EWORKSPACE;
    const int sms = sm_count();
    if (!sms) return SPEC_VERIFY_ECUDA;
    Params P;
    P.q = static_cast<const uint16_t *>(q);
    P.k = static_cast<const unsigned char *>(k_cache);
    P.v = static_cast<const unsigned char *>(v_cache);
    P.out = static_cast<uint16_t *>(out);
    P.lse = lse;
    P.q_row = q_stride;
    P.k_slot = k_slot_stride * (e4 ? 1 : 2);
    P.v_slot = v_slot_stride * (e4 ? 1 : 2);
    P.num_slots = num_slots;
    P.slot_table = slot_table;
    P.committed = committed;
    P.num_nodes = num_nodes;
    P.max_pos = max_pos;
    P.B = B;
    P.N = N;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.D = D;
    P.G = Hq / Hkv;
    P.scale_log2 = (float)((double)scale * 1.4426950408889634);
    P.dev_status = dev_status;
    P.joins = reinterpret_cast<Join *>(static_cast<char *>(workspace) + COUNTER_BYTES);
    P.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + COUNTER_BYTES + JOIN_BYTES);
    P.ctas = sms;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SPEC_VERIFY_BF16 ? (e4 ? dispatch<true, true>(P, sms, s) : dispatch<true, false>(P, sms, s))
                                                    : (e4 ? dispatch<false, true>(P, sms, s) : dispatch<false, false>(P, sms, s));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return SPEC_VERIFY_ECUDA;
    }
    return SPEC_VERIFY_OK;
}
