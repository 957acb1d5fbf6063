// sv_append.cu -- the verify forward's new keys and values into the paged cache, with the position
// rotation applied on the way, and the queries rotated beside them.
//
//   position of node n = committed + depth(n)      (chain: committed + n)
//   slot of node n     = slot_table[committed + n]
//   (x_i, x_j) -> (x_i cos - x_j sin, x_j cos + x_i sin), j = i + rot/2, or pairs (2i, 2i + 1)
//
// Bytes bound it: every row is read once and written once, and the 3 operations per element are
// nothing beside that.  For few rows its time is the chain of dependent round trips (committed,
// then slot and cosines, then the stores), so the rows' own loads are issued first and the index
// chain runs under them.  A CTA takes one node: its unit of work is a pair of 16-byte vectors,
// which under either pairing holds whole pairs (half-split: vectors rot/2 apart; adjacent: any
// two), so a thread needs one unit's cosines and sines and no exchange with its neighbours.
// Measured (GB300, copy rate 6.68 TB/s; 32 query and 8 key heads of 128, in a graph): 8194 rows 33 us for
// 204 MB, 6.2 TB/s; 384 rows 3.6 us and one row 2.9 us, the chain's length.  Narrow rows are bound by the CTAs
// that come and go, one for each: 8194 rows of 3 + 2 heads of 64 take 9.5 us for 13 MB, of 4 + 2 heads of 128
// 10.9 us for 29 MB.
#include "sv_ops.cuh"

namespace svapp {

using sv::Half2;

// Threads per CTA.  A thread has one unit in flight, whatever the row's width: with three, 8194 rows of 5 heads of
// 64 took 12.6 us against 9.5, of 12 heads of 128 15.4 against 12.9, of 48 35.4 against 33.2, of 80 52.3 against
// 52.7; a single row of 48 heads 2.75 against 2.87.
constexpr int NT = 128;

struct Params {
    const uint4 *q, *k, *v;            // rows of heads * D elements, row_*  vectors apart
    uint4 *q_out, *k_cache, *v_cache;
    int64_t q_row, k_row, v_row, q_out_row;  // in 16-byte vectors
    int64_t k_slot, v_slot;                  // slot strides, in 16-byte vectors
    int64_t num_slots;
    const int32_t *slot_table, *committed, *parents, *num_nodes;
    const float *cos_sin;
    int rot_positions, rot;
    int B, N, Hq, Hkv, D, max_pos;
    int32_t *dev_status;
};

// Rotate the pairs of one unit: c, s hold the eight angles of the vectors' elements (half-split),
// or four angles for each vector (adjacent pairs).
template <bool BF, bool ADJ>
__device__ __forceinline__ void rotate(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8])
{
    uint32_t *wa = &a.x, *wb = &b.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = Half2<BF>::unpack(wa[i]), y = Half2<BF>::unpack(wb[i]);
        if (ADJ) {
            wa[i] = Half2<BF>::pack(x.x * c[i] - x.y * s[i], x.y * c[i] + x.x * s[i]);
            wb[i] = Half2<BF>::pack(y.x * c[4 + i] - y.y * s[4 + i], y.y * c[4 + i] + y.x * s[4 + i]);
        } else {
            wa[i] = Half2<BF>::pack(x.x * c[2 * i] - y.x * s[2 * i], x.y * c[2 * i + 1] - y.y * s[2 * i + 1]);
            wb[i] = Half2<BF>::pack(y.x * c[2 * i] + x.x * s[2 * i], y.y * c[2 * i + 1] + x.y * s[2 * i + 1]);
        }
    }
}

template <bool BF, bool ADJ>
__global__ void __launch_bounds__(NT) append_kernel(const Params P)
{
    __shared__ int s_par[sv::MAX_TREE];
    __shared__ int s_bad;
    const int64_t row = blockIdx.x;
    const int b = (int)((unsigned)row / (unsigned)P.N), n = (int)(row - (int64_t)b * P.N), tid = threadIdx.x;
    [[maybe_unused]] const int64_t rows = (int64_t)P.B * P.N;
    const int hv = P.D / 8, hu = hv / 2;  // a head's vectors and units
    const int units = (P.Hq + 2 * P.Hkv) * hu;
    const int rv = P.rot / 8;  // rotated vectors of a head (even)
    const int c = SV_INB(b, P.B, 1001) ? P.committed[b] : 0;
    const int nn = P.num_nodes && SV_INB(b, P.B, 1002) ? P.num_nodes[b] : P.N;

    // A unit's two vectors: (j, j + rv/2) among the rotated ones when pairs are half a rotation
    // apart, else neighbours.
    struct Unit {
        int head, j, i0, i1;
        bool turned;
    };
    auto unit = [&](int u) {
        Unit x;
        x.head = (unsigned)u / (unsigned)hu;
        x.j = u - x.head * hu;
        x.turned = 2 * x.j < rv;
        x.i0 = !ADJ && x.turned ? x.j : 2 * x.j;
        x.i1 = !ADJ && x.turned ? x.j + rv / 2 : 2 * x.j + 1;
        return x;
    };
    auto load = [&](const Unit &x, uint4 &a, uint4 &c) {
        const bool is_q = x.head < P.Hq, is_k = x.head < P.Hq + P.Hkv;
        const uint4 *base = is_q ? P.q : is_k ? P.k : P.v;
        const int64_t stride = is_q ? P.q_row : is_k ? P.k_row : P.v_row;
        const int64_t at = row * stride + (x.head - (is_q ? 0 : is_k ? P.Hq : P.Hq + P.Hkv)) * hv;
        if (!SV_INB(n, nn, 1007) || !SV_INB(at + x.i1, (rows - 1) * stride + (is_q ? P.Hq : P.Hkv) * hv, 1006)) return;
        a = base[at + x.i0];
        c = base[at + x.i1];
    };

    // The thread's first vectors, before anything is known of where they go; a row that the caller says is not
    // there is not read.
    uint4 va, vb;
    if (n < nn && tid < units) load(unit(tid), va, vb);

    int code = 0;
    if (nn < 0 || nn > P.N || c < 0 || (int64_t)c + nn > P.max_pos) code = SPEC_VERIFY_DEV_BAD_KV_POSITION;
    const bool here = n < nn;
    int slot = 0;
    if (!code && here) {
        const int64_t i = (int64_t)b * P.max_pos + c + n;
        slot = SV_INB(i, (int64_t)P.B * P.max_pos, 1004) ? P.slot_table[i] : -1;
    }
    int depth = n;
    bool bad_tree = false;
    if (P.parents) {
        if (tid == 0) s_bad = 0;
        __syncthreads();
        if (tid < P.N && tid < nn && SV_INB((int64_t)b * P.N + tid, rows, 1003)) {
            const int p = P.parents[(int64_t)b * P.N + tid];
            s_par[tid] = p;
            if (tid == 0 ? p != -1 : (p < 0 || p >= tid)) s_bad = 1;
        }
        __syncthreads();
        bad_tree = s_bad;
        if (!bad_tree && !code && here) {
            depth = 0;
            for (int j = n; j > 0; j = s_par[j]) ++depth;
        }
    }
    // The faults, the later ones of the list only where the earlier ones leave them a meaning.
    if (!code && here && !bad_tree) {
        if (P.rot && (int64_t)c + depth >= P.rot_positions) code = SPEC_VERIFY_DEV_BAD_KV_POSITION;
        else if (slot < 0 || slot >= P.num_slots) code = SPEC_VERIFY_DEV_BAD_KV_SLOT;
    }
    if (!code && bad_tree) code = SPEC_VERIFY_DEV_BAD_TREE;
    if (code && tid == 0 && P.dev_status) atomicMax(P.dev_status, code);
    if (code || !here) {  // nothing is appended; the row's queries are zeros (absent) or NaN (a fault)
        const uint32_t w = code ? Half2<BF>::NAN2 : 0u;
        for (int i = tid; i < P.Hq * hv; i += NT)
            if (SV_INB(row * P.q_out_row + i, rows * P.q_out_row, 1005))
                P.q_out[row * P.q_out_row + i] = make_uint4(w, w, w, w);
        return;
    }
    const float *cs = P.cos_sin + ((int64_t)c + depth) * P.rot;
    for (int u = tid; u < units; u += NT) {
        const Unit x = unit(u);
        if (u != tid) load(x, va, vb);
        const bool is_q = x.head < P.Hq, is_k = x.head < P.Hq + P.Hkv;
        if (x.turned && is_k) {
            const float4 *pc = reinterpret_cast<const float4 *>(cs + 8 * x.j);
            const float4 *ps = reinterpret_cast<const float4 *>(cs + 8 * x.j + P.rot / 2);
            const float4 c0 = __ldg(pc), c1 = __ldg(pc + 1), s0 = __ldg(ps), s1 = __ldg(ps + 1);
            const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
            rotate<BF, ADJ>(va, vb, cc, ss);
        }
        uint4 *const dst = (is_q    ? P.q_out + row * P.q_out_row
                            : is_k ? P.k_cache + (int64_t)slot * P.k_slot - P.Hq * hv
                                   : P.v_cache + (int64_t)slot * P.v_slot - (P.Hq + P.Hkv) * hv) +
                           x.head * hv;
        dst[x.i0] = va;
        dst[x.i1] = vb;
    }
}

}  // namespace svapp

namespace sv {
// This module's first range violation (debug builds; 0 otherwise), cleared when read.
unsigned long long append_debug_fault()
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

extern "C" int spec_verify_kv_append(const void *q, const void *k, const void *v, int dtype, int64_t q_stride,
                                     int64_t k_stride, int64_t v_stride, void *q_out, void *k_cache, void *v_cache,
                                     int64_t num_slots, int64_t k_slot_stride, int64_t v_slot_stride,
                                     const int32_t *slot_table, int max_pos, const int32_t *committed,
                                     const int32_t *parents, const int32_t *num_nodes, const float *cos_sin,
                                     int rot_positions, int rotary_dim, int interleaved, int B, int N, int Hq, int Hkv,
                                     int D, int32_t *dev_status, void *stream)
{
    if (!q || !k || !v || !q_out || !k_cache || !v_cache || !slot_table || !committed) return SPEC_VERIFY_EINVAL;
    if (dtype != SPEC_VERIFY_BF16 && dtype != SPEC_VERIFY_FP16) return SPEC_VERIFY_EINVAL;
    if (B < 1 || N < 1 || (int64_t)B * N > 0x7fffffff || (parents && N > sv::MAX_TREE) || max_pos < 1 || num_slots < 1 ||
        num_slots > 0x7fffffff)
        return SPEC_VERIFY_EINVAL;
    if (Hq < 1 || Hkv < 1 || D < 16 || D % 16 || D > 1024 || (int64_t)(Hq + 2 * (int64_t)Hkv) * D > (1 << 24))
        return SPEC_VERIFY_EINVAL;
    if (rotary_dim < 0 || rotary_dim % 16 || rotary_dim > D || (rotary_dim && (!cos_sin || rot_positions < 1)))
        return SPEC_VERIFY_EINVAL;
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hkv * D;
    if (q_stride % 8 || k_stride % 8 || v_stride % 8 || k_slot_stride % 8 || v_slot_stride % 8) return SPEC_VERIFY_EINVAL;
    if (q_stride < qw || k_stride < kw || v_stride < kw || k_slot_stride < kw || v_slot_stride < kw)
        return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)k_cache | (uintptr_t)v_cache |
         (uintptr_t)cos_sin) % 16)
        return SPEC_VERIFY_EINVAL;
    if (((uintptr_t)slot_table | (uintptr_t)committed | (uintptr_t)parents | (uintptr_t)num_nodes |
         (uintptr_t)dev_status) % 4)
        return SPEC_VERIFY_EINVAL;
    const uintptr_t q0 = (uintptr_t)q, o0 = (uintptr_t)q_out, rows = (uintptr_t)B * N;
    if (q0 < o0 + rows * qw * 2 && o0 < q0 + ((rows - 1) * q_stride + qw) * 2) return SPEC_VERIFY_EINVAL;
    svapp::Params P;
    P.q = static_cast<const uint4 *>(q);
    P.k = static_cast<const uint4 *>(k);
    P.v = static_cast<const uint4 *>(v);
    P.q_out = static_cast<uint4 *>(q_out);
    P.k_cache = static_cast<uint4 *>(k_cache);
    P.v_cache = static_cast<uint4 *>(v_cache);
    P.q_row = q_stride / 8;
    P.k_row = k_stride / 8;
    P.v_row = v_stride / 8;
    P.q_out_row = qw / 8;
    P.k_slot = k_slot_stride / 8;
    P.v_slot = v_slot_stride / 8;
    P.num_slots = num_slots;
    P.slot_table = slot_table;
    P.committed = committed;
    P.parents = parents;
    P.num_nodes = num_nodes;
    P.cos_sin = cos_sin;
    P.rot_positions = rot_positions;
    P.rot = rotary_dim;
    P.B = B;
    P.N = N;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.D = D;
    P.max_pos = max_pos;
    P.dev_status = dev_status;
    const unsigned grid = (unsigned)((int64_t)B * N);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SPEC_VERIFY_BF16) {
        if (interleaved) svapp::append_kernel<true, true><<<grid, svapp::NT, 0, s>>>(P);
        else svapp::append_kernel<true, false><<<grid, svapp::NT, 0, s>>>(P);
    } else {
        if (interleaved) svapp::append_kernel<false, true><<<grid, svapp::NT, 0, s>>>(P);
        else svapp::append_kernel<false, false><<<grid, svapp::NT, 0, s>>>(P);
    }
    return cudaGetLastError() == cudaSuccess ? SPEC_VERIFY_OK : SPEC_VERIFY_ECUDA;
}
