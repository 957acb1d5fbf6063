// sv_attention.cu -- attention of a verification step's nodes over the paged cache.
//
//   s_j = scale * q . k_j over the positions j that node n sees: j < committed, and the positions
//   committed + a of the nodes a on the path from the root to n (a chain: a <= n)
//   out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), lse = m + ln sum_j e^(s_j - m)
//
// One CTA per (request, node, query head); its warps take the positions in turn, lanes split a
// head's dimensions, each warp keeps a running (max, sum, weighted values) and they are merged at
// the end.  A position a node does not see is skipped, so nothing stored there can matter.
#include "sv_ops.cuh"

namespace svatt {

using sv::Half2;

constexpr int NW = 4, NT = 32 * NW;
constexpr int MAXD = 128;

struct Params {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;
    int64_t q_row, k_slot, v_slot, num_slots;
    const int32_t *slot_table, *committed, *parents, *num_nodes;
    int max_pos, B, N, Hq, Hkv, D;
    float scale_log2;
    int32_t *dev_status;
};

template <bool BF>
__global__ void __launch_bounds__(NT) attention_kernel(const Params P)
{
    __shared__ float s_m[NW], s_l[NW], s_o[NW][MAXD];
    __shared__ int s_par[sv::MAX_TREE];
    __shared__ int s_code;
    __shared__ unsigned long long s_path;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % P.Hq;
    const int64_t row = blockIdx.x / P.Hq;
    const int b = (int)(row / P.N), n = (int)(row - (int64_t)b * P.N);
    const int c = P.committed[b];
    const int nn = P.num_nodes ? P.num_nodes[b] : P.N;
    if (tid == 0) s_code = nn < 0 || nn > P.N || c < 0 || (int64_t)c + nn > P.max_pos ? SPEC_VERIFY_DEV_BAD_KV_POSITION : 0;
    __syncthreads();
    if (P.parents && tid < nn && tid < P.N) {
        const int p = P.parents[(int64_t)b * P.N + tid];
        s_par[tid] = p;
        if (tid == 0 ? p != -1 : (p < 0 || p >= tid)) atomicMax(&s_code, SPEC_VERIFY_DEV_BAD_TREE);
    }
    __syncthreads();
    if (tid == 0) {
        unsigned long long path = 0;
        if (!s_code && n < nn) {
            if (P.parents)
                for (int j = n; j >= 0; j = s_par[j]) path |= 1ull << j;
            else
                path = ~0ull >> (63 - n);
        }
        s_path = path;
    }
    __syncthreads();
    const unsigned long long path = s_path;
    const int len = s_code ? 0 : c + nn;
    float qv[MAXD / 32], o[MAXD / 32], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < MAXD / 32; ++i) {
        const int d = i * 32 + lane;
        qv[i] = d < P.D ? Half2<BF>::unpack(P.q[row * P.q_row + (int64_t)h * P.D + d]).x : 0.f;
        o[i] = 0.f;
    }
    const int64_t hk = (int64_t)(h / (P.Hq / P.Hkv)) * P.D;
    for (int j = warp; j < len; j += NW) {
        const int slot = P.slot_table[(int64_t)b * P.max_pos + j];
        if (slot < 0 || slot >= P.num_slots) {
            if (lane == 0) atomicMax(&s_code, SPEC_VERIFY_DEV_BAD_KV_SLOT);
            continue;
        }
        if (n >= nn || (j >= c && !((path >> (j - c)) & 1))) continue;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < MAXD / 32; ++i) {
            const int d = i * 32 + lane;
            if (d < P.D) s += qv[i] * Half2<BF>::unpack(P.k[(int64_t)slot * P.k_slot + hk + d]).x;
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= P.scale_log2;
        const float nm = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.f : exp2f(m - nm), p = exp2f(s - nm);
        l = l * f + p;
        m = nm;
#pragma unroll
        for (int i = 0; i < MAXD / 32; ++i) {
            const int d = i * 32 + lane;
            if (d < P.D) o[i] = o[i] * f + p * Half2<BF>::unpack(P.v[(int64_t)slot * P.v_slot + hk + d]).x;
        }
    }
#pragma unroll
    for (int i = 0; i < MAXD / 32; ++i) s_o[warp][i * 32 + lane] = o[i];
    s_m[warp] = m;
    s_l[warp] = l;
    __syncthreads();
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < NW; ++w) {
        if (s_l[w] == 0.f) continue;  // the warp saw no position
        const float f = exp2f(s_m[w] - M);
        L += f * s_l[w];
        acc += f * s_o[w][tid];
    }
    const float val = s_code ? NAN : (n < nn ? acc / L : 0.f);
    if (tid < P.D) {
        const uint32_t w = Half2<BF>::pack(val, val);
        P.out[(row * P.Hq + h) * P.D + tid] = (uint16_t)w;
    }
    if (tid == 0) {
        if (P.lse) P.lse[row * P.Hq + h] = s_code ? NAN : (n < nn ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY);
        if (s_code && P.dev_status) atomicMax(P.dev_status, s_code);
    }
}

}  // namespace svatt

extern "C" size_t spec_verify_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int max_pos)
{
    if (B < 1 || B > 65536 || N < 1 || N > sv::MAX_TREE || Hq < 1 || Hkv < 1 || Hq % Hkv || D < 64 || D > svatt::MAXD ||
        D % 16 || max_pos < 1)
        return 0;
    return 256;
}

extern "C" int spec_verify_attention(const void *q, int dtype, int64_t q_stride, const void *k_cache,
                                     const void *v_cache, int64_t num_slots, int64_t k_slot_stride,
                                     int64_t v_slot_stride, const int32_t *slot_table, int max_pos,
                                     const int32_t *committed, const int32_t *parents, const int32_t *num_nodes, int B,
                                     int N, int Hq, int Hkv, int D, float scale, void *out, float *lse, void *workspace,
                                     size_t ws_bytes, int32_t *dev_status, void *stream)
{
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
    svatt::Params P;
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
    P.scale_log2 = (float)((double)scale * 1.4426950408889634);
    P.dev_status = dev_status;
    const int64_t grid = (int64_t)B * N * Hq;
    if (grid > 0x7fffffff) return SPEC_VERIFY_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SPEC_VERIFY_BF16) svatt::attention_kernel<true><<<(unsigned)grid, svatt::NT, 0, s>>>(P);
    else svatt::attention_kernel<false><<<(unsigned)grid, svatt::NT, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? SPEC_VERIFY_OK : SPEC_VERIFY_ECUDA;
}
