// sv_logprobs.cu -- what is answered beside emitted tokens: the token's log probability, its rank,
// the distribution's entropy and its most likely alternatives.
//
//   x = logits / T, m = max x, Z = sum e^(x - m)
//   logprob(t) = x_t - m - ln Z, entropy = ln Z - sum (x - m) e^(x - m) / Z, rank = 1 + #{x > x_t}
//
// One CTA per row: a pass for the maximum, one for the sums and the rank, and one per alternative
// (the largest logit below the last one taken, ties to the lower token).
#include "sv_ops.cuh"

namespace svlp {

constexpr int NT = 512;
constexpr int MAX_TOP = 32;

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
};

__device__ __forceinline__ float logit(const __nv_bfloat16 *p, int i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float logit(const float *p, int i) { return p[i]; }

struct Key {
    float v;
    int i;
};
__device__ __forceinline__ bool better(Key a, Key b) { return a.v > b.v || (a.v == b.v && a.i < b.i); }

template <typename T>
__global__ void __launch_bounds__(NT) logprobs_kernel(const Params P)
{
    __shared__ float s_a[NT / 32], s_b[NT / 32];
    __shared__ int s_n[NT / 32];
    __shared__ Key s_k[NT / 32];
    const int64_t r = blockIdx.x;
    const int b = (int)(r / P.T), t = (int)(r - (int64_t)b * P.T), tid = threadIdx.x;
    const int tok = P.tokens[r];
    const int idx = P.row_index ? P.row_index[r] : t;
    const float temp = P.temperatures ? P.temperatures[b] : P.temperature;
    int code = tok < -1 || tok >= P.V ? SPEC_VERIFY_DEV_BAD_TOKEN : idx < -1 || idx >= P.rows ? SPEC_VERIFY_DEV_BAD_ROW : 0;
    const bool here = tok >= 0 && idx >= 0;
    float lp = 0.f, ent = 0.f, M = 0.f, lz = 0.f;
    int rank = 0;
    const float inv = temp == 0.f ? 1.f : 1.f / temp;
    const T *x = nullptr;
    if (!code && here) {
        x = static_cast<const T *>(P.logits) + ((int64_t)b * P.rows + idx) * P.V;
        float m = -INFINITY;
        int bad = 0;
        for (int i = tid; i < P.V; i += NT) {
            const float y = logit(x, i);
            if (y != y || y == INFINITY) bad = 1;
            m = fmaxf(m, y);
        }
        bad = __syncthreads_or(bad);
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (tid % 32 == 0) s_a[tid / 32] = m;
        __syncthreads();
        for (int w = 0; w < NT / 32; ++w) m = fmaxf(m, s_a[w]);
        __syncthreads();
        M = m;
        if (bad || m == -INFINITY || !(temp >= 0.f)) code = SPEC_VERIFY_DEV_BAD_ROW;
        const float xt = logit(x, tok);
        float z = 0.f, e1 = 0.f;
        for (int i = tid; i < P.V; i += NT) {
            const float y = logit(x, i), d = (y - m) * inv, e = expf(d);
            z += e;
            if (e > 0.f) e1 += e * d;
            rank += y > xt;
        }
        for (int o = 16; o; o >>= 1) {
            z += __shfl_xor_sync(~0u, z, o);
            e1 += __shfl_xor_sync(~0u, e1, o);
            rank += __shfl_xor_sync(~0u, rank, o);
        }
        if (tid % 32 == 0) s_a[tid / 32] = z, s_b[tid / 32] = e1, s_n[tid / 32] = rank;
        __syncthreads();
        z = e1 = 0.f;
        rank = 1;
        for (int w = 0; w < NT / 32; ++w) z += s_a[w], e1 += s_b[w], rank += s_n[w];
        lz = logf(z);
        lp = (xt - m) * inv - lz;
        ent = lz - e1 / z;
    }
    if (code) lp = ent = NAN, rank = -1;
    if (tid == 0) {
        P.logprobs[r] = lp;
        if (P.entropy) P.entropy[r] = ent;
        if (P.ranks) P.ranks[r] = rank;
        if (code && P.dev_status) atomicMax(P.dev_status, code);
    }
    Key last = {INFINITY, -1};
    for (int k = 0; k < P.top; ++k) {
        Key best = {-INFINITY, 0x7fffffff};
        if (!code && here)
            for (int i = tid; i < P.V; i += NT) {
                const Key y = {logit(x, i), i};
                if (better(last, y) && better(y, best)) best = y;
            }
        for (int o = 16; o; o >>= 1) {
            const Key y = {__shfl_xor_sync(~0u, best.v, o), __shfl_xor_sync(~0u, best.i, o)};
            if (better(y, best)) best = y;
        }
        __syncthreads();
        if (tid % 32 == 0) s_k[tid / 32] = best;
        __syncthreads();
        for (int w = 0; w < NT / 32; ++w)
            if (better(s_k[w], best)) best = s_k[w];
        last = best;
        if (tid == 0) {
            const bool any = !code && here && best.v > -INFINITY;
            P.top_ids[r * P.top + k] = any ? best.i : -1;
            P.top_logprobs[r * P.top + k] = code ? NAN : any ? (best.v - M) * inv - lz : -INFINITY;
        }
    }
}

}  // namespace svlp

extern "C" size_t spec_verify_logprobs_workspace_bytes(int B, int T, int V, int top_n)
{
    if (B < 1 || B > 65536 || T < 1 || T > sv::MAX_TREE || V < 1 || top_n < 0 || top_n > svlp::MAX_TOP) return 0;
    return 256;
}

extern "C" int spec_verify_logprobs(const void *logits, int dtype, const int32_t *tokens, const int32_t *row_index, int B,
                                    int rows, int T, int V, const float *temperatures, float temperature, int top_n,
                                    float *logprobs, float *entropy, int32_t *ranks, int32_t *top_ids,
                                    float *top_logprobs, void *workspace, size_t ws_bytes, int32_t *dev_status,
                                    void *stream)
{
    if (!logits || !tokens || !logprobs || !workspace) return SPEC_VERIFY_EINVAL;
    if (dtype != SPEC_VERIFY_BF16 && dtype != SPEC_VERIFY_FP32) return SPEC_VERIFY_EINVAL;
    const size_t need = spec_verify_logprobs_workspace_bytes(B, T, V, top_n);
    if (!need || rows < 1 || rows > sv::MAX_TREE || (top_n && (!top_ids || !top_logprobs)) || (!row_index && T > rows))
        return SPEC_VERIFY_EINVAL;
    if (!temperatures && !(temperature >= 0.f && temperature < 3e38f)) return SPEC_VERIFY_EINVAL;
    if ((uintptr_t)logits % (dtype == SPEC_VERIFY_BF16 ? 2 : 4) ||
        ((uintptr_t)tokens | (uintptr_t)row_index | (uintptr_t)temperatures | (uintptr_t)logprobs | (uintptr_t)entropy |
         (uintptr_t)ranks | (uintptr_t)top_ids | (uintptr_t)top_logprobs | (uintptr_t)dev_status) % 4)
        return SPEC_VERIFY_EINVAL;
    if (ws_bytes < need || (uintptr_t)workspace % 256) return SPEC_VERIFY_EWORKSPACE;
    svlp::Params P = {logits, tokens, row_index, temperatures, temperature, B, rows, T, V, top_n, logprobs, entropy,
                      ranks, top_n ? top_ids : nullptr, top_n ? top_logprobs : nullptr, dev_status};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(B * T);
    if (dtype == SPEC_VERIFY_BF16) svlp::logprobs_kernel<__nv_bfloat16><<<grid, svlp::NT, 0, s>>>(P);
    else svlp::logprobs_kernel<float><<<grid, svlp::NT, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? SPEC_VERIFY_OK : SPEC_VERIFY_ECUDA;
}
