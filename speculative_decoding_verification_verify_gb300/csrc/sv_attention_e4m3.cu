// sv_attention_e4m3.cu -- attention of a verification step's nodes over a paged cache of 8-bit rows.
#include "sv_attention.cuh"

namespace sv {
bool attention_e4m3_timeouts(unsigned long long &n) { return tc::read_timeouts(n); }
bool attention_e4m3_wait_clocks(long long clocks) { return tc::set_wait_clocks(clocks); }

// This module's first range violation (debug builds; 0 otherwise), cleared when read.
unsigned long long attention_e4m3_debug_fault()
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

extern "C" size_t spec_verify_attention_e4m3_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int max_pos)
{
    return svatt::workspace_bytes(B, N, Hq, Hkv, D, max_pos, true);
}

extern "C" int spec_verify_attention_e4m3(const void *q, int dtype, int64_t q_stride, const void *k_cache,
                                          const void *v_cache, int64_t num_slots, int64_t k_slot_stride,
                                          int64_t v_slot_stride, const int32_t *slot_table, int max_pos,
                                          const int32_t *committed, const int32_t *parents, const int32_t *num_nodes, int B,
                                          int N, int Hq, int Hkv, int D, float scale, void *out, float *lse, void *workspace,
                                          size_t ws_bytes, int32_t *dev_status, void *stream)
{
    return svatt::run<true>(q, dtype, q_stride, k_cache, v_cache, num_slots, k_slot_stride, v_slot_stride, slot_table, max_pos,
                          committed, parents, num_nodes, B, N, Hq, Hkv, D, scale, out, lse, workspace, ws_bytes, dev_status,
                          stream);
}
