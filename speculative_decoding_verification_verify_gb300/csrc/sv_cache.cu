// sv_cache.cu -- what writes and reads the paged cache beside the attention kernels, its rows in 16 or in 8 bits:
// append with heads' norms and the position rotation, and positions read back as contiguous rows.
//
//   append:  x = x * w / sqrt(mean(x^2) + eps) over a head of q or k (where a weight is given), then the rotation of
//            sv_append.cu, then q to q_out and k, v to their slot: rounded to 16 bits, or to e4m3 (sv_e4m3.cuh)
//   read:    out[b][n] = the row at position first[b] + n
//
// Bytes bound both.  A thread of append has two 16-byte vectors of a head, which under either pairing hold whole
// pairs (as in sv_append.cu); the lanes that share a head are neighbours, so that a norm's sum and a head's largest
// magnitude are a few exchanges, and a row passes through registers once.
//
// Measured (GB300, copy rate 6.68 TB/s; 32 query and 8 key heads of 128; in a graph, a call waited for in a row of calls
// in brackets): append of 8194 rows with norms to 8-bit rows 44 us (48) for 185 MB, 4.2 TB/s, its instructions at 76% of the
// issue slots; to 16-bit rows 39 us (42) for 201 MB, 5.1 TB/s; 384 rows 4.5 us, one row 3 us.  Read of 48 requests' 24
// thousand 8-bit rows 27 us (29) for 127 MB, 4.7 TB/s; of 60001 rows of 4 heads of 80 28 us (31) for 117 MB, 4.2 TB/s: the
// chain slot table, slot, row at 48 warps an SM.  Of 16-bit rows, 48 x 504 in all 33 us (36) for 198 MB, 6.0 TB/s; 60001 of
// 4 x 80 28 us (31) for 154 MB, 5.5 TB/s.
#include "sv_e4m3.cuh"

#include <initializer_list>
#include <type_traits>

namespace svc {

using sv::Half2;

constexpr int NT = 128;  // threads per CTA of append: a CTA takes a row

struct Append {
    const uint4 *q, *k, *v, *q_norm, *k_norm;
    uint4 *q_out;
    unsigned char *k_cache, *v_cache;
    int64_t q_row, k_row, v_row;  // in 16-byte vectors
    int64_t k_slot, v_slot;       // in bytes
    int64_t num_slots;
    const int32_t *slot_table, *committed, *parents, *num_nodes;
    const float *cos_sin;
    float eps;
    int rot_positions, rot;
    int B, N, Hq, Hkv, D, max_pos;
    int lanes;  // that share a head: the power of two from D / 16 on
    int32_t *dev_status;
};

template <bool BF>
__device__ __forceinline__ void to_float(const uint4 &a, float (&x)[8])
{
    const uint32_t *w = &a.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Half2<BF>::unpack(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <bool BF>
__device__ __forceinline__ uint4 to_half(const float (&x)[8])
{
    return make_uint4(Half2<BF>::pack(x[0], x[1]), Half2<BF>::pack(x[2], x[3]), Half2<BF>::pack(x[4], x[5]),
                      Half2<BF>::pack(x[6], x[7]));
}

// a * b + c * d, the second product's rounding made good: two roundings are left, of the sum and of what makes it good.
// (An infinite product has no rounding: the difference is NaN, the sum is what it is.)
__device__ __forceinline__ float sum2(float a, float b, float c, float d)
{
    const float p = c * d, e = fmaf(c, d, -p), s = fmaf(a, b, p), y = s + e;
    return y == y ? y : s;
}

// What is rounded to four digits is worked out more exactly than what keeps eight: each of fp32's roundings that is saved
// is as many fewer values next to a border that fall on its other side.
template <bool FINE>
__device__ __forceinline__ void turn(float &x, float &y, float c, float s)
{
    const float a = FINE ? sum2(x, c, -y, s) : x * c - y * s, b = FINE ? sum2(y, c, x, s) : y * c + x * s;
    x = a;
    y = b;
}

// x * r * w, r the reciprocal of a root of x's head: x * r is a number of modest size, r * w may pass fp32.
template <bool FINE>
__device__ __forceinline__ float scaled(float x, float r, float w)
{
    const float p = x * r;
    if (!FINE) return p * w;
    const float e = fmaf(x, r, -p);
    return fmaf(p, w, e * w);
}

template <bool BF, bool ADJ, bool E4>
__global__ void __launch_bounds__(NT) append_kernel(const Append P)
{
    __shared__ int s_par[sv::MAX_TREE];
    __shared__ int s_bad;
    const int64_t row = blockIdx.x;
    const int b = (int)((unsigned)row / (unsigned)P.N), n = (int)(row - (int64_t)b * P.N), tid = threadIdx.x;
    [[maybe_unused]] const int64_t rows = (int64_t)P.B * P.N;
    const int hv = P.D / 8, hu = hv / 2;  // a head's vectors and pairs of them
    const int rv = P.rot / 8;             // rotated vectors of a head (even)
    const int j = tid & (P.lanes - 1), per = NT / P.lanes;  // the thread's pair of its head; heads at a time
    const int heads = P.Hq + 2 * P.Hkv;
    const bool live = j < hu;
    const bool turned = 2 * j < rv;
    const int i0 = !ADJ && turned ? j : 2 * j, i1 = !ADJ && turned ? j + rv / 2 : 2 * j + 1;
    const int c = SV_INB(b, P.B, 1201) ? P.committed[b] : 0;
    const int nn = P.num_nodes && SV_INB(b, P.B, 1202) ? P.num_nodes[b] : P.N;

    auto load = [&](int head, uint4 &x, uint4 &y) {
        const bool is_q = head < P.Hq, is_k = head < P.Hq + P.Hkv;
        const uint4 *base = is_q ? P.q : is_k ? P.k : P.v;
        const int64_t stride = is_q ? P.q_row : is_k ? P.k_row : P.v_row;
        const int64_t at = row * stride + (int64_t)(head - (is_q ? 0 : is_k ? P.Hq : P.Hq + P.Hkv)) * hv;
        if (!SV_INB(n, nn, 1207) || !SV_INB(at + i1, (rows - 1) * stride + (int64_t)(is_q ? P.Hq : P.Hkv) * hv, 1206)) return;
        x = base[at + i0];
        y = base[at + i1];
    };

    // The thread's first vectors, before anything is known of where they go; a row that the caller says is not
    // there is not read.
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    const int first = tid / P.lanes;
    if (n < nn && live && first < heads) load(first, va, vb);

    int code = 0;
    if (nn < 0 || nn > P.N || c < 0 || (int64_t)c + nn > P.max_pos) code = SPEC_VERIFY_DEV_BAD_KV_POSITION;
    const bool here = n < nn;
    int slot = 0;
    if (!code && here) {
        const int64_t i = (int64_t)b * P.max_pos + c + n;
        slot = SV_INB(i, (int64_t)P.B * P.max_pos, 1204) ? P.slot_table[i] : -1;
    }
    int depth = n;
    bool bad_tree = false;
    if (P.parents) {
        if (tid == 0) s_bad = 0;
        __syncthreads();
        if (tid < P.N && tid < nn && SV_INB((int64_t)b * P.N + tid, rows, 1203)) {
            const int p = P.parents[(int64_t)b * P.N + tid];
            s_par[tid] = p;
            if (tid == 0 ? p != -1 : (p < 0 || p >= tid)) s_bad = 1;
        }
        __syncthreads();
        bad_tree = s_bad;
        if (!bad_tree && !code && here) {
            depth = 0;
            for (int a = n; a > 0; a = s_par[a]) ++depth;
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
            if (SV_INB(row * P.Hq * hv + i, rows * P.Hq * hv, 1205)) P.q_out[row * P.Hq * hv + i] = make_uint4(w, w, w, w);
        return;
    }

    // The angles are the same for all of the thread's heads.
    float cs[8], sn[8];
    if (live && turned) {
        const float *at = P.cos_sin + ((int64_t)c + depth) * P.rot + 8 * j;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(at) + i);
            const float4 y = __ldg(reinterpret_cast<const float4 *>(at + P.rot / 2) + i);
            cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
            sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
        }
    }
    // (All lanes go through the exchanges, those beyond the last head with nothing.)
    for (int h0 = 0; h0 < heads; h0 += per) {
        const int head = h0 + first;
        const bool mine = live && head < heads;
        const bool is_q = head < P.Hq, is_k = !is_q && head < P.Hq + P.Hkv;
        float x[8], y[8];
        to_float<BF>(va, x);
        to_float<BF>(vb, y);
        if (live && head + per < heads) load(head + per, va, vb);  // the next ones' while these are worked on
        else va = vb = make_uint4(0, 0, 0, 0);
        const uint4 *weight = is_q ? P.q_norm : is_k ? P.k_norm : nullptr;
        if (P.q_norm || P.k_norm) {
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 8; ++i) part[i & 3] += x[i] * x[i] + y[i] * y[i];
            float sum = (part[0] + part[1]) + (part[2] + part[3]);
            for (int o = P.lanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (weight && mine) {
                const float r = __frsqrt_rn(sum / (float)P.D + P.eps);
                float w[8];
                to_float<BF>(__ldg(weight + i0), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = E4 && is_k ? scaled<true>(x[i], r, w[i]) : scaled<false>(x[i], r, w[i]);
                to_float<BF>(__ldg(weight + i1), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = E4 && is_k ? scaled<true>(y[i], r, w[i]) : scaled<false>(y[i], r, w[i]);
            }
        }
        auto rotate = [&](auto fine) {
            constexpr bool F = decltype(fine)::value;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!ADJ) {
                    turn<F>(x[i], y[i], cs[i], sn[i]);
                } else if (i < 4) {
                    turn<F>(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
                    turn<F>(y[2 * i], y[2 * i + 1], cs[4 + i], sn[4 + i]);
                }
            }
        };
        if (live && turned) {
            if (E4 && is_k) rotate(std::true_type());
            else if (is_q || is_k) rotate(std::false_type());
        }
        if (is_q) {
            if (mine) {
                uint4 *const dst = P.q_out + row * P.Hq * hv + head * hv;
                dst[i0] = to_half<BF>(x);
                dst[i1] = to_half<BF>(y);
            }
        }
        const int kv = head - P.Hq - (is_k ? 0 : P.Hkv);  // the key head
        unsigned char *const dst = is_k ? P.k_cache + (int64_t)slot * P.k_slot : P.v_cache + (int64_t)slot * P.v_slot;
        if (!E4) {
            if (mine && !is_q) {
                reinterpret_cast<uint4 *>(dst)[kv * hv + i0] = to_half<BF>(x);
                reinterpret_cast<uint4 *>(dst)[kv * hv + i1] = to_half<BF>(y);
            }
        } else if (h0 + per > P.Hq) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(y[i])));
            for (int o = P.lanes / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (mine && !is_q) {
                const int e = sv::e4m3_exponent(top, BF);
                const float f = sv::exp2_int(-e);
                auto pack = [&](const float (&z)[8]) {
                    return make_uint2(sv::e4m3_pack(z[0] * f, z[1] * f) | sv::e4m3_pack(z[2] * f, z[3] * f) << 16,
                                      sv::e4m3_pack(z[4] * f, z[5] * f) | sv::e4m3_pack(z[6] * f, z[7] * f) << 16);
                };
                reinterpret_cast<uint2 *>(dst)[kv * hv + i0] = pack(x);
                reinterpret_cast<uint2 *>(dst)[kv * hv + i1] = pack(y);
                if (j == 0) dst[P.Hkv * P.D + kv] = (unsigned char)(e + 127);
            }
        }
    }
    if (E4) {
        const int used = P.Hkv * (P.D + 1), pad = (int)sv::e4m3_row_bytes(P.Hkv, P.D) - used;
        if (tid < 2 * pad) {
            unsigned char *const dst = tid < pad ? P.k_cache + (int64_t)slot * P.k_slot : P.v_cache + (int64_t)slot * P.v_slot;
            dst[used + tid % pad] = 0;
        }
    }
}

struct Read {
    const unsigned char *k, *v;
    uint4 *k_out, *v_out;
    int64_t k_slot, v_slot, num_slots;  // strides in bytes
    const int32_t *slot_table, *first, *num_rows;
    int B, N, Hkv, D, max_pos;
    int units;  // of a row of k or v, 16 values each
    int32_t *dev_status;
};

// A warp takes the keys and the values of two rows, so that its lanes have their places with few divisions, and 16
// values of them a lane at a time, READ_U of those under way.  Stores of 32 bytes fill a sector each.
constexpr int READ_NT = 256, READ_SIDES = 4, READ_U = 2;

__device__ __forceinline__ void store32(void *at, const uint4 &x, const uint4 &y)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x),
                 "r"(y.y), "r"(y.z), "r"(y.w)
                 : "memory");
}

template <bool BF, bool E4>
__global__ void __launch_bounds__(READ_NT) read_kernel(const Read P)
{
    const int lane = threadIdx.x & 31, U = P.units;
    const int64_t sides = 2 * (int64_t)P.B * P.N;
    const int64_t side0 = ((int64_t)blockIdx.x * (READ_NT / 32) + (threadIdx.x >> 5)) * READ_SIDES;
    // The first lanes find the sides' rows: where they are (0: nowhere), and what is there instead.
    const unsigned char *from = nullptr;
    uint32_t fill = 0;
    if (lane < READ_SIDES && side0 + lane < sides) {
        const int64_t row = (side0 + lane) >> 1;
        const int b = (int)((unsigned)row / (unsigned)P.N), n = (int)(row - (int64_t)b * P.N);
        const int c = SV_INB(b, P.B, 1211) ? P.first[b] : 0;
        const int nn = P.num_rows && SV_INB(b, P.B, 1212) ? P.num_rows[b] : P.N;
        int code = 0;
        if (nn < 0 || nn > P.N || c < 0 || (int64_t)c + nn > P.max_pos) {
            code = SPEC_VERIFY_DEV_BAD_KV_POSITION;
        } else if (n < nn) {
            const int64_t s = (int64_t)b * P.max_pos + c + n;
            const int slot = SV_INB(s, (int64_t)P.B * P.max_pos, 1213) ? P.slot_table[s] : -1;
            if (slot < 0 || slot >= P.num_slots) code = SPEC_VERIFY_DEV_BAD_KV_SLOT;
            else from = lane & 1 ? P.v + (int64_t)slot * P.v_slot : P.k + (int64_t)slot * P.k_slot;
        }
        if (code) {
            fill = Half2<BF>::NAN2;
            if (P.dev_status) atomicMax(P.dev_status, code);
        }
    }
    const int total = (int)(sides - side0 < READ_SIDES ? (sides > side0 ? sides - side0 : 0) : READ_SIDES) * U;
    for (int i0 = 0; i0 < total; i0 += 32 * READ_U) {
        uint4 x[READ_U], y[READ_U];
        uint32_t scale[READ_U];
        unsigned char *to[READ_U];
#pragma unroll
        for (int i = 0; i < READ_U; ++i) {
            const int at = i0 + 32 * i + lane, s = min((unsigned)at / (unsigned)U, (unsigned)(READ_SIDES - 1)), u = at - s * U;
            const unsigned char *src = reinterpret_cast<const unsigned char *>(__shfl_sync(0xffffffffu, (unsigned long long)from, s));
            const uint32_t f = __shfl_sync(0xffffffffu, fill, s);
            to[i] = nullptr;
            if (at >= total) continue;
            x[i] = y[i] = make_uint4(f, f, f, f);
            scale[i] = 0;
            to[i] = reinterpret_cast<unsigned char *>((s & 1 ? P.v_out : P.k_out) + 2 * (((side0 + s) >> 1) * U + u));
            if (!src) continue;
            if (E4) {
                x[i] = __ldg(reinterpret_cast<const uint4 *>(src) + u);
                scale[i] = 1u << 31 | src[P.Hkv * P.D + (unsigned)u * 16u / (unsigned)P.D];
            } else {
                x[i] = __ldg(reinterpret_cast<const uint4 *>(src) + 2 * u);
                y[i] = __ldg(reinterpret_cast<const uint4 *>(src) + 2 * u + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < READ_U; ++i) {
            if (!to[i]) continue;
            if (E4 && scale[i]) {
                // (In bf16 as the attentions widen, so that its subnormals are the same to all.  In fp16 rows that were
                // written from bf16 may have powers that it lacks.)
                const float f = __uint_as_float(scale[i] << 23);
                const sv::E4m3Scale<true> widen(sv::E4m3Scale<true>::bits(scale[i] & 0xff));
                auto two = [&](uint32_t bits) {
                    if (BF) return widen(bits);
                    const float2 z = sv::e4m3_unpack(bits & 0xffffu);
                    return Half2<BF>::pack(z.x * f, z.y * f);
                };
                const uint4 z = x[i];
                x[i] = make_uint4(two(z.x), two(z.x >> 16), two(z.y), two(z.y >> 16));
                y[i] = make_uint4(two(z.z), two(z.z >> 16), two(z.w), two(z.w >> 16));
            }
            store32(to[i], x[i], y[i]);
        }
    }
}

static bool aligned(std::initializer_list<const void *> p, uintptr_t a)
{
    for (const void *x : p)
        if ((uintptr_t)x % a) return false;
    return true;
}

// Whether a cache's slots of these heads can be what the caller says.
static bool cache_ok(int cache_dtype, int64_t num_slots, int64_t k_stride, int64_t v_stride, int Hkv, int D)
{
    if (num_slots < 1 || num_slots > 0x7fffffff) return false;
    const int64_t need = cache_dtype == SPEC_VERIFY_E4M3 ? sv::e4m3_row_bytes(Hkv, D) : (int64_t)Hkv * D;
    const int64_t step = cache_dtype == SPEC_VERIFY_E4M3 ? 16 : 8;
    return k_stride % step == 0 && v_stride % step == 0 && k_stride >= need && v_stride >= need;
}

}  // namespace svc

namespace sv {
// This module's first range violation (debug builds; 0 otherwise), cleared when read.
unsigned long long cache_debug_fault()
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

extern "C" size_t spec_verify_kv_e4m3_row_bytes(int Hkv, int D)
{
    if (Hkv < 1 || D < 16 || D % 16 || D > 512 || (int64_t)Hkv * D > (1 << 24)) return 0;
    return (size_t)sv::e4m3_row_bytes(Hkv, D);
}

extern "C" int spec_verify_kv_append_ex(const void *q, const void *k, const void *v, int dtype, int64_t q_stride,
                                        int64_t k_stride, int64_t v_stride, void *q_out, void *k_cache, void *v_cache,
                                        int cache_dtype, int64_t num_slots, int64_t k_slot_stride, int64_t v_slot_stride,
                                        const int32_t *slot_table, int max_pos, const int32_t *committed,
                                        const int32_t *parents, const int32_t *num_nodes, const float *cos_sin,
                                        int rot_positions, int rotary_dim, int interleaved, const void *q_norm,
                                        const void *k_norm, float eps, int B, int N, int Hq, int Hkv, int D,
                                        int32_t *dev_status, void *stream)
{
    using namespace svc;
    if (!q || !k || !v || !q_out || !k_cache || !v_cache || !slot_table || !committed) return SPEC_VERIFY_EINVAL;
    if (dtype != SPEC_VERIFY_BF16 && dtype != SPEC_VERIFY_FP16) return SPEC_VERIFY_EINVAL;
    if (cache_dtype != dtype && cache_dtype != SPEC_VERIFY_E4M3) return SPEC_VERIFY_EINVAL;
    if (B < 1 || N < 1 || (int64_t)B * N > 0x7fffffff || (parents && N > sv::MAX_TREE) || max_pos < 1) return SPEC_VERIFY_EINVAL;
    if (Hq < 1 || Hkv < 1 || D < 16 || D % 16 || D > 512 || (int64_t)(Hq + 2 * (int64_t)Hkv) * D > (1 << 24))
        return SPEC_VERIFY_EINVAL;
    if (rotary_dim < 0 || rotary_dim % 16 || rotary_dim > D || (rotary_dim && (!cos_sin || rot_positions < 1)))
        return SPEC_VERIFY_EINVAL;
    if ((q_norm || k_norm) && !(eps >= 0.f && eps <= 3.4e38f)) return SPEC_VERIFY_EINVAL;
    const int64_t qw = (int64_t)Hq * D, kw = (int64_t)Hkv * D;
    if (q_stride % 8 || k_stride % 8 || v_stride % 8 || q_stride < qw || k_stride < kw || v_stride < kw ||
        !cache_ok(cache_dtype, num_slots, k_slot_stride, v_slot_stride, Hkv, D))
        return SPEC_VERIFY_EINVAL;
    if (!aligned({q, k, v, q_out, k_cache, v_cache, cos_sin, q_norm, k_norm}, 16) ||
        !aligned({slot_table, committed, parents, num_nodes, dev_status}, 4))
        return SPEC_VERIFY_EINVAL;
    const uintptr_t q0 = (uintptr_t)q, o0 = (uintptr_t)q_out, rows = (uintptr_t)B * N;
    if (q0 < o0 + rows * qw * 2 && o0 < q0 + ((rows - 1) * q_stride + qw) * 2) return SPEC_VERIFY_EINVAL;
    const int elt = cache_dtype == SPEC_VERIFY_E4M3 ? 1 : 2;
    Append P;
    P.q = static_cast<const uint4 *>(q);
    P.k = static_cast<const uint4 *>(k);
    P.v = static_cast<const uint4 *>(v);
    P.q_norm = static_cast<const uint4 *>(q_norm);
    P.k_norm = static_cast<const uint4 *>(k_norm);
    P.q_out = static_cast<uint4 *>(q_out);
    P.k_cache = static_cast<unsigned char *>(k_cache);
    P.v_cache = static_cast<unsigned char *>(v_cache);
    P.q_row = q_stride / 8;
    P.k_row = k_stride / 8;
    P.v_row = v_stride / 8;
    P.k_slot = k_slot_stride * elt;
    P.v_slot = v_slot_stride * elt;
    P.num_slots = num_slots;
    P.slot_table = slot_table;
    P.committed = committed;
    P.parents = parents;
    P.num_nodes = num_nodes;
    P.cos_sin = cos_sin;
    P.eps = eps;
    P.rot_positions = rot_positions;
    P.rot = rotary_dim;
    P.B = B;
    P.N = N;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.D = D;
    P.max_pos = max_pos;
    P.lanes = 1;
    while (P.lanes < D / 16) P.lanes *= 2;
    P.dev_status = dev_status;
    const unsigned grid = (unsigned)((int64_t)B * N);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto bf, auto e4) {
        if (interleaved) append_kernel<decltype(bf)::value, true, decltype(e4)::value><<<grid, NT, 0, s>>>(P);
        else append_kernel<decltype(bf)::value, false, decltype(e4)::value><<<grid, NT, 0, s>>>(P);
    };
    using T = std::true_type;
    using F = std::false_type;
    const bool e4 = cache_dtype == SPEC_VERIFY_E4M3;
    if (dtype == SPEC_VERIFY_BF16) e4 ? launch(T(), T()) : launch(T(), F());
    else e4 ? launch(F(), T()) : launch(F(), F());
    return cudaGetLastError() == cudaSuccess ? SPEC_VERIFY_OK : SPEC_VERIFY_ECUDA;
}

extern "C" int spec_verify_kv_read(const void *k_cache, const void *v_cache, int cache_dtype, int64_t num_slots,
                                   int64_t k_slot_stride, int64_t v_slot_stride, const int32_t *slot_table, int max_pos,
                                   const int32_t *first, const int32_t *num_rows, int B, int N, int Hkv, int D,
                                   void *k_out, void *v_out, int dtype, int32_t *dev_status, void *stream)
{
    using namespace svc;
    if (!k_cache || !v_cache || !slot_table || !first || !k_out || !v_out) return SPEC_VERIFY_EINVAL;
    if (dtype != SPEC_VERIFY_BF16 && dtype != SPEC_VERIFY_FP16) return SPEC_VERIFY_EINVAL;
    if (cache_dtype != dtype && cache_dtype != SPEC_VERIFY_E4M3) return SPEC_VERIFY_EINVAL;
    if (B < 1 || N < 1 || (int64_t)B * N > 0x7fffffff || max_pos < 1) return SPEC_VERIFY_EINVAL;
    if (Hkv < 1 || D < 16 || D % 16 || D > 512 || (int64_t)Hkv * D > (1 << 23)) return SPEC_VERIFY_EINVAL;
    if (!cache_ok(cache_dtype, num_slots, k_slot_stride, v_slot_stride, Hkv, D)) return SPEC_VERIFY_EINVAL;
    if (!aligned({k_cache, v_cache}, 16) || !aligned({k_out, v_out}, 32) || !aligned({slot_table, first, num_rows, dev_status}, 4))
        return SPEC_VERIFY_EINVAL;
    const int elt = cache_dtype == SPEC_VERIFY_E4M3 ? 1 : 2;
    Read P;
    P.k = static_cast<const unsigned char *>(k_cache);
    P.v = static_cast<const unsigned char *>(v_cache);
    P.k_out = static_cast<uint4 *>(k_out);
    P.v_out = static_cast<uint4 *>(v_out);
    P.k_slot = k_slot_stride * elt;
    P.v_slot = v_slot_stride * elt;
    P.num_slots = num_slots;
    P.slot_table = slot_table;
    P.first = first;
    P.num_rows = num_rows;
    P.B = B;
    P.N = N;
    P.Hkv = Hkv;
    P.D = D;
    P.max_pos = max_pos;
    P.units = Hkv * (D / 16);
    P.dev_status = dev_status;
    constexpr int PER = READ_SIDES * (READ_NT / 32);
    const int64_t grid = (2 * (int64_t)B * N + PER - 1) / PER;
    if (grid > 0x7fffffff) return SPEC_VERIFY_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool e4 = cache_dtype == SPEC_VERIFY_E4M3;
    if (dtype == SPEC_VERIFY_BF16)
        e4 ? read_kernel<true, true><<<(unsigned)grid, READ_NT, 0, s>>>(P) : read_kernel<true, false><<<(unsigned)grid, READ_NT, 0, s>>>(P);
    else
        e4 ? read_kernel<false, true><<<(unsigned)grid, READ_NT, 0, s>>>(P) : read_kernel<false, false><<<(unsigned)grid, READ_NT, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? SPEC_VERIFY_OK : SPEC_VERIFY_ECUDA;
}
