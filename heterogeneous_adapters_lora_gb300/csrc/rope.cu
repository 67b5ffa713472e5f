// Norm and rotation of query and key heads in one pass over the packed QKV
// rows, keys and values to their cache rows (lora_qk_norm_rope):
//   n = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// HBM-bound: every row is read once and written once (12 KB each way per
// token at 32 + 2 x 8 heads of 128).  A head is held by the D / 8 lanes of a
// group (rounded up to a power of two), each with the two 4-element pieces
// whose elements rotate with each other, so the rotation needs no exchange
// between lanes and the norm one butterfly sum.  A group does U heads of one
// token: their loads are in flight together, and the token's cosines and
// sines are read once for all of them.
#include <math.h>
#include <string.h>

#include "lora_internal.cuh"

namespace {

constexpr int kThreads = 128;

struct RopeArgs {
    const uint16_t *qkv;
    long long ld_qkv;
    int T, hq, hkv, D, rot, max_pos, heads;  // heads: query, key and (when copied) value heads
    float eps, inv_d;
    const uint16_t *qw, *kw;
    const int32_t *positions;
    const float *cs;
    uint16_t *q, *k, *v;
    long long ld_q, ld_k, ld_v;
    const int32_t *slots;
    long long n_rows;
    int32_t *status;
    int lw_log;  // log2 of the lanes of a group
    int chunks;  // head chunks of a token
};

__device__ __forceinline__ void unpack4(uint2 u, float (&f)[4]) {
    f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
}
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    return make_uint2(*(const uint32_t *)&x, *(const uint32_t *)&y);
}

template <int U, bool kPairs>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(unit / p.chunks), chunk = (int)(unit % p.chunks);
    asm volatile("griddepcontrol.launch_dependents;");
    if (t >= p.T) return;
    const int lw = 1 << p.lw_log, l = lane & (lw - 1), group = lane >> p.lw_log;
    const int head0 = (chunk * U << (5 - p.lw_log)) + group;  // heads of this group: head0 + u * groups
    const int groups = 32 >> p.lw_log;
    const bool live = l * 8 < p.D, rotated = l * 8 < p.rot;
    // the lane's two pieces: elements that rotate with each other
    const int ea = !kPairs && rotated ? 4 * l : 8 * l;
    const int eb = !kPairs && rotated ? 4 * l + p.rot / 2 : 8 * l + 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int pos = p.rot ? __ldg(p.positions + t) : 0;
    const long long slot = p.slots ? (long long)__ldg(p.slots + t) : (long long)t;
    const uint16_t *row = p.qkv + (long long)t * p.ld_qkv;
    uint2 xa[U], xb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = head0 + u * groups;
        xa[u] = xb[u] = make_uint2(0u, 0u);
        if (live && h < p.heads) {
            xa[u] = *(const uint2 *)(row + (long long)h * p.D + ea);
            xb[u] = *(const uint2 *)(row + (long long)h * p.D + eb);
        }
    }
    if ((p.rot && (pos < 0 || pos >= p.max_pos)) || slot < -1 || slot >= p.n_rows) {
        if (lane == 0 && p.status) atomicExch(p.status, (int)LORA_ERR_DEVICE_INDEX);
        return;
    }
    float4 co = make_float4(0.f, 0.f, 0.f, 0.f), si = co;
    if (rotated) {
        const float *c = p.cs + (long long)pos * p.rot + 4 * l;
        co = __ldg((const float4 *)c);
        si = __ldg((const float4 *)(c + p.rot / 2));
    }
    const uint2 ones = make_uint2(0x3f803f80u, 0x3f803f80u);
    uint2 wqa = ones, wqb = ones, wka = ones, wkb = ones;
    if (live && p.qw) { wqa = __ldg((const uint2 *)(p.qw + ea)); wqb = __ldg((const uint2 *)(p.qw + eb)); }
    if (live && p.kw) { wka = __ldg((const uint2 *)(p.kw + ea)); wkb = __ldg((const uint2 *)(p.kw + eb)); }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = head0 + u * groups;
        float a[4], b[4];
        unpack4(xa[u], a);
        unpack4(xb[u], b);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss += a[i] * a[i] + b[i] * b[i];
        for (int o = lw >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!live || h >= p.heads) continue;
        if (h >= p.hq + p.hkv) {  // a value head: stored as it is
            if (slot >= 0) {
                uint16_t *o = p.v + slot * p.ld_v + (long long)(h - p.hq - p.hkv) * p.D;
                *(uint2 *)(o + ea) = xa[u];
                *(uint2 *)(o + eb) = xb[u];
            }
            continue;
        }
        const bool is_q = h < p.hq;
        const float r = rsqrtf(ss * p.inv_d + p.eps);
        float wa[4], wb[4];
        unpack4(is_q ? wqa : wka, wa);
        unpack4(is_q ? wqb : wkb, wb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = a[i] * r * wa[i];
            b[i] = b[i] * r * wb[i];
        }
        const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
        if (!rotated) {  // past the rotated part: no partner, not even times zero
        } else if (kPairs) {  // piece a = pairs 0, 1 of the lane, piece b = pairs 2, 3
            const float e[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            float o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[2 * i] = e[2 * i] * c4[i] - e[2 * i + 1] * s4[i];
                o[2 * i + 1] = e[2 * i + 1] * c4[i] + e[2 * i] * s4[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) { a[i] = o[i]; b[i] = o[4 + i]; }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = a[i] * c4[i] - b[i] * s4[i];
                b[i] = b[i] * c4[i] + a[i] * s4[i];
                a[i] = x;
            }
        }
        if (!is_q && slot < 0) continue;
        uint16_t *o = is_q ? p.q + (long long)t * p.ld_q + (long long)h * p.D
                           : p.k + slot * p.ld_k + (long long)(h - p.hq) * p.D;
        *(uint2 *)(o + ea) = pack4(a[0], a[1], a[2], a[3]);
        *(uint2 *)(o + eb) = pack4(b[0], b[1], b[2], b[3]);
    }
}

template <int U, bool kPairs>
cudaError_t rope_launch(RopeArgs &p, cudaStream_t s) {
    const int per = U << (5 - p.lw_log);
    p.chunks = (p.heads + per - 1) / per;
    const long long units = (long long)p.T * p.chunks;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)((units + kThreads / 32 - 1) / (kThreads / 32)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, rope_kernel<U, kPairs>, p);
}

}  // namespace

extern "C" lora_status_t lora_qk_norm_rope(const lora_rope_desc_t *desc, const void *qkv, int64_t ld_qkv, int32_t T,
                                           const void *q_weight, const void *k_weight, const int32_t *positions,
                                           const float *cos_sin, void *q_out, int64_t ld_q, void *k_out, int64_t ld_k,
                                           void *v_out, int64_t ld_v, const int32_t *slots, int64_t n_rows,
                                           int32_t *status, void *stream) {
    if (!desc || T < 0) return LORA_ERR_INVALID_ARG;
    const lora_rope_desc_t d = *desc;
    if (d.n_q_heads < 1 || d.n_kv_heads < 1 || d.n_q_heads > 65536 || d.n_kv_heads > 65536 || d.head_dim < 8 ||
        d.head_dim > 256 || d.head_dim % 8 || d.rot_dim < 0 || d.rot_dim > d.head_dim || d.rot_dim % 8 ||
        (d.interleaved != 0 && d.interleaved != 1) || (d.rot_dim && d.max_pos < 1) || !(d.eps >= 0.f) || isinf(d.eps))
        return LORA_ERR_INVALID_ARG;
    const int64_t qc = (int64_t)d.n_q_heads * d.head_dim, kc = (int64_t)d.n_kv_heads * d.head_dim;
    if (ld_qkv < qc + 2 * kc || ld_qkv % 8 || ld_q < qc || ld_q % 8 || ld_k < kc || ld_k % 8 ||
        (v_out && (ld_v < kc || ld_v % 8)) || n_rows < 0 || (!slots && n_rows < T))
        return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    if (!qkv || !q_out || !k_out || (d.rot_dim && (!positions || !cos_sin)) || !lora_aligned16(qkv) ||
        !lora_aligned16(q_out) || !lora_aligned16(k_out) || !lora_aligned16(v_out) || !lora_aligned16(q_weight) ||
        !lora_aligned16(k_weight) || !lora_aligned16(cos_sin) || ((uintptr_t)positions & 3) || ((uintptr_t)slots & 3) ||
        ((uintptr_t)status & 3))
        return LORA_ERR_INVALID_ARG;
    RopeArgs p;
    memset(&p, 0, sizeof(p));
    p.qkv = (const uint16_t *)qkv;
    p.ld_qkv = ld_qkv;
    p.T = T;
    p.hq = d.n_q_heads;
    p.hkv = d.n_kv_heads;
    p.D = d.head_dim;
    p.rot = d.rot_dim;
    p.max_pos = d.max_pos;
    p.heads = d.n_q_heads + d.n_kv_heads * (v_out ? 2 : 1);
    p.eps = d.eps;
    p.inv_d = 1.0f / (float)d.head_dim;
    p.qw = (const uint16_t *)q_weight;
    p.kw = (const uint16_t *)k_weight;
    p.positions = positions;
    p.cs = cos_sin;
    p.q = (uint16_t *)q_out;
    p.k = (uint16_t *)k_out;
    p.v = (uint16_t *)v_out;
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.ld_v = ld_v;
    p.slots = slots;
    p.n_rows = n_rows;
    p.status = status;
    while ((8 << p.lw_log) < d.head_dim) ++p.lw_log;
    const int per = 4 << (5 - p.lw_log);
    if ((long long)T * ((p.heads + per - 1) / per) > 0x7fffffffLL) return LORA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    LORA_CUDA_TRY(d.interleaved ? (rope_launch<4, true>(p, s)) : (rope_launch<4, false>(p, s)));
    lora_note_launch();
    return LORA_OK;
}
