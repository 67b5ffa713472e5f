// A whole layer of experts for a few tokens: the chosen experts' products, the
// deltas of the tokens' adapters, the activation and the weighted sum.
#include <math.h>
#include <string.h>

#include "lora_internal.cuh"

namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

struct LayerArgs {
    int T, K, P, E, D, F, gelu;
    const uint16_t *x, *w13, *w2;
    long long ldx, ld13, ld2, ld_out;
    const int32_t *ids, *idx;
    const float *topk_w;
    uint16_t *out;
    int *status;
    // adapters (L = 0: none); two w13 slices or one of both
    int L, R, n13, shared;
    const uint16_t *A[3], *B[3];  // gate, up, w2
    long long a_ss[3], b_ss[3];   // elements of a slot
    long long a_es[3];            // ... of an expert of A (0: one for all)
    int b_up;                     // first up row in B of an expert (F where gate and up share a slice)
    int b_rows[3];                // rows of B per expert (0: one for all)
    const int32_t *rank, *enabled;
    const float *scale;
    float *v13, *h, *v2;          // [P][2][R], [P][F], [P][R]
};

__device__ __forceinline__ int expert_of(const LayerArgs &p, int pair, bool note) {
    const int e = p.ids[pair];
    if (e >= 0 && e < p.E) return e;
    if (note && e != -1 && p.status) atomicExch(p.status, (int)LORA_ERR_DEVICE_INDEX);
    return -1;
}
__device__ __forceinline__ int slot_of(const LayerArgs &p, int t, bool note) {
    if (!p.L) return -1;
    const int a = p.idx[t];
    if (a < 0 || a >= p.L) {
        if (note && a != -1 && p.status) atomicExch(p.status, (int)LORA_ERR_DEVICE_INDEX);
        return -1;
    }
    return p.enabled[a] && p.rank[a] > 0 ? a : -1;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
// products of 8 pairs of bf16
__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
    return bf16lo(a.x) * bf16lo(b.x) + bf16hi(a.x) * bf16hi(b.x) + bf16lo(a.y) * bf16lo(b.y) + bf16hi(a.y) * bf16hi(b.y) +
           bf16lo(a.z) * bf16lo(b.z) + bf16hi(a.z) * bf16hi(b.z) + bf16lo(a.w) * bf16lo(b.w) + bf16hi(a.w) * bf16hi(b.w);
}
__device__ __forceinline__ float dot8(uint4 a, float4 b, float4 c) {
    return bf16lo(a.x) * b.x + bf16hi(a.x) * b.y + bf16lo(a.y) * b.z + bf16hi(a.y) * b.w + bf16lo(a.z) * c.x +
           bf16hi(a.z) * c.y + bf16lo(a.w) * c.z + bf16hi(a.w) * c.w;
}
__device__ __forceinline__ float dot_bf16(const uint16_t *a, const uint16_t *b, int n, int lane) {
    float s = 0.f;
    for (int i = lane * 8; i < n; i += 256) s += dot8(__ldg((const uint4 *)(a + i)), __ldg((const uint4 *)(b + i)));
    return warp_sum(s);
}
__device__ __forceinline__ float dot_f32(const uint16_t *a, const float *b, int n, int lane) {
    float s = 0.f;
    for (int i = lane * 8; i < n; i += 256)
        s += dot8(__ldg((const uint4 *)(a + i)), __ldcg((const float4 *)(b + i)), __ldcg((const float4 *)(b + i + 4)));
    return warp_sum(s);
}

// scale * A x of every pair: a warp per (pair, slice, rank row)
__global__ void __launch_bounds__(kThreads) shrink13_kernel(const LayerArgs p) {
    const long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (long long)p.P * 2 * p.R) return;
    const int r = (int)(i % p.R), s = (int)(i / p.R % 2), pair = (int)(i / p.R / 2), t = pair / p.K;
    const int e = expert_of(p, pair, false), a = slot_of(p, t, false);
    if (e < 0 || a < 0 || r >= p.rank[a]) return;
    const int n = p.n13 == 2 ? s : 0;
    const uint16_t *A = p.A[n] + (long long)a * p.a_ss[n] + (long long)e * p.a_es[n] + (long long)r * p.D;
    const float v = dot_bf16(A, p.x + t * p.ldx, p.D, lane);
    if (lane == 0) p.v13[i] = v * p.scale[a];
}

__device__ __forceinline__ float activation(float g, int gelu) {
    if (gelu) return 0.5f * g * (1.f + tanhf(0.7978845608f * (g + 0.044715f * g * g * g)));
    return g / (1.f + expf(-g));
}

__device__ __forceinline__ float expand(const uint16_t *b, const float *v, int rank) {
    float s = 0.f;
    for (int r = 0; r < rank; ++r) s += __uint_as_float((uint32_t)b[r] << 16) * v[r];
    return s;
}

// h of every pair: a warp per (pair, f)
__global__ void __launch_bounds__(kThreads) up_kernel(const LayerArgs p) {
    const long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (long long)p.P * p.F) return;
    const int f = (int)(i % p.F), pair = (int)(i / p.F), t = pair / p.K;
    const int e = expert_of(p, pair, f == 0 && lane == 0), a = slot_of(p, t, f == 0 && lane == 0);
    if (e < 0) return;
    const uint16_t *w = p.w13 + ((long long)e * 2 * p.F + f) * p.ld13;
    float g = dot_bf16(w, p.x + t * p.ldx, p.D, lane);
    float u = dot_bf16(w + (long long)p.F * p.ld13, p.x + t * p.ldx, p.D, lane);
    if (a >= 0) {
        const int rank = p.rank[a], rs = (rank + 7) & ~7, n = p.n13 - 1;
        const float *v = p.v13 + (long long)pair * 2 * p.R;
        g += expand(p.B[0] + (long long)a * p.b_ss[0] + ((long long)e * p.b_rows[0] + f) * rs, v, rank);
        u += expand(p.B[n] + (long long)a * p.b_ss[n] + ((long long)e * p.b_rows[n] + p.b_up + f) * rs, v + p.R, rank);
    }
    if (lane == 0) p.h[i] = activation(g, p.gelu) * u;
}

// scale * A2 h of every pair: a warp per (pair, rank row)
__global__ void __launch_bounds__(kThreads) shrink2_kernel(const LayerArgs p) {
    const long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (long long)p.P * p.R) return;
    const int r = (int)(i % p.R), pair = (int)(i / p.R), t = pair / p.K;
    const int e = expert_of(p, pair, false), a = slot_of(p, t, false);
    if (e < 0 || a < 0 || r >= p.rank[a]) return;
    const uint16_t *A = p.A[2] + (long long)a * p.a_ss[2] + (long long)e * p.a_es[2] + (long long)r * p.F;
    const float v = dot_f32(A, p.h + (long long)pair * p.F, p.F, lane);
    if (lane == 0) p.v2[i] = v * p.scale[a];
}

// out of every token: a warp per (token, d)
__global__ void __launch_bounds__(kThreads) down_kernel(const LayerArgs p) {
    const long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (long long)p.T * p.D) return;
    const int d = (int)(i % p.D), t = (int)(i / p.D);
    const int a = slot_of(p, t, false);
    float sum = 0.f;
    for (int k = 0; k < p.K; ++k) {
        const int pair = t * p.K + k, e = expert_of(p, pair, false);
        if (e < 0) continue;
        float y = dot_f32(p.w2 + ((long long)e * p.D + d) * p.ld2, p.h + (long long)pair * p.F, p.F, lane);
        if (a >= 0) {
            const int rank = p.rank[a], rs = (rank + 7) & ~7;
            y += expand(p.B[2] + (long long)a * p.b_ss[2] + ((long long)e * p.b_rows[2] + d) * rs, p.v2 + (long long)pair * p.R,
                        rank);
        }
        sum += (p.topk_w ? p.topk_w[pair] : 1.f) * y;
    }
    const __nv_bfloat16 b = __float2bfloat16_rn(sum);
    if (lane == 0) p.out[t * p.ld_out + d] = *(const uint16_t *)&b;
}

bool desc_ok(const lora_moe_layer_desc_t &d) {
    return d.n_experts >= 1 && d.n_experts <= LORA_ROUTE_MAX_EXPERTS && d.top_k >= 1 && d.top_k <= LORA_ROUTE_MAX_TOP_K &&
           d.d_model >= 8 && d.d_model <= 65536 && d.d_model % 8 == 0 && d.d_mlp >= 8 && d.d_mlp <= 65536 && d.d_mlp % 8 == 0 &&
           (d.activation == 0 || d.activation == 1);
}

lora_status_t pool_ok(const lora_moe_layer_desc_t &d, const lora_pool_t *pool) {
    if (!pool) return LORA_OK;
    const lora_pool_desc_t &q = pool->desc;
    if (!pool->is_moe) return LORA_ERR_UNSUPPORTED;
    if (q.num_experts != d.n_experts || q.d_model != d.d_model || q.d_mlp != d.d_mlp) return LORA_ERR_SHAPE;
    if ((int64_t)q.n_w13_slices * q.w13_slice_width != 2 * (int64_t)d.d_mlp) return LORA_ERR_UNSUPPORTED;
    return LORA_OK;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Carve {
    size_t v13, h, v2, bytes;
};
Carve carve(const lora_moe_layer_desc_t &d, const lora_pool_t *pool, int64_t T) {
    const size_t P = (size_t)T * d.top_k, R = pool ? pool->desc.max_rank : 0;
    Carve c;
    c.v13 = 0;
    c.h = c.v13 + align256(P * 2 * R * 4);
    c.v2 = c.h + align256(P * d.d_mlp * 4);
    c.bytes = c.v2 + align256(P * R * 4) + 256;
    return c;
}

}  // namespace

extern "C" size_t lora_moe_layer_workspace_bytes(const lora_moe_layer_desc_t *desc, const lora_pool_t *pool,
                                                 int32_t max_tokens) {
    if (!desc || max_tokens < 0 || !desc_ok(*desc) || pool_ok(*desc, pool) != LORA_OK ||
        (int64_t)max_tokens * desc->top_k > LORA_MOE_LAYER_MAX_PAIRS)
        return 0;
    return carve(*desc, pool, max_tokens).bytes;
}

extern "C" lora_status_t lora_moe_layer(const lora_moe_layer_desc_t *desc, const lora_pool_t *pool, const int32_t *d_idx,
                                        const void *x, int64_t ldx, int32_t T, const int32_t *topk_ids,
                                        const float *topk_w, const void *w13, int64_t ld_w13, const void *w2,
                                        int64_t ld_w2, void *out, int64_t ld_out, int32_t *status, void *workspace,
                                        size_t ws_bytes, void *stream) {
    if (!desc || T < 0 || !desc_ok(*desc)) return LORA_ERR_INVALID_ARG;
    const lora_moe_layer_desc_t d = *desc;
    const lora_status_t st = pool_ok(d, pool);
    if (st != LORA_OK) return st;
    if (ldx < d.d_model || ldx % 8 || ld_w13 < d.d_model || ld_w13 % 8 || ld_w2 < d.d_mlp || ld_w2 % 8 ||
        ld_out < d.d_model || ld_out % 8 || ((uintptr_t)status & 3))
        return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    if (!x || !topk_ids || !w13 || !w2 || !out || !lora_aligned16(x) || !lora_aligned16(w13) || !lora_aligned16(w2) ||
        !lora_aligned16(out) || (((uintptr_t)topk_ids | (uintptr_t)topk_w | (uintptr_t)d_idx) & 3) || !pool != !d_idx)
        return LORA_ERR_INVALID_ARG;
    if ((int64_t)T * d.top_k > LORA_MOE_LAYER_MAX_PAIRS) return LORA_ERR_CAPACITY;
    if (!workspace || !lora_aligned16(workspace)) return LORA_ERR_INVALID_ARG;
    const Carve c = carve(d, pool, T);
    if (ws_bytes < c.bytes) return LORA_ERR_CAPACITY;
    int dev = 0;
    LORA_CUDA_TRY(cudaGetDevice(&dev));
    if (pool && pool->device != dev) return LORA_ERR_INVALID_ARG;
    LayerArgs p;
    memset(&p, 0, sizeof(p));
    p.T = T;
    p.K = d.top_k;
    p.P = T * d.top_k;
    p.E = d.n_experts;
    p.D = d.d_model;
    p.F = d.d_mlp;
    p.gelu = d.activation;
    p.x = (const uint16_t *)x;
    p.w13 = (const uint16_t *)w13;
    p.w2 = (const uint16_t *)w2;
    p.ldx = ldx;
    p.ld13 = ld_w13;
    p.ld2 = ld_w2;
    p.ld_out = ld_out;
    p.ids = topk_ids;
    p.idx = d_idx;
    p.topk_w = topk_w;
    p.out = (uint16_t *)out;
    p.status = status;
    char *ws = (char *)workspace;
    p.v13 = (float *)(ws + c.v13);
    p.h = (float *)(ws + c.h);
    p.v2 = (float *)(ws + c.v2);
    if (pool) {
        const lora_pool_desc_t &q = pool->desc;
        p.L = q.max_loras;
        p.R = q.max_rank;
        p.n13 = q.n_w13_slices;
        p.b_up = p.n13 == 2 ? 0 : d.d_mlp;
        p.rank = pool->d_rank;
        p.enabled = pool->d_enabled;
        p.scale = pool->d_scale;
        for (int i = 0; i < 3; ++i) {
            const int j = i == 2 ? p.n13 : i < p.n13 ? i : 0;
            p.A[i] = pool->A[j];
            p.B[i] = pool->B[j];
            p.a_ss[i] = pool->a_slot_elems[j];
            p.b_ss[i] = pool->b_slot_elems[j];
            p.a_es[i] = pool->a_experts[j] > 1 ? (long long)q.max_rank * pool->a_in[j] : 0;
            p.b_rows[i] = pool->b_experts[j] > 1 ? pool->b_out[j] : 0;
        }
    }
    cudaStream_t s = (cudaStream_t)stream;
    const auto grid = [](long long warps) { return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)); };
    if (pool) {
        shrink13_kernel<<<grid((long long)p.P * 2 * p.R), kThreads, 0, s>>>(p);
        lora_note_launch();
    }
    up_kernel<<<grid((long long)p.P * p.F), kThreads, 0, s>>>(p);
    lora_note_launch();
    if (pool) {
        shrink2_kernel<<<grid((long long)p.P * p.R), kThreads, 0, s>>>(p);
        lora_note_launch();
    }
    down_kernel<<<grid((long long)p.T * p.D), kThreads, 0, s>>>(p);
    LORA_CUDA_TRY(cudaGetLastError());
    lora_note_launch();
    return LORA_OK;
}
