// The item kernel of the attention calls (see attn.cuh): one warp per row of
// an item, keys one by one with the running maximum and sum of the softmax.
#include <math.h>
#include <string.h>

#include "attn.cuh"

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ long long key_row(const attn::Args &p, int prob, int j) {
    const int32_t *t = prob >= 0 ? p.table + (long long)prob * p.ld_table : p.ptable + (long long)(-1 - prob) * p.ld_ptable;
    const long long r = p.page ? (long long)__ldg(t + j / p.page) * p.page + j % p.page : (long long)__ldg(t) + j;
    if (r < 0 || r >= p.n_rows) {
        atomicExch(p.status, (int)LORA_ERR_DEVICE_INDEX);
        return -1;
    }
    return r;
}

__global__ void __launch_bounds__(kThreads) item_kernel(const __grid_constant__ attn::Args p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_items = p.counters[attn::kItems] * p.hkv;
    for (int w = blockIdx.x; w < n_items; w += gridDim.x) {
        const attn::Item it = p.items[w / p.hkv];
        const int kvh = w % p.hkv;
        for (int r = warp; r < it.n_tok * p.G; r += kThreads / 32) {
            const int e = r / p.G, t = it.tok0 + e, h = kvh * p.G + r % p.G;
            const int lim = min(it.kv_len, it.lim0 + (it.prob >= 0 && p.causal ? e : 0));
            const bool live = 4 * lane < p.D;
            float q[4] = {0.f, 0.f, 0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
            if (live) {
                const uint2 u = *(const uint2 *)(p.q + (long long)t * p.ldq + (long long)h * p.D + 4 * lane);
                q[0] = bf16lo(u.x); q[1] = bf16hi(u.x); q[2] = bf16lo(u.y); q[3] = bf16hi(u.y);
            }
            float m = -INFINITY, l = 0.f;
            for (int j = it.blk0 * attn::kBlock; j < min(lim, it.blk1 * attn::kBlock); ++j) {
                const long long row = key_row(p, it.prob, j);
                uint2 ku = make_uint2(0u, 0u), vu = ku;
                if (live && row >= 0) {
                    ku = *(const uint2 *)(p.k + row * p.ldk + (long long)kvh * p.D + 4 * lane);
                    vu = *(const uint2 *)(p.v + row * p.ldv + (long long)kvh * p.D + 4 * lane);
                }
                float s = q[0] * bf16lo(ku.x) + q[1] * bf16hi(ku.x) + q[2] * bf16lo(ku.y) + q[3] * bf16hi(ku.y);
#pragma unroll
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                s *= p.scale_log2;
                const float m2 = fmaxf(m, s), base = m2 == -INFINITY ? 0.f : m2;
                const float c = exp2f(m - base), w2 = exp2f(s - base);
                l = l * c + w2;
                acc[0] = acc[0] * c + w2 * bf16lo(vu.x);
                acc[1] = acc[1] * c + w2 * bf16hi(vu.x);
                acc[2] = acc[2] * c + w2 * bf16lo(vu.y);
                acc[3] = acc[3] * c + w2 * bf16hi(vu.y);
                m = m2;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] *= inv;
            if (it.part >= 0) {
                const long long row = (long long)(it.part + e) * p.hq + h;
                if (live) *(float4 *)(p.part_o + row * p.D + 4 * lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (lane == 0) p.part_lse[row] = l == 0.f ? -INFINITY : m + log2f(l);
            } else if (live) {
                const __nv_bfloat162 x = __floats2bfloat162_rn(acc[0], acc[1]), y = __floats2bfloat162_rn(acc[2], acc[3]);
                *(uint2 *)(p.out + (long long)t * p.ldo + (long long)h * p.D + 4 * lane) =
                    make_uint2(*(const uint32_t *)&x, *(const uint32_t *)&y);
            }
        }
    }
}

}  // namespace

lora_status_t lora_attn_launch(const attn::Args &a, int max_items, cudaStream_t s) {
    const long long n = (long long)max_items * a.hkv;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(n < 8 * 152 ? n : 8 * 152), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    LORA_CUDA_TRY(cudaLaunchKernelEx(&cfg, item_kernel, a));
    lora_note_launch();
    return LORA_OK;
}
