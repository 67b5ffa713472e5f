// Norm and rotation of query and key heads in one pass over the packed QKV
// rows, keys and values to their cache rows (lora_qk_norm_rope):
//   n = x * rsqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// HBM-bound: every row is read once and written once (12 KB each way per
// token at 32 + 2 x 8 heads of 128, and 512 bytes of the table).  A head is
// held by the lanes of a group (a power of two of them), each with the two
// pieces whose elements rotate with each other, so the rotation needs no
// exchange between lanes and the norm one butterfly sum.  Pieces are 16 bytes
// when the head size and its rotated part are multiples of 16 elements, else 8.
//
// Few tokens: a warp does kU heads per group of one token (256 tokens of that
// size: 3.1 us in a graph; one token: 2.2 us, of which a launch is most; calls
// one by one take 6.6 to 7.7 us, the host's time).  Many tokens: resident CTAs
// pass their tokens' rows through shared memory by bulk copies, which keeps
// three rows a CTA and six CTAs an SM in flight and writes whole rows (7995
// tokens: 35 us, 5.7 TB/s, against 47 us with a CTA per unit and 39 us with four
// rows and four CTAs).
#include <math.h>
#include <string.h>

#include <atomic>

#include "mma_common.cuh"
#include "tc_common.cuh"

namespace {

constexpr int kSms = 152;
constexpr int kThreads = 128;
constexpr int kU = 2;              // heads that a group has in hand
constexpr int kRowThreads = 128;
constexpr int kRowStages = 3;
constexpr int kRowSmem = 224 * 1024;  // of an SM, for row buffers
constexpr int kRowCtas = 8;           // per SM at most
constexpr int kRowLand = 1 << 12;     // polls (about 1.5 us each) for a copy in flight to land

__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(tc::smem_u32(src)),
                 "r"(bytes)
                 : "memory");
}

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
    int row_bytes;  // of a row buffer
    int spin_limit;
};

// A lane's piece of V elements (4 or 8) as it lies in memory.
template <int V>
struct Piece {
    uint32_t w[V / 2];
};
template <int V>
__device__ __forceinline__ Piece<V> load_piece(const uint16_t *p) {
    Piece<V> r;
    if (V == 4) {
        const uint2 u = *(const uint2 *)p;
        r.w[0] = u.x; r.w[1] = u.y;
    } else {
        const uint4 u = *(const uint4 *)p;
        r.w[0] = u.x; r.w[1] = u.y; r.w[V / 2 - 2] = u.z; r.w[V / 2 - 1] = u.w;
    }
    return r;
}
template <int V>
__device__ __forceinline__ void store_piece(uint16_t *p, const Piece<V> &r) {
    if (V == 4) *(uint2 *)p = make_uint2(r.w[0], r.w[1]);
    else *(uint4 *)p = make_uint4(r.w[0], r.w[1], r.w[V / 2 - 2], r.w[V / 2 - 1]);
}
template <int V>
__device__ __forceinline__ void unpack(const Piece<V> &r, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        f[2 * i] = bf16lo(r.w[i]);
        f[2 * i + 1] = bf16hi(r.w[i]);
    }
}
template <int V>
__device__ __forceinline__ Piece<V> pack(const float (&f)[V]) {
    Piece<V> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        r.w[i] = *(const uint32_t *)&x;
    }
    return r;
}

// One head: the norm with weights wa, wb, then the rotation of the lane's
// pieces a and b.  All lanes of a warp call it (lw lanes to a head).
template <int V, bool kPairs>
__device__ __forceinline__ void norm_rotate(float (&a)[V], float (&b)[V], const Piece<V> &pa, const Piece<V> &pb, int lw,
                                            float inv_d, float eps, bool rotated, const float (&co)[V],
                                            const float (&si)[V]) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss += a[i] * a[i] + b[i] * b[i];
    for (int o = lw >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * inv_d + eps);
    float wa[V], wb[V];
    unpack<V>(pa, wa);
    unpack<V>(pb, wb);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        a[i] = a[i] * r * wa[i];
        b[i] = b[i] * r * wb[i];
    }
    if (!rotated) return;  // past the rotated part: no partner, not even times zero
    if (kPairs) {          // pairs side by side: the first half of them in piece a
        float e[2 * V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            e[i] = a[i];
            e[V + i] = b[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = e[2 * i] * co[i] - e[2 * i + 1] * si[i];
            e[2 * i + 1] = e[2 * i + 1] * co[i] + e[2 * i] * si[i];
            e[2 * i] = x;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = e[i];
            b[i] = e[V + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = a[i] * co[i] - b[i] * si[i];
            b[i] = b[i] * co[i] + a[i] * si[i];
            a[i] = x;
        }
    }
}

// The lane's cosines and sines of a position.
template <int V>
__device__ __forceinline__ void angles(const RopeArgs &p, int pos, int l, bool rotated, float (&co)[V], float (&si)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) co[i] = si[i] = 0.f;
    if (!rotated) return;
    const float *c = p.cs + (long long)pos * p.rot + V * l;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 x = __ldg((const float4 *)(c + i)), y = __ldg((const float4 *)(c + p.rot / 2 + i));
        co[i] = x.x; co[i + 1] = x.y; co[i + 2] = x.z; co[i + 3] = x.w;
        si[i] = y.x; si[i + 1] = y.y; si[i + 2] = y.z; si[i + 3] = y.w;
    }
}

// A token's places: false when its position or slot is outside the tables.
__device__ __forceinline__ bool in_tables(const RopeArgs &p, int pos, long long slot) {
    return !(p.rot && (pos < 0 || pos >= p.max_pos)) && slot >= -1 && slot < p.n_rows;
}

template <int V, bool kPairs>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lw = 1 << p.lw_log, l = lane & (lw - 1), group = lane >> p.lw_log;
    const int groups = 32 >> p.lw_log;
    const bool live = l * 2 * V < p.D, rotated = l * 2 * V < p.rot;
    // the lane's two pieces: elements that rotate with each other
    const int ea = !kPairs && rotated ? V * l : 2 * V * l;
    const int eb = !kPairs && rotated ? V * l + p.rot / 2 : 2 * V * l + V;
    Piece<V> wqa, wqb, wka, wkb;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) wqa.w[i] = wqb.w[i] = wka.w[i] = wkb.w[i] = 0x3f803f80u;
    if (live && p.qw) { wqa = load_piece<V>(p.qw + ea); wqb = load_piece<V>(p.qw + eb); }
    if (live && p.kw) { wka = load_piece<V>(p.kw + ea); wkb = load_piece<V>(p.kw + eb); }
    const int unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = unit / p.chunks, head0 = ((unit - t * p.chunks) * kU << (5 - p.lw_log)) + group;
    if (t >= p.T) return;
    const int pos = p.rot ? __ldg(p.positions + t) : 0;
    const long long slot = p.slots ? __ldg(p.slots + t) : t;
    const uint16_t *row = p.qkv + (long long)t * p.ld_qkv;
    Piece<V> xa[kU], xb[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int h = head0 + u * groups;
        if (live && h < p.heads) {
            xa[u] = load_piece<V>(row + h * p.D + ea);
            xb[u] = load_piece<V>(row + h * p.D + eb);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) xa[u].w[i] = xb[u].w[i] = 0u;
        }
    }
    if (!in_tables(p, pos, slot)) {
        if (lane == 0 && p.status) atomicExch(p.status, (int)LORA_ERR_DEVICE_INDEX);
        return;
    }
    float co[V], si[V];
    angles<V>(p, pos, l, rotated, co, si);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int h = head0 + u * groups;
        float a[V], b[V];
        unpack<V>(xa[u], a);
        unpack<V>(xb[u], b);
        const bool is_q = h < p.hq;
        norm_rotate<V, kPairs>(a, b, is_q ? wqa : wka, is_q ? wqb : wkb, lw, p.inv_d, p.eps, rotated, co, si);
        if (!live || h >= p.heads) continue;
        if (h >= p.hq + p.hkv) {  // a value head: stored as it is
            if (slot >= 0) {
                uint16_t *o = p.v + slot * p.ld_v + (long long)(h - p.hq - p.hkv) * p.D;
                store_piece<V>(o + ea, xa[u]);
                store_piece<V>(o + eb, xb[u]);
            }
            continue;
        }
        if (!is_q && slot < 0) continue;
        uint16_t *o = is_q ? p.q + (long long)t * p.ld_q + (long long)h * p.D
                           : p.k + slot * p.ld_k + (long long)(h - p.hq) * p.D;
        store_piece<V>(o + ea, pack<V>(a));
        store_piece<V>(o + eb, pack<V>(b));
    }
}

// The same for many tokens: a CTA's tokens pass through a ring of row buffers
// in shared memory, brought and taken away by bulk copies while other rows
// are worked on in place.
template <int V, bool kPairs>
__global__ void __launch_bounds__(kRowThreads) rope_rows_kernel(const __grid_constant__ RopeArgs p) {
    extern __shared__ __align__(128) char smem[];
    __shared__ uint64_t full[kRowStages];
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRowStages; ++i) tc::mbar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tc::fence_proxy_async();
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lw = 1 << p.lw_log, l = lane & (lw - 1);
    const int group = threadIdx.x >> p.lw_log, groups = kRowThreads >> p.lw_log;
    const bool live = l * 2 * V < p.D, rotated = l * 2 * V < p.rot;
    const int ea = !kPairs && rotated ? V * l : 2 * V * l;
    const int eb = !kPairs && rotated ? V * l + p.rot / 2 : 2 * V * l + V;
    const uint32_t qb = (uint32_t)(p.hq * p.D * 2), kb = (uint32_t)(p.hkv * p.D * 2);
    const uint32_t bytes = (uint32_t)(p.heads * p.D * 2);
    Piece<V> wqa, wqb, wka, wkb;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) wqa.w[i] = wqb.w[i] = wka.w[i] = wkb.w[i] = 0x3f803f80u;
    if (live && p.qw) { wqa = load_piece<V>(p.qw + ea); wqb = load_piece<V>(p.qw + eb); }
    if (live && p.kw) { wka = load_piece<V>(p.kw + ea); wkb = load_piece<V>(p.kw + eb); }
    const int step = gridDim.x;
    auto fetch = [&](int t, int st) {
        tc::mbar_expect_tx(&full[st], bytes);
        bgmv::bulk_g2s(smem + st * p.row_bytes, p.qkv + (long long)t * p.ld_qkv, bytes, &full[st]);
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < kRowStages - 1; ++i)
            if (blockIdx.x + i * step < p.T) fetch(blockIdx.x + i * step, i);
    // a token's position, slot and angles are fetched while the one before is worked on
    int pos = 0, npos = 0;
    long long slot = 0, nslot = 0;
    float nco[V], nsi[V];
    auto places = [&](int t) {
        npos = p.rot && t < p.T ? __ldg(p.positions + t) : 0;
        nslot = t < p.T ? (p.slots ? (long long)__ldg(p.slots + t) : (long long)t) : 0;
    };
    int t = blockIdx.x;
    places(t);
    angles<V>(p, in_tables(p, npos, nslot) ? npos : 0, l, rotated, nco, nsi);
    int i = 0;
    bool gave_up = false;
    for (; t < p.T; ++i, t += step) {
        const int st = i % kRowStages;
        pos = npos;
        slot = nslot;
        float co[V], si[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            co[j] = nco[j];
            si[j] = nsi[j];
        }
        places(t + step);
        const bool good = in_tables(p, pos, slot);
        if (!good && threadIdx.x == 0 && p.status) atomicExch(p.status, (int)LORA_ERR_DEVICE_INDEX);
        const uint32_t parity = (uint32_t)((i / kRowStages) & 1);
        const bool ok = p.spin_limit < 0 ? tc::mbar_test_wait(&full[st], parity)
                                         : tc::mbar_wait(&full[st], parity, p.spin_limit);
        gave_up = __syncthreads_or(!ok);
        if (gave_up) {
            if (threadIdx.x == 0 && p.status) atomicExch(p.status, (int)LORA_ERR_TIMEOUT);
            break;
        }
        uint16_t *row = (uint16_t *)(smem + st * p.row_bytes);
        for (int h = group; h - group < p.hq + p.hkv; h += groups) {
            const bool mine = live && h < p.hq + p.hkv;
            Piece<V> xa, xb;
#pragma unroll
            for (int j = 0; j < V / 2; ++j) xa.w[j] = xb.w[j] = 0u;
            if (mine) {
                xa = load_piece<V>(row + h * p.D + ea);
                xb = load_piece<V>(row + h * p.D + eb);
            }
            float a[V], b[V];
            unpack<V>(xa, a);
            unpack<V>(xb, b);
            const bool is_q = h < p.hq;
            norm_rotate<V, kPairs>(a, b, is_q ? wqa : wka, is_q ? wqb : wkb, lw, p.inv_d, p.eps, rotated, co, si);
            if (mine) {
                store_piece<V>(row + h * p.D + ea, pack<V>(a));
                store_piece<V>(row + h * p.D + eb, pack<V>(b));
            }
        }
        angles<V>(p, in_tables(p, npos, nslot) ? npos : 0, l, rotated, nco, nsi);
        tc::fence_proxy_async();
        __syncthreads();
        if (threadIdx.x == 0) {
            if (good) {
                bulk_s2g(p.q + (long long)t * p.ld_q, row, qb);
                if (slot >= 0) {
                    bulk_s2g(p.k + slot * p.ld_k, (char *)row + qb, kb);
                    if (p.v) bulk_s2g(p.v + slot * p.ld_v, (char *)row + qb + kb, kb);
                }
            }
            tc::bulk_commit();
            // the stage of the token before is free when its rows have been read
            const int ahead = t + (kRowStages - 1) * step;
            if (ahead < p.T) {
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                fetch(ahead, (i + kRowStages - 1) % kRowStages);
            }
        }
    }
    if (threadIdx.x == 0) {
        // after a wait that gave up, this token's row and the one fetched ahead of it
        // land before the CTA ends, each waited for in its own phase
        for (int j = i; gave_up && j < i + kRowStages - 1 && t < p.T; ++j, t += step)
            tc::mbar_wait(&full[j % kRowStages], (uint32_t)((j / kRowStages) & 1), kRowLand);
        tc::bulk_wait0();
    }
}

template <int V, bool kPairs>
cudaError_t rope_launch(RopeArgs &p, int dev, cudaStream_t s) {
    p.lw_log = 0;
    while ((2 * V << p.lw_log) < p.D) ++p.lw_log;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.stream = s;
    p.row_bytes = (p.heads * p.D * 2 + 127) / 128 * 128;
    // many tokens whose rows fit the ring: two or more to each of its CTAs
    const int per_sm = kRowSmem / (kRowStages * p.row_bytes + 256);
    const int ctas = kSms * (per_sm < kRowCtas ? per_sm : kRowCtas);
    if (per_sm >= 2 && p.T >= 2 * ctas) {
        static std::atomic<bool> ready[64];  // the shared-memory limit is set once per device
        if (!ready[dev].load(std::memory_order_acquire)) {
            const cudaError_t e = cudaFuncSetAttribute(rope_rows_kernel<V, kPairs>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem / 2);
            if (e != cudaSuccess) return e;
            ready[dev].store(true, std::memory_order_release);
        }
        cfg.gridDim = dim3((unsigned)ctas, 1, 1);
        cfg.blockDim = dim3(kRowThreads, 1, 1);
        cfg.dynamicSmemBytes = (size_t)kRowStages * p.row_bytes;
        return cudaLaunchKernelEx(&cfg, rope_rows_kernel<V, kPairs>, p);
    }
    const int per = kU << (5 - p.lw_log);
    p.chunks = (p.heads + per - 1) / per;
    const long long units = (long long)p.T * p.chunks;
    cfg.gridDim = dim3((unsigned)((units + kThreads / 32 - 1) / (kThreads / 32)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    return cudaLaunchKernelEx(&cfg, rope_kernel<V, kPairs>, p);
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
    p.spin_limit = lora_spin_limit();
    if ((long long)T * p.heads > 0x7fffffffLL) return LORA_ERR_INVALID_ARG;
    int dev = 0;
    LORA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return LORA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const bool wide = d.head_dim % 16 == 0 && d.rot_dim % 16 == 0;
    LORA_CUDA_TRY(wide ? (d.interleaved ? rope_launch<8, true>(p, dev, s) : rope_launch<8, false>(p, dev, s))
                       : (d.interleaved ? rope_launch<4, true>(p, dev, s) : rope_launch<4, false>(p, dev, s)));
    lora_note_launch();
    return LORA_OK;
}
