// The item kernel of the attention calls (see attn.cuh for the terms): one
// pass over the keys with the running maximum and sum of the softmax,
//   S = Q K^T,   P = 2^(S * scale * log2 e - m),   O += P V,   out = O / l,
// both products on tcgen05, S, P and O in tensor memory.
//
// A row of an MMA tile is (token, query head of the group), so the heads that
// share a key/value head share its keys in one product, and a decode token
// fills group-many rows instead of one.  An item has two tiles (*slots*) that
// run over the same blocks of 128 keys: while one slot's softmax is computed
// by its four warps, the tensor cores do the other slot's products.
//
// Warp roles (384 threads, one CTA per SM, each CTA takes items in turn):
//   warps 0-3, 4-7  softmax of slot 0 / 1, one row per thread, and its epilogue
//   warp 8          TMA of K and V blocks into a ring of stages
//   warp 9          MMA issue
//   warp 10         TMA of the Q tiles
//   warp 11         TMEM allocation
// Tensor memory (512 columns): S of slot 0, 1 (128 columns each, P as bf16 in
// the first half of its S), O of slot 0, 1.
//
// Orders that no barrier of its own is needed for: a slot's QK of block j + 1
// is issued after its PV of block j, so "S is there" also says that O holds
// block j; a slot's PV of an item's first block waits for P, which the same
// warps write after they have read the item before's O.
#include <math.h>
#include <string.h>

#include <atomic>

#include "attn.cuh"
#include "tc_common.cuh"

namespace {

constexpr int kThreads = 384;
constexpr int kChunkBytes = attn::kBlock * 128;  // 128 rows of 64 bf16
constexpr int kMaxPolls = 1 << 25;               // of a wait (seconds)
constexpr float kLag = 8.f;                      // the maximum in use may lag by 2^8
constexpr float kExactBase = 1048576.f;          // up to here the rounding of the maximum is small against 1

struct KArgs {
    attn::Args a;
    CUtensorMap tq, tk, tv;
    int box_rows;  // rows of a K/V box: a whole block, or what pages divide it into
    int tpt;       // tokens of a slot's tile
    int q_bytes;   // bytes of a Q tile's copies
};

template <int NCH>
struct Shape {
    static constexpr int kDP = 64 * NCH;                      // head size in the products
    static constexpr int kStage = NCH * kChunkBytes;          // one K or V block
    static constexpr int kStages = NCH == 2 ? 5 : 10;
    static constexpr int kSmem = 1024 + 2 * kStage + kStages * kStage + 512;
};

struct Bars {
    uint64_t kv_full[10], kv_empty[10];
    uint64_t q_full[2], q_empty[2], s_full[2], o_full[2], fin;
    uint64_t p_full[2][2];  // of each slot: the first and the second 64 keys of P
    uint32_t tmem;
    int abort;
};

// Bounded wait; false when it gave up here or somewhere else in the CTA.
// The lanes of a warp may differ: callers vote before they leave a loop.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Bars *b, int32_t *status) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    for (int polls = 0; !tc::mbar_try_wait(bar, parity); ++polls) {
        if ((polls & 1023) == 0 && *(volatile int *)&b->abort) return false;
        if (polls > kMaxPolls) {
            *(volatile int *)&b->abort = 1;
            atomicExch(status, (int)LORA_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool all(bool ok) { return __all_sync(0xffffffffu, ok); }
// ... of a whole warp, with the vote.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Bars *b, int32_t *status) {
    return all(wait(bar, parity, b, status));
}

// What the roles of a CTA all derive from an item.
struct Work {
    attn::Item it;
    int kvh;
    int step;     // keys that each further token sees more
    int nt[2];    // tokens of the slots
    int nb[2];    // blocks of the slots
    int n;        // blocks of the item
};

__device__ __forceinline__ Work work_of(const KArgs &p, int w) {
    Work k;
    const int4 x = __ldg((const int4 *)(p.a.items + w / p.a.hkv)), y = __ldg((const int4 *)(p.a.items + w / p.a.hkv) + 1);
    k.it.tok0 = x.x; k.it.n_tok = x.y; k.it.prob = x.z; k.it.blk0 = x.w;
    k.it.blk1 = y.x; k.it.kv_len = y.y; k.it.lim0 = y.z; k.it.part = y.w;
    k.kvh = w % p.a.hkv;
    k.step = k.it.prob >= 0 && p.a.causal ? 1 : 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        k.nt[s] = min(max(k.it.n_tok - s * p.tpt, 0), p.tpt);
        const int lim = min(k.it.kv_len, k.it.lim0 + k.step * (s * p.tpt + k.nt[s] - 1));
        const int end = lim <= 0 ? 0 : (lim - 1) / attn::kBlock + 1;
        k.nb[s] = k.nt[s] ? max(0, min(k.it.blk1, end) - k.it.blk0) : 0;
    }
    k.n = max(k.nb[0], k.nb[1]);
    return k;
}

// The w-th piece of work of this CTA: items come longest first, so every
// other round runs backwards to even the CTAs out.
__device__ __forceinline__ int work_index(int round) {
    return round * (int)gridDim.x + ((round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two fp32 at a time.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 two(float lo, float hi) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 apart(f32x2 v) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&v;
}

// One lane of a converged warp, as the hardware picks it: the compiler then
// knows that what follows runs in one lane, and keeps the operands of the
// products in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}

// The products with the upper halves of the descriptors as immediates: only
// start addresses change from one to the next.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // see tc::desc_sw128
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}\n" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHi)
        : "memory");
}

template <int NCH>
__global__ void __launch_bounds__(kThreads, 1) item_kernel(const __grid_constant__ KArgs p) {
    using Sh = Shape<NCH>;
    constexpr int kNS = Sh::kStages;
    extern __shared__ char smem_raw[];
    char *smem = smem_raw + ((1024 - (smem_u32_of(smem_raw) & 1023)) & 1023);
    char *sq = smem;                       // two Q tiles
    char *ring = smem + 2 * Sh::kStage;    // K and V blocks
    Bars *bars = (Bars *)(ring + kNS * Sh::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *status = p.a.status;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kNS; ++i) {
            tc::mbar_init(&bars->kv_full[i], 1);
            tc::mbar_init(&bars->kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars->q_full[i], 1);
            tc::mbar_init(&bars->q_empty[i], 1);
            tc::mbar_init(&bars->s_full[i], 1);
            tc::mbar_init(&bars->p_full[i][0], 4);
            tc::mbar_init(&bars->p_full[i][1], 4);
            tc::mbar_init(&bars->o_full[i], 1);
        }
        tc::mbar_init(&bars->fin, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tc::fence_proxy_async();
    }
    if (warp == 11) {
        tc::tmem_alloc(&bars->tmem, 512);
        tc::tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        tc::prefetch_tmap(&p.tq);
        tc::prefetch_tmap(&p.tk);
        tc::prefetch_tmap(&p.tv);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *(volatile uint32_t *)&bars->tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int n_work = __ldg(p.a.counters + attn::kItems) * p.a.hkv;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 8) {
            // ---- K and V blocks, one stage each, in the order K0 V0 K1 V1 ..
            int fill = 0;
            bool ok = true;
            const int subs = attn::kBlock / p.box_rows;
            const int oob = (int)max(1LL, p.a.n_rows);  // a box from here on reads as zeros
            for (int r = 0; ok; ++r) {
                const int w = work_index(r);
                if (r * (int)gridDim.x >= n_work) break;
                if (w >= n_work) continue;
                const Work k = work_of(p, w);
                const int32_t *tab = k.it.prob >= 0 ? p.a.table + (long long)k.it.prob * p.a.ld_table
                                                    : p.a.ptable + (long long)(-1 - k.it.prob) * p.a.ld_ptable;
                for (int j = 0; j < k.n && ok; ++j) {
                    // this lane's box: its first row
                    int row = oob;
                    const int key = (k.it.blk0 + j) * attn::kBlock + lane * p.box_rows;
                    if (lane < subs && key < k.it.kv_len) {
                        long long x = p.a.page ? (long long)__ldg(tab + key / p.a.page) * p.a.page + key % p.a.page
                                               : (long long)__ldg(tab) + key;
                        const int need = min(p.box_rows, k.it.kv_len - key);
                        if (x < 0 || x + need > p.a.n_rows) atomicExch(status, (int)LORA_ERR_DEVICE_INDEX);
                        row = x < -(long long)p.box_rows || x > p.a.n_rows ? oob : (int)x;
                    }
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++fill) {
                        const int st = fill % kNS;
                        if (fill >= kNS && !warp_wait(&bars->kv_empty[st], (uint32_t)((fill / kNS - 1) & 1), bars, status)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) tc::mbar_expect_tx(&bars->kv_full[st], Sh::kStage);
                        __syncwarp();
                        if (lane < subs) {
                            char *dst = ring + st * Sh::kStage + lane * p.box_rows * 128;
#pragma unroll
                            for (int c = 0; c < NCH; ++c)
                                tc::tma_load_3d(dst + c * kChunkBytes, kv ? &p.tv : &p.tk, c * 64, k.kvh, row,
                                                &bars->kv_full[st]);
                        }
                    }
                }
            }
            // every copy has landed before the CTA ends
            for (int s = 0; s < kNS && s < fill; ++s) {
                const int last = fill - 1 - ((fill - 1 - s) % kNS);
                int polls = 0;
                while (!tc::mbar_try_wait(&bars->kv_full[s], (uint32_t)((last / kNS) & 1)) && ++polls < (1 << 16)) {}
            }
        } else if (warp == 10) {
            // ---- Q tiles
            int fill[2] = {0, 0};
            bool ok = true;
            for (int r = 0; ok; ++r) {
                const int w = work_index(r);
                if (r * (int)gridDim.x >= n_work) break;
                if (w >= n_work) continue;
                const Work k = work_of(p, w);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!k.nb[s] || !ok) continue;
                    if (fill[s] && !warp_wait(&bars->q_empty[s], (uint32_t)((fill[s] - 1) & 1), bars, status)) {
                        ok = false;
                        continue;
                    }
                    if (lane == 0) {
                        tc::mbar_expect_tx(&bars->q_full[s], p.q_bytes);
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            tc::tma_load_3d(sq + s * Sh::kStage + c * kChunkBytes, &p.tq, c * 64, k.kvh * p.a.G,
                                            k.it.tok0 + s * p.tpt, &bars->q_full[s]);
                    }
                    __syncwarp();
                    ++fill[s];
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                int polls = 0;
                while (fill[s] && !tc::mbar_try_wait(&bars->q_full[s], (uint32_t)((fill[s] - 1) & 1)) &&
                       ++polls < (1 << 16)) {}
            }
        } else if (warp == 9) {
            // ---- MMA issue
            constexpr uint32_t id_qk = tc::idesc_bf16(128, 128), id_pv = tc::idesc_bf16_bmn(128, Sh::kDP);
            int st = 0;                // the next stage of the ring and its parity
            uint32_t par = 0;
            auto next = [&]() {
                if (++st == kNS) {
                    st = 0;
                    par ^= 1u;
                }
            };
            uint32_t pq[2] = {0, 0}, pp[2] = {0, 0};
            bool ok = true;
            // lower halves of the descriptors (shared addresses end below 2^18): of K-major
            // tiles, and of V, whose 64-element chunks are kChunkBytes apart
            const uint32_t q_lo = (tc::smem_u32(sq) >> 4) | (1u << 16), k_lo = (tc::smem_u32(ring) >> 4) | (1u << 16);
            const uint32_t v_lo = (tc::smem_u32(ring) >> 4) | ((uint32_t)(kChunkBytes >> 4) << 16);
            auto qk = [&](int s, int stage) {  // by one lane
                const uint32_t qa = q_lo + s * (Sh::kStage >> 4), ka = k_lo + stage * (Sh::kStage >> 4);
#pragma unroll
                for (int i = 0; i < NCH * 4; ++i) {
                    const uint32_t off = (uint32_t)((i >> 2) * kChunkBytes + (i & 3) * 32) >> 4;
                    mma_ss(tmem + s * 128, qa + off, ka + off, id_qk, i != 0);
                }
                tc::mma_commit(&bars->s_full[s]);
            };
            auto pv = [&](int s, int h, int stage, bool first) {
                const uint32_t va = v_lo + stage * (Sh::kStage >> 4) + h * (8192 >> 4);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_ts(tmem + 256 + s * Sh::kDP, tmem + s * 128 + h * 32 + i * 8, va + i * (2048 >> 4), id_pv,
                           h || i ? true : !first);
            };
            for (int r = 0; ok; ++r) {
                const int w = work_index(r);
                if (r * (int)gridDim.x >= n_work) break;
                if (w >= n_work) continue;
                const Work k = work_of(p, w);
                if (!k.n) continue;
                // the first block's S
                ok &= wait(&bars->kv_full[st], par, bars, status);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!k.nb[s]) continue;
                    ok &= wait(&bars->q_full[s], pq[s], bars, status);
                    pq[s] ^= 1u;
                    tc::tc_fence_after();
                    if (elect_one()) {
                        qk(s, st);
                        if (k.nb[s] == 1) tc::mma_commit(&bars->q_empty[s]);
                    }
                }
                if (elect_one()) tc::mma_commit(&bars->kv_empty[st]);
                next();
                const int full = (k.it.kv_len >> 7) - k.it.blk0;  // blocks whose keys all count
                for (int j = 0; j < k.n; ++j) {
                    const bool more = j + 1 < k.n;
                    const int sv = st;
                    ok &= wait(&bars->kv_full[st], par, bars, status);
                    next();
                    const int sk = st;
                    if (more) {
                        ok &= wait(&bars->kv_full[st], par, bars, status);
                        next();
                    }
                    // values of a block's keys past the end count for nothing, whatever their rows hold
                    if (j >= full) {
                        char *v = ring + sv * Sh::kStage;
                        for (int i = (k.it.kv_len & 127) * 8 + lane; i < attn::kBlock * 8; i += 32)
#pragma unroll
                            for (int c = 0; c < NCH; ++c) *(uint4 *)(v + c * kChunkBytes + i * 16) = make_uint4(0, 0, 0, 0);
                        tc::fence_proxy_async();
                        __syncwarp();
                    }
                    if (!(ok = all(ok))) break;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (j >= k.nb[s]) continue;
                        ok &= wait(&bars->p_full[s][0], pp[s], bars, status);
                        tc::tc_fence_after();
                        if (elect_one()) pv(s, 0, sv, j == 0);
                        ok &= wait(&bars->p_full[s][1], pp[s], bars, status);
                        pp[s] ^= 1u;
                        tc::tc_fence_after();
                        if (elect_one()) {
                            pv(s, 1, sv, false);
                            if (j + 1 < k.nb[s]) {
                                qk(s, sk);
                                if (j + 2 == k.nb[s]) tc::mma_commit(&bars->q_empty[s]);
                            } else {
                                tc::mma_commit(&bars->o_full[s]);
                            }
                            if (s == 1 || j >= k.nb[1]) {  // the last of the slots: the stages are free
                                tc::mma_commit(&bars->kv_empty[sv]);
                                if (more) tc::mma_commit(&bars->kv_empty[sk]);
                            }
                        }
                    }
                    __syncwarp();
                }
                ok = all(ok);
            }
            // all products are done before tensor memory is given back
            if (lane == 0) tc::mma_commit(&bars->fin);
            __syncwarp();
            int polls = 0;
            while (!tc::mbar_try_wait(&bars->fin, 0) && ++polls < (1 << 20)) {}
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ---- softmax and epilogue of one slot, a row per thread
        const int s = warp >> 2, q = warp & 3, row = q * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t ts = tl + s * 128, to = tl + 256 + s * Sh::kDP;
        const int e = row / p.a.G, g = row - e * p.a.G;
        int ns = 0, no = 0;
        bool ok = true;
        for (int r = 0; ok; ++r) {
            const int w = work_index(r);
            if (r * (int)gridDim.x >= n_work) break;
            if (w >= n_work) continue;
            const Work k = work_of(p, w);
            const int nt = k.nt[s], nb = k.nb[s];
            if (!nt) continue;
            const bool live = e < nt, warp_live = __any_sync(0xffffffffu, live);
            // keys that the row sees; a row that is not there masks nothing
            const int lim = live ? min(k.it.kv_len, k.it.lim0 + k.step * (s * p.tpt + e)) : 0x7fffffff;
            const int min_lim = __reduce_min_sync(0xffffffffu, lim);
            float m = -INFINITY, l = 0.f, base = 0.f;
            bool huge = false;
            for (int j = 0; j < nb; ++j) {
                if (!(ok = warp_wait(&bars->s_full[s], (uint32_t)(ns & 1), bars, status))) break;
                ++ns;
                if (warp_live) {
                    tc::tc_fence_after();
                    uint32_t x[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::tmem_ld32(ts + c * 32, x[c]);
                    tc::tmem_wait_ld();
                    const int key0 = (k.it.blk0 + j) * attn::kBlock;
                    if (key0 + attn::kBlock > min_lim) {
                        const int rel = lim - key0;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i >= rel) x[c][i] = 0xff800000u;
                    }
                    float mx[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        mx[c] = max3(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]), __uint_as_float(x[c][2]));
#pragma unroll
                        for (int i = 3; i < 31; i += 2)
                            mx[c] = max3(mx[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
                        mx[c] = fmaxf(mx[c], __uint_as_float(x[c][31]));
                    }
                    const float bm = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                    // the maximum in use stays while no row is more than kLag above it
                    if (__any_sync(0xffffffffu, live && !((bm - m) * p.a.scale_log2 <= kLag))) {
                        const float mn = fmaxf(m, bm);
                        const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * p.a.scale_log2);
                        m = mn;
                        l *= f;
                        base = m == -INFINITY ? 0.f : m * p.a.scale_log2;
                        huge = __any_sync(0xffffffffu, live && !(fabsf(base) <= kExactBase));
#pragma unroll 1
                        for (int c = 0; j && c < Sh::kDP / 32; ++c) {  // the output so far, with the weights
                            uint32_t o[32], o0[16], o1[16];
                            tc::tmem_ld32(to + c * 32, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                o0[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                o1[i] = __float_as_uint(__uint_as_float(o[16 + i]) * f);
                            }
                            tc::tmem_st16(to + c * 32, o0);
                            tc::tmem_st16(to + c * 32 + 16, o1);
                        }
                    }
                    // 2^(x * scale - base): whatever base was rounded to divides out, unless
                    // it is so large that its rounding is
                    float sc = p.a.scale_log2, sb = -base;
                    if (huge) {
                        const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[c][i] = __float_as_uint((__uint_as_float(x[c][i]) - mm) * sc);
                        sc = 1.f;
                        sb = 0.f;
                    }
                    const f32x2 sc2 = two(sc, sc), sb2 = two(sb, sb);
                    f32x2 sum[2] = {two(0.f, 0.f), two(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 v = apart(fma2(two(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])),
                                                  sc2, sb2));
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            sum[i & 1] = add2(sum[i & 1], two(v.x, v.y));
                            pk[i] = pack2(v.x, v.y);
                        }
                        tc::tmem_st16(ts + c * 16, pk);
                        if (c == 1) {  // the first half of P (and the rescaled output) is there
                            tc::tmem_wait_st();
                            tc::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(&bars->p_full[s][0]);
                        }
                    }
                    const float2 sm = apart(add2(sum[0], sum[1]));
                    l += sm.x + sm.y;
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    if (!warp_live) tc::mbar_arrive(&bars->p_full[s][0]);
                    tc::mbar_arrive(&bars->p_full[s][1]);
                }
            }
            if (!ok) break;
            if (nb) {
                if (!(ok = warp_wait(&bars->o_full[s], (uint32_t)(no & 1), bars, status))) break;
                ++no;
                tc::tc_fence_after();
            }
            if (warp_live) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int t = k.it.tok0 + s * p.tpt + e, h = k.kvh * p.a.G + g;
                const long long prow = (long long)(k.it.part + s * p.tpt + e) * p.a.hq + h;
                uint16_t *out = p.a.out + (long long)t * p.a.ldo + (long long)h * p.a.D;
                float *po = p.a.part_o + prow * p.a.D;
#pragma unroll 1
                for (int c = 0; c < Sh::kDP / 32; ++c) {
                    uint32_t o[32];
                    if (nb) {
                        tc::tmem_ld32(to + c * 32, o);
                        tc::tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = nb && l != 0.f ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int col = c * 32 + i * 8;
                        if (col >= p.a.D) break;
                        const float *f = (const float *)&o[i * 8];
                        if (k.it.part < 0) {
                            *(uint4 *)(out + col) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                                                               pack2(f[6], f[7]));
                        } else {
                            *(float4 *)(po + col) = make_float4(f[0], f[1], f[2], f[3]);
                            *(float4 *)(po + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
                        }
                    }
                }
                if (live && k.it.part >= 0)
                    p.a.part_lse[prow] = l == 0.f ? -INFINITY : m * p.a.scale_log2 + log2f(l);
                tc::tc_fence_before();
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 11) tc::tmem_dealloc(tmem, 512);
}

std::atomic<int> g_attn_sms[64];  // SM count per device, looked up once

template <int NCH>
cudaError_t launch(KArgs &p, int grid, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(item_kernel<NCH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NCH>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Shape<NCH>::kSmem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, item_kernel<NCH>, p);
}

}  // namespace

lora_status_t lora_attn_launch(const attn::Args &a, int max_items, cudaStream_t s) {
    int dev = 0;
    LORA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return LORA_ERR_INVALID_ARG;
    int n_sms = g_attn_sms[dev].load(std::memory_order_relaxed);
    if (!n_sms) {
        LORA_CUDA_TRY(cudaDeviceGetAttribute(&n_sms, cudaDevAttrMultiProcessorCount, dev));
        n_sms = n_sms > 0 ? n_sms : 1;
        g_attn_sms[dev].store(n_sms, std::memory_order_relaxed);
    }
    KArgs p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    p.tpt = attn::tile_tokens(a.G);
    p.box_rows = attn::kBlock;
    if (a.page)
        while (a.page % p.box_rows) p.box_rows >>= 1;
    const int nch = a.D > 64 ? 2 : 1;
    p.q_bytes = nch * 128 * a.G * p.tpt;
    const long long rows = a.n_rows > 0 ? a.n_rows : 1;
    if (!lora_make_tmap_heads(&p.tq, a.q, a.D, a.hq, a.T, a.ldq, a.G, p.tpt) ||
        !lora_make_tmap_heads(&p.tk, a.k, a.D, a.hkv, rows, a.ldk, 1, p.box_rows) ||
        !lora_make_tmap_heads(&p.tv, a.v, a.D, a.hkv, rows, a.ldv, 1, p.box_rows))
        return LORA_ERR_UNSUPPORTED;
    const long long n = (long long)max_items * a.hkv;
    const int grid = (int)(n < n_sms ? n : n_sms);
    LORA_CUDA_TRY(nch == 2 ? launch<2>(p, grid, s) : launch<1>(p, grid, s));
    lora_note_launch();
    return LORA_OK;
}
