// The item kernel of the attention calls (see attn.cuh for the terms): one
// pass over the keys with the running maximum and sum of the softmax,
//   S = Q K^T,   P = 2^(S * scale * log2 e - m),   O += P V,   out = O / l,
// both products on tcgen05, S, P and O in tensor memory.
//
// A row of an MMA tile is (token, query head of the group), so the heads that
// share a key/value head share its keys in one product, and a decode token
// fills group-many rows instead of one.  A CTA works on two tiles (*slots*) at
// a time: while one slot's softmax is computed by its four warps, the tensor
// cores do the other slot's products.  The slots are the two tiles of one
// item, over the same stream of K/V blocks, or two one-tile items with a
// stream each.
//
// Warp roles (384 threads, one CTA per SM, each CTA takes units in turn):
//   warps 0-3, 4-7  softmax of slot 0 / 1, one row per thread, and its epilogue
//   warps 8, 10     TMA of K and V blocks into a ring of stages, half a block each;
//                   8 takes the units, 10 loads the Q tiles and allocates TMEM
//   warps 9, 11     MMA issue of slot 0 / 1
// Tensor memory (512 columns): S of slot 0, 1 (128 columns each, P as bf16 in
// the first half of its S), O of slot 0, 1.
//
// What bounds it: the products of two full slots take 2048 cycles a block, the
// two softmaxes (512 cycles of exponentials each and about 300 other
// instructions) run under them, and a slot's own chain (S there, softmax 1100
// to 1400 cycles, 250 to the MMA warp, 1024 of products) just fits: one prompt
// of 7995 tokens, 32 heads of 128 over 8: 298 us in a burst of twelve calls,
// 1.76 PFLOP/s, tensor pipe 76% active; 331 us, 1.58 PFLOP/s, in calls that go
// on, whose clocks the power limit lowers.  One-tile items of decode batches are
// bound by HBM (64 single tokens over up to 4000 keys: 89 us, 6.0 TB/s).  Short
// units are bound by chains of dependent steps in single warps: one of two
// one-key items takes 8600 cycles, of which reading the unit and its table and
// issuing four stages' copies is one chain of 7000, a softmax, its wait for O
// and the stores another.
//
// Roundings: scores, statistics, accumulators and partial results are fp32; P is
// rounded to bf16 once, because the products take both operands in one 16-bit
// type and V is bf16.  The sums l are of the weights before that, whose
// roundings average out: against 64 bits the outputs are 1.7e-3 to 2.3e-3 off,
// where rounding the exact ones to bf16 gives 1.5e-3 to 1.7e-3.
//
// Orders that no barrier of its own is needed for: a slot's QK of block j + 1
// is issued after its PV of block j, so "S is there" also says that O holds
// block j; a slot's PV of a unit's first block waits for P, which the same
// warps write after they have read the unit before's O.
#include <math.h>
#include <string.h>

#include <atomic>

#include "attn.cuh"
#include "tc_common.cuh"

namespace {

constexpr int kThreads = 384;
constexpr int kChunkBytes = attn::kBlock * 128;  // 128 rows of 64 bf16
constexpr int kLand = 1 << 13;                   // polls (about 1.5 us each) for what is in flight to end
constexpr float kLag = 8.f;                      // the maximum in use may lag by 2^8
constexpr float kExactBase = 1048576.f;          // up to here the rounding of the maximum is small against 1

struct KArgs {
    attn::Args a;
    CUtensorMap tq, tk, tv;
    int page_shift;  // log2 of the boxes of a page, -1 if they are no power of two
    int box_rows;  // rows of a K/V box: a whole block, or what pages divide it into
    int tpt;       // tokens of a slot's tile
    int q_bytes;   // bytes of a Q tile's copies
    int out32;     // output rows of a head begin on 32-byte boundaries, in pieces of 32
    int spin_limit;
};

// A slot's part of a unit.
struct Slot {
    int tok0, nt;       // its tokens
    int prob, kv_len;   // whose keys, and how many
    int blk0, nb;       // its blocks
    int lim0, step;     // keys that its first token sees, and that each further one sees more
    int part;           // token row of its partial result, or -1
};
struct Work {
    Slot s[2];
    int shared;  // both slots run over slot 0's stream (of n blocks)
    int n;       // blocks of the longer slot; -1: no more work
    int kvh;
};
constexpr int kWorks = 4;

struct Bars {
    uint64_t kv_full[10], kv_empty[10];
    uint64_t q_full[2], q_empty[2], s_full[2], o_full[2], fin[2];
    uint64_t turn[2];       // a slot's turn to issue, when the slots share a stream
    uint64_t p_full[2][2];  // of each slot: the first and the second 64 keys of P
    uint64_t work_full[kWorks], work_empty[kWorks];
    Work work[kWorks];
    uint32_t tmem;
    int abort, spin_limit;  // next to each other: a wait that lasts reads both
};

template <int NCH>
struct Shape {
    static constexpr int kDP = 64 * NCH;                      // head size in the products
    static constexpr int kStage = NCH * kChunkBytes;          // one K or V block
    static constexpr int kStages = NCH == 2 ? 5 : 10;
    static constexpr int kSmem = 1024 + 2 * kStage + kStages * kStage + 1024;
    static_assert(sizeof(Bars) <= 1024, "barriers and work");
};

// Bounded wait; false when it gave up here or somewhere else in the CTA.
// The lanes of a warp may differ: callers vote before they leave a loop.
// abort points at a Bars' abort and spin_limit.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort, int32_t *status) {
#pragma unroll 1
    for (int polls = 0; !tc::mbar_try_wait(bar, parity); ++polls) {
        if ((polls & 1023) == 0 && *abort) return false;
        if (polls > abort[1]) {
            *abort = 1;
            atomicExch(status, (int)LORA_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
// The warps with few registers call it; the softmax warps, whose registers
// leave a call no room, have it inline.
__device__ __noinline__ bool wait_call(uint32_t bar, uint32_t parity, volatile int *abort, int32_t *status) {
    return wait_on(bar, parity, abort, status);
}
template <bool kCall>
__device__ __forceinline__ bool wait_as(uint64_t *bar, uint32_t parity, Bars *b, int32_t *status) {
    const uint32_t at = tc::smem_u32(bar);
    if (tc::mbar_try_wait(at, parity)) return true;
    return kCall ? wait_call(at, parity, &b->abort, status) : wait_on(at, parity, &b->abort, status);
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Bars *b, int32_t *status) {
    return wait_as<true>(bar, parity, b, status);
}
template <bool kCall>
struct Call {
    static constexpr bool value = kCall;
};
__device__ __forceinline__ bool all(bool ok) { return __all_sync(0xffffffffu, ok); }
// ... of a whole warp, with the vote.
template <bool kCall>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Bars *b, int32_t *status) {
    return all(wait_as<kCall>(bar, parity, b, status));
}

__device__ __forceinline__ Slot slot_of(const KArgs &p, const int4 x, const int4 y) {
    Slot k;
    k.tok0 = x.x; k.nt = x.y; k.prob = x.z; k.blk0 = x.w;
    k.nb = y.x - x.w; k.kv_len = y.y; k.lim0 = y.z; k.part = y.w;
    k.step = k.prob >= 0 && p.a.causal ? 1 : 0;
    return k;
}
// Blocks of [blk0, blk0 + nb) that the slot's last token sees.
__device__ __forceinline__ void clip(Slot &k) {
    const int lim = min(k.kv_len, k.lim0 + k.step * (k.nt - 1));
    const int end = lim <= 0 ? 0 : (lim - 1) / attn::kBlock + 1;
    k.nb = k.nt ? max(0, min(k.nb, end - k.blk0)) : 0;
}
__device__ __forceinline__ Work work_of(const KArgs &p, int w) {
    Work k;
    const int u = w / p.a.hkv;
    k.kvh = w - u * p.a.hkv;
    const int4 *at = (const int4 *)(p.a.units + u);
    const int4 x0 = __ldg(at), y0 = __ldg(at + 1), x1 = __ldg(at + 2), y1 = __ldg(at + 3);
    k.s[0] = slot_of(p, x0, y0);
    k.s[1] = slot_of(p, x1, y1);
    k.shared = k.s[0].nt > p.tpt;
    if (k.shared) {
        k.s[1] = k.s[0];
        k.s[1].nt = k.s[0].nt - p.tpt;
        k.s[0].nt = p.tpt;
        k.s[1].tok0 += p.tpt;
        k.s[1].lim0 += k.s[0].step * p.tpt;
        if (k.s[1].part >= 0) k.s[1].part += p.tpt;
    }
    clip(k.s[0]);
    clip(k.s[1]);
    k.n = max(k.s[0].nb, k.s[1].nb);
    return k;
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
__device__ __forceinline__ void st_global32(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
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

// The products with the upper halves of the shared-memory descriptors as
// immediates: only start addresses change from one to the next (computing whole
// descriptors in a lane-0 branch issued a product every 110 cycles, this one
// every 68).  128-byte swizzle, 8 rows of 128 bytes to a group of 1024 bytes.
// Q and K lie with k contiguous.  V's rows are its k, its N elements are
// contiguous in chunks of 64, and the leading byte offset is the way to the
// next chunk; a K step of 16 rows advances the start address by 2048 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // as tc::desc_sw128 has them
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHi)
        : "memory");
}
// A from tensor memory: row r in lane r, two bf16 of consecutive k per column.
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
            tc::mbar_init(&bars->kv_empty[i], 2);  // one from each slot's MMA warp
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars->q_full[i], 1);
            tc::mbar_init(&bars->q_empty[i], 1);
            tc::mbar_init(&bars->s_full[i], 1);
            tc::mbar_init(&bars->p_full[i][0], 4);
            tc::mbar_init(&bars->p_full[i][1], 4);
            tc::mbar_init(&bars->o_full[i], 1);
            tc::mbar_init(&bars->fin[i], 1);
            tc::mbar_init(&bars->turn[i], 1);
        }
        bars->abort = 0;
        bars->spin_limit = p.spin_limit;
        for (int i = 0; i < kWorks; ++i) {
            tc::mbar_init(&bars->work_full[i], 1);
            tc::mbar_init(&bars->work_empty[i], kThreads / 32 - 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tc::fence_proxy_async();
    }
    if (warp == 10) {
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
    // The units of this CTA, as warp 8 takes them; every other warp waits for
    // the next, reads it in place and gives it back.
    int round = 0;
    auto next_work = [&](bool &ok, auto call) -> const Work * {
        ok = ok && warp_wait<decltype(call)::value>(&bars->work_full[round % kWorks], (uint32_t)((round / kWorks) & 1), bars, status);
        const Work *k = &bars->work[round % kWorks];
        return ok && k->n >= 0 ? k : nullptr;
    };
    auto done_work = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->work_empty[round % kWorks]);
        ++round;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8 || warp == 10) {
            // ---- K and V blocks, one stage each: the first K of each stream, then for each
            // block its V and the K of the block after it.  A stage is up to 16 boxes of a
            // page by two chunks, which one warp issues one after the other: of more than
            // four pieces the two warps take half each (64 single tokens, 16-row pages: 103 us
            // with one warp, 91 us with two).  Warp 8 takes the units, warp 10 loads the Q tiles.
            const int half = warp == 8 ? 0 : 1;
            const int subs = attn::kBlock / p.box_rows;
            const int oob = (int)max(1LL, p.a.n_rows);  // a box from here on reads as zeros
            const bool split = subs * NCH > 4;
            // this lane's box and chunk: of two chunks a warp has one, else every other box
            const int box0 = split ? (NCH == 2 ? lane : 2 * lane + half) : lane / NCH;
            const int chunk = split ? (NCH == 2 ? half : 0) : lane % NCH;
            const bool mine = box0 < subs && (split || !half);
            int st = 0, fill = 0;
            uint32_t par = 1;  // of the stage's last release
            int nq[2] = {0, 0};
            bool ok = true;
            // This lane's box of a block of a stream: what the table says of it, fetched a
            // step ahead, and then its first row.
            auto entry = [&](const Slot &k, int j) {
                const int box = (k.blk0 + j) * subs + box0;
                if (!mine || box * p.box_rows >= k.kv_len) return 0;
                const int32_t *tab = k.prob >= 0 ? p.a.table + (long long)k.prob * p.a.ld_table
                                                 : p.a.ptable + (long long)(-1 - k.prob) * p.a.ld_ptable;
                const int at = !p.a.page ? 0 : p.page_shift >= 0 ? box >> p.page_shift : box * p.box_rows / p.a.page;
                return __ldg(tab + at);
            };
            auto box_row = [&](const Slot &k, int j, int tab) {
                const int box = (k.blk0 + j) * subs + box0, key = box * p.box_rows;
                if (!mine || key >= k.kv_len) return oob;
                const int in = !p.a.page ? key : p.page_shift >= 0 ? key & (p.a.page - 1) : key % p.a.page;
                const long long x = p.a.page ? (long long)tab * p.a.page + in : (long long)tab + in;
                if (x < 0 || x + min(p.box_rows, k.kv_len - key) > p.a.n_rows) {
                    atomicExch(status, (int)LORA_ERR_DEVICE_INDEX);
                    // a cache of no rows has none to read (its maps have one, as maps need)
                    if (!p.a.n_rows || x < -(long long)p.box_rows || x > p.a.n_rows) return oob;
                }
                return (int)x;
            };
            auto load = [&](const CUtensorMap *map, int kvh, int row) {
                // After a wait somewhere in the CTA gave up no more copies are issued, also where
                // stages still come back: the other warp's half of one, or the bytes that it is
                // to expect, may be missing, and a barrier counts bytes only so far.
                const int gone = *(volatile int *)&bars->abort;
                ok &= wait(&bars->kv_empty[st], par, bars, status);  // at once for a stage's first fill
                ok &= !gone;
                if (ok) {
                    if (!half && lane == 0) tc::mbar_expect_tx(&bars->kv_full[st], Sh::kStage);
                    if (mine)
                        tc::tma_load_3d(ring + st * Sh::kStage + chunk * kChunkBytes + box0 * p.box_rows * 128, map,
                                        chunk * 64, kvh, row, &bars->kv_full[st]);
                    ++fill;
                }
                if (++st == kNS) {
                    st = 0;
                    par ^= 1u;
                }
            };
            auto load_q = [&](const Work &k) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!k.s[s].nb) continue;
                    if (nq[s]) ok &= wait(&bars->q_empty[s], (uint32_t)((nq[s] - 1) & 1), bars, status);
                    if (ok && lane == 0) {
                        tc::mbar_expect_tx(&bars->q_full[s], p.q_bytes);
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            tc::tma_load_3d(sq + s * Sh::kStage + c * kChunkBytes, &p.tq, c * 64, k.kvh * p.a.G,
                                            k.s[s].tok0, &bars->q_full[s]);
                    }
                    ++nq[s];
                }
            };
            // Units are taken one after the other, each when the one before is nearly loaded
            // (sooner would bind the rest of the work to whoever asked first).
            int w = blockIdx.x;  // the first is given (the plan has room for it, built or not)
            Work k;
            if (!half) k = work_of(p, w);
            const int n_work = half ? 0 : __ldg(p.a.counters + attn::kUnits) * p.a.hkv;
            while (ok) {
                if (half) {
                    const Work *at = next_work(ok, Call<true>());
                    if (!at) break;
                    k = *at;
                    done_work();
                } else {
                    if (round && (unsigned)w < (unsigned)n_work) k = work_of(p, w);
                    if (round >= kWorks)
                        ok = warp_wait<true>(&bars->work_empty[round % kWorks], (uint32_t)((round / kWorks - 1) & 1), bars, status);
                    if (lane == 0) {
                        if ((unsigned)w < (unsigned)n_work) bars->work[round % kWorks] = k; else bars->work[round % kWorks].n = -1;
                        tc::mbar_arrive(&bars->work_full[round % kWorks]);
                    }
                    __syncwarp();
                    ++round;
                    if ((unsigned)w >= (unsigned)n_work) break;
                }
                const int nb[2] = {k.shared ? k.n : k.s[0].nb, k.shared ? 0 : k.s[1].nb};
                int row[2] = {oob, oob}, tab[2];
                tab[0] = nb[0] ? entry(k.s[0], 0) : 0;
                tab[1] = nb[1] ? entry(k.s[1], 0) : 0;
                // The Q tiles are free when the unit before has issued its last QK: by then
                // some of this unit's blocks are on their way, but not more than the ring holds.
                bool q_due = half;
                if (half && (!split || !fill)) {
                    load_q(k);
                    q_due = false;
                    if (!split) {
                        ok = all(ok);
                        continue;
                    }
                }
                int taken = 0;
                const int ask = max(-1, k.n - 3);
#pragma unroll 1
                for (int j = -1; j < k.n; ++j) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (j >= 0 && j < nb[c]) load(&p.tv, k.kvh, row[c]);
                        if (q_due && j >= 0) {
                            load_q(k);
                            q_due = false;
                        }
                        if (j + 1 < nb[c]) {
                            row[c] = box_row(k.s[c], j + 1, tab[c]);
                            if (j + 2 < nb[c]) tab[c] = entry(k.s[c], j + 2);
                            load(&p.tk, k.kvh, row[c]);
                        }
                    }
                    if (!half && j == ask && lane == 0) taken = atomicAdd(p.a.tickets, 1);
                }
                w = __shfl_sync(0xffffffffu, taken, 0) + (int)gridDim.x;
                ok = all(ok);
            }
            if (!half) {
                __threadfence();  // what was taken is taken before the CTA counts as done
                if (lane == 0 && atomicAdd(p.a.tickets + 1, 1) == (int)gridDim.x - 1) {
                    p.a.tickets[0] = 0;  // the last CTA to end leaves them as they were
                    p.a.tickets[1] = 0;
                }
            }
            // every copy has landed before the CTA ends
#pragma unroll 1
            for (int s = 0; s < kNS && s < fill; ++s) {
                const int last = fill - 1 - ((fill - 1 - s) % kNS);
                int polls = 0;
#pragma unroll 1
                while (!tc::mbar_try_wait(&bars->kv_full[s], (uint32_t)((last / kNS) & 1)) && ++polls < kLand) {}
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                int polls = 0;
#pragma unroll 1
                while (nq[s] && !tc::mbar_try_wait(&bars->q_full[s], (uint32_t)((nq[s] - 1) & 1)) && ++polls < kLand) {}
            }
        } else {
            // ---- MMA issue of one slot
            constexpr uint32_t id_qk = tc::idesc_bf16(128, 128), id_pv = tc::idesc_bf16_bmn(128, Sh::kDP);
            const int s = warp == 9 ? 0 : 1;
            int st = 0;                // the next stage of the ring and its parity
            uint32_t par = 0;
            auto step = [&]() {
                if (++st == kNS) {
                    st = 0;
                    par ^= 1u;
                }
            };
            uint32_t pq = 0, pp = 0, pt = 0;
            bool ok = true;
            // lower halves of the descriptors (shared addresses end below 2^18): of K-major
            // tiles, and of V, whose 64-element chunks are kChunkBytes apart
            const uint32_t q_lo = ((tc::smem_u32(sq) + s * Sh::kStage) >> 4) | (1u << 16);
            const uint32_t k_lo = (tc::smem_u32(ring) >> 4) | (1u << 16);
            const uint32_t v_lo = (tc::smem_u32(ring) >> 4) | ((uint32_t)(kChunkBytes >> 4) << 16);
            const uint32_t ts = tmem + s * 128, to = tmem + 256 + s * Sh::kDP;
            uint64_t *s_full = &bars->s_full[s], *p_full = bars->p_full[s];
            auto qk = [&](int stage) {  // by one lane
                const uint32_t ka = k_lo + stage * (Sh::kStage >> 4);
#pragma unroll
                for (int i = 0; i < NCH * 4; ++i) {
                    const uint32_t off = (uint32_t)((i >> 2) * kChunkBytes + (i & 3) * 32) >> 4;
                    mma_ss(ts, q_lo + off, ka + off, id_qk, i != 0);
                }
                tc::mma_commit(s_full);
            };
            auto pv = [&](int h, int stage, bool first) {
                const uint32_t va = v_lo + stage * (Sh::kStage >> 4) + h * (8192 >> 4);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_ts(to, ts + h * 32 + i * 8, va + i * (2048 >> 4), id_pv, h || i ? true : !first);
            };
            // Fills of the other slot's stream.  Both warps see every phase of every stage
            // (a parity wait is exact only within one phase), so both give every stage back.
            auto pass = [&](int n) {
#pragma unroll 1
                for (; n; --n) {
                    ok &= wait(&bars->kv_full[st], par, bars, status);
                    if (elect_one()) tc::mbar_arrive(&bars->kv_empty[st]);
                    step();
                }
            };
            while (const Work *k = next_work(ok, Call<true>())) {
                const Slot &me = k->s[s];
                const int nb = me.nb, other = k->s[1 - s].nb, most = k->n;
                const bool alone = !k->shared;
                const int n = alone ? nb : most;  // blocks of the stream
                const int full = (me.kv_len >> 7) - me.blk0;  // blocks whose keys all count
                // step j: PV of block j and QK of block j + 1, from -1 on
#pragma unroll 1
                for (int j = -1; j < most; ++j) {
                    // fills of the other stream that come between
                    const int between = alone ? (j >= 0 && j < other) + (j + 1 < other) : 0;
                    if (s) pass(between);
                    // The slots of one stream issue by turns, so that one slot's products are
                    // done, and its softmax begins, while the other's are still to come.
                    auto turn = [&]() {
                        if (alone || (!s && j <= 0) || j < 0) return;
                        ok &= wait(&bars->turn[s], pt, bars, status);
                        pt ^= 1u;
                    };
                    if (j < n) {
                        const bool has = j >= 0, more = j + 1 < n;
                        const int sv = st;
                        const uint32_t par_v = par;
                        if (has) step();
                        const int sk = st;
                        const uint32_t par_k = par;
                        if (more) step();
                        if (has) ok &= wait(&bars->kv_full[sv], par_v, bars, status);
                        if (more) ok &= wait(&bars->kv_full[sk], par_k, bars, status);
                        if (has && j >= full) {
                            // values past the last key count for nothing, whatever their rows
                            // hold (boxes past the one it is in are zeros already; the slots of
                            // one stream both write the same zeros)
                            const int left = me.kv_len - (me.blk0 + j) * attn::kBlock;
                            const int end = (left + p.box_rows - 1) / p.box_rows * p.box_rows * 8;
                            char *v = ring + sv * Sh::kStage;
#pragma unroll 1
                            for (int i = left * 8 + lane; i < end; i += 32)
#pragma unroll
                                for (int c = 0; c < NCH; ++c)
                                    *(uint4 *)(v + c * kChunkBytes + i * 16) = make_uint4(0, 0, 0, 0);
                            tc::fence_proxy_async();
                        }
                        const bool pv_due = has && j < nb, qk_due = j + 1 < nb;
                        if (pv_due) ok &= wait(&p_full[0], pp, bars, status);
                        turn();
                        if (pv_due) {
                            tc::tc_fence_after();
                            if (elect_one()) pv(0, sv, j == 0);
                            ok &= wait(&p_full[1], pp, bars, status);
                            pp ^= 1u;
                        }
                        if (!has && qk_due) {
                            ok &= wait(&bars->q_full[s], pq, bars, status);
                            pq ^= 1u;
                        }
                        tc::tc_fence_after();
                        if (elect_one()) {
                            if (pv_due) pv(1, sv, false);
                            if (qk_due) {
                                qk(sk);
                                if (j + 2 == nb) tc::mma_commit(&bars->q_empty[s]);
                            } else if (pv_due) {
                                tc::mma_commit(&bars->o_full[s]);
                            }
                            if (has && !alone && (more || !s)) tc::mbar_arrive(&bars->turn[1 - s]);
                            if (has) tc::mma_commit(&bars->kv_empty[sv]);
                            if (more) tc::mma_commit(&bars->kv_empty[sk]);
                        }
                    }
                    if (!s) pass(between);
                }
                ok = all(ok);
                done_work();
            }
            // all products are done before tensor memory is given back, also those of a unit
            // that was given up (a commit counts the products of the lane that issues it)
            if (elect_one()) tc::mma_commit(&bars->fin[s]);
            __syncwarp();
            int polls = 0;
#pragma unroll 1
            while (!tc::mbar_try_wait(&bars->fin[s], 0) && ++polls < kLand) {}
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- softmax and epilogue of one slot, a row per thread
        const int s = warp >> 2, q = warp & 3, row = q * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t ts = tl + s * 128, to = tl + 256 + s * Sh::kDP;
        const int e = row / p.a.G, g = row - e * p.a.G;
        const float scale = p.a.scale_log2;
        uint32_t ps = 0, po = 0;
        bool ok = true;
        while (const Work *at = next_work(ok, Call<false>())) {
            const Slot k = at->s[s];
            const int kvh = at->kvh;
            done_work();
            if (!k.nt) continue;
            const bool live = e < k.nt, warp_live = __any_sync(0xffffffffu, live);
            // keys that the row sees; a row that is not there masks nothing
            const int lim = live ? min(k.kv_len, k.lim0 + k.step * e) : 0x7fffffff;
            const int min_lim = __reduce_min_sync(0xffffffffu, lim);
            float m = -INFINITY, l = 0.f, base = 0.f;
            bool huge = false;
#pragma unroll 1
            for (int j = 0; j < k.nb; ++j) {
                if (!(ok = warp_wait<false>(&bars->s_full[s], ps, bars, status))) break;
                ps ^= 1u;
                if (warp_live) {
                    tc::tc_fence_after();
                    uint32_t x[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::tmem_ld32(ts + c * 32, x[c]);
                    tc::tmem_wait_ld();
                    const int key0 = (k.blk0 + j) * attn::kBlock;
                    if (key0 + attn::kBlock > min_lim) {
                        const int rel = lim - key0;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (key0 + c * 32 + 32 <= min_lim) continue;  // seen whole by all rows
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i >= rel) x[c][i] = 0xff800000u;
                        }
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
                    // the maximum in use stays while no row's scores are more than kLag above it
                    if (__any_sync(0xffffffffu, live && !((bm - m) * scale <= kLag))) {
                        const float mn = fmaxf(m, bm);
                        const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * scale);
                        m = mn;
                        l *= f;
                        base = m == -INFINITY ? 0.f : m * scale;
                        huge = __any_sync(0xffffffffu, live && !(fabsf(base) <= kExactBase));
#pragma unroll 1
                        for (int c = 0; j && c < Sh::kDP / 16; ++c) {  // the output so far, with the weights
                            uint32_t o[16];
                            tc::tmem_ld16(to + c * 16, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tc::tmem_st16(to + c * 16, o);
                        }
                    }
                    // 2^(x * scale - base): whatever base was rounded to divides out, unless
                    // it is so large that its rounding is; then x - maximum goes first
                    f32x2 sc2 = two(scale, scale), sb2 = two(-base, -base), s0 = two(0.f, 0.f), s1 = s0;
                    if (huge) {
                        const float mm = m == -INFINITY ? 0.f : m;
                        tc::tmem_st32(ts, x[0]);
                        tc::tmem_st32(ts + 32, x[1]);
                        tc::tmem_st32(ts + 64, x[2]);
                        tc::tmem_st32(ts + 96, x[3]);
                        tc::tmem_wait_st();
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[16];
                            tc::tmem_ld16(ts + c * 16, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint((__uint_as_float(o[i]) - mm) * scale);
                            tc::tmem_st16(ts + c * 16, o);
                        }
                        tc::tmem_wait_st();
#pragma unroll
                        for (int c = 0; c < 4; ++c) tc::tmem_ld32(ts + c * 32, x[c]);
                        tc::tmem_wait_ld();
                        sc2 = two(1.f, 1.f);
                        sb2 = two(0.f, 0.f);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 v = apart(fma2(two(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])),
                                                  sc2, sb2));
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            if (i & 1) s1 = add2(s1, two(v.x, v.y)); else s0 = add2(s0, two(v.x, v.y));
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
                    const float2 sm = apart(add2(s0, s1));
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
            if (k.nb) {
                if (!(ok = warp_wait<false>(&bars->o_full[s], po, bars, status))) break;
                po ^= 1u;
                tc::tc_fence_after();
            }
            if (warp_live) {
                const bool some = k.nb && l != 0.f;  // a row that saw no key gets zeros
                const float inv = some ? 1.f / l : 0.f;
                const int rows = k.nt * p.a.G;
                const long long prow = (long long)k.part * p.a.hq + (long long)kvh * rows;
                uint16_t *out = p.a.out + (long long)(k.tok0 + e) * p.a.ldo + (long long)(kvh * p.a.G + g) * p.a.D;
                float *part = p.a.part_o + prow * p.a.D + 8 * row;
                // a loop, though of few rounds: code that a unit runs once comes from beyond
                // the instruction cache, and unrolled this took longer than its work
#pragma unroll 1
                for (int c = 0; c < p.a.D; c += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(to + c, o);
                    tc::tmem_wait_ld();
                    if (!live) continue;
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = some ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
                    if (k.part >= 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (c + 8 * i < p.a.D) st_global32(part, o + 8 * i);
                            part += 8 * rows;
                        }
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = pack2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                    if (p.out32) {  // whole 32-byte sectors
                        st_global32(out + c, o);
                        if (c + 16 < p.a.D) st_global32(out + c + 16, o + 8);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (c + 8 * i < p.a.D)
                                *(uint4 *)(out + c + 8 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (live && k.part >= 0) p.a.part_lse[prow + row] = l == 0.f ? -INFINITY : m * scale + log2f(l);
                tc::tc_fence_before();
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 10) tc::tmem_dealloc(tmem, 512);
}

std::atomic<int> g_attn_sms[64];  // SM count per device, looked up once

template <int NCH>
cudaError_t launch(KArgs &p, int dev, int grid, cudaStream_t s) {
    static std::atomic<bool> ready[64];  // the shared-memory limit is set once per device
    if (!ready[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(item_kernel<NCH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<NCH>::kSmem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
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
    p.spin_limit = lora_spin_limit();
    p.tpt = attn::tile_tokens(a.G);
    p.box_rows = attn::kBlock;
    if (a.page)
        while (a.page % p.box_rows) p.box_rows >>= 1;
    const int boxes = a.page / p.box_rows;
    p.page_shift = boxes & (boxes - 1) ? -1 : 0;
    while (p.page_shift >= 0 && boxes >> (p.page_shift + 1)) ++p.page_shift;
    const int nch = a.D > 64 ? 2 : 1;
    p.q_bytes = nch * 128 * a.G * p.tpt;
    p.out32 = a.D % 16 == 0 && a.ldo % 16 == 0 && ((uintptr_t)a.out & 31) == 0;
    const long long rows = a.n_rows > 0 ? a.n_rows : 1;
    if (!lora_make_tmap_heads(&p.tq, a.q, a.D, a.hq, a.T, a.ldq, a.G, p.tpt) ||
        !lora_make_tmap_heads(&p.tk, a.k, a.D, a.hkv, rows, a.ldk, 1, p.box_rows) ||
        !lora_make_tmap_heads(&p.tv, a.v, a.D, a.hkv, rows, a.ldv, 1, p.box_rows))
        return LORA_ERR_UNSUPPORTED;
    const long long n = (long long)max_items * a.hkv;
    const int grid = (int)(n < n_sms ? n : n_sms);
    LORA_CUDA_TRY(nch == 2 ? launch<2>(p, dev, grid, s) : launch<1>(p, dev, grid, s));
    lora_note_launch();
    return LORA_OK;
}
