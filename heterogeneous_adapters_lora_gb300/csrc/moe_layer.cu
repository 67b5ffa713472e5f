// A whole layer of experts for a few tokens: the chosen experts' products, the
// deltas of the tokens' adapters, the activation and the weighted sum.
//
// With few tokens the time is that of reading the chosen experts' weights once.
// Two kernels of the same make stream them through the tensor cores, W13 and
// then W2, with the roles of a product turned round: 128 rows of a weight are the MMA's
// M, the pairs (token, expert) of one expert its N, so a weight goes from DRAM to shared
// memory by TMA and from there straight into tcgen05.mma, past the registers, and up to
// 64 pairs cost what one costs.
//
//   shrink13   v[p] = scale A13 x        (with adapters; runs under the start of up)
//   up         g, u = W13 x + B13 v; h = act(g) u; parts of A2 h      per 128 columns of h
//   down       y[p] = w (W2 h + B2 (scale A2 h))                     per 256 rows of W2
//   combine    out[t] = sum of y over the token's pairs, in their order, one rounding
//
// Work is cut by bytes, not by tiles.  A unit is 256 weight rows (128 of gate and 128
// of up, or 256 of W2) for one group (an expert and up to 64 of its pairs), a block 64 columns of
// them (32 KB).  All units' blocks in a row are divided evenly among one CTA per SM,
// so a unit may be shared: its other CTAs leave fp32 sums in the workspace, and the one
// that has its last block adds them, lower columns first, and finishes the unit.  A CTA works from its
// last unit to its first, so what others wait for comes first, and only CTAs of
// lower index are waited for, which have started earlier.  Every CTA finds its groups from
// topk_ids by itself (a histogram and a scan in shared memory).
//
// Roles (320 threads): warp 0 issues the TMA copies, one lane the two weight boxes of a
// block, the others four gathered rows each (tile::gather4 by token, or by pair); warp 1 issues the MMAs;
// warps 2-9 are the epilogue, a row per thread, two warps per quarter of the accumulator's lanes
// which take turns at four columns (pairs) each, under the next unit's MMAs (two accumulators).
//
// Roundings: sums are fp32 throughout (accumulators, v, parts, y).  h enters the second
// product in 16 bits: as two bf16, h = hi + lo, in separate columns whose sums are
// added (2^-17 of h instead of 2^-9; the weights' bytes bound the kernel, not its MMAs).
#include <math.h>
#include <stddef.h>
#include <string.h>

#include <atomic>

#include "lora_internal.cuh"
#include "tc_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxE = LORA_ROUTE_MAX_EXPERTS, kMaxP = LORA_MOE_LAYER_MAX_PAIRS;
constexpr int kGroup = 64;                    // pairs of a group
constexpr int kRows = 256, kTile = 128;       // weight rows of a unit, of an MMA
constexpr int kBK = 64;                       // columns of a block: one 128-byte swizzle row
constexpr uint32_t kABytes = kRows * kBK * 2;
constexpr int kStreamThreads = 320, kEpi0 = 2, kEpiThreads = 256;
constexpr int kSms = 152;                     // where no device answers
constexpr int kLeast = 4;                     // fewest blocks worth a CTA

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
    float *v13;                   // [P][2][R], scaled
    uint16_t *h;                  // [2][P][F]: hi, lo
    float *v2;                    // [P][ceil(F / 128)][R], parts of A2 h
    float *y;                     // [P][D], weighted
    float *part;                  // [CTA][2][kGroup][kTile] sums of shared units
    int *flags;                   // [2][CTA] part is there (up, down)
    int grid, spin_limit;
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
__device__ __forceinline__ float dot_bf16(const uint16_t *a, const uint16_t *b, int n, int lane) {
    float s = 0.f;
    for (int i = lane * 8; i < n; i += 256) s += dot8(__ldg((const uint4 *)(a + i)), __ldg((const uint4 *)(b + i)));
    return warp_sum(s);
}

// scale * A x of every pair: a warp per (pair, slice, rank row)
__global__ void __launch_bounds__(kThreads) shrink13_kernel(const LayerArgs p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
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

// ------------------------------------------------------------ streamed products

struct StreamArgs {
    CUtensorMap tm_w, tm_b;
    LayerArgs a;
    int KB, MT;  // blocks of a unit, units of a group
};

template <bool DOWN>
struct Shape {
    static constexpr int kCols = DOWN ? 2 * kGroup : kGroup;  // accumulator columns of a tile (down: hi, then lo)
    static constexpr uint32_t kStage = kABytes + kCols * 128;
    static constexpr int kStages = DOWN ? 4 : 5;
    static constexpr int kTmem = 4 * kCols;  // two tiles, two buffers
};

struct Shared {
    uint64_t full[5], empty[5], accf[2], acce[2];
    uint32_t tmem;
    int abort;
    uint16_t groups[kMaxE + 8], pairs[kMaxE + 8];  // groups and pairs of the experts before this one
    uint16_t list[kMaxP];                          // pairs of this CTA's experts, by expert
    int slot[kGroup], rank[kGroup];                // of a unit's pairs: adapter slot (-1: none), its rank
    float scale[kGroup], weight[kGroup];
    union alignas(16) {
        struct {
            int count[kMaxE];
            uint16_t ids[kMaxP];
        } g;                                                 // while groups are found
        float h[2][2][4][kTile + 4];                         // up: four columns of h of each half of the warps, twice
        float v2[2][4][LORA_MAX_RANK];                       // down: scale A2 h of four pairs
    } u;
};

static_assert(offsetof(Shared, u) % 16 == 0 && sizeof(float[kTile + 4]) % 16 == 0, "columns of h are read 16 bytes at a time");

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

// Operands in 128-byte swizzled rows, 8 rows to 1024 bytes; only start addresses change.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)acc), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem) { return ((smem >> 4) & 0x3fffu) | (1u << 16); }

// Four rows of a matrix (64 columns from x on) to consecutive 128-byte lines.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int x, int4 rows, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(tc::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void note_timeout(const LayerArgs &p, Shared &s) {
    *(volatile int *)&s.abort = 1;
    if (p.status) atomicExch(p.status, (int)LORA_ERR_TIMEOUT);
}
// Waits for a phase of a barrier; false once any wait of the CTA has given up.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const LayerArgs &p, Shared &s) {
    int polls = 0;
    while (!tc::mbar_try_wait(bar, parity)) {
        if (*(volatile int *)&s.abort) return false;
        if (++polls > p.spin_limit) {
            note_timeout(p, s);
            return false;
        }
    }
    return true;
}
constexpr int kLand = 1 << 20;  // polls for copies and products in flight, before a CTA ends
__device__ __forceinline__ void land(uint64_t *bar, uint32_t parity) {
    int polls = 0;
    while (!tc::mbar_try_wait(bar, parity) && ++polls < kLand) {}
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A barrier that tells all of its threads whether `ok` holds in every one.
__device__ __forceinline__ bool bar_and(int id, int threads, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)ok), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// The groups of the batch, as prefix sums over the experts.
__device__ int find_groups(const LayerArgs &p, Shared &s) {
    for (int i = threadIdx.x; i < p.E; i += kStreamThreads) s.u.g.count[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.P; i += kStreamThreads) {
        const int e = p.ids[i];
        const bool ok = e >= 0 && e < p.E;
        s.u.g.ids[i] = ok ? (uint16_t)e : 0xffffu;
        if (ok) atomicAdd(&s.u.g.count[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int groups = 0, pairs = 0;
        for (int e0 = 0; e0 <= p.E; e0 += 32) {
            const int c = e0 + lane < p.E ? s.u.g.count[e0 + lane] : 0, n = (c + kGroup - 1) / kGroup;
            int cs = c, ns = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(kAll, cs, o), b = __shfl_up_sync(kAll, ns, o);
                if (lane >= o) cs += a, ns += b;
            }
            if (e0 + lane <= p.E) {
                s.groups[e0 + lane] = (uint16_t)(groups + ns - n);
                s.pairs[e0 + lane] = (uint16_t)(pairs + cs - c);
            }
            groups += __shfl_sync(kAll, ns, 31);
            pairs += __shfl_sync(kAll, cs, 31);
        }
    }
    __syncthreads();
    return s.groups[p.E];
}
__device__ __forceinline__ int expert_of_group(const LayerArgs &p, const Shared &s, int g) {
    int lo = 0, hi = p.E;  // groups[lo] <= g < groups[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.groups[mid] <= g) lo = mid;
        else hi = mid;
    }
    return lo;
}
// The pairs of experts e0..e1 in their order, each expert's by a warp.
__device__ void list_pairs(const LayerArgs &p, Shared &s, int e0, int e1) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = e0 + warp; e <= e1; e += kStreamThreads / 32) {
        int at = s.pairs[e] - s.pairs[e0];
        if (s.pairs[e + 1] == s.pairs[e]) continue;
        for (int i = 0; i < p.P; i += 32) {
            const bool mine = i + lane < p.P && s.u.g.ids[i + lane] == e;
            const unsigned m = __ballot_sync(kAll, mine);
            if (mine) s.list[at + __popc(m & ((1u << lane) - 1))] = (uint16_t)(i + lane);
            at += __popc(m);
        }
    }
}

// What a CTA does: blocks [b0, b1) of all the units' blocks in a row.
struct Range {
    int b0, b1, total, n;  // n CTAs share them
    __device__ __forceinline__ int start(int c) const { return (int)((long long)total * c / n); }
};

// The CTA's part of unit u, and what the unit is.
struct Part {
    int k0, k1;        // blocks of the unit
    int e, m, n, at;   // expert, place in it, pairs, first of them in the list
};
__device__ __forceinline__ Part part_of(const StreamArgs &q, const Shared &s, const Range &r, int u, int e_first) {
    Part x;
    x.k0 = max(r.b0 - u * q.KB, 0);
    x.k1 = min(r.b1 - u * q.KB, q.KB);
    const int g = u / q.MT;
    x.m = u - g * q.MT;
    x.e = expert_of_group(q.a, s, g);
    const int first = s.pairs[x.e] + (g - s.groups[x.e]) * kGroup;
    x.n = min(kGroup, s.pairs[x.e + 1] - first);
    x.at = first - s.pairs[e_first];
    return x;
}

// sum_r b[r] v[r] of up to 4 rows of B (16 bytes each 8 ranks), v in shared or global memory
template <int N>
__device__ __forceinline__ void expand_rows(float (&acc)[N], const uint16_t *const (&b)[N], const float *const (&v)[N],
                                            const int (&rank)[N], int most) {
    for (int r = 0; r < most; r += 8) {
        uint4 w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = r < rank[j] ? __ldg((const uint4 *)(b[j] + r)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (r >= rank[j]) continue;
            const uint32_t c[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r + i < rank[j]) acc[j] += (i & 1 ? bf16hi(c[i >> 1]) : bf16lo(c[i >> 1])) * v[j][r + i];
        }
    }
}

template <bool DOWN>
constexpr size_t stream_smem() {
    return 1024 + (size_t)Shape<DOWN>::kStages * Shape<DOWN>::kStage + sizeof(Shared);
}
static_assert(stream_smem<false>() <= 227 * 1024 && stream_smem<true>() <= 227 * 1024, "shared memory of a CTA");

template <bool DOWN>
__global__ void __launch_bounds__(kStreamThreads, 1) stream_kernel(const __grid_constant__ StreamArgs q) {
    typedef Shape<DOWN> Sh;
    extern __shared__ __align__(1024) char smem_raw[];
    char *ring = smem_raw + ((1024u - (smem_u32_of(smem_raw) & 1023u)) & 1023u);
    Shared &s = *(Shared *)(ring + (size_t)Sh::kStages * Sh::kStage);
    const LayerArgs &p = q.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Without adapters the kernel before up is the caller's, which may have written
    // topk_ids; shrink13, and up before down, let this one start when those are complete.
    if (!DOWN && !p.L) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        s.abort = 0;
        for (int i = 0; i < Sh::kStages; ++i) {
            tc::mbar_init(&s.full[i], 1);
            tc::mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.accf[i], 1);
            tc::mbar_init(&s.acce[i], kEpiThreads / 32);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tc::tmem_alloc(&s.tmem, Sh::kTmem);
        tc::tmem_relinquish();
    }
    Range r;
    r.total = find_groups(p, s) * q.MT * q.KB;
    r.n = min((int)gridDim.x, max(1, r.total / kLeast));
    const int c = blockIdx.x;
    const bool any = c < r.n && r.total > 0;
    r.b0 = any ? r.start(c) : 0;
    r.b1 = any ? r.start(c + 1) : 0;
    const int u_lo = any ? r.b0 / q.KB : 0, u_hi = any ? (r.b1 - 1) / q.KB : -1;
    const int e_first = any ? expert_of_group(p, s, u_lo / q.MT) : 0;
    if (any) list_pairs(p, s, e_first, expert_of_group(p, s, u_hi / q.MT));
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s.tmem;

    if (warp == 0) {
        // ---- copies.  Weights are nobody's results: those of the first stages are asked for before
        // the kernel before this one is complete, the gathered rows after it.
        int done = 0;  // blocks asked for
        const auto weights = [&](const Part &x, int k, int st) {
            char *dst = ring + (size_t)st * Sh::kStage;
            // rows of the expert's second tile that are there at all
            const bool two = !DOWN || x.m * kRows + kTile < p.D;
            const int n4 = (x.n + 3) & ~3;
            tc::mbar_expect_tx(&s.full[st], (two ? kABytes : kABytes / 2) + (uint32_t)n4 * 128 * (DOWN ? 2 : 1));
            if (DOWN) {
                tc::tma_load_3d(dst, &q.tm_w, k * kBK, x.m * kRows, x.e, &s.full[st]);
                if (two) tc::tma_load_3d(dst + kABytes / 2, &q.tm_w, k * kBK, x.m * kRows + kTile, x.e, &s.full[st]);
            } else {
                tc::tma_load_3d(dst, &q.tm_w, k * kBK, x.m * kTile, 2 * x.e, &s.full[st]);
                tc::tma_load_3d(dst + kABytes / 2, &q.tm_w, k * kBK, x.m * kTile, 2 * x.e + 1, &s.full[st]);
            }
        };
        int ahead = 0;
        if (lane == 0) {
            tc::prefetch_tmap(&q.tm_w);
            tc::prefetch_tmap(&q.tm_b);
            for (int u = u_hi; u >= u_lo && ahead < Sh::kStages; --u) {
                const Part x = part_of(q, s, r, u, e_first);
                for (int k = x.k0; k < x.k1 && ahead < Sh::kStages; ++k) weights(x, k, ahead++);
            }
        }
        ahead = __shfl_sync(kAll, ahead, 0);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("fence.proxy.async.global;" ::: "memory");
        bool ok = true;
        for (int u = u_hi; u >= u_lo && ok; --u) {
            const Part x = part_of(q, s, r, u, e_first);
            // this lane's four rows: of x by token, of h by pair (hi, in the upper lanes lo)
            const int quad = DOWN ? lane & 15 : lane;
            const bool mine = quad * 4 < x.n;
            int4 rows = make_int4(0, 0, 0, 0);
            if (mine) {
                const auto row = [&](int i) {
                    const int pair = s.list[x.at + min(quad * 4 + i, x.n - 1)];
                    return DOWN ? pair + (lane >> 4) * p.P : pair / p.K;
                };
                rows = make_int4(row(0), row(1), row(2), row(3));
            }
            const uint32_t off = kABytes + (uint32_t)(quad * 4 + (DOWN ? (lane >> 4) * ((x.n + 7) & ~7) : 0)) * 128;
            for (int k = x.k0; k < x.k1; ++k) {
                const int st = done % Sh::kStages;
                if (done >= ahead) {
                    if (lane == 0) {
                        ok = wait(&s.empty[st], (uint32_t)((done / Sh::kStages - 1) & 1), p, s);
                        if (ok) weights(x, k, st);
                    }
                    ok = __shfl_sync(kAll, (int)ok, 0);
                    if (!ok) break;
                }
                if (mine) tma_gather4(tc::smem_u32(ring) + st * Sh::kStage + off, &q.tm_b, k * kBK, rows, &s.full[st]);
                ++done;
            }
        }
        // every copy has landed before the CTA ends (given up or not: all that was asked for comes)
        if (lane == 0)
            for (int i = max(0, done - Sh::kStages); i < done; ++i)
                land(&s.full[i % Sh::kStages], (uint32_t)((i / Sh::kStages) & 1));
    } else if (warp == 1) {
        // ---- products
        int done = 0, i = 0;
        bool ok = true;
        for (int u = u_hi; u >= u_lo && ok; --u, ++i) {
            const Part x = part_of(q, s, r, u, e_first);
            const int buf = i & 1;
            const bool two = !DOWN || x.m * kRows + kTile < p.D;
            const int cols = DOWN ? 2 * ((x.n + 7) & ~7) : (x.n + 15) & ~15;
            const uint32_t idesc = tc::idesc_bf16(kTile, cols);
            if (i >= 2) ok = __all_sync(kAll, wait(&s.acce[buf], (uint32_t)(((i >> 1) - 1) & 1), p, s));
            tc::tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(buf * 2 * Sh::kCols);
            for (int k = x.k0; k < x.k1 && ok; ++k, ++done) {
                const int st = done % Sh::kStages;
                ok = __all_sync(kAll, wait(&s.full[st], (uint32_t)((done / Sh::kStages) & 1), p, s));
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t base = tc::smem_u32(ring) + (uint32_t)st * Sh::kStage;
                const uint32_t a0 = desc_lo(base), a1 = desc_lo(base + kABytes / 2), b = desc_lo(base + kABytes);
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kBK / 16; ++j) {
                        mma_ss(d, a0 + j * 2, b + j * 2, idesc, (k - x.k0) | j);
                        if (two) mma_ss(d + Sh::kCols, a1 + j * 2, b + j * 2, idesc, (k - x.k0) | j);
                    }
                    tc::mma_commit(&s.empty[st]);
                    if (k == x.k1 - 1) tc::mma_commit(&s.accf[buf]);
                }
            }
        }
        // products in flight read the ring and write tensor memory: the next stage's barrier tells their end
        if (done > 0 && lane == 0) {
            const int last = done - 1;
            land(&s.empty[last % Sh::kStages], (uint32_t)((last / Sh::kStages) & 1));
        }
        __syncwarp();
    } else {
        // ---- epilogue
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int tid = threadIdx.x - kEpi0 * 32;
        const int quarter = warp & 3, half = (warp - kEpi0) >> 2, row = quarter * 32 + lane;
        const int htid = quarter * 32 + lane;  // thread of its half
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        float *const my_part = p.part + (size_t)c * 2 * kGroup * kTile;
        int *const flags = p.flags + (DOWN ? p.grid : 0);
        int i = 0;
        for (int u = u_hi; u >= u_lo; --u, ++i) {
            const Part x = part_of(q, s, r, u, e_first);
            const int buf = i & 1;
            const bool last = x.k1 == q.KB;
            const uint32_t acc = tmem + lanes + (uint32_t)(buf * 2 * Sh::kCols);
            const int lo_col = (x.n + 7) & ~7;
            bar_sync(1, kEpiThreads);  // the last unit's slots are no longer read
            if (last && tid < x.n) {
                const int pair = s.list[x.at + tid], slot = slot_of(p, pair / p.K, false);
                s.slot[tid] = slot;
                s.rank[tid] = slot >= 0 ? p.rank[slot] : 0;
                s.scale[tid] = slot >= 0 ? p.scale[slot] : 0.f;
                s.weight[tid] = p.topk_w ? p.topk_w[pair] : 1.f;
            }
            bool ok = wait(&s.accf[buf], (uint32_t)((i >> 1) & 1), p, s);
            // sums that other CTAs have left of this unit
            int from = c;
            if (last && x.k0 > 0) {
                // the CTA that has the unit's first block: start(f) <= u KB < start(f + 1)
                from = (int)((long long)u * q.KB * r.n / r.total);
                while (r.start(from) > u * q.KB) --from;
                while (r.start(from + 1) <= u * q.KB) ++from;
                if (tid < c - from) {
                    int polls = 0;
                    while (ok && ld_acquire_gpu(flags + from + tid) == 0) {
                        if (*(volatile int *)&s.abort) ok = false;
                        else if (++polls > p.spin_limit) {
                            note_timeout(p, s);
                            ok = false;
                        } else
                            __nanosleep(64);
                    }
                }
            }
            // one wait that gave up ends the work of all
            ok = bar_and(1, kEpiThreads, ok);
            if (!ok) break;
            tc::tc_fence_after();
            int turn = 0;
#pragma unroll 1
            for (int col = half * 4; col < x.n; col += 8) {
                float g[4], v[4];  // gate and up; or the two tiles' rows
                tmem_ld4(acc + col, g);
                tmem_ld4(acc + Sh::kCols + col, v);
                if (DOWN) {
                    float gl[4], vl[4];
                    tmem_ld4(acc + lo_col + col, gl);
                    tmem_ld4(acc + Sh::kCols + lo_col + col, vl);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) g[j] += gl[j], v[j] += vl[j];
                } else {
                    tc::tmem_wait_ld();
                }
                if (!last) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        __stcg(my_part + (size_t)(col + j) * kTile + row, g[j]);
                        __stcg(my_part + (size_t)(kGroup + col + j) * kTile + row, v[j]);
                    }
                    continue;
                }
                for (int f = from; f < c; ++f) {
                    const float *o = p.part + (size_t)f * 2 * kGroup * kTile;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        g[j] += __ldcg(o + (size_t)(col + j) * kTile + row);
                        v[j] += __ldcg(o + (size_t)(kGroup + col + j) * kTile + row);
                    }
                }
                int pair[4], slot[4], rank[4], most = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = min(col + j, x.n - 1);
                    pair[j] = s.list[x.at + k];
                    slot[j] = s.slot[k];
                    rank[j] = col + j < x.n ? s.rank[k] : 0;
                    most = max(most, rank[j]);
                }
                if (!DOWN) {
                    const int f = x.m * kTile + row;
                    const bool there = f < p.F;
                    if (most && there) {
                        const uint16_t *b[4];
                        const float *vv[4];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int n = t ? p.n13 - 1 : 0, first = t ? p.b_up : 0;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int rs = (rank[j] + 7) & ~7;
                                b[j] = p.B[n] + (long long)slot[j] * p.b_ss[n] + ((long long)x.e * p.b_rows[n] + first + f) * rs;
                                vv[j] = p.v13 + ((long long)pair[j] * 2 + t) * p.R;
                            }
                            expand_rows<4>(t ? v : g, b, vv, rank, most);
                        }
                    }
                    float(*sh)[kTile + 4] = s.u.h[half][turn];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float h = there ? activation(g[j], p.gelu) * v[j] : 0.f;
                        if (most) sh[j][row] = h;
                        if (there && col + j < x.n) {
                            const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                            const __nv_bfloat16 lo = __float2bfloat16_rn(h - __bfloat162float(hi));
                            p.h[(long long)pair[j] * p.F + f] = *(const uint16_t *)&hi;
                            p.h[(long long)(p.P + pair[j]) * p.F + f] = *(const uint16_t *)&lo;
                        }
                    }
                    if (most) {
                        turn ^= 1;
                        bar_sync(2 + half, kEpiThreads / 2);
                        // this warp's pair: its column's part of A2 h
                        const int j = quarter, k = min(col + j, x.n - 1), mine = col + j < x.n ? s.rank[k] : 0;
                        if (mine) {
                            const int f0 = x.m * kTile + lane * 4;
                            const float4 h4 = *(const float4 *)&sh[j][lane * 4];
                            const uint16_t *A = p.A[2] + (long long)s.slot[k] * p.a_ss[2] + (long long)x.e * p.a_es[2] + f0;
                            float *out = p.v2 + ((long long)s.list[x.at + k] * q.MT + x.m) * p.R;
                            for (int r0 = 0; r0 < mine; r0 += 8) {
                                float d[8];
#pragma unroll
                                for (int t = 0; t < 8; ++t) {
                                    uint2 w = make_uint2(0, 0);
                                    if (r0 + t < mine && f0 < p.F) w = __ldg((const uint2 *)(A + (long long)(r0 + t) * p.F));
                                    d[t] = bf16lo(w.x) * h4.x + bf16hi(w.x) * h4.y + bf16lo(w.y) * h4.z + bf16hi(w.y) * h4.w;
                                }
                                // eight sums over 32 lanes: halves of the values change lanes, so that 8 lanes end with one each
#pragma unroll
                                for (int t = 0; t < 4; ++t) {
                                    const float give = lane & 16 ? d[t] : d[t + 4], keep = lane & 16 ? d[t + 4] : d[t];
                                    d[t] = keep + __shfl_xor_sync(kAll, give, 16);
                                }
#pragma unroll
                                for (int t = 0; t < 2; ++t) {
                                    const float give = lane & 8 ? d[t] : d[t + 2], keep = lane & 8 ? d[t + 2] : d[t];
                                    d[t] = keep + __shfl_xor_sync(kAll, give, 8);
                                }
                                {
                                    const float give = lane & 4 ? d[0] : d[1], keep = lane & 4 ? d[1] : d[0];
                                    d[0] = keep + __shfl_xor_sync(kAll, give, 4);
                                }
                                d[0] += __shfl_xor_sync(kAll, d[0], 2);
                                d[0] += __shfl_xor_sync(kAll, d[0], 1);
                                const int rr = r0 + (lane & 16 ? 4 : 0) + (lane & 8 ? 2 : 0) + (lane & 4 ? 1 : 0);
                                if (!(lane & 3) && rr < mine) out[rr] = d[0];
                            }
                        }
                    }
                } else {
                    float(*sv)[LORA_MAX_RANK] = s.u.v2[half];
                    const int parts = (p.F + kTile - 1) / kTile;
                    if (p.L) {
                        bar_sync(2 + half, kEpiThreads / 2);  // the last four pairs' sums are no longer read
                        for (int j = 0; j < 4; ++j) {
                            const int k = min(col + j, x.n - 1), mine = col + j < x.n ? s.rank[k] : 0;
                            const float *in = p.v2 + (long long)s.list[x.at + k] * parts * p.R;
                            for (int rr = htid; rr < mine; rr += kEpiThreads / 2) {
                                float sum = 0.f;
                                for (int m = 0; m < parts; ++m) sum += __ldcg(in + (long long)m * p.R + rr);
                                sv[j][rr] = sum * s.scale[k];
                            }
                        }
                        bar_sync(2 + half, kEpiThreads / 2);
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int d = x.m * kRows + t * kTile + row;
                        if (d >= p.D) continue;
                        if (most) {
                            const uint16_t *b[4];
                            const float *vv[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int rs = (rank[j] + 7) & ~7;
                                b[j] = p.B[2] + (long long)slot[j] * p.b_ss[2] + ((long long)x.e * p.b_rows[2] + d) * rs;
                                vv[j] = sv[j];
                            }
                            expand_rows<4>(t ? v : g, b, vv, rank, most);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (col + j < x.n) __stcg(p.y + (long long)pair[j] * p.D + d, (t ? v[j] : g[j]) * s.weight[col + j]);
                    }
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.acce[buf]);
            if (!last) {
                __threadfence();
                bar_sync(1, kEpiThreads);
                if (tid == 0) {
                    __threadfence();
                    asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(flags + c), "r"(1) : "memory");
                }
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, Sh::kTmem);
}

// The pairs' results of a token in their order; the flags are left as they were found.
__global__ void __launch_bounds__(kThreads) combine_kernel(const LayerArgs p) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i < 2 * p.grid) p.flags[i] = 0;
    const int per = p.D / 8;
    if (i >= (long long)p.T * per) return;
    const int t = (int)(i / per), d = (int)(i % per) * 8;
    if (d == 0) slot_of(p, t, true);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < p.K; ++k) {
        const int pair = t * p.K + k;
        if (expert_of(p, pair, d == 0) < 0) continue;
        const float *y = p.y + (long long)pair * p.D + d;
        const float4 a = __ldcg((const float4 *)y), b = __ldcg((const float4 *)(y + 4));
        sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
        sum[4] += b.x, sum[5] += b.y, sum[6] += b.z, sum[7] += b.w;
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(sum[2 * j], sum[2 * j + 1]);
        o[j] = *(const uint32_t *)&b;
    }
    *(uint4 *)(p.out + t * p.ld_out + d) = make_uint4(o[0], o[1], o[2], o[3]);
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
    size_t flags, part, v13, h, v2, y, bytes;
};
Carve carve(const lora_moe_layer_desc_t &d, const lora_pool_t *pool, int64_t T, int sms) {
    const size_t P = (size_t)T * d.top_k, R = pool ? pool->desc.max_rank : 0;
    Carve c;
    c.flags = 0;
    c.part = c.flags + align256((size_t)2 * sms * 4);
    c.v13 = c.part + (size_t)sms * 2 * kGroup * kTile * 4;
    c.h = c.v13 + align256(P * 2 * R * 4);
    c.v2 = c.h + align256(2 * P * d.d_mlp * 2);
    c.y = c.v2 + align256(P * lora_ceil_div(d.d_mlp, kTile) * R * 4);
    c.bytes = c.y + align256(P * d.d_model * 4);
    return c;
}

struct Device {
    std::atomic<int> sms;  // 0: not looked up yet
};
Device g_devices[64];

// SM count of the current device; the kernels' attributes are set on the way.
cudaError_t device_sms(int &dev, int &sms) {
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    sms = g_devices[dev].sms.load(std::memory_order_acquire);
    if (sms) return cudaSuccess;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(stream_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)stream_smem<false>())) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(stream_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)stream_smem<true>())) !=
            cudaSuccess)
        return e;
    g_devices[dev].sms.store(sms, std::memory_order_release);
    return cudaSuccess;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) lora_note_launch();
    return e;
}

}  // namespace

extern "C" size_t lora_moe_layer_workspace_bytes(const lora_moe_layer_desc_t *desc, const lora_pool_t *pool,
                                                 int32_t max_tokens) {
    if (!desc || max_tokens < 0 || !desc_ok(*desc) || pool_ok(*desc, pool) != LORA_OK ||
        (int64_t)max_tokens * desc->top_k > LORA_MOE_LAYER_MAX_PAIRS)
        return 0;
    int dev = 0, sms = 0;
    const bool found = device_sms(dev, sms) == cudaSuccess;
    return carve(*desc, pool, max_tokens, found ? sms : kSms).bytes;
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
    int dev = 0, sms = 0;
    const cudaError_t found = device_sms(dev, sms);
    const Carve c = carve(d, pool, T, found == cudaSuccess ? sms : kSms);
    if (ws_bytes < c.bytes) return LORA_ERR_CAPACITY;
    LORA_CUDA_TRY(found);
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
    p.flags = (int *)(ws + c.flags);
    p.part = (float *)(ws + c.part);
    p.v13 = (float *)(ws + c.v13);
    p.h = (uint16_t *)(ws + c.h);
    p.v2 = (float *)(ws + c.v2);
    p.y = (float *)(ws + c.y);
    p.grid = sms;
    p.spin_limit = lora_spin_limit();
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
    StreamArgs up, down;
    memset(&up, 0, sizeof(up));
    memset(&down, 0, sizeof(down));
    up.KB = lora_ceil_div(d.d_model, kBK);
    up.MT = lora_ceil_div(d.d_mlp, kTile);
    down.KB = lora_ceil_div(d.d_mlp, kBK);
    down.MT = lora_ceil_div(d.d_model, kRows);
    if (!lora_make_tmap_3d(&up.tm_w, w13, d.d_model, d.d_mlp, 2LL * d.n_experts, ld_w13, (long long)d.d_mlp * ld_w13, kBK, kTile) ||
        !lora_make_tmap_2d(&up.tm_b, x, d.d_model, T, ldx, kBK, 1, true) ||
        !lora_make_tmap_3d(&down.tm_w, w2, d.d_mlp, d.d_model, d.n_experts, ld_w2, (long long)d.d_model * ld_w2, kBK, kTile) ||
        !lora_make_tmap_2d(&down.tm_b, p.h, d.d_mlp, 2LL * p.P, d.d_mlp, kBK, 1, true))
        return LORA_ERR_UNSUPPORTED;
    up.a = down.a = p;
    if (pool)
        LORA_CUDA_TRY(launch(shrink13_kernel, (unsigned)lora_ceil_div((int64_t)p.P * 2 * p.R, kThreads / 32), kThreads, 0, s, p));
    LORA_CUDA_TRY(launch(stream_kernel<false>, (unsigned)sms, kStreamThreads, stream_smem<false>(), s, up));
    LORA_CUDA_TRY(launch(stream_kernel<true>, (unsigned)sms, kStreamThreads, stream_smem<true>(), s, down));
    const int64_t pieces = (int64_t)T * (d.d_model / 8), most = pieces > 2 * sms ? pieces : 2 * sms;
    LORA_CUDA_TRY(launch(combine_kernel, (unsigned)lora_ceil_div(most, kThreads), kThreads, 0, s, p));
    return LORA_OK;
}
