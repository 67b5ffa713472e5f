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
//   shrink13   v[p] = scale A13 x        (with adapters; up's CTAs start as its CTAs leave)
//   up         g, u = W13 x + B13 v; h = act(g) u; parts of A2 h      per 128 columns of h
//   down       y[p] = w (W2 h + B2 (scale A2 h))                      per 256 rows of W2
//   combine    out[t] = sum of y over the token's pairs, in their order, one rounding
//
// Work is cut by bytes, not by tiles.  A unit is 256 weight rows (128 of gate and 128
// of up, or 256 of W2) for one group (an expert and up to 64 of its pairs), a block 64 columns of
// them (32 KB).  All units' blocks in a row are divided evenly among one CTA per SM (whole units where they are small),
// so a unit may be shared: its other CTAs leave fp32 sums in the workspace, and the one
// that has its last block adds them, lower columns first, and finishes the unit.  A CTA works from its
// last unit to its first, so what others wait for comes first, and only CTAs of
// lower index are waited for, which have started earlier.  Every CTA finds its groups from
// topk_ids by itself (a histogram and a scan in shared memory).
//
// Roles (352 threads): warp 0 issues the TMA copies, one lane the two weight boxes of a
// block, others the pairs' rows (x by token, four rows to a tile::gather4; h, which up leaves in the order
// of the groups, in boxes of eight); warp 1 issues the MMAs; warps 2-9 are the epilogue, a row per
// thread, two warps per quarter of the accumulator's lanes which take four of eight columns (pairs) each, under
// the next unit's MMAs (two accumulators); warp 10 says that a shared unit's sums are there (the
// fence behind stores takes some 5 us while the memory is busy, which the epilogue would wait out).
//
// The adapters' part of eight pairs is small (256 rows of B, some ranks) and goes by m16n8k16
// products in the epilogue's warps while a unit's weights are still on their way, for up to 32 pairs (down: 24): the rows of
// B, or of A2, come from global memory straight into registers, once per adapter among eight pairs, and of its product the columns
// of its own pairs are kept.
//
// Measured on one GB300 with 64 experts of 2048 x 1408, 8 a token (us; in brackets what their bytes take at the
// copy rate): 1 token 36.2 (20.4), 16 157 (144), 64 182 (163), 256 217 (163); with 8 adapters of rank 16 40.5 (20.7),
// 181 (149), 229 (178), 294 (188).  The weights go at 86% of the copy rate once they flow.  What is left are the
// kernels' starts (3 us each until products flow), shrink13, which keeps up off its SMs (4, 8, 14 and 25 us), and the last unit's
// epilogue, which no weights hide (1 to 8 us).
//
// Roundings: sums are fp32 throughout (accumulators, v, parts of A2 h, y), and h and v enter their products with all 24 bits: as
// the sum of three bf16, a number's leading, middle and last 8 bits.  The weights' bytes bound the kernel, not its MMAs.
#include <math.h>
#include <stddef.h>
#include <string.h>

#include <atomic>

#include "lora_internal.cuh"
#include "mma_common.cuh"
#include "tc_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxE = LORA_ROUTE_MAX_EXPERTS, kMaxP = LORA_MOE_LAYER_MAX_PAIRS;
constexpr int kGroup = 64;                    // most pairs of a group
constexpr int kRows = 256, kTile = 128;       // weight rows of a unit, of an MMA
constexpr int kBK = 64;                       // columns of a block: one 128-byte swizzle row
constexpr uint32_t kABytes = kRows * kBK * 2;
constexpr int kStreamThreads = 352, kEpi0 = 2, kEpiThreads = 256;
constexpr int kSms = 152;                     // where no device answers
constexpr int kLeast = 8;                     // fewest blocks of a unit worth a CTA of their own

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
    int R8;
    float *v13;                   // [P][2][R8], scaled (shared outer: by token), zeros past the adapter's rank
    uint16_t *h;                  // [3][P][F]: leading, middle and last bits, in the order of the groups
    float *v2;                    // [P][ceil(F / 128)][R8], parts of A2 h
    float *y;                     // [P][D], weighted
    float *part;                  // [CTA][2][kGroup][kTile] sums of shared units
    int *flags;                   // [2][CTA] part is there (up, down)
    int grid, spin_limit;
    int group;                    // pairs of a group (8, 16, 32 or 64)
    int single;                   // shrink13: a pair to a CTA
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

// A number is the sum of three bf16 without error: its leading 8 bits, the leading 8 of what they leave, and the last 8 (of 24
// bits; what is below bf16's smallest number is lost).  An infinite one or NaN is the first of them.
__device__ __forceinline__ float rest(float v) {
    return fabsf(v) < INFINITY ? v - __uint_as_float(__float_as_uint(v) & 0xffff0000u) : 0.f;
}
__device__ __forceinline__ uint16_t leading(float v) { return (uint16_t)(__float_as_uint(v) >> 16); }
__device__ __forceinline__ uint32_t leading(float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); }
__device__ __forceinline__ float4 rest(const float4 &v) { return make_float4(rest(v.x), rest(v.y), rest(v.z), rest(v.w)); }

// v = scale A13 x.  A CTA takes an expert (shared outer: the slots of one
// remainder by the number of CTAs), a slice and 16 ranks.  It finds the expert's pairs (the slots'
// tokens), sorts them by slot and reads an adapter's rows once for up to 8 of them: 16 ranks x 8
// pairs is one m16n8k16 product, whose operands come from global memory straight into registers
// (any order of k will do as long as both have the same), a warp per eighth of the columns.
// Several CTAs (gridDim.z) share an expert's batches of 8.  Bound by its chain of dependent reads (ids
// and slots, then rows; rank and scale come with the rows, which are zeros past a rank) and by
// the adapters' bytes (256 tokens of 8 adapters of rank 16: 67 MB in 20 us).
constexpr int kBatch = 8, kRanks = 16;
__global__ void __launch_bounds__(kThreads, 3) shrink13_kernel(const LayerArgs p, int chunks) {
    constexpr int kWarps = kThreads / 32, kAhead = 4;
    extern __shared__ uint32_t found[];  // slot << 12 | pair; behind them in order
    __shared__ float sums[2][kWarps][kRanks][kBatch];
    __shared__ int s_n;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int which = (int)blockIdx.y / chunks, r0 = (int)blockIdx.y % chunks * kRanks;
    if (tid == 0) s_n = 0;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int count = p.shared ? p.T : p.P, sets = gridDim.x, me = blockIdx.x;
    uint32_t *key = found + count;
    // few pairs: a CTA takes one, whoever else has its adapter
    const bool single = !p.shared && gridDim.z == 1 && sets == p.P && p.single;
    int e_me = me;
    if (single) {
        const int e = p.ids[me], a = p.idx[me / p.K];
        if (e < 0 || e >= p.E || a < 0 || a >= p.L) return;
        e_me = e;
        if (tid == 0) key[0] = (uint32_t)a << 12 | (uint32_t)me, s_n = 1;
    }
    for (int i0 = single ? count : tid; i0 < count; i0 += kAhead * kThreads) {
        int e[kAhead], a[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            e[j] = i >= count ? -1 : p.shared ? me : p.ids[i];
            a[j] = i >= count ? -1 : p.idx[p.shared ? i : i / p.K];
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (e[j] == me && a[j] >= 0 && a[j] < p.L && (!p.shared || a[j] % sets == me))
                found[atomicAdd(&s_n, 1)] = (uint32_t)a[j] << 12 | (uint32_t)(i0 + j * kThreads);
    }
    __syncthreads();
    const int n = s_n;
    // in order, whatever order they were found in; those of slots without an adapter go unused
    for (int i = tid; i < n && !single; i += kThreads) {
        const uint32_t mine = found[i];
        int before = 0;
        for (int j = 0; j < n; ++j) before += found[j] < mine;
        key[before] = mine;
    }
    __syncthreads();
    const int m = p.n13 == 2 ? which : 0;
    const int g = lane >> 2, c0 = (lane & 3) * 8;  // row of the fragments, first of this lane's 8 columns of 32
    for (int at = 0, b = 0, turn = 0; at < n; ++b) {
        const int slot = (int)(key[at] >> 12);
        int few = 1;
        while (few < kBatch && at + few < n && (int)(key[at + few] >> 12) == slot) ++few;
        const int first = at;
        at += few;
        if (b % (int)gridDim.z != (int)blockIdx.z) continue;
        const int rank = p.rank[slot];
        const float scale = p.scale[slot];
        const uint16_t *A = p.A[m] + (long long)slot * p.a_ss[m] + (p.shared ? 0 : (long long)e_me * p.a_es[m]);
        const int i = (int)(key[first + min(g, few - 1)] & 0xfffu);
        const uint16_t *x = p.x + (long long)(p.shared ? i : i / p.K) * p.ldx + c0;
        const uint16_t *row0 = A + (long long)min(r0 + g, p.R - 1) * p.D + c0, *row1 = A + (long long)min(r0 + g + 8, p.R - 1) * p.D + c0;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = warp * 32; c < p.D; c += kAhead * kWarps * 32) {
            uint4 a0[kAhead], a1[kAhead], v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int k = c + j * kWarps * 32;
                a0[j] = a1[j] = v[j] = make_uint4(0, 0, 0, 0);
                if (k + c0 < p.D) {
                    a0[j] = ldg_stream(row0 + k);
                    a1[j] = ldg_stream(row1 + k);
                    v[j] = __ldg((const uint4 *)(x + k));
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                bgmv::mma16816(d, a0[j].x, a1[j].x, a0[j].y, a1[j].y, v[j].x, v[j].y);
                bgmv::mma16816(d, a0[j].z, a1[j].z, a0[j].w, a1[j].w, v[j].z, v[j].w);
            }
        }
        float(*sum)[kRanks][kBatch] = sums[turn];
        turn ^= 1;
        sum[warp][g][(lane & 3) * 2] = d[0];
        sum[warp][g][(lane & 3) * 2 + 1] = d[1];
        sum[warp][g + 8][(lane & 3) * 2] = d[2];
        sum[warp][g + 8][(lane & 3) * 2 + 1] = d[3];
        __syncthreads();
        const int r = r0 + (tid & 15), j = tid >> 4;
        if (j < few && r < p.R8) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += sum[w][tid & 15][j];
            // ranks past the adapter's meet zeros: finite, whatever x is
            p.v13[((long long)(key[first + j] & 0xfffu) * 2 + which) * p.R8 + r] = r < rank ? v * scale : 0.f;
        }
    }
}

__device__ __forceinline__ float activation(float g, int gelu) {
    if (gelu) return 0.5f * g * (1.f + tanhf(0.7978845608f * (g + 0.044715f * g * g * g)));
    return g / (1.f + expf(-g));
}

// ------------------------------------------------------------ streamed products

struct StreamArgs {
    CUtensorMap tm_w, tm_b;  // weights, the pairs' rows (x or h)
    LayerArgs a;
    int KB, MT;  // blocks of a unit, units of a group
};

template <bool DOWN>
struct Shape {
    static constexpr int kCols = DOWN ? 2 * kGroup : kGroup;  // accumulator columns of a tile
    static constexpr int kParts = DOWN ? 3 : 1;  // rows of a pair in a block
    static constexpr uint32_t kStage = kABytes + kParts * kGroup * 128;
    // (2 and 3 stages: 16 tokens without adapters 176 and 156 us, 256 with adapters 294 and 293, 91 pairs over 51 experts of 672 x 568
    // 32 and 29, 904 over 18 of 432 x 760 57 and 60; there is no room for 4)
    static constexpr int kStages = 3;
    static constexpr int kTmem = 4 * kCols;  // two tiles, two buffers
};

constexpr int kBatchCols = 8;                // columns that the epilogue takes at a time
constexpr int kDPitch = kRows + 4;           // of the adapters' part of a column: no two of a product's lanes on one bank
// ... whose adapters' part is there at once.  Down has room for fewer beside v of all 64 pairs of rank 64, which stays from unit to unit.
template <bool DOWN>
constexpr int kLotCols = DOWN ? 24 : 32;
constexpr int kVFloats = 4096;
static_assert(kVFloats / (2 * LORA_MAX_RANK) >= kBatchCols, "v of eight pairs");
constexpr int kHPitch = kTile + 4;           // of a column of h: no two of 8 lanes' 16 bytes on one bank

template <bool DOWN, bool ADAPT>
struct SharedOf {
    uint64_t full[3], empty[3], accf[2], acce[2];
    uint32_t tmem;
    int abort;
    uint16_t groups[kMaxE + 8], pairs[kMaxE + 8];  // groups and pairs of the experts before this one
    uint16_t list[kMaxP];                          // pairs of this CTA's experts, by expert
    // of the pairs of a group, and of the next one
    struct Pairs {
        unsigned long long starts;       // columns where another adapter begins
        int slot[kGroup], rank[kGroup];  // adapter (-1: none) and its rank
        float weight[kGroup];
    } of[2];
    alignas(16) union {
        struct {
            int count[kMaxE];
            uint16_t ids[kMaxP], at[kMaxP], slots[ADAPT ? kMaxP : 1];  // of a pair: expert, place among the expert's as counted
            uint32_t key[kMaxP];                                       // slot << 12 | pair, by expert
        } g;  // while groups are found
        struct {
            float delta[ADAPT ? kLotCols<DOWN> : 1][kDPitch];  // the adapters' part of a lot of columns
            float v[ADAPT ? kVFloats : 1];     // scale A x or scale A2 h of some pairs
            alignas(16) float h[ADAPT && !DOWN ? kGroup : 1][kHPitch];  // the unit's columns of h
        } e;  // epilogue
    } u;
};
static_assert(kDPitch % 4 == 0 && kHPitch % 4 == 0, "read 16 bytes at a time");

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
// Columns that a group's pairs have in an accumulator, and rows in a block.  Down: leading, middle and last bits follow each other, all
// three in one product; above 32 pairs two in one, and the last ones are added to the middle ones' columns by another (each product's
// operands are read anew, and three a block made 3 tokens of 512 x 256 1.1 us slower).
constexpr int kFew = 32;
template <bool DOWN>
__device__ __forceinline__ int columns_of(int pairs) {
    return DOWN && pairs > kFew ? kGroup : (pairs + 15) & ~15;
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

// A box of weights, which nobody reads again: L2 is to give their lines up first, and to keep
// what is read often (instructions above all: a fetch from DRAM takes microseconds behind the weights).
__device__ __forceinline__ uint64_t evict_first() {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void tma_weights(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], "
        "[%5], %6;" ::"r"(tc::smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
                 : "r"(taddr)
                 : "memory");
}

template <class Shared>
__device__ __forceinline__ void note_timeout(const LayerArgs &p, Shared &s) {
    *(volatile int *)&s.abort = 1;
    if (p.status) atomicExch(p.status, (int)LORA_ERR_TIMEOUT);
}
// Waits for a phase of a barrier; false once any wait of the CTA has given up.
template <class Shared>
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
template <class Shared>
__device__ int find_groups(const LayerArgs &p, Shared &s) {
#pragma unroll 1
    for (int i = threadIdx.x; i < p.E; i += kStreamThreads) s.u.g.count[i] = 0;
    __syncthreads();
    constexpr int kIds = 4;
    constexpr bool kSlots = sizeof(s.u.g.slots) > 2;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < p.P; i0 += kIds * kStreamThreads) {
        int e[kIds], a[kIds];
#pragma unroll
        for (int j = 0; j < kIds; ++j) {
            const int i = i0 + j * kStreamThreads;
            e[j] = i < p.P ? p.ids[i] : -1;
            a[j] = kSlots && i < p.P ? p.idx[i / p.K] : -1;
        }
#pragma unroll
        for (int j = 0; j < kIds; ++j) {
            const int i = i0 + j * kStreamThreads;
            if (i >= p.P) break;
            const bool ok = e[j] >= 0 && e[j] < p.E;
            s.u.g.ids[i] = ok ? (uint16_t)e[j] : 0xffffu;
            if (kSlots) s.u.g.slots[i] = (uint16_t)min((unsigned)a[j], 0xffffu);
            if (ok) s.u.g.at[i] = (uint16_t)atomicAdd(&s.u.g.count[e[j]], 1);
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int groups = 0, pairs = 0;
#pragma unroll 1
        for (int e0 = 0; e0 <= p.E; e0 += 32) {
            const int c = e0 + lane < p.E ? s.u.g.count[e0 + lane] : 0, n = (c + p.group - 1) / p.group;
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
template <class Shared>
__device__ __forceinline__ int expert_of_group(const LayerArgs &p, const Shared &s, int g) {
    int lo = 0, hi = p.E;  // groups[lo] <= g < groups[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.groups[mid] <= g) lo = mid;
        else hi = mid;
    }
    return lo;
}
// The pairs of experts e0..e1, an expert's by slot (with adapters) and in their order: the same in every CTA, whatever
// the order in which they were counted.  A pair is compared with all others of its expert, here and in shrink13, which hides behind
// the weights up to some 500 of them and not above (D = F = 64, 4096 pairs without and with adapters: for one expert 1103 and 1751 us,
// evenly for 64 of them 29 and 68; 512 pairs with adapters 58 and 25).
template <class Shared>
__device__ void list_pairs(const LayerArgs &p, Shared &s, int e0, int e1) {
    const int base = s.pairs[e0];
#pragma unroll 1
    for (int i = threadIdx.x; i < p.P; i += kStreamThreads) {
        const int e = s.u.g.ids[i];
        if (e < e0 || e > e1) continue;
        const uint32_t slot = sizeof(s.u.g.slots) > 2 ? s.u.g.slots[i] : 0u;
        s.u.g.key[s.pairs[e] - base + s.u.g.at[i]] = slot << 12 | (uint32_t)i;
    }
    __syncthreads();
    const int n = s.pairs[e1 + 1] - base;
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += kStreamThreads) {
        const uint32_t mine = s.u.g.key[i];
        const int e = s.u.g.ids[mine & 0xfffu], first = s.pairs[e] - base, end = s.pairs[e + 1] - base;
        int place = first;
#pragma unroll 4
        for (int j = first; j < end; ++j) place += s.u.g.key[j] < mine;
        s.list[place] = (uint16_t)(mine & 0xfffu);
    }
}

// What a CTA does: blocks [b0, b1) of all the units' blocks in a row.  A unit of less than 2 kLeast blocks is not cut, and of
// others a CTA gets kLeast blocks at least, and all CTAs with any equal parts (160 pairs over 49 experts of
// 136 x 128 23 us, 34 where units of 2 and 3 blocks are cut; kLeast of 4, 6, 8 and 10: 37 tokens of three over 6 of 1040 x 272 29.2, 27.3,
// 27.3 and 28.7, 904 pairs over 18 of 432 x 760 68, 68, 60 and 60).
struct Range {
    int b0, b1, grains, grain, n;  // n CTAs share them, in grains of a block or a unit
    // grains * c / n, whose parts stay below 2^31
    __device__ __forceinline__ int start(int c) const {
        return grain * (grains / n * c + (int)((unsigned)(grains % n * c) / (unsigned)n));
    }
};

// The CTA's part of unit u, and what the unit is.
struct Part {
    int k0, k1;        // blocks of the unit
    int e, m, n, at;   // expert, place in it, pairs, first of them in the list
    int pos;           // ... and in the order of the groups
};
template <class Shared>
__device__ __forceinline__ Part part_of(const StreamArgs &q, const Shared &s, const Range &r, int u, int e_first) {
    Part x;
    x.k0 = max(r.b0 - u * q.KB, 0);
    x.k1 = min(r.b1 - u * q.KB, q.KB);
    const int g = u / q.MT;
    x.m = u - g * q.MT;
    x.e = expert_of_group(q.a, s, g);
    const int first = s.pairs[x.e] + (g - s.groups[x.e]) * q.a.group;
    x.n = min(q.a.group, s.pairs[x.e + 1] - first);
    x.pos = first;
    x.at = first - s.pairs[e_first];
    return x;
}

// What the epilogue does for adapters; all of its threads call these together.  The code is kept
// small and in one place each, here and in the roles (loops stay rolled: 37 tokens over 6 experts 32.2 -> 30.5 us): what
// a unit runs once comes from L2 instruction by instruction.
template <bool DOWN, bool ADAPT>
struct Epilogue {
    typedef SharedOf<DOWN, ADAPT> Shared;
    typedef typename Shared::Pairs Pairs;
    const LayerArgs &p;
    Shared &s;
    const int tid, warp, lane, g, t4;  // g, t4: row and column of a product's fragments
    const int per, lot;                // floats of v of a pair, pairs of them at a time

    __device__ __forceinline__ Epilogue(const LayerArgs &p, Shared &s, int tid)
        : p(p), s(s), tid(tid), warp(tid >> 5), lane(tid & 31), g((tid & 31) >> 2), t4(tid & 3),
          per(ADAPT ? p.R8 * (DOWN ? 1 : p.n13) : 1), lot(kVFloats / per & ~(kBatchCols - 1)) {}

    // The weights and adapters of a group's pairs.  A barrier has to follow.
    __device__ __forceinline__ void note(const Part &x, Pairs &o) {
        if (warp >= 2) return;
        int slot = -1;
        if (tid < x.n) {
            const int pair = s.list[x.at + tid];
            if (DOWN) o.weight[tid] = p.topk_w ? p.topk_w[pair] : 1.f;
            if (ADAPT) slot = slot_of(p, pair / p.K, false);
        }
        if (!ADAPT) return;
        o.slot[tid] = slot;
        o.rank[tid] = slot >= 0 ? p.rank[slot] : 0;
        int left = __shfl_up_sync(kAll, slot, 1);
        if (lane == 0) left = -1;  // an adapter that goes on past column 32 begins there again
        const unsigned starts = __ballot_sync(kAll, slot >= 0 && slot != left);
        if (lane == 0) ((unsigned *)&o.starts)[warp] = starts;
    }

    // v of a lot of a group's pairs, to shared memory: scale A x as shrink13 left it (up), or scale A2 h, the sum of
    // its parts, of which four lanes take one each in turn (down).  A barrier has to follow.
    __device__ __forceinline__ void fill(const Part &x, const Pairs &o, int b0) {
        const int n = min(lot, x.n - b0);
        if (DOWN) {
            const int parts = (p.F + kTile - 1) / kTile;
            const unsigned quad = 0xfu << (lane & 28);
#pragma unroll 1
            for (int i = tid >> 2; i < n * per; i += kEpiThreads / 4) {
                const int k = b0 + i / per, r = i - (k - b0) * per;
                float sum = 0.f;
                if (r < o.rank[k]) {
                    const float *in = p.v2 + (long long)s.list[x.at + k] * parts * per + r;
#pragma unroll 4
                    for (int m = t4; m < parts; m += 4) sum += __ldcg(in + (long long)m * per);
                    sum *= p.scale[o.slot[k]];
                }
                sum += __shfl_xor_sync(quad, sum, 1);
                sum += __shfl_xor_sync(quad, sum, 2);
                if (t4 == 0) s.u.e.v[i] = sum;
            }
        } else {
#pragma unroll 1
            for (int i = tid * 4; i < n * per; i += kEpiThreads * 4) {
                const int k = b0 + i / per, r = i - (k - b0) * per, pair = s.list[x.at + k];
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (o.slot[k] >= 0) f = __ldcg((const float4 *)(p.v13 + (long long)(p.shared ? pair / p.K : pair) * 2 * p.R8 + r));
                *(float4 *)&s.u.e.v[i] = f;
            }
        }
    }

    // Rows of B for 16 ranks of an adapter, four such at a time, in the order of eight columns' adapters.
    struct Rows {
        uint2 w[4][4];
        int run[4], r0[4];
        int left, r;  // adapters to come (the first of them from rank r on)
    };
    __device__ __forceinline__ int runs(const Pairs &o, int b0) const {  // columns of eight where an adapter begins or goes on
        return ((int)(o.starts >> b0) & 0xff) | (o.slot[b0] >= 0 ? 1 : 0);
    }
    __device__ __forceinline__ int tile() const { return DOWN ? 0 : warp >> 2; }
    __device__ __forceinline__ void ask(Rows &q, const Part &x, const Pairs &o, int b0) {
        const int which = DOWN ? 2 : tile() ? p.n13 - 1 : 0, rows = DOWN ? p.D : p.F;
        const int row0 = x.m * (DOWN ? kRows : kTile) + (DOWN ? warp : warp & 3) * 32 + g;
        const long long brow = (long long)x.e * p.b_rows[which] + (tile() ? p.b_up : 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            q.run[k] = -1;
            q.r0[k] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) q.w[k][j] = make_uint2(0, 0);
            if (!q.left) continue;
            const int run = __ffs(q.left) - 1, rank = o.rank[b0 + run], rs = (rank + 7) & ~7, r = q.r + t4 * 4;
            const uint16_t *b = p.B[which] + (long long)o.slot[b0 + run] * p.b_ss[which] + brow * rs + r;
            q.run[k] = run;
            q.r0[k] = q.r;
            if (r < rs)
#pragma unroll
                for (int j = 0; j < 4; ++j) q.w[k][j] = __ldg((const uint2 *)(b + (long long)min(row0 + j * 8, rows - 1) * rs));
            q.r += 16;
            if (q.r >= rank) {
                q.r = 0;
                q.left &= q.left - 1;
            }
        }
    }
    // B v of eight columns from b0 on for the unit's 256 rows, to s.u.e.delta: a warp takes 32 rows.  The
    // first rows of B may have been asked for.  A barrier has to follow.
    __device__ __forceinline__ void rows(Rows &q, bool asked, const Part &x, const Pairs &o, int b0) {
        float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int all = runs(o, b0);
        int run[2];  // of the columns whose results this lane has
#pragma unroll
        for (int j = 0; j < 2; ++j)
            run[j] = o.slot[b0 + t4 * 2 + j] >= 0 ? 31 - __clz(all & ((2 << (t4 * 2 + j)) - 1)) : -2;
        const float *v = s.u.e.v + (b0 + g) % lot * per + (p.n13 == 2 && tile() ? p.R8 : 0) + t4 * 4;
        if (!asked) q.left = all, q.r = 0;
#pragma unroll 1
        for (;;) {
            if (!asked) ask(q, x, o, b0);
            asked = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (q.run[k] < 0) break;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (q.r0[k] + t4 * 4 < p.R8) f = *(const float4 *)(v + q.r0[k]);
                float e[2][4];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i >> 2][i & 3] = d[i >> 2][i & 3];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint32_t b0 = leading(f.x, f.y), b1 = leading(f.z, f.w);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        bgmv::mma16816(e[j], q.w[k][2 * j].x, q.w[k][2 * j + 1].x, q.w[k][2 * j].y, q.w[k][2 * j + 1].y, b0, b1);
                    f = rest(f);
                }
                // other adapters' columns keep what they have: a weight that is not finite is NaN even in a product with 0
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (q.run[k] == run[i & 1]) d[i >> 2][i & 3] = e[i >> 2][i & 3];
            }
            if (!q.left) break;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) s.u.e.delta[b0 % kLotCols<DOWN> + t4 * 2 + (k & 1)][warp * 32 + j * 16 + g + (k >> 1) * 8] = d[j][k];
    }

    // 16 ranks of an adapter's A2, this unit's columns of them: what a warp multiplies with h at a time (up).
    struct Task {
        uint4 w[4][2];
        unsigned long long left;  // adapters from the task's on
        int r0, rank, skip;       // skip: tasks from this one to the next of the warp
    };
    __device__ __forceinline__ bool next_task(Task &q, const Part &x, const Pairs &o) {
#pragma unroll 1
        for (; q.left; q.left &= q.left - 1, q.r0 = 0) {
            q.rank = o.rank[__ffsll(q.left) - 1];
            const int tiles = (q.rank - q.r0 + 15) / 16;
            if (q.skip < tiles) break;
            q.skip -= tiles;
        }
        if (!q.left) return false;
        q.r0 += q.skip * 16;
        q.skip = kEpiThreads / 32;
        const int f0 = x.m * kTile + t4 * 8;
        const uint16_t *A = p.A[2] + (long long)o.slot[__ffsll(q.left) - 1] * p.a_ss[2] + (long long)x.e * p.a_es[2] + f0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                q.w[j][k] = f0 + j * 32 < p.F ? __ldg((const uint4 *)(A + (long long)min(q.r0 + k * 8 + g, q.rank - 1) * p.F + j * 32))
                                              : make_uint4(0, 0, 0, 0);
        return true;
    }
    __device__ __forceinline__ void run_task(const Task &q, const Part &x, const Pairs &o, int parts) {
        const int run = __ffsll(q.left) - 1, slot = o.slot[run];
        const unsigned long long next = q.left & (q.left - 1);
        int end = next ? __ffsll(next) - 1 : x.n;
        while (o.slot[end - 1] != slot) --end;  // pairs without an adapter come behind it
#pragma unroll 1
        for (int c = run; c < end; c += 8) {
            float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // of the leading bits, of the rest
            const float *h = &s.u.e.h[min(c + g, kGroup - 1)][t4 * 8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 f0 = *(const float4 *)(h + j * 32), f1 = *(const float4 *)(h + j * 32 + 4);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    bgmv::mma16816(d[i > 0], q.w[j][0].x, q.w[j][1].x, q.w[j][0].y, q.w[j][1].y, leading(f0.x, f0.y), leading(f0.z, f0.w));
                    bgmv::mma16816(d[i > 0], q.w[j][0].z, q.w[j][1].z, q.w[j][0].w, q.w[j][1].w, leading(f1.x, f1.y), leading(f1.z, f1.w));
                    f0 = rest(f0);
                    f1 = rest(f1);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = c + t4 * 2 + (k & 1), r = q.r0 + g + (k >> 1) * 8;
                if (at < end && r < q.rank) p.v2[((long long)s.list[x.at + at] * parts + x.m) * p.R8 + r] = d[0][k] + d[1][k];
            }
        }
    }
};

template <bool DOWN, bool ADAPT>
constexpr size_t stream_smem() {
    return 1024 + (size_t)Shape<DOWN>::kStages * Shape<DOWN>::kStage + sizeof(SharedOf<DOWN, ADAPT>);
}
static_assert(stream_smem<false, true>() <= 227 * 1024 && stream_smem<true, true>() <= 227 * 1024, "shared memory of a CTA");

// (168 registers a thread are what 352 threads can have; up with adapters spills one)
template <bool DOWN, bool ADAPT>
__global__ void __launch_bounds__(kStreamThreads, 1) stream_kernel(const __grid_constant__ StreamArgs q) {
    typedef Shape<DOWN> Sh;
    typedef SharedOf<DOWN, ADAPT> Shared;
    extern __shared__ __align__(1024) char smem_raw[];
    char *ring = smem_raw + ((1024u - (smem_u32_of(smem_raw) & 1023u)) & 1023u);
    Shared &s = *(Shared *)(ring + (size_t)Sh::kStages * Sh::kStage);
    const LayerArgs &p = q.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Without adapters the kernel before up is the caller's, which may have written
    // topk_ids; shrink13, and up before down, let this one start when those are complete.
    if (!DOWN && !ADAPT) asm volatile("griddepcontrol.wait;" ::: "memory");
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
    const int units = find_groups(p, s) * q.MT, parts = max(1, q.KB / kLeast);
    r.grain = parts == 1 ? q.KB : 1;
    r.grains = parts == 1 ? units : units * q.KB;
    r.n = max(1, min((int)gridDim.x, units * parts));
    const int c = blockIdx.x;
    const bool any = c < r.n && units > 0;
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
        // the kernel before this one is complete, the pairs' rows after it.
        const uint64_t policy = evict_first();
        const auto weights = [&](const Part &x, int k, int st) {
            char *dst = ring + (size_t)st * Sh::kStage;
            if (DOWN) {
                const bool two = x.m * kRows + kTile < p.D;  // rows of the second tile that are there at all
                tc::mbar_expect_tx(&s.full[st], (two ? kABytes : kABytes / 2) + (uint32_t)((x.n + 7) & ~7) * 128 * Sh::kParts);
                tma_weights(dst, &q.tm_w, k * kBK, x.m * kRows, x.e, &s.full[st], policy);
                if (two) tma_weights(dst + kABytes / 2, &q.tm_w, k * kBK, x.m * kRows + kTile, x.e, &s.full[st], policy);
            } else {
                tc::mbar_expect_tx(&s.full[st], kABytes + (uint32_t)((x.n + 3) & ~3) * 128);
                tma_weights(dst, &q.tm_w, k * kBK, x.m * kTile, 2 * x.e, &s.full[st], policy);
                tma_weights(dst + kABytes / 2, &q.tm_w, k * kBK, x.m * kTile, 2 * x.e + 1, &s.full[st], policy);
            }
        };
        int done = 0, ahead = 0;  // blocks asked for; of the first ones the weights alone
        if (lane == 0) {
            tc::prefetch_tmap(&q.tm_w);
            tc::prefetch_tmap(&q.tm_b);
#pragma unroll 1
            for (int u = u_hi; u >= u_lo && ahead < Sh::kStages; --u) {
                const Part x = part_of(q, s, r, u, e_first);
#pragma unroll 1
                for (int k = x.k0; k < x.k1 && ahead < Sh::kStages; ++k) weights(x, k, ahead++);
            }
        }
        ahead = __shfl_sync(kAll, ahead, 0);
        if (DOWN) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            asm volatile("fence.proxy.async.global;" ::: "memory");
        }
        bool ok = true;
#pragma unroll 1
        for (int u = u_hi; u >= u_lo && ok; --u) {
            const Part x = part_of(q, s, r, u, e_first);
            // this lane's rows: four of x by token, or eight of h (leading bits, in lanes 8-15 middle ones, then the last)
            const bool mine = DOWN ? lane < 8 * Sh::kParts && (lane & 7) * 8 < x.n : lane * 4 < x.n;
            const uint32_t off =
                kABytes + (uint32_t)(DOWN ? (lane & 7) * 8 + (lane >> 3) * columns_of<DOWN>(x.n) : lane * 4) * 128;
            const int row = x.pos + (lane & 7) * 8 + (lane >> 3) * p.P;
            int4 rows = make_int4(0, 0, 0, 0);
            if (!DOWN && mine) {
                const auto token = [&](int i) { return s.list[x.at + min(lane * 4 + i, x.n - 1)] / p.K; };
                rows = make_int4(token(0), token(1), token(2), token(3));
            }
#pragma unroll 1
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
                char *dst = ring + (size_t)st * Sh::kStage + off;
                if (mine) {
                    if (DOWN) tc::tma_load_2d(dst, &q.tm_b, k * kBK, row, &s.full[st]);
                    else tma_gather4(tc::smem_u32(dst), &q.tm_b, k * kBK, rows, &s.full[st]);
                }
                ++done;
            }
        }
        if (!DOWN) asm volatile("griddepcontrol.wait;" ::: "memory");
        // every copy has landed before the CTA ends (given up or not: all that was asked for comes)
        if (lane == 0)
#pragma unroll 1
            for (int i = max(0, done - Sh::kStages); i < done; ++i)
                land(&s.full[i % Sh::kStages], (uint32_t)((i / Sh::kStages) & 1));
    } else if (warp == 1) {
        // ---- products
        int done = 0, i = 0;
        bool ok = true;
#pragma unroll 1
        for (int u = u_hi; u >= u_lo && ok; --u, ++i) {
            const Part x = part_of(q, s, r, u, e_first);
            const int buf = i & 1;
            const bool two = !DOWN || x.m * kRows + kTile < p.D;
            const int cols = columns_of<DOWN>(x.n);
            const bool few = x.n <= kFew;
            const uint32_t idesc = tc::idesc_bf16(kTile, cols * (DOWN ? few ? 3 : 2 : 1)), idesc_last = tc::idesc_bf16(kTile, kGroup);
            if (i >= 2) ok = __all_sync(kAll, wait(&s.acce[buf], (uint32_t)(((i >> 1) - 1) & 1), p, s));
            tc::tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(buf * 2 * Sh::kCols);
#pragma unroll 1
            for (int k = x.k0; k < x.k1 && ok; ++k) {
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
                        if (DOWN && !few) {
                            const uint32_t last = b + (uint32_t)(2 * kGroup * 128 >> 4) + j * 2;
                            mma_ss(d + kGroup, a0 + j * 2, last, idesc_last, true);
                            if (two) mma_ss(d + Sh::kCols + kGroup, a1 + j * 2, last, idesc_last, true);
                        }
                    }
                    tc::mma_commit(&s.empty[st]);
                    if (k == x.k1 - 1) tc::mma_commit(&s.accf[buf]);
                }
                ++done;
            }
        }
        // products in flight read the ring and write tensor memory: the next stage's barrier tells their end
        if (done > 0 && lane == 0) {
            const int last = done - 1;
            land(&s.empty[last % Sh::kStages], (uint32_t)((last / Sh::kStages) & 1));
        }
        __syncwarp();
    } else if (warp < kEpi0 + kEpiThreads / 32) {
        // ---- epilogue
        const int tid = threadIdx.x - kEpi0 * 32;
        const int quarter = warp & 3, half = (warp - kEpi0) >> 2, row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        float *const my_part = p.part + (size_t)c * 2 * kGroup * kTile;
        int *const flags = p.flags + (DOWN ? p.grid : 0);
        typedef Epilogue<DOWN, ADAPT> Epi;
        Epi epi(p, s, tid);
        typename Epi::Rows rows;
        typename Epi::Task task;
        bool asked = false, waited = false;
        int now = 0, noted = -1, filled = -1;  // of[now] is of this unit's group; `noted` is noted, `filled` the lot of v that is there
        int i = 0;
        Part x = part_of(q, s, r, any ? u_hi : 0, e_first);
        if ((DOWN || ADAPT) && any && x.k1 == q.KB) {
            epi.note(x, s.of[0]);
            noted = u_hi / q.MT;
            bar_sync(1, kEpiThreads);
        }
        if (!ADAPT) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 1
        for (int u = u_hi; u >= u_lo; --u, ++i) {
            const int buf = i & 1;
            const bool last = x.k1 == q.KB, more = u > u_lo;
            const uint32_t acc = tmem + lanes + (uint32_t)(buf * 2 * Sh::kCols);
            const Part y = part_of(q, s, r, more ? u - 1 : u, e_first);  // the next unit
            int next = now;
            if (DOWN || ADAPT) {
                bar_sync(1, kEpiThreads);  // nothing of the last unit is read any more
                if (more && (u - 1) / q.MT != noted) {
                    next ^= 1;
                    noted = (u - 1) / q.MT;
                    epi.note(y, s.of[next]);
                }
            }
            const typename Shared::Pairs &of = s.of[now];
            bool any_delta = false, ok = true;
            int from = c;
            unsigned with = 0;  // batches of the lot that have an adapter's part
#pragma unroll 1
            for (int b0 = 0; b0 < x.n; b0 += kBatchCols) {
                if (ADAPT && b0 % kLotCols<DOWN> == 0) {
                    // the adapters' part of a lot of columns, before their products are there
                    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
                    waited = true;
                    const int to = min(x.n, b0 + kLotCols<DOWN>);
                    with = 0;
                    if (last)
#pragma unroll 1
                        for (int b = b0; b < to; b += kBatchCols) {
                            if (!epi.runs(of, b)) continue;
                            with |= 1u << (b - b0) / kBatchCols;
                            const int lot = (u / q.MT) * kGroup + b / epi.lot;
                            if (lot != filled) {
                                if (b > 0) bar_sync(1, kEpiThreads);  // v is no longer read
                                epi.fill(x, of, b / epi.lot * epi.lot);
                                bar_sync(1, kEpiThreads);
                            }
                            filled = lot;
                            epi.rows(rows, asked, x, of, b);
                            asked = false;
                        }
                    any_delta |= with != 0;
                    bar_sync(1, kEpiThreads);
                    // rows of B of the columns after these, and rows of A2, are on their way while these are worked on
                    const bool end = to == x.n;
                    const Part &z = end ? y : x;
                    const typename Shared::Pairs &oz = end ? s.of[next] : of;
                    const int bz = end ? 0 : to;
                    if (end ? more : last) {
                        rows.left = epi.runs(oz, bz);
                        rows.r = 0;
                        asked = rows.left != 0;
                        if (asked) epi.ask(rows, z, oz, bz);
                    }
                    if (!DOWN && end && any_delta) {
                        task.left = of.starts;
                        task.r0 = 0;
                        task.skip = tid >> 5;
                        epi.next_task(task, x, of);
                    }
                }
                const bool delta = with >> b0 % kLotCols<DOWN> / kBatchCols & 1;
                const int col = b0 + half * 4;
                if (b0 == 0 && last && x.k0 > 0) {
                    // Sums that other CTAs have left of this unit, while its products are still to come.
                    // The CTA that has the unit's first block: start(f) <= u KB < start(f + 1)
                    from = max(0, c - (int)((unsigned)x.k0 * (unsigned)r.n / (unsigned)r.grains) - 1);
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
                    ok = bar_and(1, kEpiThreads, ok);
                }
                float pg[4] = {0.f, 0.f, 0.f, 0.f}, pv[4] = {0.f, 0.f, 0.f, 0.f};
                if (col < x.n && ok)
#pragma unroll 1
                    for (int f = from; f < c; ++f) {
                        const float *o = p.part + (size_t)f * 2 * kGroup * kTile;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            pg[j] += __ldcg(o + (size_t)(col + j) * kTile + row);
                            pv[j] += __ldcg(o + (size_t)(kGroup + col + j) * kTile + row);
                        }
                    }
                if (b0 == 0) {
                    ok = ok && wait(&s.accf[buf], (uint32_t)((i >> 1) & 1), p, s);
                    // one wait that gave up ends the work of all
                    ok = bar_and(1, kEpiThreads, ok);
                    if (!ok) break;
                    tc::tc_fence_after();
                }
                if (col < x.n) {
                    float g[4], v[4];  // gate and up; or the two tiles' rows
                    tmem_ld4(acc + col, g);
                    tmem_ld4(acc + Sh::kCols + col, v);
                    if (DOWN) {
                        const int cols = columns_of<DOWN>(x.n);
                        float gl[4], vl[4];
#pragma unroll 1
                        for (int at = cols; at < (x.n <= kFew ? 3 * cols : 2 * cols); at += cols) {
                            tmem_ld4(acc + at + col, gl);
                            tmem_ld4(acc + Sh::kCols + at + col, vl);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 4; ++j) g[j] += gl[j], v[j] += vl[j];
                        }
                    } else {
                        tc::tmem_wait_ld();
                    }
                    if (!last) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            __stcg(my_part + (size_t)(col + j) * kTile + row, g[j]);
                            __stcg(my_part + (size_t)(kGroup + col + j) * kTile + row, v[j]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) g[j] += pg[j], v[j] += pv[j];
                        const int at = x.m * (DOWN ? kRows : kTile) + row;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (col + j >= x.n) break;
                            if (delta) {
                                g[j] += s.u.e.delta[col % kLotCols<DOWN> + j][row];
                                v[j] += s.u.e.delta[col % kLotCols<DOWN> + j][kTile + row];
                            }
                            if (DOWN) {
                                float *y = p.y + (long long)s.list[x.at + col + j] * p.D + at;
                                const float w = of.weight[col + j];
                                if (at < p.D) __stcg(y, g[j] * w);
                                if (at + kTile < p.D) __stcg(y + kTile, v[j] * w);
                            } else {
                                float h = 0.f;
                                if (at < p.F) {
                                    h = activation(g[j], p.gelu) * v[j];
                                    uint16_t *to = p.h + (long long)(x.pos + col + j) * p.F + at;
                                    const long long part = (long long)p.P * p.F;
                                    const float middle = rest(h);
                                    to[0] = leading(h);
                                    to[part] = leading(middle);
                                    to[2 * part] = leading(rest(middle));
                                }
                                if (ADAPT) s.u.e.h[col + j][row] = h;
                            }
                        }
                    }
                }
                // the lot's delta is no longer read; at the end, all of h is there
                if (ADAPT && last && ((b0 + kBatchCols) % kLotCols<DOWN> == 0 || b0 + kBatchCols >= x.n)) bar_sync(1, kEpiThreads);
            }
            if (!ok) {
                if (!last) asm volatile("bar.arrive 3, %0;" ::"r"(kEpiThreads + 32) : "memory");
                break;
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.acce[buf]);
            if (!last) asm volatile("bar.arrive 3, %0;" ::"r"(kEpiThreads + 32) : "memory");
            if (ADAPT && !DOWN && any_delta) {
#pragma unroll 1
                while (task.left) {
                    epi.run_task(task, x, of, q.MT);
                    if (!epi.next_task(task, x, of)) break;
                }
            }
            x = y;
            now = next;
        }
        asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
        // ---- whoever waits for this CTA's sums of a shared unit (its first one) is told
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (any && part_of(q, s, r, u_hi, e_first).k1 < q.KB) {
            bar_sync(3, kEpiThreads + 32);
            if (lane == 0)
                asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p.flags + (DOWN ? p.grid : 0) + c), "r"(1) : "memory");
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, Sh::kTmem);
}

// The pairs' results of a token in their order, 8 columns a thread; the flags are left as they were found.  Bound by reading y
// back from L2 (256 tokens of 8 pairs and 2048 columns, 16.8 MB: 5 us).
__global__ void __launch_bounds__(kThreads) combine_kernel(const LayerArgs p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int per = p.D / 8;
    const bool mine = i < (long long)p.T * per;
    const int t = (int)(i / per), d = (int)(i % per) * 8;
    unsigned there = 0;  // pairs that have an expert (ids are older than the kernel before this one)
    if (mine)
        for (int k = 0; k < p.K; ++k) there |= (unsigned)(expert_of(p, t * p.K + k, d == 0) >= 0) << k;
    if (mine && d == 0) slot_of(p, t, true);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (i < 2 * p.grid) p.flags[i] = 0;
    if (!mine) return;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < p.K; ++k) {
        const int pair = t * p.K + k;
        if (!(there >> k & 1)) continue;
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
    const size_t P = (size_t)T * d.top_k, R = pool ? pool->R8 : 0;
    Carve c;
    c.flags = 0;
    c.part = c.flags + align256((size_t)2 * sms * 4);
    c.v13 = c.part + (size_t)sms * 2 * kGroup * kTile * 4;
    c.h = c.v13 + align256(P * 2 * R * 4);
    c.v2 = c.h + align256(3 * P * d.d_mlp * 2);
    c.y = c.v2 + align256(P * lora_ceil_div(d.d_mlp, kTile) * R * 4);
    c.bytes = c.y + align256(P * d.d_model * 4);
    return c;
}

// Pairs of a group.  Groups of an expert read its weights once each: the batch's pairs make up to P / group of them
// more, at some 0.5 us for a block and an SM.  A group's epilogue, of which the last one of each of the two kernels is seen, takes some
// 1 us there for eight pairs, 2 with adapters, and a token's favourite experts may get many (91 pairs over 51 experts of 672 x 568, most
// for one of them: groups of 64 57.9 us, of 16 27.7, of 8 28.7; 904 pairs over 18 of 432 x 760 73, of 16 60; 2048 pairs over 64 of
// 2048 x 1408 293 us, of 32 363).  And where units are few, smaller groups share out the work behind the products
// (111 pairs over 6 of 1040 x 272 with adapters: groups of 64 43.6 us, of 8 27.3).
int group_of(const lora_moe_layer_desc_t &d, int P, bool adapters, int sms) {
    const int experts = P < d.n_experts ? P : d.n_experts, each = lora_ceil_div(P, experts);
    const int mt = lora_ceil_div(d.d_mlp, kTile);
    const int64_t blocks = (int64_t)mt * lora_ceil_div(d.d_model, kBK) + (int64_t)lora_ceil_div(d.d_model, kRows) * lora_ceil_div(d.d_mlp, kBK);
    int best = kGroup;
    double least = 1e30;
    for (int g = kGroup; g >= kBatchCols; g /= 2) {
        const double cost = 0.5 * (double)P / g * (double)blocks / sms + (adapters ? 4.0 : 2.0) * g / kBatchCols;
        if (cost < least) {
            least = cost;
            best = g;
        }
    }
    while (best > kBatchCols && (int64_t)experts * lora_ceil_div(each, best) * mt * 2 <= sms) best /= 2;
    return best;
}

struct Device {
    std::atomic<int> sms;  // 0: not looked up yet
};
Device g_devices[64];

template <bool DOWN, bool ADAPT>
cudaError_t set_smem() {
    return cudaFuncSetAttribute(stream_kernel<DOWN, ADAPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)stream_smem<DOWN, ADAPT>());
}

// SM count of the current device; the kernels' attributes are set on the way.
cudaError_t device_sms(int &dev, int &sms) {
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    sms = g_devices[dev].sms.load(std::memory_order_acquire);
    if (sms) return cudaSuccess;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = set_smem<false, false>()) != cudaSuccess || (e = set_smem<false, true>()) != cudaSuccess ||
        (e = set_smem<true, false>()) != cudaSuccess || (e = set_smem<true, true>()) != cudaSuccess ||
        (e = cudaFuncSetAttribute(shrink13_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxP * 8)) != cudaSuccess)
        return e;
    g_devices[dev].sms.store(sms, std::memory_order_release);
    return cudaSuccess;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = grid;
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
    p.group = group_of(d, p.P, pool != nullptr, sms);
    // A pair to a CTA of shrink13: no search for pairs, but rows of A that pairs share are read for each.
    p.single = p.P <= 256;
    if (pool) {
        const lora_pool_desc_t &q = pool->desc;
        p.L = q.max_loras;
        p.R = q.max_rank;
        p.R8 = pool->R8;
        p.shared = q.shared_outer;
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
        !lora_make_tmap_2d(&down.tm_b, p.h, d.d_mlp, 3LL * p.P, d.d_mlp, kBK, 8, true))
        return LORA_ERR_UNSUPPORTED;
    up.a = down.a = p;
    if (pool) {
        // experts, or as many sets of slots as there can be; CTAs that share the batches of one
        const int chunks = lora_ceil_div(p.R, kRanks), sets = !p.shared ? p.single ? p.P : p.E : p.L < T ? p.L : T;
        const int slots = 3 * sms / (sets * p.n13 * chunks), share = p.single || slots < 1 ? 1 : slots > 16 ? 16 : slots;
        const dim3 grid((unsigned)sets, (unsigned)(p.n13 * chunks), (unsigned)(share < T ? share : T));
        LORA_CUDA_TRY(launch(shrink13_kernel, grid, kThreads, (size_t)p.P * 8, s, p, chunks));
    }
    const unsigned grid = (unsigned)sms;
    if (pool) {
        LORA_CUDA_TRY(launch(stream_kernel<false, true>, grid, kStreamThreads, stream_smem<false, true>(), s, up));
        LORA_CUDA_TRY(launch(stream_kernel<true, true>, grid, kStreamThreads, stream_smem<true, true>(), s, down));
    } else {
        LORA_CUDA_TRY(launch(stream_kernel<false, false>, grid, kStreamThreads, stream_smem<false, false>(), s, up));
        LORA_CUDA_TRY(launch(stream_kernel<true, false>, grid, kStreamThreads, stream_smem<true, false>(), s, down));
    }
    const int64_t pieces = (int64_t)T * (d.d_model / 8), most = pieces > 2 * sms ? pieces : 2 * sms;
    LORA_CUDA_TRY(launch(combine_kernel, (unsigned)lora_ceil_div(most, kThreads), kThreads, 0, s, p));
    return LORA_OK;
}
