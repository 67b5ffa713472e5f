// Plans of attention batches, the join of partial results, and the entry
// points of the attention calls (see attn.cuh for the terms).
#include <math.h>
#include <string.h>

#include <atomic>
#include <chrono>

#include "attn.cuh"

using attn::Item;

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;  // of the sort of items by length

// A token with partial results: first those of its own tile, then its prefix's;
// or with own keys that no item covers, of sequence part[0].base.
struct Parts {
    int base, nt;      // first token row of its slot in the first of them, tokens of the slot
    int at;            // which of the slot's tokens it is
    int apart, n;      // token rows from one to the next, and how many there are
};
struct Join {
    int token;
    Parts part[2];
    int keys;
};
static_assert(sizeof(Join) == 48, "joins are 12 words");

struct PlanArgs {
    const int32_t *cu_q, *kv_len, *group_start, *prefix_len;
    int n_seqs, n_groups, T, max_kv, max_prefix;
    int tpi;      // tokens of an item
    int hkv, causal, tpt;
    Item *items;
    attn::Unit *units;
    int32_t *tiles, *token_tiles, *first_tile, *counters;
    Join *joins;
    int max_tokens;
    unsigned long long binding;
};

struct Problem {
    int tok0, n_tok, len, causal;
};

// Problems are the groups' prefixes, then the sequences.
__device__ __forceinline__ Problem problem(const PlanArgs &p, int i) {
    Problem r;
    if (i < p.n_groups) {
        r.tok0 = __ldg(p.cu_q + __ldg(p.group_start + i));
        r.n_tok = __ldg(p.cu_q + __ldg(p.group_start + i + 1)) - r.tok0;
        r.len = __ldg(p.prefix_len + i);
        r.causal = 0;
    } else {
        const int b = i - p.n_groups;
        r.tok0 = __ldg(p.cu_q + b);
        r.n_tok = __ldg(p.cu_q + b + 1) - r.tok0;
        r.len = __ldg(p.kv_len + b);
        r.causal = p.causal;
    }
    return r;
}

// Exclusive sum over the CTA; *total gets the whole sum.  All threads call it.
__device__ int block_scan(int v, int *total) {
    __shared__ int warp_sum[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    const int before = warp ? warp_sum[warp - 1] : 0;
    *total = warp_sum[kPlanThreads / 32 - 1];
    __syncthreads();
    return before + x - v;
}

// Blocks of keys that tile j (tokens from j * tpi on) of a problem has to see.
__device__ __forceinline__ int tile_blocks(const Problem &q, int j, int tpi) {
    const int end = min(q.n_tok, (j + 1) * tpi);
    const long long lim = q.causal ? min((long long)q.len, (long long)q.len - q.n_tok + end) : (long long)q.len;
    return lim <= 0 ? 0 : (int)((lim + attn::kBlock - 1) / attn::kBlock);
}

// Own keys of a single token that the join takes.
__device__ __forceinline__ bool is_short(const PlanArgs &p, const Problem &q, int i) {
    return i >= p.n_groups && p.n_groups && q.n_tok == 1 && q.len <= attn::kShortKeys;
}

// The problem of a tile: the last one whose first tile is at or before it.
__device__ __forceinline__ int find_problem(const int32_t *first, int n, int tile) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs p) {
    __shared__ int hist[2][kBuckets];  // items of two tiles, of one
    __shared__ unsigned long long total_time;
    __shared__ int fit[attn::kMostFit + 1];  // units, were no range longer
    __shared__ int bad;
    const int tid = threadIdx.x;
    const int n = p.n_groups + p.n_seqs;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
        total_time = 0;
        bad = 0;
    }
    // The status word stays as calls left it until it is read.  Only the first build of a
    // binding clears it, also when a captured build is replayed.  Whose it is is asked for
    // here and looked at in the end: waited for here, it would add 0.3 us.
    unsigned long long *binding = (unsigned long long *)(p.counters + attn::kBinding);
    const unsigned long long of = tid == 0 ? *(volatile unsigned long long *)binding : 0;
    auto own_status = [&]() {
        if (of == p.binding) return;
        *binding = p.binding;
        p.counters[attn::kStatus] = LORA_OK;
    };
    for (int i = tid; i < kBuckets; i += kPlanThreads) hist[0][i] = hist[1][i] = 0;
    if (tid <= attn::kMostFit) fit[tid] = 0;
    __syncthreads();
    // the lengths keep to the rules, or the plan is empty
    for (int b = tid; b < p.n_seqs; b += kPlanThreads) {
        const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1), len = __ldg(p.kv_len + b);
        if (c0 < 0 || c1 < c0 || c1 > p.T || (b == 0 && c0 != 0) || (b == p.n_seqs - 1 && c1 != p.T) || len < 0 ||
            len > p.max_kv)
            bad = 1;
    }
    for (int g = tid; g < p.n_groups; g += kPlanThreads) {
        const int g0 = __ldg(p.group_start + g), g1 = __ldg(p.group_start + g + 1), len = __ldg(p.prefix_len + g);
        if (g0 < 0 || g1 < g0 || g1 > p.n_seqs || (g == 0 && g0 != 0) || (g == p.n_groups - 1 && g1 != p.n_seqs) ||
            len < 0 || len > p.max_prefix)
            bad = 1;
    }
    for (int t = tid; t < p.T; t += kPlanThreads) p.token_tiles[t] = p.token_tiles[p.max_tokens + t] = -1;
    __syncthreads();
    if (bad) {
        if (tid == 0) {
            p.counters[attn::kItems] = p.counters[attn::kUnits] = 0;
            p.counters[attn::kPartTokens] = p.counters[attn::kTiles] = p.counters[attn::kJoins] = 0;
            own_status();
            atomicExch(p.counters + attn::kStatus, (int)LORA_ERR_DEVICE_INDEX);
        }
        return;
    }
    // first tile of every problem
    int n_tiles = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int tiles = 0, sum;
        if (i < n) {
            const Problem q = problem(p, i);
            tiles = (q.n_tok + p.tpi - 1) / p.tpi;
        }
        const int at = block_scan(tiles, &sum);
        if (i < n) p.first_tile[i] = n_tiles + at;
        n_tiles += sum;
    }
    __syncthreads();
    // an SM's share of the time, hence the lengths of the ranges
    unsigned long long mine = 0;
    for (int t = tid; t < n_tiles; t += kPlanThreads) {
        const int i = find_problem(p.first_tile, n, t), j = t - p.first_tile[i];
        const Problem q = problem(p, i);
        if (is_short(p, q, i)) continue;
        const unsigned long long b = tile_blocks(q, j, p.tpi);
        mine += 2 * min(p.tpi, q.n_tok - j * p.tpi) <= p.tpi ? attn::kOneBlock * b + attn::kOneItem
                                                             : attn::kPairBlock * b + attn::kPairItem;
        if (n_tiles > attn::kSms) continue;
        for (int r = attn::kMinPrefixBlocks; r <= attn::kMostFit; ++r)
            atomicAdd(&fit[r], i >= p.n_groups && b <= attn::kMinBlocks ? 1 : max(1, (int)((b + r - 1) / r)));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if ((tid & 31) == 0 && mine) atomicAdd(&total_time, mine);
    __syncthreads();
    const unsigned long long share = total_time * (unsigned long long)p.hkv / attn::kSms;
    const unsigned long long share_pair = share / attn::kPairBlock + 1, share_one = share / (2 * attn::kOneBlock) + 1;
    int fits = attn::kMinPrefixBlocks;
    while (fits <= attn::kMostFit && (n_tiles > attn::kSms || fit[fits] * p.hkv > attn::kSms)) ++fits;
    auto range_of = [&](bool prefix, int n_tok) {
        const int least = fits > attn::kMostFit ? attn::kMinBlocks - prefix
                                                : max(fits, prefix ? attn::kMinPrefixBlocks : attn::kMinOwnBlocks);
        return (int)max((unsigned long long)least, 2 * n_tok <= p.tpi ? share_one : share_pair);
    };
    // items and partial rows of each tile; the histogram of item lengths
    int n_part = 0;
    for (int t0 = 0; t0 < n_tiles; t0 += kPlanThreads) {
        const int t = t0 + tid;
        int parts = 0, rows = 0, sum, blocks = 0, range = 1, n_tok = 0, tok0 = 0, i = 0;
        bool joined = false;
        if (t < n_tiles) {
            i = find_problem(p.first_tile, n, t);
            const Problem q = problem(p, i);
            const int j = t - p.first_tile[i];
            blocks = tile_blocks(q, j, p.tpi);
            tok0 = q.tok0 + j * p.tpi;
            n_tok = min(p.tpi, q.n_tok - j * p.tpi);
            int ahead = i < p.n_groups ? 1 : 0;  // this tile's result joins a prefix's
            if (i >= p.n_groups && p.n_groups) {
                int lo = 0, hi = p.n_groups - 1;  // the last group that starts at or before the sequence
                const int b = i - p.n_groups;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (__ldg(p.group_start + mid) <= b) lo = mid; else hi = mid - 1;
                }
                ahead = __ldg(p.prefix_len + lo) > 0;
            }
            const bool few = is_short(p, q, i);
            if (few) p.token_tiles[tok0] = -2 - (i - p.n_groups);
            range = range_of(i < p.n_groups, n_tok);
            if (i >= p.n_groups && blocks <= attn::kMinBlocks) range = attn::kMinBlocks;
            parts = few ? 0 : (blocks + range - 1) / range;
            // no keys: zeros are written, unless a prefix has the tokens' result
            if (parts == 0 && !ahead && !few) parts = 1;
            joined = parts > 1 || ahead;
            if (joined) rows = parts * n_tok;
        }
        const int part0 = n_part + block_scan(rows, &sum);
        n_part += sum;
        if (t < n_tiles) {
            *(int4 *)(p.tiles + 4 * (long long)t) = make_int4(joined ? part0 : -1, parts, tok0, n_tok);
            if (joined && parts) {
                int32_t *map = p.token_tiles + (i < p.n_groups ? p.max_tokens : 0);
                for (int e = 0; e < n_tok; ++e) map[tok0 + e] = t;
            }
            // whole ranges and what is left: the short ones even the CTAs out
            for (int s = 0; s < parts; ++s) {
                const int len = min(blocks - s * range, range);
                atomicAdd(&hist[2 * n_tok <= p.tpi][min(len, kBuckets - 1)], 1);
            }
        }
    }
    __syncthreads();
    // where each length starts, the longest first
    int pairs, singles;
    {
        const int b = kBuckets - 1 - tid;
        const int at0 = block_scan(hist[0][b], &pairs), at1 = block_scan(hist[1][b], &singles);
        hist[0][b] = at0;
        hist[1][b] = pairs + at1;
    }
    __syncthreads();
    for (int t = tid; t < n_tiles; t += kPlanThreads) {
        const int4 e = *(const int4 *)(p.tiles + 4 * (long long)t);
        const int i = find_problem(p.first_tile, n, t);
        const Problem q = problem(p, i);
        const int j = t - p.first_tile[i], blocks = tile_blocks(q, j, p.tpi);
        const int range = e.y == 1 ? max(1, blocks) : range_of(i < p.n_groups, e.w);
        for (int s = 0; s < e.y; ++s) {
            Item it;
            it.blk0 = s * range;
            it.blk1 = min(blocks, (s + 1) * range);
            it.tok0 = e.z;
            it.n_tok = e.w;
            it.prob = i < p.n_groups ? -1 - i : i - p.n_groups;
            it.kv_len = q.len;
            it.lim0 = q.causal ? q.len - q.n_tok + j * p.tpi + 1 : q.len;
            it.part = e.x < 0 ? -1 : e.x + s * e.w;
            const int at = atomicAdd(&hist[2 * it.n_tok <= p.tpi][min(it.blk1 - it.blk0, kBuckets - 1)], 1);
            int4 *dst = (int4 *)(p.items + at);
            dst[0] = make_int4(it.tok0, it.n_tok, it.prob, it.blk0);
            dst[1] = make_int4(it.blk1, it.kv_len, it.lim0, it.part);
        }
    }
    __syncthreads();
    // units: one-tile items go two to a CTA when there are more of them than
    // CTAs; all units by the time they take, the longest first
    const int per = (long long)singles * p.hkv > attn::kSms ? 2 : 1;
    const int n_units = pairs + (singles + per - 1) / per;
    const long long top = max(attn::kPairBlock * (long long)range_of(false, p.tpi) + attn::kPairItem,
                              2LL * (attn::kOneBlock * range_of(false, 0) + attn::kOneItem));
    for (int i = tid; i < kBuckets; i += kPlanThreads) hist[0][i] = 0;
    __syncthreads();
    auto unit = [&](int u, int *first, bool *both) {
        const int at = u < pairs ? u : pairs + (u - pairs) * per;
        const bool two = u >= pairs && per == 2 && at + 1 < pairs + singles;
        *first = at;
        *both = two;
        auto blocks = [&](int i) { return (long long)(p.items[i].blk1 - p.items[i].blk0); };
        const long long time = u < pairs ? attn::kPairBlock * blocks(at) + attn::kPairItem
                                         : attn::kOneBlock * (blocks(at) + (two ? blocks(at + 1) : 0)) +
                                               attn::kOneItem * (two ? 2 : 1);
        return (int)min((long long)kBuckets - 1, time * (kBuckets - 1) / top);
    };
    int first;
    bool both;
    for (int u = tid; u < n_units; u += kPlanThreads) atomicAdd(&hist[0][unit(u, &first, &both)], 1);
    __syncthreads();
    {
        int sum;
        const int b = kBuckets - 1 - tid;
        const int at = block_scan(hist[0][b], &sum);
        hist[0][b] = at;
    }
    __syncthreads();
    for (int u = tid; u < n_units; u += kPlanThreads) {
        const int b = unit(u, &first, &both);
        const int4 *from = (const int4 *)(p.items + first);
        int4 *to = (int4 *)(p.units + atomicAdd(&hist[0][b], 1));
        to[0] = from[0];
        to[1] = from[1];
        to[2] = both ? from[2] : make_int4(0, 0, 0, 0);
        to[3] = both ? from[3] : make_int4(0, 0, 0, 0);
    }
    // the tokens with own keys for the join, which can begin with them while the
    // last items are still computed, then those that have only partial results
    int n_joins = 0;
    for (int keys = 1; keys >= 0; --keys) {
        for (int t0 = 0; t0 < p.T && (keys ? p.n_groups : n_part); t0 += kPlanThreads) {
            const int t = t0 + tid;
            const int own = t < p.T ? p.token_tiles[t] : -1;
            const int has = keys ? own < -1 : own >= 0 || (own == -1 && t < p.T && p.token_tiles[p.max_tokens + t] >= 0);
            int sum;
            const int at = block_scan(has, &sum);
            if (has) {
                Join r;
                r.token = t;
                r.keys = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int tile = p.token_tiles[k * p.max_tokens + t];
                    r.part[k] = {0, 1, 0, 0, 0};
                    if (tile < -1) {
                        r.part[k].base = -2 - tile;
                        r.keys = __ldg(p.kv_len + r.part[k].base);
                    }
                    if (tile < 0) continue;
                    const int4 e = *(const int4 *)(p.tiles + 4 * (long long)tile);
                    const int i = t - e.z, slot = i / p.tpt;  // slots of tpt tokens, the last one of what is left
                    r.part[k] = {e.x + slot * p.tpt, min(p.tpt, e.w - slot * p.tpt), i - slot * p.tpt, e.w, e.y};
                }
                p.joins[n_joins + at] = r;
            }
            n_joins += sum;
        }
    }
    if (tid == 0) {
        p.counters[attn::kJoins] = n_joins;
        p.counters[attn::kItems] = pairs + singles;
        p.counters[attn::kUnits] = n_units;
        p.counters[attn::kPartTokens] = n_part;
        p.counters[attn::kTiles] = n_tiles;
        own_status();
    }
}

// ---------------------------------------------------------------- join

struct JoinArgs {
    const Join *joins;
    const int32_t *counters;
    int hq, hkv, G, D;
    const float *part_o, *part_lse;
    uint16_t *out;
    long long ldo;
    // for the tokens whose own keys no item covers
    const uint16_t *q, *k, *v;
    long long ldq, ldk, ldv, n_rows, ld_table;
    const int32_t *table;
    int32_t *status;
    int page, page_shift;  // page_shift: log2 of the page, -1 if it is no power of two
    float scale_log2;
};

constexpr int kJoinThreads = 128;

__device__ __forceinline__ void ld_global32(float *v, const float *p) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p)
                 : "memory");
}

// 8 bf16 as floats.
__device__ __forceinline__ void floats(float *y, uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(w[i] << 16);
        y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load16(float *y, const uint16_t *x, const bool (&in)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        floats(y + 8 * h, in[h] ? *(const uint4 *)(x + 64 * h) : make_uint4(0, 0, 0, 0));
}

// out[t][h] = sum_s 2^lse_s o_s / sum_s 2^lse_s over the partial results of
// the token's own tile and of its prefix tile, in that order (so the result
// does not depend on which item ended first).  A warp takes a token and kHeads
// heads of one key/value head, whose rows are neighbours in a partial result:
// eight lanes have a head, a lane 8 of its elements and the 8 that lie 64 on.
// The 4 / kHeads groups of eight lanes that share a head share its parts out,
// and are added up in the end.  Bound by latency with few tokens (about 2.5 us
// of a call, most of it one read of what other SMs wrote), by L2 with many.
// With elements of four heads in a lane, 16 bytes each, it read half sectors,
// a line per lane: 889 tokens of 28 heads in two to three parts 16 us, now 6.
// Own keys that no item covers are taken like partial results of one key, whose
// outputs are the rows of V and whose statistics the scores, here a dot product
// over the eight lanes of a head.
template <int kHeads, int kAhead, bool kOwn>
__global__ void __launch_bounds__(kJoinThreads, kHeads == 4 ? 4 : 1) join_kernel(const __grid_constant__ JoinArgs p) {
    constexpr int kSlices = 4 / kHeads;
    // The plan was complete before the item kernel began, which lets this one
    // start: only the partial results are waited for.
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, c0 = lane & 7, u = (lane >> 3) % kHeads, slice = (lane >> 3) / kHeads;
    const int per = (p.G + kHeads - 1) / kHeads * p.hkv;  // warps of a token
    const int step = gridDim.x * (kJoinThreads / 32);
    int w = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
    auto entry = [&](int i) {
        Join r;
        const int4 *at = (const int4 *)(p.joins + i);
        *(int4 *)&r.token = __ldg(at);
        *((int4 *)&r.token + 1) = __ldg(at + 1);
        *((int4 *)&r.token + 2) = __ldg(at + 2);
        return r;
    };
    const long long n = (long long)__ldg(p.counters + attn::kJoins) * per;
    bool waited = false;
#pragma unroll 1
    for (; w < n; w += step) {
        const Join r = entry(w / per);
        const int kvh = (w % per) % p.hkv, g = (w % per) / p.hkv * kHeads + u;
        const int all = r.part[0].n + r.part[1].n, n0 = r.part[0].n;
        const int rows0 = r.part[0].nt * p.G, rows1 = r.part[1].nt * p.G;
        const int at0 = r.part[0].at * p.G + g, at1 = r.part[1].at * p.G + g;
        const long long first0 = (long long)r.part[0].base * p.hq + kvh * rows0, apart0 = (long long)r.part[0].apart * p.hq;
        const long long first1 = (long long)r.part[1].base * p.hq + kvh * rows1, apart1 = (long long)r.part[1].apart * p.hq;
        const int mine = g < p.G ? all : 0;  // parts that there are for this lane
        float top = -INFINITY, sum = 0.f, acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        // to the maximum m: what the sums so far are rescaled by is made theirs
        auto raise = [&](float m) {
            const float base = m == -INFINITY ? 0.f : m, old = exp2f(top - base);
            top = m;
            sum *= old;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] *= old;
            return base;
        };
        if (kOwn) {
            const int keys = r.keys;
            const long long head = (long long)kvh * p.D + 8 * c0;
            const bool in[2] = {g < p.G && 8 * c0 < p.D, g < p.G && 8 * c0 + 64 < p.D};
            float q[16];
            if (keys) load16(q, p.q + r.token * p.ldq + ((long long)kvh * p.G + g) * p.D + 8 * c0, in);
            // the rows of the keys, a lane's each; -1: outside the cache, zeros
            static_assert(attn::kShortKeys <= 32, "a lane for each own key");
            long long row = -1;
            if (lane < keys) {
                const int at = !p.page ? 0 : p.page_shift >= 0 ? lane >> p.page_shift : lane / p.page;
                const long long tab = __ldg(p.table + (long long)r.part[0].base * p.ld_table + at);
                row = p.page ? tab * p.page + (lane - at * p.page) : tab + lane;
                if (row < 0 || row >= p.n_rows) {
                    atomicExch(p.status, (int)LORA_ERR_DEVICE_INDEX);
                    row = -1;
                }
            }
            if (row >= 0) {  // all of them asked for at once
                const uint16_t *kr = p.k + row * p.ldk + (long long)kvh * p.D, *vr = p.v + row * p.ldv + (long long)kvh * p.D;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(kr));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(vr));
                if (p.D > 64) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(kr + 64));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(vr + 64));
                }
            }
            // no more at a time than there are
            constexpr int kOwnAhead = kAhead * kSlices <= attn::kShortKeys ? kAhead : attn::kShortKeys / kSlices;
#pragma unroll 1
            for (int i0 = 0; i0 < keys; i0 += kOwnAhead * kSlices) {
                uint4 k[kOwnAhead][2], v[kOwnAhead][2];
                float score[kOwnAhead];
#pragma unroll
                for (int a = 0; a < kOwnAhead; ++a) {
                    const int i = i0 + a * kSlices + slice;
                    const int x = __shfl_sync(0xffffffffu, (int)row, i & 31);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool is = in[h] && i < keys && x >= 0;
                        k[a][h] = is ? *(const uint4 *)(p.k + x * p.ldk + head + 64 * h) : make_uint4(0, 0, 0, 0);
                        v[a][h] = is ? *(const uint4 *)(p.v + x * p.ldv + head + 64 * h) : make_uint4(0, 0, 0, 0);
                    }
                }
                float m = top;
#pragma unroll
                for (int a = 0; a < kOwnAhead; ++a) {
                    float y[16], d = 0.f;
                    floats(y, k[a][0]);
                    floats(y + 8, k[a][1]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) d += q[i] * y[i];
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                    score[a] = i0 + a * kSlices + slice < keys ? d * p.scale_log2 : -INFINITY;
                    m = fmaxf(m, score[a]);
                }
                const float base = raise(m);
#pragma unroll
                for (int a = 0; a < kOwnAhead; ++a) {
                    const float x = exp2f(score[a] - base);
                    if (x == 0.f) continue;
                    float y[16];
                    floats(y, v[a][0]);
                    floats(y + 8, v[a][1]);
                    sum += x;
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[i] += x * y[i];
                }
            }
        }
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
        // kAhead parts at a time, their loads together; the sums so far are
        // rescaled when a part's maximum is above theirs
#pragma unroll 1
        for (int s0 = slice; s0 < all; s0 += kAhead * kSlices) {
            float lse[kAhead], v[kAhead][16];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int s = s0 + a * kSlices;
                const bool second = s >= n0;
                const int rows = second ? rows1 : rows0, at = second ? at1 : at0;
                const long long first = second ? first1 + (s - n0) * apart1 : first0 + s * apart0;
                const float *o = p.part_o + first * p.D + (c0 * rows + at) * 8;
                lse[a] = s < mine ? p.part_lse[first + at] : -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (s < mine && 8 * c0 + 64 * h < p.D) {
                        ld_global32(v[a] + 8 * h, o + 64 * h * rows);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[a][8 * h + i] = 0.f;
                    }
                }
            }
            float m = top;
#pragma unroll
            for (int a = 0; a < kAhead; ++a) m = fmaxf(m, lse[a]);
            const float base = raise(m);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                // a part without keys weighs nothing; a NaN or infinite score makes its weight NaN
                const float x = exp2f(lse[a] - base);
                if (x == 0.f) continue;
                sum += x;
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] += x * v[a][i];
            }
        }
#pragma unroll
        for (int o = 8 * kHeads; o < 32; o <<= 1) {
            const float m = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float x = exp2f(top - (m == -INFINITY ? 0.f : m));
            top = m;
            sum *= x;
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                acc[i] *= x;
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            }
        }
        const float f = sum == 0.f ? 0.f : 1.f / sum;
        uint16_t *out = p.out + (long long)r.token * p.ldo + (long long)(kvh * p.G + g) * p.D + 8 * c0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (slice || g >= p.G || 8 * c0 + 64 * h >= p.D) continue;
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 y = __floats2bfloat162_rn(acc[8 * h + 2 * i] * f, acc[8 * h + 2 * i + 1] * f);
                x[i] = *(const uint32_t *)&y;
            }
            *(uint4 *)(out + 64 * h) = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
    // a kernel after this one must not start on what the item kernel still writes
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- host

bool desc_ok(const lora_attn_desc_t &d) {
    if (d.n_kv_heads < 1 || d.n_q_heads < d.n_kv_heads || d.n_q_heads % d.n_kv_heads || d.n_q_heads > (1 << 20))
        return false;
    if (d.n_q_heads / d.n_kv_heads > attn::kTileRows) return false;
    if (d.head_dim < 8 || d.head_dim > 128 || d.head_dim % 8) return false;
    if (d.page_size < 0 || d.page_size % 8 || (d.causal != 0 && d.causal != 1)) return false;
    return isfinite(d.scale) && d.scale > 0.f && isfinite(d.scale * 1.44269504f);
}

constexpr int kMostRanges = 2 * attn::kSms;

struct Caps {
    long long tpi, items, tiles, part;
};

// What a batch of the given size can need.  A range of a tile beyond its first
// stands for a range's length of blocks; all ranges of one length take at
// least half an SM's share each, so there are at most 2 * kSms of them (times
// key/value heads).  A tile of two or more ranges has at most twice the ranges
// that it has beyond the first; with prefixes every token also has one partial
// result of its own keys and one of its prefix.
Caps caps(const lora_attn_desc_t &d, long long tokens, long long seqs, long long groups) {
    Caps c;
    c.tpi = 2 * attn::tile_tokens(d.n_q_heads / d.n_kv_heads);
    const long long extra = kMostRanges / d.n_kv_heads;
    c.tiles = (tokens / c.tpi + seqs) + (groups ? tokens / c.tpi + groups : 0);
    c.items = c.tiles + extra;
    const long long most = c.tpi < tokens ? c.tpi : tokens;
    c.part = 2 * extra * most + (groups ? 2 * tokens : 0);
    return c;
}

// A number for each binding of a plan, which memory that another one left does not hold by
// chance: the time of the first binding, spread over 64 bits by an odd factor, and a count.
uint64_t next_binding() {
    static const uint64_t first =
        (uint64_t)std::chrono::system_clock::now().time_since_epoch().count() * 0x9e3779b97f4a7c15ull;
    static std::atomic<uint64_t> n{0};
    return first + n.fetch_add(1, std::memory_order_relaxed);
}

size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

size_t plan_bytes(const Caps &c, long long tokens, long long seqs, long long groups) {
    return align16((size_t)c.items * sizeof(Item)) + (size_t)c.items * sizeof(attn::Unit) + align16((size_t)c.tiles * 16) +
           align16((size_t)tokens * 8) + (size_t)tokens * sizeof(Join) + align16((size_t)(seqs + groups) * 4) + 32;
}

bool caps_ok(const lora_attn_desc_t *desc, int32_t max_tokens, int32_t max_seqs, int32_t max_groups, Caps *c) {
    if (!desc || !desc_ok(*desc) || max_tokens < 1 || max_seqs < 1 || max_groups < 0)
        return false;
    *c = caps(*desc, max_tokens, max_seqs, max_groups);
    return c->items * desc->n_kv_heads <= 0x7fffffffLL && (long long)max_tokens * desc->n_q_heads <= 0x3fffffffLL &&
           c->part <= 0x7fffffffLL && c->tiles <= 0x1fffffffLL;
}

size_t part_bytes(const lora_attn_plan_t &p) {
    return (size_t)p.max_part * p.desc.n_q_heads * (p.desc.head_dim + 1) * 4 + 32;  // the first on 32 bytes
}

constexpr size_t kWsHead = 256;  // control words at the start of a workspace

cudaLaunchConfig_t config(int grid, int threads, cudaStream_t s, cudaLaunchAttribute *at) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = s;
    return cfg;
}

// CTAs of the join with so many heads to a warp, were each warp to take one token.
long long join_ctas(const attn::Args &a, int heads) {
    const long long warps = (long long)a.T * ((a.G + heads - 1) / heads * a.hkv);
    return (warps + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
}

template <int kHeads, int kAhead>
cudaError_t join_launch(const JoinArgs &j, bool own, long long ctas, int per_sm, cudaStream_t s) {
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = config((int)(ctas < per_sm * attn::kSms ? ctas : per_sm * attn::kSms), kJoinThreads, s, at);
    return own ? cudaLaunchKernelEx(&cfg, join_kernel<kHeads, kAhead, true>, j)
               : cudaLaunchKernelEx(&cfg, join_kernel<kHeads, kAhead, false>, j);
}

lora_status_t attention(const lora_attn_plan_t *plan, const void *q, int64_t ldq, const void *k, int64_t ldk,
                        const void *v, int64_t ldv, int64_t n_rows, const int32_t *table, int64_t ld_table,
                        const int32_t *ptable, int64_t ld_ptable, void *out, int64_t ldo, void *workspace,
                        size_t ws_bytes, bool prefix, void *stream) {
    if (!plan || !plan->counters || plan->total_q < 0 || plan->n_seqs < 0) return LORA_ERR_INVALID_ARG;
    if ((plan->n_groups > 0) != prefix) return LORA_ERR_UNSUPPORTED;
    const lora_attn_desc_t &d = plan->desc;
    const int64_t qc = (int64_t)d.n_q_heads * d.head_dim, kc = (int64_t)d.n_kv_heads * d.head_dim;
    if (ldq < qc || ldq % 8 || ldk < kc || ldk % 8 || ldv < kc || ldv % 8 || ldo < qc || ldo % 8 || n_rows < 0 ||
        n_rows > attn::kMostRows)
        return LORA_ERR_INVALID_ARG;
    const int64_t page = d.page_size;
    if (plan->max_kv_len > 0 &&
        (!table || ((uintptr_t)table & 3) || (page ? ld_table * page < plan->max_kv_len : ld_table < 1)))
        return LORA_ERR_INVALID_ARG;
    if (plan->max_prefix_len > 0 &&
        (!ptable || ((uintptr_t)ptable & 3) || (page ? ld_ptable * page < plan->max_prefix_len : ld_ptable < 1)))
        return LORA_ERR_INVALID_ARG;
    if (plan->total_q == 0) return LORA_OK;
    if (!q || !k || !v || !out || !lora_aligned16(q) || !lora_aligned16(k) || !lora_aligned16(v) ||
        !lora_aligned16(out))
        return LORA_ERR_INVALID_ARG;
    if (!workspace || !lora_aligned16(workspace)) return LORA_ERR_INVALID_ARG;
    if (ws_bytes < kWsHead + part_bytes(*plan)) return LORA_ERR_CAPACITY;
    cudaStream_t s = (cudaStream_t)stream;
    attn::Args a;
    memset(&a, 0, sizeof(a));
    a.units = (const attn::Unit *)plan->units;
    a.counters = plan->counters;
    a.tickets = (int32_t *)workspace;
    a.status = plan->counters + attn::kStatus;
    a.hq = d.n_q_heads;
    a.hkv = d.n_kv_heads;
    a.G = d.n_q_heads / d.n_kv_heads;
    a.D = d.head_dim;
    a.page = d.page_size;
    a.causal = d.causal;
    a.T = plan->total_q;
    a.scale_log2 = d.scale * 1.44269504088896340736f;
    a.q = (const uint16_t *)q;
    a.k = (const uint16_t *)k;
    a.v = (const uint16_t *)v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.n_rows = n_rows;
    a.ldo = ldo;
    a.table = table;
    a.ptable = ptable;
    a.ld_table = ld_table;
    a.ld_ptable = ld_ptable;
    a.out = (uint16_t *)out;
    a.part_o = (float *)(((uintptr_t)workspace + kWsHead + 31) & ~(uintptr_t)31);
    a.part_lse = a.part_o + (size_t)plan->max_part * d.n_q_heads * d.head_dim;
    const Caps c = caps(d, plan->total_q, plan->n_seqs, plan->n_groups);
    const lora_status_t st = lora_attn_launch(a, (int)c.items, s);  // no more units than items
    if (st != LORA_OK) return st;
    // without prefixes, tiles of up to kMinBlocks blocks are never split
    if (!prefix && plan->max_kv_len <= attn::kMinBlocks * attn::kBlock) return LORA_OK;
    JoinArgs j;
    memset(&j, 0, sizeof(j));
    j.joins = (const Join *)plan->joins;
    j.counters = plan->counters;
    j.hq = d.n_q_heads;
    j.hkv = d.n_kv_heads;
    j.G = a.G;
    j.D = d.head_dim;
    j.part_o = a.part_o;
    j.part_lse = a.part_lse;
    j.out = a.out;
    j.ldo = ldo;
    j.q = a.q;
    j.k = a.k;
    j.v = a.v;
    j.ldq = ldq;
    j.ldk = ldk;
    j.ldv = ldv;
    j.n_rows = n_rows;
    j.table = table;
    j.ld_table = ld_table;
    j.status = a.status;
    j.page = d.page_size;
    for (j.page_shift = 0; j.page_shift < 31 && 1 << j.page_shift < d.page_size;) ++j.page_shift;
    if (1 << j.page_shift != d.page_size) j.page_shift = -1;
    j.scale_log2 = a.scale_log2;
    // One head to a warp while all its warps fit the SMs at once (their registers let two
    // CTAs be resident) or where no heads share keys, then two, then four: 16 tokens behind a
    // prefix of 8000 20 us against 28 with four heads, 64 tokens over 4000 keys 17.9 with two
    // against 18.9 with four and 19.9 with one, 256 tokens behind 8190 86 with four against 98
    // with one; 240 tokens of 16 heads of their own 67 with one against 75 with four.
    const long long one = join_ctas(a, 1), two = join_ctas(a, 2), all = join_ctas(a, 4);
    cudaError_t e;
    if (one <= 2 * attn::kSms) e = join_launch<1, 8>(j, prefix, one, 2, s);
    else if (a.G == 1) e = join_launch<1, 4>(j, prefix, one, 3, s);
    else if (two <= 3 * attn::kSms) e = join_launch<2, 4>(j, prefix, two, 3, s);
    else e = join_launch<4, 3>(j, prefix, all, 4, s);
    LORA_CUDA_TRY(e);
    lora_note_launch();
    return LORA_OK;
}

}  // namespace

extern "C" size_t lora_attn_plan_bytes(const lora_attn_desc_t *desc, int32_t max_tokens, int32_t max_seqs,
                                       int32_t max_groups) {
    Caps c;
    if (!caps_ok(desc, max_tokens, max_seqs, max_groups, &c)) return 0;
    return plan_bytes(c, max_tokens, max_seqs, max_groups);
}

extern "C" lora_status_t lora_attn_plan_bind(lora_attn_plan_t *plan, const lora_attn_desc_t *desc, void *d_buf,
                                             size_t bytes, int32_t max_tokens, int32_t max_seqs, int32_t max_groups) {
    Caps c;
    if (!plan || !caps_ok(desc, max_tokens, max_seqs, max_groups, &c) || !d_buf || !lora_aligned16(d_buf))
        return LORA_ERR_INVALID_ARG;
    if (bytes < plan_bytes(c, max_tokens, max_seqs, max_groups)) return LORA_ERR_CAPACITY;
    memset(plan, 0, sizeof(*plan));
    plan->desc = *desc;
    plan->max_tokens = max_tokens;
    plan->max_seqs = max_seqs;
    plan->max_groups = max_groups;
    plan->max_items = (int32_t)c.items;
    plan->max_tiles = (int32_t)c.tiles;
    plan->max_part = (int32_t)c.part;
    plan->n_seqs = plan->total_q = -1;  // nothing built yet
    plan->binding = next_binding();
    char *at = (char *)d_buf;
    plan->counters = (int32_t *)at;
    at += 32;
    plan->items = (int32_t *)at;
    at += align16((size_t)c.items * sizeof(Item));
    plan->units = (int32_t *)at;
    at += (size_t)c.items * sizeof(attn::Unit);
    plan->tiles = (int32_t *)at;
    at += align16((size_t)c.tiles * 16);
    plan->token_tiles = (int32_t *)at;
    at += align16((size_t)max_tokens * 8);
    plan->joins = (int32_t *)at;
    at += (size_t)max_tokens * sizeof(Join);
    plan->first_tile = (int32_t *)at;
    return LORA_OK;
}

extern "C" lora_status_t lora_attn_build_plan(lora_attn_plan_t *plan, int32_t n_seqs, int32_t total_q,
                                              const int32_t *d_cu_q, const int32_t *d_kv_len, int32_t n_groups,
                                              const int32_t *d_group_start, const int32_t *d_prefix_len,
                                              int32_t max_kv_len, int32_t max_prefix_len, void *stream) {
    if (!plan || !plan->counters || n_seqs < 0 || total_q < 0 || n_groups < 0 || max_kv_len < 0 ||
        max_prefix_len < 0 || max_kv_len > attn::kMostKeys || max_prefix_len > attn::kMostKeys ||
        (n_seqs == 0 && total_q > 0))
        return LORA_ERR_INVALID_ARG;
    if (n_seqs > plan->max_seqs || total_q > plan->max_tokens || n_groups > plan->max_groups) return LORA_ERR_CAPACITY;
    if (n_seqs > 0 && (!d_cu_q || !d_kv_len || ((uintptr_t)d_cu_q & 3) || ((uintptr_t)d_kv_len & 3)))
        return LORA_ERR_INVALID_ARG;
    if (n_groups > 0 && (!d_group_start || !d_prefix_len || ((uintptr_t)d_group_start & 3) ||
                         ((uintptr_t)d_prefix_len & 3)))
        return LORA_ERR_INVALID_ARG;
    PlanArgs p;
    memset(&p, 0, sizeof(p));
    p.cu_q = d_cu_q;
    p.kv_len = d_kv_len;
    p.group_start = d_group_start;
    p.prefix_len = d_prefix_len;
    p.n_seqs = n_seqs;
    p.n_groups = n_seqs ? n_groups : 0;  // groups of no sequences at all: no lengths to read
    p.T = total_q;
    p.max_kv = max_kv_len;
    p.max_prefix = max_prefix_len;
    p.tpi = 2 * attn::tile_tokens(plan->desc.n_q_heads / plan->desc.n_kv_heads);
    p.hkv = plan->desc.n_kv_heads;
    p.causal = plan->desc.causal;
    p.items = (Item *)plan->items;
    p.units = (attn::Unit *)plan->units;
    p.tiles = plan->tiles;
    p.token_tiles = plan->token_tiles;
    p.joins = (Join *)plan->joins;
    p.tpt = attn::tile_tokens(plan->desc.n_q_heads / plan->desc.n_kv_heads);
    p.first_tile = plan->first_tile;
    p.counters = plan->counters;
    p.max_tokens = plan->max_tokens;
    p.binding = plan->binding;
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = config(1, kPlanThreads, (cudaStream_t)stream, at);
    LORA_CUDA_TRY(cudaLaunchKernelEx(&cfg, plan_kernel, p));
    lora_note_launch();
    plan->n_seqs = n_seqs;
    plan->total_q = total_q;
    plan->n_groups = n_groups;
    plan->max_kv_len = max_kv_len;
    plan->max_prefix_len = n_groups ? max_prefix_len : 0;
    return LORA_OK;
}

extern "C" size_t lora_attn_workspace_bytes(const lora_attn_plan_t *plan) {
    if (!plan || !plan->counters) return 0;
    return kWsHead + part_bytes(*plan);
}

extern "C" lora_status_t lora_prompt_attention(const lora_attn_plan_t *plan, const void *q, int64_t ldq, const void *k,
                                               int64_t ldk, const void *v, int64_t ldv, int64_t n_rows,
                                               const int32_t *table, int64_t ld_table, void *out, int64_t ldo,
                                               void *workspace, size_t ws_bytes, void *stream) {
    return attention(plan, q, ldq, k, ldk, v, ldv, n_rows, table, ld_table, nullptr, 0, out, ldo, workspace, ws_bytes,
                     false, stream);
}

extern "C" lora_status_t lora_prefix_attention(const lora_attn_plan_t *plan, const void *q, int64_t ldq, const void *k,
                                               int64_t ldk, const void *v, int64_t ldv, int64_t n_rows,
                                               const int32_t *table, int64_t ld_table, const int32_t *prefix_table,
                                               int64_t ld_prefix, void *out, int64_t ldo, void *workspace,
                                               size_t ws_bytes, void *stream) {
    return attention(plan, q, ldq, k, ldk, v, ldv, n_rows, table, ld_table, prefix_table, ld_prefix, out, ldo,
                     workspace, ws_bytes, true, stream);
}

extern "C" lora_status_t lora_attn_get_status(const lora_attn_plan_t *plan, void *stream) {
    if (!plan || !plan->counters) return LORA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    int32_t c[8];
    LORA_CUDA_TRY(cudaMemcpyAsync(c, plan->counters, sizeof(c), cudaMemcpyDeviceToHost, s));
    LORA_CUDA_TRY(cudaStreamSynchronize(s));
    uint64_t binding;
    memcpy(&binding, c + attn::kBinding, sizeof(binding));
    // memory that no build of this binding has reached yet says nothing
    if (binding != plan->binding || c[attn::kStatus] == LORA_OK) return LORA_OK;
    LORA_CUDA_TRY(cudaMemsetAsync(plan->counters + attn::kStatus, 0, 4, s));
    LORA_CUDA_TRY(cudaStreamSynchronize(s));
    return (lora_status_t)c[attn::kStatus];
}
