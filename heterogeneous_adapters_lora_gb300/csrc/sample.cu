// The next token of every row of logits: temperature, top-k, top-p, min-p and a
// draw by a given random number.
//
// A row of bf16 logits has few distinct values: at most 65536, and a few
// thousand in practice.  So the columns are counted by value (atomics in shared memory), and
// everything else works on the counts: the weight exp((l - largest) / T) of a value times its
// count, running sums of those in descending order, and the places where such a sum
// passes a bound.  Only the position of the chosen column among its equals asks for the row again.
//
// The bounds of top-p and of the draw are compared with sums of up to 257024
// weights, and one column more or less is another token.  So weights are
// integers, 2^62 for the largest, from 64-bit products (weight62), and sums are 128-bit
// integers: exact, whatever their order.  fp64 would do too, but GB300 has few units for it
// (4096 weights took longer than reading the row).
//
// Counting takes 13 instructions for two columns, all of them on both at once but the
// addresses; columns outside of the counted range (masked ones, zeros) leave that path by eights.  Adds to 32 random
// banks take some 3.5 passes, which bound it (256 rows of 128256 columns 51 us, with a bank to each lane 36).
// Where rows are few a cluster of up to 8 CTAs shares one: each counts its part, tells which groups of 128
// values it has any of, and adds up all parts' counts of its share of those over distributed shared memory.
// The rest is a chain of dependent steps: the entries in order (3 us), their weights and running sums (4), up to three bounds, which the
// first warp of every CTA finds for itself (3 to 6), and the chosen column's position in the row (5).  256 rows of 128256 columns
// take 58 us: with two of them to an SM counting takes 28, in the last to end 35, the rest of that one's chain 19.
//
// Keys are bf16 bits mapped to integers that grow with the value.  A window is a
// range of keys that is counted at once:
//   one     the keys of 0 and of magnitudes in (2^-55, 2^9), 16384 places: all that
//           takes part in most rows
//   many    otherwise 16 windows of 4096 keys each, in descending order, each
//           counted when it is asked for, by the first CTA of the cluster alone
#include <math.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "lora_internal.cuh"
#include "mma_common.cuh"

namespace {

typedef unsigned long long u64;
typedef unsigned __int128 u128;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMagLo = 72 * 128, kMags = 64 * 128;  // magnitudes [2^-55, 2^9) as bf16 bits
constexpr int kBins = 2 * kMags + 1;                // by magnitude, the sign above it, 0 last
constexpr int kPlaces = 2 * kMags;                  // of the order; +2^-55 has none
constexpr int kGroups = kPlaces / 128;              // of places: four to a lane of a warp
constexpr int kRounds = kGroups / kWarps;           // most of them to a warp
constexpr int kMostCtas = 8;
constexpr int kWinBins = 4096;
constexpr int kWindows = 65536 / kWinBins;
constexpr unsigned kKeyMax = 0xff7fu;  // key of the largest finite number

struct SampleArgs {
    const uint16_t *logits;
    long long ld;
    int T, V, C;  // C CTAs share a row
    const float *temperature, *top_p, *min_p, *uniform;
    const int32_t *top_k;
    int32_t *tokens;
    float *logprobs;
};

// Key of a logit's bits: grows with the value, 0 = takes no part.
__device__ __forceinline__ unsigned key_of(unsigned b) {
    const unsigned mag = b & 0x7fffu;
    if (mag > 0x7f80u || b == 0xff80u) return 0u;  // NaN, -inf
    if (mag == 0u) return 0x8000u;                 // -0 equals +0
    if (b == 0x7f80u) return kKeyMax;              // +inf
    return (b & 0x8000u) ? 0x7fffu - mag : 0x8000u | mag;
}
__device__ __forceinline__ float value_of(unsigned key) {
    const unsigned b = (key & 0x8000u) ? key & 0x7fffu : 0x8000u | (0x7fffu - key);
    return __uint_as_float(b << 16);
}

// Places of the one window, in descending order of values: positive magnitudes, 0, negative ones (bins
// kMags - 1 to 1, the one of 0, kMags to 2 kMags - 1).
__device__ __forceinline__ unsigned key_of_place(int place, int window) {
    if (window >= 0) return (unsigned)(window * kWinBins + kWinBins - 1 - place);
    if (place == kMags - 1) return 0x8000u;
    return place < kMags ? 0x8000u | (unsigned)(kMagLo + kMags - 1 - place) : 0x7fffu - (unsigned)(kMagLo + place - kMags);
}

// 2^(-2^-j) for j = 1..18 in units of 2^-63.
__device__ const u64 kRoots[18] = {0x5a827999fcef3242ull, 0x6ba27e656b4eb57aull, 0x75606373ee921c97ull,
                                   0x7a92be8a92436616ull, 0x7d41d96db915019dull, 0x7e9f06067a4360baull,
                                   0x7f4f08ae3dc7c426ull, 0x7fa765aca88f6453ull, 0x7fd3ab290e46d769ull,
                                   0x7fe9d3a8e07bf086ull, 0x7ff4e9597bed93abull, 0x7ffa748dff8dc61full,
                                   0x7ffd3a3f50020332ull, 0x7ffe9d1dbc0a75aaull, 0x7fff4e8e6306ed59ull,
                                   0x7fffa74712c3cdfdull, 0x7fffd3a381b1fa29ull, 0x7fffe9d1beed018aull};
constexpr u64 kOne63 = 1ull << 63;

__device__ __forceinline__ u64 mul63(u64 a, u64 b) { return __umul64hi(a, b) << 1; }

// The factors 2^(-i / 64), 2^(-i / 4096) and 2^(-i / 2^18), i < 64, of weight62.
__device__ __forceinline__ void fill_powers(u64 *pw) {
#pragma unroll 1
    for (int i = threadIdx.x; i < 192; i += kThreads) {
        u64 v = kOne63;
#pragma unroll
        for (int b = 0; b < 6; ++b)
            if ((i & 63) >> (5 - b) & 1) v = mul63(v, kRoots[(i >> 6) * 6 + b]);
        pw[i] = v;
    }
}

struct Scale {
    float up;      // a power of two that logits are multiplied by, so that fp32 holds what follows
    float hi, lo;  // log2(e) / temperature / up as a sum
    float top;     // the largest logit, times up
    int e;         // exponent of the temperature
};

// With temperature = m 2^e, m in [0.5, 1): log2(e) / m, a quotient and its remainder's; and logits times
// 2^-e.  Where the power would make the largest logit exceed 2^100, a smaller one does: distinct logits
// are then at least 2^91 apart, and every weight but the largest is 0 whatever the factor.
__device__ __forceinline__ Scale begin_scale(float temperature) {
    constexpr float kLog2e = 1.4426950408889634f, kRest = (float)(1.4426950408889634 - (double)kLog2e);
    Scale r;
    r.hi = r.lo = 0.f;
    r.e = 2;
    if (temperature < INFINITY) {
        const float m = frexpf(temperature, &r.e);
        r.hi = kLog2e / m;
        r.lo = (fmaf(-r.hi, m, kLog2e) + kRest) / m;
    }
    return r;
}
__device__ __forceinline__ void end_scale(Scale &r, float top) {
    int s = max(-126, min(126, -r.e));
    if (top != 0.f) s = min(s, 100 - ilogbf(top));
    const float rest = exp2f((float)min(-r.e - s, 30));
    r.hi *= rest;
    r.lo *= rest;
    r.up = __int_as_float((s + 127) << 23);
    r.top = top * r.up;
}

// (top - v) * log2(e) / temperature as hi + lo, to about 2^-46 of it.
__device__ __forceinline__ void distance(const Scale &c, float v, float &hi, float &lo) {
    v *= c.up;
    const float d = c.top - v;  // d + e is the difference without error
    const float bb = d - c.top;
    const float e = (c.top - (d - bb)) + (-v - bb);
    hi = d * c.hi;
    lo = fmaf(d, c.lo, fmaf(e, c.hi, fmaf(d, c.hi, -hi)));
}

// exp((v - top) / temperature) in units of 2^-62: y = i + i1 / 64 + i2 / 4096 + i3 /
// 2^18 + r, the three powers from tables, 2^-r by its series (r < 2^-18: the
// cubic term is below 2^-56).  Off by at most (y + 1) 2^-47 of itself, from y, and 2^-62 of the largest, as it is cut.
__device__ __forceinline__ u64 weight62(const Scale &c, float v, const u64 *pw) {
    float hi, lo;
    distance(c, v, hi, lo);
    const float sum = __fadd_rn(hi, lo);  // (lo can exceed a step of hi)
    lo -= __fadd_rn(sum, -hi);
    hi = sum;
    if (!(hi < 62.f)) return 0ull;
    // y in units of 2^-50: its multiple of 2^-24, and the rest (half a step of hi at most, 2^-19), each a 32-bit conversion
    const int whole = __float2int_rd(hi * 0x1p24f);
    const int rest = __float2int_rn((lo + (hi - (float)whole * 0x1p-24f)) * 0x1p50f);
    long long y = ((long long)whole << 26) + rest;
    y = y < 0 ? 0 : y;
    const unsigned low = (unsigned)y, high = (unsigned)((u64)y >> 32);  // r; i3 (6 bits), i2, i1, i
    const unsigned q = __umulhi(low, 0xb17217f8u);                      // r ln 2 in units of 2^-50
    u64 w = kOne63 - ((u64)q << 13) + (__umulhi(q, q) >> 6);
    w = mul63(w, pw[high >> 12 & 63]);
    w = mul63(w, pw[64 + (high >> 6 & 63)]);
    w = mul63(w, pw[128 + (high & 63)]);
    return w >> (1 + (high >> 18));
}

struct Sums {
    u128 mass;
    int n;
};

struct Found {
    unsigned key;
    int rank, n;  // which of the key's columns; columns up to and with it
    u64 lo, hi;   // ... and their weight
};

// What a CTA tells the others of its row.
struct Told {
    int top;       // first place of its part that is not empty
    uint8_t some[kWarps];  // groups of its part that are not empty, a bit each
    unsigned low;  // largest key below the one window
    int odd;       // a key in the gaps of the one window, or above it
    u64 lo, hi, least_lo, least_hi;  // weight of its slice, and of the beginning of at least min_p a column
    int n, least_n;
    int entries;   // places of its slice that are not empty
    int matches;   // columns of its part with the chosen key
};

struct Shared {
    alignas(16) unsigned bins[kBins + 7];             // by bits; or a window's in descending order
    u64 pw[192];
    unsigned groups[kGroups / 32];         // that are not empty in any part, as bits
    uint8_t group_at[kGroups];             // ... and in their order
    u64 warp_lo[kWarps], warp_hi[kWarps];  // 128-bit partial sums
    int warp_n[kWarps], last;
    Told told;
    Told all[kMostCtas];  // of every CTA
    Found found;
    Scale scale;
    // many windows
    int coarse[kWindows];
    u64 win_lo[kWindows], win_hi[kWindows];
    int win_n[kWindows];
};

// Sums ahead of a thread's entries.
struct Pre {
    u64 lo[kThreads], hi[kThreads];
    unsigned n[kThreads];
};

// Behind the rest of shared memory: the entries of a CTA's share, where several have the row (one has them where the
// counts were), and Pre.  Of two CTAs Pre lies where the counts were, so that half of a long row can be kept.
constexpr size_t kExtra = (sizeof(Shared) + 15) & ~(size_t)15;
__host__ __device__ constexpr size_t list_bytes(int C) { return C == 1 ? 0 : (size_t)kPlaces / C * 4; }
__host__ __device__ constexpr size_t extra_bytes(int C) { return list_bytes(C) + (C == 2 ? 0 : sizeof(Pre)); }
static_assert(sizeof(Pre) <= sizeof(unsigned[kPlaces / 2]) && kWinBins <= kPlaces / 2, "Pre in the second half of the counts");

__device__ __forceinline__ u128 join(u64 hi, u64 lo) { return ((u128)hi << 64) | lo; }

// Sums over the threads before this one, and over all of them.
__device__ __forceinline__ Sums scan(Shared &s, Sums mine, Sums &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 hi = __shfl_up_sync(kAll, (u64)(inc.mass >> 64), o), lo = __shfl_up_sync(kAll, (u64)inc.mass, o);
        const int n = __shfl_up_sync(kAll, inc.n, o);
        if (lane >= o) {
            inc.mass += join(hi, lo);
            inc.n += n;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.warp_hi[warp] = (u64)(inc.mass >> 64);
        s.warp_lo[warp] = (u64)inc.mass;
        s.warp_n[warp] = inc.n;
    }
    __syncthreads();
    static_assert(kWarps == 16, "a warp's sums to a lane of half a warp");
    Sums all = {join(s.warp_hi[lane & 15], s.warp_lo[lane & 15]), s.warp_n[lane & 15]};
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const u64 hi = __shfl_up_sync(kAll, (u64)(all.mass >> 64), o, 16), lo = __shfl_up_sync(kAll, (u64)all.mass, o, 16);
        const int n = __shfl_up_sync(kAll, all.n, o, 16);
        if ((lane & 15) >= o) {
            all.mass += join(hi, lo);
            all.n += n;
        }
    }
    total.mass = join(__shfl_sync(kAll, (u64)(all.mass >> 64), 15), __shfl_sync(kAll, (u64)all.mass, 15));
    total.n = __shfl_sync(kAll, all.n, 15);
    const int ahead = warp ? warp - 1 : 0;
    Sums before = {join(__shfl_sync(kAll, (u64)(all.mass >> 64), ahead), __shfl_sync(kAll, (u64)all.mass, ahead)),
                   __shfl_sync(kAll, all.n, ahead)};
    if (!warp) before = {0, 0};
    before.mass += inc.mass - mine.mass;
    before.n += inc.n - mine.n;
    return before;
}

// A row's columns from `begin` on, 8 at a time: f(column, its 8 bits' words), and g(column, bits) for
// those of a last vector that is not whole.
template <int kAhead, typename F, typename G>
__device__ __forceinline__ void each_vector(const uint16_t *row, int begin, int end, int at, int step, F f, G g) {
    const int whole = begin + ((end - begin) & ~7);
#pragma unroll 1
    for (int i = begin + at * 8; i < whole; i += kAhead * step * 8) {
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i + j * step * 8 < whole) v[j] = __ldg((const uint4 *)(row + i + j * step * 8));
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i + j * step * 8 < whole) f(i + j * step * 8, v[j]);
    }
    if (at == 0)
#pragma unroll 1
        for (int i = whole; i < end; ++i) g(i, (unsigned)row[i]);
}
// The vectors of columns that are kept in shared memory, and a last one that is not whole from the row itself.
template <typename F, typename G>
__device__ __forceinline__ void each_kept(const uint16_t *row, const uint4 *kept, int begin, int end, int at, int step, F f, G g) {
    const int n = (end - begin) >> 3;
#pragma unroll 2
    for (int i = at; i < n; i += step) f(begin + i * 8, kept[i]);
    if (at == 0)
#pragma unroll 1
        for (int i = begin + n * 8; i < end; ++i) g(i, (unsigned)row[i]);
}
// (where time matters less than the size of the code)
template <typename G>
__device__ __forceinline__ void each_column(const uint16_t *row, int end, G g) {
#pragma unroll 1
    for (int i = threadIdx.x; i < end; i += kThreads) g((unsigned)row[i]);
}

// What a CTA has of the order: the places that are not empty, as place << 18 | columns (a row has
// fewer than 2^18), an equal number of them to a thread, in a row.
struct Entries {
    unsigned *list;
    int n, window;  // window: -1, the one
    Sums before;    // sums ahead of them
};
__device__ __forceinline__ u64 weight_of(const Shared &s, unsigned entry, int window) {
    return weight62(s.scale, value_of(key_of_place((int)(entry >> 18), window)), s.pw);
}
__device__ __forceinline__ int each_of(int n) { return (n + kThreads - 1) / kThreads; }
constexpr unsigned kColumns = (1u << 18) - 1;
static_assert(LORA_MAX_VOCAB <= kColumns && kPlaces <= 1 << 14 && kWinBins <= 1 << 14, "an entry's parts");

// Writes the entries of the warps' groups, one warp's after the other's.  group(j): a warp's group number j, of
// `rounds`; four(j): the columns of this lane's four places of it.  `list` may be where the counts are.
template <int MAX, typename G, typename F>
__device__ __forceinline__ int write_entries(Shared &s, unsigned *list, int rounds, G group, F four) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4 c[MAX];
    unsigned some = 0;  // rounds in which the warp has any
    int mine = 0;
#pragma unroll
    for (int j = 0; j < MAX; ++j) {
        c[j] = j < rounds ? four(j) : make_uint4(0, 0, 0, 0);
        const int here = (c[j].x != 0) + (c[j].y != 0) + (c[j].z != 0) + (c[j].w != 0);
        mine += here;
        if (__any_sync(kAll, here)) some |= 1u << j;
    }
    mine = (int)__reduce_add_sync(kAll, (unsigned)mine);
    if (lane == 0) s.warp_n[warp] = mine;
    __syncthreads();  // (all counts have been read)
    const int all = s.warp_n[lane & 15], n = (int)__reduce_add_sync(kAll, lane < 16 ? (unsigned)all : 0u);
    int at = (int)__reduce_add_sync(kAll, lane < warp ? (unsigned)all : 0u);
#pragma unroll
    for (int j = 0; j < MAX; ++j) {
        if (!(some >> j & 1)) continue;
        const unsigned q[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
        const unsigned first = (unsigned)(group(j) * 128 + lane * 4);
        int to = at;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned some_k = __ballot_sync(kAll, q[k] != 0);
            to += __popc(some_k & ((1u << lane) - 1));
            at += __popc(some_k);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (q[k]) list[to++] = (first + k) << 18 | q[k];
    }
    __syncthreads();
    return n;
}

// The columns of four places of the one window: of 0 and ahead of it they come in descending order of the bins.
__device__ __forceinline__ int bin_of_places(int place) { return place < kMags ? kMags - 4 - place : place; }
__device__ __forceinline__ uint4 in_order(int place, uint4 v) { return place < kMags ? make_uint4(v.w, v.z, v.y, v.x) : v; }

__device__ __forceinline__ void put(Pre &pre, const Sums &before) {
    pre.hi[threadIdx.x] = (u64)(before.mass >> 64);
    pre.lo[threadIdx.x] = (u64)before.mass;
    pre.n[threadIdx.x] = (unsigned)before.n;
}

// Sums of the entries in `total`; returns those ahead of this thread's.  Of their beginning that weighs at
// least `least` a column in s.told.
__device__ __forceinline__ Sums add_up(Shared &s, const Entries &q, u64 least, Sums &total) {
    Sums much = {0, 0}, own = {0, 0};
    const int each = each_of(q.n), begin = min(q.n, (int)threadIdx.x * each), end = min(q.n, begin + each);
#pragma unroll 1
    for (int i = begin; i < end; ++i) {
        const unsigned entry = q.list[i];
        const int c = (int)(entry & kColumns);
        const u64 w = weight_of(s, entry, q.window);
        own.mass += (u128)w * (unsigned)c;
        own.n += c;
        if (w >= least) much = own;
    }
    const Sums before = scan(s, own, total);
    if (!least) return before;
    // the last thread that has some ends that beginning
    if (threadIdx.x == 0) s.last = -1, s.told.least_n = 0, s.told.least_hi = 0, s.told.least_lo = 0;
    __syncthreads();
    const unsigned some = __ballot_sync(kAll, much.n > 0);
    if (some && (threadIdx.x & 31) == 0) atomicMax(&s.last, (int)threadIdx.x + 31 - __clz(some));
    __syncthreads();
    if ((int)threadIdx.x == s.last) {
        much.mass += before.mass;
        much.n += before.n;
        s.told.least_hi = (u64)(much.mass >> 64);
        s.told.least_lo = (u64)much.mass;
        s.told.least_n = much.n;
    }
    return before;
}

// ------------------------------------------------------------ clusters

template <bool SHARE>
__device__ __forceinline__ void cluster_sync() {
    if (!SHARE) {
        __syncthreads();
        return;
    }
    bgmv::cluster_arrive();
    bgmv::cluster_wait();
}
__device__ __forceinline__ uint32_t peer_address(const void *local, int peer) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32_of(local)), "r"(peer));
    return a;
}
__device__ __forceinline__ unsigned load_peer(uint32_t a) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ u64 load_peer8(uint32_t a) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 load_peer4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
// A number of a CTA of the row.
template <bool SHARE>
__device__ __forceinline__ unsigned peers(const unsigned *local, int peer) {
    return SHARE ? load_peer(peer_address(local, peer)) : *(const volatile unsigned *)local;
}
template <bool SHARE>
__device__ __forceinline__ u64 peers(const u64 *local, int peer) {
    return SHARE ? load_peer8(peer_address(local, peer)) : *(const volatile u64 *)local;
}
// What every CTA of the row tells, in s.all.
template <bool SHARE>
__device__ __forceinline__ void hear(Shared &s, int C) {
    cluster_sync<SHARE>();  // all have told
    constexpr int kWords = sizeof(Told) / 4;
#pragma unroll 1
    for (int i = threadIdx.x; i < C * kWords; i += kThreads)
        ((unsigned *)s.all)[i] = peers<SHARE>((unsigned *)&s.told + i % kWords, i / kWords);
    __syncthreads();
}

// The first column of the order at which the sum of weights exceeds `mass`, or that is number `n`,
// whichever comes first, if it is among the entries of CTA `peer` (q.n of them at q.list, behind q.before).
// A warp's work: the thread that has it by two ballots over `pre`, then that thread's entries, one a lane.
template <bool SHARE>
__device__ __forceinline__ Found look(const Shared &s, const Pre &pre, const Entries &q, int peer, u128 mass, int n) {
    const int lane = threadIdx.x & 31, each = each_of(q.n);
    int who = lane < kWarps ? lane * 32 : 0, n0 = 0;
    u128 before = 0;
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
        before = q.before.mass + join(peers<SHARE>(&pre.hi[who], peer), peers<SHARE>(&pre.lo[who], peer));
        n0 = q.before.n + (int)peers<SHARE>(&pre.n[who], peer);
        const unsigned upto = __ballot_sync(kAll, before <= mass && n0 < n && (level || lane < kWarps));
        const int at = upto ? 31 - __clz(upto) : 0;  // (that of lane 0 always is)
        if (level) {
            before = join(__shfl_sync(kAll, (u64)(before >> 64), at), __shfl_sync(kAll, (u64)before, at));
            n0 = __shfl_sync(kAll, n0, at);
            who = who - lane + at;
        } else {
            who = at * 32 + lane;
        }
    }
    const int i = who * each + lane;
    const unsigned entry = lane < each && i < q.n ? peers<SHARE>(&q.list[i], peer) : 0u;
    const int c = (int)(entry & kColumns);
    const u64 w = c ? weight_of(s, entry, q.window) : 0ull;
    Sums sum = {(u128)w * (unsigned)c, c};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 h = __shfl_up_sync(kAll, (u64)(sum.mass >> 64), o), l = __shfl_up_sync(kAll, (u64)sum.mass, o);
        const int k = __shfl_up_sync(kAll, sum.n, o);
        if (lane >= o) {
            sum.mass += join(h, l);
            sum.n += k;
        }
    }
    sum.mass += before;
    sum.n += n0;
    const unsigned past = __ballot_sync(kAll, c && (sum.mass > mass || sum.n >= n));
    const int winner = past ? __ffs(past) - 1 : 0;
    Found f = {0, 0, 0, 0, 0};
    if (lane == winner) {
        const u128 m0 = sum.mass - (u128)w * (unsigned)c;
        const int k0 = sum.n - c, last = min(c, n - k0) - 1;
        // smallest r with m0 + (r + 1) w > mass, at most the number asked for: a quotient below 2^18, from fp32 to within one
        int r = last;
        if (sum.mass > mass) {
            const u128 gap = mass - m0;
            const int down = gap >> 64 ? 64 - __clzll((u64)(gap >> 64)) : 0;
            const float quotient = (float)(u64)(gap >> down) / (float)w * exp2f((float)down);
            r = quotient < (float)last ? (int)quotient : last;
            while (r > 0 && m0 + (u128)w * (unsigned)r > mass) --r;
            while (r < last && m0 + (u128)w * (unsigned)(r + 1) <= mass) ++r;
        }
        const u128 m = m0 + (u128)w * (unsigned)(r + 1);
        f.key = key_of_place((int)(entry >> 18), q.window);
        f.rank = r;
        f.n = k0 + r + 1;
        f.hi = (u64)(m >> 64);
        f.lo = (u64)m;
    }
    f.key = __shfl_sync(kAll, f.key, winner);
    f.rank = __shfl_sync(kAll, f.rank, winner);
    f.n = __shfl_sync(kAll, f.n, winner);
    f.hi = __shfl_sync(kAll, f.hi, winner);
    f.lo = __shfl_sync(kAll, f.lo, winner);
    return f;
}

// ------------------------------------------------------------ many windows (one CTA)

__device__ __noinline__ void count_window(Shared &s, const uint16_t *row, int V, int window) {
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < kWinBins; i += kThreads) s.bins[i] = 0;
    __syncthreads();
    each_column(row, V, [&](unsigned b) {
        const unsigned k = key_of(b);
        if (k && (int)(k / kWinBins) == window) atomicAdd(&s.bins[kWinBins - 1 - (k % kWinBins)], 1u);
    });
    __syncthreads();
}

__device__ __noinline__ void window_entries(Shared &s, Pre &pre, const uint16_t *row, int V, int window, u64 least, Entries &q, Sums &all) {
    count_window(s, row, V, window);
    constexpr int kPer = kWinBins / kThreads / 4;
    q.list = s.bins;
    q.window = window;
    const int own = (int)(threadIdx.x >> 5) * kPer;
    q.n = write_entries<kPer>(s, s.bins, kPer, [&](int j) { return own + j; },
                              [&](int j) { return *(const uint4 *)&s.bins[(own + j) * 128 + (int)(threadIdx.x & 31) * 4]; });
    put(pre, add_up(s, q, least, all));
}

__device__ __noinline__ void window_sums(Shared &s, Pre &pre, const uint16_t *row, int V, u64 least, Sums &total, Sums &heavy) {
    if (threadIdx.x < kWindows) s.coarse[threadIdx.x] = 0;
    __syncthreads();
    each_column(row, V, [&](unsigned b) {
        const unsigned k = key_of(b);
        if (k) atomicAdd(&s.coarse[k / kWinBins], 1);
    });
    __syncthreads();
    total = heavy = {0, 0};
#pragma unroll 1
    for (int w = kWindows - 1; w >= 0; --w) {
        Sums all = {0, 0};
        if (s.coarse[w]) {
            Entries q;
            window_entries(s, pre, row, V, w, least, q, all);
            __syncthreads();
            if (least && s.told.least_n) heavy = {total.mass + join(s.told.least_hi, s.told.least_lo), total.n + s.told.least_n};
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            s.win_hi[w] = (u64)(all.mass >> 64);
            s.win_lo[w] = (u64)all.mass;
            s.win_n[w] = all.n;
        }
        total.mass += all.mass;
        total.n += all.n;
    }
    __syncthreads();
}

// The window where a sum passes a bound, and its entries.
__device__ __noinline__ void window_of(Shared &s, Pre &pre, const uint16_t *row, int V, u128 mass, int n, Entries &q) {
    Sums at = {0, 0}, all;
    int w = kWindows - 1;
#pragma unroll 1
    for (; w > 0; --w) {
        const u128 m = at.mass + join(s.win_hi[w], s.win_lo[w]);
        if (m > mass || at.n + s.win_n[w] >= n) break;
        at.mass = m;
        at.n += s.win_n[w];
    }
    window_entries(s, pre, row, V, w, 0, q, all);
    q.before = at;
}

// floor(m * f) for 0 <= f < 1, and whether that is m * f itself.
__device__ __forceinline__ u128 times(u128 m, float f, bool &exact) {
    exact = true;
    if (!(f > 0.f)) return 0;
    int e;
    const float mant = frexpf(f, &e);  // f = mant 2^e, mant in [0.5, 1)
    const u128 product = m * (u128)(unsigned)(mant * 0x1p24f);
    const int shift = 24 - e;
    const u128 down = shift > 127 ? 0 : product >> shift;
    exact = shift <= 127 && down << shift == product;
    return down;
}

// A share of the largest weight, in units of 2^-62, from below.
__device__ __forceinline__ u64 share62(float f) {
    if (!(f > 0.f)) return 0ull;
    if (f >= 1.f) return 1ull << 62;
    const unsigned b = __float_as_uint(f), m = (b & 0x7fffffu) | 0x800000u;
    const int up = (int)(b >> 23) - 88;  // f = m 2^(exponent - 150)
    return up >= 0 ? (u64)m << up : up > -24 && b >> 23 ? (u64)(m >> -up) : 0ull;
}

// Adds the columns of a vector to the bins, which lie at `bins` in shared memory.
struct Counter {
    unsigned *bins;
    unsigned low = 0, odd = 0;
    __device__ __forceinline__ void add(unsigned address) {
        asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(address) : "memory");
    }
    __device__ __forceinline__ void rare(unsigned b) {  // outside of the counted range
        const unsigned mag = b & 0x7fffu;
        if (mag == 0u) atomicAdd(&bins[2 * kMags], 1u);
        else if (mag > 0x7f80u || b == 0xff80u) return;  // NaN, -inf
        else if ((b & 0x8000u) && mag > kMagLo) low = max(low, key_of(b));
        else odd = 1;
    }
    __device__ __forceinline__ void one(unsigned b) {
        const unsigned mag = b & 0x7fffu;
        if (mag - kMagLo < (unsigned)kMags) atomicAdd(&bins[(mag - kMagLo) | (b >> 2 & 0x2000u)], 1u);
        else rare(b);
    }
    __device__ __forceinline__ void eight(const uint4 &v) {
        static_assert(kMagLo == 0x2400 && kMags == 0x2000, "with 0x1c00 added the range is 0x4000 to 0x5fff");
        const unsigned base = smem_u32_of(bins);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t t[4], out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            t[k] = (w[k] & 0x7fff7fffu) + 0x1c001c00u;
            out[k] = (t[k] ^ 0x40004000u) & 0x60006000u;
        }
        // four times (magnitude | sign << 13)
        const auto lower = [&](int k) { return base + ((t[k] << 2 & 0x7ffcu) | (w[k] & 0x8000u)); };
        const auto upper = [&](int k) { return base + ((t[k] >> 14 & 0x7ffcu) | (w[k] >> 16 & 0x8000u)); };
        if (!(out[0] | out[1] | out[2] | out[3])) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                add(lower(k));
                add(upper(k));
            }
            return;
        }
        uint32_t odd_one = 0;  // halves outside of the range that are not -inf, as the halves' highest bits
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x = w[k] ^ 0xff80ff80u;
            odd_one |= (out[k] + 0x60006000u) & (((x & 0x7fff7fffu) + 0x7fff7fffu) | x) & 0x80008000u;
            if (!(out[k] & 0xffffu)) add(lower(k));
            if (!(out[k] >> 16)) add(upper(k));
        }
        if (odd_one)
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                const unsigned b = w[k >> 1] >> (k & 1) * 16 & 0xffffu;
                if ((b & 0x7fffu) - kMagLo >= (unsigned)kMags) rare(b);
            }
    }
};

__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32_of(to)), "l"(from) : "memory");
}

// How many of 8 columns count as the largest finite number: it or +inf (rare, and kept out of the way).
__device__ __noinline__ int eight_largest(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) n += (key_of(w[k] & 0xffffu) == kKeyMax) + (key_of(w[k] >> 16) == kKeyMax);
    return n;
}

// SHARE: CTAs share a row (p.C of them; otherwise one has it).  KEEP: a CTA keeps its part of the row in shared memory; others run two to an
// SM, with 64 registers a thread (two of those that share a row are spilled).
template <bool SHARE, bool KEEP>
__global__ void __launch_bounds__(kThreads, KEEP ? 1 : 2) sample_kernel(const SampleArgs p) {
    extern __shared__ __align__(16) char smem[];
    Shared &s = *(Shared *)smem;
    const int C = SHARE ? p.C : 1, c = SHARE ? (int)bgmv::cluster_rank() : 0;
    unsigned *const extra = (unsigned *)(smem + kExtra);
    Pre &pre = *(Pre *)(C == 2 ? s.bins + kPlaces / 2 : SHARE ? extra + kPlaces / C : extra);
    const int t = (int)blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint16_t *row = p.logits + (long long)t * p.ld;
    asm volatile("griddepcontrol.launch_dependents;");
    fill_powers(s.pw);
    if (tid == 0) s.told.low = 0, s.told.odd = 0, s.told.top = kPlaces;
#pragma unroll 1
    for (int i = tid; i < kBins; i += kThreads) s.bins[i] = 0;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const float temperature = p.temperature ? p.temperature[t] : 1.f;
    const bool greedy = !(temperature > 0.f);
    const float min_p = p.min_p ? p.min_p[t] : 0.f, top_p = p.top_p ? p.top_p[t] : 1.f, u = p.uniform ? p.uniform[t] : 0.f;
    const int top_k = p.top_k ? p.top_k[t] : 0;

    // counts of this CTA's part of the row
    const int part = ((p.V + C - 1) / C + 7) & ~7, begin = min(p.V, c * part), end = min(p.V, begin + part);
    Counter counter;
    counter.bins = s.bins;
    uint4 *const kept = (uint4 *)(smem + kExtra + extra_bytes(C));
    if (KEEP) {
        // a thread copies and counts the same vectors, in two halves
        const int n = (end - begin) >> 3, half = n >> 1;
#pragma unroll 1
        for (int i = tid; i < half; i += kThreads) copy16(&kept[i], row + begin + i * 8);
        asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 1
        for (int i = half + tid; i < n; i += kThreads) copy16(&kept[i], row + begin + i * 8);
        asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            if (h) asm volatile("cp.async.wait_group 0;" ::: "memory");
            else asm volatile("cp.async.wait_group 1;" ::: "memory");
            const int to = h ? n : half;
#pragma unroll 2
            for (int i = (h ? half : 0) + tid; i < to; i += kThreads) counter.eight(kept[i]);
        }
        if (tid == 0)
#pragma unroll 1
            for (int i = begin + n * 8; i < end; ++i) counter.one((unsigned)row[i]);
    } else {
        each_vector<2>(row, begin, end, tid, kThreads, [&](int, const uint4 &v) { counter.eight(v); }, [&](int, unsigned b) { counter.one(b); });
    }
    const unsigned low = __reduce_max_sync(kAll, counter.low);
    if (lane == 0 && low) atomicMax(&s.told.low, low);
    if (__any_sync(kAll, counter.odd) && lane == 0) s.told.odd = 1;
    __syncthreads();
    if (tid == 0) {
        if (s.bins[0]) s.told.odd = 1;  // +2^-55, whose place is that of 0
        s.bins[0] = s.bins[2 * kMags];
    }
    __syncthreads();
    const u64 least = greedy ? 0ull : share62(min_p);
    if (tid == 0) s.scale = begin_scale(greedy ? 1.f : temperature);
    unsigned lowest = s.told.low;
    int odd = s.told.odd, top = kPlaces;
    int n_groups = kGroups;
    if (SHARE) {
        // Most groups of places are empty: those that are not are found, and shared out.
        unsigned some = 0;
#pragma unroll 4
        for (int j = 0; j < kRounds; ++j) {
            const int place = (warp * kRounds + j) * 128 + lane * 4;
            const uint4 v = in_order(place, *(const uint4 *)&s.bins[bin_of_places(place)]);
            const unsigned lanes = __ballot_sync(kAll, (v.x | v.y | v.z | v.w) != 0);
            if (lanes && !some && lane == __ffs(lanes) - 1) atomicMin(&s.told.top, place + (v.x ? 0 : v.y ? 1 : v.z ? 2 : 3));
            some |= (lanes ? 1u : 0u) << j;
        }
        if (lane == 0) s.told.some[warp] = (uint8_t)some;
        hear<SHARE>(s, C);
        bool mine = false;  // group `tid` has any
#pragma unroll 1
        for (int k = 0; k < C; ++k) {
            const Told &o = s.all[k];
            top = min(top, o.top);
            lowest = max(lowest, o.low);
            odd |= o.odd;
            if (tid < kGroups) mine |= o.some[tid / kRounds] >> tid % kRounds & 1;
        }
        if (warp < kGroups / 32) {
            const unsigned bits = __ballot_sync(kAll, mine);
            if (lane == 0) s.groups[warp] = bits;
        }
        __syncthreads();
        n_groups = 0;
        int ahead = 0;
#pragma unroll
        for (int k = 0; k < kGroups / 32; ++k) {
            if (k < warp) ahead += __popc(s.groups[k]);
            if (k == warp) ahead += __popc(s.groups[k] & ((1u << lane) - 1));
            n_groups += __popc(s.groups[k]);
        }
        if (mine) s.group_at[ahead] = (uint8_t)tid;
        __syncthreads();
    }
    Entries entries;
    {
        const int g0 = c * n_groups / C, few = (c + 1) * n_groups / C - g0;
        const int w0 = few * warp / kWarps, rounds = few * (warp + 1) / kWarps - w0;
        unsigned *const list = SHARE ? extra : s.bins;
        const auto group = [&](int j) { return SHARE ? (int)s.group_at[g0 + w0 + j] : w0 + j; };
        if (SHARE) {
            // the counts of all parts
#pragma unroll 1
            for (int j = 0; j < rounds; ++j) {
                const int place = group(j) * 128 + lane * 4, bin = bin_of_places(place);
                uint4 sum = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kMostCtas; ++k)
                    if (k < C) {
                        const uint4 v = load_peer4(peer_address(&s.bins[bin], k));
                        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                    }
                *(uint4 *)&list[(w0 + j) * 128 + lane * 4] = in_order(place, sum);
            }
        }
        entries.list = list;
        entries.window = -1;
        entries.before = {0, 0};
        entries.n = write_entries<kRounds>(s, list, rounds, group, [&](int j) {
            const int place = group(j) * 128 + lane * 4;
            return SHARE ? *(const uint4 *)&list[(w0 + j) * 128 + lane * 4] : in_order(place, *(const uint4 *)&list[bin_of_places(place)]);
        });
        if (!SHARE && entries.n) top = (int)(list[0] >> 18);
    }
    if (tid == 0 && top < kPlaces) end_scale(s.scale, value_of(key_of_place(top, -1)));
    __syncthreads();
    // The one window is enough if nothing lies outside of it but numbers too low to weigh anything.
    bool one = !odd && top < kPlaces;
    if (one) one = lowest == 0 || weight62(s.scale, value_of(lowest), s.pw) == 0;
    Sums total, heavy = {0, 0};
    if (!one) {
        // the first CTA does the row alone
        cluster_sync<SHARE>();  // (and is no longer read by the others)
        if (c) return;
        unsigned key = 0;
        each_column(row, p.V, [&](unsigned b) { key = max(key, key_of(b)); });
        key = __reduce_max_sync(kAll, key);
        if (lane == 0) s.warp_n[warp] = (int)key;
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) key = max(key, (unsigned)s.warp_n[w]);
        if (key == 0) {  // nothing to choose from
            if (tid == 0) {
                p.tokens[t] = -1;
                if (p.logprobs) p.logprobs[t] = -INFINITY;
            }
            return;
        }
        if (tid == 0) {
            s.scale = begin_scale(greedy ? 1.f : temperature);
            end_scale(s.scale, value_of(key));
        }
        window_sums(s, pre, row, p.V, least, total, heavy);
    } else {
        const Sums before = add_up(s, entries, least, total);
        if (C != 2) put(pre, before);
        if (tid == 0) {
            s.told.hi = (u64)(total.mass >> 64);
            s.told.lo = (u64)total.mass;
            s.told.n = total.n;
            s.told.entries = entries.n;
        }
        hear<SHARE>(s, C);
        if (C == 2) {
            // (nobody reads the counts any more)
            put(pre, before);
            cluster_sync<SHARE>();
        }
        total = {0, 0};
#pragma unroll 1
        for (int k = 0; k < C; ++k) {
            const Told &o = s.all[k];
            if (least && o.least_n) heavy = {total.mass + join(o.least_hi, o.least_lo), total.n + o.least_n};
            total.mass += join(o.hi, o.lo);
            total.n += o.n;
        }
    }
    // What is kept is n columns that weigh `mass`: by top-k, by top-p, by min-p.  The last step is the draw.
    // With the one window the first warp of every CTA takes these steps for itself.
    if (!one || warp == 0) {
        int n = total.n;
        u128 mass = total.mass;
        if (greedy) {
            n = 1;
            mass = (u128)1 << 62;
        }
        const float draw = u < 1.f ? u : u >= 1.f ? 0x1.fffffep-1f : 0.f;
        Found f;
#pragma unroll 1
        for (int step = greedy ? 2 : 0; step < 3; ++step) {
            u128 bound = ~(u128)0;  // the column at which sums exceed it
            int most = n;           // ... or which is this one
            if (step == 0) {
                if (top_k < 1 || top_k >= n) continue;
                most = top_k;
            } else {
                if (step == 1 && !(top_p < 1.f)) continue;
                if (step == 2 && least && heavy.n < n) {
                    most = heavy.n;
                    mass = heavy.mass;
                }
                bool exact;
                bound = times(mass, step == 1 ? top_p : draw, exact);
                // a share of the weight has to be reached: the next integer below exceeded
                if (step == 1 && exact && bound) --bound;
            }
            int peer = c;
            if (!one) {
                window_of(s, pre, row, p.V, bound, most, entries);
                __syncthreads();
            } else {
                Sums upto = {0, 0};
#pragma unroll 1
                for (int k = 0; k < C; ++k) {
                    peer = k;
                    entries.before = upto;
                    entries.n = s.all[k].entries;
                    upto.mass += join(s.all[k].hi, s.all[k].lo);
                    upto.n += s.all[k].n;
                    if (upto.mass > bound || upto.n >= most) break;
                }
            }
            f = look<SHARE>(s, pre, entries, peer, bound, most);
            n = f.n;
            mass = join(f.hi, f.lo);
            if (!one) __syncthreads();
        }
        if (tid == 0) s.found = f;
    }
    __syncthreads();

    // which column that is: number `rank` of those with the found key.  A warp's columns follow each other.
    const unsigned key = s.found.key;
    const int rank = s.found.rank;
    const int from = one ? begin : 0, to = one ? end : p.V;
    const int chunk = ((to - from + kWarps - 1) / kWarps + 255) & ~255;
    const int w0 = min(to, from + warp * chunk), w1 = min(to, w0 + chunk);
    const unsigned bits = key == 0x8000u ? 0u : __float_as_uint(value_of(key)) >> 16, both = bits | bits << 16;
    const unsigned signs = key == 0x8000u ? 0x7fff7fffu : 0xffffffffu;  // -0 is 0
    const bool largest = key == kKeyMax;                                // +inf counts as that, too
    // how many of 8 columns have it
    const auto matches = [&](const uint4 &v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        int n = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x = (w[k] ^ both) & signs;
            n += __popc(~(((x & 0x7fff7fffu) + 0x7fff7fffu) | x) & 0x80008000u);  // halves of 0
        }
        if (largest) n = eight_largest(v);
        return n;
    };
    int found = 0;
    const bool here = KEEP && one;
    if (here)
        each_kept(row, kept + ((w0 - begin) >> 3), w0, w1, lane, 32, [&](int, const uint4 &v) { found += matches(v); },
                  [&](int, unsigned b) { found += key_of(b) == key; });
    else
        each_vector<4>(row, w0, w1, lane, 32, [&](int, const uint4 &v) { found += matches(v); }, [&](int, unsigned b) { found += key_of(b) == key; });
    found = (int)__reduce_add_sync(kAll, (unsigned)found);
    __syncthreads();
    if (lane == 0) s.warp_n[warp] = found;
    __syncthreads();
    int ahead = 0;
    if (SHARE && one) {
        if (tid == 0) {
            int sum = 0;
#pragma unroll 1
            for (int w = 0; w < kWarps; ++w) sum += s.warp_n[w];
            s.told.matches = sum;
        }
        hear<SHARE>(s, C);
#pragma unroll 1
        for (int k = 0; k < c; ++k) ahead += s.all[k].matches;
        cluster_sync<SHARE>();  // nobody is read any more
    }
    ahead += (int)__reduce_add_sync(kAll, lane < warp ? (unsigned)s.warp_n[lane] : 0u);
    if (ahead > rank || rank >= ahead + found) return;
    // the warp's columns again, 256 at a time, from L1 or L2
    int found_at = -1;
#pragma unroll 1
    for (int i = w0; i < w1; i += 256) {
        const int at = i + lane * 8, few = min(8, w1 - at);
        uint4 v = make_uint4(0, 0, 0, 0);
        int n = 0;
        if (few == 8) {
            v = here ? kept[(at - begin) >> 3] : __ldg((const uint4 *)(row + at));
            n = matches(v);
        } else {
#pragma unroll 1
            for (int k = 0; k < few; ++k) n += key_of(row[at + k]) == key;
        }
        const int all = (int)__reduce_add_sync(kAll, (unsigned)n);
        if (rank >= ahead + all) {
            ahead += all;
            continue;
        }
        int upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int k = __shfl_up_sync(kAll, upto, o);
            if (lane >= o) upto += k;
        }
        ahead += upto - n;  // ahead of this lane's columns
        if (ahead <= rank && rank < ahead + n)
#pragma unroll 1
            for (int k = 0; k < few; ++k)
                if (key_of(row[at + k]) == key && ahead++ == rank) found_at = at + k;
        break;
    }
    if (found_at < 0) return;
    p.tokens[t] = found_at;
    if (p.logprobs) {
        float hi, lo;
        distance(s.scale, value_of(key), hi, lo);
        // ln of the sum, whose largest weight is 2^62, one: accurate where the others are little, too
        constexpr float kLn2 = 0.6931471805599453f, kLn2Rest = (float)(0.6931471805599453 - (double)kLn2);
        const u128 others = total.mass - ((u128)1 << 62);
        const int down = others >> 64 ? 64 - __clzll((u64)(others >> 64)) : 0;
        const float sum = log1pf(ldexpf((float)(u64)(others >> down), down - 62));
        p.logprobs[t] = -fmaf(hi, kLn2, fmaf(hi, kLn2Rest, fmaf(lo, kLn2, sum)));
    }
}

// CTAs that share a row: as many as all find room at once, two to an SM, of 12000 columns at least; a short
// row is not shared, as the cluster's barriers and what goes around take 3 us (one row, by 1, 2, 4 and 8 CTAs:
// of 4000 columns 10.0, 13.2, 13.4 and 13.9 us, of 32007 15.3, 16.4, 15.8 and 15.7, of 128256 27.9, 23.3, 17.6 and 15.9).
int ctas_of_a_row(int T, int V, int sms) {
    int C = 1;
    if (V < 40000) return C;
    while (C < kMostCtas && (long long)T * C * 2 <= 2LL * sms && V >= C * 2 * 12000) C *= 2;
    return C;
}

constexpr int kMostSmem = 227 * 1024;  // of a CTA
// A row's part in shared memory: one CTA to an SM, so only where all rows find room at once.  It is read
// once, and more of it at a time (64 rows of 32007 columns 19.2 -> 16.3 us, one 18.0 -> 16.8, with all filters).
// Half as many CTAs to a row that have that room are faster than all without it (18 rows of 128256 columns by four
// 18.5 us, by eight 22.4; 64 of 100000 by two 21.6, by four 25.9).
struct Device {
    std::atomic<int> sms;  // 0: not looked up yet
    int rooms[4];          // clusters of 1, 2, 4 and 8 such CTAs that run at once
};
Device g_devices[64];

size_t part_of(int V, int C) { return (size_t)((lora_ceil_div(V, C) + 7) & ~7); }
bool kept(const Device &d, int T, int V, int C) {
    return kExtra + extra_bytes(C) + part_of(V, C) * 2 <= (size_t)kMostSmem && T <= d.rooms[C == 1 ? 0 : C == 2 ? 1 : C == 4 ? 2 : 3];
}

void configure(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *at, int T, int C, size_t smem, cudaStream_t stream) {
    memset(&cfg, 0, sizeof(cfg));
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 2 : 1;
    cfg.gridDim = dim3((unsigned)T * (unsigned)C, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
}

template <bool SHARE, bool KEEP>
cudaError_t set_smem() {
    return cudaFuncSetAttribute(sample_kernel<SHARE, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, KEEP ? kMostSmem : (int)(kExtra + extra_bytes(2)));
}

// What the current device has; looked up once (the kernels' attributes are set on the way).
cudaError_t device_of(Device *&d) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    d = &g_devices[dev];
    if (d->sms.load(std::memory_order_acquire)) return cudaSuccess;
    int sms = 0, rooms[4];
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = set_smem<false, false>()) != cudaSuccess || (e = set_smem<false, true>()) != cudaSuccess ||
        (e = set_smem<true, false>()) != cudaSuccess || (e = set_smem<true, true>()) != cudaSuccess)
        return e;
    rooms[0] = sms;
    for (int i = 1; i < 4; ++i) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute at[2];
        configure(cfg, at, 1, 1 << i, kMostSmem, nullptr);
        if ((e = cudaOccupancyMaxActiveClusters(&rooms[i], sample_kernel<true, true>, &cfg)) != cudaSuccess) return e;
    }
    static std::mutex lock;
    std::lock_guard<std::mutex> hold(lock);
    if (d->sms.load(std::memory_order_relaxed)) return cudaSuccess;
    for (int i = 0; i < 4; ++i) d->rooms[i] = rooms[i];
    d->sms.store(sms, std::memory_order_release);
    return cudaSuccess;
}

}  // namespace

extern "C" lora_status_t lora_sample(const void *logits, int64_t ld, int32_t T, int32_t vocab_size,
                                     const float *temperature, const int32_t *top_k, const float *top_p,
                                     const float *min_p, const float *uniform, int32_t *tokens, float *logprobs,
                                     void *stream) {
    if (T < 0) return LORA_ERR_INVALID_ARG;
    if (vocab_size < 1 || vocab_size > LORA_MAX_VOCAB) return LORA_ERR_SHAPE;
    if (ld < vocab_size || ld % 8) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    if (T > 0x7fffffff / kMostCtas) return LORA_ERR_INVALID_ARG;
    if (!logits || !tokens || !lora_aligned16(logits) ||
        (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)uniform |
          (uintptr_t)tokens | (uintptr_t)logprobs) & 3))
        return LORA_ERR_INVALID_ARG;
    Device *dev = nullptr;
    LORA_CUDA_TRY(device_of(dev));
    SampleArgs p;
    p.logits = (const uint16_t *)logits;
    p.ld = ld;
    p.T = T;
    p.V = vocab_size;
    p.C = ctas_of_a_row(T, vocab_size, dev->sms);
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.uniform = uniform;
    p.tokens = tokens;
    p.logprobs = logprobs;
    if (!kept(*dev, T, vocab_size, p.C) && p.C > 1 && kept(*dev, T, vocab_size, p.C / 2)) p.C /= 2;
    const bool keep = kept(*dev, T, vocab_size, p.C);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at[2];
    configure(cfg, at, T, p.C, kExtra + extra_bytes(p.C) + (keep ? part_of(vocab_size, p.C) * 2 : 0), (cudaStream_t)stream);
    if (p.C > 1)
        LORA_CUDA_TRY(keep ? cudaLaunchKernelEx(&cfg, sample_kernel<true, true>, p) : cudaLaunchKernelEx(&cfg, sample_kernel<true, false>, p));
    else
        LORA_CUDA_TRY(keep ? cudaLaunchKernelEx(&cfg, sample_kernel<false, true>, p) : cudaLaunchKernelEx(&cfg, sample_kernel<false, false>, p));
    lora_note_launch();
    return LORA_OK;
}
