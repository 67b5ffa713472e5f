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
// addresses; columns outside of the counted range (masked ones, zeros) leave that path by eights.
// A cluster of up to 8 CTAs shares a row: each counts its part, the counts are added up by slices
// over distributed shared memory, and sums before a slice go around with a cluster barrier.
//
// Keys are bf16 bits mapped to integers that grow with the value.  A window is a
// range of keys that is counted at once:
//   one     the keys of 0 and of magnitudes in [2^-23, 2^9), 8193 bins: all that
//           takes part in most rows
//   many    otherwise 16 windows of 4096 keys each, in descending order, each
//           counted when it is asked for, by the first CTA of the cluster alone
#include <math.h>
#include <string.h>

#include <atomic>

#include "lora_internal.cuh"
#include "mma_common.cuh"

namespace {

typedef unsigned long long u64;
typedef unsigned __int128 u128;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMagLo = 104 * 128, kMags = 32 * 128;  // magnitudes [2^-23, 2^9) as bf16 bits
constexpr int kBins = 2 * kMags + 1;
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

// Places of the one window, in descending order of values: positive magnitudes, 0, negative ones.
// Its bins lie by their bits instead: magnitude, the sign above it, 0 last.
__device__ __forceinline__ int bin_of_place(int place) {
    return place < kMags ? kMags - 1 - place : place == kMags ? 2 * kMags : place - 1;
}
__device__ __forceinline__ unsigned key_of_place(int place, int window) {
    if (window >= 0) return (unsigned)(window * kWinBins + kWinBins - 1 - place);
    if (place == kMags) return 0x8000u;
    return place < kMags ? 0x8000u | (unsigned)(kMagLo + kMags - 1 - place) : 0x7fffu - (unsigned)(kMagLo + place - kMags - 1);
}

// 2^(-2^-j) for j = 1..18 in units of 2^-63, and ln 2 in units of 2^-64.
__device__ const u64 kRoots[18] = {0x5a827999fcef3242ull, 0x6ba27e656b4eb57aull, 0x75606373ee921c97ull,
                                   0x7a92be8a92436616ull, 0x7d41d96db915019dull, 0x7e9f06067a4360baull,
                                   0x7f4f08ae3dc7c426ull, 0x7fa765aca88f6453ull, 0x7fd3ab290e46d769ull,
                                   0x7fe9d3a8e07bf086ull, 0x7ff4e9597bed93abull, 0x7ffa748dff8dc61full,
                                   0x7ffd3a3f50020332ull, 0x7ffe9d1dbc0a75aaull, 0x7fff4e8e6306ed59ull,
                                   0x7fffa74712c3cdfdull, 0x7fffd3a381b1fa29ull, 0x7fffe9d1beed018aull};
constexpr u64 kOne63 = 1ull << 63;
constexpr u64 kLn2 = 0xb17217f7d1cf79acull;

__device__ __forceinline__ u64 mul63(u64 a, u64 b) { return __umul64hi(a, b) << 1; }

// The factors 2^(-i / 64), 2^(-i / 4096) and 2^(-i / 2^18), i < 64, of weight62.
__device__ __forceinline__ void fill_powers(u64 *pw) {
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
};

// With c = log2(e) / temperature = m 2^e, m in [1, 2): logits times 2^e, and m.  Where that
// would make the largest logit exceed 2^100, a smaller power does: distinct logits are then
// at least 2^91 apart, and every weight but the largest is 0 whatever the factor.
__device__ __forceinline__ Scale make_scale(float temperature, float top) {
    Scale r;
    int s = -2;
    double c = 0.0;
    if (temperature < INFINITY) {
        c = 1.4426950408889634 / (double)temperature;
        s = max(-126, min(126, ilogb(c)));
        if (top != 0.f) s = min(s, 100 - ilogbf(top));
        c = fmin(ldexp(c, -s), 0x1p30);
    }
    r.up = __int_as_float((s + 127) << 23);
    r.hi = (float)c;
    r.lo = (float)(c - (double)r.hi);
    r.top = top * r.up;
    return r;
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
// cubic term is below 2^-56).
__device__ __forceinline__ u64 weight62(const Scale &c, float v, const u64 *pw) {
    float hi, lo;
    distance(c, v, hi, lo);
    if (!(hi < 62.f)) return 0ull;
    long long y = __float2ll_rn(hi * 0x1p50f) + __float2ll_rn(lo * 0x1p50f);
    y = y < 0 ? 0 : y;
    const u64 f = (u64)y & ((1ull << 50) - 1);
    const u64 q = __umul64hi((f & 0xffffffffull) << 14, kLn2);  // r ln 2 in units of 2^-64
    u64 w = kOne63 - (q >> 1) + (__umul64hi(q, q) >> 2);
    w = mul63(w, pw[f >> 44]);
    w = mul63(w, pw[64 + ((f >> 38) & 63)]);
    w = mul63(w, pw[128 + ((f >> 32) & 63)]);
    return w >> (1 + (int)(y >> 50));
}

struct Found {
    unsigned key;
    int rank, n;  // which of the key's columns; columns up to and with it
    u64 lo, hi;   // ... and their weight
};

struct Sums {
    u128 mass;
    int n;
};

// What a CTA tells the others of its row.
struct Told {
    int top;       // first place that is not empty
    unsigned low;  // largest key below the one window
    int odd;       // a key in the gaps of the one window, or above it
    u64 lo, hi, least_lo, least_hi;  // weight of its slice, and of the weights of at least min_p in it
    int n, least_n;
    int matches;   // columns of its part with the chosen key
};

struct Shared {
    unsigned bins[kBins + 7];                   // by bits; or a window's in descending order
    unsigned merged[(kBins / 2 + kThreads) / kThreads * kThreads + kThreads];  // a slice's counts of all CTAs, two CTAs at least
    u64 pw[192];
    u64 warp_lo[kWarps], warp_hi[kWarps];  // 128-bit partial sums
    int warp_n[kWarps];
    Told told;
    Told all[kMostCtas];  // of every CTA
    Found found;
    Scale scale;
    // many windows
    int coarse[kWindows];
    u64 win_lo[kWindows], win_hi[kWindows];
    int win_n[kWindows];
};

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
    Sums before = {0, 0};
    total = {0, 0};
    for (int w = 0; w < kWarps; ++w) {
        const u128 m = join(s.warp_hi[w], s.warp_lo[w]);
        if (w < warp) {
            before.mass += m;
            before.n += s.warp_n[w];
        }
        total.mass += m;
        total.n += s.warp_n[w];
    }
    before.mass += inc.mass - mine.mass;
    before.n += inc.n - mine.n;
    return before;
}

// A row's columns from `begin` on, 8 at a time: f(column, its 8 bits' words), and g(column, bits) for
// those of a last vector that is not whole.
template <typename F, typename G>
__device__ __forceinline__ void each_vector(const uint16_t *row, int begin, int end, int at, int step, F f, G g) {
    constexpr int kAhead = 4;
    const int whole = begin + ((end - begin) & ~7);
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
        for (int i = whole; i < end; ++i) g(i, (unsigned)row[i]);
}
template <typename G>
__device__ __forceinline__ void each_column(const uint16_t *row, int begin, int end, int at, int step, G g) {
    each_vector(row, begin, end, at, step,
                [&](int i, const uint4 &v) {
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) g(i + k, u[k >> 1] >> (k & 1) * 16 & 0xffffu);
                },
                g);
}

// Counts of a slice: places [first, first + per) are this thread's, in descending order.
struct Slice {
    const unsigned *counts;
    int base, window;  // merged counts start at place `base`; -1: bins by bits
    bool by_bits;
    __device__ __forceinline__ unsigned count(int place) const {
        if (!by_bits) return counts[place - base];
        return place < kBins ? counts[bin_of_place(place)] : 0u;
    }
    __device__ __forceinline__ u64 weight(const Shared &s, int place) const {
        return weight62(s.scale, value_of(key_of_place(place, window)), s.pw);
    }
};

// Sums over a thread's places, and over those of them that weigh at least `least`.
__device__ __forceinline__ void add_up(const Shared &s, const Slice &q, int first, int per, u64 least, Sums &sum, Sums &heavy) {
    sum = heavy = {0, 0};
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const unsigned c = q.count(first + i);
        if (!c) continue;
        const u64 w = q.weight(s, first + i);
        const u128 m = (u128)w * c;
        sum.mass += m;
        sum.n += (int)c;
        if (w >= least) {
            heavy.mass += m;
            heavy.n += (int)c;
        }
    }
}

// The first column of the order at which the sum of weights exceeds `mass`, or that is number `n`,
// whichever comes first, if it lies within this thread's places (`before`: sums ahead of them,
// `own`: theirs).  The thread's warp looks through its places, one a lane.
__device__ __forceinline__ bool look(const Shared &s, const Slice &q, int first, int per, Sums before, const Sums &own, u128 mass, int n,
                                     Found &out) {
    const int lane = threadIdx.x & 31;
    const bool here = before.mass <= mass && before.n < n && (before.mass + own.mass > mass || before.n + own.n >= n);
    const unsigned who = __ballot_sync(kAll, here);
    if (!who) return false;
    const int owner = __ffs(who) - 1;
    first = __shfl_sync(kAll, first, owner);
    const u64 hi = __shfl_sync(kAll, (u64)(before.mass >> 64), owner), lo = __shfl_sync(kAll, (u64)before.mass, owner);
    const int n0 = __shfl_sync(kAll, before.n, owner);
    const unsigned c = lane < per ? q.count(first + lane) : 0u;
    const u64 w = c ? q.weight(s, first + lane) : 0ull;
    Sums sum = {(u128)w * c, (int)c};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 h = __shfl_up_sync(kAll, (u64)(sum.mass >> 64), o), l = __shfl_up_sync(kAll, (u64)sum.mass, o);
        const int k = __shfl_up_sync(kAll, sum.n, o);
        if (lane >= o) {
            sum.mass += join(h, l);
            sum.n += k;
        }
    }
    sum.mass += join(hi, lo);
    sum.n += n0;
    const unsigned past = __ballot_sync(kAll, c && (sum.mass > mass || sum.n >= n));
    if (lane != __ffs(past) - 1) return false;
    const u128 m0 = sum.mass - (u128)w * c;
    const int k0 = sum.n - (int)c;
    // smallest r with m0 + (r + 1) w > mass, bounded by the number asked for
    int a = 0, b = min((int)c, n - k0) - 1;
    while (a < b) {
        const int mid = (a + b) >> 1;
        if (m0 + (u128)w * (unsigned)(mid + 1) > mass) b = mid;
        else a = mid + 1;
    }
    const u128 m = m0 + (u128)w * (unsigned)(a + 1);
    out.key = key_of_place(first + lane, q.window);
    out.rank = a;
    out.n = k0 + a + 1;
    out.hi = (u64)(m >> 64);
    out.lo = (u64)m;
    return true;
}

// ------------------------------------------------------------ many windows (one CTA)

__device__ __noinline__ void count_window(Shared &s, const uint16_t *row, int V, int window) {
    __syncthreads();
    for (int i = threadIdx.x; i < kWinBins; i += kThreads) s.bins[i] = 0;
    __syncthreads();
    each_column(row, 0, V, threadIdx.x, kThreads, [&](int, unsigned b) {
        const unsigned k = key_of(b);
        if (k && (int)(k / kWinBins) == window) atomicAdd(&s.bins[kWinBins - 1 - (k % kWinBins)], 1u);
    });
    __syncthreads();
}

__device__ __noinline__ void window_sums(Shared &s, const uint16_t *row, int V, u64 least, Sums &total, Sums &heavy) {
    constexpr int kPer = kWinBins / kThreads;
    if (threadIdx.x < kWindows) s.coarse[threadIdx.x] = 0;
    __syncthreads();
    each_column(row, 0, V, threadIdx.x, kThreads, [&](int, unsigned b) {
        const unsigned k = key_of(b);
        if (k) atomicAdd(&s.coarse[k / kWinBins], 1);
    });
    __syncthreads();
    total = heavy = {0, 0};
    for (int w = kWindows - 1; w >= 0; --w) {
        Sums all = {0, 0}, some = {0, 0};
        if (s.coarse[w]) {
            count_window(s, row, V, w);
            Sums own, much;
            add_up(s, {s.bins, 0, w, false}, threadIdx.x * kPer, kPer, least, own, much);
            scan(s, own, all);
            scan(s, much, some);
        }
        if (threadIdx.x == 0) {
            s.win_hi[w] = (u64)(all.mass >> 64);
            s.win_lo[w] = (u64)all.mass;
            s.win_n[w] = all.n;
        }
        total.mass += all.mass;
        total.n += all.n;
        heavy.mass += some.mass;
        heavy.n += some.n;
    }
    __syncthreads();
}

__device__ __noinline__ void find_by_windows(Shared &s, const uint16_t *row, int V, u128 mass, int n) {
    constexpr int kPer = kWinBins / kThreads;
    Sums at = {0, 0};
    int w = kWindows - 1;
    for (; w > 0; --w) {
        const u128 m = at.mass + join(s.win_hi[w], s.win_lo[w]);
        if (m > mass || at.n + s.win_n[w] >= n) break;
        at.mass = m;
        at.n += s.win_n[w];
    }
    count_window(s, row, V, w);
    const Slice q = {s.bins, 0, w, false};
    Sums own, unused, total;
    add_up(s, q, threadIdx.x * kPer, kPer, 0, own, unused);
    Sums before = scan(s, own, total);
    before.mass += at.mass;
    before.n += at.n;
    Found f;
    if (look(s, q, threadIdx.x * kPer, kPer, before, own, mass, n, f)) s.found = f;
    __syncthreads();
}

// ------------------------------------------------------------ clusters

__device__ __forceinline__ void cluster_sync(int C) {
    if (C == 1) {
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
__device__ __forceinline__ void store_peer(uint32_t a, unsigned v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
// What every CTA of the row tells, in s.all.
__device__ __forceinline__ void hear(Shared &s, int C) {
    cluster_sync(C);  // all have told
    constexpr int kWords = sizeof(Told) / 4;
    for (int i = threadIdx.x; i < C * kWords; i += kThreads)
        ((unsigned *)s.all)[i] = C == 1 ? ((unsigned *)&s.told)[i] : load_peer(peer_address((unsigned *)&s.told + i % kWords, i / kWords));
    __syncthreads();
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

// Adds the columns of a vector to the bins, which lie at `bins` in shared memory.
struct Counter {
    unsigned *bins;
    unsigned low = 0, odd = 0;
    __device__ __forceinline__ void add(unsigned address) {
        asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(address) : "memory");
    }
    __device__ __forceinline__ void one(unsigned b) {
        const unsigned mag = b & 0x7fffu;
        if (mag - kMagLo < (unsigned)kMags) atomicAdd(&bins[(mag - kMagLo) | (b >> 3 & 0x1000u)], 1u);
        else if (mag == 0u) atomicAdd(&bins[2 * kMags], 1u);
        else if (mag > 0x7f80u || b == 0xff80u) return;  // NaN, -inf
        else if ((b & 0x8000u) && mag > kMagLo) low = max(low, key_of(b));
        else odd = 1;
    }
    __device__ __forceinline__ void eight(const uint4 &v) {
        static_assert(kMagLo == 0x3400 && kMags == 0x1000, "the range ends at a multiple of its size with 0xc00 added");
        const unsigned base = smem_u32_of(bins);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t t[4], out = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            t[k] = (w[k] & 0x7fff7fffu) + 0x0c000c00u;
            out |= (t[k] ^ 0x40004000u) & 0x70007000u;
        }
        if (out) {
#pragma unroll 1
            for (int k = 0; k < 8; ++k) one(w[k >> 1] >> (k & 1) * 16 & 0xffffu);
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // four times (magnitude | sign << 12)
            add(base + ((t[k] << 2 & 0x3ffcu) | (w[k] >> 1 & 0x4000u)));
            add(base + ((t[k] >> 14 & 0x3ffcu) | (w[k] >> 17 & 0x4000u)));
        }
    }
};

__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs p) {
    extern __shared__ __align__(16) char smem[];
    Shared &s = *(Shared *)smem;
    const int C = p.C, c = C > 1 ? (int)bgmv::cluster_rank() : 0;
    const int t = (int)blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint16_t *row = p.logits + (long long)t * p.ld;
    asm volatile("griddepcontrol.launch_dependents;");
    fill_powers(s.pw);
    if (tid == 0) s.told.low = 0, s.told.odd = 0, s.told.top = kBins;
    for (int i = tid; i < kBins; i += kThreads) s.bins[i] = 0;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // counts of this CTA's part of the row
    const int part = ((p.V + C - 1) / C + 7) & ~7, begin = min(p.V, c * part), end = min(p.V, begin + part);
    Counter counter;
    counter.bins = s.bins;
    each_vector(row, begin, end, tid, kThreads, [&](int, const uint4 &v) { counter.eight(v); }, [&](int, unsigned b) { counter.one(b); });
    const unsigned low = __reduce_max_sync(kAll, counter.low);
    if (lane == 0 && low) atomicMax(&s.told.low, low);
    if (__any_sync(kAll, counter.odd) && lane == 0) s.told.odd = 1;
    __syncthreads();
    int top = kBins;
    for (int i = tid; i < kBins; i += kThreads)
        if (s.bins[bin_of_place(i)]) {
            top = i;
            break;
        }
    top = (int)__reduce_min_sync(kAll, (unsigned)top);
    if (lane == 0) atomicMin(&s.told.top, top);
    const float temperature = p.temperature ? p.temperature[t] : 1.f;
    const bool greedy = !(temperature > 0.f);
    const float min_p = p.min_p ? p.min_p[t] : 0.f, top_p = p.top_p ? p.top_p[t] : 1.f, u = p.uniform ? p.uniform[t] : 0.f;
    const int top_k = p.top_k ? p.top_k[t] : 0;
    const u64 least = !(min_p > 0.f) ? 0ull : min_p >= 1.f ? 1ull << 62 : (u64)((double)min_p * 0x1p62);
    hear(s, C);
    unsigned lowest = 0;
    int odd = 0;
    top = kBins;
    for (int k = 0; k < C; ++k) {
        top = min(top, s.all[k].top);
        lowest = max(lowest, s.all[k].low);
        odd |= s.all[k].odd;
    }
    // The one window is enough if nothing lies outside of it but numbers too low to weigh anything.
    bool one = !odd && top < kBins;
    if (one) {
        if (tid == 0) s.scale = make_scale(greedy ? 1.f : temperature, value_of(key_of_place(top, -1)));
        __syncthreads();
        one = lowest == 0 || weight62(s.scale, value_of(lowest), s.pw) == 0;
    }
    Sums total, heavy, own, before = {0, 0};
    const int per = (kBins + C * kThreads - 1) / (C * kThreads), first = (c * kThreads + tid) * per;
    const Slice slice = {C == 1 ? s.bins : s.merged, c * kThreads * per, -1, C == 1};
    if (!one) {
        // the first CTA does the row alone
        cluster_sync(C);  // (and is no longer read by the others)
        if (c) return;
        unsigned key = 0;
        each_column(row, 0, p.V, tid, kThreads, [&](int, unsigned b) { key = max(key, key_of(b)); });
        key = __reduce_max_sync(kAll, key);
        if (lane == 0) s.warp_n[warp] = (int)key;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) key = max(key, (unsigned)s.warp_n[w]);
        if (key == 0) {  // nothing to choose from
            if (tid == 0) {
                p.tokens[t] = -1;
                if (p.logprobs) p.logprobs[t] = -INFINITY;
            }
            return;
        }
        if (tid == 0) s.scale = make_scale(greedy ? 1.f : temperature, value_of(key));
        window_sums(s, row, p.V, least, total, heavy);
    } else {
        if (C > 1) {
            // the slice's counts in the parts of all
            for (int i = 0; i < per; ++i) {
                const int place = c * kThreads * per + i * kThreads + tid;
                unsigned sum = 0;
                if (place < kBins) {
                    const unsigned *at = s.bins + bin_of_place(place);
#pragma unroll 1
                    for (int k = 0; k < C; ++k) sum += load_peer(peer_address(at, k));
                }
                s.merged[i * kThreads + tid] = sum;
            }
            __syncthreads();
        }
        Sums much, slice_total, slice_heavy;
        add_up(s, slice, first, per, least, own, much);
        before = scan(s, own, slice_total);
        scan(s, much, slice_heavy);
        if (tid == 0) {
            s.told.hi = (u64)(slice_total.mass >> 64);
            s.told.lo = (u64)slice_total.mass;
            s.told.n = slice_total.n;
            s.told.least_hi = (u64)(slice_heavy.mass >> 64);
            s.told.least_lo = (u64)slice_heavy.mass;
            s.told.least_n = slice_heavy.n;
        }
        hear(s, C);
        total = heavy = {0, 0};
        for (int k = 0; k < C; ++k) {
            const Told &o = s.all[k];
            if (k == c) {
                before.mass += total.mass;
                before.n += total.n;
            }
            total.mass += join(o.hi, o.lo);
            total.n += o.n;
            heavy.mass += join(o.least_hi, o.least_lo);
            heavy.n += o.least_n;
        }
    }
    // the column of the order where sums pass a bound, in s.found of every CTA
    const auto find = [&](u128 mass, int n) {
        if (!one) {
            find_by_windows(s, row, p.V, mass, n);
            return;
        }
        Found f;
        if (look(s, slice, first, per, before, own, mass, n, f)) {
            if (C == 1) s.found = f;
            else
                for (int k = 0; k < C; ++k) {
                    const uint32_t to = peer_address(&s.found, k);
#pragma unroll
                    for (int i = 0; i < (int)(sizeof(Found) / 4); ++i) store_peer(to + i * 4, ((const unsigned *)&f)[i]);
                }
        }
        cluster_sync(C);
    };
    // what is kept: n columns that weigh `mass`
    int n = total.n;
    u128 mass = total.mass;
    if (greedy) {
        n = 1;
        mass = (u128)1 << 62;
    } else {
        if (top_k > 0 && top_k < n) {
            find(~(u128)0, top_k);
            n = top_k;
            mass = join(s.found.hi, s.found.lo);
            cluster_sync(one ? C : 1);
        }
        if (top_p < 1.f) {
            // the sum has to reach top_p * mass, so it has to exceed the next integer below
            bool exact;
            const u128 down = times(mass, top_p, exact);
            find(exact && down ? down - 1 : down, n);
            n = s.found.n;
            mass = join(s.found.hi, s.found.lo);
            cluster_sync(one ? C : 1);
        }
        if (least && heavy.n < n) {
            n = heavy.n;
            mass = heavy.mass;
        }
    }
    bool exact;
    find(times(mass, u < 1.f ? u : u >= 1.f ? 0x1.fffffep-1f : 0.f, exact), n);

    // which column that is: number `rank` of those with the found key.  A warp's columns follow each other.
    const unsigned key = s.found.key;
    const int rank = s.found.rank;
    const int from = one ? begin : 0, to = one ? end : p.V;
    const int chunk = ((to - from + kWarps - 1) / kWarps + 255) & ~255;
    const int w0 = min(to, from + warp * chunk), w1 = min(to, w0 + chunk);
    const unsigned bits = key == 0x8000u ? 0u : __float_as_uint(value_of(key)) >> 16, both = bits | bits << 16;
    const unsigned odd_keys = key == 0x8000u || key == kKeyMax;  // those that several bits stand for
    int mine = 0;
    each_vector(
        row, w0, w1, lane, 32,
        [&](int, const uint4 &v) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t hit = odd_keys;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t x = w[k] ^ both;
                hit |= (x - 0x00010001u) & ~x & 0x80008000u;  // not 0 where a half of x is
            }
            if (!hit) return;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) mine += key_of(w[k >> 1] >> (k & 1) * 16 & 0xffffu) == key;
        },
        [&](int, unsigned b) { mine += key_of(b) == key; });
    mine = (int)__reduce_add_sync(kAll, (unsigned)mine);
    __syncthreads();
    if (lane == 0) s.warp_n[warp] = mine;
    __syncthreads();
    int ahead = 0;
    if (one && C > 1) {
        if (tid == 0) {
            int sum = 0;
            for (int w = 0; w < kWarps; ++w) sum += s.warp_n[w];
            s.told.matches = sum;
        }
        hear(s, C);
        for (int k = 0; k < c; ++k) ahead += s.all[k].matches;
        cluster_sync(C);  // nobody is read any more
    }
    for (int w = 0; w < warp; ++w) ahead += s.warp_n[w];
    if (ahead > rank || rank >= ahead + mine) return;
    for (int i = w0; i < w1; i += 32) {
        const int at = i + lane;
        const unsigned hit = __ballot_sync(kAll, at < w1 && key_of(row[at]) == key);
        if (rank < ahead + __popc(hit)) {
            if ((hit >> lane & 1) && ahead + __popc(hit & ((1u << lane) - 1)) == rank) {
                p.tokens[t] = at;
                if (p.logprobs) {
                    float hi, lo;
                    distance(s.scale, value_of(key), hi, lo);
                    // ln of the sum: 2^62 is one
                    const int lead = total.mass >> 64 ? 64 - __clzll((u64)(total.mass >> 64)) : 0;
                    const float m = (float)(u64)(total.mass >> lead);
                    p.logprobs[t] = -(hi * 0.69314718056f + (logf(m * 0x1p-62f) + (float)lead * 0.69314718056f));
                }
            }
            break;
        }
        ahead += __popc(hit);
    }
}

// CTAs that share a row: as many as all find room at once, two to an SM, of 4096 columns at least.
int ctas_of_a_row(int T, int V, int sms) {
    int C = 1;
    while (C < kMostCtas && (long long)T * C * 2 <= 2LL * sms && V >= C * 2 * 4096) C *= 2;
    return C;
}

std::atomic<int> g_sample_sms[64];  // SM count per device, looked up once (the kernel's attribute is set on the way)
cudaError_t device_sms(int &sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    sms = g_sample_sms[dev].load(std::memory_order_acquire);
    if (sms) return cudaSuccess;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    if (e == cudaSuccess) g_sample_sms[dev].store(sms, std::memory_order_release);
    return e;
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
    int sms = 0;
    LORA_CUDA_TRY(device_sms(sms));
    SampleArgs p;
    p.logits = (const uint16_t *)logits;
    p.ld = ld;
    p.T = T;
    p.V = vocab_size;
    p.C = ctas_of_a_row(T, vocab_size, sms);
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.uniform = uniform;
    p.tokens = tokens;
    p.logprobs = logprobs;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)p.C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.C > 1 ? 2 : 1;
    cfg.gridDim = dim3((unsigned)T * (unsigned)p.C, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = (cudaStream_t)stream;
    LORA_CUDA_TRY(cudaLaunchKernelEx(&cfg, sample_kernel, p));
    lora_note_launch();
    return LORA_OK;
}
