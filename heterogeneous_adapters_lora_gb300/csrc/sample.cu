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
// Keys are bf16 bits mapped to integers that grow with the value.  A window is a
// range of keys that is counted at once:
//   one     the keys of 0 and of magnitudes in [2^-23, 2^9), 8193 bins: all that
//           takes part in most rows
//   many    otherwise 16 windows of 4096 keys each, in descending order, each
//           counted when it is asked for
#include <math.h>
#include <string.h>

#include "lora_internal.cuh"

namespace {

typedef unsigned long long u64;
typedef unsigned __int128 u128;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMagLo = 104 * 128, kMags = 32 * 128;  // magnitudes [2^-23, 2^9) as bf16 bits
constexpr int kBins = 2 * kMags + 1;
constexpr int kBinsPad = (kBins + kThreads - 1) / kThreads * kThreads;
constexpr int kPerThread = kBinsPad / kThreads;
constexpr int kWinBins = 4096;
constexpr int kWindows = 65536 / kWinBins;
constexpr unsigned kKeyMax = 0xff7fu;  // key of the largest finite number

struct SampleArgs {
    const uint16_t *logits;
    long long ld;
    int T, V;
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

// Bin of the one window, in descending order of values, and back.
__device__ __forceinline__ int bin_of(unsigned key) {
    if (key == 0x8000u) return kMags;
    return key & 0x8000u ? kMagLo + kMags - 1 - (int)(key & 0x7fffu) : kMags + 1 + (int)(0x7fffu - key) - kMagLo;
}
__device__ __forceinline__ unsigned bin_key(int bin, int window) {
    if (window >= 0) return (unsigned)(window * kWinBins + kWinBins - 1 - bin);
    if (bin == kMags) return 0x8000u;
    return bin < kMags ? 0x8000u | (unsigned)(kMagLo + kMags - 1 - bin) : 0x7fffu - (unsigned)(kMagLo + bin - kMags - 1);
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

struct Shared {
    unsigned bins[kBinsPad];
    u64 pw[192];
    u64 warp_lo[kWarps], warp_hi[kWarps];  // 128-bit partial sums
    int warp_n[kWarps];
    int coarse[kWindows];
    u64 win_lo[kWindows], win_hi[kWindows];
    int win_n[kWindows];
    unsigned top;        // largest key
    unsigned low;        // largest key below the one window
    int odd;             // a key in the gaps of the one window, or above it
    Scale scale;
    // what find() leaves
    unsigned found_key;
    int found_rank, found_n;
    u64 found_lo, found_hi;
    int token;
};

__device__ __forceinline__ u128 join(u64 hi, u64 lo) { return ((u128)hi << 64) | lo; }

struct Sums {
    u128 mass;
    int n;
};

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

// Every column's bits, 8 at a time.
template <typename F>
__device__ __forceinline__ void each_column(const uint16_t *row, int begin, int end, int at, int step, F f) {
    for (int i = begin + at * 8; i < end; i += step * 8) {
        if (i + 8 <= end) {
            const uint4 v = __ldg((const uint4 *)(row + i));
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f(i + 2 * k, u[k] & 0xffffu);
                f(i + 2 * k + 1, u[k] >> 16);
            }
        } else {
            for (int k = i; k < end; ++k) f(k, (unsigned)row[k]);
        }
    }
}

__device__ __forceinline__ void clear_bins(Shared &s, int bins) {
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += kThreads) s.bins[i] = 0;
    __syncthreads();
}

__device__ void count_window(Shared &s, const uint16_t *row, int V, int window) {
    clear_bins(s, kWinBins);
    each_column(row, 0, V, threadIdx.x, kThreads, [&](int, unsigned b) {
        const unsigned k = key_of(b);
        if (k && (int)(k / kWinBins) == window) atomicAdd(&s.bins[kWinBins - 1 - (k % kWinBins)], 1u);
    });
    __syncthreads();
}

// Sums over this thread's bins; with `least`, of weights of at least that much only.
__device__ __forceinline__ Sums own_bins(const Shared &s, int per, int window, u64 least) {
    Sums r = {0, 0};
    for (int i = 0; i < per; ++i) {
        const int bin = threadIdx.x * per + i;
        const unsigned c = s.bins[bin];
        if (!c) continue;
        const u64 w = weight62(s.scale, value_of(bin_key(bin, window)), s.pw);
        if (w < least) continue;
        r.mass += (u128)w * c;
        r.n += (int)c;
    }
    return r;
}

// The first column of the order at which the sum of weights exceeds `mass`, or
// that is number `n`, whichever comes first (of the counted window, behind `at`);
// the thread that has it writes it down.
__device__ __forceinline__ void find_in_window(Shared &s, int per, int window, Sums at, u128 mass, int n) {
    const Sums mine = own_bins(s, per, window, 0);
    Sums total;
    Sums before = scan(s, mine, total);
    before.mass += at.mass;
    before.n += at.n;
    const bool here = before.mass <= mass && before.n < n && (before.mass + mine.mass > mass || before.n + mine.n >= n);
    if (here) {
        Sums sum = before;
        for (int i = 0; i < per; ++i) {
            const int bin = threadIdx.x * per + i;
            const unsigned c = s.bins[bin];
            if (!c) continue;
            const unsigned key = bin_key(bin, window);
            const u64 w = weight62(s.scale, value_of(key), s.pw);
            if (sum.mass + (u128)w * c > mass || sum.n + (int)c >= n) {
                // smallest r with sum + (r + 1) w > mass, bounded by the number asked for
                int lo = 0, hi = min((int)c, n - sum.n) - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (sum.mass + (u128)w * (unsigned)(mid + 1) > mass) hi = mid;
                    else lo = mid + 1;
                }
                sum.mass += (u128)w * (unsigned)(lo + 1);
                s.found_key = key;
                s.found_rank = lo;
                s.found_n = sum.n + lo + 1;
                s.found_hi = (u64)(sum.mass >> 64);
                s.found_lo = (u64)sum.mass;
                break;
            }
            sum.mass += (u128)w * c;
            sum.n += (int)c;
        }
    }
    __syncthreads();
}

__device__ void find(Shared &s, const uint16_t *row, int V, bool one, u128 mass, int n) {
    if (one) {
        find_in_window(s, kPerThread, -1, {0, 0}, mass, n);
        return;
    }
    Sums at = {0, 0};
    int w = kWindows - 1;
    for (; w > 0; --w) {
        const u128 m = at.mass + join(s.win_hi[w], s.win_lo[w]);
        if (m > mass || at.n + s.win_n[w] >= n) break;
        at.mass = m;
        at.n += s.win_n[w];
    }
    count_window(s, row, V, w);
    find_in_window(s, kWinBins / kThreads, w, at, mass, n);
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

__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs p) {
    extern __shared__ __align__(16) char smem[];
    Shared &s = *(Shared *)smem;
    const int t = blockIdx.x;
    const uint16_t *row = p.logits + (long long)t * p.ld;
    asm volatile("griddepcontrol.launch_dependents;");
    fill_powers(s.pw);
    if (threadIdx.x < kWindows) s.coarse[threadIdx.x] = 0;
    if (threadIdx.x == 0) s.top = s.low = 0, s.odd = 0;
    clear_bins(s, kBinsPad);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // counts by value, as far as the one window reaches
    unsigned top = 0, low = 0, odd = 0;
    each_column(row, 0, p.V, threadIdx.x, kThreads, [&](int, unsigned b) {
        const unsigned k = key_of(b);
        if (!k) return;
        top = max(top, k);
        const unsigned mag = b & 0x7fffu;
        if (mag - kMagLo < (unsigned)kMags || mag == 0u) atomicAdd(&s.bins[bin_of(k)], 1u);
        else if ((b & 0x8000u) && mag >= kMagLo + kMags) low = max(low, k);
        else odd = 1;
    });
    atomicMax(&s.top, __reduce_max_sync(kAll, top));
    atomicMax(&s.low, __reduce_max_sync(kAll, low));
    if (__any_sync(kAll, odd)) s.odd = 1;
    __syncthreads();
    if (s.top == 0) {  // nothing to choose from
        if (threadIdx.x == 0) {
            p.tokens[t] = -1;
            if (p.logprobs) p.logprobs[t] = -INFINITY;
        }
        return;
    }
    const float temperature = p.temperature ? p.temperature[t] : 1.f;
    const bool greedy = !(temperature > 0.f);
    if (threadIdx.x == 0) s.scale = make_scale(greedy ? 1.f : temperature, value_of(s.top));
    __syncthreads();
    const float min_p = p.min_p ? p.min_p[t] : 0.f;
    const u64 least = !(min_p > 0.f) ? 0ull : min_p >= 1.f ? 1ull << 62 : (u64)((double)min_p * 0x1p62);
    // the one window is enough if nothing lies outside of it but numbers too low to weigh anything
    const bool one = !s.odd && (s.low == 0 || weight62(s.scale, value_of(s.low), s.pw) == 0);
    Sums total, heavy;
    if (one) {
        scan(s, own_bins(s, kPerThread, -1, 0), total);
        if (least) scan(s, own_bins(s, kPerThread, -1, least), heavy);
    } else {
        each_column(row, 0, p.V, threadIdx.x, kThreads, [&](int, unsigned b) {
            const unsigned k = key_of(b);
            if (k) atomicAdd(&s.coarse[k / kWinBins], 1);
        });
        __syncthreads();
        total = heavy = {0, 0};
        for (int w = kWindows - 1; w >= 0; --w) {
            Sums sum = {0, 0}, some = {0, 0};
            if (s.coarse[w]) {
                count_window(s, row, p.V, w);
                scan(s, own_bins(s, kWinBins / kThreads, w, 0), sum);
                if (least) scan(s, own_bins(s, kWinBins / kThreads, w, least), some);
            }
            if (threadIdx.x == 0) {
                s.win_hi[w] = (u64)(sum.mass >> 64);
                s.win_lo[w] = (u64)sum.mass;
                s.win_n[w] = sum.n;
            }
            total.mass += sum.mass;
            total.n += sum.n;
            heavy.mass += some.mass;
            heavy.n += some.n;
        }
        __syncthreads();
    }
    // what is kept: n columns that weigh `mass`
    int n = total.n;
    u128 mass = total.mass;
    if (greedy) {
        n = 1;
        mass = (u128)1 << 62;
    } else {
        const int k = p.top_k ? p.top_k[t] : 0;
        if (k > 0 && k < n) {
            find(s, row, p.V, one, ~(u128)0, k);
            n = k;
            mass = join(s.found_hi, s.found_lo);
            __syncthreads();
        }
        const float top_p = p.top_p ? p.top_p[t] : 1.f;
        if (top_p < 1.f) {
            // the sum has to reach top_p * mass, so it has to exceed the next integer below
            bool exact;
            const u128 down = times(mass, top_p, exact);
            find(s, row, p.V, one, exact && down ? down - 1 : down, n);
            n = s.found_n;
            mass = join(s.found_hi, s.found_lo);
            __syncthreads();
        }
        if (least && heavy.n < n) {
            n = heavy.n;
            mass = heavy.mass;
        }
    }
    const float u = p.uniform ? p.uniform[t] : 0.f;
    bool exact;
    find(s, row, p.V, one, times(mass, u < 1.f ? u : u >= 1.f ? 0x1.fffffep-1f : 0.f, exact), n);
    // which column that is: number found_rank of those with the found key
    const unsigned key = s.found_key;
    const int rank = s.found_rank;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = ((p.V + kWarps - 1) / kWarps + 255) / 256 * 256;
    const int begin = min(p.V, warp * part), end = min(p.V, begin + part);
    int mine = 0;
    each_column(row, begin, end, lane, 32, [&](int, unsigned b) { mine += key_of(b) == key; });
    mine = __reduce_add_sync(kAll, mine);
    if (lane == 0) s.warp_n[warp] = mine;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s.warp_n[w];
    if (before <= rank && rank < before + mine) {
        for (int i = begin; i < end; i += 32) {
            const int c = i + lane;
            const unsigned hit = __ballot_sync(kAll, c < end && key_of(row[c]) == key);
            if (rank < before + __popc(hit)) {
                if ((hit >> lane & 1) && before + __popc(hit & ((1u << lane) - 1)) == rank) {
                    p.tokens[t] = c;
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
            before += __popc(hit);
        }
    }
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
    if (!logits || !tokens || !lora_aligned16(logits) ||
        (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)uniform |
          (uintptr_t)tokens | (uintptr_t)logprobs) & 3))
        return LORA_ERR_INVALID_ARG;
    SampleArgs p;
    p.logits = (const uint16_t *)logits;
    p.ld = ld;
    p.T = T;
    p.V = vocab_size;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.uniform = uniform;
    p.tokens = tokens;
    p.logprobs = logprobs;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)T, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = (cudaStream_t)stream;
    static_assert(sizeof(Shared) <= 48 * 1024, "fits without an attribute");
    LORA_CUDA_TRY(cudaLaunchKernelEx(&cfg, sample_kernel, p));
    lora_note_launch();
    return LORA_OK;
}
