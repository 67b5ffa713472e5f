// The router's choice: the top_k experts of every token by score (softmax or
// logistic function of the logits) plus a bias, and their weights.
//
// A warp takes a token and keeps its logits in registers, experts lane * N to lane * N + N - 1
// in a lane: the lowest lane that has the largest key then has the lowest id of equal ones.  Choosing needs no
// scores where they grow with the logits (no bias): the order is that of the logits, exact in fp32.
// The choice is top_k rounds: the largest of the lanes' keys, order-preserving integers (redux.sync), is taken out.
// With many tokens and more than two experts a lane, rounds over the lanes' own largest first give a bound that leaves
// a dozen experts, which go to a lane each: a round over those is a few instructions.  Many tokens are bound by issuing
// some 1200 instructions each in chains (half of all issue slots are used); few by the launch and one
// read.  Warps walk over tokens and read the next one's logits ahead.  One token of 64 experts takes 2.4
// us, 7995 of 256 with a bias 14.8 (their bytes 0.7).
//
// With a bias the fp32 scores may be off by a few 2^-24, which could order two
// experts wrongly.  So rounds go on until the next expert is further behind than twice the error bound, and
// where neighbours of the order are nearer than that the ones that were found, one in a lane, are
// ordered again by scores in 64 bits (a logistic function each; a softmax's sum takes all of the token's).
#include <float.h>
#include <string.h>

#include <atomic>

#include "lora_internal.cuh"

namespace {

constexpr int kThreads = 128;
// CTAs of an SM, which walk over the tokens in one wave: as many as registers allow before spills cost (7995 tokens of 256 experts
// with a bias by 6 to 10 CTAs 15.0, 18.2 and 20 us; without one by 5 to 12 14.2, 11.7, 10.9, 10.5 and 9.9, the last with one register spilled).
template <int N, bool BIAS>
__host__ __device__ constexpr int ctas_per_sm() {
    return N == 2 ? 8 : N == 8 ? (BIAS ? 6 : 12) : BIAS ? 2 : 4;
}
constexpr unsigned kAll = 0xffffffffu;
// Bounds on the absolute error of an fp32 score with the rounding of its biased sum, for sums
// of magnitude 1 or less (larger ones in proportion).  Scores that decide take the fast exp and division: e =
// exp(x) is off by 2^-22 and by 2^-24 * 1.45 |x| of itself, the quotient by 2 ulp.  Logistic
// function: s (1 - s) <= 1/4 and s (1 - s) |x| < 0.23, so 2e-7 with the quotient's.  Softmax: all in proportion to the largest
// score, s |x - top| < 0.37 of it, the sum of up to 1024 terms in 32 lanes and 5 steps takes 37 roundings, 3e-6.  The sum with
// the bias 6e-8.
constexpr float kEpsSigmoid = 1.0e-6f, kEpsSoftmax = 1.0e-5f, kEpsSum = 2.0e-7f;  // (softmax: of the largest score, and kEpsSum)

struct RouteArgs {
    const void *logits;
    long long ld;
    int T, E, k, sigmoid, renormalize, wide, vec, many;
    float scale;
    const float *bias;
    int32_t *ids;
    float *w;
};

// Order-preserving map of floats to unsigned integers; 0 = takes no part.
__device__ __forceinline__ unsigned order_key(float v) {
    if (!(v > -INFINITY)) return 0u;  // -inf or NaN
    v += 0.0f;                        // -0 equals +0
    const unsigned b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long order_key(double v) {
    if (!(v > -(double)INFINITY)) return 0ull;
    v += 0.0;
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ unsigned warp_max(unsigned v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
    const unsigned hi = __reduce_max_sync(kAll, (unsigned)(v >> 32));
    const unsigned lo = __reduce_max_sync(kAll, (unsigned)(v >> 32) == hi ? (unsigned)v : 0u);
    return ((unsigned long long)hi << 32) | lo;
}

// One round: the expert of the largest key, taken out; -1 if none is left.  `mine`: this lane's largest.
template <int N, typename K>
__device__ __forceinline__ int take_best(K (&key)[N], K &mine, K &best, int lane) {
    best = warp_max(mine);
    if (best == 0) return -1;
    const int who = __ffs(__ballot_sync(kAll, mine == best)) - 1;
    int at = 0;
    if (lane == who) {
        K next = 0;
        bool taken = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (!taken && key[j] == best) {
                key[j] = 0;
                at = j;
                taken = true;
            }
            next = key[j] > next ? key[j] : next;
        }
        mine = next;
    }
    return who * N + __shfl_sync(kAll, at, who);
}
template <int N, typename K>
__device__ __forceinline__ K largest(const K (&key)[N]) {
    K m = key[0];
#pragma unroll
    for (int j = 1; j < N; ++j) m = key[j] > m ? key[j] : m;
    return m;
}

__device__ __forceinline__ float load_logit(const RouteArgs &p, long long t, int e) {
    if (p.wide) return ((const float *)p.logits)[t * p.ld + e];
    return __uint_as_float((uint32_t)((const uint16_t *)p.logits)[t * p.ld + e] << 16);
}
// What a logit counts as: NaN and -inf take no part, +inf is the largest number.
__device__ __forceinline__ float counted(float v) { return v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY; }

// This lane's logits of token t.  `vec`: rows are aligned to pairs.
template <int N>
__device__ __forceinline__ void load_logits(const RouteArgs &p, long long t, int lane, float (&x)[N]) {
    if (p.vec && lane * N + N <= p.E) {
        if (p.wide) {
            const float *row = (const float *)p.logits + t * p.ld + lane * N;
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const float2 v = __ldg((const float2 *)(row + j));
                x[j] = v.x;
                x[j + 1] = v.y;
            }
        } else {
            const uint16_t *row = (const uint16_t *)p.logits + t * p.ld + lane * N;
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const uint32_t v = __ldg((const uint32_t *)(row + j));
                x[j] = bf16lo(v);
                x[j + 1] = bf16hi(v);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane * N + j;
            x[j] = e < p.E ? load_logit(p, t, e) : -INFINITY;
        }
    }
}

// The first k of `found` candidates (lane r has the one of round r) by scores in 64 bits; lane r gets number r.
template <int N>
__device__ __noinline__ int order_exactly(const RouteArgs &p, long long t, float top, int lane, int candidate, int found) {
    double total = 1.0;
    if (!p.sigmoid) {
        double part = 0.0;
#pragma unroll 1
        for (int j = 0; j < N; ++j) {
            const int e = lane * N + j;
            if (e < p.E) part += exp((double)counted(load_logit(p, t, e)) - (double)top);
        }
        total = warp_sum(part);
    }
    unsigned long long key = 0;
    if (lane < found) {
        const double v = (double)counted(load_logit(p, t, candidate));
        const double s = p.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)top) / total;
        key = order_key(s + (double)p.bias[candidate]);
    }
    int place = 0;  // of equal keys the lower id comes first
    for (int r = 0; r < found; ++r) {
        const unsigned long long other = __shfl_sync(kAll, key, r);
        const int id = __shfl_sync(kAll, candidate, r);
        place += other > key || (other == key && id < candidate);
    }
    int chosen = -1;
    for (int r = 0; r < found; ++r) {
        const int at = __shfl_sync(kAll, place, r), id = __shfl_sync(kAll, candidate, r);
        if (at == lane) chosen = id;
    }
    return lane < p.k ? chosen : -1;
}

// The same for a token with more than 32 of them: all experts by scores in 64 bits.
template <int N>
__device__ __noinline__ int choose_exactly(const RouteArgs &p, long long t, float top, int lane) {
    double total = 1.0;
    unsigned long long key[N], best;
    for (int pass = p.sigmoid; pass < 2; ++pass) {  // the sum, then the keys
        double part = 0.0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane * N + j;
            const float v = counted(e < p.E ? load_logit(p, t, e) : -INFINITY);
            const double s = v == -INFINITY ? 0.0 : p.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top) / total;
            part += s;
            key[j] = v == -INFINITY ? 0ull : order_key(s + (double)p.bias[e]);
        }
        if (pass == 0) total = warp_sum(part);
    }
    unsigned long long mine = largest<N>(key);
    int chosen = -1;
    for (int r = 0; r < p.k; ++r) {
        const int e = take_best<N>(key, mine, best, lane);
        if (r == lane) chosen = e;
    }
    return chosen;
}

// The chosen scores' shares of their sum, in 64 bits: where one of them is below fp32's normal numbers, as far logits' are that a
// bias has chosen.
__device__ __noinline__ float share_exactly(float v, float top, int sigmoid) {  // v: -inf where none is chosen
    const double s = v == -INFINITY ? 0.0 : sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top);
    const double sum = warp_sum(s);
    return sum > 0.0 ? (float)(s / sum) : 0.f;
}

// The rounds.  Lane r gets the expert of round r (as who has it times M plus its place there); with a bias they go on past
// top_k while neighbours are near: `near` says that some are, `found` how many rounds there were (33: more than lanes).
template <int M, bool BIAS>
__device__ __forceinline__ int rounds(const RouteArgs &p, unsigned (&key)[M], unsigned mine, float eps, int lane, bool &near, int &found) {
    unsigned best;
    int chosen = -1;
    found = 0;
    near = false;
    if (!BIAS) {
#pragma unroll 1
        for (int r = 0; r < p.k; ++r) {
            const int e = take_best<M>(key, mine, best, lane);
            if (e < 0) break;
            if (r == lane) chosen = e;
        }
        return chosen;
    }
    float before = 0.f, widest = 1.f;
#pragma unroll 1
    for (int r = 0;; ++r) {
        const int e = take_best<M>(key, mine, best, lane);
        if (e < 0) break;
        const float v = key_value(best);
        widest = fmaxf(widest, fabsf(v));
        const bool close = r > 0 && !(before - v > 2.f * eps * widest);
        if (r >= p.k && !close) break;  // and all that follow are further behind
        near |= close;
        found = r + 1;
        if (r >= 32) break;
        before = v;
        if (r == lane) chosen = e;
    }
    return chosen;
}

// N: experts of a lane (32 N in all).  Up to 64 without a bias keep to 32 registers, so that the CTAs of the next launch find room beside
// these (7995 tokens of 64 experts, one launch behind the other, 6.3 us, with 37 registers 8.9).
template <int N, bool BIAS>
__global__ void __launch_bounds__(kThreads, N == 2 && !BIAS ? 16 : ctas_per_sm<N, BIAS>()) route_kernel(const RouteArgs p) {
    const int lane = threadIdx.x & 31, step = (int)gridDim.x * (kThreads / 32);
    long long t = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ unsigned s_key[N > 2 ? kThreads : 1];  // the few that can be chosen, a lane's each
    __shared__ uint16_t s_id[N > 2 ? kThreads : 1];
    float bias[BIAS ? N : 1], ahead[N];
    if (BIAS)
#pragma unroll
        for (int j = 0; j < N; ++j) bias[j] = lane * N + j < p.E ? p.bias[lane * N + j] : 0.f;
    if (t < p.T) load_logits<N>(p, t, lane, ahead);
    for (; t < p.T; t += step) {
        float x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = counted(ahead[j]);
        if (t + step < p.T) load_logits<N>(p, t + step, lane, ahead);
        const unsigned top_key = warp_max(order_key(largest<N>(x)));
        const float top = top_key ? key_value(top_key) : 0.f;
        unsigned key[N];
        int chosen = -1;  // of round `lane`
        float total = 1.f;  // of exp(x - top)
        if (!p.sigmoid) {
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) part += BIAS ? __expf(x[j] - top) : expf(x[j] - top);
            total = warp_sum(part);
        }
        const float inv = 1.f / total;  // the largest score of a softmax
        const float eps = p.sigmoid ? kEpsSigmoid : fmaf(kEpsSoftmax, inv, kEpsSum);
        if (!BIAS) {
#pragma unroll
            for (int j = 0; j < N; ++j) key[j] = order_key(x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float s = p.sigmoid ? __fdividef(1.f, 1.f + fminf(__expf(-x[j]), 1e30f)) : __expf(x[j] - top) * inv;
                key[j] = x[j] > -INFINITY ? order_key(s + bias[j]) : 0u;
            }
        }
        const unsigned mine = largest<N>(key);
        bool near = false, few = false;
        int found = 0;
        if (N > 2 && p.many) {
            // Number k of the lanes' largest is a bound: what is below it is not chosen, nor (with a bias) what is
            // below it by more than the widest distance that counts as near.
            unsigned m = mine, least = 0, most = 0;
#pragma unroll 1
            for (int r = 0; r < p.k; ++r) {
                least = warp_max(m);
                if (r == 0) most = least;
                if (!least) break;
                if (lane == __ffs(__ballot_sync(kAll, m == least)) - 1) m = 0;
            }
            if (BIAS && least) {
                const float v = key_value(least);
                least = order_key(v - 4.f * eps * fmaxf(1.f, fmaxf(fabsf(v), fabsf(key_value(most)))));
            }
            least = max(least, 1u);
            int at = 0, n = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const unsigned some = __ballot_sync(kAll, key[j] >= least);
                at += __popc(some & ((1u << lane) - 1));
                n += __popc(some);
            }
            few = n <= 32;
            if (few) {
                unsigned *const keys = s_key + (threadIdx.x & ~31u);
                uint16_t *const ids = s_id + (threadIdx.x & ~31u);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (key[j] >= least) {
                        keys[at] = key[j];
                        ids[at++] = (uint16_t)(lane * N + j);
                    }
                __syncwarp();
                unsigned one[1] = {lane < n ? keys[lane] : 0u};
                const int who = rounds<1, BIAS>(p, one, one[0], eps, lane, near, found);
                chosen = who >= 0 ? (int)ids[who] : -1;
                __syncwarp();
            }
        }
        if (!few) chosen = rounds<N, BIAS>(p, key, mine, eps, lane, near, found);
        if (BIAS) {
            if (!p.sigmoid) {  // the weights' sum, of exp itself
                float part = 0.f;
#pragma unroll
                for (int j = 0; j < N; ++j) part += expf(x[j] - top);
                total = warp_sum(part);
            }
            // (nothing of the row is needed any more, so these calls save few registers)
            if (found > 32) chosen = choose_exactly<N>(p, t, top, lane);
            else if (near) chosen = order_exactly<N>(p, t, top, lane, chosen, found);
        }
        float s = 0.f, v = -INFINITY;
        if (chosen >= 0) {
            v = counted(load_logit(p, t, chosen));
            s = p.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / total;
        }
        if (p.renormalize) {
            if (__any_sync(kAll, chosen >= 0 && s < FLT_MIN)) {
                s = share_exactly(v, top, p.sigmoid);
            } else {
                const float sum = warp_sum(s);
                s = sum > 0.f ? s / sum : 0.f;
            }
        }
        if (lane < p.k) {
            p.ids[t * p.k + lane] = chosen;
            p.w[t * p.k + lane] = chosen >= 0 ? s * p.scale : 0.f;
        }
    }
}

template <int N, bool BIAS>
cudaError_t route_launch(RouteArgs p, int sms, cudaStream_t s) {
    const int size = p.wide ? 4 : 2;
    // few tokens wait for their chains, which are shorter without the bound (13 tokens of 236 experts 3.9 us, with it 4.3)
    p.many = p.T >= 8 * sms;
    p.vec = p.ld % 2 == 0 && ((uintptr_t)p.logits & (2 * size - 1)) == 0;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const int need = lora_ceil_div(p.T, kThreads / 32), most = sms * ctas_per_sm<N, BIAS>();
    cfg.gridDim = dim3((unsigned)(need < most ? need : most), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, route_kernel<N, BIAS>, p);
}

std::atomic<int> g_route_sms[64];  // SM count per device, looked up once

}  // namespace

extern "C" lora_status_t lora_moe_route(const lora_route_desc_t *desc, const void *logits, int64_t ld_logits, int32_t T,
                                        const float *bias, int32_t *topk_ids, float *topk_w, void *stream) {
    if (!desc || T < 0) return LORA_ERR_INVALID_ARG;
    const lora_route_desc_t d = *desc;
    if (d.n_experts < 1 || d.n_experts > LORA_ROUTE_MAX_EXPERTS || d.top_k < 1 || d.top_k > LORA_ROUTE_MAX_TOP_K ||
        d.top_k > d.n_experts || (d.scoring != 0 && d.scoring != 1) || (d.renormalize != 0 && d.renormalize != 1) ||
        (d.logits_f32 != 0 && d.logits_f32 != 1) || !(d.scale >= -FLT_MAX && d.scale <= FLT_MAX) || ld_logits < d.n_experts)
        return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    if (!logits || !topk_ids || !topk_w || ((uintptr_t)logits & (d.logits_f32 ? 3 : 1)) || ((uintptr_t)bias & 3) ||
        ((uintptr_t)topk_ids & 3) || ((uintptr_t)topk_w & 3))
        return LORA_ERR_INVALID_ARG;
    RouteArgs p;
    p.logits = logits;
    p.ld = ld_logits;
    p.T = T;
    p.E = d.n_experts;
    p.k = d.top_k;
    p.sigmoid = d.scoring;
    p.renormalize = d.renormalize;
    p.wide = d.logits_f32;
    p.scale = d.scale;
    p.bias = bias;
    p.ids = topk_ids;
    p.w = topk_w;
    cudaStream_t s = (cudaStream_t)stream;
    int dev = 0;
    LORA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return LORA_ERR_INVALID_ARG;
    int sms = g_route_sms[dev].load(std::memory_order_relaxed);
    if (!sms) {
        LORA_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        g_route_sms[dev].store(sms, std::memory_order_relaxed);
    }
    if (bias)
        LORA_CUDA_TRY(d.n_experts <= 64    ? (route_launch<2, true>(p, sms, s))
                      : d.n_experts <= 256 ? (route_launch<8, true>(p, sms, s))
                                           : (route_launch<32, true>(p, sms, s)));
    else
        LORA_CUDA_TRY(d.n_experts <= 64    ? (route_launch<2, false>(p, sms, s))
                      : d.n_experts <= 256 ? (route_launch<8, false>(p, sms, s))
                                           : (route_launch<32, false>(p, sms, s)));
    lora_note_launch();
    return LORA_OK;
}
