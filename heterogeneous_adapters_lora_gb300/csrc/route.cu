// The router's choice: the top_k experts of every token by score (softmax or
// logistic function of the logits) plus a bias, and their weights.
//
// A warp takes a token and keeps its logits in registers, expert j * 32 + lane
// in element j.  Choosing needs no scores where they grow with the logits (no
// bias): the order is that of the logits, exact in fp32.  The choice is top_k
// rounds of a maximum over order-preserving integers (redux.sync) and the lowest
// id among those that have it.  A round costs the same for every token, so a
// call is bound by its launch for few tokens, and by these rounds for many.
//
// With a bias the fp32 scores may be off by a few 2^-24, which could order two
// experts wrongly.  So one more expert than asked for is looked at, and where two
// neighbours of the order are nearer than twice the error bound the
// token is done again with scores in 64 bits.
#include <float.h>
#include <string.h>

#include "lora_internal.cuh"

namespace {

constexpr int kThreads = 128;
constexpr unsigned kAll = 0xffffffffu;
// Bounds on the relative error of an fp32 score with the rounding of its biased
// sum.  Logistic function: exp 2 ulp, three more roundings.  Softmax: a logit minus the
// largest is rounded once, 2^-24 of up to 104 past which the score is 0; exp 2 ulp; the sum
// of up to 1024 terms in 32 lanes and 5 steps 37 roundings; the product and the bias two more.
constexpr float kEpsSigmoid = 1.0e-6f, kEpsSoftmax = 1.0e-5f;

struct RouteArgs {
    const void *logits;
    long long ld;
    int T, E, k, sigmoid, renormalize, wide;
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

// One round: the expert of the largest key, taken out; -1 if none is left.
template <int N, typename K>
__device__ __forceinline__ int take_best(K (&key)[N], K &best, int lane) {
    K mine = key[0];
#pragma unroll
    for (int j = 1; j < N; ++j) mine = key[j] > mine ? key[j] : mine;
    best = warp_max(mine);
    if (best == 0) return -1;
    int at = 0x7fffffff;
#pragma unroll
    for (int j = N - 1; j >= 0; --j) at = key[j] == best ? j * 32 + lane : at;
    at = (int)__reduce_min_sync(kAll, (unsigned)at);
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j * 32 + lane == at) key[j] = 0;
    return at;
}

__device__ __forceinline__ float load_logit(const RouteArgs &p, long long t, int e) {
    if (p.wide) return ((const float *)p.logits)[t * p.ld + e];
    return __uint_as_float((uint32_t)((const uint16_t *)p.logits)[t * p.ld + e] << 16);
}

// The choice by scores in 64 bits, for a token whose fp32 scores are too near to each other.
template <int N>
__device__ __noinline__ int choose_exactly(const RouteArgs &p, const float (&x)[N], float top, int lane, int k_lane) {
    double s[N], total = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        s[j] = p.sigmoid ? 1.0 / (1.0 + exp(-(double)x[j])) : exp((double)x[j] - (double)top);
        total += s[j];
    }
    total = p.sigmoid ? 1.0 : warp_sum(total);
    unsigned long long key[N], best;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = j * 32 + lane;
        key[j] = e < p.E && x[j] > -INFINITY ? order_key(s[j] / total + (double)p.bias[e]) : 0ull;
    }
    int chosen = -1;
    for (int r = 0; r < p.k; ++r) {
        const int e = take_best<N>(key, best, lane);
        if (r == k_lane) chosen = e;
    }
    return chosen;
}

// N: elements per lane (experts up to 32 N).
template <int N>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs p) {
    const int lane = threadIdx.x & 31;
    const long long t = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (t >= p.T) return;
    float x[N];
    unsigned key[N], best;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = j * 32 + lane;
        const float v = e < p.E ? load_logit(p, t, e) : -INFINITY;
        x[j] = v > -INFINITY ? fminf(v, FLT_MAX) : -INFINITY;  // NaN takes no part either
    }
    float mine = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) mine = fmaxf(mine, x[j]);
    const unsigned top_key = __reduce_max_sync(kAll, order_key(mine));
    const float top = top_key ? key_value(top_key) : 0.f;
    // the scores' common factor: 1 / sum of exp(x - top), or 1
    float inv = 1.f;
    float part = 0.f;
    if (!p.sigmoid) {
#pragma unroll
        for (int j = 0; j < N; ++j) part += expf(x[j] - top);
        inv = 1.f / warp_sum(part);
    }
    // score of a logit
    const auto score = [&](float v) { return p.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) * inv; };
    int chosen = -1;  // of round `lane`
    if (!p.bias) {
#pragma unroll
        for (int j = 0; j < N; ++j) key[j] = order_key(x[j]);
        for (int r = 0; r < p.k; ++r) {
            const int e = take_best<N>(key, best, lane);
            if (r == lane) chosen = e;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = j * 32 + lane;
            key[j] = e < p.E && x[j] > -INFINITY ? order_key(score(x[j]) + p.bias[e]) : 0u;
        }
        float before = 0.f, widest = 1.f;
        bool near = false;
        const float eps = p.sigmoid ? kEpsSigmoid : kEpsSoftmax;
        for (int r = 0; r <= p.k; ++r) {
            const int e = take_best<N>(key, best, lane);
            if (e < 0) break;
            const float v = key_value(best);
            widest = fmaxf(widest, fabsf(v));
            if (r > 0 && !(before - v > 2.f * eps * widest)) near = true;
            before = v;
            if (r == lane && r < p.k) chosen = e;
        }
        if (near) chosen = choose_exactly<N>(p, x, top, lane, lane);
    }
    float s = 0.f;
    if (chosen >= 0) {
        float v = load_logit(p, t, chosen);
        s = score(fminf(v, FLT_MAX));
    }
    if (p.renormalize) {
        const float sum = warp_sum(s);
        s = sum > 0.f ? s / sum : 0.f;
    }
    if (lane < p.k) {
        p.ids[t * p.k + lane] = chosen;
        p.w[t * p.k + lane] = chosen >= 0 ? s * p.scale : 0.f;
    }
}

template <int N>
cudaError_t route_launch(const RouteArgs &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)lora_ceil_div(p.T, kThreads / 32), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, route_kernel<N>, p);
}

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
    LORA_CUDA_TRY(d.n_experts <= 64    ? route_launch<2>(p, s)
                  : d.n_experts <= 256 ? route_launch<8>(p, s)
                                       : route_launch<32>(p, s));
    lora_note_launch();
    return LORA_OK;
}
