// router.cu -- top-k routing of tokens from router logits, and its gradient.
//
// One warp per token, the token's logits in registers (expert i * 32 + lane in
// slot i) as order-preserving integers of logit or score plus bias. Ties go to the lowest
// expert. The weights need the chosen logits only, except for the softmax over all
// experts, which adds one sum. Instructions and their latency bound it, not memory:
// 8192 tokens of 256 bf16 logits (4.2 MB) take 8.0 us forward (10.1 with the bias on
// the scores) and 4.0 backward, 128 tokens of 64 about 2 either way.
#include "launch.cuh"

#include <cfloat>
#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

namespace ep {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct TopkParams {
    const void *logits;
    const float *bias, *dweights;
    int32_t *ids;
    const int32_t *ids_in;
    float *weights;
    void *dlogits;
    int tokens, E, K, score, renormalize, bias_on_score;
    float scale;
};

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *p, size_t at) {
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[at]) : static_cast<const float *>(p)[at];
}

// Order-preserving integer of a float; 0 (below every float's) for NaN and -inf.
// Adding 0 turns -0 into +0, so that the two tie.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v >= -FLT_MAX)) return 0u;
    const uint32_t u = __float_as_uint(v + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float warp_max(float v) {
    for (int d = 16; d > 0; d /= 2) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// log of the sigmoid, without overflow on either side
__device__ __forceinline__ float log_sigmoid(float z) { return fminf(z, 0.f) - log1pf(expf(-fabsf(z))); }

// The softmax over all experts, as (maximum, sum): NaN logits count for nothing and
// +inf as the largest finite number.
template <int N>
__device__ __forceinline__ float2 softmax_stats(const float (&z)[N]) {
    float m = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, z[i]);
    m = warp_max(m);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += expf(z[i] - m);
    return make_float2(m, warp_sum(s));
}

// The score of a logit among all.
__device__ __forceinline__ float score_of(const TopkParams &p, float z, float2 all) {
    return p.score == EP_SCORE_SOFTMAX ? expf(z - all.x) / all.y : 1.f / (1.f + expf(-z));
}

// The unscaled weight of the lane's chosen logit (`on`: the lane holds one).
__device__ __forceinline__ float weight_of(const TopkParams &p, float z, bool on, float2 all) {
    if (!p.renormalize) {
        const float w = score_of(p, z, all);
        return on ? w : 0.f;
    }
    // the chosen scores over their sum, as a softmax of their logarithms: the scores
    // themselves may all underflow
    const float l = !on ? -INFINITY : p.score == EP_SCORE_SOFTMAX ? z : log_sigmoid(z);
    const float m = warp_max(l);
    const float e = on ? expf(l - m) : 0.f;
    const float s = warp_sum(e);
    return on ? e / s : 0.f;
}

// A logit as the scores use it: NaN and -inf to -inf, +inf to the largest float.
__device__ __forceinline__ float usable(float z) { return z >= -FLT_MAX ? fminf(z, FLT_MAX) : -INFINITY; }

// SCORED: the bias goes on the score. A kernel of its own: as a branch it slowed the choice by
// logits, which does not take it (8192 tokens, 256 experts: 8.0 -> 8.9 us).
template <int N, bool BF16, bool SCORED>
__global__ void __launch_bounds__(kThreads) topk_kernel(const TopkParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % 32;
    const int t = blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= p.tokens) return;
    float z[N];
    uint32_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = i * 32 + lane;
        z[i] = e < p.E ? load_logit<BF16>(p.logits, (size_t)t * p.E + e) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = i * 32 + lane;
        key[i] = order_key(z[i]);
        if (!SCORED && p.bias && e < p.E && key[i]) key[i] = order_key(z[i] + p.bias[e]);
        z[i] = usable(z[i]);
    }
    float2 all = make_float2(0.f, 1.f);
    if (p.score == EP_SCORE_SOFTMAX && (!p.renormalize || SCORED)) all = softmax_stats(z);
    if (SCORED) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 32 + lane;
            if (e < p.E && key[i]) key[i] = order_key(score_of(p, z[i], all) + p.bias[e]);
        }
    }

    int rank = p.K, id = -1;   // this lane's choice, if it has one: place and expert
    int n = 0;                 // choices of the row
    bool done = false;
    if constexpr (N >= 4) {
        // The top_k-th largest of the lanes' maxima bounds the top_k-th largest logit from
        // below. What is not smaller is usually little more than top_k: those go to a lane
        // each, in expert order, and count who is ahead of them. (8192 tokens, 256 experts,
        // top 8: 11.0 -> 7.9 us against a round per choice.)
        __shared__ uint2 kept[kWarps][32];
        uint32_t most = key[0];
#pragma unroll
        for (int i = 1; i < N; ++i) most = max(most, key[i]);
        uint32_t bound = 0;
        for (int k = 0; k < p.K; ++k) {
            bound = __reduce_max_sync(kAll, most);
            if (most == bound) most = 0;
        }
        bound = max(bound, 1u);
        uint32_t held[N];
        int total = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            held[i] = __ballot_sync(kAll, key[i] >= bound);
            total += __popc(held[i]);
        }
        if (total <= 32) {
            uint2 *slot = kept[threadIdx.x / 32];
            int at = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (key[i] >= bound) slot[at + __popc(held[i] & lanemask_lt())] = make_uint2(key[i], i * 32 + lane);
                at += __popc(held[i]);
            }
            __syncwarp();
            const uint2 own = lane < total ? slot[lane] : make_uint2(0u, 0u);
            int ahead = 0;
            for (int j = 0; j < total; ++j) {
                const uint32_t other = __shfl_sync(kAll, own.x, j);
                ahead += other > own.x || (other == own.x && j < lane);
            }
            if (lane < total && ahead < p.K) rank = ahead, id = (int)own.y;
            n = min(total, p.K);
            done = true;
        }
    }
    if (!done) {   // few experts, or many ties: a round per choice, kept by lane k
        for (int k = 0; k < p.K; ++k) {
            uint32_t best = 0;
            int slot = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (key[i] > best) best = key[i], slot = i;
            const uint32_t top = __reduce_max_sync(kAll, best);
            if (top == 0) break;
            const int mine = slot * 32 + lane;
            const int e = (int)__reduce_min_sync(kAll, best == top ? (uint32_t)mine : 0xFFFFFFFFu);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (e == i * 32 + lane) key[i] = 0;
            if (lane == k) rank = k, id = e;
            ++n;
        }
    }
    // the chosen logits again, from cache: picking them out of the registers would
    // need a run-time index
    const float chosen = id >= 0 ? usable(load_logit<BF16>(p.logits, (size_t)t * p.E + id)) : 0.f;
    const float w = p.scale * weight_of(p, chosen, id >= 0, all);
    const size_t out = (size_t)t * p.K;
    if (id >= 0) {
        p.ids[out + rank] = id;
        p.weights[out + rank] = w;
    }
    if (lane >= n && lane < p.K) {
        p.ids[out + lane] = -1;
        p.weights[out + lane] = 0.f;
    }
}

// With q the unscaled weights, dq = scale * dweights and m = sum_k dq_k q_k:
//   softmax, renormalised   dz_k = q_k (dq_k - m)              (chosen only)
//   softmax                 dz_e = p_e (dq_e [chosen] - m)     (every expert)
//   sigmoid, renormalised   dz_k = q_k (1 - s_k) (dq_k - m)
//   sigmoid                 dz_k = q_k (1 - s_k) dq_k
template <int N, bool BF16>
__global__ void __launch_bounds__(kThreads) topk_backward_kernel(const TopkParams p) {
    __shared__ float rows[kWarps][N * 32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int t = blockIdx.x * kWarps + warp;
    if (t >= p.tokens) return;
    const size_t base = (size_t)t * p.E;
    const bool whole = p.score == EP_SCORE_SOFTMAX && !p.renormalize;
    int id = -1;
    float dq = 0.f, zk = 0.f;
    if (lane < p.K) {
        id = p.ids_in[(size_t)t * p.K + lane];
        if (id < 0 || id >= p.E) id = -1;
        if (id >= 0) {
            dq = p.scale * p.dweights[(size_t)t * p.K + lane];
            zk = usable(load_logit<BF16>(p.logits, base + id));
        }
    }
    float z[N];
    float2 all = make_float2(0.f, 1.f);
    if (whole) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 32 + lane;
            z[i] = e < p.E ? usable(load_logit<BF16>(p.logits, base + e)) : -INFINITY;
        }
        all = softmax_stats(z);
    }
    const float q = weight_of(p, zk, id >= 0, all);
    const float m = warp_sum(dq * q);
    float d;
    if (p.score == EP_SCORE_SOFTMAX) {
        d = whole ? q * dq : q * (dq - m);
    } else {
        const float rest = 1.f / (1.f + expf(zk));   // 1 - sigmoid
        d = q * rest * (p.renormalize ? dq - m : dq);
    }
    float *row = rows[warp];
    const float part = all.y > 0.f ? -m / all.y : 0.f;   // no expert left: no gradient
#pragma unroll
    for (int i = 0; i < N; ++i) row[i * 32 + lane] = whole ? expf(z[i] - all.x) * part : 0.f;
    __syncwarp();
    if (id >= 0) row[id] += d;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = i * 32 + lane;
        if (e >= p.E) break;
        const float v = row[e];
        if (BF16)
            static_cast<__nv_bfloat16 *>(p.dlogits)[base + e] = __float2bfloat16_rn(v);
        else
            static_cast<float *>(p.dlogits)[base + e] = v;
    }
}

template <bool BACKWARD, int N>
int launch_n(const TopkParams &p, bool bf16, cudaStream_t st) {
    const int grid = (p.tokens - 1) / kWarps + 1;   // tokens may be 2^31 - 1
    const auto kernel = BACKWARD ? (bf16 ? topk_backward_kernel<N, true> : topk_backward_kernel<N, false>)
                        : p.bias && p.bias_on_score ? (bf16 ? topk_kernel<N, true, true> : topk_kernel<N, false, true>)
                                                    : (bf16 ? topk_kernel<N, true, false> : topk_kernel<N, false, false>);
    return launch_after(kernel, dim3((unsigned)grid), kThreads, st, p) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

template <bool BACKWARD>
int launch_topk(const TopkParams &p, bool bf16, cudaStream_t st) {
    if (p.E <= 32) return launch_n<BACKWARD, 1>(p, bf16, st);
    if (p.E <= 64) return launch_n<BACKWARD, 2>(p, bf16, st);
    if (p.E <= 128) return launch_n<BACKWARD, 4>(p, bf16, st);
    if (p.E <= 256) return launch_n<BACKWARD, 8>(p, bf16, st);
    if (p.E <= 512) return launch_n<BACKWARD, 16>(p, bf16, st);
    return launch_n<BACKWARD, 32>(p, bf16, st);
}

bool topk_params(const ep_topk_t *a, const void *logits, TopkParams &p) {
    if (!a || a->tokens < 0 || a->E < 1 || a->E > EP_MAX_E || a->top_k < 1 || a->top_k > EP_MAX_TOPK ||
        a->top_k > a->E || (a->renormalize != 0 && a->renormalize != 1) ||
        ((a->score & ~EP_BIAS_ON_SCORE) != EP_SCORE_SOFTMAX && (a->score & ~EP_BIAS_ON_SCORE) != EP_SCORE_SIGMOID) ||
        (a->logits_dtype != EP_BF16 && a->logits_dtype != EP_F32))
        return false;
    p = {};
    p.logits = logits;
    p.tokens = a->tokens;
    p.E = a->E;
    p.K = a->top_k;
    p.score = a->score & ~EP_BIAS_ON_SCORE;
    p.bias_on_score = (a->score & EP_BIAS_ON_SCORE) != 0;
    p.renormalize = a->renormalize;
    p.scale = a->scale;
    return true;
}

bool aligned_to(const void *q, size_t n) { return q && reinterpret_cast<uintptr_t>(q) % n == 0; }

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

}  // namespace

}  // namespace ep

using namespace ep;

extern "C" int ep_topk_route(const ep_topk_t *a, const void *logits, const float *bias, int32_t *topk_ids,
                             float *topk_weights, void *stream) {
    TopkParams p;
    if (!topk_params(a, logits, p)) return EP_ERR_INVALID_ARG;
    if (a->tokens == 0) return EP_OK;
    const bool bf16 = a->logits_dtype == EP_BF16;
    if (!aligned_to(logits, bf16 ? 2 : 4) || !aligned_to(topk_ids, 4) || !aligned_to(topk_weights, 4) ||
        (bias && !aligned_to(bias, 4)))
        return EP_ERR_INVALID_ARG;
    p.bias = bias;
    p.ids = topk_ids;
    p.weights = topk_weights;
    Range range("ep:topk_route");
    return launch_topk<false>(p, bf16, static_cast<cudaStream_t>(stream));
}

extern "C" int ep_topk_route_backward(const ep_topk_t *a, const float *dweights, const void *logits,
                                      const int32_t *topk_ids, void *dlogits, void *stream) {
    TopkParams p;
    if (!topk_params(a, logits, p)) return EP_ERR_INVALID_ARG;
    if (a->tokens == 0) return EP_OK;
    const bool bf16 = a->logits_dtype == EP_BF16;
    if (!aligned_to(logits, bf16 ? 2 : 4) || !aligned_to(dlogits, bf16 ? 2 : 4) || !aligned_to(topk_ids, 4) ||
        !aligned_to(dweights, 4))
        return EP_ERR_INVALID_ARG;
    p.dweights = dweights;
    p.ids_in = topk_ids;
    p.dlogits = dlogits;
    Range range("ep:topk_route_backward");
    return launch_topk<true>(p, bf16, static_cast<cudaStream_t>(stream));
}
