// balance.cu -- the router's balance loss and per-expert counts, its z loss, and the gradient
// of both.
//
// Tokens form pools (all of a call, or one per sequence). With c_e the choices of expert e in a
// pool of N tokens, p_e(t) token t's probabilities and f_e = E c_e / (K N),
//   balance = mean over the pools with tokens of sum_e f_e (1/N) sum_t p_e(t)
//   z       = mean over all tokens of L(t)^2, L = log sum_e exp(logit_e)
// and with d0, d1 the losses' gradients, g_e = d0 f_e / (pools N)
//   softmax  dz_e = p_e (g_e - sum_j g_j p_j + 2 d1 / N_all L)
//   sigmoid  dz_e = p_e (1 - s_e) (g_e - sum_j g_j p_j) + 2 d1 / N_all L softmax_e
// where a sigmoid gate's p_e = s_e / sum_j s_j.
//
// A token's logits are read once, by a group of 8, 16 or 32 lanes with 8 consecutive experts
// (or more) to a lane, 16 bytes a load. Each lane adds its experts' probabilities up over its
// tokens; a CTA's sums go to the workspace and a second, small kernel adds the CTAs' up in
// order, so that nothing depends on the order of atomics (counts, whole numbers, are added
// atomically in shared memory).
//
// Instructions and their latency bound it: 64000 tokens of 256 fp32 logits (66 MB) take 48 us in both
// directions (about 20 for the sums, 5 to join them, 22 for the gradient; 20 would be the bytes'), 8
// sequences of 1024 19 us, 128 tokens of 64 experts 7 for the losses alone.
#include "launch.cuh"

#include <cfloat>
#include <cuda_bf16.h>
#include <nvtx3/nvToolsExt.h>

#include "act.cuh"

namespace ep {

namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kMaxChunks = 304;      // CTAs of all pools together, two per SM, while pools allow it
constexpr int kMaxChunk = 4096;      // tokens of a CTA, at most: bounds the chain of a fp32 sum
constexpr int kFinishThreads = 1024;
constexpr int kSlice = 32;           // experts of a finishing CTA
constexpr int kBackThreads = 256;
constexpr unsigned kMaxBackCtas = 4 * kMaxChunks;   // eight per SM
constexpr float kLn2 = 0.69314718055994531f;

struct BalanceParams {
    const void *logits;
    const int32_t *ids, *num_tokens;
    int32_t *counts;
    const int32_t *counts_in;
    float *losses;
    const float *dlosses;
    void *dlogits;
    uint32_t *ticket;
    float *slots;     // [pools][slices]
    float *zpart;     // [pools][chunks]
    float *part;      // [pools][chunks][E]
    int32_t *cpart;   // [pools][chunks][E]
    int seqs, T, E, K, pools, rows;   // rows = tokens of a pool, used or not
    int chunks, chunk;                // CTAs of a pool, tokens of each
    int sigmoid, accumulate;
};

// Where token r of a pool lies, and whether it is in use.
struct Token {
    long long at;   // its row among all
    bool used;
};
__device__ __forceinline__ int length_of(const BalanceParams &p, int s) {
    return p.num_tokens ? max(0, min(p.num_tokens[s], p.T)) : p.T;
}
__device__ __forceinline__ Token token_of(const BalanceParams &p, int pool, long long r, int end) {
    if (r >= end) return {0, false};
    if (!p.num_tokens) return {p.pools == p.seqs ? (long long)pool * p.T + r : r, true};
    if (p.pools == p.seqs) return {(long long)pool * p.T + r, r < length_of(p, pool)};
    const int s = (int)r / p.T;
    return {r, (int)r - s * p.T < length_of(p, s)};
}

// The expert in a lane's slot j: runs of 8, or for rows that allow no wide loads one by one.
template <int G, bool VEC>
__device__ __forceinline__ int expert_of(int lane, int j) {
    return VEC ? ((j / 8) * G + lane) * 8 + j % 8 : j * G + lane;
}

// A logit as the losses use it: NaN and -inf to -inf (no part), +inf to the largest float.
__device__ __forceinline__ float usable(float z) { return fminf(fmaxf(z, -INFINITY), FLT_MAX); }

template <int G, int M, bool BF16, bool VEC>
__device__ __forceinline__ void load_row(const BalanceParams &p, Token t, int lane, float (&z)[M]) {
    if (VEC) {
#pragma unroll
        for (int c = 0; c < M / 8; ++c) {
            const int e = (c * G + lane) * 8;
            const bool on = t.used && e < p.E;
            const size_t at = (size_t)t.at * p.E + e;
            if (BF16) {
                uint4 v = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);   // -inf
                if (on) v = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.logits) + at);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 f = unpack_bf16x2(w[q]);
                    z[8 * c + 2 * q] = f.x, z[8 * c + 2 * q + 1] = f.y;
                }
            } else {
                float4 a = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), b = a;
                if (on) {
                    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p.logits) + at);
                    a = q[0], b = q[1];
                }
                z[8 * c] = a.x, z[8 * c + 1] = a.y, z[8 * c + 2] = a.z, z[8 * c + 3] = a.w;
                z[8 * c + 4] = b.x, z[8 * c + 5] = b.y, z[8 * c + 6] = b.z, z[8 * c + 7] = b.w;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const int e = expert_of<G, VEC>(lane, j);
            z[j] = -INFINITY;
            if (t.used && e < p.E) {
                const size_t at = (size_t)t.at * p.E + e;
                z[j] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[at])
                            : static_cast<const float *>(p.logits)[at];
            }
        }
    }
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
    if constexpr (G == 32) {
        float m;
        asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(v));
        return m;
    } else {
#pragma unroll
        for (int d = G / 2; d > 0; d /= 2) v = max_nan(v, __shfl_xor_sync(kAll, v, d));
        return v;
    }
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = G / 2; d > 0; d /= 2) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// A token's largest logit. Where a warp's tokens have NaN, infinite or large ones, or none, the
// logits become usable and the exponentials take another step (`odd`, the same for the warp):
// looking at the maximum alone saves two instructions a logit.
struct Top {
    float m;
    bool odd;
};
// Up to here the short way's rounding of the maximum times log2(e) (half a unit of 2^17) is 2^-8 at most.
constexpr float kLarge = 65536.f;

template <int G, int M>
__device__ __forceinline__ Top top_of(float (&z)[M]) {
    float m = z[0];
#pragma unroll
    for (int j = 1; j < M; ++j) m = max_nan(m, z[j]);
    m = group_max<G>(m);
    const bool odd = __any_sync(kAll, !(fabsf(m) <= kLarge));
    if (odd) {
        m = -FLT_MAX;
#pragma unroll
        for (int j = 0; j < M; ++j) z[j] = usable(z[j]), m = fmaxf(m, z[j]);
        m = group_max<G>(m);
    }
    return {m, odd};
}

__device__ __forceinline__ float log2_f(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(z - m) of every slot into e, up to a factor that all share; their sum's inverse (0 for a row
// without a usable logit) and the logits' logsumexp (then 0). The factor is 2 to the power of what
// rounding takes from m log2(e): the logsumexp takes it back, and within 2^-8 of 0 that power overflows
// nothing. Past kLarge it would (|m| = 1e10: a power of 440), so there z - m is formed first.
// Exponentials by ex2.approx: right to (2 + |z - m| 1.5) 2^-23 of themselves, so that what carries the
// sum is right to a few units of fp32; the logarithm to 2^-22.
template <int G, int M>
__device__ __forceinline__ float softmax_of(const float (&z)[M], Top top, float (&e)[M], float &lse) {
    float sum = 0.f;
    const float shift = top.m * kLog2E;   // rounded: the factor
    if (!top.odd) {
#pragma unroll
        for (int j = 0; j < M; ++j) {
            e[j] = exp2_f(fmaf(z[j], kLog2E, -shift));
            sum += e[j];
        }
        sum = group_sum<G>(sum);
        lse = (shift + log2_f(sum)) * kLn2;
        return rcp_f(sum);
    }
#pragma unroll
    for (int j = 0; j < M; ++j) {
        e[j] = exp2_f((z[j] - top.m) * kLog2E);
        sum += e[j];
    }
    sum = group_sum<G>(sum);
    lse = sum > 0.f ? top.m + log2_f(sum) * kLn2 : 0.f;
    return sum > 0.f ? rcp_f(sum) : 0.f;
}

// Sigmoids up to a common factor (exp(-mu), mu the largest logit where that is negative: the
// sigmoids themselves may all underflow) into s, what is left to 1 into rest, the sum's inverse.
template <int G, int M, bool REST>
__device__ __forceinline__ float sigmoid_of(const float (&z)[M], float m, float (&s)[M], float (&rest)[M]) {
    const float mu = fminf(m, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < M; ++j) {
        const float v = exp2_f(-kLog2E * fabsf(z[j])), r = rcp_f(1.f + v);
        const float low = mu == 0.f ? v : exp2_f((z[j] - mu) * kLog2E);
        s[j] = z[j] >= 0.f ? r : low * r;
        if (REST) rest[j] = z[j] >= 0.f ? v * r : r;
        sum += s[j];
    }
    sum = group_sum<G>(sum);
    return sum > 0.f ? rcp_f(sum) : 0.f;
}

template <int M>
constexpr int kSumThreads = M <= 8 ? 512 : 256;   // so that the warps' sums fit in 32 KB

template <int G, int M, bool BF16, bool VEC>
__global__ void __launch_bounds__(kSumThreads<M>) balance_sums_kernel(const BalanceParams p) {
    constexpr int kWarps = kSumThreads<M> / 32, kRow = G * M;
    __shared__ float sums[kWarps][kRow];
    __shared__ int32_t count[kRow];
    __shared__ float zs[kWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % G, sub = threadIdx.x % 32 / G;
    for (int e = threadIdx.x; e < kRow; e += kSumThreads<M>) count[e] = 0;
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
    __syncthreads();
    const int pool = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const long long lo = (long long)chunk * p.chunk;
    int end = (int)min((long long)p.rows, lo + p.chunk);
    if (p.pools == p.seqs) end = min(end, length_of(p, pool));
    float acc[M], z2 = 0.f;
#pragma unroll
    for (int j = 0; j < M; ++j) acc[j] = 0.f;
    constexpr int kAtOnce = kSumThreads<M> / G, kPerWarp = 32 / G;
    for (long long r0 = lo + warp * kPerWarp; r0 < end; r0 += kAtOnce) {
        const Token t = token_of(p, pool, r0 + sub, end);
        float z[M], e[M], lse;
        load_row<G, M, BF16, VEC>(p, t, lane, z);
        if (t.used) {
            for (int k = lane; k < p.K; k += G) {
                const int id = p.ids[t.at * p.K + k];
                if (id >= 0 && id < p.E) atomicAdd(&count[id], 1);
            }
        }
        const Top top = top_of<G, M>(z);
        float inv = softmax_of<G, M>(z, top, e, lse);
        z2 += lse * lse;
        if (p.sigmoid) {
            float rest[M];
            inv = sigmoid_of<G, M, false>(z, top.m, e, rest);
        }
#pragma unroll
        for (int j = 0; j < M; ++j) acc[j] = fmaf(e[j], inv, acc[j]);
    }
    // the warp's groups, its lanes' slots in expert order, then the CTA's warps
#pragma unroll
    for (int d = G; d < 32; d *= 2) {
        z2 += __shfl_xor_sync(kAll, z2, d);
#pragma unroll
        for (int j = 0; j < M; ++j) acc[j] += __shfl_xor_sync(kAll, acc[j], d);
    }
    if (sub == 0) {
#pragma unroll
        for (int j = 0; j < M; ++j) sums[warp][expert_of<G, VEC>(lane, j)] = acc[j];
    }
    if (threadIdx.x % 32 == 0) zs[warp] = z2;
    __syncthreads();
    const size_t out = (size_t)blockIdx.x * p.E;
    for (int e = threadIdx.x; e < p.E; e += kSumThreads<M>) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[w][e];
        p.part[out + e] = s;
        p.cpart[out + e] = count[e];
    }
    if (threadIdx.x == 0) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w) s += zs[w];
        p.zpart[blockIdx.x] = s;
    }
}

// Tokens in use of all sequences, and how many sequences have any. A warp, or the warps of a block with a
// part each, walk the sequences. (When every CTA did, and CTAs were as many as the sequences, the time
// grew with their square: 16384 of one token took 10 ms.)
struct Lengths {
    long long all;
    int some;
};
__device__ __forceinline__ Lengths warp_lengths(Lengths n) {
    for (int d = 16; d > 0; d /= 2) {
        n.all += __shfl_xor_sync(kAll, n.all, d);
        n.some += __shfl_xor_sync(kAll, n.some, d);
    }
    return n;
}
// Of the sequences first, first + step, ... of each thread, for a whole warp.
__device__ __forceinline__ void put_lengths(const BalanceParams &p, int first, int step, Lengths &out) {
    Lengths n = {0, 0};
    if (p.num_tokens) {
#pragma unroll 4
        for (long long s = first; s < p.seqs; s += step) {
            const int own = length_of(p, (int)s);
            n.all += own, n.some += own > 0;
        }
        n = warp_lengths(n);
    } else if (first < 32) {
        n = {(long long)p.seqs * p.T, p.seqs};
    }
    if (threadIdx.x % 32 == 0) out = n;
}
template <int WARPS>
__device__ __forceinline__ Lengths total_lengths(const Lengths (&parts)[WARPS]) {
    const int lane = threadIdx.x % 32;
    return warp_lengths(lane < WARPS ? parts[lane] : Lengths{0, 0});
}
// Pools that have tokens.
__device__ __forceinline__ int pools_in_use(const BalanceParams &p, Lengths n) {
    return p.pools == p.seqs ? n.some : n.all > 0;
}

// A fp32 sum with what rounding took from it. (In 64 bits, of which this GPU does two additions a
// cycle and SM, the second kernel and the gradient's few divisions took more time than all the rest:
// 8 sequences of 1024 tokens, both directions, 46 us.)
struct Sum {
    float s = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float sum = __fadd_rn(s, v), part = __fsub_rn(sum, s);
        lost += __fadd_rn(__fsub_rn(s, __fsub_rn(sum, part)), __fsub_rn(v, part));
        s = sum;
    }
    __device__ __forceinline__ float value() const { return s <= FLT_MAX ? s + lost : s; }   // (infinite: lost is NaN)
};
__device__ __forceinline__ float warp_sum(float v) {
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// One CTA per pool and slice of 32 experts: the chunks' sums in order, the counts, and the
// slice's part of the pool's loss; the last CTA to finish adds the parts up.
__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(const BalanceParams p) {
    constexpr int kRows = kFinishThreads / kSlice;
    __shared__ float ps[kRows][kSlice + 1];
    __shared__ int32_t cs[kRows][kSlice + 1];
    __shared__ float parts[2][kFinishThreads / 32];
    __shared__ Lengths lens[kFinishThreads / 32];
    __shared__ bool last;
    pdl_launch_dependents();
    pdl_wait();
    const int slices = (p.E + kSlice - 1) / kSlice;
    const int pool = blockIdx.x / slices, slice = blockIdx.x % slices;
    const int col = threadIdx.x % kSlice, row = threadIdx.x / kSlice, e = slice * kSlice + col;
    const bool own = p.pools == p.seqs;   // a pool is a sequence
    const bool few = !p.num_tokens || p.seqs <= kFinishThreads;   // one warp walks them while the others add up
    const int length = own ? length_of(p, pool) : 0;
    Sum sum;
    int32_t count = 0;
    if (e < p.E) {
        const size_t at = (size_t)pool * p.chunks * p.E + e;
#pragma unroll 5
        for (int c = row; c < p.chunks; c += kRows) {
            sum.add(p.part[at + (size_t)c * p.E]);
            count += p.cpart[at + (size_t)c * p.E];
        }
    }
    ps[row][col] = sum.value(), cs[row][col] = count;
    if (few) {
        if (row == kRows - 1) put_lengths(p, col, 32, lens[0]);
    } else if (!own) {
        put_lengths(p, threadIdx.x, kFinishThreads, lens[row]);
    }
    __syncthreads();
    const long long tokens = own ? length : few ? lens[0].all : total_lengths(lens).all;
    // a warp per expert adds the rows up by a tree
    const float psum = warp_sum(ps[col][row]);
    const int32_t csum = __reduce_add_sync(kAll, cs[col][row]);
    const int e2 = slice * kSlice + row;
    if (col == 0) {
        float v = 0.f;
        if (e2 < p.E) {
            p.counts[(size_t)pool * p.E + e2] = csum;
            if (tokens > 0) v = (float)csum * p.E / ((float)p.K * tokens) * (psum / tokens);
        }
        parts[0][row] = v;
    }
    __syncthreads();
    if (row == 0) {
        const float v = warp_sum(parts[0][col]);
        if (col == 0) {
            p.slots[blockIdx.x] = v;
            __threadfence();
            last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (own && !few) put_lengths(p, threadIdx.x, kFinishThreads, lens[row]);
    Sum b, z;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kFinishThreads) b.add(__ldcg(p.slots + i));
    const long long all = (long long)p.pools * p.chunks;
    for (long long i = threadIdx.x; i < all; i += kFinishThreads) z.add(p.zpart[i]);
    const float bw = warp_sum(b.value()), zw = warp_sum(z.value());
    if (threadIdx.x % 32 == 0) parts[0][threadIdx.x / 32] = bw, parts[1][threadIdx.x / 32] = zw;
    __syncthreads();
    if (threadIdx.x < 32) {
        const float bs = warp_sum(parts[0][threadIdx.x]), zt = warp_sum(parts[1][threadIdx.x]);
        const Lengths n = few ? lens[0] : total_lengths(lens);
        const int pools = pools_in_use(p, n);
        if (threadIdx.x == 0) {
            p.losses[0] = pools > 0 ? bs / pools : 0.f;
            p.losses[1] = n.all > 0 ? zt / n.all : 0.f;
        }
    }
}

template <int G, int M, bool BF16, bool VEC>
__device__ __forceinline__ void store_row(const BalanceParams &p, long long row, int lane, float (&d)[M]) {
    if (VEC) {
#pragma unroll
        for (int c = 0; c < M / 8; ++c) {
            const int e = (c * G + lane) * 8;
            if (e >= p.E) continue;
            const size_t at = (size_t)row * p.E + e;
            float *v = d + 8 * c;
            if (BF16) {
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.dlogits) + at);
                if (p.accumulate) {
                    const uint4 old = *out;
                    const uint32_t w[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 f = unpack_bf16x2(w[q]);
                        v[2 * q] += f.x, v[2 * q + 1] += f.y;
                    }
                }
                *out = make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                                  pack_bf16x2_rn(v[6], v[7]));
            } else {
                float4 *out = reinterpret_cast<float4 *>(static_cast<float *>(p.dlogits) + at);
                if (p.accumulate) {
                    const float4 a = out[0], b = out[1];
                    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
                    v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
                }
                out[0] = make_float4(v[0], v[1], v[2], v[3]);
                out[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const int e = expert_of<G, VEC>(lane, j);
            if (e >= p.E) continue;
            const size_t at = (size_t)row * p.E + e;
            if (BF16) {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.dlogits) + at;
                *out = __float2bfloat16_rn(p.accumulate ? __bfloat162float(*out) + d[j] : d[j]);
            } else {
                float *out = static_cast<float *>(p.dlogits) + at;
                *out = p.accumulate ? *out + d[j] : d[j];
            }
        }
    }
}

template <int G, int M, bool BF16, bool VEC>
__device__ __forceinline__ void backward_chunk(const BalanceParams &p, Lengths n, int pool, int chunk) {
    constexpr int kAtOnce = kBackThreads / G, kPerWarp = 32 / G;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % G, sub = threadIdx.x % 32 / G;
    const int pools = pools_in_use(p, n);
    const float d0 = p.dlosses[0], d1 = p.dlosses[1];
    const float zunit = n.all > 0 ? 2.f * d1 / n.all : 0.f;
    const long long tokens = p.pools == p.seqs ? length_of(p, pool) : n.all;
    const float unit = tokens > 0 ? d0 * p.E / ((float)p.K * tokens) / ((float)tokens * pools) : 0.f;
    float g[M];
#pragma unroll
    for (int j = 0; j < M; ++j) {
        const int e = expert_of<G, VEC>(lane, j);
        g[j] = e < p.E ? unit * p.counts_in[(size_t)pool * p.E + e] : 0.f;
    }
    const long long lo = (long long)chunk * p.chunk;
    const int end = (int)min((long long)p.rows, lo + p.chunk);
    for (long long r0 = lo + warp * kPerWarp; r0 < end; r0 += kAtOnce) {
        const long long r = r0 + sub;
        const Token t = token_of(p, pool, r, end);
        float z[M], e[M], lse;
        load_row<G, M, BF16, VEC>(p, t, lane, z);
        const Top top = top_of<G, M>(z);
        const float inv = softmax_of<G, M>(z, top, e, lse);
        // The z loss's part. The logsumexp of large logits times its unit may pass the largest float where its
        // share for an expert does not (and then meet a probability of 0): there the share comes first.
        const float zc = zunit != 0.f && !top.odd ? zunit * lse : 0.f;   // (no part where the z loss has none)
        float dot = 0.f;
        if (p.sigmoid) {
            float s[M], rest[M];
            const float sinv = sigmoid_of<G, M, true>(z, top.m, s, rest);
#pragma unroll
            for (int j = 0; j < M; ++j) s[j] *= sinv, dot = fmaf(g[j], s[j], dot);
            dot = group_sum<G>(dot);
#pragma unroll
            for (int j = 0; j < M; ++j) e[j] *= inv, z[j] = fmaf(s[j] * rest[j], g[j] - dot, e[j] * zc);
        } else {
#pragma unroll
            for (int j = 0; j < M; ++j) e[j] *= inv, dot = fmaf(g[j], e[j], dot);
            dot = group_sum<G>(dot) - zc;
#pragma unroll
            for (int j = 0; j < M; ++j) z[j] = e[j] * (g[j] - dot);
        }
        if (top.odd && zunit != 0.f && lse != 0.f) {
#pragma unroll
            for (int j = 0; j < M; ++j) z[j] = fmaf(e[j] * lse, zunit, z[j]);
        }
        if (r >= end || (p.accumulate && !t.used)) continue;   // a group's lanes agree
        if (!t.used) {
#pragma unroll
            for (int j = 0; j < M; ++j) z[j] = 0.f;
        }
        store_row<G, M, BF16, VEC>(p, p.pools == p.seqs ? (long long)pool * p.T + r : r, lane, z);
    }
}

// A CTA for each chunk; with MANY a CTA takes several, so that the sequences are not walked as often as there
// are chunks. (A loop around all cases takes registers from the tokens: 64000 of 256, 26.2 us without, 28.6 with.
// Five CTAs an SM hold the registers of narrow groups at 48, from 59 to 62 otherwise.)
template <int G, int M, bool BF16, bool VEC, bool MANY>
__global__ void __launch_bounds__(kBackThreads, VEC && G < 32 && !MANY ? 5 : 0) balance_backward_kernel(const BalanceParams p) {
    __shared__ Lengths lens[kBackThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const bool few = !p.num_tokens || p.seqs <= kBackThreads;
    if (!few) put_lengths(p, threadIdx.x, kBackThreads, lens[threadIdx.x / 32]);
    else if (threadIdx.x < 32) put_lengths(p, threadIdx.x, 32, lens[0]);
    __syncthreads();
    const Lengths n = few ? lens[0] : total_lengths(lens);
    if (!MANY) return backward_chunk<G, M, BF16, VEC>(p, n, blockIdx.x / p.chunks, blockIdx.x % p.chunks);
    for (unsigned at = blockIdx.x; at < (unsigned)p.pools * (unsigned)p.chunks; at += gridDim.x)
        backward_chunk<G, M, BF16, VEC>(p, n, at / p.chunks, at % p.chunks);
}

constexpr long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Tokens that a CTA of the sums takes at once, for E experts.
int sum_step(int E) { return E <= 64 ? 64 : E <= 128 ? 32 : E <= 256 ? 16 : 8; }

// Chunks of a pool's rows: two CTAs per SM over all pools, each with a step's tokens at least.
void cut(BalanceParams &p, int step, int most) {
    const long long share = most / p.pools > 1 ? most / p.pools : 1;
    const long long steps = ceil_div(p.rows, step);
    long long chunk = ceil_div(steps, steps < share ? steps : share) * step;
    if (chunk > kMaxChunk) chunk = kMaxChunk;
    p.chunk = (int)chunk;
    p.chunks = (int)ceil_div(p.rows, chunk);
}

bool balance_params(const ep_balance_t *a, BalanceParams &p) {
    if (!a || a->seqs < 0 || a->tokens < 0 || a->E < 1 || a->E > EP_MAX_E || a->top_k < 1 || a->top_k > EP_MAX_TOPK ||
        a->top_k > a->E || (a->score != EP_SCORE_SOFTMAX && a->score != EP_SCORE_SIGMOID) ||
        (a->per_sequence != 0 && a->per_sequence != 1) || (a->logits_dtype != EP_BF16 && a->logits_dtype != EP_F32) ||
        (long long)a->seqs * a->tokens > INT32_MAX || reinterpret_cast<uintptr_t>(a->num_tokens) % 4)
        return false;
    p = {};
    p.num_tokens = a->num_tokens;
    p.seqs = a->seqs;
    p.T = a->tokens;
    p.E = a->E;
    p.K = a->top_k;
    p.sigmoid = a->score == EP_SCORE_SIGMOID;
    p.pools = a->per_sequence ? a->seqs : 1;
    p.rows = a->per_sequence ? a->tokens : a->seqs * a->tokens;
    // (with one sequence the two are the same)
    return true;
}

size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }

// Places the workspace's parts behind `base`; returns their size.
size_t place(BalanceParams &p, uint8_t *base) {
    const size_t slices = ceil_div(p.E, kSlice), chunks = (size_t)p.pools * p.chunks;
    size_t at = 0;
    p.ticket = reinterpret_cast<uint32_t *>(base);
    at += 16;
    p.slots = reinterpret_cast<float *>(base + at);
    at += align16(p.pools * slices * 4);
    p.zpart = reinterpret_cast<float *>(base + at);
    at += align16(chunks * 4);
    p.part = reinterpret_cast<float *>(base + at);
    at += align16(chunks * p.E * 4);
    p.cpart = reinterpret_cast<int32_t *>(base + at);
    return at + align16(chunks * p.E * 4);
}

bool aligned_to(const void *q, size_t n) { return q && reinterpret_cast<uintptr_t>(q) % n == 0; }

template <int G, int M, bool MANY>
cudaError_t launch_backward(const BalanceParams &p, bool bf16, bool vec, unsigned ctas, cudaStream_t st) {
    const auto kernel = bf16 ? (vec ? balance_backward_kernel<G, M, true, true, MANY> : balance_backward_kernel<G, M, true, false, MANY>)
                             : (vec ? balance_backward_kernel<G, M, false, true, MANY> : balance_backward_kernel<G, M, false, false, MANY>);
    return launch_after(kernel, dim3(ctas), kBackThreads, st, p);
}

template <bool BACKWARD, int G, int M>
cudaError_t launch_n(const BalanceParams &p, bool bf16, bool vec, cudaStream_t st) {
    const unsigned ctas = (unsigned)(p.pools * (long long)p.chunks);
    if (BACKWARD) {
        // (without lengths there is nothing to walk)
        if (p.num_tokens && ctas > kMaxBackCtas) return launch_backward<G, M, true>(p, bf16, vec, kMaxBackCtas, st);
        return launch_backward<G, M, false>(p, bf16, vec, ctas, st);
    }
    const auto kernel = bf16 ? (vec ? balance_sums_kernel<G, M, true, true> : balance_sums_kernel<G, M, true, false>)
                             : (vec ? balance_sums_kernel<G, M, false, true> : balance_sums_kernel<G, M, false, false>);
    return launch_after(kernel, dim3(ctas), kSumThreads<M>, st, p);
}

// Lanes of a token: few experts leave lanes of a warp to other tokens.
template <bool BACKWARD>
cudaError_t launch_rows(const BalanceParams &p, bool bf16, cudaStream_t st) {
    const void *other = BACKWARD ? p.dlogits : p.logits;
    const bool vec = p.E % 8 == 0 && aligned_to(p.logits, 16) && aligned_to(other, 16);
    if (p.E <= 64) return launch_n<BACKWARD, 8, 8>(p, bf16, vec, st);
    if (p.E <= 128) return launch_n<BACKWARD, 16, 8>(p, bf16, vec, st);
    if (p.E <= 256) return launch_n<BACKWARD, 32, 8>(p, bf16, vec, st);
    if (p.E <= 512) return launch_n<BACKWARD, 32, 16>(p, bf16, vec, st);
    return launch_n<BACKWARD, 32, 32>(p, bf16, vec, st);
}

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

}  // namespace

}  // namespace ep

using namespace ep;

extern "C" int ep_balance_workspace_bytes(const ep_balance_t *a, size_t *bytes) {
    BalanceParams p;
    if (!bytes || !balance_params(a, p)) return EP_ERR_INVALID_ARG;
    *bytes = 0;
    if (p.pools == 0 || p.rows == 0) return EP_OK;
    cut(p, sum_step(p.E), kMaxChunks);
    *bytes = place(p, nullptr);
    return EP_OK;
}

extern "C" int ep_balance_loss(const ep_balance_t *a, const void *logits, const int32_t *topk_ids, float *losses,
                               int32_t *counts, void *workspace, size_t workspace_bytes, void *stream) {
    BalanceParams p;
    if (!balance_params(a, p)) return EP_ERR_INVALID_ARG;
    if (!aligned_to(losses, 4) || (p.pools > 0 && !aligned_to(counts, 4))) return EP_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    Range range("ep:balance_loss");
    if (p.pools == 0 || p.rows == 0) {   // no tokens
        if (cudaMemsetAsync(losses, 0, 2 * sizeof(float), st) != cudaSuccess) return EP_ERR_CUDA;
        if (p.pools > 0 && cudaMemsetAsync(counts, 0, (size_t)p.pools * p.E * 4, st) != cudaSuccess) return EP_ERR_CUDA;
        return EP_OK;
    }
    const bool bf16 = a->logits_dtype == EP_BF16;
    if (!aligned_to(logits, bf16 ? 2 : 4) || !aligned_to(topk_ids, 4)) return EP_ERR_INVALID_ARG;
    cut(p, sum_step(p.E), kMaxChunks);
    if (!aligned_to(workspace, 16) || workspace_bytes < place(p, static_cast<uint8_t *>(workspace)))
        return EP_ERR_WORKSPACE;
    const long long slices = ceil_div(p.E, kSlice);
    if (p.pools * slices > INT32_MAX || p.pools * (long long)p.chunks > INT32_MAX) return EP_ERR_INVALID_ARG;
    p.logits = logits;
    p.ids = topk_ids;
    p.losses = losses;
    p.counts = counts;
    if (launch_rows<false>(p, bf16, st) != cudaSuccess) return EP_ERR_CUDA;
    return launch_after(balance_finish_kernel, dim3((unsigned)(p.pools * slices)), kFinishThreads, st, p) == cudaSuccess
               ? EP_OK
               : EP_ERR_CUDA;
}

extern "C" int ep_balance_loss_backward(const ep_balance_t *a, const float *dlosses, const void *logits,
                                        const int32_t *counts, int32_t accumulate, void *dlogits, void *stream) {
    BalanceParams p;
    if (!balance_params(a, p) || (accumulate != 0 && accumulate != 1)) return EP_ERR_INVALID_ARG;
    if (p.pools == 0 || p.rows == 0) return EP_OK;
    const bool bf16 = a->logits_dtype == EP_BF16;
    if (!aligned_to(dlosses, 4) || !aligned_to(logits, bf16 ? 2 : 4) || !aligned_to(counts, 4) ||
        !aligned_to(dlogits, bf16 ? 2 : 4))
        return EP_ERR_INVALID_ARG;
    // a CTA reads the counts and lengths once, so it takes several steps where tokens are many
    const int at_once = kBackThreads / (p.E <= 64 ? 8 : p.E <= 128 ? 16 : 32);
    cut(p, at_once, kMaxBackCtas);
    if (p.pools * (long long)p.chunks > INT32_MAX) return EP_ERR_INVALID_ARG;
    p.dlosses = dlosses;
    p.logits = logits;
    p.counts_in = counts;
    p.accumulate = accumulate;
    p.dlogits = dlogits;
    Range range("ep:balance_loss_backward");
    return launch_rows<true>(p, bf16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
