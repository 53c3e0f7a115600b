// w4_rows.cu -- products with 4-bit weights for few rows of x, and the entry point.
//
// The weight's codes bound it. A CTA takes 16 (or 32) rows of the weight and all of k, split
// over its warps; each lane reads 16 bytes of codes, 32 elements, of two weight rows straight
// into registers, makes bf16 pairs of them and multiplies them with up to four tiles of eight
// rows of x by mma.sync (m16n8k16, the weight's rows along m): an MMA's contraction may take the
// elements in any order that both operands share, so a lane's elements are those that lie
// together in memory. (tcgen05.mma wants its operands in shared or tensor memory and 64 or 128
// weight rows at once; few rows of x make no use of its rate.) The warps' sums are joined in
// shared memory, in order.
#include "w4.cuh"

#include <nvtx3/nvToolsExt.h>

#include "act.cuh"

namespace ep {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 128;     // elements of k that a warp takes at once: 32 per lane of a row's four
constexpr int kFewRows = 16;   // row slots of a group for which this kernel is the faster one
constexpr int kFlight = 2;     // steps whose codes are on their way together

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// MT tiles of 16 weight rows, up to NT tiles of 8 rows of x at once. A gated tile holds 8 gate
// rows and the 8 up rows that belong to them, which are 8 apart in an accumulator.
template <int MT, int NT, bool FP4, bool GATED>
__global__ void __launch_bounds__(kThreads) w4_rows_kernel(const W4Params p) {
    constexpr int kFeatures = MT * (GATED ? 8 : 16);   // of the output
    constexpr int kCols = NT * 8;
    __shared__ float sums[kWarps][MT * 16][kCols + 1];
    pdl_launch_dependents();
    pdl_wait();
    const int g = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int count = p.counts ? max(0, min(p.counts[g], p.rows)) : p.rows;
    const int f0 = blockIdx.x * kFeatures;
    const int r = lane / 4, t = lane % 4;
    // this lane's weight rows (past the last feature: the last, which nobody looks at)
    int row[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i)
        row[i] = GATED ? min(f0 + (i / 2) * 8 + r, p.n - 1) + (i % 2) * p.n : min(f0 + i * 8 + r, p.n - 1);
    const uint8_t *codes = p.codes + (size_t)g * p.wide * (p.k / 2);
    const __nv_bfloat16 *scales = p.scales + (size_t)g * (p.k >> p.group_shift) * p.wide;
    const int steps = (p.k + kStep - 1) / kStep;
    for (int c0 = 0; c0 < count; c0 += kCols) {
        const __nv_bfloat16 *x = p.x + ((size_t)g * p.rows + c0) * p.k;
        const int cols = min(kCols, count - c0);
        float acc[MT][NT][4] = {};
        for (int s0 = warp; s0 < steps; s0 += kWarps * kFlight) {
            uint4 code[kFlight][2 * MT];
            __nv_bfloat16 raw[kFlight][2 * MT];
#pragma unroll
            for (int q = 0; q < kFlight; ++q) {
                const int e = (s0 + q * kWarps) * kStep + t * 32;   // this lane's first element
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                    code[q][i] = make_uint4(0, 0, 0, 0);
                    raw[q][i] = __ushort_as_bfloat16(0);
                    if (e < p.k) {
                        code[q][i] = __ldcs(reinterpret_cast<const uint4 *>(codes + (size_t)row[i] * (p.k / 2) + e / 2));
                        raw[q][i] = scales[(size_t)(e >> p.group_shift) * p.wide + row[i]];
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kFlight; ++q) {
                const int e = (s0 + q * kWarps) * kStep + t * 32;
                if (s0 + q * kWarps >= steps) break;   // the same for the whole warp
                bool large = false;
                W4Scale<FP4> scale[2 * MT];
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                    scale[i] = W4Scale<FP4>(raw[q][i]);
                    large |= scale[i].large();
                }
                large = __any_sync(0xFFFFFFFFu, large);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a[2 * MT][4];
#pragma unroll
                    for (int i = 0; i < 2 * MT; ++i) {
                        const uint4 c = code[q][i];
                        const uint32_t word = w == 0 ? c.x : w == 1 ? c.y : w == 2 ? c.z : c.w;
                        if (large) w4_values<FP4, true>(word, scale[i], a[i]);
                        else w4_values<FP4, false>(word, scale[i], a[i]);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if (j * 8 >= cols) break;
                        uint4 b = make_uint4(0, 0, 0, 0);
                        if (e < p.k && j * 8 + r < cols)
                            b = *reinterpret_cast<const uint4 *>(x + (size_t)(j * 8 + r) * p.k + e + w * 8);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            mma_16x8x16(acc[m][j], a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], b.x, b.y);
                            mma_16x8x16(acc[m][j], a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], b.z, b.w);
                        }
                    }
                }
            }
        }
        __syncthreads();   // the last tile's sums have been read
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[warp][m * 16 + (i / 2) * 8 + r][j * 8 + t * 2 + i % 2] = acc[m][j][i];
        __syncthreads();
        for (int i = threadIdx.x; i < kFeatures * cols; i += kThreads) {
            const int f = i % kFeatures, c = i / kFeatures;
            if (f0 + f >= p.n) continue;
            const int at = GATED ? f / 8 * 16 + f % 8 : f;
            float z = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                z += sums[w][at][c];
                if (GATED) up += sums[w][at + 8][c];
            }
            if (p.bias) {
                const __nv_bfloat16 *b = p.bias + (size_t)g * p.wide + f0 + f;
                z += __bfloat162float(*b);
                if (GATED) up += __bfloat162float(b[p.n]);
            }
            float y = GATED ? act_value(z, EP_ACT_SILU) * up : act_value(z, p.act);
            const size_t o = ((size_t)g * p.rows + c0 + c) * p.n + f0 + f;
            if (p.residual) y += __bfloat162float(p.residual[o]);
            p.out[o] = __float2bfloat16_rn(y);
        }
    }
}

template <int MT, int NT>
cudaError_t launch_n(const W4Params &p, bool fp4, cudaStream_t st) {
    const bool gated = p.act == EP_ACT_SWIGLU;
    const int features = MT * (gated ? 8 : 16);
    const dim3 grid((unsigned)((p.n + features - 1) / features), (unsigned)p.groups);
    const auto kernel = gated ? (fp4 ? w4_rows_kernel<MT, NT, true, true> : w4_rows_kernel<MT, NT, false, true>)
                              : (fp4 ? w4_rows_kernel<MT, NT, true, false> : w4_rows_kernel<MT, NT, false, false>);
    return launch_after(kernel, grid, kThreads, st, p);
}

bool aligned16(const void *q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

}  // namespace

cudaError_t launch_w4_rows(const W4Params &p, bool fp4, cudaStream_t st) {
    if (p.rows <= 8) return launch_n<1, 1>(p, fp4, st);
    if (p.rows <= 16) return launch_n<1, 2>(p, fp4, st);
    return launch_n<1, 4>(p, fp4, st);
}

}  // namespace ep

using namespace ep;

extern "C" int ep_product_w4(const ep_w4_t *a, const void *x, const void *codes, const void *scales, const void *bias,
                             const void *residual, void *out, void *stream) {
    if (!a || a->groups < 1 || a->groups > EP_MAX_E || a->rows < 0 || (long long)a->groups * a->rows >= (1LL << 31))
        return EP_ERR_INVALID_ARG;
    if (a->kind != EP_W4_INT4 && a->kind != EP_W4_FP4) return EP_ERR_INVALID_ARG;
    if (a->group != 32 && a->group != 64 && a->group != 128) return EP_ERR_INVALID_ARG;
    if (a->k < a->group || a->k % a->group || a->k > EP_W4_MAX_K || a->n < 8 || a->n % 8 || a->n > (1 << 24))
        return EP_ERR_INVALID_ARG;
    // a tensor map's strides stay below 2^40 bytes
    if (4LL * a->k * a->rows >= (1LL << 38) || 4LL * a->n * a->rows >= (1LL << 38)) return EP_ERR_INVALID_ARG;
    if (a->act < EP_ACT_NONE || a->act > EP_ACT_SWIGLU) return EP_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->counts) % 4 || reinterpret_cast<uintptr_t>(a->status) % 4) return EP_ERR_INVALID_ARG;
    if (a->rows == 0) return EP_OK;
    if (!x || !codes || !scales || !out || !aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(bias) ||
        !aligned16(residual) || !aligned16(out))
        return EP_ERR_INVALID_ARG;
    W4Params p = {};
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.codes = static_cast<const uint8_t *>(codes);
    p.scales = static_cast<const __nv_bfloat16 *>(scales);
    p.bias = static_cast<const __nv_bfloat16 *>(bias);
    p.residual = static_cast<const __nv_bfloat16 *>(residual);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.counts = a->counts;
    p.groups = a->groups;
    p.rows = a->rows;
    p.k = a->k;
    p.n = a->n;
    p.wide = a->act == EP_ACT_SWIGLU ? 2 * a->n : a->n;
    p.group_shift = a->group == 32 ? 5 : a->group == 64 ? 6 : 7;
    p.act = a->act;
    Range range("ep:product_w4");
    const bool fp4 = a->kind == EP_W4_FP4;
    if (a->rows > kFewRows) return launch_w4_tiles(p, fp4, a->status, static_cast<cudaStream_t>(stream));
    return launch_w4_rows(p, fp4, static_cast<cudaStream_t>(stream)) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
