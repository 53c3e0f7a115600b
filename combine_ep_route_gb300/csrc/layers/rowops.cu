// rowops.cu -- row-wise companions of the products: the bias gradient (a sum of
// rows per group), which latency bounds, and the gradient through an activation that no
// product follows, which HBM does. Both read each byte once.
#include "launch.cuh"

#include <cooperative_groups.h>
#include <nvtx3/nvToolsExt.h>

#include "act.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;        // of the activation's gradient
constexpr int kSumThreads = 512;
constexpr int kVecs = 8;             // 16-byte vectors of a row one CTA covers (64 columns)
constexpr int kRowLanes = kSumThreads / kVecs;
constexpr int kInFlight = 8;         // rows a thread has on their way
constexpr int kSplit = 8;            // CTAs of a cluster that share a group's rows

__device__ __forceinline__ void add_vec(float (&a)[8], uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float2 f = unpack_bf16x2(w[q]);
        a[2 * q] += f.x, a[2 * q + 1] += f.y;
    }
}

// Sums over rows, fp32, in a fixed order: each thread walks rows r, r + 64 * split, ...,
// then the CTA's 64 row threads (by eights) and the cluster's CTAs are added in order.
// Latency bounds it: 5001 x 2048 take 9 us after a weight gradient (20 MB, 3 us at the
// copy's rate); starting beside that kernel's end instead took 7, and was not worth its care.
template <bool OUT_F32>
__global__ void __launch_bounds__(kSumThreads) row_sums_kernel(const uint4 *src, const int32_t *counts, int rows,
                                                               int n, int split, int accumulate, void *out) {
    __shared__ float part[kRowLanes][kVecs * 8 + 1];
    __shared__ float eighth[8][kVecs * 8];
    __shared__ float sums[kVecs * 8];
    pdl_launch_dependents();
    pdl_wait();
    const int g = blockIdx.y, part_id = blockIdx.x % split, tile = blockIdx.x / split;
    const int v = tile * kVecs + threadIdx.x % kVecs, r0 = threadIdx.x / kVecs;
    const int nvec = n / 8;
    const int count = counts ? max(0, min(counts[g], rows)) : rows;
    float a[8] = {};
    if (v < nvec) {
        const uint4 *p = src + (size_t)g * rows * nvec + v;
        const int step = kRowLanes * split;
        for (long long r = part_id * kRowLanes + r0; r < count; r += (long long)kInFlight * step) {
            uint4 x[kInFlight];
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const long long at = r + (long long)i * step;
                x[i] = at < count ? p[(size_t)at * nvec] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) add_vec(a, x[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[r0][(threadIdx.x % kVecs) * 8 + i] = a[i];
    __syncthreads();
    const int c = threadIdx.x;
    {
        const int col = c % (kVecs * 8), e = c / (kVecs * 8);
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRowLanes / 8; ++r) s += part[e * (kRowLanes / 8) + r][col];
        eighth[e][col] = s;
    }
    __syncthreads();
    if (c < kVecs * 8) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += eighth[e][c];
        sums[c] = s;
    }
    if (split > 1) {
        namespace cg = cooperative_groups;
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (part_id == 0 && c < kVecs * 8) {
            float s = 0.f;
            for (int i = 0; i < split; ++i) s += *cluster.map_shared_rank(&sums[c], i);
            sums[c] = s;
        }
        cluster.sync();
    }
    const int col = tile * kVecs * 8 + c;
    if (part_id == 0 && c < kVecs * 8 && col < n) {
        const size_t at = (size_t)g * n + col;
        if (OUT_F32) {
            float *o = static_cast<float *>(out);
            o[at] = accumulate ? o[at] + sums[c] : sums[c];
        } else {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out);
            o[at] = __float2bfloat16_rn(accumulate ? __bfloat162float(o[at]) + sums[c] : sums[c]);
        }
    }
}

// One thread per 16-byte vector of dy, rows in use only. 8192 x 7168: gelu 59.0 us (6.0 TB/s),
// gelu_tanh 56.5 (6.2), relu 56.0 (6.3); 8192 x 4096 through swiglu 52.5 (6.4).
__global__ void __launch_bounds__(kThreads) act_grad_kernel(const uint4 *dy, const uint4 *z, uint4 *dz,
                                                            const int32_t *counts, int rows, int nvec, int act) {
    pdl_launch_dependents();
    pdl_wait();
    const bool gated = act == EP_ACT_SWIGLU;
    const int g = blockIdx.y;
    const int count = counts ? max(0, min(counts[g], rows)) : rows;
    const long long items = (long long)count * nvec;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < items;
         i += (long long)gridDim.x * kThreads) {
        const size_t row = (size_t)g * rows + (size_t)(i / nvec);
        const int v = (int)(i % nvec);
        const size_t zi = row * nvec * (gated ? 2 : 1) + v;
        const uint4 d4 = dy[row * nvec + v], a4 = z[zi];
        const uint4 b4 = gated ? z[zi + nvec] : make_uint4(0, 0, 0, 0);
        const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w}, a[4] = {a4.x, a4.y, a4.z, a4.w},
                       b[4] = {b4.x, b4.y, b4.z, b4.w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 dv = unpack_bf16x2(d[q]), zv = unpack_bf16x2(a[q]), uv = unpack_bf16x2(b[q]);
            if (gated) {
                float2 dg, du;
                swiglu_grad(dv.x, zv.x, uv.x, dg.x, du.x);
                swiglu_grad(dv.y, zv.y, uv.y, dg.y, du.y);
                oa[q] = pack_bf16x2_rn(dg.x, dg.y);
                ob[q] = pack_bf16x2_rn(du.x, du.y);
            } else {
                oa[q] = pack_bf16x2_rn(dv.x * act_slope(zv.x, act), dv.y * act_slope(zv.y, act));
                ob[q] = 0;
            }
        }
        dz[zi] = make_uint4(oa[0], oa[1], oa[2], oa[3]);
        if (gated) dz[zi + nvec] = make_uint4(ob[0], ob[1], ob[2], ob[3]);
    }
}

}  // namespace

cudaError_t launch_row_sums(const void *src, const int32_t *counts, int groups, int rows, int n, bool out_f32,
                            bool accumulate, void *out, cudaStream_t st) {
    const int tiles = (n + kVecs * 8 - 1) / (kVecs * 8);
    // few column tiles with many rows: a cluster's CTAs share the rows
    const int split = (long long)tiles * groups < 512 && rows > 2 * kRowLanes ? kSplit : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split * tiles, groups);
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const uint4 *s = static_cast<const uint4 *>(src);
    return out_f32 ? cudaLaunchKernelEx(&cfg, row_sums_kernel<true>, s, counts, rows, n, split, (int)accumulate, out)
                   : cudaLaunchKernelEx(&cfg, row_sums_kernel<false>, s, counts, rows, n, split, (int)accumulate, out);
}

}  // namespace ep

using namespace ep;

extern "C" int ep_act_grad(const ep_product_t *a, const void *dy, const void *preact, void *dz, void *stream) {
    if (!a || a->groups < 1 || a->groups > EP_MAX_E || a->rows < 0 || a->n < 8 || a->n % 8 || a->n > (1 << 24) ||
        (long long)a->groups * a->rows >= (1LL << 31) || a->act <= EP_ACT_NONE || a->act > EP_ACT_SWIGLU ||
        a->out_dtype != EP_BF16)
        return EP_ERR_INVALID_ARG;
    if (a->rows == 0) return EP_OK;
    if (!dy || !preact || !dz || reinterpret_cast<uintptr_t>(a->counts) % 4)
        return EP_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(preact) | reinterpret_cast<uintptr_t>(dz)) % 16)
        return EP_ERR_INVALID_ARG;
    const long long per_group = ((long long)a->rows * (a->n / 8) + kThreads - 1) / kThreads;
    // about sixteen CTAs per SM in all, however many groups share them
    const long long want = 2432 / a->groups + 1;
    const dim3 grid((unsigned)(per_group < want ? per_group : want), (unsigned)a->groups);
    nvtxRangePushA("ep:act_grad");
    const cudaError_t e = launch_after(act_grad_kernel, grid, kThreads, static_cast<cudaStream_t>(stream),
                                       static_cast<const uint4 *>(dy), static_cast<const uint4 *>(preact),
                                       static_cast<uint4 *>(dz), a->counts, a->rows, a->n / 8, a->act);
    nvtxRangePop();
    return e == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
