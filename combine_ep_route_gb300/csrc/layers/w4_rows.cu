// w4_rows.cu -- products with 4-bit weights for few rows of x, and the entry point.
//
// The weight's codes bound it, and for a single small weight the latency of getting them. A CTA
// takes 16 rows of the weight (of a gated one 8 gate rows and the 8 up rows that belong to them)
// and all of k, which bulk copies bring to shared memory in one piece where three CTAs' pieces fit
// an SM, else in chunks, three on their way at a time; a chunk's elements are split over the warps.
// Each lane takes 32 elements, 16 bytes, of two weight rows at a time, makes bf16 pairs of them and multiplies them with one or two tiles of
// eight rows of x by mma.sync (m16n8k16, the weight's rows along m): an MMA's contraction may take the
// elements in any order that both operands share, so a lane's elements are those that lie
// together in memory. (tcgen05.mma wants 128 weight rows at once; few rows of x make no use of its
// rate.) The warps' sums are joined in shared memory, in order. One row, 7168 x 7168: 9.5 us with the
// weight in L2, 11.7 from HBM (2.2 TB/s; 3.8 us at the copy's rate), of which about 7 are start and end.
#include "w4.cuh"

#include <nvtx3/nvToolsExt.h>

#include "act.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace ep {

namespace {

constexpr int kFewRows = 16;   // row slots of a group that this kernel takes
constexpr long long kFewBytes = 28 << 20;   // through L2, for up to eight rows whole
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;      // of the weight
constexpr int kSub = 128;      // elements of k that a warp takes at once: 32 per lane of a row's four
constexpr int kStages = 3;
constexpr int kSmBytes = 228 * 1024;     // shared memory of an SM
constexpr int kWholeBytes = 74 * 1024;   // of a piece, so that three CTAs fit an SM
constexpr int kCodePad = 64;   // bytes between rows of codes, of x: their banks differ
constexpr int kXPad = 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr uint32_t kSleepNs = 1000000;
constexpr uint64_t kPollNs = 100000;     // limits below are kept by polling: a suspended try may last 20 us

struct RowsParams {
    W4Params w;
    int chunk;        // elements of k of a stage, a multiple of kSub * kWarps
    int stages, stage_bytes;
    int32_t *status;
    uint64_t wait_limit_ns;
    uint32_t sleep_ns;   // of a try at a wait, at most; 0: polled
};

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Whether a stage is there: after a suspended try, or at once.
__device__ __forceinline__ bool try_stage(uint64_t *bar, uint32_t parity, uint32_t sleep_ns) {
    if (sleep_ns > 0) return mbar_try_wait_ns(bar, parity, sleep_ns);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// 32 elements of two weight rows against NT tiles of x.
template <int NT, bool FP4, bool LARGE>
__device__ __forceinline__ void multiply(float (&acc)[NT][4], const uint4 (&code)[2], const __nv_bfloat16 (&raw)[2],
                                         const uint8_t *x, uint32_t x_stride, int cols, int r) {
    const W4Scale<FP4> s0(raw[0]), s1(raw[1]);
    const uint32_t words[2][4] = {{code[0].x, code[0].y, code[0].z, code[0].w}, {code[1].x, code[1].y, code[1].z, code[1].w}};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t a[2][4];
        w4_values<FP4, LARGE>(words[0][w], s0, a[0]);
        w4_values<FP4, LARGE>(words[1][w], s1, a[1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint4 b = make_uint4(0, 0, 0, 0);
            if (j * 8 + r < cols) b = *reinterpret_cast<const uint4 *>(x + (j * 8) * x_stride + w * 16);
            mma_16x8x16(acc[j], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
            mma_16x8x16(acc[j], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
        }
    }
}

template <int NT, bool FP4, bool GATED>
__global__ void __launch_bounds__(kThreads) w4_rows_kernel(const RowsParams q) {
    constexpr int kFeatures = GATED ? 8 : 16;   // of the output
    constexpr int kCols = NT * 8;
    const W4Params &p = q.w;
    extern __shared__ __align__(128) uint8_t stages[];
    __shared__ uint64_t full[kStages];
    __shared__ int abort;
    auto &sums = *reinterpret_cast<float(*)[kWarps][kRows][kCols + 1]>(stages);   // once the stages have been read
    const int g = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
        abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    const int f0 = blockIdx.x * kFeatures;
    if (warp == 0 && !p.counts) {
        // the codes on their way to L2 while the kernel before ends (no read: what that may still write to
        // them is written to L2 as well); two rows, which are neighbours, to every fourth lane
        const int i = lane / 4 * 2, f = f0 + (GATED ? i % 8 : i);
        if (lane % 4 == 0 && f < p.n)
            prefetch_l2(p.codes + ((size_t)g * p.wide + f + (GATED ? i / 8 * p.n : 0)) * (p.k / 2), p.k);
    }
    pdl_wait();
    const int count = p.counts ? max(0, min(p.counts[g], p.rows)) : p.rows;
    if (count == 0) return;
    const int cols = min(count, kCols);   // (rows fit: the launch takes NT for them)
    const int chunks = (p.k + q.chunk - 1) / q.chunk;
    const uint32_t code_stride = q.chunk / 2 + kCodePad, x_stride = q.chunk * 2 + kXPad;
    // row i of the CTA's 16 (past the last feature: the last, which nobody looks at)
    const auto weight_row = [&](int i) {
        return GATED ? min(f0 + i % 8, p.n - 1) + i / 8 * p.n : min(f0 + i, p.n - 1);
    };
    const uint8_t *codes = p.codes + (size_t)g * p.wide * (p.k / 2);
    const uint8_t *x = reinterpret_cast<const uint8_t *>(p.x + (size_t)g * p.rows * p.k);

    // A chunk's copies: a lane for each row of codes and of x.
    const auto load = [&](int c) {
        const int s = c % q.stages, k0 = c * q.chunk, n = min(q.chunk, p.k - k0);
        uint8_t *stage = stages + s * q.stage_bytes;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], kRows * n / 2 + cols * n * 2);
        __syncwarp();
        if (lane < kRows)
            bulk_g2s(stage + lane * code_stride, codes + (size_t)weight_row(lane) * (p.k / 2) + k0 / 2, n / 2, &full[s]);
        else if (lane - kRows < cols)
            bulk_g2s(stage + kRows * code_stride + (lane - kRows) * x_stride, x + ((size_t)(lane - kRows) * p.k + k0) * 2,
                     n * 2, &full[s]);
    };
    if (warp == 0)
        for (int c = 0; c < min(chunks, q.stages); ++c) load(c);

    const int r = lane / 4, t = lane % 4;
    const int row[2] = {weight_row(r), weight_row(r + 8)};
    const __nv_bfloat16 *scales = p.scales + (size_t)g * (p.k >> p.group_shift) * p.wide;
    const int subs = q.chunk / (kSub * kWarps);   // of a chunk, for each warp
    const auto load_scales = [&](int e, __nv_bfloat16 (&raw)[2]) {   // of 32 elements from e on
#pragma unroll
        for (int i = 0; i < 2; ++i)
            raw[i] = e < p.k ? scales[(size_t)(e >> p.group_shift) * p.wide + row[i]] : __ushort_as_bfloat16(0);
    };
    float acc[NT][4] = {};
    bool ok = true;
    int c = 0;
    for (; c < chunks; ++c) {
        const int s = c % q.stages, k0 = c * q.chunk;
        __nv_bfloat16 next[2];   // on their way while the copies are waited for, and a step ahead from then on
        load_scales(k0 + warp * kSub + t * 32, next);
        if (!try_stage(&full[s], (c / q.stages) & 1, q.sleep_ns)) {
            const uint64_t since = global_ns();
            while (!try_stage(&full[s], (c / q.stages) & 1, q.sleep_ns)) {
                if (*(volatile int *)&abort || global_ns() - since > q.wait_limit_ns) {
                    abort = 1;
                    atomicCAS(q.status, 0, EP_ERR_TIMEOUT);
                    ok = false;
                    break;
                }
            }
        }
        if (__syncthreads_or(!ok)) break;   // (one has given up: all leave together)
        const uint8_t *stage = stages + s * q.stage_bytes;
        for (int u = 0; u < subs; ++u) {
            const int at = (u * kWarps + warp) * kSub + t * 32;   // this lane's first element in the chunk
            if (k0 + at - t * 32 >= p.k) break;                   // the same for the whole warp
            const __nv_bfloat16 raw[2] = {next[0], next[1]};
            if (u + 1 < subs) load_scales(k0 + at + kWarps * kSub, next);
            uint4 code[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            const bool in = k0 + at < p.k;
            if (in) {
                code[0] = *reinterpret_cast<const uint4 *>(stage + r * code_stride + at / 2);
                code[1] = *reinterpret_cast<const uint4 *>(stage + (r + 8) * code_stride + at / 2);
            }
            const uint8_t *xs = stage + kRows * code_stride + r * x_stride + at * 2;
            const int use = in ? cols : 0;
            if (__any_sync(kAll, is_large<FP4>(raw[0]) || is_large<FP4>(raw[1])))
                multiply<NT, FP4, true>(acc, code, raw, xs, x_stride, use, r);
            else
                multiply<NT, FP4, false>(acc, code, raw, xs, x_stride, use, r);
        }
        if (c + q.stages < chunks) {
            __syncthreads();   // the stage has been read
            if (warp == 0) load(c + q.stages);
        }
    }
    if (c < chunks) {   // a wait ran out: the copies in flight are to finish (bounded)
        if (threadIdx.x == 0) {
            const uint64_t since = global_ns();
            for (int i = c; i < min(chunks, c + q.stages); ++i)
                while (!mbar_try_wait(&full[i % q.stages], (i / q.stages) & 1) && global_ns() - since < 100000000ull)
                    ;
        }
        __syncthreads();
        return;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[warp][(i / 2) * 8 + r][j * 8 + t * 2 + i % 2] = acc[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kFeatures * cols; i += kThreads) {
        const int f = i % kFeatures, col = i / kFeatures;
        if (f0 + f >= p.n) continue;
        float z = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            z += sums[w][f][col];
            if (GATED) up += sums[w][f + 8][col];
        }
        if (p.bias) {
            const __nv_bfloat16 *b = p.bias + (size_t)g * p.wide + f0 + f;
            z += __bfloat162float(*b);
            if (GATED) up += __bfloat162float(b[p.n]);
        }
        float y = GATED ? act_value(z, EP_ACT_SILU) * up : act_value(z, p.act);
        const size_t o = ((size_t)g * p.rows + col) * p.n + f0 + f;
        if (p.residual) y += __bfloat162float(p.residual[o]);
        p.out[o] = __float2bfloat16_rn(y);
    }
}

template <int NT>
cudaError_t launch_n(const RowsParams &q, bool fp4, cudaStream_t st) {
    const bool gated = q.w.act == EP_ACT_SWIGLU;
    const int features = gated ? 8 : 16;
    const auto kernel = gated ? (fp4 ? w4_rows_kernel<NT, true, true> : w4_rows_kernel<NT, false, true>)
                              : (fp4 ? w4_rows_kernel<NT, true, false> : w4_rows_kernel<NT, false, false>);
    const size_t sums = (size_t)kWarps * kRows * (NT * 8 + 1) * sizeof(float), stages = (size_t)q.stages * q.stage_bytes;
    const size_t smem = stages > sums ? stages : sums;
    // (raised from 47 KB on: the default limit counts the kernel's own variables too)
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(kernel), smem + 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((q.w.n + features - 1) / features), (unsigned)q.w.groups);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, q);
}

bool aligned16(const void *q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

// How a call is cut: the elements of a piece, and the pieces a CTA holds.
void cut_rows(const W4Params &w, RowsParams &q) {
    const int rows = w.rows < kFewRows ? w.rows : kFewRows, unit = kSub * kWarps;
    const auto bytes = [&](int chunk) {
        return (kRows * (chunk / 2 + kCodePad) + rows * (chunk * 2 + kXPad) + 127) / 128 * 128;
    };
    // All of k with a copy for a row, where it fits (one row of x, 7168 x 7168, the weight in L2: 11.6 us in
    // chunks of 2048 elements, 9.6 whole; from HBM 11.7 either way). Else three stages of 1024 elements, or
    // of 2048 where x is small.
    const int whole = (w.k + unit - 1) / unit * unit;
    q.chunk = bytes(whole) <= kWholeBytes ? whole : rows <= 2 ? 2 * unit : unit;
    q.stages = q.chunk == whole ? 1 : kStages;
    q.stage_bytes = bytes(q.chunk);
}

// Whether this kernel takes a call (of 16 row slots at most), or the tiles. A CTA for 16 weight rows reads
// all of x again, so beside n k / 2 bytes of codes rows / 4 times as many of x pass through L2; the tiles
// read x once for 128 or 256 weight rows, but begin later. Measured, in us, here / the tiles:
// 1. up to 8 rows held whole: 4096 x 2048 with 1, 8 rows 4.8 / 8.1, 5.1 / 8.2; at 24 MiB through L2 8 x 2048 x
//    1024 7.7 / 8.1; at 35, 28672 x 1024 with 6 rows 11.2 / 11.5, and past that even or slower (64 experts of
//    7168 x 2048 with 4 row slots 192 / 115). One row alone, held whole, wins at any n: 7168 x 7168 11.5 / 14.6;
// 2. while all CTAs find room at once, three an SM or what their shared memory allows, more rows win too:
//    7168 x 2048 with 14 rows 5.8 / 9.1. A second round costs as much again: 4096 x 2048 with 14, 15 rows (in
//    chunks, one CTA an SM) 5.4 / 8.3, 10.0 / 8.3; 1024 CTAs of 32 x 512 x 512 with 12 rows 10.5 / 7.3;
// 3. each chunk of k costs 2.2 us, and the tiles share a long k among CTAs where no counts are given: 1024 x
//    7168 with 8 rows 13.3 / 9.8 without, 13.3 / 19.3 with counts; one row, 2048 x 16384, 20.6 / 15.1.
// Over 252 calls of 1 to 16 rows (both kernels timed on each) the one taken is within 8 % of the better but for
// eight, which lose 1.6 us at most.
bool few_rows_here(const W4Params &w, int sms) {
    RowsParams q = {};
    cut_rows(w, q);
    const bool whole = q.stages == 1;
    if (whole && w.groups == 1 && w.rows == 1) return true;
    const long long codes = (long long)w.groups * w.wide * w.k / 2;   // below 2^50
    if (whole && w.rows <= 8 && codes * (4 + w.rows) / 4 <= kFewBytes) return true;
    const int held = kSmBytes / (q.stages * q.stage_bytes + 1024);
    const bool at_once = (long long)w.groups * ((w.wide + kRows - 1) / kRows) <= (long long)sms * (held < 3 ? held : 3);
    return at_once && (whole || w.counts || w.k <= 2 * q.chunk);
}

}  // namespace

cudaError_t launch_w4_rows(const W4Params &w, bool fp4, int32_t *status, cudaStream_t st) {
    RowsParams q = {};
    q.w = w;
    q.status = status;
    q.wait_limit_ns = product_wait_limit();
    q.sleep_ns = q.wait_limit_ns < kPollNs ? 0 : q.wait_limit_ns < kSleepNs ? (uint32_t)q.wait_limit_ns : kSleepNs;
    cut_rows(w, q);
    return w.rows <= 8 ? launch_n<1>(q, fp4, st) : launch_n<2>(q, fp4, st);
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
    bool few = a->rows <= kFewRows;
    if (few) {
        int sms;
        if (sm_count(&sms) != cudaSuccess) return EP_ERR_CUDA;
        few = few_rows_here(p, sms);
    }
    int32_t *status = a->status;
    if (!status && product_status_word(&status) != cudaSuccess) return EP_ERR_CUDA;
    if (!few) return launch_w4_tiles(p, fp4, status, static_cast<cudaStream_t>(stream));
    return launch_w4_rows(p, fp4, status, static_cast<cudaStream_t>(stream)) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
