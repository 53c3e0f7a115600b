// gradnorm.cu -- the global norm of many gradients and their clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * max_norm / norm where norm is finite and above max_norm, else g
//
// Two kernels over the same list of pieces (runs of up to 16384 elements of a tensor): one
// adds squares up, a double per CTA in a fixed place; the other adds those up, again in a
// fixed order, and scales. HBM bounds both: the second walks the pieces backwards, so that
// what the first read last is still in L2, and is over at once where nothing is to be changed.
// 1.44 G elements in 160 tensors (3.26 GB, read twice and written once) take 1509 us, 6.5 TB/s; 200 M in
// 50 tensors 216, 5.9 TB/s; 0.3 M in 12 tensors 8.7 us on the device and 38 with the call's lists.
//
// A square of a fp32 (or bf16) number overflows from 1.8e19 and loses digits below 1e-19, so
// a vector of 16 bytes whose largest magnitude lies outside 2^-50 .. 2^50 is scaled by 2^100
// or 2^-100 before it is squared and goes to a sum of its own.
#include "launch.cuh"

#include <algorithm>
#include <cuda_bf16.h>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "act.cuh"

namespace ep {

namespace {

constexpr int kThreads = 512;        // of the sums' kernel,
constexpr int kMaxCtas = 456;        // whose CTAs are three per SM
// And of the scaling one, which reads and writes: fewer threads on their way do better (1.4 G elements
// with 2, 3, 4, 6 CTAs of 256 per SM: 1757, 1661, 1786, 1812 us in all; three of 512: 1775).
constexpr int kScaleThreads = 256, kMaxScaleCtas = 456;
// Elements of a piece: small ones where all tensors together would leave SMs idle otherwise.
constexpr int kPiece = 16384, kSmallPiece = 2048;
constexpr long long kSmallTotal = 4 << 20;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr double kDoubleMax = 1.7976931348623157e308;

// The tensors of one launch, passed by value: a list in device memory would have to be copied
// there before the launch. Three sizes, since a launch takes longer the more it carries.
template <int N>
struct List {
    const void *in[N];
    void *out[N];
    long long numel[N];
    uint32_t first[N + 1];   // pieces before it
    uint32_t bf16[(N + 31) / 32];
    int n, piece;
};

struct ClipParams {
    double *partial;      // one per CTA of the sums, of all launches
    int partials, base;   // how many there are; where this launch's begin
    float *norm;
    float max_norm;
    int write_norm, copy; // whether this launch writes the norm; copy where nothing is scaled
};

struct Piece {
    const void *in;
    void *out;
    long long begin;
    int count;
    bool bf16;
};

template <int N>
__device__ __forceinline__ Piece piece_of(const List<N> &list, uint32_t i) {
    int lo = 0, hi = list.n;   // first[lo] <= i < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (list.first[mid] <= i) lo = mid;
        else hi = mid;
    }
    Piece x;
    x.begin = (long long)(i - list.first[lo]) * list.piece;
    x.count = (int)min((long long)list.piece, list.numel[lo] - x.begin);
    x.bf16 = (list.bf16[lo / 32] >> (lo % 32)) & 1;
    const size_t at = (size_t)x.begin * (x.bf16 ? 2 : 4);
    x.in = static_cast<const uint8_t *>(list.in[lo]) + at;
    x.out = static_cast<uint8_t *>(list.out[lo]) + at;
    return x;
}

// A sum and what rounding took from it. (This GPU does two 64-bit additions a cycle and SM, so they
// are few: some for a warp's sum and one for each warp and CTA.)
struct Kept {
    float sum = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float s = __fadd_rn(sum, v), part = __fsub_rn(s, sum);
        lost += __fadd_rn(__fsub_rn(sum, __fsub_rn(s, part)), __fsub_rn(v, part));
        sum = s;
    }
    // The warp's, in all lanes.
    __device__ __forceinline__ double warp_total() {
        for (int d = 16; d > 0; d /= 2) {
            const float other = __shfl_xor_sync(kAll, sum, d);
            lost += __shfl_xor_sync(kAll, lost, d);
            // (the same in both: the larger first)
            const float a = fmaxf(sum, other), b = fminf(sum, other);
            sum = sum == sum && other == other ? a : sum + other;
            add(sum == sum ? b : 0.f);
        }
        // (past the largest float `lost` is NaN, and the sum infinite)
        return sum <= 3.402823466e38f ? (double)sum + lost : (double)sum;
    }
};

// mid, low and high are of the piece at hand; kept and odd are of those before it. (Low and high ones kept over all
// pieces in 32 bits alone: 2^30 squares of 1e-32 were off by 6 2^-20. In 64 bits, where there are any, the norm of
// 2^28 elements of 1e-17 or 1e17 takes 157 us instead of 154, that of 1.44 G ordinary ones 495 instead of 488.)
struct Squares {
    float mid = 0.f, low = 0.f, high = 0.f;
    Kept kept;
    double odd = 0.;
    __device__ __forceinline__ void end_piece() {
        kept.add(mid);
        mid = 0.f;
        if (low != 0.f || high != 0.f) {
            odd += (double)low * 0x1p-200 + (double)high * 0x1p200;
            low = high = 0.f;
        }
    }
    // The warp's sum, in all lanes.
    __device__ __forceinline__ double warp_total() {
        const double sum = kept.warp_total();
        if (__any_sync(kAll, odd != 0.))
            for (int d = 16; d > 0; d /= 2) odd += __shfl_xor_sync(kAll, odd, d);
        return sum + odd;
    }
};

template <int N>
__device__ __forceinline__ void add_squares(Squares &s, const float (&v)[N]) {
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) most = fmaxf(most, fabsf(v[j]));
    if (most >= 0x1p-50f && most <= 0x1p50f) {
        float sum = v[0] * v[0];
#pragma unroll
        for (int j = 1; j < N; ++j) sum = fmaf(v[j], v[j], sum);
        s.mid += sum;
    } else {   // (also NaN alone, which leaves the maximum at 0)
        const bool up = most < 1.f;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float u = v[j] * (up ? 0x1p100f : 0x1p-100f);
            sum = fmaf(u, u, sum);
        }
        if (up) s.low += sum;
        else s.high += sum;
    }
}

// Elements before the first that is aligned to 16 bytes.
__device__ __forceinline__ int head_of(const void *p, int size, int count) {
    const int off = (int)(reinterpret_cast<uintptr_t>(p) % 16);
    return off ? min(count, (16 - off) / size) : 0;
}

template <bool BF16>
__device__ __forceinline__ float element(const void *p, int i) {
    return BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void unpack(uint4 x, float (&v)[BF16 ? 8 : 4]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (BF16) {
            const float2 f = unpack_bf16x2(w[q]);
            v[2 * q] = f.x, v[2 * q + 1] = f.y;
        } else {
            v[q] = __uint_as_float(w[q]);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void piece_squares(const Piece &x, Squares &s) {
    constexpr int kVec = BF16 ? 8 : 4, kFlight = 4;
    const int head = head_of(x.in, BF16 ? 2 : 4, x.count);
    const int vecs = (x.count - head) / kVec, tail = head + vecs * kVec;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x.in) + head * (BF16 ? 2 : 4));
    for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * kFlight) {
        uint4 u[kFlight];
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
            const int i = i0 + q * kThreads;
            u[q] = i < vecs ? p[i] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
            float v[kVec];
            unpack<BF16>(u[q], v);
            add_squares(s, v);
        }
    }
    const int rest = head + (x.count - tail);   // at most 14 elements
    if (threadIdx.x < rest) {
        const int i = (int)threadIdx.x < head ? (int)threadIdx.x : tail + (int)threadIdx.x - head;
        const float v[1] = {element<BF16>(x.in, i)};
        add_squares(s, v);
    }
    s.end_piece();
}

template <int N>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ List<N> list, const ClipParams p) {
    __shared__ double parts[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    Squares s;
    const uint32_t pieces = list.first[list.n];
    for (uint32_t i = blockIdx.x; i < pieces; i += gridDim.x) {
        const Piece x = piece_of(list, i);
        if (x.bf16) piece_squares<true>(x, s);
        else piece_squares<false>(x, s);
    }
    const double sum = s.warp_total();
    if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0;
        for (int w = 0; w < kThreads / 32; ++w) all += parts[w];
        p.partial[p.base + blockIdx.x] = all;
    }
}

// What elements are multiplied with: factor, then more, which is 1 unless the two's product is below the
// smallest normal float (a norm of 1e39, or a bound of 1e-30 and elements of 1e10), where one factor would have lost
// its last digits or all.
struct Scale {
    float factor, more;
    __device__ __forceinline__ float of(float v) const { return v * factor * more; }
};

// The norm from the sums, the same in every CTA, and the scale that it asks for (factor -1: none).
__device__ __forceinline__ Scale scale_of(const ClipParams &p, bool write) {
    __shared__ Scale scale;
    if (threadIdx.x < 32) {
        double sum = 0;
        for (int i = threadIdx.x; i < p.partials; i += 32) sum += p.partial[i];
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(kAll, sum, d);
        if (threadIdx.x == 0) {
            const double norm = sqrt(sum);
            if (write) *p.norm = (float)norm;
            // (a NaN compares false)
            const bool clip = norm > (double)p.max_norm && norm <= kDoubleMax;
            const double by = clip ? (double)p.max_norm / norm : -1.;
            const bool tiny = clip && by < 0x1p-126;
            scale = {(float)(tiny ? by * 0x1p126 : by), tiny ? 0x1p-126f : 1.f};
        }
    }
    __syncthreads();
    return scale;
}

template <bool BF16>
__device__ __forceinline__ void scale_piece(const Piece &x, Scale scale) {
    constexpr int kVec = BF16 ? 8 : 4, kFlight = 4, kSize = BF16 ? 2 : 4;
    const bool wide = (reinterpret_cast<uintptr_t>(x.in) - reinterpret_cast<uintptr_t>(x.out)) % 16 == 0;
    const int head = wide ? head_of(x.in, kSize, x.count) : x.count;
    const int vecs = (x.count - head) / kVec, tail = head + vecs * kVec;
    // (plain loads and stores: streaming ones took 3 % longer)
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x.in) + head * kSize);
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(x.out) + head * kSize);
    for (int i0 = threadIdx.x; i0 < vecs; i0 += kScaleThreads * kFlight) {
        uint4 u[kFlight];
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
            const int i = i0 + q * kScaleThreads;
            if (i < vecs) u[q] = p[i];
        }
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
            const int i = i0 + q * kScaleThreads;
            if (i >= vecs) continue;
            float v[kVec];
            unpack<BF16>(u[q], v);
            uint4 r;
            if constexpr (BF16)
                r = make_uint4(pack_bf16x2_rn(scale.of(v[0]), scale.of(v[1])), pack_bf16x2_rn(scale.of(v[2]), scale.of(v[3])),
                               pack_bf16x2_rn(scale.of(v[4]), scale.of(v[5])), pack_bf16x2_rn(scale.of(v[6]), scale.of(v[7])));
            else
                r = make_uint4(__float_as_uint(scale.of(v[0])), __float_as_uint(scale.of(v[1])),
                               __float_as_uint(scale.of(v[2])), __float_as_uint(scale.of(v[3])));
            o[i] = r;
        }
    }
    const int rest = head + (x.count - tail);   // all of it where the two are not alike aligned
    for (int j = threadIdx.x; j < rest; j += kScaleThreads) {
        const int i = j < head ? j : tail + j - head;
        const float v = scale.of(element<BF16>(x.in, i));
        if (BF16) static_cast<__nv_bfloat16 *>(x.out)[i] = __float2bfloat16_rn(v);
        else static_cast<float *>(x.out)[i] = v;
    }
}

template <int N>
__global__ void __launch_bounds__(kScaleThreads) scale_kernel(const __grid_constant__ List<N> list, const ClipParams p) {
    pdl_launch_dependents();
    pdl_wait();
    Scale scale = scale_of(p, p.write_norm && blockIdx.x == 0);
    if (scale.factor < 0.f) {   // nothing to scale
        if (!p.copy) return;
        scale.factor = 1.f;
    }
    const uint32_t pieces = list.first[list.n];
    for (uint32_t i = blockIdx.x; i < pieces; i += gridDim.x) {
        const Piece x = piece_of(list, pieces - 1 - i);
        if (x.bf16) scale_piece<true>(x, scale);
        else scale_piece<false>(x, scale);
    }
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const ClipParams p) {
    pdl_launch_dependents();
    pdl_wait();
    scale_of(p, true);
}

// The tensors [from, to) of the list, as one launch takes them.
struct Part {
    int from, to;
    uint32_t pieces;
    int ctas, base;   // of the sums' kernel, and those of the parts before
};

constexpr int kMost = 512;                     // tensors of a launch
constexpr uint32_t kMostPieces = 1u << 31;     // pieces of a launch

long long pieces_of(long long numel, int piece) { return (numel + piece - 1) / piece; }

int piece_size(const ep_grads_t *a) {
    long long total = 0;
    for (int i = 0; i < a->n && total < kSmallTotal; ++i) total += a->numel[i];
    return total < kSmallTotal ? kSmallPiece : kPiece;
}

// False where a tensor alone has too many pieces.
bool cut(const ep_grads_t *a, std::vector<Part> &parts) {
    const int piece = piece_size(a);
    int base = 0;
    for (int i = 0; i < a->n;) {
        Part x = {i, i, 0, 0, base};
        long long pieces = 0;
        while (x.to < a->n && x.to - x.from < kMost && pieces + pieces_of(a->numel[x.to], piece) < (long long)kMostPieces)
            pieces += pieces_of(a->numel[x.to++], piece);
        if (x.to == x.from) return false;
        x.pieces = (uint32_t)pieces;
        x.ctas = (int)(pieces < kMaxCtas ? pieces : kMaxCtas);
        base += x.ctas;
        i = x.to;
        if (pieces > 0) parts.push_back(x);
    }
    return true;
}

template <int N>
void fill(const ep_grads_t *a, const Part &x, List<N> &list) {
    list.n = 0;
    list.piece = piece_size(a);
    for (uint32_t &w : list.bf16) w = 0;
    uint32_t first = 0;
    for (int i = x.from; i < x.to; ++i) {
        if (a->numel[i] == 0) continue;
        const int at = list.n++;
        list.in[at] = a->grads[i];
        list.out[at] = a->out ? a->out[i] : const_cast<void *>(a->grads[i]);   // (in place)
        list.numel[at] = a->numel[i];
        list.first[at] = first;
        if (a->dtypes[i] == EP_BF16) list.bf16[at / 32] |= 1u << (at % 32);
        first += (uint32_t)pieces_of(a->numel[i], list.piece);
    }
    list.first[list.n] = first;
}

template <int N>
cudaError_t launch_n(const ep_grads_t *a, const Part &x, const ClipParams &p, bool scale, cudaStream_t st) {
    List<N> list;
    fill(a, x, list);
    if (!scale) return launch_after(squares_kernel<N>, dim3((unsigned)x.ctas), kThreads, st, list, p);
    const uint32_t ctas = x.pieces < (uint32_t)kMaxScaleCtas ? x.pieces : (uint32_t)kMaxScaleCtas;
    return launch_after(scale_kernel<N>, dim3(ctas), kScaleThreads, st, list, p);
}

cudaError_t launch_part(const ep_grads_t *a, const Part &x, const ClipParams &p, bool scale, cudaStream_t st) {
    if (x.to - x.from <= 16) return launch_n<16>(a, x, p, scale, st);
    if (x.to - x.from <= 128) return launch_n<128>(a, x, p, scale, st);
    return launch_n<kMost>(a, x, p, scale, st);
}

bool grads_ok(const ep_grads_t *a) {
    if (!a || a->n < 0 || (a->n > 0 && (!a->numel || !a->dtypes))) return false;
    for (int i = 0; i < a->n; ++i)
        if (a->numel[i] < 0 || a->numel[i] >= (1LL << 44) || (a->dtypes[i] != EP_BF16 && a->dtypes[i] != EP_F32)) return false;
    return true;
}

// Whether any two of the byte ranges that are written (or of the gradients, which count once
// each) share a byte, or one that is written overlaps another tensor's gradient.
bool overlap(const ep_grads_t *a) {
    struct Span {
        uintptr_t lo, hi;
        int id;
        bool written;
    };
    std::vector<Span> spans;
    spans.reserve((size_t)a->n * 2);
    for (int i = 0; i < a->n; ++i) {
        if (a->numel[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)a->numel[i] * (a->dtypes[i] == EP_BF16 ? 2 : 4);
        const uintptr_t g = reinterpret_cast<uintptr_t>(a->grads[i]);
        const uintptr_t o = a->out ? reinterpret_cast<uintptr_t>(a->out[i]) : g;
        spans.push_back({g, g + bytes, i, o == g});
        if (o != g) spans.push_back({o, o + bytes, i, true});
    }
    std::sort(spans.begin(), spans.end(), [](const Span &x, const Span &y) { return x.lo < y.lo; });
    uintptr_t read_hi = 0, write_hi = 0;   // ends of what came before
    for (const Span &s : spans) {
        if (s.lo < write_hi || (s.written && s.lo < read_hi)) return true;
        read_hi = std::max(read_hi, s.hi);
        if (s.written) write_hi = std::max(write_hi, s.hi);
    }
    return false;
}

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

int clip(const ep_grads_t *a, float max_norm, float *norm, void *workspace, size_t workspace_bytes, cudaStream_t st) {
    std::vector<Part> parts;
    if (!cut(a, parts)) return EP_ERR_INVALID_ARG;
    ClipParams p = {};
    for (const Part &x : parts) p.partials += x.ctas;
    if (p.partials > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 ||
                           workspace_bytes < (size_t)p.partials * sizeof(double)))
        return EP_ERR_WORKSPACE;
    p.partial = static_cast<double *>(workspace);
    p.norm = norm;
    p.max_norm = max_norm;
    p.copy = a->out != nullptr;
    for (const Part &x : parts) {
        p.base = x.base;
        if (launch_part(a, x, p, false, st) != cudaSuccess) return EP_ERR_CUDA;
    }
    // nothing can be above infinity, so nothing is to be scaled
    if (parts.empty() || (max_norm == __builtin_inff() && !p.copy))
        return launch_after(norm_kernel, dim3(1), kThreads, st, p) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
    // backwards here too; each launch reads all the sums
    for (size_t i = parts.size(); i-- > 0;) {
        p.write_norm = i == 0;
        if (launch_part(a, parts[i], p, true, st) != cudaSuccess) return EP_ERR_CUDA;
    }
    return EP_OK;
}

}  // namespace

}  // namespace ep

using namespace ep;

extern "C" int ep_clip_workspace_bytes(const ep_grads_t *a, size_t *bytes) {
    if (!bytes || !grads_ok(a)) return EP_ERR_INVALID_ARG;
    try {
        std::vector<Part> parts;
        if (!cut(a, parts)) return EP_ERR_INVALID_ARG;
        *bytes = 0;
        for (const Part &x : parts) *bytes += (size_t)x.ctas * sizeof(double);
        return EP_OK;
    } catch (...) {
        return EP_ERR_INVALID_ARG;
    }
}

extern "C" int ep_clip_grad_norm(const ep_grads_t *a, float max_norm, float *norm, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    if (!grads_ok(a) || !(max_norm >= 0.f) || !norm || reinterpret_cast<uintptr_t>(norm) % 4) return EP_ERR_INVALID_ARG;
    for (int i = 0; i < a->n; ++i) {
        if (a->numel[i] == 0) continue;
        const uintptr_t size = a->dtypes[i] == EP_BF16 ? 2 : 4;
        if (!a->grads || !a->grads[i] || reinterpret_cast<uintptr_t>(a->grads[i]) % size) return EP_ERR_INVALID_ARG;
        if (a->out && (!a->out[i] || reinterpret_cast<uintptr_t>(a->out[i]) % size)) return EP_ERR_INVALID_ARG;
    }
    try {
        if (overlap(a)) return EP_ERR_INVALID_ARG;
        Range range("ep:clip_grad_norm");
        return clip(a, max_norm, norm, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
    } catch (...) {   // no host memory
        return EP_ERR_INVALID_ARG;
    }
}
