// product.cu -- the layers' matrix products on the 5th-generation tensor cores:
// forward (bias, activation, residual), input gradient (through an activation)
// and weight gradient, for one weight or one per expert with ragged row counts.
//
// All three are D[col][lane] = sum_r A[lane][r] B[col][r] with fp32 sums in
// tensor memory. The weights' features sit on the 128 accumulator lanes and the
// tokens on the columns, because the column count of an MMA may be any multiple
// of 16: an expert with 20 rows pays for 32 columns, not for a tile of 128.
// An accumulator column is then one token's row, whose features are contiguous
// in memory across a warp's lanes, so results go out without a transpose.
//
// A gated forward product (silu(gate) * up) takes 64 gate and 64 up rows into
// one lane tile, interleaved in blocks of 8 or 16 by the tensor map alone, so
// that both halves of an output element are in the same warp.
//
// One persistent CTA per SM: a TMA warp per operand, an MMA warp, a warp that
// zeroes the rows past a group's count in the weight gradient's last block (a
// count can end inside it, and whatever lies there may be NaN), and eight epilogue
// warps that drain one accumulator while the next fills. Large products run on
// pairs of CTAs (cta_group::2, 256 lanes x 256 columns): each holds half of either
// operand, which halves what a tile reads through shared memory, the limit of a
// single CTA (8192 x 7168 x 4096: 287 against 346 us; a cuBLAS product 279). Products
// with few tiles run on single CTAs, up to four of them sharing a tile's reduction
// and joining their sums through distributed shared memory, in order.
//
// What bounds it: the tensor cores under the power limit for long dense products
// (1680 TFLOP/s of 1729 sustained by cuBLAS), the weights' bytes for few rows per
// expert (128 experts of 4096 x 7168 with 16 rows each: 1.135 ms, 6.62 TB/s of the
// copy's 6.67). In between, both at once reach the power limit (256 rows each: 1.38 to
// 1.43 ms at 1.3 GHz), and two stages of 64 KB instead of three cost 15 %.
#include "product.cuh"

#include <atomic>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "act.cuh"
#include "tensor_map.cuh"

namespace ep {

namespace {

constexpr int kEpilogueWarps = 8;    // two per quarter of the accumulator lanes
constexpr int kThreads = 128 + 32 * kEpilogueWarps;
constexpr int kLanes = 128;          // accumulator lanes of a CTA
constexpr int kColMax = 256;         // accumulator columns, at most
constexpr int kSubRed = 64;          // reduction elements of a sub-block: one 128-byte swizzled line
constexpr int kMaxStages = 12;
constexpr int kChunkBytes = kSubRed * 128;   // MN-major: 64 reduction lines of 64 elements
constexpr int kTmemCols = 512;       // two accumulators of 256 columns
constexpr int kMaxSplit = 4;         // clusters of four fill 144 of 152 SMs, of eight 120
constexpr int kNarrowCols = 32;      // most columns for narrow lane tiles (see plan_dense)
constexpr float kNarrowSubUs = .08f;  // least time of a sub-block
constexpr int kChainF32 = 1024;      // reduction elements summed in one accumulator (see Sums)
constexpr int kChainBf16 = 16384;
constexpr int kBand = 8;             // lane tiles of a band (see find_tile)
constexpr uint32_t kSleepNs = 1000000;   // of one attempt at a wait, at most
constexpr uint64_t kWaitLimitNs = 2000000000ull;   // every other wait is for a pass at most
constexpr uint64_t kBlockNs = 10000;

// What calls without a status word have reported, one word per device, and what of it the
// last ep_product_status took.
__device__ int32_t device_status, status_taken;

__global__ void take_status() { status_taken = atomicExch(&device_status, 0); }

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], tail[kMaxStages];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
    // the groups in the order they are worked on
    int count[EP_MAX_E];             // rows in use
    int first[EP_MAX_E + 1];         // column tiles before it
    uint16_t group[EP_MAX_E];        // which it is
};

constexpr size_t kSmemMax = 227 * 1024;
constexpr size_t kStageSpace = kSmemMax - 1024 - sizeof(Shared);
// a split tile's partial sums take the place of the stages
static_assert((size_t)kLanes * kColMax * 4 + kEpilogueWarps * 4096 <= kStageSpace, "partial sums fit");

// A position in the ring of stages: stage and phase parity.
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) s = 0, phase ^= 1;
    }
};

// A wait of one of the kernel's roles: bounded (by `more` ns beyond the limit), and cut short
// once any role of the CTA has given up.
__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, Shared *sh, const ProductParams &p,
                                          uint64_t more = 0) {
    if (mbar_try_wait_ns(bar, parity, p.sleep_ns)) return true;
    const uint64_t t0 = global_ns();
    volatile int *abort = &sh->abort;
    while (!mbar_try_wait_ns(bar, parity, p.sleep_ns)) {
        if (*abort) return false;
        if (global_ns() - t0 > p.wait_limit_ns + more) {
            *abort = 1;
            atomicCAS(p.status ? p.status : &device_status, 0, EP_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

struct Tile {
    int g, lane0;            // group; this CTA's first output feature
    int col0, cols, n_mma;   // first column, columns in use, columns of the MMA
    int red, blocks;         // reduction length and blocks
};

// Column tiles of a group are of equal width (a multiple of 16 per CTA), so 260
// rows make two tiles of 144 and 116 (of a pair: 160 and 100) and not of 256 and 4.
template <int MODE>
__device__ __forceinline__ int col_tiles(const ProductParams &p, int count) {
    const int cols = MODE == PRODUCT_WGRAD ? p.cols : count;
    return cols > 0 ? (cols - 1) / p.col_max + 1 : 0;
}

// a / b for 0 <= a, 0 < b: by reciprocal and correction where fp32 holds a exactly (an
// integer division takes several times as long, and short tiles wait for it).
__device__ __forceinline__ int quotient(int a, int b) {
    if (a >= 1 << 22) return a / b;
    int q = (int)__fdividef((float)a, (float)b);
    const int r = a - q * b;
    if (r < 0) --q;
    if (r >= b) ++q;
    return q;
}

// Columns of each of ct tiles over `all` > 0.
template <int CG>
__device__ __forceinline__ int tile_width(int all, int ct) {
    constexpr int kUnit = 16 * CG;
    return ((ct == 1 ? all : quotient(all - 1, ct) + 1) + kUnit - 1) / kUnit * kUnit;
}

// Reads the groups' counts and puts the groups in order, the dearest tiles first (the
// widest, or of a weight gradient the longest), so that the last round, which not every
// SM takes part in, is a cheap one: 64 experts' input gradient 466 -> 452 us, 128 experts'
// gated product 1669 -> 1615, 64 experts of a decode batch 99.1 -> 99.6. A group's place
// is the number of groups ahead of it; with more groups than threads the order matters
// little and stays. Called by every thread, ends in a barrier.
template <int MODE, int CG>
__device__ __forceinline__ void order_groups(const ProductParams &p, Shared *sh) {
    const int own = threadIdx.x;
    if (p.groups > kThreads || !p.counts) {
        for (int g = own; g < p.groups; g += kThreads) {
            sh->count[g] = p.counts ? max(0, min(p.counts[g], p.rows)) : p.rows;
            sh->group[g] = (uint16_t)g;
        }
        __syncthreads();
        return;
    }
    int count = 0, key = 0;
    if (own < p.groups) {
        count = max(0, min(p.counts[own], p.rows));
        key = MODE == PRODUCT_WGRAD || count == 0 ? count : tile_width<CG>(count, col_tiles<MODE>(p, count));
        sh->first[own] = key;
    }
    __syncthreads();
    if (own < p.groups) {
        int ahead = 0;
        for (int g = 0; g < p.groups; ++g) {
            const int other = sh->first[g];
            ahead += other > key || (other == key && g < own);
        }
        sh->count[ahead] = count;
        sh->group[ahead] = (uint16_t)own;
    }
    __syncthreads();
}

// A role's place in the launch's tiles, which it visits in rising order: the current
// group, the first tile after it, and what its tiles have in common.
struct Walk {
    int at = -1, begin = 0, end = 0;  // the group's place, its tiles [begin, end)
    int g = 0;
    int ct = 0, all = 0, width = 0;   // column tiles, columns, columns of a tile
    int red = 0, blocks = 0;
};

template <int MODE, int CG>
__device__ __forceinline__ Tile find_tile(const ProductParams &p, const Shared *sh, int t, uint32_t rank, Walk &w) {
    constexpr int kUnit = 16 * CG;
    if (t >= w.end) {
        do {
            ++w.at;
            w.begin = w.end;
            w.end = sh->first[w.at + 1] * p.lane_tiles;
        } while (t >= w.end);
        w.g = sh->group[w.at];
        w.ct = sh->first[w.at + 1] - sh->first[w.at];
        const int count = sh->count[w.at];
        w.all = MODE == PRODUCT_WGRAD ? p.cols : count;
        w.width = tile_width<CG>(w.all, w.ct);
        w.red = MODE == PRODUCT_WGRAD ? count : p.red;
        w.blocks = (int)(((uint32_t)w.red + p.block_red - 1) >> p.block_shift);   // red may be 2^31 - 1
    }
    // bands of kBand lane tiles, lane tiles innermost: the tiles in flight at a time form
    // a square rather than a strip, so each operand block is fetched by several of them
    const int r = t - w.begin;
    const int band = w.ct == 1 ? r / kBand : quotient(r, kBand * w.ct), in_band = r - band * kBand * w.ct;
    const int high = min(kBand, p.lane_tiles - band * kBand);
    const int c = w.ct == 1 ? 0 : high == kBand ? in_band / kBand : quotient(in_band, high);
    const int lt = band * kBand + in_band - c * high;
    Tile x;
    x.g = w.g;
    x.lane0 = (CG == 1 ? lt : lt * 2 + (int)rank) * p.lane_step;
    x.col0 = c * w.width;
    x.cols = min(w.width, w.all - x.col0);
    x.n_mma = (x.cols + kUnit - 1) / kUnit * kUnit;
    x.red = w.red;
    x.blocks = w.blocks;
    return x;
}

// The blocks [lo, hi) of a tile's reduction that this CTA sums.
__device__ __forceinline__ void my_blocks(const ProductParams &p, const Tile &x, uint32_t rank, int &lo, int &hi) {
    lo = 0, hi = x.blocks;
    if (p.split > 1) {
        lo = (int)((long long)x.blocks * rank / p.split);
        hi = (int)((long long)x.blocks * (rank + 1) / p.split);
    }
}

// The tensor cores truncate each step's sum to fp32, and its terms to the place of the sum's
// last bits: a chain of steps is off towards zero, and more than in proportion to its length
// (non-negative terms: 1.7e-6 of the sum after 64 steps, 7.2e-5 after 1024, 3.5e-4 after 4096),
// where rounded sums err by less than 1e-6 at any length. So a chain ends after p.chain blocks: 64
// steps for an fp32 result, 1024 for a bf16 one (a twenty-seventh of the least half unit).
//
// A pass is what goes to one accumulator before the epilogue takes it. An fp32 result whose
// columns leave room has several chains side by side in it, added up with rounding by the
// epilogue. What is longer takes several passes in the same accumulator; the epilogue warps
// keep the running sums, rounded, in the other, and the MMAs wait meanwhile (fp32 8192 x 7168 x 4096:
// 271 -> 307 us; a bf16 weight gradient of 65536 rows, 4096 x 2048: 662 -> 664). Such products
// have kernels of their own (LONG): in one kernel for both the others lost 1 to 2 % (7 x 7168 x 7168
// 22.8 -> 23.0 us, the gradients of 5001 x 4096 x 2048 137.2 -> 139.5).
struct Sums {
    int apart;    // columns between the chains of a pass
    int chain;    // blocks of a chain
    int pass;     // blocks of a pass; the tile's, unless it takes several
};
template <bool LONG>
__device__ __forceinline__ Sums sums_of(const ProductParams &p, const Tile &x, int blocks) {
    const int shift = !p.out_f32 ? 0 : x.n_mma <= 64 ? 2 : x.n_mma <= 128 ? 1 : 0;   // log2 of the chains
    int pass = blocks;
    if (LONG && blocks > p.chain << shift) {
        const int passes = (blocks - 1) / (p.chain << shift) + 1;
        pass = (blocks - 1) / passes + 1;
    }
    return {kColMax >> shift, (pass + (1 << shift) - 1) >> shift, pass};
}

// Two output features (f, f + 1) of token column j or j + 1: lanes trade with
// their neighbour so that each holds a pair of one token, ready for a packed
// store. Even lanes end with column j, odd lanes with column j + 1.
__device__ __forceinline__ float2 trade_pair(float vj, float vj1, bool odd) {
    const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? vj : vj1, 1);
    return odd ? make_float2(got, vj1) : make_float2(vj, got);
}

__device__ __forceinline__ uint32_t ld_pair(const __nv_bfloat16 *ptr) {
    return *reinterpret_cast<const uint32_t *>(ptr);
}
__device__ __forceinline__ void st_pair(__nv_bfloat16 *ptr, uint32_t v) {
    *reinterpret_cast<uint32_t *>(ptr) = v;
}

// What the epilogue of one chunk reads from memory (residual, pre-activations or
// the output added to), fetched before the accumulators are waited for.
struct Side {
    uint32_t a[16], b[16];
};

// Where a lane's pairs of a chunk of 32 columns lie: its first feature, and the
// column of its i-th pair (see trade_pair; a gated forward chunk ends in 8 pairs).
template <int MODE, bool GATED>
struct Place {
    int f;
    bool ok, odd, up;
    __device__ __forceinline__ Place(const ProductParams &p, const Tile &x, int quad, int lane) {
        odd = lane & 1;
        if (MODE == PRODUCT_FORWARD && GATED) {
            const int il = p.interleave;   // 8 or 16
            up = lane & il;
            f = quad * 16 + (il == 8 ? (lane >> 4) * 8 : 0) + (lane & (il - 1) & ~1);
        } else {
            up = false;
            f = quad * 32 + (lane & ~1);
        }
        ok = f < p.lane_step;   // lanes past a narrow tile hold nothing
        f += x.lane0;
        ok = ok && f < p.lanes;
    }
    __device__ __forceinline__ int column(int i) const {
        return MODE == PRODUCT_FORWARD && GATED ? 4 * i + (up ? 2 : 0) + odd : 2 * i + odd;
    }
};

// Read once: streaming loads, which leave the operands in L2 (gradient through relu,
// 5001 x 2048 x 4096: 62.1 -> 59.4 us, with no prefetch into L2 beside them).
__device__ __forceinline__ uint32_t ld_once(const __nv_bfloat16 *ptr) {
    return __ldcs(reinterpret_cast<const uint32_t *>(ptr));
}

template <int MODE, bool GATED>
__device__ __forceinline__ void load_side(const ProductParams &p, size_t row0, int n, const Place<MODE, GATED> &at,
                                          Side &side) {
    constexpr int kPairs = MODE == PRODUCT_FORWARD && GATED ? 8 : 16;
    if (!at.ok) return;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int j = at.column(i);
        if (j >= n) continue;
        if (MODE == PRODUCT_FORWARD) {
            side.a[i] = ld_once(p.residual + (row0 + j) * p.lanes + at.f);
        } else if (MODE == PRODUCT_DGRAD) {
            const __nv_bfloat16 *z = p.z + (row0 + j) * (GATED ? 2 : 1) * p.lanes + at.f;
            side.a[i] = ld_once(z);
            if (GATED) side.b[i] = ld_once(z + p.lanes);
        } else if (p.out_f32) {
            const float2 v = __ldcs(reinterpret_cast<const float2 *>(static_cast<const float *>(p.out) +
                                                                    (row0 + j) * p.lanes + at.f));
            side.a[i] = __float_as_uint(v.x), side.b[i] = __float_as_uint(v.y);
        } else {
            side.a[i] = ld_once(static_cast<const __nv_bfloat16 *>(p.out) + (row0 + j) * p.lanes + at.f);
        }
    }
}

template <int ACT, int N>
__device__ __forceinline__ void act_pairs(float2 (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(act_value(v[i].x, ACT), act_value(v[i].y, ACT));
}
template <int ACT, int N>
__device__ __forceinline__ void slope_pairs(float2 (&v)[N], const uint32_t (&z)[16]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 s = unpack_bf16x2(z[i]);
        v[i].x *= act_slope(s.x, ACT), v[i].y *= act_slope(s.y, ACT);
    }
}

// Pairs i of v to output rows row0 + column(i), `wide` elements apart, at `off`.
template <int MODE, bool GATED, int N>
__device__ __forceinline__ void store_pairs(const ProductParams &p, const float2 (&v)[N], size_t row0, int n,
                                            const Place<MODE, GATED> &at, size_t wide, size_t off) {
    if (!at.ok) return;
    if (p.out_f32) {
        float *o = static_cast<float *>(p.out) + row0 * wide + off;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (at.column(i) < n) *reinterpret_cast<float2 *>(o + at.column(i) * wide) = v[i];
    } else {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + row0 * wide + off;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (at.column(i) < n) st_pair(o + at.column(i) * wide, pack_bf16x2_rn(v[i].x, v[i].y));
    }
}

// Where a warp's 32 x 32 output tile is staged, and its place in the output.
struct OutTile {
    uint8_t *smem;
    int lane, row, group;
};

// Full tiles leave through shared memory and a TMA store: as stores of each lane they
// kept the epilogue warps waiting on the memory pipe, and with the short reductions of
// a weight gradient the epilogue sets the pace (885 -> 725 us on 32 experts of 4096 x
// 7168 with 256 rows each, in fp32). Lanes past the last feature are cut by the map.
template <int MODE, bool GATED>
__device__ __forceinline__ void tile_pairs(const ProductParams &p, const float2 (&v)[16], const Place<MODE, GATED> &at,
                                           const OutTile &tile, int half) {
    if (elect_one()) bulk_wait_read<0>();   // the tile's last contents are on their way
    __syncwarp();
    const int pair = (threadIdx.x % 32) / 2;
    if (p.out_f32) {
        float2 *o = reinterpret_cast<float2 *>(tile.smem) + pair;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[(2 * i + at.odd) * 16] = v[i];
    } else {
        uint32_t *o = reinterpret_cast<uint32_t *>(tile.smem) + pair;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[(2 * i + at.odd) * 16] = pack_bf16x2_rn(v[i].x, v[i].y);
    }
    fence_async();
    __syncwarp();
    if (elect_one() && tile.lane < p.lanes) {
        tma_store_4d(&p.o, tile.smem, tile.lane, half, tile.row, tile.group);
        bulk_commit();
    }
}

// The accumulators as they are, in fp32.
__device__ __forceinline__ void tile_lanes(const ProductParams &p, const float (&acc)[32], const OutTile &tile) {
    if (elect_one()) bulk_wait_read<0>();
    __syncwarp();
    float *o = reinterpret_cast<float *>(tile.smem) + threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < 32; ++j) o[j * 32] = acc[j];
    fence_async();
    __syncwarp();
    if (elect_one() && tile.lane < p.lanes) {
        tma_store_4d(&p.o, tile.smem, tile.lane, 0, tile.row, tile.group);
        bulk_commit();
    }
}

// The epilogue of 32 accumulator columns of one warp's 32 lanes, of which n are
// output rows row0 .. row0 + n - 1. Straight-line over the 16 pairs, so that
// their arithmetic and stores overlap.
template <int MODE, bool GATED, bool SIDE>
__device__ __forceinline__ void epilogue_chunk(const ProductParams &p, const float (&acc)[32], size_t row0, int n,
                                               const Place<MODE, GATED> &at, float2 bias, const Side &side,
                                               const OutTile &tile) {
    const size_t L = (size_t)p.lanes;
    if constexpr (MODE == PRODUCT_WGRAD) {
        if (!SIDE && n == 32 && p.out_f32) {   // nothing to pair up: lanes side by side already
            tile_lanes(p, acc, tile);
            return;
        }
    }
    float2 v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = trade_pair(acc[2 * i], acc[2 * i + 1], at.odd);
    if constexpr (MODE == PRODUCT_FORWARD) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i].x += bias.x, v[i].y += bias.y;
        if (p.preact && at.ok) {
            const size_t wide = GATED ? 2 * L : L;
            __nv_bfloat16 *z = p.preact + row0 * wide + (GATED && at.up ? L : 0) + at.f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (2 * i + at.odd < n) st_pair(z + (2 * i + at.odd) * wide, pack_bf16x2_rn(v[i].x, v[i].y));
        }
    }
    if constexpr (MODE == PRODUCT_FORWARD && GATED) {
        float2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // of two pairs, gate lanes give their second for the up pair of the first
            const float2 a = v[2 * i], b = v[2 * i + 1], give = at.up ? a : b;
            float2 got;
            got.x = __shfl_xor_sync(0xFFFFFFFFu, give.x, p.interleave);
            got.y = __shfl_xor_sync(0xFFFFFFFFu, give.y, p.interleave);
            const float2 gate = at.up ? got : a, up = at.up ? b : got;
            y[i] = make_float2(act_value(gate.x, EP_ACT_SILU) * up.x, act_value(gate.y, EP_ACT_SILU) * up.y);
        }
        if (SIDE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 r = unpack_bf16x2(side.a[i]);
                y[i].x += r.x, y[i].y += r.y;
            }
        }
        store_pairs(p, y, row0, n, at, L, at.f);
    } else if constexpr (MODE == PRODUCT_DGRAD && GATED) {
        float2 d[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 g = unpack_bf16x2(side.a[i]), u = unpack_bf16x2(side.b[i]);
            swiglu_grad(v[i].x, g.x, u.x, d[i].x, v[i].x);
            swiglu_grad(v[i].y, g.y, u.y, d[i].y, v[i].y);
        }
        if (n == 32) {
            tile_pairs(p, d, at, tile, 0);
            tile_pairs(p, v, at, tile, 1);
        } else {
            store_pairs(p, d, row0, n, at, 2 * L, at.f);
            store_pairs(p, v, row0, n, at, 2 * L, L + at.f);
        }
    } else {
        if (MODE == PRODUCT_FORWARD) {
            switch (p.act) {
                case EP_ACT_RELU: act_pairs<EP_ACT_RELU>(v); break;
                case EP_ACT_SILU: act_pairs<EP_ACT_SILU>(v); break;
                case EP_ACT_GELU: act_pairs<EP_ACT_GELU>(v); break;
                case EP_ACT_GELU_TANH: act_pairs<EP_ACT_GELU_TANH>(v); break;
                default: break;
            }
        } else if (MODE == PRODUCT_DGRAD && SIDE) {
            switch (p.act) {
                case EP_ACT_RELU: slope_pairs<EP_ACT_RELU>(v, side.a); break;
                case EP_ACT_SILU: slope_pairs<EP_ACT_SILU>(v, side.a); break;
                case EP_ACT_GELU: slope_pairs<EP_ACT_GELU>(v, side.a); break;
                case EP_ACT_GELU_TANH: slope_pairs<EP_ACT_GELU_TANH>(v, side.a); break;
                default: break;
            }
        }
        if (MODE != PRODUCT_DGRAD && SIDE) {
            const bool wide = MODE == PRODUCT_WGRAD && p.out_f32;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 r = wide ? make_float2(__uint_as_float(side.a[i]), __uint_as_float(side.b[i]))
                                      : unpack_bf16x2(side.a[i]);
                v[i].x += r.x, v[i].y += r.y;
            }
        }
        if (n == 32 && (MODE != PRODUCT_FORWARD || p.lane_step == kLanes))
            tile_pairs(p, v, at, tile, 0);
        else
            store_pairs(p, v, row0, n, at, L, at.f);
    }
}

template <int MODE, bool GATED, int CG, bool SIDE, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ ProductParams p) {
    constexpr bool kMnA = MODE != PRODUCT_FORWARD, kMnB = MODE == PRODUCT_WGRAD;
    extern __shared__ uint8_t raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Shared *sh = reinterpret_cast<Shared *>(stages + kStageSpace / 1024 * 1024);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool clustered = CG == 2 || p.split > 1;
    const uint32_t rank = clustered ? cluster_rank() : 0;
    const int per_cluster = CG == 2 ? 2 : p.split;
    const int t0 = blockIdx.x / per_cluster, t_step = gridDim.x / per_cluster;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&sh->full[s], 2 * CG);   // an arrival per operand and CTA
            mbar_init(&sh->empty[s], 1);
            mbar_init(&sh->tail[s], 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], kEpilogueWarps * CG);
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.a);
        tma_prefetch_map(&p.b[0]);
    }
    if (warp == 3) tmem_alloc<CG>(&sh->tmem, kTmemCols);
    pdl_wait();   // nothing above reads or writes global memory
    pdl_launch_dependents();
    order_groups<MODE, CG>(p, sh);
    if (warp == 0) {   // exclusive prefix of the groups' column tiles
        int base = 0;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const int g = g0 + lane;
            const int own = g < p.groups ? col_tiles<MODE>(p, sh->count[g]) : 0;
            int sum = own;
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += v;
            }
            if (g < p.groups) sh->first[g] = base + sum - own;
            base += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) sh->first[p.groups] = base;
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();   // both CTAs' barriers are ready before either signals the other's
    tc_fence_after();
    const int total = sh->first[p.groups] * p.lane_tiles;
    const uint32_t tmem = sh->tmem;

    Ring ring;
    Walk walk;
    int acc = 0;                            // the accumulator in turn,
    uint32_t acc_phase = 0;                 // and a bit for each: the phase of its next use
    int issued = 0;                         // producer: blocks so far
    uint32_t on_tail = 0, tail_phase = 0;   // producer, a bit per stage: last load signals tail[], and its phase
    if (warp == 0 || warp == 3) {
        // ---- TMA: this CTA's part of one operand (warp 0: lanes, warp 3: columns) of every
        // block into the next free stage. One warp for both took as long to issue a block's
        // loads as the tensor cores to use them.
        const bool lanes = warp == 0;
        bool ok = true;
        for (int t = t0; t < total && ok; t += t_step) {
            const Tile x = find_tile<MODE, CG>(p, sh, t, rank, walk);
            const int own_cols = x.n_mma / CG;
            // (of the last tile it may lie past the columns, where loads read zeros)
            const int col0 = (int)((uint32_t)x.col0 + (CG == 2 ? rank * own_cols : 0u));
            const int chunks = (own_cols + 63) / 64;
            const uint32_t sub_bytes = lanes ? p.a_bytes : kMnB ? chunks * kChunkBytes : own_cols * 128;
            const int lane_block = x.lane0 / (GATED && MODE == PRODUCT_FORWARD ? p.interleave : 1);
            int lo, hi;
            my_blocks(p, x, rank, lo, hi);
            for (int kb = lo; kb < hi; ++kb, ++issued, ring.next(p.stages)) {
                const int s = ring.s;
                ok = role_wait(&sh->empty[s], ring.phase ^ 1, sh, p);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const int r0 = kb * p.block_red, left = x.red - r0;
                const int subs = left >= p.block_red ? p.subs : (left + kSubRed - 1) / kSubRed;
                // a weight gradient's block that ends past the count goes through the
                // zeroing warp before the MMA warp sees it
                const bool tail = kMnB && left < p.block_red && left % kSubRed != 0;
                if (kMnB) {
                    if (tail) tail_phase ^= 1u << s;   // phase of the stage's next tail
                    on_tail = (on_tail & ~(1u << s)) | (tail ? 1u << s : 0u);
                }
                if (elect_one()) {
                    uint64_t *local = tail ? &sh->tail[s] : &sh->full[s];
                    uint32_t bar;
                    if (CG == 2 && !tail) {
                        bar = map_rank(local, 0);
                        mbar_arrive_expect_tx_cluster(bar, sub_bytes * subs);
                    } else {
                        bar = smem_u32(local);
                        mbar_arrive_expect_tx(local, sub_bytes * subs);
                    }
                    uint8_t *dst = stages + (size_t)s * p.stage_bytes + (lanes ? 0 : p.a_bytes);
                    for (int sub = 0; sub < subs; ++sub, dst += p.sub_bytes) {
                        const int r = r0 + sub * kSubRed;
                        if (lanes) {
                            if (MODE == PRODUCT_FORWARD) {
                                if (GATED)
                                    tma_load_5d<CG>(dst, &p.a, r, 0, 0, lane_block, x.g, bar);
                                else
                                    tma_load_3d<CG>(dst, &p.a, r, lane_block, x.g, bar);
                            } else {
                                tma_load_3d<CG>(dst, &p.a, x.lane0, r, x.g, bar);
                                tma_load_3d<CG>(dst + kChunkBytes, &p.a, x.lane0 + 64, r, x.g, bar);
                            }
                        } else if (kMnB) {
                            for (int c = 0; c < chunks; ++c)
                                tma_load_3d<CG>(dst + c * kChunkBytes, &p.b[0], col0 + 64 * c, r, x.g, bar);
                        } else {
                            // a box for every width: a second TMA for what is left costs more
                            // than its bytes (tiles of 160 columns 8 % slower)
                            const int more = CG == 1 && own_cols > 128 ? own_cols - 128 : 0;
                            tma_load_3d<CG>(dst, &p.b[(own_cols - more) / 16 - 1], r, col0, x.g, bar);
                            if (CG == 1 && more)
                                tma_load_3d<CG>(dst + 128 * 128, &p.b[more / 16 - 1], r, col0 + 128, x.g, bar);
                        }
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp == 1 && (CG == 1 || rank == 0)) {
        // ---- MMA: one thread issues the steps of 16 of each block
        bool ok = true;
        for (int t = t0; t < total && ok; t += t_step) {
            const Tile x = find_tile<MODE, CG>(p, sh, t, rank, walk);
            int lo, hi;
            my_blocks(p, x, rank, lo, hi);
            if (lo == hi) continue;
            const uint32_t idesc = mma_idesc(kLanes * CG, x.n_mma, kMnA, kMnB);
            const Sums sums = sums_of<LONG>(p, x, hi - lo);
            for (int kb = lo; kb < hi && ok;) {
                const int end = LONG ? min(kb + sums.pass, hi) : hi;
                ok = role_wait(&sh->acc_empty[acc], ((acc_phase >> acc) & 1) ^ 1, sh, p);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                uint32_t d = tmem + acc * kColMax;
                for (int in_chain = 0; kb < end; ++kb, ++in_chain, ring.next(p.stages)) {
                    if (in_chain == sums.chain) in_chain = 0, d += sums.apart;
                    const int s = ring.s;
                    ok = role_wait(&sh->full[s], ring.phase, sh, p);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        uint32_t sa = smem_u32(stages + (size_t)s * p.stage_bytes);
                        int left = x.red - kb * p.block_red;
                        for (int sub = 0; sub < p.subs && left > 0; ++sub, sa += p.sub_bytes, left -= kSubRed) {
                            const uint64_t da = kMnA ? smem_desc(sa, kChunkBytes, 1024) : smem_desc(sa, 16, 1024);
                            // (of a narrow tile the MMA reads on past its rows, within shared memory,
                            // for lanes nobody looks at)
                            const uint64_t db = kMnB ? smem_desc(sa + p.a_bytes, kChunkBytes, 1024)
                                                     : smem_desc(sa + p.a_bytes, 16, 1024);
                            constexpr uint32_t kStepA = (kMnA ? 2048 : 32) / 16, kStepB = (kMnB ? 2048 : 32) / 16;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (left > 16 * i)
                                    mma_bf16<CG>(d, da + kStepA * i, db + kStepB * i, idesc,
                                                 in_chain > 0 || sub > 0 || i > 0);
                        }
                        mma_commit<CG>(&sh->empty[s]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) mma_commit<CG>(&sh->acc_full[acc]);
                __syncwarp();
                acc_phase ^= 1u << acc;
            }
            if (!LONG || sums.pass == hi - lo) acc ^= 1;   // after several passes the next tile goes on in the same
        }
    } else if (warp == 2 && kMnB) {
        // ---- rows at or past the count, in the last block: zero in both operands
        uint32_t used = 0;   // a bit per stage: parity of its next use here
        bool ok = true;
        for (int t = t0; t < total && ok; t += t_step) {
            const Tile x = find_tile<MODE, CG>(p, sh, t, rank, walk);
            int lo, hi;
            my_blocks(p, x, rank, lo, hi);
            const int left = x.red % kSubRed;
            for (int kb = lo; kb < hi; ++kb, ring.next(p.stages)) {
                if (left == 0 || kb + 1 < x.blocks) continue;
                const int s = ring.s;
                // (for the whole reduction, so its length counts; a block takes 0.2 to 0.4 us)
                ok = role_wait(&sh->tail[s], (used >> s) & 1, sh, p, (uint64_t)(hi - lo) * kBlockNs);
                ok = __all_sync(0xFFFFFFFFu, ok);
                used ^= 1u << s;
                if (!ok) break;
                // rows up to the MMA's last step of 16
                const int rows = ((left + 15) & ~15) - left;
                const int chunks = 2 + (x.n_mma / CG + 63) / 64;
                const int sub = (x.red - kb * p.block_red) / kSubRed;
                uint8_t *sa = stages + (size_t)s * p.stage_bytes + sub * p.sub_bytes;
                for (int i = lane; i < rows * chunks * 8; i += 32) {
                    const int c = i / (rows * 8), r = i % (rows * 8) / 8, v = i % 8;
                    *reinterpret_cast<uint4 *>(sa + c * kChunkBytes + (left + r) * 128 + v * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_async();
                __syncwarp();
                if (lane < 2) {   // for both operands' loads
                    if (CG == 2)
                        mbar_arrive_cluster(map_rank(&sh->full[s], 0));
                    else
                        mbar_arrive(&sh->full[s]);
                }
            }
        }
    } else if (warp >= 4) {
        // ---- epilogue: 32 lanes and every other 32 columns of each accumulator
        const int quad = warp % 4, half = (warp - 4) / 4;
        OutTile tile;
        tile.smem = stages + p.out_at + (warp - 4) * (p.out_f32 ? 4096 : 2048);
        // accumulator a may be overwritten: this warp's part is in registers (nothing in
        // memory is handed over)
        auto free_acc = [&](int a) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2)
                    mbar_arrive_cluster_relaxed(map_rank(&sh->acc_empty[a], 0));
                else
                    mbar_arrive(&sh->acc_empty[a]);
            }
        };
        auto wait_acc = [&](int a) {
            const bool full = role_wait(&sh->acc_full[a], (acc_phase >> a) & 1, sh, p);
            acc_phase ^= 1u << a;
            const bool all = __all_sync(0xFFFFFFFFu, full);
            tc_fence_after();
            return all;
        };
        bool ok = true;
        for (int t = t0; t < total && ok; t += t_step) {
            const Tile x = find_tile<MODE, CG>(p, sh, t, rank, walk);
            int lo, hi;
            my_blocks(p, x, rank, lo, hi);
            if (p.split == 1 && lo == hi && MODE == PRODUCT_WGRAD && p.accumulate) continue;
            const Place<MODE, GATED> at(p, x, quad, lane);
            const size_t row0 = (size_t)x.g * (MODE == PRODUCT_WGRAD ? p.cols : p.rows) + x.col0;
            float2 bias = make_float2(0.f, 0.f);
            if (MODE == PRODUCT_FORWARD && p.bias && at.ok)
                bias = unpack_bf16x2(ld_pair(p.bias + (size_t)x.g * (GATED ? 2 : 1) * p.lanes +
                                             (at.up ? p.lanes : 0) + at.f));
            tile.lane = x.lane0 + quad * 32, tile.group = x.g;
            const Sums sums = sums_of<LONG>(p, x, hi - lo);
            const uint32_t quad_lanes = (uint32_t)(quad * 32) << 16;
            uint32_t at_acc = tmem + acc * kColMax + quad_lanes;   // where the sums are read,
            int chain = sums.chain;                                // and the blocks of each part
            if (LONG && sums.pass < hi - lo) {
                const uint32_t kept = tmem + (acc ^ 1) * kColMax + quad_lanes;
                for (int kb = lo; kb < hi; kb += sums.pass) {
                    ok = wait_acc(acc);
                    if (!ok) break;
                    const int n = min(sums.pass, hi - kb);
                    for (int c = half * 32; c < x.cols; c += 64) {
                        uint32_t r[32], more[32];
                        tmem_ld32(at_acc + c, r);
                        for (int i = 0, done = sums.chain; done < n; done += sums.chain) {
                            tmem_ld32(at_acc + c + ++i * sums.apart, more);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(more[j]));
                        }
                        if (kb > lo) {
                            tmem_ld32(kept + c, more);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(more[j]));
                        }
                        tmem_ld_wait();
                        tmem_st32(kept + c, r);
                    }
                    tmem_st_wait();
                    if (kb + sums.pass < hi) free_acc(acc);   // the last goes with the sums kept
                }
                if (!ok) break;
                at_acc = kept, chain = hi - lo;
            }
            Side side;
            if (SIDE && p.split == 1 && half * 32 < x.cols)
                load_side(p, row0 + half * 32, min(32, x.cols - half * 32), at, side);
            if (lo < hi && (!LONG || sums.pass == hi - lo)) {
                ok = wait_acc(acc);
                if (!ok) break;
            }
            for (int c = half * 32; c < x.cols; c += 64) {
                float v[32];
                if (lo < hi) {
                    uint32_t r[32], from = at_acc + c;
                    tmem_ld32(from, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                    for (int done = chain; done < hi - lo; done += chain) {
                        from += sums.apart;
                        tmem_ld32(from, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(r[j]);
                    }
                    if (c + 64 >= x.cols) free_acc(acc);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                }
                if (p.split > 1) {   // to shared memory, [column][lane]; joined below
                    float *part = reinterpret_cast<float *>(stages) + quad * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < x.cols) part[(c + j) * kLanes] = v[j];
                } else {
                    tile.row = x.col0 + c;
                    const Side now = side;
                    if (SIDE && c + 64 < x.cols) load_side(p, row0 + c + 64, min(32, x.cols - c - 64), at, side);
                    epilogue_chunk<MODE, GATED, SIDE>(p, v, row0 + c, min(32, x.cols - c), at, bias, now, tile);
                }
            }
            if (lo < hi) {
                if (half * 32 >= x.cols) free_acc(acc);   // a warp with no columns here
                if (!LONG || sums.pass == hi - lo) acc ^= 1;
            }
        }
        if (elect_one()) bulk_wait_all();
    }
    __syncthreads();
    if (sh->abort && threadIdx.x < 64) {
        // a wait ran out: let the copies and MMAs in flight finish (bounded) before
        // shared and tensor memory are given up
        const uint64_t t0 = global_ns();
        if (threadIdx.x == 0 && (CG == 1 || rank == 0)) {
            for (int i = max(0, issued - p.stages); i < issued; ++i) {
                const int s = i % p.stages;
                const bool tail = (on_tail >> s) & 1;
                const uint32_t phase = tail ? ((tail_phase >> s) & 1) ^ 1 : (uint32_t)(i / p.stages) & 1;
                while (!mbar_try_wait(tail ? &sh->tail[s] : &sh->full[s], phase) &&
                       global_ns() - t0 < 100000000ull)
                    ;
            }
        } else if (threadIdx.x == 32 && (CG == 1 || rank == 0)) {
            mma_commit<CG>(&sh->drain);
            while (!mbar_try_wait(&sh->drain, 0) && global_ns() - t0 < 100000000ull)
                ;
        }
        while (global_ns() - t0 < 1000000ull)   // the other CTA's copies, which it cannot see end
            ;
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 1 && p.split > 1) {
        // ---- the split tile: every CTA has its partial sums in shared memory; each adds up
        // its share of the columns, in rank order, and finishes them
        cluster_sync();
        if (t0 < total && warp >= 4) {
            const int quad = warp % 4, half = (warp - 4) / 4;
            walk = Walk();
            const Tile x = find_tile<MODE, CG>(p, sh, t0, rank, walk);
            const Place<MODE, GATED> at(p, x, quad, lane);
            const size_t row0 = (size_t)x.g * (MODE == PRODUCT_WGRAD ? p.cols : p.rows) + x.col0;
            float2 bias = make_float2(0.f, 0.f);
            if (MODE == PRODUCT_FORWARD && p.bias && at.ok)
                bias = unpack_bf16x2(ld_pair(p.bias + (size_t)x.g * (GATED ? 2 : 1) * p.lanes +
                                             (at.up ? p.lanes : 0) + at.f));
            OutTile tile;
            tile.smem = stages + p.out_at + (warp - 4) * (p.out_f32 ? 4096 : 2048);
            tile.lane = x.lane0 + quad * 32, tile.group = x.g;
            const int share = (x.cols + p.split - 1) / p.split;
            const int c1 = min(x.cols, ((int)rank + 1) * share);
            for (int c = (int)rank * share + half * 32; c < c1; c += 64) {
                const int n = min(32, c1 - c);
                Side side;
                if (SIDE) load_side(p, row0 + c, n, at, side);
                float acc[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[j] = 0.f;
                for (int i = 0; i < p.split; ++i) {
                    const uint32_t part =
                        map_rank(reinterpret_cast<float *>(stages) + c * kLanes + quad * 32 + lane, i);
                    float got[32];   // all loads on their way before the first is used
#pragma unroll
                    for (int j = 0; j < 32; ++j) got[j] = j < n ? ld_cluster_f32(part + j * kLanes * 4) : 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[j] += got[j];
                }
                tile.row = x.col0 + c;
                epilogue_chunk<MODE, GATED, SIDE>(p, acc, row0 + c, n, at, bias, side, tile);
            }
            if (elect_one()) bulk_wait_all();
        }
        cluster_sync();   // no CTA leaves while another reads its shared memory
    }
    if (CG == 2) cluster_sync();
    tc_fence_after();
    if (warp == 3) tmem_free<CG>(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side

// The output [groups][rows][halves][lanes], written in boxes of 32 lanes and 32 rows.
bool make_out_map(CUtensorMap *m, void *out, bool f32, uint64_t halves, uint64_t lanes, uint64_t rows,
                  uint64_t groups) {
    EncodeTiled enc = encoder();
    if (!enc) return false;
    const uint64_t size = f32 ? 4 : 2;
    const cuuint64_t dims[4] = {lanes, halves, rows, groups};
    const cuuint64_t strides[3] = {lanes * size, lanes * halves * size, lanes * halves * rows * size};
    const cuuint32_t box[4] = {32, 1, 32, 1}, one[4] = {1, 1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, out, dims, strides, box,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// How a product is cut: CTAs per MMA, widest column tile, CTAs that share a tile's reduction.
struct Plan {
    int cg, col_max, split;
    int lane_step;   // 0 = full lane tiles
};

// Ragged groups, whose row counts the host does not know: pairs of CTAs where one tile
// per group and lane tile, or full groups, fill the GPU; single CTAs otherwise.
Plan plan_ragged(long long lane_tiles, long long groups, long long cols, int sms) {
    const long long pairs = ceil_div(lane_tiles, 2) * groups * ceil_div(cols, kColMax);
    return {lane_tiles > 1 && 2 * pairs >= sms ? 2 : 1, kColMax, 1, 0};
}

// Dense products: the cut with the least estimated time. A round (one tile on every SM)
// costs, per 64 reduction elements, the share kCost of what a pair's tile of 256 lanes x
// 256 columns takes (0.363 us), measured by column width on 8192 x 7168 x 4096, a tile
// of 128 lanes on a single CTA included. Narrow tiles are dear (both operands pass through
// shared memory for fewer MMAs), so they pay only where wide ones leave SMs idle; sharing
// a reduction adds a join of about 2 us, and the last epilogue shows, 2.3 us for 256 columns.
// Measured against pairs of full tiles where those fill the GPU and single CTAs otherwise:
// 512 x 7168 x 4096 33.8 -> 28.5 us, 1024 x 4096 x 4096 29.7 -> 27.2, 3000 x 4096 x 1024
// 27.6 -> 22.6, 1024 x 7168 x 7168 78 -> 79.
//
// Few columns on many features (a decoding step's forward product) leave the weight's bytes
// as the floor. There lane tiles may be narrower than the accumulator, so that one round
// covers the SMs evenly without a join: `narrow` is 1, or 2 for a gated product's two rows
// per feature, or 0. 7 x 7168 x 7168: 24.8 -> 22.5 us, 16 x 2048 x 7168 10.7 -> 10.5,
// 16 x 4096 x 4096 13.3 -> 13.7; at 64 rows it no longer pays (23.5 -> 23.9).
Plan plan_dense(long long lane_tiles, long long groups, long long cols, long long red, long long lanes, int narrow,
                int sms) {
    static const float kCost[2][8] = {{.51f, .54f, .65f, .73f, .88f, .91f, 1.05f, 1.19f},
                                      {.46f, .47f, .51f, .58f, .75f, .78f, .91f, 1.f}};
    const float blocks = (float)ceil_div(red, kSubRed);
    const float dram_us = (float)(groups * lanes * (narrow > 1 ? 2 : 1) * red) * 2.f / 6.4e6f;
    Plan best = {1, kColMax, 1, 0};
    float best_us = 0.f;
    for (int cg = 1; cg <= 2; ++cg) {
        if (cg == 2 && lane_tiles < 2) break;
        const int slots = sms / cg;
        for (int w = 1; w <= kColMax / 32; ++w) {
            const long long tiles = ceil_div(lane_tiles, cg) * groups * ceil_div(cols, 32 * w);
            for (int split = 1; split <= (cg == 1 ? kMaxSplit : 1); split *= 2) {
                // (clusters of four fit on all but a few SMs: 144 of 152)
                if (split > 1 && (split * tiles > (split == 4 ? sms - sms / 16 : sms) || blocks < 8 * split)) break;
                const float rounds = split > 1 ? 1.f : (float)ceil_div(tiles, slots);
                const float sums = rounds * kCost[cg - 1][w - 1] * .363f * blocks / split;
                const float us = (sums > dram_us ? sums : dram_us) + (split > 1 ? 2.f : 0.f) + 2.3f / 8 * w / split;
                if (best_us == 0.f || us < best_us) best_us = us, best = {cg, 32 * w, split, 0};
            }
            if (32 * w >= cols) break;
        }
    }
    if (narrow && cols <= kNarrowCols) {
        const long long step = ceil_div(ceil_div(groups * lanes, sms), 16) * 16;   // one round
        const long long rows = step * narrow;
        if (rows < kLanes) {
            const float sub = (float)(rows + ceil_div(cols, 16) * 16) * 128.f / 95e3f;   // at 95 GB/s a CTA
            const float rounds = (float)ceil_div(groups * ceil_div(lanes, step), sms);
            const float sums = (sub > kNarrowSubUs ? sub : kNarrowSubUs) * blocks * rounds;
            const float us = (sums > dram_us ? sums : dram_us) + 2.3f / 8 * ceil_div(cols, 32);
            if (us < best_us) best = {1, (int)(ceil_div(cols, 32) * 32), 1, (int)step};
        }
    }
    return best;
}

template <int MODE, bool GATED, int CG, bool SIDE>
int launch(const ProductParams &p, bool is_long, int clusters, cudaStream_t st) {
    const auto kernel = is_long ? &product_kernel<MODE, GATED, CG, SIDE, true> : &product_kernel<MODE, GATED, CG, SIDE, false>;
    if (ensure_dyn_smem(reinterpret_cast<const void *>(kernel), kSmemMax) != cudaSuccess) return EP_ERR_CUDA;
    const int size = CG == 2 ? 2 : p.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    // the set-up (barriers, tensor memory) overlaps the end of the kernel before
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

std::atomic<uint64_t> wait_limit_ns{kWaitLimitNs};

// Plans and launches: `a` is the lane operand (a weight, or wgrad's x), `b` the column
// operand, [groups][rows][width].
template <int MODE>
int launch(ProductParams &p, const void *a, const void *b, int width, cudaStream_t st) {
    const bool gated = p.act == EP_ACT_SWIGLU, two = gated && MODE == PRODUCT_FORWARD;
    const int full_step = two ? kLanes / 2 : kLanes;
    const long long cols = MODE == PRODUCT_WGRAD ? p.cols : p.rows;
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return EP_ERR_CUDA;
    p.wait_limit_ns = wait_limit_ns.load(std::memory_order_relaxed);
    p.sleep_ns = p.wait_limit_ns < kSleepNs ? (uint32_t)p.wait_limit_ns : kSleepNs;
    const long long full_tiles = ceil_div(p.lanes, full_step);
    const Plan plan = p.counts ? plan_ragged(full_tiles, p.groups, cols, sms)
                               : plan_dense(full_tiles, p.groups, cols, MODE == PRODUCT_WGRAD ? p.rows : p.red, p.lanes,
                                            MODE != PRODUCT_FORWARD ? 0 : two ? 2 : 1, sms);
    const int cg = plan.cg;
    p.col_max = plan.col_max;
    p.split = plan.split;
    p.lane_step = plan.lane_step ? plan.lane_step : full_step;
    p.lane_tiles = (int)ceil_div(ceil_div(p.lanes, p.lane_step), cg);
    const int lane_rows = p.lane_step * (two ? 2 : 1);
    p.a_bytes = lane_rows * kSubRed * 2;
    const int unit = 16 * cg;
    const int widest = (int)(cols < p.col_max ? ceil_div(cols, unit) * unit : p.col_max);
    p.sub_bytes = p.a_bytes + (MODE == PRODUCT_WGRAD ? (widest / cg + 63) / 64 * kChunkBytes
                                                     : (widest / cg * 128 + 1023) / 1024 * 1024);
    const int out_bytes = kEpilogueWarps * (p.out_f32 ? 4096 : 2048);
    const int space = (int)(kStageSpace / 1024 * 1024) - out_bytes;
    // two sub-blocks per stage (of narrow tiles, four) halve the barrier traffic; one where
    // that leaves fewer than three stages (8192 x 7168 x 4096: 288 against 305 us; 7 rows:
    // 26.7 against 28.7)
    p.subs = plan.lane_step ? 4 : 2;
    while (p.subs > 1 && space / (p.subs * p.sub_bytes) < 3) p.subs /= 2;
    p.block_red = p.subs * kSubRed;
    p.block_shift = p.subs == 4 ? 8 : p.subs == 2 ? 7 : 6;
    p.chain = (p.out_f32 ? kChainF32 : kChainBf16) / p.block_red;
    // whether a tile may take several passes (see Sums; the widest has the fewest chains)
    const long long own_blocks = ceil_div(ceil_div(MODE == PRODUCT_WGRAD ? p.rows : p.red, p.block_red), p.split);
    const bool is_long = own_blocks > (long long)p.chain << (!p.out_f32 ? 0 : widest <= 64 ? 2 : widest <= 128 ? 1 : 0);
    p.stage_bytes = p.subs * p.sub_bytes;
    p.stages = space / p.stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.out_at = (int)(kStageSpace / 1024 * 1024) - out_bytes;
    const uint64_t L = p.lanes, K = p.red, G = p.groups;
    bool ok;
    if (two) {
        // w [G][gate, up][n][k] read as k x il x (gate, up) x n / il blocks
        p.interleave = p.lanes % 16 == 0 ? 16 : 8;
        const uint64_t il = p.interleave;
        const uint64_t dims[5] = {K, il, 2, L / il, G}, strides[4] = {K, L * K, il * K, 2 * L * K};
        const uint32_t box[5] = {64, (uint32_t)il, 2, (uint32_t)(p.lane_step / il), 1};
        ok = make_map(&p.a, a, 5, dims, strides, box);
    } else if (MODE == PRODUCT_FORWARD) {
        ok = make_map3(&p.a, a, K, L, G, lane_rows);
    } else {
        ok = make_map3(&p.a, a, L, MODE == PRODUCT_DGRAD ? K : p.rows, G, kSubRed);
    }
    if (!ok) return EP_ERR_CUDA;
    if (MODE == PRODUCT_WGRAD) {
        if (!make_map3(&p.b[0], b, width, p.rows, p.groups, kSubRed)) return EP_ERR_CUDA;
    } else {
        const int boxes = widest / cg > 128 ? kBoxes : widest / cg / 16;
        for (int i = 0; i < boxes; ++i)
            if (!make_map3(&p.b[i], b, width, p.rows, p.groups, 16u * (i + 1))) return EP_ERR_CUDA;
    }
    if (!make_out_map(&p.o, p.out, p.out_f32, MODE == PRODUCT_DGRAD && gated ? 2 : 1, p.lanes, cols, p.groups))
        return EP_ERR_CUDA;
    const long long most = (long long)p.lane_tiles * p.groups * ceil_div(cols, p.col_max);
    if (most >= (1LL << 30)) return EP_ERR_INVALID_ARG;   // tile numbers stay within int
    const long long room = p.split > 1 ? most : sms / cg;
    const int clusters = (int)(most < room ? most : room);
    // whether the epilogue reads from memory: residual, pre-activations, output added to
    const bool side = MODE == PRODUCT_FORWARD ? p.residual != nullptr : MODE == PRODUCT_DGRAD ? p.z != nullptr : p.accumulate;
    if constexpr (MODE != PRODUCT_WGRAD) {
        if (gated && side)
            return cg == 2 ? launch<MODE, true, 2, true>(p, is_long, clusters, st) : launch<MODE, true, 1, true>(p, is_long, clusters, st);
    }
    if constexpr (MODE == PRODUCT_FORWARD) {   // (a gated gradient always reads its pre-activation)
        if (gated)
            return cg == 2 ? launch<MODE, true, 2, false>(p, is_long, clusters, st) : launch<MODE, true, 1, false>(p, is_long, clusters, st);
    }
    if (side) return cg == 2 ? launch<MODE, false, 2, true>(p, is_long, clusters, st) : launch<MODE, false, 1, true>(p, is_long, clusters, st);
    return cg == 2 ? launch<MODE, false, 2, false>(p, is_long, clusters, st) : launch<MODE, false, 1, false>(p, is_long, clusters, st);
}

bool aligned16(const void *q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

bool product_ok(const ep_product_t *a, bool wgrad) {
    if (!a || a->groups < 1 || a->groups > EP_MAX_E || a->rows < 0) return false;
    if (a->k < 8 || a->n < 8 || a->k % 8 || a->n % 8 || a->k > (1 << 24) || a->n > (1 << 24)) return false;
    if ((long long)a->groups * a->rows >= (1LL << 31)) return false;
    // a tensor map's strides stay below 2^40 bytes
    const long long wide = 4LL * (a->k > a->n ? a->k : a->n);   // elements of the widest row, and both its halves
    if (wide * a->rows >= (1LL << 38) || 4LL * a->n * a->k >= (1LL << 38)) return false;
    if (a->act < EP_ACT_NONE || a->act > EP_ACT_SWIGLU || (wgrad && a->act != EP_ACT_NONE)) return false;
    if (a->out_dtype != EP_BF16 && a->out_dtype != EP_F32) return false;
    return reinterpret_cast<uintptr_t>(a->counts) % 4 == 0 && reinterpret_cast<uintptr_t>(a->status) % 4 == 0;
}

ProductParams base_params(const ep_product_t *a) {
    ProductParams p = {};
    p.counts = a->counts;
    p.groups = a->groups;
    p.rows = a->rows;
    p.act = a->act;
    p.out_f32 = a->out_dtype == EP_F32;
    p.status = a->status;
    return p;
}

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

}  // namespace

cudaError_t product_status_word(int32_t **word) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int32_t *> cached[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (*word = cached[dev].load(std::memory_order_relaxed))) return cudaSuccess;
    void *at = nullptr;
    e = cudaGetSymbolAddress(&at, device_status);
    *word = static_cast<int32_t *>(at);
    if (e == cudaSuccess && dev < kMaxDevices) cached[dev].store(*word, std::memory_order_relaxed);
    return e;
}

uint64_t product_wait_limit() { return wait_limit_ns.load(std::memory_order_relaxed); }

}  // namespace ep

using namespace ep;

extern "C" int ep_product(const ep_product_t *a, const void *x, const void *w, const void *bias,
                          const void *residual, void *out, void *preact, void *stream) {
    if (!product_ok(a, false)) return EP_ERR_INVALID_ARG;
    if (a->rows == 0) return EP_OK;
    if (!x || !w || !out || !aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) ||
        !aligned16(out) || !aligned16(preact))
        return EP_ERR_INVALID_ARG;
    ProductParams p = base_params(a);
    p.lanes = a->n;
    p.red = a->k;
    p.bias = static_cast<const __nv_bfloat16 *>(bias);
    p.residual = static_cast<const __nv_bfloat16 *>(residual);
    p.preact = static_cast<__nv_bfloat16 *>(preact);
    p.out = out;
    Range range("ep:product");
    return launch<PRODUCT_FORWARD>(p, w, x, a->k, static_cast<cudaStream_t>(stream));
}

extern "C" int ep_product_dgrad(const ep_product_t *a, const void *dy, const void *w, const void *preact,
                                void *dx, void *stream) {
    if (!product_ok(a, false)) return EP_ERR_INVALID_ARG;
    if (a->rows == 0) return EP_OK;
    if (!dy || !w || !dx || !aligned16(dy) || !aligned16(w) || !aligned16(preact) || !aligned16(dx))
        return EP_ERR_INVALID_ARG;
    if ((a->act != EP_ACT_NONE) != (preact != nullptr)) return EP_ERR_INVALID_ARG;
    ProductParams p = base_params(a);
    p.lanes = a->k;
    p.red = a->n;
    p.z = static_cast<const __nv_bfloat16 *>(preact);
    p.out = dx;
    Range range("ep:product_dgrad");
    return launch<PRODUCT_DGRAD>(p, w, dy, a->n, static_cast<cudaStream_t>(stream));
}

extern "C" int ep_product_wgrad(const ep_product_t *a, const void *dy, const void *x, int32_t accumulate,
                                void *dw, void *dbias, void *stream) {
    if (!product_ok(a, true) || (accumulate != 0 && accumulate != 1)) return EP_ERR_INVALID_ARG;
    if (!dw || !aligned16(dw) || !aligned16(dbias)) return EP_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const uint64_t K = a->k, N = a->n, G = a->groups;
    const size_t size = a->out_dtype == EP_F32 ? 4 : 2;
    Range range("ep:product_wgrad");
    if (a->rows == 0) {   // no rows: the sums are empty
        if (accumulate) return EP_OK;
        if (cudaMemsetAsync(dw, 0, G * N * K * size, st) != cudaSuccess) return EP_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, G * N * size, st) != cudaSuccess) return EP_ERR_CUDA;
        return EP_OK;
    }
    if (!dy || !x || !aligned16(dy) || !aligned16(x)) return EP_ERR_INVALID_ARG;
    ProductParams p = base_params(a);
    p.lanes = a->k;
    p.cols = a->n;
    p.accumulate = accumulate;
    p.out = dw;
    const int rc = launch<PRODUCT_WGRAD>(p, x, dy, a->n, st);
    if (rc != EP_OK || !dbias) return rc;
    return launch_row_sums(dy, a->counts, a->groups, a->rows, a->n, p.out_f32, accumulate, dbias, st) ==
                   cudaSuccess
               ? EP_OK
               : EP_ERR_CUDA;
}

extern "C" int ep_product_status(void *stream) {
    static std::mutex one;   // status_taken is shared
    std::lock_guard<std::mutex> lock(one);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t status = 0;
    take_status<<<1, 1, 0, st>>>();
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&status, status_taken, sizeof(status), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return EP_ERR_CUDA;
    return status;
}

extern "C" int ep_product_wait_limit(int64_t ns) {
    if (ns < 1000 || ns > 60000000000LL) return EP_ERR_INVALID_ARG;
    wait_limit_ns.store((uint64_t)ns, std::memory_order_relaxed);
    return EP_OK;
}
