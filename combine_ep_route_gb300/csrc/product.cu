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
// One persistent CTA per SM: a TMA warp, an MMA warp, a warp that zeroes the
// rows past a group's count in the weight gradient's last block (a count can
// end inside it, and whatever lies there may be NaN), and four epilogue warps
// that drain one accumulator while the next fills.
#include "product.cuh"

#include <atomic>

#include <nvtx3/nvToolsExt.h>

#include "act.cuh"

namespace ep {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 128;          // accumulator lanes of a tile
constexpr int kColMax = 256;         // accumulator columns of a tile, at most
constexpr int kBlockRed = 64;        // reduction elements per stage: one 128-byte swizzled line
constexpr int kStages = 4;
constexpr int kABytes = kLanes * kBlockRed * 2;
constexpr int kBBytes = kColMax * kBlockRed * 2;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kChunkBytes = kBlockRed * 128;   // MN-major: 64 reduction lines of 64 elements
constexpr int kTmemCols = 512;       // two accumulators of 256 columns
constexpr uint64_t kWaitLimitNs = 2000000000ull;

struct Shared {
    uint64_t full[kStages], empty[kStages], tail[kStages];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
    int count[EP_MAX_E];             // rows in use per group
    int first[EP_MAX_E + 1];         // column tiles before each group
};

constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kStageBytes + sizeof(Shared);

// A wait of one of the kernel's roles: bounded, and cut short once any role of
// the CTA has given up.
__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, Shared *sh,
                                          const ProductParams &p) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    volatile int *abort = &sh->abort;
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (global_ns() - t0 > p.wait_limit_ns) {
            *abort = 1;
            if (p.status) atomicCAS(p.status, 0, EP_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

struct Tile {
    int g, lane0, col0, cols, n_mma, red, blocks;
};

// Column tiles of a group are of equal width (a multiple of 16), so 260 rows
// make two tiles of 144 and 116 and not of 256 and 4.
template <int MODE>
__device__ __forceinline__ int col_tiles(const ProductParams &p, int count) {
    const int cols = MODE == PRODUCT_WGRAD ? p.cols : count;
    return (cols + p.col_max - 1) / p.col_max;
}

template <int MODE, bool GATED>
__device__ __forceinline__ Tile find_tile(const ProductParams &p, const Shared *sh, int t) {
    int lo = 0, hi = p.groups;       // first[lo] * lane_tiles <= t < first[hi] * lane_tiles
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh->first[mid] * p.lane_tiles <= t)
            lo = mid;
        else
            hi = mid;
    }
    Tile x;
    x.g = lo;
    const int r = t - sh->first[lo] * p.lane_tiles;
    const int ct = sh->first[lo + 1] - sh->first[lo];
    const int count = sh->count[lo];
    const int all = MODE == PRODUCT_WGRAD ? p.cols : count;
    const int lt = r / ct;
    const int width = ((all + ct - 1) / ct + 15) & ~15;
    x.lane0 = lt * (GATED && MODE == PRODUCT_FORWARD ? kLanes / 2 : kLanes);
    x.col0 = (r - lt * ct) * width;
    x.cols = min(width, all - x.col0);
    x.n_mma = (x.cols + 15) & ~15;
    x.red = MODE == PRODUCT_WGRAD ? count : p.red;
    x.blocks = (x.red + kBlockRed - 1) / kBlockRed;
    return x;
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
__device__ __forceinline__ void st_out(const ProductParams &p, size_t at, float2 v) {
    if (p.out_f32)
        *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at) = v;
    else
        st_pair(static_cast<__nv_bfloat16 *>(p.out) + at, pack_bf16x2_rn(v.x, v.y));
}

// What the epilogue of one chunk reads from memory (residual, pre-activations or
// the output added to), fetched before the accumulators are waited for.
struct Side {
    uint32_t a[16], b[16];
};

// Where a lane's pairs of a chunk of 32 columns lie: its first feature, and the
// column of its i-th pair (see trade_pair; a gated forward chunk has 8 pairs).
template <int MODE, bool GATED>
struct Place {
    int f;
    bool ok, odd, up;
    __device__ __forceinline__ Place(const ProductParams &p, const Tile &x, int quad, int lane) {
        odd = lane & 1;
        if (MODE == PRODUCT_FORWARD && GATED) {
            const int il = p.interleave;   // 8 or 16
            up = lane & il;
            f = x.lane0 + quad * 16 + (il == 8 ? (lane >> 4) * 8 : 0) + (lane & (il - 1) & ~1);
        } else {
            up = false;
            f = x.lane0 + quad * 32 + (lane & ~1);
        }
        ok = f < p.lanes;
    }
    __device__ __forceinline__ int column(int i) const {
        return MODE == PRODUCT_FORWARD && GATED ? 4 * i + (up ? 2 : 0) + odd : 2 * i + odd;
    }
};

template <int MODE, bool GATED>
__device__ __forceinline__ void load_side(const ProductParams &p, size_t row0, int n,
                                          const Place<MODE, GATED> &at, Side &side) {
    constexpr int kPairs = MODE == PRODUCT_FORWARD && GATED ? 8 : 16;
    const bool want = MODE == PRODUCT_FORWARD ? p.residual != nullptr
                                              : MODE == PRODUCT_DGRAD ? GATED || p.act != EP_ACT_NONE : p.accumulate;
    if (!want || !at.ok) return;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int j = at.column(i);
        if (j >= n) continue;
        if (MODE == PRODUCT_FORWARD) {
            side.a[i] = ld_pair(p.residual + (row0 + j) * p.lanes + at.f);
        } else if (MODE == PRODUCT_DGRAD) {
            const __nv_bfloat16 *z = p.z + (row0 + j) * (GATED ? 2 : 1) * p.lanes + at.f;
            side.a[i] = ld_pair(z);
            if (GATED) side.b[i] = ld_pair(z + p.lanes);
        } else if (p.out_f32) {
            const float2 v = *reinterpret_cast<const float2 *>(static_cast<const float *>(p.out) +
                                                               (row0 + j) * p.lanes + at.f);
            side.a[i] = __float_as_uint(v.x), side.b[i] = __float_as_uint(v.y);
        } else {
            side.a[i] = ld_pair(static_cast<const __nv_bfloat16 *>(p.out) + (row0 + j) * p.lanes + at.f);
        }
    }
}

// The epilogue of 32 accumulator columns of one warp's 32 lanes, of which n are
// output rows row0 .. row0 + n - 1.
template <int MODE, bool GATED>
__device__ __forceinline__ void epilogue_chunk(const ProductParams &p, const float (&acc)[32], size_t row0,
                                               int n, const Place<MODE, GATED> &at, float2 bias,
                                               const Side &side) {
    if constexpr (MODE == PRODUCT_FORWARD && GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (4 * i >= n) break;
            float2 a = trade_pair(acc[4 * i], acc[4 * i + 1], at.odd);
            float2 b = trade_pair(acc[4 * i + 2], acc[4 * i + 3], at.odd);
            a.x += bias.x, a.y += bias.y, b.x += bias.x, b.y += bias.y;
            if (p.preact && at.ok) {
                const int ja = 4 * i + at.odd, jb = ja + 2;
                __nv_bfloat16 *z = p.preact + (at.up ? p.lanes : 0) + at.f;
                if (ja < n) st_pair(z + (row0 + ja) * 2 * p.lanes, pack_bf16x2_rn(a.x, a.y));
                if (jb < n) st_pair(z + (row0 + jb) * 2 * p.lanes, pack_bf16x2_rn(b.x, b.y));
            }
            // gate lanes give their second token's pair for the up pair of the first
            const float2 give = at.up ? a : b;
            float2 got;
            got.x = __shfl_xor_sync(0xFFFFFFFFu, give.x, p.interleave);
            got.y = __shfl_xor_sync(0xFFFFFFFFu, give.y, p.interleave);
            const float2 gate = at.up ? got : a, up = at.up ? b : got;
            const int j = at.column(i);
            if (at.ok && j < n) {
                float2 y = make_float2(act_value(gate.x, EP_ACT_SILU) * up.x,
                                       act_value(gate.y, EP_ACT_SILU) * up.y);
                if (p.residual) {
                    const float2 r = unpack_bf16x2(side.a[i]);
                    y.x += r.x, y.y += r.y;
                }
                st_out(p, (row0 + j) * p.lanes + at.f, y);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (2 * i >= n) break;
            float2 v = trade_pair(acc[2 * i], acc[2 * i + 1], at.odd);
            const int j = at.column(i);
            if (!at.ok || j >= n) continue;
            if (MODE == PRODUCT_DGRAD && GATED) {
                const float2 zg = unpack_bf16x2(side.a[i]), zu = unpack_bf16x2(side.b[i]);
                const size_t o = (row0 + j) * 2 * p.lanes + at.f;
                st_out(p, o, make_float2(v.x * zu.x * act_slope(zg.x, EP_ACT_SILU),
                                         v.y * zu.y * act_slope(zg.y, EP_ACT_SILU)));
                st_out(p, o + p.lanes, make_float2(v.x * act_value(zg.x, EP_ACT_SILU),
                                                   v.y * act_value(zg.y, EP_ACT_SILU)));
                continue;
            }
            const size_t o = (row0 + j) * p.lanes + at.f;
            if (MODE == PRODUCT_FORWARD) {
                v.x += bias.x, v.y += bias.y;
                if (p.preact) st_pair(p.preact + o, pack_bf16x2_rn(v.x, v.y));
                v = make_float2(act_value(v.x, p.act), act_value(v.y, p.act));
                if (p.residual) {
                    const float2 r = unpack_bf16x2(side.a[i]);
                    v.x += r.x, v.y += r.y;
                }
            } else if (MODE == PRODUCT_DGRAD) {
                if (p.act != EP_ACT_NONE) {
                    const float2 z = unpack_bf16x2(side.a[i]);
                    v.x *= act_slope(z.x, p.act), v.y *= act_slope(z.y, p.act);
                }
            } else if (p.accumulate) {
                const float2 was = p.out_f32 ? make_float2(__uint_as_float(side.a[i]), __uint_as_float(side.b[i]))
                                             : unpack_bf16x2(side.a[i]);
                v.x += was.x, v.y += was.y;
            }
            st_out(p, o, v);
        }
    }
}

template <int MODE, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ ProductParams p) {
    constexpr bool kMnA = MODE != PRODUCT_FORWARD, kMnB = MODE == PRODUCT_WGRAD;
    extern __shared__ uint8_t raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    Shared *sh = reinterpret_cast<Shared *>(stages + (size_t)kStages * kStageBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    for (int g = threadIdx.x; g < p.groups; g += kThreads)
        sh->count[g] = p.counts ? max(0, min(p.counts[g], p.rows)) : p.rows;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->empty[s], 1);
            mbar_init(&sh->tail[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 4);
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.a);
        tma_prefetch_map(&p.b[0]);
    }
    if (warp == 3) tmem_alloc(&sh->tmem, kTmemCols);
    __syncthreads();
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
    tc_fence_after();
    const int total = sh->first[p.groups] * p.lane_tiles;
    const uint32_t tmem = sh->tmem;

    uint32_t it = 0;       // reduction blocks so far: stage it % kStages, phase (it / kStages) & 1
    uint32_t n_acc = 0;    // accumulators so far
    uint32_t on_tail = 0, tail_phase = 0;   // producer, a bit per stage: last load signals tail[], and its phase
    if (warp == 0) {
        // ---- TMA: both operands of every block into the next free stage
        if (lane == 0) {
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Tile x = find_tile<MODE, GATED>(p, sh, t);
                for (int kb = 0; kb < x.blocks; ++kb, ++it) {
                    const int s = it % kStages;
                    ok = role_wait(&sh->empty[s], ((it / kStages) & 1) ^ 1, sh, p);
                    if (!ok) break;
                    uint8_t *sa = stages + (size_t)s * kStageBytes, *sb = sa + kABytes;
                    const int r0 = kb * kBlockRed;
                    const int chunks = (x.n_mma + 63) / 64;
                    const uint32_t bytes = kABytes + (kMnB ? chunks * kChunkBytes : x.n_mma * 128);
                    // a weight gradient's block that ends past the count goes through the
                    // zeroing warp before the MMA warp sees it
                    const bool tail = kMnB && x.red - r0 < kBlockRed;
                    uint64_t *bar = tail ? &sh->tail[s] : &sh->full[s];
                    if (kMnB) {
                        // phase bit of the next use: flipped by each use
                        if (tail) tail_phase ^= 1u << s;
                        on_tail = (on_tail & ~(1u << s)) | (tail ? 1u << s : 0u);
                    }
                    mbar_arrive_expect_tx(bar, bytes);
                    if (MODE == PRODUCT_FORWARD) {
                        if (GATED)
                            tma_load_5d(sa, &p.a, r0, 0, 0, x.lane0 / p.interleave, x.g, bar);
                        else
                            tma_load_3d(sa, &p.a, r0, x.lane0, x.g, bar);
                    } else {
                        tma_load_3d(sa, &p.a, x.lane0, r0, x.g, bar);
                        tma_load_3d(sa + kChunkBytes, &p.a, x.lane0 + 64, r0, x.g, bar);
                    }
                    if (kMnB) {
                        for (int c = 0; c < chunks; ++c)
                            tma_load_3d(sb + c * kChunkBytes, &p.b[0], x.col0 + 64 * c, r0, x.g, bar);
                    } else {
                        int done = 0;
                        for (int b = 0; b < kBoxes; ++b)
                            for (const int box = 128 >> b; x.n_mma - done >= box; done += box)
                                tma_load_3d(sb + done * 128, &p.b[b], r0, x.col0 + done, x.g, bar);
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---- MMA: one thread issues four steps of 16 per block
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile x = find_tile<MODE, GATED>(p, sh, t);
            if (x.blocks == 0) continue;
            const int a = n_acc & 1;
            ok = role_wait(&sh->acc_empty[a], ((n_acc / 2) & 1) ^ 1, sh, p);
            if (!ok) break;
            tc_fence_after();
            const uint32_t idesc = mma_idesc(kLanes, x.n_mma, kMnA, kMnB);
            const uint32_t d = tmem + a * kColMax;
            for (int kb = 0; kb < x.blocks; ++kb, ++it) {
                const int s = it % kStages;
                ok = role_wait(&sh->full[s], (it / kStages) & 1, sh, p);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t sa = smem_u32(stages + (size_t)s * kStageBytes), sb = sa + kABytes;
                    const int steps = min(4, (x.red - kb * kBlockRed + 15) / 16);
                    for (int i = 0; i < steps; ++i) {
                        const uint64_t da = kMnA ? smem_desc(sa + i * 2048, kChunkBytes, 1024)
                                                 : smem_desc(sa + i * 32, 16, 1024);
                        const uint64_t db = kMnB ? smem_desc(sb + i * 2048, kChunkBytes, 1024)
                                                 : smem_desc(sb + i * 32, 16, 1024);
                        mma_bf16(d, da, db, idesc, kb > 0 || i > 0);
                    }
                    mma_commit(&sh->empty[s]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) mma_commit(&sh->acc_full[a]);
            __syncwarp();
            ++n_acc;
        }
    } else if (warp == 2 && kMnB) {
        // ---- rows at or past the count, in the last block: zero in both operands
        uint32_t used = 0;   // a bit per stage: parity of its next use here
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile x = find_tile<MODE, GATED>(p, sh, t);
            it += x.blocks;
            const int left = x.red % kBlockRed;
            if (left == 0) continue;
            const int s = (it - 1) % kStages;
            ok = role_wait(&sh->tail[s], (used >> s) & 1, sh, p);
            used ^= 1u << s;
            if (!ok) break;
            // rows up to the MMA's last step of 16
            const int rows = ((left + 15) & ~15) - left;
            const int chunks = 2 + (x.n_mma + 63) / 64;
            uint8_t *sa = stages + (size_t)s * kStageBytes;
            for (int i = lane; i < rows * chunks * 8; i += 32) {
                const int c = i / (rows * 8), r = i % (rows * 8) / 8, v = i % 8;
                *reinterpret_cast<uint4 *>(sa + c * kChunkBytes + (left + r) * 128 + v * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->full[s]);
        }
    } else if (warp >= 4) {
        // ---- epilogue: this warp's 32 lanes of every accumulator
        const int quad = warp - 4;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile x = find_tile<MODE, GATED>(p, sh, t);
            if (x.blocks == 0 && MODE == PRODUCT_WGRAD && p.accumulate) continue;
            const Place<MODE, GATED> at(p, x, quad, lane);
            const size_t row0 = (size_t)x.g * (MODE == PRODUCT_WGRAD ? p.cols : p.rows) + x.col0;
            float2 bias = make_float2(0.f, 0.f);
            if (MODE == PRODUCT_FORWARD && p.bias && at.ok)
                bias = unpack_bf16x2(ld_pair(p.bias + (size_t)x.g * (GATED ? 2 : 1) * p.lanes +
                                             (at.up ? p.lanes : 0) + at.f));
            const int a = n_acc & 1;
            if (x.blocks > 0) {
                ok = role_wait(&sh->acc_full[a], (n_acc / 2) & 1, sh, p);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            for (int c = 0; c < x.cols; c += 32) {
                float acc[32];
                Side side;
                const int n = min(32, x.cols - c);
                load_side(p, row0 + c, n, at, side);
                if (x.blocks > 0) {
                    uint32_t r[32];
                    tmem_ld32(tmem + a * kColMax + c + ((uint32_t)(quad * 32) << 16), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[j] = __uint_as_float(r[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[j] = 0.f;
                }
                epilogue_chunk(p, acc, row0 + c, n, at, bias, side);
            }
            if (x.blocks > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->acc_empty[a]);
                ++n_acc;
            }
        }
    }
    __syncthreads();
    if (sh->abort && threadIdx.x < 64) {
        // a wait ran out: let the copies and MMAs in flight finish (bounded) before
        // shared and tensor memory are given up
        const uint64_t t0 = global_ns();
        if (threadIdx.x == 0) {
            for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) {
                const int s = i % kStages;
                uint64_t *bar = (on_tail >> s) & 1 ? &sh->tail[s] : &sh->full[s];
                const uint32_t phase = (on_tail >> s) & 1 ? ((tail_phase >> s) & 1) ^ 1 : (i / kStages) & 1;
                while (!mbar_try_wait(bar, phase) && global_ns() - t0 < 100000000ull)
                    ;
            }
        } else if (threadIdx.x == 32) {
            mma_commit(&sh->drain);
            while (!mbar_try_wait(&sh->drain, 0) && global_ns() - t0 < 100000000ull)
                ;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_free(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library links no driver library).
EncodeTiled encoder() {
    static std::atomic<EncodeTiled> found{nullptr};
    EncodeTiled e = found.load(std::memory_order_acquire);
    if (e) return e;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    e = reinterpret_cast<EncodeTiled>(fn);
    found.store(e, std::memory_order_release);
    return e;
}

// A bf16 tensor of `rank` dimensions (innermost first, strides in elements of
// dimensions 1..), read in boxes with the 128-byte swizzle and zeros outside.
bool make_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
              const uint32_t *box) {
    EncodeTiled enc = encoder();
    if (!enc) return false;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i > 0) s[i - 1] = strides[i - 1] * 2;
    }
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), d, s, b, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [groups][rows][cols] read in boxes of 64 columns and box_rows rows.
bool make_map3(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t groups,
               uint32_t box_rows) {
    const uint64_t dims[3] = {cols, rows, groups}, strides[2] = {cols, cols * rows};
    const uint32_t box[3] = {64, box_rows, 1};
    return make_map(m, base, 3, dims, strides, box);
}

// The multiprocessor count of the current device.
cudaError_t sm_count(int *out) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (*out = cached[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < kMaxDevices) cached[dev].store(*out, std::memory_order_relaxed);
    return e;
}

template <int MODE, bool GATED>
int launch(const ProductParams &p, int grid, cudaStream_t st) {
    const void *fn = reinterpret_cast<const void *>(&product_kernel<MODE, GATED>);
    if (ensure_dyn_smem(fn, kSmemBytes) != cudaSuccess) return EP_ERR_CUDA;
    product_kernel<MODE, GATED><<<grid, kThreads, kSmemBytes, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

template <int MODE>
int launch(ProductParams &p, cudaStream_t st) {
    const bool gated = p.act == EP_ACT_SWIGLU;
    const int per_tile = gated && MODE == PRODUCT_FORWARD ? kLanes / 2 : kLanes;
    p.lane_tiles = (p.lanes + per_tile - 1) / per_tile;
    p.col_max = kColMax;
    p.wait_limit_ns = kWaitLimitNs;
    const long long cols = MODE == PRODUCT_WGRAD ? p.cols : p.rows;
    const long long most = (long long)p.lane_tiles * p.groups * ((cols + p.col_max - 1) / p.col_max);
    if (most >= (1LL << 31)) return EP_ERR_INVALID_ARG;
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return EP_ERR_CUDA;
    const int grid = (int)(most < sms ? most : sms);
    if constexpr (MODE != PRODUCT_WGRAD) {
        if (gated) return launch<MODE, true>(p, grid, st);
    }
    return launch<MODE, false>(p, grid, st);
}

bool aligned16(const void *q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

bool product_ok(const ep_product_t *a, bool wgrad) {
    if (!a || a->groups < 1 || a->groups > EP_MAX_E || a->rows < 0) return false;
    if (a->k < 8 || a->n < 8 || a->k % 8 || a->n % 8 || a->k > (1 << 24) || a->n > (1 << 24)) return false;
    if ((long long)a->groups * a->rows >= (1LL << 31)) return false;
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

}  // namespace ep

using namespace ep;

extern "C" int ep_product(const ep_product_t *a, const void *x, const void *w, const void *bias,
                          const void *residual, void *out, void *preact, void *stream) {
    if (!product_ok(a, false)) return EP_ERR_INVALID_ARG;
    if (a->rows == 0) return EP_OK;
    if (!x || !w || !out || !aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) ||
        !aligned16(out) || !aligned16(preact))
        return EP_ERR_INVALID_ARG;
    const bool gated = a->act == EP_ACT_SWIGLU;
    ProductParams p = base_params(a);
    p.lanes = a->n;
    p.red = a->k;
    p.bias = static_cast<const __nv_bfloat16 *>(bias);
    p.residual = static_cast<const __nv_bfloat16 *>(residual);
    p.preact = static_cast<__nv_bfloat16 *>(preact);
    p.out = out;
    const uint64_t K = a->k, N = a->n, G = a->groups;
    bool ok;
    if (gated) {
        // w [G][gate, up][n][k] read as k x il x (gate, up) x n / il blocks
        p.interleave = a->n % 16 == 0 ? 16 : 8;
        const uint64_t il = p.interleave;
        const uint64_t dims[5] = {K, il, 2, N / il, G}, strides[4] = {K, N * K, il * K, 2 * N * K};
        const uint32_t box[5] = {64, (uint32_t)il, 2, (uint32_t)(64 / il), 1};
        ok = make_map(&p.a, w, 5, dims, strides, box);
    } else {
        ok = make_map3(&p.a, w, K, N, G, kLanes);
    }
    for (int b = 0; b < kBoxes && ok; ++b) ok = make_map3(&p.b[b], x, K, a->rows, G, 128u >> b);
    if (!ok) return EP_ERR_CUDA;
    Range range("ep:product");
    return launch<PRODUCT_FORWARD>(p, static_cast<cudaStream_t>(stream));
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
    const uint64_t K = a->k, N = a->n, G = a->groups;
    bool ok = make_map3(&p.a, w, K, N, G, kBlockRed);
    for (int b = 0; b < kBoxes && ok; ++b) ok = make_map3(&p.b[b], dy, N, a->rows, G, 128u >> b);
    if (!ok) return EP_ERR_CUDA;
    Range range("ep:product_dgrad");
    return launch<PRODUCT_DGRAD>(p, static_cast<cudaStream_t>(stream));
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
    if (!make_map3(&p.a, x, K, a->rows, G, kBlockRed) || !make_map3(&p.b[0], dy, N, a->rows, G, kBlockRed))
        return EP_ERR_CUDA;
    const int rc = launch<PRODUCT_WGRAD>(p, st);
    if (rc != EP_OK || !dbias) return rc;
    return launch_row_sums(dy, a->counts, a->groups, a->rows, a->n, p.out_f32, accumulate, dbias, st) ==
                   cudaSuccess
               ? EP_OK
               : EP_ERR_CUDA;
}
