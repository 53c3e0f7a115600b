// w4_tiles.cu -- products with 4-bit weights on the 5th-generation tensor cores.
//
// D[lane][col] = sum_k w[lane][k] x[col][k]: 128 rows of the weight on the accumulator's lanes,
// up to 128 rows of x on its columns. The weight is the operand that sits in tensor memory:
// TMA brings steps of 256 elements of 4-bit codes and their scales, sixteen warps make bf16 of
// them (a lane its own row, 64 bytes of codes at a time) and store them to tensor memory, from
// where the MMAs read them; x goes by TMA to shared memory with the 128-byte swizzle. So the
// expanded weight never passes through shared memory, whose bandwidth the MMAs' other operand
// needs (an MMA of 128 columns takes 65-74 cycles that way, 107 with both operands in shared
// memory). A gated product's gate and up rows are interleaved by eights by the tensor maps alone.
//
// One persistent CTA per SM: a TMA warp for the codes and scales, one for x, an MMA warp, two pairs
// of groups of four warps that expand a step each, half a step to a group, and eight epilogue warps
// that drain one accumulator while the next fills. Where tiles are many, pairs of CTAs share an MMA
// of 256 weight rows (cta_group::2): each holds half of x, which is what most of the bytes from L2 are.
// Dense products with few tiles let up to four CTAs of a cluster share a tile's reduction and join
// their sums through distributed shared memory.
//
// What bounds it: no one unit is full. With few rows of x, the codes' stream with its waits and the expanding
// instructions (64 experts of 7168 x 2048 with four rows each, int4: 115 us, 4.4 TB/s, the copies alone 97; issue
// slots 66 % used, and warps wait for barriers and copies more than for anything else; yet fp4, whose decode takes
// 17 instructions a word instead of 9, takes 133, and groups of 32 or 128 the same). With about 120 rows the same
// and the gated epilogue (64 experts of 2 x 1024 x 2048: int4 63 us, fp4 68 to 70, 920 TFLOP/s; tensor pipe 49 %
// busy). With more, each 128 rows expand their weight again, which keeps the tensor pipe at 68 % (64 experts of
// 2 x 2048 x 4096 under Zipf: 309 to 315 us, 1.2 PFLOP/s). What each step gave (us, the three): the first kernel 228 / 111 / 476; one thread waits and issues 181 / 95 / 396;
// steps of 256 158 / 93 / 347; warps that skip to their own steps 130 / 87 / 323; pairs of CTAs, x in a
// ring of its own 134 / 76 / 304; x by one copy a step 120 / 76 / 289.
#include "w4.cuh"

#include <nvtx3/nvToolsExt.h>

#include "act.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace ep {

namespace {

// Pairs of groups of four warps that expand steps by turns, half a step to a group. No more pairs
// than slots in tensor memory: then what a group has seen of its last step tells it that its slot's
// last use but one is over, so that the parity it waits for is not that of an older phase.
constexpr int kTurns = 2;
constexpr int kExpandWarps = kTurns * 8;
constexpr int kEpilogueWarps = 8;    // two per quarter of the accumulator lanes
constexpr int kThreads = 128 + (kExpandWarps + kEpilogueWarps) * 32;
constexpr int kFirstEpilogue = 4 + kExpandWarps;
constexpr int kLanes = 128;          // weight rows of a tile
constexpr int kStep = 256;           // elements of k of a block: rows of codes of 128 bytes
constexpr int kColMax = 128;         // rows of x of a tile, at most
constexpr int kBoxes = kColMax / 16;   // boxes of 16, 32, ... 128 rows of x
constexpr int kChunk = 16;           // columns that an epilogue warp takes at once
constexpr int kACols = kStep / 2;    // tensor-memory columns of a step: two elements to one
constexpr int kTmemCols = 512;       // two accumulators, then steps of the weight
constexpr int kMaxSlots = (kTmemCols - 2 * 32) / kACols;
constexpr int kMaxXSlots = 8;
constexpr int kCodeBytes = kLanes * kStep / 2;
constexpr int kCodeSlot = kCodeBytes + kLanes * (kStep / 32) * 2;   // with the scales, at most
constexpr int kMaxCodeSlots = 8;
static_assert(kMaxCodeSlots % kTurns == 0, "a slot's uses are one pair of groups'");
constexpr int kMaxSplit = 4;
constexpr uint32_t kSleepNs = 1000000;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct TileParams {
    CUtensorMap codes, scales;
    CUtensorMap x[kBoxes];    // boxes of a step (k a multiple of 64), or of one line of 64 elements
    W4Params w;
    int lane_step, lane_tiles;       // output features of a tile, tiles per group
    int col_max;                     // widest column tile
    int code_slots;                  // ring of codes and scales
    int slots;                       // ring of expanded steps in tensor memory
    int x_slots, x_bytes;            // ring of x; bytes of a slot
    int acc_stride;                  // columns of an accumulator
    int scale_parts;                 // groups of a step
    int whole_lines;                 // k is a multiple of 64
    int steps, split;                // steps of k; CTAs of a cluster that share them
    int32_t *status;
    uint64_t wait_limit_ns;
    uint32_t sleep_ns;
};

struct Shared {
    uint64_t code_full[kMaxCodeSlots], code_empty[kMaxCodeSlots];
    uint64_t x_full[kMaxXSlots], x_empty[kMaxXSlots];
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort;
    int count[EP_MAX_E];             // rows in use, of the groups in the order they are worked on
    int first[EP_MAX_E + 1];         // column tiles before it
    uint16_t group[EP_MAX_E];
};

constexpr size_t kSmemMax = 227 * 1024;
constexpr size_t kRingSpace = (kSmemMax - 1024 - sizeof(Shared)) / 1024 * 1024;

struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++s == slots) s = 0, phase ^= 1;
    }
    __device__ __forceinline__ void skip(int n, int slots) {   // n <= slots
        s += n;
        if (s >= slots) s -= slots, phase ^= 1;
    }
};

// 32 weights from 16 bytes of codes.
template <bool FP4, bool LARGE>
__device__ __forceinline__ void expand(uint4 c, const W4Scale<FP4> &scale, uint32_t *r) {
    const uint32_t words[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t pair[4];
        w4_values<FP4, LARGE>(words[q], scale, pair);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[q * 4 + j] = pair[j];
    }
}

// D (+)= A * B over 16 elements, A from tensor memory.
template <int CG>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int u, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
            : "memory");
}

// 16 columns of this warp's 32 lanes; valid after tmem_ld_wait().
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// An arrival on a barrier of any CTA of the cluster, after this thread's stores to tensor memory
// (which it has waited for and fenced). At cluster scope the release would wait for all of the
// thread's memory traffic, once per step.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A bounded wait, cut short once any role of the CTA has given up.
__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, Shared *sh, const TileParams &p) {
    if (mbar_try_wait_ns(bar, parity, p.sleep_ns)) return true;
    const uint64_t t0 = global_ns();
    volatile int *abort = &sh->abort;
    while (!mbar_try_wait_ns(bar, parity, p.sleep_ns)) {
        if (*abort) return false;
        if (global_ns() - t0 > p.wait_limit_ns) {
            *abort = 1;
            atomicCAS(p.status, 0, EP_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
// The same by a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Shared *sh, const TileParams &p) {
    return __all_sync(kAll, role_wait(bar, parity, sh, p));
}

// Waits (bounded) for the MMAs that this thread has issued.
template <int CG>
__device__ __forceinline__ void drain_mma(Shared *sh) {
    const uint64_t since = global_ns();
    mma_commit<CG>(&sh->drain);
    while (!mbar_try_wait(&sh->drain, 0) && global_ns() - since < 100000000ull)
        ;
}

// Columns of each of ct tiles over `all` > 0 columns: 130 rows make 80 and 50, not 128 and 2.
template <int CG>
__device__ __forceinline__ int tile_width(int all, int ct) {
    constexpr int kUnit = 16 * CG;
    return ((all - 1) / ct + kUnit) / kUnit * kUnit;
}

// The groups' row counts, dearest tiles first, so that the last round is a cheap one. Ends in a barrier.
__device__ __forceinline__ void order_groups(const TileParams &p, Shared *sh) {
    const int own = threadIdx.x, groups = p.w.groups;
    const int32_t *counts = p.w.counts;
    if (groups > kThreads || !counts) {
        for (int g = own; g < groups; g += kThreads) {
            sh->count[g] = counts ? max(0, min(counts[g], p.w.rows)) : p.w.rows;
            sh->group[g] = (uint16_t)g;
        }
        __syncthreads();
        return;
    }
    int count = 0;
    if (own < groups) {
        count = max(0, min(counts[own], p.w.rows));
        sh->first[own] = min(count, kColMax);
    }
    __syncthreads();
    if (own < groups) {
        const int key = min(count, kColMax);
        int ahead = 0;
        for (int g = 0; g < groups; ++g) {
            const int other = sh->first[g];
            ahead += other > key || (other == key && g < own);
        }
        sh->count[ahead] = count;
        sh->group[ahead] = (uint16_t)own;
    }
    __syncthreads();
}

struct Tile {
    int g, lane0;            // group, first output feature
    int col0, cols, n_mma;   // first row of x, rows in use, columns of the MMA
};
struct Walk {
    int at = -1, begin = 0, end = 0;   // the current group's place, its tiles [begin, end)
    int ct = 0, width = 0;
};

// Column tiles innermost: the CTAs that share a lane tile's weight work at the same time, so
// all but one find it in L2.
template <int CG>
__device__ __forceinline__ Tile find_tile(const TileParams &p, const Shared *sh, int t, uint32_t rank, Walk &w) {
    if (t >= w.end) {
        do {
            ++w.at;
            w.begin = w.end;
            w.end = sh->first[w.at + 1] * p.lane_tiles;
        } while (t >= w.end);
        w.ct = sh->first[w.at + 1] - sh->first[w.at];
        w.width = tile_width<CG>(sh->count[w.at], w.ct);
    }
    const int r = t - w.begin, lt = w.ct == 1 ? r : r / w.ct, c = r - lt * w.ct;
    Tile x;
    x.g = sh->group[w.at];
    x.lane0 = (CG == 1 ? lt : lt * 2 + (int)rank) * p.lane_step;
    x.col0 = c * w.width;
    x.cols = min(w.width, sh->count[w.at] - x.col0);
    x.n_mma = (x.cols + 16 * CG - 1) / (16 * CG) * (16 * CG);
    return x;
}

template <int ACT>
__device__ __forceinline__ void act_all(float (&v)[kChunk]) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) v[j] = act_value(v[j], ACT);
}

// kChunk columns of one warp's 32 lanes: bias, activation, residual, out. n of them are rows in use.
// Lanes first trade columns with a partner, so that each ends with half of them: of a gated product
// gate lanes (0-7, 16-23) take the even ones' ups from the lanes eight further and give the odd
// ones' gates; otherwise neighbours end with two features of the even or the odd columns.
template <bool GATED>
__device__ __forceinline__ void epilogue_chunk(const TileParams &p, float (&v)[kChunk], size_t row0, int n, int quad, int lane,
                                               int lane0, float bias) {
    const W4Params &w = p.w;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) v[j] += bias;
    if (!GATED) {
        switch (w.act) {
            case EP_ACT_RELU: act_all<EP_ACT_RELU>(v); break;
            case EP_ACT_SILU: act_all<EP_ACT_SILU>(v); break;
            case EP_ACT_GELU: act_all<EP_ACT_GELU>(v); break;
            case EP_ACT_GELU_TANH: act_all<EP_ACT_GELU_TANH>(v); break;
            default: break;
        }
    }
    const bool odd = GATED ? lane & 8 : lane & 1;
    const int f = GATED ? lane0 + quad * 16 + (lane >> 4) * 8 + (lane & 7) : lane0 + quad * 32 + (lane & ~1);
    const int last = f < w.n ? n - odd : 0;   // this lane's columns are those of 0, 2, .. below it
    const size_t step = 2 * (size_t)w.n, at = (row0 + odd) * w.n + f;
    __nv_bfloat16 *out = w.out + at;
    const __nv_bfloat16 *residual = w.residual ? w.residual + at : nullptr;
#pragma unroll
    for (int i = 0; i < kChunk / 2; ++i, out += step) {
        const float got = __shfl_xor_sync(kAll, odd ? v[2 * i] : v[2 * i + 1], GATED ? 8 : 1);
        float lo = odd ? got : v[2 * i], hi = odd ? v[2 * i + 1] : got;
        if (GATED) {
            lo = act_value(lo, EP_ACT_SILU) * hi;
            if (residual && 2 * i < last) lo += __bfloat162float(residual[i * step]);
            if (2 * i < last) *out = __float2bfloat16_rn(lo);
        } else {
            if (residual && 2 * i < last) {
                const float2 r = unpack_bf16x2(*reinterpret_cast<const uint32_t *>(residual + i * step));
                lo += r.x, hi += r.y;
            }
            if (2 * i < last) *reinterpret_cast<uint32_t *>(out) = pack_bf16x2_rn(lo, hi);
        }
    }
}

template <bool GATED>
__device__ __forceinline__ float bias_of(const TileParams &p, const Tile &x, int quad, int lane) {
    if (!p.w.bias) return 0.f;
    const int f = GATED ? x.lane0 + quad * 16 + (lane >> 4) * 8 + (lane & 7) : x.lane0 + quad * 32 + lane;
    if (f >= p.w.n) return 0.f;
    return __bfloat162float(p.w.bias[(size_t)x.g * p.w.wide + (GATED && (lane & 8) ? p.w.n : 0) + f]);
}

template <bool FP4, bool GATED, int CG>
__global__ void __launch_bounds__(kThreads, 1) w4_tiles_kernel(const __grid_constant__ TileParams p) {
    extern __shared__ uint8_t raw[];
    uint8_t *rings = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *xs = rings, *cs = rings + (size_t)p.x_slots * p.x_bytes;
    Shared *sh = reinterpret_cast<Shared *>(rings + kRingSpace);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 || p.split > 1 ? cluster_rank() : 0;
    const int per_cluster = CG == 2 ? 2 : p.split;
    const int t0 = blockIdx.x / per_cluster, t_step = gridDim.x / per_cluster;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.code_slots; ++s) {
            mbar_init(&sh->code_full[s], 1);
            mbar_init(&sh->code_empty[s], 8);   // the warps that expand it
        }
        for (int s = 0; s < p.slots; ++s) {
            mbar_init(&sh->full[s], 8 * CG);
            mbar_init(&sh->empty[s], 1);
        }
        for (int s = 0; s < p.x_slots; ++s) {
            mbar_init(&sh->x_full[s], CG);
            mbar_init(&sh->x_empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], kEpilogueWarps * CG);
        }
        mbar_init(&sh->drain, 1);
        sh->abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.codes);
        tma_prefetch_map(&p.scales);
    }
    if (warp == 2) tmem_alloc<CG>(&sh->tmem, kTmemCols);
    pdl_wait();   // nothing above reads or writes global memory
    pdl_launch_dependents();
    order_groups(p, sh);
    if (warp == 0) {   // exclusive prefix of the groups' column tiles
        int base = 0;
        for (int g0 = 0; g0 < p.w.groups; g0 += 32) {
            const int g = g0 + lane;
            const int own = g < p.w.groups ? (sh->count[g] + p.col_max - 1) / p.col_max : 0;
            int sum = own;
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(kAll, sum, d);
                if (lane >= d) sum += v;
            }
            if (g < p.w.groups) sh->first[g] = base + sum - own;
            base += __shfl_sync(kAll, sum, 31);
        }
        if (lane == 0) sh->first[p.w.groups] = base;
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();   // both CTAs' barriers are ready before either signals the other's
    tc_fence_after();
    const int total = sh->first[p.w.groups] * p.lane_tiles;
    const uint32_t tmem = sh->tmem;
    const int part = CG == 2 ? 0 : (int)rank;
    const int lo = p.steps * part / p.split, hi = p.steps * (part + 1) / p.split;   // this CTA's steps of a tile

    Walk walk;
    Ring ring;
    int issued = 0;   // producers: loads into their ring so far
    bool ok = true;
    if (warp == 0) {
        // ---- TMA: codes and scales
        for (int t = t0; t < total && ok; t += t_step) {
            const Tile x = find_tile<CG>(p, sh, t, rank, walk);
            for (int ks = lo; ks < hi; ++ks, ++issued, ring.next(p.code_slots)) {
                ok = warp_wait(&sh->code_empty[ring.s], ring.phase ^ 1, sh, p);
                if (!ok) break;
                if (elect_one()) {
                    uint64_t *full = &sh->code_full[ring.s];
                    mbar_arrive_expect_tx(full, kCodeBytes + kLanes * 2 * p.scale_parts);
                    const uint32_t bar = smem_u32(full);
                    uint8_t *dst = cs + ring.s * kCodeSlot;
                    if (GATED) tma_load_5d<1>(dst, &p.codes, ks * (kStep / 2), 0, 0, x.lane0 / 8, x.g, bar);
                    else tma_load_3d<1>(dst, &p.codes, ks * (kStep / 2), x.lane0, x.g, bar);
                    // scales of 64 rows, then of 64 more: gated, of the gates and of the ups
                    const int group0 = (ks * kStep) >> p.w.group_shift;
                    dst += kCodeBytes;
                    tma_load_3d<1>(dst, &p.scales, x.lane0, group0, x.g, bar);
                    tma_load_3d<1>(dst + kLanes * p.scale_parts, &p.scales, x.lane0 + (GATED ? p.w.n : kLanes / 2), group0,
                                   x.g, bar);
                }
                __syncwarp();
            }
        }
    } else if (warp == 3) {
        // ---- TMA: rows of x
        for (int t = t0; t < total && ok; t += t_step) {
            const Tile x = find_tile<CG>(p, sh, t, rank, walk);
            // of a pair each CTA holds half of the MMA's columns (the second's may hold no row in use:
            // then what lies there makes columns that nobody looks at)
            const int own = x.n_mma / CG, first = x.col0 + (CG == 2 ? (int)rank * own : 0);
            const bool any = first < x.col0 + x.cols;
            const CUtensorMap *map = &p.x[own / 16 - 1];
            for (int ks = lo; ks < hi; ++ks, ++issued, ring.next(p.x_slots)) {
                ok = warp_wait(&sh->x_empty[ring.s], ring.phase ^ 1, sh, p);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t *dst = xs + (size_t)ring.s * p.x_bytes;
                    const int subs = p.whole_lines ? kStep / 64 : min(kStep / 64, (p.w.k - ks * kStep + 63) / 64);
                    const uint32_t bytes = any ? subs * own * 128 : 0;
                    uint32_t bar;
                    if (CG == 2) {
                        bar = map_rank(&sh->x_full[ring.s], 0);
                        mbar_arrive_expect_tx_cluster(bar, bytes);
                    } else {
                        bar = smem_u32(&sh->x_full[ring.s]);
                        mbar_arrive_expect_tx(&sh->x_full[ring.s], bytes);
                    }
                    if (any) {
                        if (p.whole_lines)
                            tma_load_4d<CG>(dst, map, 0, first, ks * (kStep / 64), x.g, bar);
                        else
                            for (int i = 0; i < subs; ++i)
                                tma_load_3d<CG>(dst + i * own * 128, map, ks * kStep + i * 64, first, x.g, bar);
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        // ---- MMA: one thread waits and issues (by the whole warp, with a vote after each wait, a step of 128
        // took over 1100 cycles, whatever its columns)
        if ((CG == 1 || rank == 0) && elect_one()) {
            int acc = 0;
            uint32_t acc_phase = 0;
            Ring a_ring;
            const uint64_t base = smem_desc(smem_u32(xs), 16, 1024);
            for (int t = t0; t < total && ok; t += t_step) {
                const Tile x = find_tile<CG>(p, sh, t, rank, walk);
                const uint32_t idesc = mma_idesc(kLanes * CG, x.n_mma, false, false), d = tmem + acc * p.acc_stride;
                ok = role_wait(&sh->acc_empty[acc], ((acc_phase >> acc) & 1) ^ 1, sh, p);
                if (!ok) break;
                acc_phase ^= 1u << acc;
                const uint32_t line = x.n_mma / CG * 8;   // 64 elements of all rows, in 16 bytes
                for (int ks = lo; ks < hi; ++ks, ring.next(p.x_slots), a_ring.next(p.slots)) {
                    ok = role_wait(&sh->x_full[ring.s], ring.phase, sh, p) &&
                         role_wait(&sh->full[a_ring.s], a_ring.phase, sh, p);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t from = tmem + 2 * p.acc_stride + a_ring.s * kACols;
                    const uint64_t b = base + (uint32_t)(ring.s * p.x_bytes) / 16;
                    const int left = p.w.k - ks * kStep;
                    if (left >= kStep) {
#pragma unroll
                        for (int i = 0; i < kStep / 16; ++i)
                            mma_ts<CG>(d, from + i * 8, b + (i / 4) * line + (i % 4) * 2, idesc, i > 0 || ks > lo);
                    } else {
                        for (int i = 0; i * 16 < left; ++i)
                            mma_ts<CG>(d, from + i * 8, b + (i / 4) * line + (i % 4) * 2, idesc, i > 0 || ks > lo);
                    }
                    mma_commit<CG>(&sh->x_empty[ring.s]);
                    mma_commit<CG>(&sh->empty[a_ring.s]);
                }
                if (!ok) break;
                mma_commit<CG>(&sh->acc_full[acc]);
                acc ^= 1;
            }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < kFirstEpilogue) {
        // ---- codes to bf16, from shared to tensor memory; pairs of groups take turns. What tile a step
        // belongs to does not matter here, so a group goes from one of its steps straight to the next.
        const int turn = (warp - 4) / 8, half = (warp - 4) / 4 % 2, quad = warp % 4, row = quad * 32 + lane;
        const int tiles = t0 < total ? (total - t0 - 1) / t_step + 1 : 0;
        const long long steps = (long long)tiles * (hi - lo);
        // this lane's scales: of row 64 h + j, or gated of feature j, gate (h = 0) or up
        const int h = GATED ? (row >> 3) & 1 : row / 64, j = GATED ? (row >> 4) * 8 + (row & 7) : row % 64;
        const uint32_t scale_at = kCodeBytes + (h * (kLanes / 2) * p.scale_parts + j) * 2;
        const uint32_t row_at = row * 128, turned = (row & 7) << 4;   // (the 128-byte swizzle)
        const uint32_t to0 = tmem + 2 * p.acc_stride + half * (kACols / 2) + ((uint32_t)(quad * 32) << 16);
        ring.skip(turn, p.code_slots);
        Ring to_ring;
        to_ring.skip(turn, p.slots);
        for (long long b = turn; b < steps; b += kTurns, ring.skip(kTurns, p.code_slots), to_ring.skip(kTurns, p.slots)) {
            ok = warp_wait(&sh->code_full[ring.s], ring.phase, sh, p);
            if (!ok) break;
            const uint8_t *slot = cs + ring.s * kCodeSlot;
            const uint32_t to = to0 + to_ring.s * kACols;
            uint4 c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = *reinterpret_cast<const uint4 *>(slot + row_at + ((64 * half + 16 * i) ^ turned));
            __nv_bfloat16 raw[4];   // of 32 elements each
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[i] = *reinterpret_cast<const __nv_bfloat16 *>(
                    slot + scale_at + ((half * 4 + i) >> (p.w.group_shift - 5)) * kLanes);
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // 64 elements, 32 columns of tensor memory, at a time
                uint32_t r[32];
                const W4Scale<FP4> s0(raw[2 * i]), s1(raw[2 * i + 1]);
                if (__any_sync(kAll, is_large<FP4>(raw[2 * i]) || is_large<FP4>(raw[2 * i + 1]))) {
                    expand<FP4, true>(c[2 * i], s0, r);
                    expand<FP4, true>(c[2 * i + 1], s1, r + 16);
                } else {
                    expand<FP4, false>(c[2 * i], s0, r);
                    expand<FP4, false>(c[2 * i + 1], s1, r + 16);
                }
                if (i == 0) {   // (the slot's MMAs may take as long as the first part)
                    ok = warp_wait(&sh->empty[to_ring.s], to_ring.phase ^ 1, sh, p);
                    if (!ok) break;
                    tc_fence_after();
                }
                tmem_st32(to + i * 32, r);
            }
            if (!ok) break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh->code_empty[ring.s]);
                if (CG == 2) mbar_arrive_remote(map_rank(&sh->full[to_ring.s], 0));
                else mbar_arrive(&sh->full[to_ring.s]);
            }
        }
    } else if (warp >= kFirstEpilogue) {
        // ---- epilogue: 32 lanes and every other kChunk columns of each accumulator
        const int quad = warp % 4, half = (warp - kFirstEpilogue) / 4;
        int acc = 0;
        uint32_t acc_phase = 0;
        // accumulator a may be overwritten: this warp's part is in registers
        auto free_acc = [&](int a) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) mbar_arrive_cluster_relaxed(map_rank(&sh->acc_empty[a], 0));
                else mbar_arrive(&sh->acc_empty[a]);
            }
        };
        for (int t = t0; t < total && ok; t += t_step) {
            const Tile x = find_tile<CG>(p, sh, t, rank, walk);
            const float bias = bias_of<GATED>(p, x, quad, lane);
            const size_t row0 = (size_t)x.g * p.w.rows + x.col0;
            ok = warp_wait(&sh->acc_full[acc], (acc_phase >> acc) & 1, sh, p);
            if (!ok) break;
            acc_phase ^= 1u << acc;
            tc_fence_after();
            const uint32_t from = tmem + acc * p.acc_stride + ((uint32_t)(quad * 32) << 16);
            for (int c = half * kChunk; c < x.cols; c += 2 * kChunk) {
                uint32_t r[kChunk];
                float v[kChunk];
                tmem_ld16(from + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < kChunk; ++j) v[j] = __uint_as_float(r[j]);
                if (p.split > 1) {   // to shared memory, [column][lane]; joined below
                    float *part = reinterpret_cast<float *>(rings) + quad * 32 + lane;
#pragma unroll
                    for (int j = 0; j < kChunk; ++j)
                        if (c + j < x.cols) part[(c + j) * kLanes] = v[j];
                } else {
                    if (c + 2 * kChunk >= x.cols) free_acc(acc);
                    epilogue_chunk<GATED>(p, v, row0 + c, min(kChunk, x.cols - c), quad, lane, x.lane0, bias);
                }
            }
            if (p.split == 1 && half * kChunk >= x.cols) free_acc(acc);   // a warp with no columns here
            acc ^= 1;
        }
    }
    __syncthreads();
    // where a wait ran out, what is in flight is to finish (bounded) before shared and tensor
    // memory are given up
    if (sh->abort && warp == 1 && (CG == 1 || rank == 0) && elect_one()) drain_mma<CG>(sh);
    if (sh->abort && (threadIdx.x == 0 || threadIdx.x == 96)) {
        const uint64_t since = global_ns();
        const int slots = threadIdx.x == 0 ? p.code_slots : p.x_slots;
        uint64_t *full = threadIdx.x == 0 ? sh->code_full : sh->x_full;
        if (CG == 1 || threadIdx.x == 0)
            for (int i = max(0, issued - slots); i < issued; ++i)
                while (!mbar_try_wait(&full[i % slots], (uint32_t)(i / slots) & 1) && global_ns() - since < 100000000ull)
                    ;
        while (CG == 2 && global_ns() - since < 1000000ull)   // a pair's copies of x, whose barrier counts both CTAs'
            ;
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 1 && p.split > 1) {
        // ---- a shared tile: every CTA has its sums in shared memory; each adds up its share of
        // the columns, in rank order, and finishes them
        cluster_sync();
        if (t0 < total && warp >= kFirstEpilogue) {
            const int quad = warp % 4, half = (warp - kFirstEpilogue) / 4;
            walk = Walk();
            const Tile x = find_tile<CG>(p, sh, t0, rank, walk);
            const float bias = bias_of<GATED>(p, x, quad, lane);
            const size_t row0 = (size_t)x.g * p.w.rows + x.col0;
            const int share = (x.cols + p.split - 1) / p.split, c1 = min(x.cols, ((int)rank + 1) * share);
            for (int c = (int)rank * share + half * kChunk; c < c1; c += 2 * kChunk) {
                const int n = min(kChunk, c1 - c);
                float v[kChunk];
#pragma unroll
                for (int j = 0; j < kChunk; ++j) v[j] = 0.f;
                for (int i = 0; i < p.split; ++i) {
                    const uint32_t part = map_rank(reinterpret_cast<float *>(rings) + c * kLanes + quad * 32 + lane, i);
                    float got[kChunk];   // all loads on their way before the first is used
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) got[j] = j < n ? ld_cluster_f32(part + j * kLanes * 4) : 0.f;
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) v[j] += got[j];
                }
                epilogue_chunk<GATED>(p, v, row0 + c, n, quad, lane, x.lane0, bias);
            }
        }
        cluster_sync();   // no CTA leaves while another reads its shared memory
    }
    if (CG == 2) cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_free<CG>(tmem, kTmemCols);
}

constexpr long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Pairs of CTAs, where a tile for each pair fills the GPU.
bool plan_pairs(const W4Params &w, long long lane_tiles, int sms) {
    const long long pairs = ceil_div(lane_tiles, 2) * w.groups * ceil_div(w.rows, kColMax);
    return lane_tiles > 1 && 2 * pairs >= sms;
}

template <bool FP4, bool GATED, int CG>
cudaError_t launch(const TileParams &p, long long clusters, cudaStream_t st) {
    const auto kernel = &w4_tiles_kernel<FP4, GATED, CG>;
    const unsigned size = CG == 2 ? 2 : (unsigned)p.split;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void *>(kernel), kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)clusters * size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

int launch_w4_tiles(const W4Params &w, bool fp4, int32_t *status, cudaStream_t st) {
    const bool gated = w.act == EP_ACT_SWIGLU;
    TileParams p = {};
    p.w = w;
    p.status = status;
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) return EP_ERR_CUDA;
    p.wait_limit_ns = product_wait_limit();
    p.sleep_ns = p.wait_limit_ns < kSleepNs ? (uint32_t)p.wait_limit_ns : kSleepNs;
    p.lane_step = gated ? kLanes / 2 : kLanes;
    const long long single = ceil_div(w.n, p.lane_step);
    const int cg = plan_pairs(w, single, sms) ? 2 : 1, unit = 16 * cg;
    p.lane_tiles = (int)ceil_div(single, cg);
    p.col_max = w.rows < kColMax ? (int)ceil_div(w.rows, unit) * unit : kColMax;
    p.steps = (int)ceil_div(w.k, kStep);
    const long long most = (long long)p.lane_tiles * w.groups * ceil_div(w.rows, p.col_max);
    if (most >= (1LL << 30)) return EP_ERR_INVALID_ARG;   // tile numbers stay within int
    // dense products with few tiles share each one's reduction (clusters of four fill 144 SMs)
    p.split = 1;
    if (!w.counts && cg == 1)
        while (p.split < kMaxSplit && most * p.split * 2 <= sms - sms / 16 && p.steps >= 2 * p.split) p.split *= 2;
    p.x_bytes = p.col_max / cg * kStep * 2;
    p.scale_parts = kStep >> w.group_shift;
    p.acc_stride = (p.col_max + 31) / 32 * 32;
    p.slots = (kTmemCols - 2 * p.acc_stride) / kACols;   // 2 for 128 columns, 3 for 64
    // The rings: x waits in its own until the MMAs take it, codes only until they are expanded, up to
    // `slots` steps earlier, so x gets what four slots of codes leave. Slots of codes are a multiple of
    // kTurns: then a slot's uses are all of one pair of groups, and the parity that it waits for is not
    // that of an older phase. (With three, copies that arrive out of order let a pair see the phase before
    // the one of the other pair's step, read what was not there yet and upset the barriers' counts.)
    p.x_slots = (int)(kRingSpace - 4 * kCodeSlot) / p.x_bytes;
    if (p.x_slots > kMaxXSlots) p.x_slots = kMaxXSlots;
    p.code_slots = (int)(kRingSpace - (size_t)p.x_slots * p.x_bytes) / kCodeSlot / kTurns * kTurns;
    if (p.code_slots > kMaxCodeSlots) p.code_slots = kMaxCodeSlots;
    const uint64_t K = w.k, N = w.n, W = w.wide, G = w.groups, parts = K >> w.group_shift;
    bool good;
    if (gated) {
        // gate and up rows by turns of eight: 8 rows x (gate, up) x n / 8
        const uint64_t dims[5] = {K / 2, 8, 2, N / 8, G}, strides[4] = {K / 2, N * K / 2, 8 * K / 2, 2 * N * K / 2};
        const uint32_t box[5] = {kStep / 2, 8, 2, 8, 1};
        good = make_map(&p.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w.codes, 5, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
        const uint64_t dims[3] = {K / 2, N, G}, strides[2] = {K / 2, N * K / 2};
        const uint32_t box[3] = {kStep / 2, kLanes, 1};
        good = make_map(&p.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w.codes, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    const uint64_t sdims[3] = {W, parts, G}, sstrides[2] = {W, W * parts};
    const uint32_t sbox[3] = {kLanes / 2, (uint32_t)p.scale_parts, 1};
    good = good && make_map(&p.scales, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, w.scales, 3, sdims, sstrides, sbox,
                            CU_TENSOR_MAP_SWIZZLE_NONE);
    p.whole_lines = w.k % 64 == 0;
    for (int i = 0; good && i < p.col_max / cg / 16; ++i) {
        const uint32_t rows = 16u * (i + 1);
        if (p.whole_lines) {   // a step's lines of 64 elements, each with its rows
            const uint64_t dims[4] = {64, (uint64_t)w.rows, K / 64, G}, strides[3] = {K, 64, K * w.rows};
            const uint32_t box[4] = {64, rows, kStep / 64, 1};
            good = make_map(&p.x[i], w.x, 4, dims, strides, box);
        } else {
            good = make_map3(&p.x[i], w.x, K, w.rows, G, rows);
        }
    }
    if (!good) return EP_ERR_CUDA;
    const long long room = p.split > 1 ? most : sms / cg, clusters = most < room ? most : room;
    cudaError_t e;
    if (cg == 2)
        e = gated ? (fp4 ? launch<true, true, 2>(p, clusters, st) : launch<false, true, 2>(p, clusters, st))
                  : (fp4 ? launch<true, false, 2>(p, clusters, st) : launch<false, false, 2>(p, clusters, st));
    else
        e = gated ? (fp4 ? launch<true, true, 1>(p, clusters, st) : launch<false, true, 1>(p, clusters, st))
                  : (fp4 ? launch<true, false, 1>(p, clusters, st) : launch<false, false, 1>(p, clusters, st));
    return e == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

}  // namespace ep
