// product.cuh -- parameters of the tensor-core products (product.cu).
#pragma once

#include <cuda_bf16.h>

#include "tcgen05.cuh"

namespace ep {

enum ProductMode { PRODUCT_FORWARD = 0, PRODUCT_DGRAD = 1, PRODUCT_WGRAD = 2 };

constexpr int kBoxes = 8;   // token-row boxes of the column operand: 16, 32, ..., 128 rows

// One product, seen by the kernel as D[col][lane] = sum_r A[lane][r] B[col][r]:
//   forward  lanes = output features n, columns = tokens, r = k
//   dgrad    lanes = input features k,  columns = tokens, r = n
//   wgrad    lanes = k, columns = n, r = tokens in use
struct ProductParams {
    CUtensorMap a;            // lane operand
    CUtensorMap b[kBoxes];    // column operand (wgrad: b[0] only)
    CUtensorMap o;            // output as {lanes, halves, rows, groups}, boxes of 32 lanes x 32 rows
    const int32_t *counts;    // rows in use per group, or null (= rows)
    int groups, rows;
    int lanes;                // output features (gated forward: of the activation's output)
    int cols;                 // wgrad: n
    int red;                  // forward: k, dgrad: n (wgrad: the group's rows in use)
    int lane_tiles, col_max;  // lane tiles per group; widest column tile
    int lane_step;            // output features of a CTA's lane tile
    int a_bytes;              // a sub-block of its lane operand
    int stages, stage_bytes;  // ring of operand blocks in shared memory,
    int subs, sub_bytes;      // each of this many sub-blocks of 64 reduction elements
    int block_red, block_shift;   // subs * 64, and its logarithm
    int chain;                // blocks summed in one accumulator, at most (see Sums)
    int out_at;               // offset of the epilogue warps' output tiles, after the stages
    int split;                // CTAs of a cluster that share one tile's reduction (1 = none)
    int act, interleave;      // gated forward: 8 or 16 gate rows, then as many up rows
    int out_f32, accumulate;
    const __nv_bfloat16 *bias, *residual;
    const __nv_bfloat16 *z;   // dgrad: pre-activation of the product's input
    __nv_bfloat16 *preact;    // forward: pre-activation kept for the backward pass
    void *out;
    int32_t *status;          // or null (= the device's own word)
    uint64_t wait_limit_ns;
    uint32_t sleep_ns;        // of one attempt at a wait
};

}  // namespace ep
