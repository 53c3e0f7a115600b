// w4.cuh -- products with 4-bit weights: parameters and the codes' values, shared by the
// kernel for few rows (w4_rows.cu) and the one for many (w4_tiles.cu).
//
// A weight's row holds its codes in words of eight: the four low fields of 4 bits are elements
// 0, 2, 4, 6 and the four high ones 1, 3, 5, 7, so that a mask of one shift of the word leaves
// two neighbours in the halves of a register, ready to become a pair of bf16. The weight is
// w = bf16(value * scale), rounded once: exactly the bf16 weight that ep_product would be given
// for it, and what an MMA takes. Scales lie [k / group][rows of the weight], so that the
// scales of neighbouring rows are side by side.
#pragma once

#include <cuda_bf16.h>

#include "launch.cuh"

namespace ep {

struct W4Params {
    const __nv_bfloat16 *x;
    const uint8_t *codes;
    const __nv_bfloat16 *scales, *bias, *residual;
    __nv_bfloat16 *out;
    const int32_t *counts;
    int groups, rows, k, n;
    int wide;         // rows of a weight: n, or 2 n where gated
    int group_shift;  // log2 of the elements of a scale
    int act;
};

// Two rows' scale in both halves.
__device__ __forceinline__ __nv_bfloat162 bf162_of(uint32_t v) { return *reinterpret_cast<__nv_bfloat162 *>(&v); }
__device__ __forceinline__ uint32_t u32_of(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t *>(&v); }

// (a & b) ^ c and (a & b) | c as one instruction
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// A scale in both halves of a register. fp4 codes read as value * 2^-126 (below), so their scale
// carries 2^126, which is exact and saves a product; a scale of 4 and more would overflow
// (`large`) and takes that product.
template <bool FP4>
struct W4Scale {
    __nv_bfloat162 v;
    __device__ __forceinline__ W4Scale() : v(bf162_of(0)) {}
    __device__ __forceinline__ explicit W4Scale(__nv_bfloat16 scale) : v(__bfloat162bfloat162(scale)) {}
    __device__ __forceinline__ bool large() const { return (u32_of(v) & 0x7FFFu) >= 0x4080u; }   // |scale| >= 4, or NaN
};

// The eight weights of a word, in order, as four pairs.
//   int4 (two's complement): a field with its top bit turned is value + 8; under the exponent
//     of 128 it reads 136 + value.
//   fp4 (sign, two bits of exponent, one of mantissa): moved to bf16's sign, the low end of its
//     exponent and the top of its mantissa, it reads value * 2^-126, subnormals included.
// All steps but the scale's product are exact, so a weight is rounded once.
template <bool FP4, bool LARGE>
__device__ __forceinline__ void w4_values(uint32_t word, const W4Scale<FP4> &scale, uint32_t (&pair)[4]) {
    if (FP4) {
        const uint32_t s[4] = {word << 12, word << 8, word << 4, word};
        const uint32_t m[4] = {word << 6, word << 2, word >> 2, word >> 6};
        const __nv_bfloat162 up = bf162_of(0x7E807E80u);   // 2^126
        const __nv_bfloat162 by = LARGE ? scale.v : __hmul2(scale.v, up);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = bf162_of(and_or(s[j], 0x80008000u, m[j] & 0x01C001C0u));
            pair[j] = u32_of(__hmul2(LARGE ? __hmul2(v, up) : v, by));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = and_xor(word >> (4 * j), 0x000F000Fu, 0x43084308u);
            pair[j] = u32_of(__hmul2(__hsub2(bf162_of(v), bf162_of(0x43084308u)), scale.v));   // 136
        }
    }
}

cudaError_t launch_w4_rows(const W4Params &p, bool fp4, cudaStream_t st);
int launch_w4_tiles(const W4Params &p, bool fp4, int32_t *status, cudaStream_t st);

}  // namespace ep
