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

// A group's scale, in both halves of a register each time. A masked field is a subnormal bf16
// (below), so the scale carries the power of two that makes up for it; where that would overflow
// (is_large: rare for a weight) the values are brought up first, in a product
// more each.
//   int4: by = scale * 2^133, by16 = scale * 2^129, off = -8 scale, for scales below 2^-5
//   fp4:  by = scale * 2^126, for scales below 4
template <bool FP4>
struct W4Scale {
    __nv_bfloat162 scale, by, by16, off;
    __device__ __forceinline__ W4Scale() : scale(bf162_of(0)), by(bf162_of(0)), by16(bf162_of(0)), off(bf162_of(0)) {}
    __device__ __forceinline__ explicit W4Scale(__nv_bfloat16 s) : scale(__bfloat162bfloat162(s)) {
        if (FP4) {
            by = __hmul2(scale, bf162_of(0x7E807E80u));                       // 2^126
        } else {
            by16 = __hmul2(__hmul2(scale, bf162_of(0x7E807E80u)), bf162_of(0x41004100u));   // 2^3 more
            by = __hmul2(by16, bf162_of(0x41804180u));                        // 2^4 more
            off = __hmul2(scale, bf162_of(0xC100C100u));                      // -8
        }
    }
};

// Whether a scale is too large for the powers above, infinite or NaN.
template <bool FP4>
__device__ __forceinline__ bool is_large(__nv_bfloat16 scale) {
    return (__bfloat16_as_ushort(scale) & 0x7FFFu) >= (FP4 ? 0x4080u : 0x3D00u);   // 4, 2^-5
}

// The eight weights of a word, in order, as four pairs. All steps but the last are exact, so a
// weight is rounded once, from value * scale.
//   int4 (two's complement): a field with its top bit turned is u = value + 8. Bits 0-7 of a bf16
//     read as an integer times 2^-133 (its subnormals and their first normal binade), so a field there
//     is u 2^-133 or 16 u 2^-133 as it stands, and one fused product-sum makes u scale - 8 scale of it.
//   fp4 (sign, two bits of exponent, one of mantissa): at the low end of bf16's exponent and the top
//     of its mantissa a code reads value * 2^-126, subnormals included. One product by 2^6 + 2^12 brings
//     a field there and its sign to the top.
template <bool FP4, bool LARGE>
__device__ __forceinline__ void w4_values(uint32_t word, const W4Scale<FP4> &s, uint32_t (&pair)[4]) {
    const uint32_t w[2] = {word, word >> 8};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t field = (j & 1) ? 0x00F000F0u : 0x000F000Fu;
        if (FP4) {
            const __nv_bfloat162 v = bf162_of(((w[j / 2] & field) * ((j & 1) ? 0x104u : 0x1040u)) & 0x81C081C0u);
            pair[j] = u32_of(LARGE ? __hmul2(__hmul2(v, bf162_of(0x7E807E80u)), s.scale) : __hmul2(v, s.by));
        } else if (LARGE) {
            // under the exponent of 128 the field reads 136 + value
            const __nv_bfloat162 v = bf162_of(and_xor(word >> (4 * j), 0x000F000Fu, 0x43084308u));
            pair[j] = u32_of(__hmul2(__hsub2(v, bf162_of(0x43084308u)), s.scale));
        } else {
            const __nv_bfloat162 v = bf162_of(and_xor(w[j / 2], field, field & 0x00880088u));
            pair[j] = u32_of(__hfma2(v, (j & 1) ? s.by16 : s.by, s.off));
        }
    }
}

cudaError_t launch_w4_rows(const W4Params &p, bool fp4, int32_t *status, cudaStream_t st);
int launch_w4_tiles(const W4Params &p, bool fp4, int32_t *status, cudaStream_t st);

}  // namespace ep
