// act.cuh -- the activations of the products' epilogues and their derivatives,
// in fp32. The exponential and division are CUDA's fast forms (a few units in
// the last place of fp32), far below the rounding of the bf16 they end in.
#pragma once

#include <cuda_bf16.h>

#include "ep_internal.cuh"

namespace ep {

__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// tanh through one exponential: 1 - 2 / (1 + e^(2u)); the absolute error of a
// few 2^-24 is what counts, as it is used as 1 + t.
__device__ __forceinline__ float tanh_f(float u) { return 1.f - __fdividef(2.f, 1.f + __expf(2.f * u)); }

constexpr float kSqrtHalf = 0.70710678118654752f;     // sqrt(1/2)
constexpr float kSqrt2OverPi = 0.79788456080286536f;  // sqrt(2/pi)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;   // 1/sqrt(2 pi)
constexpr float kGeluCubic = 0.044715f;

// act(z) of the elementwise activations.
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case EP_ACT_RELU: return z < 0.f ? 0.f : z;   // NaN stays NaN
        case EP_ACT_SILU: return __fdividef(z, 1.f + __expf(-z));
        case EP_ACT_GELU: return 0.5f * z * (1.f + erff(z * kSqrtHalf));
        case EP_ACT_GELU_TANH:
            return 0.5f * z * (1.f + tanh_f(kSqrt2OverPi * (z + kGeluCubic * z * z * z)));
        default: return z;
    }
}

// d act(z) / dz of the elementwise activations (0 at z = 0 for relu).
__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case EP_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case EP_ACT_SILU: {
            const float s = sigmoid_f(z);
            return s * (1.f + z * (1.f - s));
        }
        case EP_ACT_GELU:
            return 0.5f * (1.f + erff(z * kSqrtHalf)) + z * kInvSqrt2Pi * __expf(-0.5f * z * z);
        case EP_ACT_GELU_TANH: {
            const float t = tanh_f(kSqrt2OverPi * (z + kGeluCubic * z * z * z));
            return 0.5f * (1.f + t) +
                   0.5f * z * (1.f - t * t) * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
        }
        default: return 1.f;
    }
}

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace ep
