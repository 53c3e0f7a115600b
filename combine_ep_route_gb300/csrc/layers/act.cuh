// act.cuh -- the activations of the products' epilogues and their derivatives,
// in fp32. Exponentials and reciprocals are the hardware's approximations (PTX
// ex2.approx and rcp.approx, a unit or two in the last place of fp32), since an
// epilogue has about as many cycles as its instructions need. Values and slopes are
// right to about (16 + 6 a) 2^-24 of themselves, where e^a is the exponential taken (a up
// to 87 before a tail underflows: at worst 3.2e-5, where half a unit of bf16 is 2e-3 or more);
// a slope near its zero, to that share of its terms.
#pragma once

#include <cuda_bf16.h>

#include "launch.cuh"

namespace ep {

__device__ __forceinline__ float exp2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_f(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f(float z) { return rcp_f(1.f + exp2_f(-kLog2E * z)); }

constexpr float kSqrt2OverPi = 0.79788456080286536f;  // sqrt(2/pi)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;   // 1/sqrt(2 pi)
constexpr float kGeluCubic = 0.044715f;

// gelu_tanh's factor (1 + tanh u) / 2, u = sqrt(2/pi) (z + c z^3), as the sigmoid of 2u: the
// same function, but 1 + tanh u cancels below z = -3 (4 % off at -4.5, nothing left at -5),
// and the sigmoid keeps its relative precision down to the smallest floats. z2 = z * z.
__device__ __forceinline__ float gelu_tanh_factor(float z, float z2) {
    return rcp_f(1.f + exp2_f(-2.f * kLog2E * kSqrt2OverPi * z * fmaf(kGeluCubic, z2, 1.f)));
}

// Phi(z), the normal distribution's, and its density's exponential e^(-z^2 / 2). The tail
// Phi(-|z|) is that exponential times Mills' ratio over sqrt(2 pi), which falls slowly and is
// a polynomial in t = 1 / (1 + p |z|) to 1.1e-7 of itself on [0, 15] (minimax in the relative
// error, fitted to scipy's erfcx; 3.8e-7 with fp32 roundings). So a tail is as precise, relative to itself, as
// its exponential, whose argument's rounding grows with z^2 / 2. A value and a slope share
// the exponential. erff and a separate one made the epilogue of a gradient through gelu
// take longer than the product (18 against 16 thousand cycles for a tile of 2048 terms).
__device__ __forceinline__ float normal_cdf(float z, float &density_exp) {
    const float t = rcp_f(fmaf(0.305f, fabsf(z), 1.f));
    const float e = exp2_f(-0.5f * kLog2E * z * z);
    float q = 0.036427464f;
    q = fmaf(q, t, -0.15189704f);
    q = fmaf(q, t, 0.18390650f);
    q = fmaf(q, t, -0.036374345f);
    q = fmaf(q, t, 0.12020738f);
    q = fmaf(q, t, 0.10365756f);
    q = fmaf(q, t, 0.12243050f);
    q = fmaf(q, t, 0.12164200f);
    const float tail = q * t * e;
    density_exp = e;
    return z < 0.f ? tail : 1.f - tail;
}

// act(z) of the elementwise activations.
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case EP_ACT_RELU: return z < 0.f ? 0.f : z;   // NaN stays NaN
        case EP_ACT_SILU: return z * sigmoid_f(z);
        case EP_ACT_GELU: {
            float e;
            return z * normal_cdf(z, e);
        }
        case EP_ACT_GELU_TANH: return z * gelu_tanh_factor(z, z * z);
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
        case EP_ACT_GELU: {
            float e;
            const float cdf = normal_cdf(z, e);
            return cdf + z * kInvSqrt2Pi * e;
        }
        case EP_ACT_GELU_TANH: {
            // s + z s (1 - s) 2u'. Past |z| = 16 the factor is 0 or 1 to the last digit; z * z
            // stops there, so that no infinity meets s (1 - s) = 0.
            const float z2 = fminf(z * z, 256.f), s = gelu_tanh_factor(z, z2);
            return fmaf(z * (s * (1.f - s)), 2.f * kSqrt2OverPi * fmaf(3.f * kGeluCubic, z2, 1.f), s);
        }
        default: return 1.f;
    }
}

// Of y = silu(gate) * up, given dy: the gradients of gate and up.
__device__ __forceinline__ void swiglu_grad(float dy, float gate, float up, float &dgate, float &dup) {
    const float s = sigmoid_f(gate), v = gate * s;
    dup = dy * v;
    dgate = dy * up * (s + v * (1.f - s));
}

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace ep
