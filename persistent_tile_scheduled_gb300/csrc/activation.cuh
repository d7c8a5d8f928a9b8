// Activations and their derivatives, in fp32, and conversions of 16-bit rows.
//
// Both sigmoid forms are written as z / (1 + exp(-y)): 0.5 (1 + tanh(u)) equals
// 1 / (1 + exp(-2u)), and so keeps its relative precision where the tanh form
// cancels.  exp and the division are CUDA's fast ones (__expf, __fdividef: some
// 1e-6 of the value, far below a rounding to 16 bits).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace pts {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_SILU = 5, ACT_GATED = 0x10 };

constexpr float kSqrtHalf = 0.70710678f;         // sqrt(1 / 2)
constexpr float kGeluTanhTwice = 1.5957691f;     // 2 sqrt(2 / pi)
constexpr float kGeluTanhCube = 0.044715f;
constexpr float kNormalPeak = 0.39894228f;       // 1 / sqrt(2 pi)

template <int ACT>
__device__ __forceinline__ float act(float z)
{
    if constexpr (ACT == ACT_RELU) return fmaxf(z, 0.0f);
    if constexpr (ACT == ACT_RELU2) {
        const float p = fmaxf(z, 0.0f);
        return p * p;
    }
    if constexpr (ACT == ACT_GELU) return 0.5f * z * erfcf(-kSqrtHalf * z);
    if constexpr (ACT == ACT_GELU_TANH) return __fdividef(z, 1.0f + __expf(-kGeluTanhTwice * z * fmaf(kGeluTanhCube * z, z, 1.0f)));
    if constexpr (ACT == ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
    return z;
}

// act(z) and its derivative.
template <int ACT>
__device__ __forceinline__ float2 act_and_slope(float z)
{
    if constexpr (ACT == ACT_RELU) return make_float2(fmaxf(z, 0.0f), z > 0.0f ? 1.0f : 0.0f);
    if constexpr (ACT == ACT_RELU2) {
        const float p = fmaxf(z, 0.0f);
        return make_float2(p * p, 2.0f * p);
    }
    if constexpr (ACT == ACT_GELU) {
        const float p = 0.5f * erfcf(-kSqrtHalf * z);
        return make_float2(z * p, fmaf(kNormalPeak * z, __expf(-0.5f * z * z), p));
    }
    if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        // z s(y): s + z s (1 - s) y', with 1 - s = exp(-y) s
        float y = z, dy = 1.0f;
        if constexpr (ACT == ACT_GELU_TANH) {
            y = kGeluTanhTwice * z * fmaf(kGeluTanhCube * z, z, 1.0f);
            dy = kGeluTanhTwice * fmaf(3.0f * kGeluTanhCube * z, z, 1.0f);
        }
        // (exp(-y) is kept finite: below s = exp(-80) the slope is 0 to any precision kept)
        const float e = __expf(fminf(-y, 80.0f)), s = __fdividef(1.0f, 1.0f + e);
        return make_float2(z * s, fmaf(z * dy * s, e * s, s));
    }
    return make_float2(z, 1.0f);
}

// f(std::integral_constant-like tag) with the activation as a constant.
template <int V>
struct ActTag {
    static constexpr int value = V;
};

template <class F>
__device__ __forceinline__ void with_act(int a, F f)
{
    switch (a & ~ACT_GATED) {
    case ACT_RELU: f(ActTag<ACT_RELU>()); break;
    case ACT_RELU2: f(ActTag<ACT_RELU2>()); break;
    case ACT_GELU: f(ActTag<ACT_GELU>()); break;
    case ACT_GELU_TANH: f(ActTag<ACT_GELU_TANH>()); break;
    case ACT_SILU: f(ActTag<ACT_SILU>()); break;
    default: f(ActTag<ACT_NONE>()); break;
    }
}

// ---- 16-bit values (KIND 0 fp16, else bf16) -------------------------------------

template <int KIND>
__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if constexpr (KIND == 0) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}

template <int KIND>
__device__ __forceinline__ uint32_t pack2f(float lo, float hi)
{
    if constexpr (KIND == 0) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int KIND>
__device__ __forceinline__ float unpack1(uint32_t bits16)
{
    return unpack2<KIND>(bits16).x;
}

}  // namespace pts
