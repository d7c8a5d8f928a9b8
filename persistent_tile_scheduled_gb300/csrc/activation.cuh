// Activations and their derivatives, in fp32, and conversions of 16-bit rows.
//
// silu and the tanh form of gelu are z / (1 + exp(-y)): 0.5 (1 + tanh(u)) equals
// 1 / (1 + exp(-2u)), and so keeps its relative precision where the tanh form
// cancels.  gelu's Phi(-a) = exp(-a^2 / 2) g(a), a = |z|, with g = erfcx(a /
// sqrt 2) / 2, which falls slowly and is taken as a polynomial without constant
// term in t = 1 / (1 + 0.36 a), fitted here to the least relative error over 0 <=
// a <= 13.5 (a linear program over 4000 Chebyshev points; off by 1.1e-6 of it in
// fp32, behind 13.5 the exponential is 0).  With CUDA's erfcf instead, 4101 rows
// of 4224 x 4096 with bias, gelu and residual took 131 us where this takes 98.
// 2^x and 1 / x are the approximate instructions (off by 2^-22 of the value; of
// exp(-y) the argument's rounding adds 2^-24 |y|): far below a rounding to 16 bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace pts {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_SILU = 5, ACT_GATED = 0x10 };

constexpr float kLog2E = 1.44269504f;
constexpr float kGeluTanhTwice = 1.5957691f;     // 2 sqrt(2 / pi)
constexpr float kGeluTanhCube = 0.044715f;
constexpr float kNormalPeak = 0.39894228f;       // 1 / sqrt(2 pi)

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(-z^2 / 2), and Phi(-|z|) from it
__device__ __forceinline__ float normal_exp(float z) { return exp2_fast(-0.5f * kLog2E * z * z); }

__device__ __forceinline__ float normal_tail(float z, float e)
{
    const float t = rcp_fast(fmaf(0.36f, fabsf(z), 1.0f));
    float g = 0.047314238f;
    g = fmaf(g, t, -0.18064261f);
    g = fmaf(g, t, 0.18214381f);
    g = fmaf(g, t, 0.025731557f);
    g = fmaf(g, t, 0.14001835f);
    g = fmaf(g, t, 0.14171756f);
    g = fmaf(g, t, 0.14371697f);
    return g * t * e;
}

// max(z, 0), and NaN for NaN
__device__ __forceinline__ float positive(float z) { return z <= 0.0f ? 0.0f : z; }

template <int ACT>
__device__ __forceinline__ float act(float z)
{
    if constexpr (ACT == ACT_RELU) return positive(z);
    if constexpr (ACT == ACT_RELU2) return positive(z) * positive(z);
    // z Phi(z): z - z Phi(-z) above 0 (the factor of the tail, 0 from 14 on, is kept finite)
    if constexpr (ACT == ACT_GELU) return fmaf(-fminf(fabsf(z), 16.0f), normal_tail(z, normal_exp(z)), positive(z));
    if constexpr (ACT == ACT_GELU_TANH)
        return z * rcp_fast(1.0f + exp2_fast(z * fmaf(-kLog2E * kGeluTanhTwice * kGeluTanhCube * z, z, -kLog2E * kGeluTanhTwice)));
    if constexpr (ACT == ACT_SILU) return z * rcp_fast(1.0f + exp2_fast(-kLog2E * z));
    return z;
}

// act(z) and its derivative.
template <int ACT>
__device__ __forceinline__ float2 act_and_slope(float z)
{
    if constexpr (ACT == ACT_RELU) return make_float2(positive(z), z > 0.0f ? 1.0f : 0.0f);
    if constexpr (ACT == ACT_RELU2) return make_float2(positive(z) * positive(z), 2.0f * positive(z));
    if constexpr (ACT == ACT_GELU) {
        const float e = normal_exp(z), q = normal_tail(z, e), p = z > 0.0f ? 1.0f - q : q;
        return make_float2(z * p, fmaf(kNormalPeak * z, e, p));
    }
    if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        // z s(y), s = 1 / (1 + exp(-y)): s + z s (1 - s) y', with 1 - s = exp(-y) s
        float y = -kLog2E * z, dy = 1.0f;   // (y: the exponent of 2)
        if constexpr (ACT == ACT_GELU_TANH) {
            const float z2 = fminf(z * z, 4096.0f);   // (dy stays finite; there the slope is 0 or 1)
            y = z * fmaf(-kLog2E * kGeluTanhTwice * kGeluTanhCube, z2, -kLog2E * kGeluTanhTwice);
            dy = fmaf(3.0f * kGeluTanhTwice * kGeluTanhCube, z2, kGeluTanhTwice);
        }
        // (exp(-y) is kept finite: there s and the slope are 2^-110 and less)
        const float e = exp2_fast(fminf(y, 110.0f)), s = rcp_fast(1.0f + e);
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
