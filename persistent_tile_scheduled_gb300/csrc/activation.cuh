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

// g = t (kTail[0] + t (kTail[1] + ...))
__device__ constexpr float kTail[7] = {0.14371697f, 0.14171756f, 0.14001835f, 0.025731557f, 0.18214381f, -0.18064261f, 0.047314238f};

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
    float g = fmaf(kTail[6], t, kTail[5]);
#pragma unroll
    for (int i = 4; i >= 0; --i) g = fmaf(g, t, kTail[i]);
    return g * t * e;
}

// max(z, 0), and NaN for NaN
__device__ __forceinline__ float positive(float z) { return z <= 0.0f ? 0.0f : z; }

// max(z, lo), and NaN for NaN
__device__ __forceinline__ float at_least(float z, float lo)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(z), "f"(lo));
    return y;
}

// min(z, hi), and NaN for NaN
__device__ __forceinline__ float at_most(float z, float hi)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(z), "f"(hi));
    return y;
}

// silu and the tanh form of gelu of anything below this are less than 2^-54 away from 0:
// there z counts as this, -infinity too, since the factor that it meets stops falling.
constexpr float kLowest = -44.0f;

// From here on the slopes of gelu, its tanh form and silu are 1 to within 2^-86: there z counts
// as this in them, infinity too (it meets a 0, and so did a large z whose product overflowed).
constexpr float kHighest = 64.0f;

template <int ACT>
__device__ __forceinline__ float act(float z)
{
    if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) z = at_least(z, kLowest);
    if constexpr (ACT == ACT_RELU) return positive(z);
    if constexpr (ACT == ACT_RELU2) return positive(z) * positive(z);
    // z Phi(z): z - z Phi(-z) above 0 (the factor of the tail, 0 from 14 on, is kept finite)
    if constexpr (ACT == ACT_GELU) return fmaf(-fminf(fabsf(z), 16.0f), normal_tail(z, normal_exp(z)), positive(z));
    if constexpr (ACT == ACT_GELU_TANH)
        return z * rcp_fast(1.0f + exp2_fast(z * fmaf(-kLog2E * kGeluTanhTwice * kGeluTanhCube * z, z, -kLog2E * kGeluTanhTwice)));
    if constexpr (ACT == ACT_SILU) return z * rcp_fast(1.0f + exp2_fast(-kLog2E * z));
    return z;
}

// Two values side by side: one instruction computes both (PTX's f32x2 forms).
struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair pair(float x, float y)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ Pair pair(float2 f) { return pair(f.x, f.y); }
__device__ __forceinline__ Pair both(float x) { return pair(x, x); }
__device__ __forceinline__ float2 values(Pair p)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
    return f;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b)
{
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
    return p;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    Pair p;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
    return p;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c)
{
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return p;
}
template <class F>
__device__ __forceinline__ Pair each(Pair p, F f)
{
    const float2 v = values(p);
    return pair(f(v.x), f(v.y));
}

// 1 / a of two values of 1 to 2^61 by one reciprocal: the unit of approximate functions
// takes 8 cycles a warp, and bounds an epilogue that needs two of them per value.
__device__ __forceinline__ Pair rcp_fast(Pair a)
{
    const float2 v = values(a);
    const float r = rcp_fast(v.x * v.y);
    return both(r) * pair(v.y, v.x);
}

// exp(-z^2 / 2) and Phi(-|z|)
__device__ __forceinline__ void normal_tail(Pair z, Pair &e, Pair &q)
{
    e = each(z * z * both(-0.5f * kLog2E), [](float v) { return exp2_fast(v); });
    const Pair t = rcp_fast(fma(both(0.36f), each(z, [](float v) { return fminf(fabsf(v), 16.0f); }), both(1.0f)));
    Pair g = fma(both(kTail[6]), t, both(kTail[5]));
#pragma unroll
    for (int i = 4; i >= 0; --i) g = fma(g, t, both(kTail[i]));
    q = g * t * e;
}

__device__ __forceinline__ Pair at_least(Pair z, float lo)
{
    return each(z, [=](float v) { return at_least(v, lo); });
}

__device__ __forceinline__ Pair at_most(Pair z, float hi)
{
    return each(z, [=](float v) { return at_most(v, hi); });
}

// 2^y, y at most 60: 1 / (1 + 2^60), of kLowest at most, is next to nothing, and two of
// them have a product (a NaN is taken for 60: it comes back with z, and not into the other value)
__device__ __forceinline__ Pair exp2_limited(Pair y)
{
    return each(y, [](float v) { return exp2_fast(fminf(v, 60.0f)); });
}

template <int ACT>
__device__ __forceinline__ Pair act(Pair z)
{
    if constexpr (ACT == ACT_RELU) return each(z, [](float v) { return positive(v); });
    if constexpr (ACT == ACT_RELU2) {
        const Pair p = each(z, [](float v) { return positive(v); });
        return p * p;
    }
    if constexpr (ACT == ACT_GELU) {
        Pair e, q;
        normal_tail(z, e, q);
        return fma(each(z, [](float v) { return -fminf(fabsf(v), 16.0f); }), q, each(z, [](float v) { return positive(v); }));
    }
    if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        Pair y = z * both(-kLog2E);
        if constexpr (ACT == ACT_GELU_TANH) y = z * fma(both(-kLog2E * kGeluTanhTwice * kGeluTanhCube) * z, z, both(-kLog2E * kGeluTanhTwice));
        return at_least(z, kLowest) * rcp_fast(exp2_limited(y) + both(1.0f));
    }
    return z;
}

// act(z) and its derivative, of two values.
template <int ACT>
__device__ __forceinline__ void act_and_slope(Pair z, Pair &a, Pair &slope)
{
    if constexpr (ACT == ACT_RELU) {
        a = each(z, [](float v) { return positive(v); });
        slope = each(z, [](float v) { return v > 0.0f ? 1.0f : positive(v); });   // (0, or NaN)
    } else if constexpr (ACT == ACT_RELU2) {
        const Pair p = each(z, [](float v) { return positive(v); });
        a = p * p;
        slope = p + p;
    } else if constexpr (ACT == ACT_GELU) {
        // Phi(z) = q below 0, 1 - q above; Phi + z phi(z)
        z = at_least(z, -16.0f);   // (e is 0 there; -infinity times it would not be)
        Pair e, tail;
        normal_tail(z, e, tail);
        const float2 q = values(tail), v = values(z);
        const Pair p = pair(v.x > 0.0f ? 1.0f - q.x : q.x, v.y > 0.0f ? 1.0f - q.y : q.y);
        a = z * p;
        slope = fma(at_most(z, kHighest) * both(kNormalPeak), e, p);
    } else if constexpr (ACT == ACT_GELU_TANH || ACT == ACT_SILU) {
        // z s(y), s = 1 / (1 + exp(-y)): s + z s (1 - s) y', with 1 - s = exp(-y) s
        z = at_least(z, kLowest);
        const Pair x = at_most(z, kHighest);
        Pair y, dy;   // (y: the exponent of 2)
        if constexpr (ACT == ACT_GELU_TANH) {
            const Pair x2 = x * x;
            y = x * fma(both(-kLog2E * kGeluTanhTwice * kGeluTanhCube), x2, both(-kLog2E * kGeluTanhTwice));
            dy = x * fma(both(3.0f * kGeluTanhTwice * kGeluTanhCube), x2, both(kGeluTanhTwice));
        } else {
            y = x * both(-kLog2E);
            dy = x;
        }
        const Pair e = exp2_limited(y), s = rcp_fast(e + both(1.0f));
        a = z * s;
        slope = fma(dy * s, e * s, s);
    } else {
        a = z;
        slope = both(1.0f);
    }
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
