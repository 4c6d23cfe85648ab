// Activations and their slopes for the linear layers' epilogues (part of library.hip).
#pragma once

namespace {

// An activation a(z) and its slope a'(z) as value * f^3 and slope * f^3.  f is 1,
// except where a and a' are too small for fp32 (very negative z): then it is the
// third root of what they hold of an exponential, a normal number, and each factor
// beside the activation takes an f first, so that a large one meets a small one
// before anything overflows or is lost.
struct Activated {
    float f, value, slope;

    __device__ __forceinline__ float times(float x) const { return (x * f) * (value * f) * f; }
    // x y alone may overflow beside a small slope, y times a slope be lost beside a large x.
    __device__ __forceinline__ float slope_times(float x, float y) const
    {
        const float xf = x * f, yf = y * f, sf = slope * f;
        return f > 0.01f ? xf * (yf * sf) : xf * yf * sf;
    }
    __device__ __forceinline__ float slope_times(float x) const { return (x * f) * (slope * f) * f; }
};

// z times the logistic function of v(z), with z v'(z) for the slope: silu (v = z)
// and gelu's usual approximation (v = z (a + b z^2)).  Where s(v) is exp(v) to
// fp32, it is f^3 (low_gate).
template <bool SLOPE>
__device__ __forceinline__ Activated z_logistic(float z, float v, float zdv)
{
    if (v < (SLOPE ? kLowGateGrad : kLowGate)) {
        const LowGate l = low_gate(v);
        // Minus infinity times zero: NaN, as the formula has it.
        return {l.f, z == -__builtin_inff() ? __builtin_nanf("") : z, 1.0f + zdv};
    }
    if constexpr (SLOPE) {
        const Sigmoid s = sigmoid(v);
        return {1.0f, z * s.s, s.s * __builtin_fmaf(zdv, s.c, 1.0f)};
    }
    return {1.0f, logistic_times(v, z), 0.0f};
}

// z times the normal distribution function Phi(z).  With a = |z| the tail is
//
//   Phi(-a) = h(a) exp(-a^2 / 2),   h(a) = exp(a^2 / 2) erfc(a / sqrt 2) / 2
//
// and h a polynomial in t = 1 / (1 + 0.275 a), fitted by weighted least squares for
// the smallest relative error over 0 <= a <= 60 (2.5e-6 in fp32, a thousandth of
// bf16's step).  exp(-a^2 / 2) is f^3.  The slope is Phi(z) + z phi(z), phi the
// density exp(-a^2 / 2) / sqrt(2 pi).
template <bool SLOPE>
__device__ __forceinline__ Activated z_normal(float z)
{
    constexpr float kThird = 0x1.ec709ep-3f;   // log2(e) / 6
    constexpr float kDensity = 0.398942280f;   // 1 / sqrt(2 pi)
    const float a = __builtin_fabsf(z) > 40.0f ? 40.0f : __builtin_fabsf(z);   // keeps NaN
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.275f, a, 1.0f));
    float h = -0.0551880188f;
    h = __builtin_fmaf(h, t, 0.129638717f);
    h = __builtin_fmaf(h, t, 0.00414652424f);
    h = __builtin_fmaf(h, t, 0.103499249f);
    h = __builtin_fmaf(h, t, 0.0982339233f);
    h = __builtin_fmaf(h, t, 0.109967098f);
    h = __builtin_fmaf(h, t, 0.109701574f);
    h *= t;
    const float f = __builtin_amdgcn_exp2f(-kThird * (a * a));
    const float bump = __builtin_fmaf(-kDensity, a, h);   // the slope's tail over f^3
    if (z <= 0.0f)
        return {f, z == -__builtin_inff() ? __builtin_nanf("") : z * h, bump};
    const float f3 = f * f * f;
    return {1.0f, __builtin_fmaf(-z * f3, h, z), __builtin_fmaf(-f3, bump, 1.0f)};
}

// Activation `act` (uniform), with its slope where SLOPE.
template <bool SLOPE>
__device__ __forceinline__ Activated activated(int act, float z)
{
    if (act == GEMM_ACT_SILU)
        return z_logistic<SLOPE>(z, z, z);
    if (act == GEMM_ACT_GELU_TANH) {
        constexpr float kA = 1.59576912f, kB = 0.0713548163f;   // 2 sqrt(2 / pi), that times 0.044715
        // Past 30 the logistic function is 0 or 1 and z^3 may overflow.
        const float c = z > 30.0f ? 30.0f : z < -30.0f ? -30.0f : z, c2 = c * c;
        return z_logistic<SLOPE>(z, c * __builtin_fmaf(kB, c2, kA), c * __builtin_fmaf(3.0f * kB, c2, kA));
    }
    if (act == GEMM_ACT_GELU)
        return z_normal<SLOPE>(z);
    if (act == GEMM_ACT_RELU)   // NaN stays
        return {1.0f, z < 0.0f ? 0.0f : z, z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z};
    return {1.0f, z, 1.0f};
}

}  // namespace
