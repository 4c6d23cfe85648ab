// Activations and their slopes, 8 values at a time, for the linear layers'
// epilogues (part of library.hip).
//
// Every step is right to fp32's rounding: one exponential and one reciprocal a value,
// to an ulp each, an exponential's argument rounded once (which is |v| half ulps of
// the result), and the normal distribution's tail from a polynomial to fp32.  So what
// is left where a slope's two terms cancel (gelu's at z = -0.7518) is as good as the
// terms are.  The steps count: beside memory, a small k's epilogues wait for them (4096 x
// 8192 over 1024: none 63.5 us, silu 68.3, gelu 75.5; with a tail right to 1.6e-5 only,
// whose slope was 0.4% off at z = -0.75, 74.5).  Arguments in two parts and a Newton step
// on the reciprocal, which would take away the |v| and half an ulp, cost 7 to 11% there
// and 1 to 3% of the large products, for less than a hundredth of bf16's half step: not
// taken.
// Very negative z, whose exponential or its reciprocal leaves fp32's normal range,
// take another way: a branch that no lane of most waves takes.
#pragma once

namespace {

// x times y times a slope of at most 1.13: half the slope goes with the larger of the two
// first, so that neither a product overflows where the result does not, nor a small
// one is lost before the third factor brings it back.
__device__ __forceinline__ float times_slope(float x, float y, float slope)
{
    const bool x_larger = __builtin_fabsf(x) > __builtin_fabsf(y);
    return 2.0f * ((x_larger ? x : y) * (0.5f * slope) * (x_larger ? y : x));
}

// a(z) and a'(z) as value * f^3 and slope * f^3, where the two are too small for fp32: f is
// the third root of what they hold of an exponential, a normal number, and each factor
// beside the activation takes an f first.
struct Activated {
    float f, value, slope;

    __device__ __forceinline__ float times(float x) const { return (x * f) * (value * f) * f; }
    __device__ __forceinline__ float slope_times(float x) const { return (x * f) * (slope * f) * f; }
    __device__ __forceinline__ float slope_times(float x, float y) const
    {
        const bool x_larger = __builtin_fabsf(x) > __builtin_fabsf(y);
        return ((x_larger ? x : y) * f) * (slope * f) * (x_larger ? y : x) * f;
    }
};

// Gelu's usual approximation is z p(v) with p the logistic function and v = z (a +
// b z^2); silu is z p(z).
constexpr float kTanhA = 1.59576912f, kTanhB = 0.0713548163f;   // 2 sqrt(2 / pi), that times 0.044715
constexpr float kDensity = 0.398942280f;                        // 1 / sqrt(2 pi)
constexpr float kLog2e = 1.44269504f;

// The normal distribution's tail, with a >= 0:
//
//   Phi(-a) = h(a) exp(-a^2 / 2),   h(a) = exp(a^2 / 2) erfc(a / sqrt 2) / 2
//
// h as a polynomial in t = 1 / (1 + 0.275 a), fitted by weighted least squares for
// the smallest relative error over 0 <= a <= 45: 7e-8, and 3e-7 with the roundings of
// its steps.  The slope of z Phi(z) is Phi(z) + z phi(z), phi the density exp(-z^2 /
// 2) / sqrt(2 pi).
__device__ __forceinline__ float normal_tail(float a)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.275f, a, 1.0f));
    float h = 0.0268538259f;
    h = __builtin_fmaf(h, t, -0.109358527f);
    h = __builtin_fmaf(h, t, 0.127873257f);
    h = __builtin_fmaf(h, t, -0.0329990834f);
    h = __builtin_fmaf(h, t, 0.0868154764f);
    h = __builtin_fmaf(h, t, 0.0793257654f);
    h = __builtin_fmaf(h, t, 0.102117389f);
    h = __builtin_fmaf(h, t, 0.109661452f);
    h = __builtin_fmaf(h, t, 0.109710418f);
    return h * t;
}

// The z below which the usual way loses what exp(v), or exp(-z^2 / 2), holds.
__device__ __forceinline__ float lowest_usual(int act)
{
    return act == GEMM_ACT_SILU ? -80.0f : act == GEMM_ACT_GELU ? -12.5f : -9.5f;
}

// Those z.  There the logistic function is exp(v) to fp32.
__device__ __forceinline__ Activated activated_low(int act, float z)
{
    // Minus infinity times zero: NaN, as the formulas have it.
    const float zn = z == -__builtin_inff() ? __builtin_nanf("") : z;
    if (act == GEMM_ACT_GELU) {
        const float a = __builtin_fminf(-z, 40.0f), h = normal_tail(a);
        return {__builtin_amdgcn_exp2f((-kLog2e / 6.0f) * (a * a)), zn * h, __builtin_fmaf(kDensity, zn, h)};
    }
    const bool silu = act == GEMM_ACT_SILU;
    const float c = silu ? z : z < -30.0f ? -30.0f : z, c2 = c * c;   // exp(v) is 0 at -30, and z^3 may overflow
    const float v = silu ? z : c * __builtin_fmaf(kTanhB, c2, kTanhA);
    const float zdv = silu ? zn : __builtin_fmaf(0.0f, zn, c * __builtin_fmaf(3.0f * kTanhB, c2, kTanhA));
    return {low_gate(v).f, zn, 1.0f + zdv};
}

template <bool SLOPE>
__device__ __forceinline__ void logistic_usual(float z, float minus_v, float dv, float& value, float& slope)
{
    const float e = __builtin_amdgcn_exp2f(minus_v * kLog2e), p = __builtin_amdgcn_rcpf(1.0f + e);
    value = z * p;
    if constexpr (SLOPE)
        slope = __builtin_fmaf(z * (e * p) * dv, p, p);
}

// f(i, a) for the activation a of z[i], i = 0 .. 7, and again with another a for the z
// that take the other way; `act` is uniform.
template <bool SLOPE, class F>
__device__ __forceinline__ void activate(int act, const float (&z)[kChunk], F&& f)
{
    struct Usual {
        float value, slope;
        __device__ __forceinline__ float times(float x) const { return x * value; }
        __device__ __forceinline__ float slope_times(float x) const { return x * slope; }
        __device__ __forceinline__ float slope_times(float x, float y) const { return times_slope(x, y, slope); }
    };
    Usual u;
    if (act <= GEMM_ACT_RELU) {   // NaN stays
        const bool relu = act == GEMM_ACT_RELU;
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            f(i, Usual{relu && z[i] < 0.0f ? 0.0f : z[i], relu && !(z[i] > 0.0f) ? (z[i] <= 0.0f ? 0.0f : z[i]) : 1.0f});
        return;
    }
    if (act == GEMM_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            logistic_usual<SLOPE>(z[i], -z[i], 1.0f, u.value, u.slope);
            f(i, u);
        }
    } else if (act == GEMM_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            const float z2 = z[i] * z[i];
            const float c = __builtin_amdgcn_fmed3f(z[i], -10.0f, 30.0f);   // the slope is 1 there, and z^2 may overflow
            logistic_usual<SLOPE>(z[i], z[i] * __builtin_fmaf(-kTanhB, z2, -kTanhA),
                                  __builtin_fmaf(3.0f * kTanhB * c, c, kTanhA), u.value, u.slope);
            f(i, u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            // The bounds keep infinity out of the value's product with zero, which the slope's
            // formula has; NaN comes through e.
            const float a = __builtin_amdgcn_fmed3f(__builtin_fabsf(z[i]), 0.0f, 30.0f), h = normal_tail(a);
            const float e = __builtin_amdgcn_exp2f((-0.5f * kLog2e) * (z[i] * z[i]));
            u.value = __builtin_fmaf(-a, h * e, __builtin_amdgcn_fmed3f(z[i], 0.0f, __builtin_inff()));
            if constexpr (SLOPE) {
                const float tail = e * __builtin_fmaf(-kDensity, __builtin_fabsf(z[i]), h);
                u.slope = z[i] > 0.0f ? 1.0f - tail : tail;
            }
            f(i, u);
        }
    }
    float low = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
        low = __builtin_fminf(low, z[i]);
    const float bound = lowest_usual(act);
    if (__builtin_expect(low < bound, 0)) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            if (z[i] < bound)
                f(i, activated_low(act, z[i]));
    }
}

}  // namespace
