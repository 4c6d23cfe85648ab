// The gated unit y = silu(g) * u and its gradient (part of library.hip).
//
// Bound by memory: every value is read once and written once, 8 at a time.  A
// unit of work is 128 columns of a row, 16 lanes of one chunk, so that an 8-bit
// output's scale is a maximum over one DPP row.  8192 x 8192 to 8 bits, 335 MB:
// 68 us, 4.9 TB/s; the gradient at 2047 x 5005, 102 MB, whose odd rows start at
// any byte: 20 us, 5.1 TB/s (a large copy reaches 5.1).
#pragma once

namespace {

// s = 1 / (1 + exp(-x)) and c = 1 - s, from t = exp(-|x|) <= 1:
//
//   s = (x < 0 ? t : 1) / (1 + t),   c = (x < 0 ? 1 : t) / (1 + t)
//
// so nothing overflows and neither of the two cancels.  t = 2^(-|x| log2 e): the
// product with log2 e is split into its rounded value and the rest, which
// enters to first order (a single rounded product would be off by |x| ulp).
// v_exp_f32 returns zero where the result is subnormal, so it computes the
// square root of t; the product of two roots keeps the subnormal values.  |x|
// is bounded where t is zero anyway, which leaves no infinity minus infinity;
// a NaN passes the comparison.
struct Sigmoid {
    float s, c;
};

__device__ __forceinline__ Sigmoid sigmoid(float x)
{
    constexpr float kLog2e = 0x1.715476p+0f;      // log2 e rounded to fp32
    constexpr float kLog2eRest = 0x1.4ae0cp-26f;  // log2 e - kLog2e
    constexpr float kLn2 = 0x1.62e430p-1f;
    const float ax = __builtin_fabsf(x), nx = ax > 150.0f ? -150.0f : -ax;
    const float p = nx * kLog2e;
    const float rest = __builtin_fmaf(nx, kLog2e, -p) + nx * kLog2eRest;
    const float root = __builtin_amdgcn_exp2f(0.5f * p);
    const float t = root * __builtin_fmaf(root, rest * kLn2, root);
    // 1 <= 1 + t <= 2: the hardware reciprocal and one Newton step.
    const float d = 1.0f + t, r0 = __builtin_amdgcn_rcpf(d);
    const float r = __builtin_fmaf(__builtin_fmaf(-d, r0, 1.0f), r0, r0);
    const float tr = t * r;
    return x < 0.0f ? Sigmoid{tr, r} : Sigmoid{r, tr};
}

// silu(x) * u alone, in fewer steps (the 8-bit forward kernel is bound by its
// vector instructions as much as by memory): x u / (1 + exp(-x)) for x from
// kLowGate on, where exp(-x) stays below 2^127.7.  The denominator is taken times
// 1/4, so that its reciprocal stays a normal number, which v_rcp_f32 needs, and x
// with it, so that no product passes |x|; a Newton step corrects the reciprocal
// (its ulp alone turned twice as many 8-bit roundings as the other steps; 3 us at
// 8192 x 8192).
constexpr float kLowGate = -88.5f;
// The gradients': higher, so that u s stays a normal number for every u that matters.
constexpr float kLowGateGrad = -40.0f;

__device__ __forceinline__ float silu_times(float x, float u)
{
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e430p-1f;
    const float nx = x > 150.0f ? -150.0f : -x;
    const float p = nx * kLog2e;
    const float rest = __builtin_fmaf(nx, kLog2eRest, __builtin_fmaf(nx, kLog2e, -p));
    const float e0 = __builtin_amdgcn_exp2f(p);
    const float e = __builtin_fmaf(e0, rest * kLn2, e0);
    const float d = __builtin_fmaf(e, 0.25f, 0.25f), r0 = __builtin_amdgcn_rcpf(d);
    const float r = __builtin_fmaf(__builtin_fmaf(-d, r0, 1.0f), r0, r0);
    return (0.25f * x) * r * u;
}

// Below these gates 1 + exp(-x) is exp(-x) to fp32, and exp(x) the third power of f =
// exp(x / 3), a normal number: each of the factors beside exp(x) takes an f first,
// so that a large one meets a small one before anything overflows or is lost.
// v_exp_f32 makes f zero from -262 on down, where what is left is below bf16's
// smallest value (beside one large factor; beside two, below 2^-114).  The bound
// on x keeps infinities out of the products; minus infinity is left to the formula.
struct LowGate {
    float x, f;
};

__device__ __forceinline__ LowGate low_gate(float x)
{
    constexpr float kThird = 0x1.ec709ep-2f, kThirdRest = -0x1.e2fe02p-29f, kLn2 = 0x1.62e430p-1f;   // (log2 e) / 3
    const float xc = x < -1000.0f ? -1000.0f : x;
    const float p = xc * kThird;
    const float rest = __builtin_fmaf(xc, kThirdRest, __builtin_fmaf(xc, kThird, -p));
    const float f0 = __builtin_amdgcn_exp2f(p);
    return {x == -__builtin_inff() ? __builtin_nanf("") : xc, __builtin_fmaf(f0, rest * kLn2, f0)};
}

__device__ __forceinline__ float silu_times_low(float x, float u)
{
    const LowGate l = low_gate(x);
    return (u * l.f) * (l.x * l.f) * l.f;
}

__device__ __forceinline__ float lowest(u32x4_t gv)
{
    float low = 0.0f;
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
        low = __builtin_fminf(low, chunk_at(gv, e));
    return low;
}

// 8 gates and their u.  Gates below kLowGate are rare: a branch that no lane of
// most waves takes, with both ways whole (8192 x 8192 to 8 bits: 68 us; 73 with the
// low gates corrected after the others).
__device__ __forceinline__ void silu_chunk(u32x4_t gv, u32x4_t uv, float (&y)[kChunk])
{
    if (__builtin_expect(lowest(gv) < kLowGate, 0)) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            const float g = chunk_at(gv, e), u = chunk_at(uv, e);
            y[e] = g < kLowGate ? silu_times_low(g, u) : silu_times(g, u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            y[e] = silu_times(chunk_at(gv, e), chunk_at(uv, e));
    }
}

struct SwigluParams {
    const uint16_t* dy;   // gradient only
    const uint16_t* gu;
    void* y;              // bf16 or e4m3; the gradient of gu
    float* scale;
    int64_t M, F, lddy, ldgu, ldy, lds;
    int64_t units;        // M * ceil(F / 128)
    int32_t per_row;      // ceil(F / 128)
};

template <bool FP8, bool EVEN>
__global__ void __launch_bounds__(256) k_swiglu(SwigluParams p)
{
    for (int64_t u0 = (int64_t)blockIdx.x * kUnits; u0 < p.units; u0 += (int64_t)gridDim.x * kUnits) {
        if (u0 + threadIdx.x / kLanes >= p.units)
            continue;   // whole 16-lane groups drop out: the maximum stays inside a group
        int64_t row, c;
        unit_place(u0, p.per_row, row, c);
        const int n = left(p.F, c);
        const uint16_t* src = p.gu + row * p.ldgu + c;
        const u32x4_t gv = load_chunk<EVEN>(src, n, c), uv = load_chunk<EVEN>(src + p.F, n, c);
        float y[kChunk];
        silu_chunk(gv, uv, y);
        if constexpr (FP8) {
            const BlockScale b = block_scale(block_top(y));
            store_chunk8<EVEN>((uint8_t*)p.y + row * p.ldy + c, n, chunk_fp8(y, b));
            if ((threadIdx.x & (kLanes - 1)) == 0)
                p.scale[c / kBlock * p.lds + row] = b.scale;
        } else {
            store_chunk<EVEN>((uint16_t*)p.y + row * p.ldy + c, n, chunk_bf16(y));
        }
    }
}

template <bool EVEN>
__global__ void __launch_bounds__(256) k_swiglu_bwd(SwigluParams p)
{
    for (int64_t u0 = (int64_t)blockIdx.x * kUnits; u0 < p.units; u0 += (int64_t)gridDim.x * kUnits) {
        if (u0 + threadIdx.x / kLanes >= p.units)
            continue;
        int64_t row, c;
        unit_place(u0, p.per_row, row, c);
        const int n = left(p.F, c);
        const uint16_t* src = p.gu + row * p.ldgu + c;
        const u32x4_t gv = load_chunk<EVEN>(src, n, c), uv = load_chunk<EVEN>(src + p.F, n, c);
        const u32x4_t dv = load_chunk<EVEN>(p.dy + row * p.lddy + c, n, c);
        float dg[kChunk], du[kChunk];
        auto gradient = [&](int e) {
            const float g = chunk_at(gv, e), d = chunk_at(dv, e);
            const Sigmoid s = sigmoid(g);
            du[e] = d * (g * s.s);
            dg[e] = d * (chunk_at(uv, e) * (s.s * __builtin_fmaf(g, s.c, 1.0f)));   // d * u alone may overflow
        };
        if (__builtin_expect(lowest(gv) < kLowGateGrad, 0)) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                if (chunk_at(gv, e) < kLowGateGrad) {
                    const LowGate l = low_gate(chunk_at(gv, e));
                    const float d = chunk_at(dv, e) * l.f;
                    du[e] = d * (l.x * l.f) * l.f;
                    dg[e] = d * (chunk_at(uv, e) * l.f) * ((1.0f + l.x) * l.f);
                } else {
                    gradient(e);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                gradient(e);
        }
        uint16_t* dst = (uint16_t*)p.y + row * p.ldy + c;
        store_chunk<EVEN>(dst, n, chunk_bf16(dg));
        store_chunk<EVEN>(dst + p.F, n, chunk_bf16(du));
    }
}

int swiglu_shape(int64_t M, int64_t F)
{
    if (M < 0 || F < 0)
        return GEMM_ERR_INVALID_VALUE;
    return M > kMaxRows || F > kMaxRows / 2 ? GEMM_ERR_UNSUPPORTED_SHAPE : GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_swiglu(int64_t M, int64_t F, const void* GU, int64_t ldgu, void* Y, int64_t ldy, int y_type, float* scale,
                int64_t lds, void* stream)
{
    if (int rc = swiglu_shape(M, F))
        return rc;
    const bool fp8 = y_type == GEMM_TYPE_FP8;
    if (!fp8 && y_type != GEMM_TYPE_BF16)
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || F == 0)
        return GEMM_OK;
    const int64_t per_row = (F + kBlock - 1) / kBlock;
    const Operand gu{GU, M, 2 * F, ldgu, 2}, y{Y, M, F, ldy, fp8 ? 1 : 2}, s{fp8 ? scale : nullptr, per_row, M, lds, 4};
    const Operand all[] = {gu, y, s};
    if (const int rc = check_operands(all, fp8 ? 3 : 2))
        return rc;
    if (meet(y, gu) || meet(s, gu) || meet(s, y))
        return GEMM_ERR_ALIAS;
    int cus = 0;
    if (const int rc = device_info(&cus))
        return rc;
    const SwigluParams p{nullptr, (const uint16_t*)GU, Y, scale, M, F, 0, ldgu, ldy, lds, M * per_row, (int32_t)per_row};
    const dim3 grid(unit_grid(p.units));
    auto run = [&]<bool EVEN>() {
        if (fp8)
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_swiglu<true, EVEN>), grid, dim3(256), 0, (hipStream_t)stream, p);
        else
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_swiglu<false, EVEN>), grid, dim3(256), 0, (hipStream_t)stream, p);
    };
    F % kChunk == 0 ? run.template operator()<true>() : run.template operator()<false>();
    return launched();
}

int gemm_swiglu_bwd(int64_t M, int64_t F, const void* dY, int64_t lddy, const void* GU, int64_t ldgu, void* dGU,
                    int64_t lddgu, void* stream)
{
    if (int rc = swiglu_shape(M, F))
        return rc;
    if (M == 0 || F == 0)
        return GEMM_OK;
    const Operand dy{dY, M, F, lddy, 2}, gu{GU, M, 2 * F, ldgu, 2}, dgu{dGU, M, 2 * F, lddgu, 2};
    const Operand all[] = {dy, gu, dgu};
    if (const int rc = check_operands(all, 3))
        return rc;
    // A lane reads its g and u before it writes their gradients in the same places.
    if (meet(dgu, dy) || (meet(dgu, gu) && !same_memory(dgu, gu)))
        return GEMM_ERR_ALIAS;
    int cus = 0;
    if (const int rc = device_info(&cus))
        return rc;
    const int64_t per_row = (F + kBlock - 1) / kBlock;
    const SwigluParams p{(const uint16_t*)dY, (const uint16_t*)GU, dGU, nullptr, M, F, lddy, ldgu, lddgu, 0,
                         M * per_row, (int32_t)per_row};
    if (F % kChunk == 0)
        hipLaunchKernelGGL(k_swiglu_bwd<true>, dim3(unit_grid(p.units)), dim3(256), 0, (hipStream_t)stream, p);
    else
        hipLaunchKernelGGL(k_swiglu_bwd<false>, dim3(unit_grid(p.units)), dim3(256), 0, (hipStream_t)stream, p);
    return launched();
}

}  // extern "C"
