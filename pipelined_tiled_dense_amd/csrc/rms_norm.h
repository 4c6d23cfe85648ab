// Root-mean-square norm with the residual's addition, and its gradients (part
// of library.hip).
//
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight
//
// Bound by memory: a row is read once, held in registers across the row's sum of
// squares, and written once (8192 x 8192 with residual to 8 bits, 470 MB: 84 us, 5.6
// TB/s; a large copy reaches 5.1).  Off the multiple of 8 over 16384 wide, 5 registers
// (8 to bf16) of a lane's go through scratch memory: 2048 x 32761 to 8 bits 134 us,
// 32768 105.  One row: 2.7 us, the latency of two loads, the row's sum and a store.
#pragma once

namespace {

// Lanes per row: a whole number of waves, each lane holding NCH chunks of 8
// values, chunk i of lane t being chunk i * lanes + t of the row.  A row of one
// wave needs no workgroup reduction, so a workgroup takes 4 such rows.
struct NormParams {
    const uint16_t* x;
    const uint16_t* residual;   // null: h = x
    const uint16_t* weight;
    uint16_t* h;                // null without a residual
    void* y;                    // bf16 or e4m3
    float* scale;               // e4m3 only
    float* rstd;                // may be null
    int64_t M, ldx, ldr, ldh, ldy, lds;
    int32_t D;
    float eps, inv_d;
};

// Sum over the `nw` waves of a workgroup, in wave order, on every lane.  Slots
// of `red` alternate between calls (the caller's parity), so that one barrier
// separates a call's writes from its reads and from the next call's writes.
__device__ __forceinline__ float group_sum(float x, float* red, int nw)
{
    x = wave_sum(x);
    if (nw == 1)
        return x;
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < nw; ++i)
        s += red[i];
    return s;
}

// Where a mean square is sure to hold no subnormal or lost squares, and a sum no
// infinite ones.
constexpr float kLeastMean = 0x1p-100f, kMostSum = 0x1.fffffep127f;

// Six waves per SIMD where the registers would allow five for the sake of a few
// values (6220 x 5001 to bf16: 63.7 us, 67.4 with five); four, as 1024 threads have
// at the least, leaves the other forms as they come out.
template <int NCH, bool FP8, bool EVEN>
__global__ void __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(NCH == 2 && !FP8 && !EVEN ? 6 : 4)))
k_rms_norm(NormParams p, int nw)
{
    __shared__ float red[2][16];
    const int lane_t = nw == 1 ? (threadIdx.x & 63) : threadIdx.x;
    const int lanes = nw * 64;
    const int rows_per_wg = nw == 1 ? (int)(blockDim.x >> 6) : 1;
    const int sub = nw == 1 ? (int)(threadIdx.x >> 6) : 0;
    const int64_t groups = (p.M + rows_per_wg - 1) / rows_per_wg;
    int parity = 0;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        const int64_t row = g * rows_per_wg + sub;
        if (row >= p.M)
            continue;   // single-wave rows only: no barrier is skipped
        const uint16_t* x = p.x + row * p.ldx;
        const uint16_t* r = p.residual ? p.residual + row * p.ldr : nullptr;
        u32x4_t xv[NCH], rv[NCH], wv[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * lanes + lane_t) * kChunk;
            xv[i] = load_chunk<EVEN>(x + c, p.D - c, c);
            if (r)
                rv[i] = load_chunk<EVEN>(r + c, p.D - c, c);
            wv[i] = load_chunk<EVEN>(p.weight + c, p.D - c, c);
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                const float v = r ? chunk_at(xv[i], e) + chunk_at(rv[i], e) : chunk_at(xv[i], e);
                ss = __builtin_fmaf(v, v, ss);
            }
        ss = group_sum(ss, red[parity], nw);
        parity ^= 1;
        float mean = ss * p.inv_d + p.eps, size = 1.0f;
        // Squares beyond fp32's range, from |h| = 2^64 / sqrt(D) up or, with eps near
        // zero, below 2^-50: the row's sum again, of values times a power of two.
        // Every lane of the row holds the same sum, so the row's lanes branch together.
        if (__builtin_expect(!(mean >= kLeastMean && ss <= kMostSum), 0)) {
            size = mean < 1.0f ? 0x1p80f : 0x1p-80f;
            ss = 0.0f;
#pragma unroll
            for (int i = 0; i < NCH; ++i)
#pragma unroll
                for (int e = 0; e < kChunk; ++e) {
                    const float v = size * (r ? chunk_at(xv[i], e) + chunk_at(rv[i], e) : chunk_at(xv[i], e));
                    ss = __builtin_fmaf(v, v, ss);
                }
            ss = group_sum(ss, red[parity], nw);
            parity ^= 1;
            mean = ss * p.inv_d + p.eps * size * size;
        }
        const float rstd = size / __builtin_sqrtf(mean);
        if (p.rstd && lane_t == 0)
            p.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * lanes + lane_t) * kChunk;
            float h[kChunk], y[kChunk];
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                h[e] = r ? chunk_at(xv[i], e) + chunk_at(rv[i], e) : chunk_at(xv[i], e);
                y[e] = h[e] * rstd * chunk_at(wv[i], e);
            }
            if (r)
                store_chunk<EVEN>(p.h + row * p.ldh + c, p.D - c, chunk_bf16(h));
            if constexpr (FP8) {
                // Every lane takes part: lanes past the row hold zeros.
                const BlockScale b = block_scale(block_top(y));
                store_chunk8<EVEN>((uint8_t*)p.y + row * p.ldy + c, p.D - c, chunk_fp8(y, b));
                if ((lane_t & (kLanes - 1)) == 0 && c < p.D)
                    p.scale[(int64_t)(c / kBlock) * p.lds + row] = b.scale;
            } else {
                store_chunk<EVEN>((uint16_t*)p.y + row * p.ldy + c, p.D - c, chunk_bf16(y));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Gradients.  Per row, with n = h * rstd and t = dy * weight:
//
//   dx = dres + rstd * (t - n * mean(t * n)),    dweight += dy * n
//
// One pass: a workgroup takes every gridDim-th row (so that neighbouring rows
// are in flight together), keeps each row in registers across the mean, and sums
// its rows' share of dweight in registers; the workgroups' shares go to temporary
// memory and a second, small launch adds them in workgroup order, so the sum does
// not depend on timing.  Bound by memory (8191 x 4096, 268 MB: 54 us, 5.0 TB/s; 4096 x
// 16384 90 us).  Over 16384 wide a lane's four chunks of dy, h, dres, the weight and
// its sums do not fit 128 registers, what 1024 threads leave, and 116 of them (103 off
// the multiple of 8) go through scratch memory: 2048 x 32768 274 us, three times as
// long as the same bytes at 16384.
// ---------------------------------------------------------------------------
struct NormBwdParams {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* weight;
    const float* rstd;
    const uint16_t* dres;   // may be null
    uint16_t* dx;
    float* part;            // [gridDim.x][D]
    int64_t M, lddy, ldh, lddr, lddx;
    int32_t D;
    float inv_d;
};

template <int NCH, bool EVEN>
__global__ void __launch_bounds__(1024) k_rms_norm_bwd(NormBwdParams p, int nw)
{
    __shared__ float red[2][16];
    const int lanes = nw * 64, t = threadIdx.x;
    u32x4_t wv[NCH];
    float dw[NCH][kChunk];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = (i * lanes + t) * kChunk;
        wv[i] = load_chunk<EVEN>(p.weight + c, p.D - c, c);
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            dw[i][e] = 0.0f;
    }
    struct Row {
        u32x4_t g[NCH], h[NCH], s[NCH];
        float rstd;
    };
    // Fetched a row ahead where the registers last (one chunk a lane: 8191 x 4096
    // 59.0 us without, 54.1 with; two: 4096 x 16384 116 us without, 135 with).
    auto fetch = [&](int64_t row) {
        Row v;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * lanes + t) * kChunk;
            v.g[i] = load_chunk<EVEN>(p.dy + row * p.lddy + c, p.D - c, c);
            v.h[i] = load_chunk<EVEN>(p.h + row * p.ldh + c, p.D - c, c);
            if (p.dres)
                v.s[i] = load_chunk<EVEN>(p.dres + row * p.lddr + c, p.D - c, c);
        }
        v.rstd = p.rstd[row];
        return v;
    };
    constexpr bool AHEAD = NCH == 1;
    Row v, next;
    if constexpr (AHEAD)
        next = fetch(blockIdx.x);
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        if constexpr (AHEAD) {
            v = next;
            if (row + gridDim.x < p.M)
                next = fetch(row + gridDim.x);
        } else {
            v = fetch(row);
        }
        const float rs = v.rstd;
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                const float g = chunk_at(v.g[i], e), n = chunk_at(v.h[i], e) * rs;
                dw[i][e] = __builtin_fmaf(g, n, dw[i][e]);
                dot = __builtin_fmaf(g * chunk_at(wv[i], e), n, dot);
            }
        const float mean = group_sum(dot, red[parity], nw) * p.inv_d;
        parity ^= 1;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = (i * lanes + t) * kChunk;
            float d[kChunk];
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                const float n = chunk_at(v.h[i], e) * rs;
                d[e] = rs * (chunk_at(v.g[i], e) * chunk_at(wv[i], e) - n * mean);
                if (p.dres)
                    d[e] += chunk_at(v.s[i], e);
            }
            store_chunk<EVEN>(p.dx + row * p.lddx + c, p.D - c, chunk_bf16(d));
        }
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            const int c = (i * lanes + t) * kChunk + e;
            if (c < p.D)
                p.part[(int64_t)blockIdx.x * p.D + c] = dw[i][e];
        }
}

// dweight[j] = sum over `n` workgroups of their shares: a workgroup takes 16
// columns, its 64 groups of 16 lanes a contiguous part of the shares each, added
// in order.  (Few columns a workgroup, so that there are enough workgroups to
// read the shares at once: 8191 x 4096, 64 columns 10.8 us.)
__global__ void __launch_bounds__(1024) k_norm_weight_grad(const float* part, int32_t n, int32_t D, float* dw)
{
    __shared__ float sum[64][17];
    const int lane = threadIdx.x & 15, w = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + lane;
    float s = 0.0f;
    if (c < D) {
        const float* at = part + c;
#pragma unroll 8
        for (int32_t i = n * w / 64; i < n * (w + 1) / 64; ++i)
            s += at[(int64_t)i * D];
    }
    sum[w][lane] = s;
    __syncthreads();
    if (threadIdx.x < 16 && c < D) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i)
            s += sum[i][lane];
        dw[c] = s;
    }
}

// Waves per row and chunks per lane for D values: 4 waves before a lane takes
// another chunk (8192 x 4096 forward 39.0 us, with 8 waves of one chunk 41.2; 8192 x
// 2048 20.3, with 2 waves of two 19.5), up to max_nch chunks as long as the row fits
// 16 waves, and then as many as it needs.
struct RowShape {
    int nch, nw;
};

RowShape row_shape(int64_t D, int max_nch)
{
    const int64_t chunks = (D + kChunk - 1) / kChunk;
    int nch = 1;
    while (nch < max_nch && chunks > 64 * 4 * nch)
        nch *= 2;
    while (chunks > 64 * 16 * nch)
        nch *= 2;
    return RowShape{nch, (int)((chunks + 64 * nch - 1) / (64 * nch))};
}

// Calls f.template operator()<NCH, EVEN>() for the shape and width.
template <class F>
void with_row_shape(const RowShape& rs, int64_t D, F&& f)
{
    const bool even = D % kChunk == 0;
    if (rs.nch == 1)
        even ? f.template operator()<1, true>() : f.template operator()<1, false>();
    else if (rs.nch == 2)
        even ? f.template operator()<2, true>() : f.template operator()<2, false>();
    else
        even ? f.template operator()<4, true>() : f.template operator()<4, false>();
}

// Workgroups of the gradients' kernel.  Each writes D partial sums, so there are only as
// many as give a compute unit 8 waves (8191 x 4096, 8 waves a row, both launches: one
// workgroup each 54.1 us, two 59.5), and none with fewer than 2 rows.  A few rows: one
// workgroup, whose sums are the weight's gradient, in one launch (3 x 4096 5.5 us, in
// two launches 9.2; 8 rows are level at 4096 wide, 20.1 against 17.5 at 16384).
int64_t norm_bwd_grid(int64_t M, int64_t D, int cus)
{
    const int nw = row_shape(D, 1).nw;
    if (M <= 4)
        return M > 0 ? 1 : 0;
    return std::min<int64_t>((int64_t)cus * ((8 + nw - 1) / nw), (M + 1) / 2);
}

int norm_shape(int64_t M, int64_t D)
{
    if (M < 0 || D < 1)
        return GEMM_ERR_INVALID_VALUE;
    return M > kMaxRows || D > GEMM_NORM_MAX_WIDTH ? GEMM_ERR_UNSUPPORTED_SHAPE : GEMM_OK;
}

// `take`: where the workgroups' shares of the weight's gradient come from.
int rms_norm_bwd(int64_t M, int64_t D, const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* weight,
                 const float* rstd, const void* dres, int64_t lddr, void* dX, int64_t lddx, float* dweight,
                 int (*take)(TempMem&, int64_t, hipStream_t, void**, hipEvent_t*), void* workspace,
                 int64_t workspace_bytes, void* stream)
{
    if (int rc = norm_shape(M, D))
        return rc;
    const Operand dw{dweight, 1, D, D, 4};
    int rc = check_operand(dw);
    if (rc != GEMM_OK)
        return rc;
    const Operand dy{dY, M, D, lddy, 2}, h{H, M, D, ldh, 2}, w{weight, 1, D, D, 2}, v{rstd, 1, M, M, 4};
    const Operand s{dres, M, D, lddr, 2}, dx{dX, M, D, lddx, 2};
    if (M > 0) {
        const Operand in[] = {dy, h, w, v, s};
        rc = check_operands(in, dres ? 5 : 4);
        if (rc == GEMM_OK)
            rc = check_operand(dx);
        if (rc != GEMM_OK)
            return rc;
        // As in the forward pass, a lane has read its values of the row before it writes them.
        for (const Operand& i : in) {
            if (meet(dw, i) || (meet(dx, i) && !((i.p == dy.p || i.p == s.p) && same_memory(dx, i))))
                return GEMM_ERR_ALIAS;
        }
        if (meet(dx, dw))
            return GEMM_ERR_ALIAS;
    }
    if (workspace) {
        if (workspace_bytes < 0)
            return GEMM_ERR_INVALID_VALUE;
        if ((uintptr_t)workspace & 255)
            return GEMM_ERR_MISALIGNED;
        const Operand t{workspace, 1, workspace_bytes, workspace_bytes, 1};
        for (const Operand& o : {dy, h, w, v, s, dx, dw})
            if (meet(t, o))
                return GEMM_ERR_ALIAS;
    }
    int cus = 0;
    TempMem tm;
    rc = device_info(&cus, &tm.pool, nullptr, &tm.info);
    if (rc != GEMM_OK)
        return rc;
    tm.given(workspace, workspace_bytes);
    hipStream_t st = (hipStream_t)stream;
    const RowShape rs = row_shape(D, 1);
    const int64_t grid = norm_bwd_grid(M, D, cus);
    void* ws = nullptr;
    hipEvent_t done = nullptr;
    if (grid > 1) {
        rc = take(tm, grid * D * 4, st, &ws, &done);
        if (rc != GEMM_OK)
            return rc;
    }
    if (grid > 0) {
        NormBwdParams p{(const uint16_t*)dY, (const uint16_t*)H, (const uint16_t*)weight, rstd, (const uint16_t*)dres,
                        (uint16_t*)dX, grid > 1 ? (float*)ws : dweight, M, lddy, ldh, lddr, lddx, (int32_t)D,
                        1.0f / (float)D};
        const dim3 g((unsigned)grid), b((unsigned)(rs.nw * 64));
        with_row_shape(rs, D, [&]<int NCH, bool EVEN>() {
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_rms_norm_bwd<NCH, EVEN>), g, b, 0, st, p, rs.nw);
        });
        rc = launched();
    }
    if (rc == GEMM_OK && grid != 1) {
        // The shares' last use: its completion records the block's event.
        hipExtLaunchKernelGGL(k_norm_weight_grad, dim3((unsigned)((D + 15) / 16)), dim3(1024), 0, st, nullptr, done, 0,
                              (const float*)ws, (int32_t)grid, (int32_t)D, dweight);
        rc = launched();
    }
    const int frc = temp_give(tm, ws, st, rc == GEMM_OK && done != nullptr);
    return rc != GEMM_OK ? rc : frc;
}

}  // namespace

extern "C" {

int gemm_rms_norm(int64_t M, int64_t D, const void* X, int64_t ldx, const void* residual, int64_t ldr,
                  const void* weight, float eps, void* H, int64_t ldh, void* Y, int64_t ldy, int y_type, float* scale,
                  int64_t lds, float* rstd, void* stream)
{
    if (int rc = norm_shape(M, D))
        return rc;
    const bool fp8 = y_type == GEMM_TYPE_FP8;
    if ((!fp8 && y_type != GEMM_TYPE_BF16) || !(eps >= 0.0f) || eps > 3.0e38f)
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0)
        return GEMM_OK;
    const Operand x{X, M, D, ldx, 2}, r{residual, M, D, ldr, 2}, w{weight, 1, D, D, 2};
    const Operand h{residual ? H : nullptr, M, D, ldh, 2}, y{Y, M, D, ldy, fp8 ? 1 : 2};
    const Operand s{fp8 ? scale : nullptr, (D + kBlock - 1) / kBlock, M, lds, 4}, v{rstd, 1, M, M, 4};
    const Operand in[] = {x, w, r}, out[] = {y, h, s, v};
    int rc = check_operands(in, residual ? 3 : 2);
    if (rc == GEMM_OK)
        rc = check_operand(y);
    if (rc == GEMM_OK && residual)
        rc = check_operand(h);
    if (rc == GEMM_OK && fp8)
        rc = check_operand(s);
    if (rc == GEMM_OK && rstd)
        rc = check_operand(v);
    if (rc != GEMM_OK)
        return rc;
    // Each lane reads its values of a row before it writes any of them, so a
    // row may be written over itself.
    for (const Operand& o : out) {
        for (const Operand& i : in) {
            const bool self = (o.p == h.p && (i.p == x.p || i.p == r.p)) || (o.p == y.p && i.p == x.p);
            if (meet(o, i) && !(self && same_memory(o, i)))
                return GEMM_ERR_ALIAS;
        }
        for (const Operand& q : out)
            if (&q != &o && meet(o, q))
                return GEMM_ERR_ALIAS;
    }
    int cus = 0;
    rc = device_info(&cus);
    if (rc != GEMM_OK)
        return rc;
    NormParams p{(const uint16_t*)X, (const uint16_t*)residual, (const uint16_t*)weight, (uint16_t*)H, Y, scale, rstd,
                 M, ldx, ldr, ldh, ldy, lds, (int32_t)D, eps, 1.0f / (float)D};
    // With rows for every compute unit twice over, two chunks a lane: more of a row
    // in flight from fewer waves (2048 x 8192 20.6 us, with one 23.1); with fewer rows
    // one, which has each lane's work done sooner (1 x 4096 2.7 us, with two 3.0; 512
    // rows are level).
    const RowShape rs = row_shape(D, M < 2 * cus ? 1 : 2);
    const int threads = rs.nw == 1 ? 256 : rs.nw * 64;
    const int64_t groups = rs.nw == 1 ? (M + 3) / 4 : M;
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)));
    with_row_shape(rs, D, [&]<int NCH, bool EVEN>() {
        if (fp8)
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_rms_norm<NCH, true, EVEN>), grid, dim3(threads), 0,
                               (hipStream_t)stream, p, rs.nw);
        else
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_rms_norm<NCH, false, EVEN>), grid, dim3(threads), 0,
                               (hipStream_t)stream, p, rs.nw);
    });
    return launched();
}

int gemm_rms_norm_bwd(int64_t M, int64_t D, const void* dY, int64_t lddy, const void* H, int64_t ldh,
                      const void* weight, const float* rstd, const void* dres, int64_t lddr, void* dX, int64_t lddx,
                      float* dweight, void* stream)
{
    return rms_norm_bwd(M, D, dY, lddy, H, ldh, weight, rstd, dres, lddr, dX, lddx, dweight, temp_take, nullptr, 0, stream);
}

int gemm_rms_norm_bwd_given(int64_t M, int64_t D, const void* dY, int64_t lddy, const void* H, int64_t ldh,
                            const void* weight, const float* rstd, const void* dres, int64_t lddr, void* dX,
                            int64_t lddx, float* dweight, void* workspace, int64_t workspace_bytes, void* stream)
{
    return rms_norm_bwd(M, D, dY, lddy, H, ldh, weight, rstd, dres, lddr, dX, lddx, dweight, temp_take_outside_graphs,
                        workspace, workspace_bytes, stream);
}

int64_t gemm_rms_norm_bwd_scratch_cus(int64_t M, int64_t D, int compute_units)
{
    if (const int rc = norm_shape(M, D))
        return rc;
    if (compute_units < 1)
        return GEMM_ERR_INVALID_VALUE;
    const int64_t grid = norm_bwd_grid(M, D, compute_units);
    return grid > 1 ? align256(grid * D * 4) : 0;
}

}  // extern "C"
