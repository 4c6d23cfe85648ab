// Quantisation of bf16 matrices to e4m3 with a scale for each block of 128 (part
// of library.hip).
//
// Bound by memory: 2 bytes in and 1 out per value.  Row scales of X itself need
// only a maximum over 16 lanes (k_quantize_rows).  Blocks of 128 x 128, and the
// transpose, take a 128 x 128 tile of X in one workgroup's registers
// (k_quantize_tile): 8192 x 4096 transposed, 101 MB, 21 us, 4.8 TB/s.
#pragma once

namespace {

struct QuantParams {
    const uint16_t* x;
    uint8_t* q;
    float* scale;
    int64_t M, K, ldx, ldq, lds;
    int64_t units;       // rows: M * per_row; tiles: tiles of 128 x 128
    int32_t per_row;     // ceil(K / 128)
};

template <bool EVEN>
__global__ void __launch_bounds__(256) k_quantize_rows(QuantParams p)
{
    for (int64_t u0 = (int64_t)blockIdx.x * kUnits; u0 < p.units; u0 += (int64_t)gridDim.x * kUnits) {
        if (u0 + threadIdx.x / kLanes >= p.units)
            continue;   // whole 16-lane groups drop out
        int64_t row, c;
        unit_place(u0, p.per_row, row, c);
        const int n = left(p.K, c);
        const u32x4_t v = load_chunk<EVEN>(p.x + row * p.ldx + c, n, c);
        float y[kChunk];
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            y[e] = chunk_at(v, e);
        const BlockScale b = block_scale(block_top(y));
        store_chunk8<EVEN>(p.q + row * p.ldq + c, n, chunk_fp8(y, b));
        if ((threadIdx.x & (kLanes - 1)) == 0)
            p.scale[c / kBlock * p.lds + row] = b.scale;
    }
}

// A 128 x 128 tile per workgroup of 256 threads: thread t holds the 8 x 8 values
// at rows 8 (t / 16) .. and columns 8 (t % 16) .. of the tile.  Each of its 8
// loads is 16 bytes, and 16 lanes read a 256-byte row piece.
//
// TRANSPOSED writes Q = X^T: v_cvt_pk_fp8_f32 packs any two registers, so the
// bytes of 8 consecutive rows of one column come out as two dwords without
// further moves.  They pass through LDS, whose rows are the tile's columns, and
// leave as whole 128-byte rows of Q.  An 8-byte write serves 32 lanes at a time:
// 16 columns, 8 rows of LDS apart, at 2 neighbouring chunks.  Rows of 136 bytes
// put the columns on 4 starting banks, 16 apart, and moving the chunks by 4 in
// every other run of 32 columns and by 2 in every other run of 64 fills the
// banks between, so that the 64 words take one cycle (rows of 136 bytes alone:
// 0.65 of the LDS cycles were conflicts and 8192 x 4096 took 22.0 us; 0.39, all
// of them of the reads, and 20.6 us so).
constexpr int kTileLd = kBlock + 8;

__device__ __forceinline__ int tile_at(int col, int row8)
{
    return col * kTileLd + (row8 ^ (((col >> 5) & 1) * 32 + ((col >> 6) & 1) * 16));
}

template <bool BLOCKS, bool TRANSPOSED>
__global__ void __launch_bounds__(256, 4) k_quantize_tile(QuantParams p)
{
    static_assert(BLOCKS || TRANSPOSED, "row scales of X itself are k_quantize_rows'");
    __shared__ uint32_t tops[4][kBlock];
    __shared__ __attribute__((aligned(16))) uint8_t tile[TRANSPOSED ? kBlock * kTileLd : 16];
    const int t = threadIdx.x, w = t >> 6;
    const int r8 = (t >> 4) * kChunk, c8 = (t & 15) * kChunk;
    for (int64_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        const int64_t tr = unit / p.per_row, tc = unit - tr * p.per_row;
        const int64_t r0 = tr * kBlock, c0 = tc * kBlock;
        const int nr = (int)min(p.M - r0, (int64_t)kBlock), nc = (int)min(p.K - c0, (int64_t)kBlock);
        u32x4_t v[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
            v[i] = load_chunk<false>(p.x + (r0 + min(r8 + i, nr - 1)) * p.ldx + c0 + min(c8, nc - 1),
                              r8 + i < nr ? nc - c8 : 0, c0 + c8);
        BlockScale b[kChunk];   // of each column; of the tile in b[0]
        if constexpr (BLOCKS) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
#pragma unroll
                for (int e = 0; e < kChunk; ++e)
                    m = max(m, magnitude(chunk_at(v[i], e)));
            m = row16_max(m);
            m = max(m, (uint32_t)__shfl_xor((int)m, 16));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32));
            if ((t & 63) == 0)
                tops[w][0] = m;
            __syncthreads();
            m = max(max(tops[0][0], tops[1][0]), max(tops[2][0], tops[3][0]));
            b[0] = block_scale(m);
            if (t == 0)
                p.scale[TRANSPOSED ? tr * p.lds + tc : tc * p.lds + tr] = b[0].scale;
        } else {
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    m = max(m, magnitude(chunk_at(v[i], e)));
                m = max(m, (uint32_t)__shfl_xor((int)m, 16));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32));
                if ((t & 63) < 16)
                    tops[w][c8 + e] = m;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                b[e] = block_scale(max(max(tops[0][c8 + e], tops[1][c8 + e]), max(tops[2][c8 + e], tops[3][c8 + e])));
            if (t < 16) {
#pragma unroll
                for (int e = 0; e < kChunk; ++e)
                    if (c8 + e < nc)
                        p.scale[tr * p.lds + c0 + c8 + e] = b[e].scale;
            }
        }
        if constexpr (TRANSPOSED) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                const BlockScale& s = b[BLOCKS ? 0 : e];
                float y[kChunk];
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    y[i] = chunk_at(v[i], e);
                *(u32x2_t*)(tile + tile_at(c8 + e, r8)) = chunk_fp8(y, s);
            }
            __syncthreads();
            // 16 lanes write one row of Q: 8 bytes each, 16 rows at a time.
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                const int c = i * 16 + (t >> 4);
                if (c < nc)
                    store_chunk8<false>(p.q + (c0 + c) * p.ldq + r0 + c8, nr - c8,
                                 *(const u32x2_t*)(tile + tile_at(c, c8)));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                float y[kChunk];
#pragma unroll
                for (int e = 0; e < kChunk; ++e)
                    y[e] = chunk_at(v[i], e);
                if (r8 + i < nr)
                    store_chunk8<false>(p.q + (r0 + r8 + i) * p.ldq + c0 + c8, nc - c8, chunk_fp8(y, b[0]));
            }
        }
        __syncthreads();   // tops and tile are free for the next unit
    }
}

}  // namespace

extern "C" {

int gemm_quantize_fp8(int64_t M, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq, float* scale,
                      int64_t lds, int block_rows, int transposed, void* stream)
{
    if (M < 0 || K < 0 || (block_rows != 1 && block_rows != kBlock))
        return GEMM_ERR_INVALID_VALUE;
    if (M > kMaxRows || K > kMaxRows)
        return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || K == 0)
        return GEMM_OK;
    const int64_t R = transposed ? K : M, L = transposed ? M : K;
    const Operand x{X, M, K, ldx, 2}, q{Q, R, L, ldq, 1};
    const Operand s{scale, (L + kBlock - 1) / kBlock, block_rows == 1 ? R : (R + kBlock - 1) / kBlock, lds, 4};
    const Operand all[] = {x, q, s};
    if (const int rc = check_operands(all, 3))
        return rc;
    if (meet(q, x) || meet(s, x) || meet(s, q))
        return GEMM_ERR_ALIAS;
    int cus = 0;
    if (const int rc = device_info(&cus))
        return rc;
    QuantParams p{(const uint16_t*)X, (uint8_t*)Q, scale, M, K, ldx, ldq, lds, 0, (int32_t)((K + kBlock - 1) / kBlock)};
    hipStream_t st = (hipStream_t)stream;
    if (block_rows == 1 && !transposed) {
        p.units = M * p.per_row;
        if (K % kChunk == 0)
            hipLaunchKernelGGL(k_quantize_rows<true>, dim3(unit_grid(p.units)), dim3(256), 0, st, p);
        else
            hipLaunchKernelGGL(k_quantize_rows<false>, dim3(unit_grid(p.units)), dim3(256), 0, st, p);
        return launched();
    }
    p.units = (M + kBlock - 1) / kBlock * p.per_row;
    const dim3 grid((unsigned)(p.units < (1 << 22) ? p.units : (1 << 22)));
    if (block_rows == 1)
        hipLaunchKernelGGL(HIP_KERNEL_NAME(k_quantize_tile<false, true>), grid, dim3(256), 0, st, p);
    else if (transposed)
        hipLaunchKernelGGL(HIP_KERNEL_NAME(k_quantize_tile<true, true>), grid, dim3(256), 0, st, p);
    else
        hipLaunchKernelGGL(HIP_KERNEL_NAME(k_quantize_tile<true, false>), grid, dim3(256), 0, st, p);
    return launched();
}

}  // extern "C"
