// Device and host helpers shared by the 8-bit operators (part of library.hip).
#pragma once

namespace {

// ---------------------------------------------------------------------------
// Memory: 8 values at a time.
//
// Lane c of a row takes the 8 values 8c .. 8c+7, one 16-byte access in bf16 and
// one 8-byte access in e4m3.  The hardware takes these accesses at any byte
// address (global memory on gfx950 runs in unaligned mode and the compiler
// emits one dwordx4 for the copies below), so odd strides and offsets need no
// variant of their own; only the last, partial chunk of a row goes by element.
// ---------------------------------------------------------------------------
constexpr int kChunk = 8;
// A scale covers 128 values along k: 16 lanes of one chunk each, which is one
// DPP row, so a block's maximum takes four cross-lane moves and no LDS.
constexpr int kBlock = 128;
constexpr int kLanes = kBlock / kChunk;

// `n` (<= 8) valid bf16 values at p, as they are stored; zeros beyond.  A partial
// chunk that is not the row's first (`c` > 0 values precede it) is read from the
// row's last 16 bytes and shifted into place: one load, where guarded loads of
// single values would each wait for the one before.  EVEN: the row is a multiple
// of 8 long, a chunk whole or absent; kernels bound by memory have a form of
// their own for it, since the code for the tail costs them registers and with
// them waves (962 x 4224 norm to 8 bits: 7.8 us, 9.8 with it).
template <bool EVEN>
__device__ __forceinline__ u32x4_t load_chunk(const uint16_t* p, int n, int64_t c)
{
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (EVEN ? n > 0 : n >= kChunk) {
        __builtin_memcpy(&v, p, 16);
    } else if (!EVEN && n > 0 && c > 0) {
        uint64_t x[2];
        __builtin_memcpy(x, p - (kChunk - n), 16);
        const int s = 16 * (kChunk - n);   // 16 .. 112
        const uint64_t lo = s >= 64 ? x[1] : x[0], hi = s >= 64 ? 0u : x[1];
        x[0] = (s & 63) ? (lo >> (s & 63)) | (hi << (64 - (s & 63))) : lo;
        x[1] = hi >> (s & 63);
        __builtin_memcpy(&v, x, 16);
    } else if (!EVEN) {
#pragma unroll
        for (int e = 0; e < kChunk - 1; ++e)
            if (e < n)
                v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    return v;
}

template <bool EVEN>
__device__ __forceinline__ void store_chunk(uint16_t* p, int n, u32x4_t v)
{
    if (EVEN ? n > 0 : n >= kChunk) {
        __builtin_memcpy(p, &v, 16);
    } else if (!EVEN) {
#pragma unroll
        for (int e = 0; e < kChunk - 1; ++e)
            if (e < n)
                p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
}

template <bool EVEN>
__device__ __forceinline__ void store_chunk8(uint8_t* p, int n, u32x2_t v)
{
    if (EVEN ? n > 0 : n >= kChunk) {
        __builtin_memcpy(p, &v, 8);
    } else if (!EVEN) {
#pragma unroll
        for (int e = 0; e < kChunk - 1; ++e)
            if (e < n)
                p[e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
    }
}

// Value e (a constant) of a chunk.
__device__ __forceinline__ float chunk_at(u32x4_t v, int e)
{
    const uint32_t w = v[e >> 1];
    return __builtin_bit_cast(float, (e & 1) ? (w & 0xFFFF0000u) : (w << 16));
}

// 8 values rounded to bf16 (round to nearest even).
__device__ __forceinline__ u32x4_t chunk_bf16(const float (&f)[kChunk])
{
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return v;
}

// ---------------------------------------------------------------------------
// Cross-lane reductions.
// ---------------------------------------------------------------------------
// The value of the lane that DPP control CTRL names.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}

// Lane moves that make a butterfly over a row of 16 lanes: exchange with the
// neighbour, within the quad, mirror the half row (its quads already agree),
// mirror the row (its halves already agree).
constexpr int kDppQuad1 = 0xB1;       // quad_perm [1, 0, 3, 2]
constexpr int kDppQuad2 = 0x4E;       // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;
constexpr int kDppMirror = 0x140;

__device__ __forceinline__ uint32_t row16_max(uint32_t x)
{
    x = max(x, dpp<kDppQuad1>(x));
    x = max(x, dpp<kDppQuad2>(x));
    x = max(x, dpp<kDppHalfMirror>(x));
    return max(x, dpp<kDppMirror>(x));
}

__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t as_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

__device__ __forceinline__ float row16_sum(float x)
{
    x += as_float(dpp<kDppQuad1>(as_bits(x)));
    x += as_float(dpp<kDppQuad2>(as_bits(x)));
    x += as_float(dpp<kDppHalfMirror>(as_bits(x)));
    return x + as_float(dpp<kDppMirror>(as_bits(x)));
}

__device__ __forceinline__ float wave_sum(float x)
{
    x = row16_sum(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// ---------------------------------------------------------------------------
// Quantising a block.
// ---------------------------------------------------------------------------
constexpr float kFp8Max = 448.0f;
constexpr float kMinScale = 0x1p-126f;

// |x| as an unsigned integer: ordered as the magnitudes are, with infinity
// above every number and NaN above infinity, so an integer maximum keeps both.
__device__ __forceinline__ uint32_t magnitude(float x) { return as_bits(x) & 0x7FFFFFFFu; }

struct BlockScale {
    float scale, inv;
};

// The scale of a block whose largest magnitude is `top`.  The lower bound
// keeps 1 / scale finite, for a block of zeros too; NaN passes through.  The
// division by 448 is a product and one residual step, which rounds correctly
// in three instructions instead of a dozen; the reciprocal may be an ulp off
// (quotient corrects for it).
__device__ __forceinline__ BlockScale block_scale(uint32_t top)
{
    constexpr float kInv = 1.0f / kFp8Max;
    const float t = as_float(top), s0 = t * kInv;
    const float s = __builtin_fmaf(__builtin_fmaf(-s0, kFp8Max, t), kInv, s0);
    BlockScale b;
    b.scale = s < kMinScale ? kMinScale : s;
    const float r = __builtin_amdgcn_rcpf(b.scale);
    b.inv = __builtin_fmaf(__builtin_fmaf(-b.scale, r, 1.0f), r, r);
    return b;
}

// y / scale, clamped to the e4m3 range.  The product with the reciprocal is
// off by up to an ulp of fp32, which turns many ties of the 8-bit rounding (a
// bf16 input has plenty of them) into the wrong neighbour; one residual step
// makes the quotient the correctly rounded one at the cost of two fused
// multiply-adds instead of a division's ten instructions.
__device__ __forceinline__ float quotient(float y, const BlockScale& b)
{
    const float q = y * b.inv;
    const float r = __builtin_fmaf(__builtin_fmaf(-q, b.scale, y), b.inv, q);
    return __builtin_amdgcn_fmed3f(r, -kFp8Max, kFp8Max);
}

// Four values to e4m3 bytes (v_cvt_pk_fp8_f32 rounds to nearest even; the
// operands are inside its range, so its overflow mode does not matter).
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

__device__ __forceinline__ u32x2_t chunk_fp8(const float (&y)[kChunk], const BlockScale& b)
{
    u32x2_t v;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        v[i] = pack_fp8x4(quotient(y[4 * i], b), quotient(y[4 * i + 1], b), quotient(y[4 * i + 2], b),
                          quotient(y[4 * i + 3], b));
    return v;
}

// The largest magnitude of the block whose 16 lanes hold one chunk each.
__device__ __forceinline__ uint32_t block_top(const float (&y)[kChunk])
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
        m = max(m, magnitude(y[e]));
    return row16_max(m);
}

// A unit is one block of 128 columns of a row, 16 lanes of one chunk each, so
// that a block's maximum stays inside the unit; a workgroup of 256 takes 16
// units in a row from u0 on.  The row and first column of a lane's chunk.  Only
// the workgroup's first unit is divided in full; the others lie in the same row
// or the next, or, with short rows, a few rows on.
constexpr int kUnits = 256 / kLanes;

__device__ __forceinline__ void unit_place(int64_t u0, int32_t per_row, int64_t& row, int64_t& c)
{
    const int64_t row0 = (u0 >> 32) == 0 ? (int64_t)((uint32_t)u0 / (uint32_t)per_row) : u0 / per_row;
    const uint32_t at = (uint32_t)(u0 - row0 * per_row) + threadIdx.x / kLanes;
    const uint32_t more = per_row >= kUnits ? (at >= (uint32_t)per_row ? 1u : 0u) : at / (uint32_t)per_row;
    row = row0 + more;
    c = (int64_t)(at - more * (uint32_t)per_row) * kBlock + (threadIdx.x & (kLanes - 1)) * kChunk;
}

__device__ __forceinline__ int left(int64_t n, int64_t c)
{
    return n - c >= kChunk ? kChunk : (int)max(n - c, (int64_t)0);
}

// ---------------------------------------------------------------------------
// Host: launch shapes and argument checks.
// ---------------------------------------------------------------------------
// Workgroups for `units` of 16 lanes: one pass up to a limit the launch can
// hold, whole strides beyond.
unsigned unit_grid(int64_t units)
{
    const int64_t n = (units + kUnits - 1) / kUnits;
    return (unsigned)(n < (1 << 22) ? n : (1 << 22));
}

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

// An operand as the checks see it: `rows` rows of `cols` elements of `esz`
// bytes, `ld` elements apart (ld counts only with more than one row).
struct Operand {
    const void* p;
    int64_t rows, cols, ld;
    int esz;

    bool ok_ld() const { return rows <= 1 || (ld >= cols && ld <= kMaxRows); }
    // Its extent, at most 2^62 (ld and rows are below 2^31 and cols below 2^32, so
    // that the elements are countable, but not always their bytes).
    int64_t bytes() const
    {
        constexpr int64_t kMost = (int64_t)1 << 62;
        const int64_t n = rows <= 0 || cols <= 0 ? 0 : rows > 1 ? (rows - 1) * ld + cols : cols;
        return n > kMost / esz ? kMost : n * esz;
    }
};

// The status of one operand with values to read or write.
int check_operand(const Operand& o)
{
    if (!o.p || !o.ok_ld())
        return GEMM_ERR_INVALID_VALUE;
    return ((uintptr_t)o.p & (uintptr_t)(o.esz - 1)) ? GEMM_ERR_MISALIGNED : GEMM_OK;
}

bool same_memory(const Operand& a, const Operand& b)
{
    return a.p == b.p && a.esz == b.esz && a.rows == b.rows && a.cols == b.cols && (a.ld == b.ld || a.rows <= 1);
}

bool meet(const Operand& a, const Operand& b)
{
    return a.p && b.p && overlaps(a.p, a.bytes(), b.p, b.bytes());
}

// The first bad status of `n` operands that are all read or written.
int check_operands(const Operand* o, int n)
{
    for (int i = 0; i < n; ++i)
        if (const int rc = check_operand(o[i]))
            return rc;
    return GEMM_OK;
}

int launched() { return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

}  // namespace
