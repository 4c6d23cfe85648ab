// Linear layers on the bf16 product (part of library.hip): bias, activation,
// residual and gate in the product's epilogue, and the products of the backward
// pass.
//
//   linear                y = act(x w^T + bias) + residual
//   linear, input's grad  dx = (dy w + dres) act'(z)
//   linear, weight's grad dw = dy^T x,  dbias = column sums of dy
//   gated                 y = act(g) u,  [g, u] = x [wg; wu]^T + bias
//   gated, input's grad   dg = t u act'(g),  du = t act(g),  t = dy w
//
// The main loops are the bf16 product's (k_gemm_win, k_gemm): these operators are
// parameter types with a store_tile of their own, and configurations that load A
// stored K x M (the weight's gradient contracts over the rows of both operands)
// and B as two factors whose 16-row blocks alternate, so that one wave holds g and
// u of the same elements.
#pragma once

namespace {

enum { FUSE_LINEAR, FUSE_DX, FUSE_DW, FUSE_GATED, FUSE_DGATED };

constexpr bool fuse_paired(int mode) { return mode == FUSE_GATED; }

// What an epilogue reads and writes, row-major with `ld` elements between rows.
//   LINEAR  in0 residual, out0 y, out1 z              (bias)
//   DX      in0 z, in1 dres, out0 dx
//   DW      out0 dw (fp32 or bf16)
//   GATED   out0 y, out1 [g, u]                       (bias)
//   DGATED  in0 [g, u], out0 [dg, du], out1 y
// All but LINEAR's y, DX's dx, DW's dw, GATED's y and DGATED's in0 and out0 may be
// null.
struct Epilogue {
    const uint16_t* bias;
    const uint16_t* in0;
    const uint16_t* in1;
    void* out0;
    uint16_t* out1;
    int64_t ld_in0, ld_in1, ld_out0, ld_out1;
    int64_t M, N;            // of the output (a gated unit's N: of one factor)
    int32_t act;
    int32_t fp32;            // DW: dw is fp32
};

// ---------------------------------------------------------------------------
// The elementwise part: 8 consecutive columns of one row, from fp32 sums.
// ---------------------------------------------------------------------------
struct EpilogueIn {
    u32x4_t a, b;
};

// Outputs go out non-temporal, as the product's C does (see Cfg::STORE_C).
typedef u32x4_t __attribute__((aligned(2))) u32x4_any_t;
typedef f32x4_t __attribute__((aligned(4))) f32x4_any_t;

// A chunk without its first n (< 8) elements, zeros behind the others.
__device__ __forceinline__ u32x4_t shifted_chunk(u32x4_t v, int n)
{
    uint64_t x[2];
    __builtin_memcpy(x, &v, 16);
    const int s = 16 * n;
    const uint64_t lo = s >= 64 ? x[1] : x[0], hi = s >= 64 ? 0u : x[1];
    x[0] = (s & 63) ? (lo >> (s & 63)) | (hi << (64 - (s & 63))) : lo;
    x[1] = hi >> (s & 63);
    __builtin_memcpy(&v, x, 16);
    return v;
}

// Where a chunk is: 8 columns from c on, the n (<= 8) of them that exist, of row
// `row`, in matrices of any alignment and stride.
struct ChunkAt {
    int64_t row, c;
    int n;

    __device__ __forceinline__ bool any() const { return n > 0; }
    __device__ __forceinline__ u32x4_t load(const uint16_t* base, int64_t ld) const
    {
        return load_chunk<false>(base + row * ld + c, n, c);
    }
    __device__ __forceinline__ u32x4_t placed(u32x4_t v) const { return v; }
    __device__ __forceinline__ void store(uint16_t* base, int64_t ld, u32x4_t v) const
    {
        uint16_t* p = base + row * ld + c;
        if (n >= kChunk)
            __builtin_nontemporal_store(v, (u32x4_any_t*)p);
        else
            store_chunk<false>(p, n, v);
    }
};

// The same for 8 rows of a tile, from `first` (uniform) on, without branches: a branch
// that may skip a store makes a loop's next wait for a load wait for every store
// before it (4 us a tile).  The resource ends with the matrix's last row, and an offset
// past it drops a lane of columns that do not exist.  `part` (uniform): the columns end
// inside a chunk, which is loaded from the row's last 16 bytes and stored by element.
// For leading dimensions up to kMaxTileLd and rows of 8 and more.
constexpr int64_t kMaxTileLd = (int64_t)1 << 27;

struct TileAt {
    int64_t first, rows;     // the first row, and how many exist from there on
    int32_t cols;            // of the matrix
    int32_t lane_row, c;     // this lane's, c < cols + 256
    bool part;

    __device__ __forceinline__ int n() const { return min(max(cols - c, 0), kChunk); }
    __device__ __forceinline__ bool any() const { return true; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint16_t* base, int64_t ld) const
    {
        return make_rsrc(base + first * ld, rows <= 0 ? 0 : ((rows - 1) * ld + cols) * 2);
    }
    __device__ __forceinline__ uint32_t offset(int64_t ld, int32_t col) const
    {
        return ((uint32_t)lane_row * (uint32_t)ld + (uint32_t)col) * 2u;
    }
    __device__ __forceinline__ u32x4_t load(const uint16_t* base, int64_t ld) const
    {
        const int m = n();
        const uint32_t at = offset(ld, part ? min(c, cols - kChunk) : c);
        return __builtin_bit_cast(u32x4_t,
                                  __builtin_amdgcn_raw_buffer_load_b128(rsrc(base, ld), m > 0 ? at : kOOB, 0, 0));
    }
    // What was loaded, in place.  Not in load: it would wait for the load there.
    __device__ __forceinline__ u32x4_t placed(u32x4_t v) const
    {
        return part ? shifted_chunk(v, (kChunk - n()) & 7) : v;   // lanes of whole chunks: 0
    }
    __device__ __forceinline__ void store(uint16_t* base, int64_t ld, u32x4_t v) const
    {
        const __amdgpu_buffer_rsrc_t r = rsrc(base, ld);
        const int m = n();
        const uint32_t at = offset(ld, c);
        __builtin_amdgcn_raw_buffer_store_b128(v, r, m >= kChunk ? at : kOOB, 0, kStoreNonTemporal);
        if (part) {
#pragma unroll
            for (int i = 0; i < kChunk - 1; ++i)
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[i >> 1] >> (16 * (i & 1))), r,
                                                      m < kChunk && i < m ? at + 2 * i : kOOB, 0, 0);
        }
    }
};

template <int MODE, class At>
__device__ __forceinline__ EpilogueIn epilogue_load(const Epilogue& e, const At& at)
{
    EpilogueIn in;
    if constexpr (MODE == FUSE_LINEAR || MODE == FUSE_DX) {
        if (e.in0)
            in.a = at.load(e.in0, e.ld_in0);
    }
    if constexpr (MODE == FUSE_DX) {
        if (e.in1)
            in.b = at.load(e.in1, e.ld_in1);
    }
    if constexpr (MODE == FUSE_DGATED) {
        in.a = at.load(e.in0, e.ld_in0);
        in.b = at.load(e.in0 + e.N, e.ld_in0);
    }
    return in;
}

// The biases of the columns of `at`, a chunk of the first of one row.
template <int MODE, class At>
__device__ __forceinline__ EpilogueIn epilogue_bias(const Epilogue& e, const At& at)
{
    EpilogueIn b{};
    if constexpr (MODE == FUSE_LINEAR || MODE == FUSE_GATED) {
        if (e.bias) {
            b.a = at.load(e.bias, 0);
            if constexpr (MODE == FUSE_GATED)
                b.b = at.load(e.bias + e.N, 0);
        }
    }
    return b;
}

__device__ __forceinline__ void chunk_values(float (&v)[kChunk], u32x4_t x)
{
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
        v[e] = chunk_at(x, e);
}

__device__ __forceinline__ void add_chunk(float (&v)[kChunk], u32x4_t x)
{
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
        v[e] += chunk_at(x, e);
}

// s: the sums (GATED: of the gate, and t those of the other factor).  `next` is called
// once what was read is in use, to read again.
template <int MODE, class At, class F>
__device__ __forceinline__ void epilogue_finish(const Epilogue& e, const EpilogueIn& in, const EpilogueIn& bias,
                                                const At& at, float (&s)[kChunk], float (&t)[kChunk], F&& next)
{
    if (!at.any())
        return;
    uint16_t* out = (uint16_t*)e.out0;   // not DW's, which may be fp32
    float a[kChunk], b[kChunk], o[kChunk], r[kChunk];
    if constexpr (MODE == FUSE_LINEAR) {
        if (e.in0)
            chunk_values(a, at.placed(in.a));
        next();
        add_chunk(s, at.placed(bias.a));
        if (e.out1)
            at.store(e.out1, e.ld_out1, chunk_bf16(s));
        activate<false>(e.act, s, [&](int i, const auto& x) { o[i] = x.times(1.0f); });
        if (e.in0) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                o[i] += a[i];
        }
        at.store(out, e.ld_out0, chunk_bf16(o));
    }
    if constexpr (MODE == FUSE_DX) {
        if (e.in1)
            add_chunk(s, at.placed(in.b));
        if (e.in0) {
            chunk_values(a, at.placed(in.a));
            next();
            activate<true>(e.act, a, [&](int i, const auto& x) { o[i] = x.slope_times(s[i]); });
            at.store(out, e.ld_out0, chunk_bf16(o));
        } else {
            next();
            at.store(out, e.ld_out0, chunk_bf16(s));
        }
    }
    if constexpr (MODE == FUSE_DW) {
        if constexpr (std::is_same_v<At, ChunkAt>) {   // a tile's fp32 sums take a way of their own
            if (e.fp32) {
                float* p = (float*)e.out0 + at.row * e.ld_out0 + at.c;
                if (at.n >= kChunk) {
                    __builtin_nontemporal_store(f32x4_t{s[0], s[1], s[2], s[3]}, (f32x4_any_t*)p);
                    __builtin_nontemporal_store(f32x4_t{s[4], s[5], s[6], s[7]}, (f32x4_any_t*)(p + 4));
                } else {
#pragma unroll
                    for (int i = 0; i < kChunk - 1; ++i)
                        if (i < at.n)
                            p[i] = s[i];
                }
                return;
            }
        }
        at.store(out, e.ld_out0, chunk_bf16(s));
    }
    if constexpr (MODE == FUSE_GATED) {
        add_chunk(s, at.placed(bias.a));
        add_chunk(t, at.placed(bias.b));
        if (e.out1) {
            at.store(e.out1, e.ld_out1, chunk_bf16(s));
            at.store(e.out1 + e.N, e.ld_out1, chunk_bf16(t));
        }
        activate<false>(e.act, s, [&](int i, const auto& x) { o[i] = x.times(t[i]); });
        at.store(out, e.ld_out0, chunk_bf16(o));
    }
    if constexpr (MODE == FUSE_DGATED) {
        chunk_values(a, at.placed(in.a));
        chunk_values(b, at.placed(in.b));
        next();
        float y[kChunk];
        activate<true>(e.act, a, [&](int i, const auto& x) {
            o[i] = x.slope_times(s[i], b[i]);
            r[i] = x.times(s[i]);
            y[i] = x.times(b[i]);
        });
        if (e.out1)
            at.store(e.out1, e.ld_out1, chunk_bf16(y));
        at.store(out, e.ld_out0, chunk_bf16(o));
        at.store(out + e.N, e.ld_out0, chunk_bf16(r));
    }
}

// ---------------------------------------------------------------------------
// Tiles.
// ---------------------------------------------------------------------------
// 256 x 256 tiles on the split-window ring, 8 waves: the bf16 product's default.
// 192 x 256 tiles on the same ring, where A is K-contiguous and B one matrix: a round
// of them takes 0.84 of the time, for sizes that leave fewer compute units idle so
// (6952 x 1344 x 5952: 222 tiles 103 us, 168 of 256 rows 123; 4088 x 7608 x 1728: 3
// rounds 116, 2 of 256 rows 102).
// 128 x 128 tiles on a four-stage ring, 8 waves (4 where B is paired: a wave needs both
// factors' 64 columns), where those give the compute units too little to share (1936 x
// 1024 x 1216: 15 us, 29 in tiles of 192 rows and k chunks; 1400 x 2272 x 3200: 29 and
// 39; but 8200 x 1856 x 960 46 and 47, 6952 x 1344 x 5952 139 and 103).
enum { TILES_BIG, TILES_192, TILES_SMALL, TILES_WAVE };

template <bool BT_, bool AT_, bool PAIRED_, int KIND_>
struct LinearCfg : Cfg<KIND_ == TILES_192 ? 192 : 256, 256, 64, 2, PAIRED_ ? 4 : 2, PAIRED_ ? 2 : 4, SYNC_BARRIER, BT_, 0,
                       true, 16> {
    static_assert(KIND_ == TILES_BIG || (!AT_ && !PAIRED_), "192 rows: 96 a wave, of a K-contiguous A");
    static constexpr bool AT = AT_, PAIRED = PAIRED_, ANY_SIZE = true;
};

template <bool BT_, bool AT_, bool PAIRED_>
struct LinearCfg<BT_, AT_, PAIRED_, TILES_SMALL>
    : Cfg<128, 128, 64, 4, 4, PAIRED_ ? 1 : 2, SYNC_BARRIER, BT_, 0, false, 16> {
    static constexpr bool AT = AT_, PAIRED = PAIRED_, ANY_SIZE = true;
};
static_assert(LinearCfg<true, false, false, TILES_BIG>::THREADS == 512 && LinearCfg<true, false, true, TILES_BIG>::THREADS == 512 &&
                  LinearCfg<true, false, false, TILES_192>::THREADS == 512,
              "8 waves, as k_linear_wave (gemm_linear_plan_cus)");

// Sums of the k chunks: chunk sp's of the launch's u-th tile are piece sp * span +
// u of the workspace, a tile's rows (of both factors, one after the other) in fp32.
template <int MODE>
struct LinearParams : Params {
    Epilogue e;

    // What an epilogue reads and writes beside the accumulators bounds it first: 8192 x 8192
    // over 4096 takes 407 us as a plain gradient, 435 through relu and 437 through silu (134 MB
    // more), 470 with both factors' (268 MB more each way), since all workgroups reach theirs
    // at about the same time, and then wait for memory.  Activations with more steps add to that
    // (gelu 450, and activations.h).
    //
    // The accumulators, 8 rows by 64 columns of each factor at a time, through the
    // wave's strip of LDS into rows, 8 consecutive columns a lane.  A rolled loop,
    // whose rounds differ only in the accumulators that a uniform switch picks, so
    // that the elementwise part is there once, with every activation in it.  (Loads three
    // and four rounds ahead instead of two were no faster.)
    //
    // Strip: 16 rows of 256 bytes, the 16-byte chunk XORed with the row: 16 rows of
    // one factor, written every other round, or 8 rows of both.  A write's 16 lanes
    // of one column group hold 16 rows (8 of both), a read's 16 lanes two rows at
    // chunks of one parity: either way all chunks differ, and with them all banks.
    template <class C>
    __device__ __forceinline__ void store_tile(typename C::Acc (&acc)[C::FM][C::FN], lds_char* strip, int32_t tm,
                                               int32_t tn, int32_t piece, int wm, int wn, int lane_in) const
    {
        constexpr int FACTORS = fuse_paired(MODE) ? 2 : 1, BNO = C::BN / FACTORS;   // output columns of a tile
        const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * BNO;
        if (partial || (MODE == FUSE_DW && e.fp32))
            store_rows<C, true>(acc, strip, m0, n0, piece, wm, wn, lane_in);
        else
            store_rows<C, false>(acc, strip, m0, n0, piece, wm, wn, lane_in);
    }

    template <class C, bool SUMS>
    __device__ __forceinline__ void store_rows(typename C::Acc (&acc)[C::FM][C::FN], lds_char* strip, int64_t m0,
                                               int64_t n0, int32_t piece, int wm, int wn, int lane_in) const
    {
        constexpr bool PAIR = fuse_paired(MODE);
        static_assert(C::PAIRED == PAIR && C::EPI_WAVE_BYTES == 16 * 64 * 4, "the strip");
        constexpr int FACTORS = PAIR ? 2 : 1, ROUNDS = C::FM * 2, BNO = C::BN / FACTORS;
        static_assert(C::FN == 4 * FACTORS && ROUNDS <= 16, "64 columns of a factor per wave");
        const int lane = (int)opaque((uint32_t)lane_in);
        const int wrow = lane & 15, wq = lane >> 4, rrow = lane >> 3, c8 = lane & 7;
        const int32_t r0 = wm * C::TM, w0 = wn * (C::TN / FACTORS);
        // The rows of `round`, written with its pass's first round, or, of two factors, by
        // the lanes that hold them.  A wave's LDS operations complete in order, so neither
        // writes nor reads are waited for before the others.
        auto write = [&](int round) {
            const int half = round & 1;
            if (PAIR ? (wrow >> 3) == half : half == 0) {
                auto pass = [&]<int P>() {
                    if constexpr (P < ROUNDS / 2) {
#pragma unroll
                        for (int h = 0; h < FACTORS; ++h)
#pragma unroll
                            for (int jj = 0; jj < 4; ++jj) {
                                const int row = PAIR ? (wrow & 7) + 8 * h : wrow;
                                *(LDS_AS f32x4_t*)(strip + row * 256 + (((4 * jj + wq) ^ row) << 4)) =
                                    acc[P][jj * FACTORS + h];
                            }
                        // Tells the cases apart: merged, they would index the accumulators.
                        asm volatile("; rows %0" ::"n"(P));
                    }
                };
                switch (round >> 1) {
                case 0: pass.template operator()<0>(); break;
                case 1: pass.template operator()<1>(); break;
                case 2: pass.template operator()<2>(); break;
                case 3: pass.template operator()<3>(); break;
                case 4: pass.template operator()<4>(); break;
                case 5: pass.template operator()<5>(); break;
                case 6: pass.template operator()<6>(); break;
                default: pass.template operator()<7>(); break;
                }
            }
            COMPILER_FENCE();
        };
        auto strip_row = [&](int round, int h) { return rrow + 8 * (PAIR ? h : round & 1); };
        if constexpr (SUMS) {
            // fp32 sums as they are, 4 columns a lane, whole 128-byte lines a store: columns
            // 4 c8 .. and, 32 further, the others, in this order in even rows (whose reads then
            // meet the odd rows' on no bank).
            const bool whole = !partial;
            const int64_t ld = whole ? e.ld_out0 : BNO, c = (whole ? n0 : 0) + w0 + 4 * c8;
            float* out = whole ? (float*)e.out0 + (m0 + r0) * ld
                               : partial + (int64_t)piece * (C::BM * BNO * FACTORS) + (int64_t)r0 * ld;
#pragma clang loop unroll(disable)
            for (int round = 0; round < ROUNDS; ++round) {
                write(round);
                const bool in_rows = !whole || rrow < e.M - (m0 + r0 + 8 * round);
#pragma unroll
                for (int h = 0; h < FACTORS; ++h) {
                    const int row = strip_row(round, h);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int second = q ^ (rrow & 1);
                        const f32x4_t x = *(const LDS_AS f32x4_t*)(strip + row * 256 + (((c8 + 8 * second) ^ row) << 4));
                        const int64_t col = c + 32 * second, n = whole ? e.N - col : 4;
                        float* to = out + h * (C::BM * BNO) + (rrow * ld + col);
                        if (!in_rows)
                            continue;
                        if (!whole)
                            *(f32x4_t*)to = x;
                        else if (n >= 4)
                            __builtin_nontemporal_store(x, (f32x4_any_t*)to);
                        else
#pragma unroll
                            for (int i = 0; i < 3; ++i)
                                if (i < n)
                                    to[i] = x[i];
                    }
                }
                COMPILER_FENCE();
                out += 8 * ld;
            }
        } else {
            const int32_t cols = (int32_t)e.N, c = (int32_t)n0 + w0 + c8 * kChunk;
            const bool part = cols % kChunk != 0 && cols - (int32_t)n0 - w0 < 64;
            auto at = [&](int round) {
                const int64_t first = m0 + r0 + 8 * round;
                return TileAt{first, e.M - first, cols, rrow, c, part};
            };
            const EpilogueIn bias = epilogue_bias<MODE>(e, TileAt{0, 1, cols, 0, c, part});
            // What a round reads is on its way two rounds before.
            EpilogueIn in[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                in[i] = epilogue_load<MODE>(e, at(i));
            auto one = [&](EpilogueIn& now, int round) {
                write(round);
                float v[FACTORS][kChunk];
#pragma unroll
                for (int h = 0; h < FACTORS; ++h) {
                    const int row = strip_row(round, h);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const f32x4_t x = *(const LDS_AS f32x4_t*)(strip + row * 256 + (((2 * c8 + q) ^ row) << 4));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[h][4 * q + i] = x[i];
                    }
                }
                COMPILER_FENCE();
                // Past the last round the last rows are read again, and not used.
                auto next = [&] { now = epilogue_load<MODE>(e, at(min(round + 2, ROUNDS - 1))); };
                epilogue_finish<MODE>(e, now, bias, at(round), v[0], v[FACTORS - 1], next);
            };
#pragma clang loop unroll(disable)
            for (int round = 0; round < ROUNDS; round += 2) {
                one(in[0], round);
                one(in[1], round + 1);
            }
        }
    }
};

// Sums of columns in parts: part[r * cols + c], r = 0 .. runs - 1, added in order.
struct ColumnSums {
    const float* part;
    float* to;
    int64_t cols;
    int32_t runs;
    unsigned blocks;   // of 16 columns, that add them
};

__device__ __forceinline__ void join_column_sums(const ColumnSums& p, unsigned block)
{
    __shared__ float sums[16][16];
    const int cl = threadIdx.x & 15, rl = threadIdx.x >> 4;
    const int64_t c = (int64_t)block * 16 + cl;
    float t = 0.0f;
    if (c < p.cols) {
#pragma unroll 4
        for (int32_t r = rl; r < p.runs; r += 16)
            t += p.part[r * p.cols + c];
    }
    sums[rl][cl] = t;
    __syncthreads();
    if (rl == 0 && c < p.cols) {
        t = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            t += sums[r][cl];
        p.to[c] = t;
    }
}

__global__ void __launch_bounds__(256) k_join_column_sums(ColumnSums p) { join_column_sums(p, blockIdx.x); }

// The epilogue over the sums of k chunks, added in chunk order (with no chunk, K ==
// 0: over zeros), for the launch's span of tiles of bm x bn outputs.  A thread takes 8
// columns, of fp32 results 4, so that its stores are next to its neighbours'.  The
// first blocks add the column sums of a weight's gradient, where there are any.  Bound by
// the sums' bytes: 1024 x 1024 in 16 chunks 12.8 us, 5.3 TB/s; 300 x 1000 in 3 chunks 4.5.
template <int MODE>
__global__ void __launch_bounds__(256) k_linear_finish(LinearParams<MODE> p, int32_t bm, int32_t bn, ColumnSums sums)
{
    if (blockIdx.x < sums.blocks) {
        join_column_sums(sums, blockIdx.x);
        return;
    }
    constexpr int FACTORS = fuse_paired(MODE) ? 2 : 1;
    const bool fp32 = MODE == FUSE_DW && p.e.fp32;
    const int32_t width = fp32 ? 4 : kChunk, per_row = bn / width, units = bm * per_row;
    const int64_t total = (int64_t)p.span * units, piece = (int64_t)bm * bn * FACTORS;
    for (int64_t q = (int64_t)(blockIdx.x - sums.blocks) * 256 + threadIdx.x; q < total;
         q += (int64_t)(gridDim.x - sums.blocks) * 256) {
        const int32_t u = (int32_t)(q / units), at = (int32_t)(q - (int64_t)u * units), r = at / per_row;
        const int32_t cc = (at - r * per_row) * width;
        int32_t tm, tn;
        raster_tile(p, p.tile_base + u, tm, tn);
        const int64_t c = (int64_t)tn * bn + cc, row = (int64_t)tm * bm + r;
        if (row >= p.e.M || c >= p.e.N)
            continue;
        const float* first = p.partial + u * piece + (int64_t)r * bn + cc;
        if (fp32) {
            f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
            for (int32_t sp = 0; sp < p.splits; ++sp)
                v += *(const f32x4_t*)(first + sp * (int64_t)p.span * piece);
            float* to = (float*)p.e.out0 + row * p.e.ld_out0 + c;
            if (p.e.N - c >= 4)
                __builtin_nontemporal_store(v, (f32x4_any_t*)to);
            else
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < p.e.N - c)
                        to[i] = v[i];
            continue;
        }
        const ChunkAt here{row, c, left(p.e.N, c)};
        const EpilogueIn in = epilogue_load<MODE>(p.e, here);
        float v[2][kChunk] = {};
#pragma unroll 4
        for (int32_t sp = 0; sp < p.splits; ++sp) {
            const float* src = first + sp * (int64_t)p.span * piece;
#pragma unroll
            for (int h = 0; h < FACTORS; ++h) {
                float x[kChunk];
                __builtin_memcpy(x, src + (int64_t)h * bm * bn, 32);
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    v[h][i] += x[i];
            }
        }
        epilogue_finish<MODE>(p.e, in, epilogue_bias<MODE>(p.e, ChunkAt{0, here.c, here.n}), here, v[0], v[1], [] {});
    }
}

// ---------------------------------------------------------------------------
// Small products and few rows, which latency or one operand's bytes bound: the 8
// waves of a workgroup share out the 64-wide blocks along k (wave w takes blocks w, w
// + 8, ...) of 16 MF rows by 16 NF columns (of each factor) and add their sums through
// LDS in wave order.  So a workgroup has loads in flight over the whole of k, nothing
// waits for another wave before the end, and there is little code to fetch (a launch
// of the tiles' kernel takes 5 us longer for that alone).  512 x 512 x 512: 9 us, 11 in
// tiles; the gated gradient of 25 x 72 over 1344 9.5 and 19.  One row reads the weight at
// 5 TB/s (8192 x 4096 in 13 us); 300 x 1000 x 4112 takes 13.9 in 240 workgroups that load
// 138 MB, 27 of them from memory: each wave has two or three blocks in series, and which
// of the start, the loads and the join is the time was not separated.
//
// A wave loads DEPTH blocks ahead into registers, a block's 16-byte chunks in rows
// (lanes 8 i .. 8 i + 7 a row's 128 bytes), writes them to LDS of its own and reads
// MFMA fragments back: plain reads where k is contiguous, transposing ones where it
// is not.  A wave's LDS operations complete in order, so there is nothing to wait
// for but the loads.  EVEN: operands as the tiles read them (rows of whole 16-byte
// chunks on 16-byte boundaries), by range-checked loads; otherwise any alignment and
// stride, by 16-byte loads at any byte, and a row's last chunk from its last bytes.
//
// Swizzles of a 64-row block: with k along the rows of 128 bytes as the tiles' (swz_k:
// a read's 16 lanes hold 16 rows at one chunk).  With k across, a transposing read's 32
// lanes hold rows r, r + 8 (r = 0 .. 3) at two chunks, and rows of one parity share
// the same banks: the chunk's pair is XORed with bits 1 and 3 of the row.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;

__device__ __forceinline__ int swz_across(int krow) { return (krow & 2) | ((krow >> 1) & 4); }

// One operand's part of a wave: 16 X rows (columns, where k is across) of it.
template <int X, bool ACROSS, bool EVEN>
struct WaveOperand {
    static_assert(!ACROSS || X == 4, "rows of 128 bytes");
    const uint16_t* base;   // the first row's (column's) k = 0
    const uint16_t* end;    // EVEN, across: past the last row's last whole chunk
    int64_t ld, first;      // first: column of `base`, across
    int32_t count, K;       // rows (columns) that exist from base on
    __amdgpu_buffer_rsrc_t rsrc;

    __device__ __forceinline__ WaveOperand(const char* p, int64_t ld_, int64_t at, int64_t total, int64_t k)
    {
        ld = ld_;
        first = ACROSS ? at : 0;
        count = (int32_t)min(total - at, (int64_t)X * 16);
        K = (int32_t)k;
        base = (const uint16_t*)p + (ACROSS ? at : at * ld);
        if constexpr (EVEN) {
            if constexpr (ACROSS)
                end = (const uint16_t*)p + (k - 1) * ld + total;
            else
                rsrc = make_rsrc(base, ((count - 1) * ld + k) * 2);
        }
    }

    __device__ __forceinline__ void load(u32x4_t (&v)[2 * X], int32_t kb) const
    {
        const int lane = threadIdx.x & 63, lr = lane >> 3, lc = lane & 7;
        if constexpr (EVEN) {
            const __amdgpu_buffer_rsrc_t r =
                ACROSS ? make_rsrc(base + (int64_t)kb * 64 * ld, (end - (base + (int64_t)kb * 64 * ld)) * 2) : rsrc;
            const bool in = ACROSS ? lc * 8 < count : kb * 64 + lc * 8 < K;
#pragma unroll
            for (int t = 0; t < 2 * X; ++t) {
                const int row = 8 * t + lr;
                const bool ok = in && (ACROSS || row < count);
                v[t] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                    r, ok ? (uint32_t)row * (uint32_t)(ld * 2) + lc * 16 : kOOB, ACROSS ? 0 : kb * 128, 0));
            }
        } else {
#pragma unroll
            for (int t = 0; t < 2 * X; ++t) {
                const int row = 8 * t + lr;
                if constexpr (ACROSS) {
                    const int64_t k = (int64_t)kb * 64 + row;
                    v[t] = load_chunk<false>(base + k * ld + lc * 8, k < K ? left(count, lc * 8) : 0, first + lc * 8);
                } else {
                    const int32_t k = kb * 64 + lc * 8;
                    v[t] = load_chunk<false>(base + row * ld + k, row < count ? left(K, k) : 0, k);
                }
            }
        }
    }

    __device__ __forceinline__ void stage(lds_char* to, const u32x4_t (&v)[2 * X]) const
    {
        const int lane = threadIdx.x & 63, lr = lane >> 3, lc = lane & 7;
#pragma unroll
        for (int t = 0; t < 2 * X; ++t) {
            const int row = 8 * t + lr;
            *(LDS_AS u32x4_t*)(to + row * 128 + ((lc ^ (ACROSS ? swz_across(row) : swz_k<64>(row))) << 4)) = v[t];
        }
    }

    // Fragments of k-step ks (32 wide).
    __device__ __forceinline__ void fragments(bf16x8_t (&f)[X], const lds_char* from, int ks) const
    {
        const int lane = threadIdx.x & 63, r16 = lane & 15, h = lane >> 4;
#pragma unroll
        for (int i = 0; i < X; ++i) {
            if constexpr (ACROSS) {
                const int rr = r16 >> 2, q = r16 & 3;
                i16x4_t half[2];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int krow = 32 * ks + 8 * h + 4 * hh + rr;
                    half[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (LDS_AS i16x4_t*)(from + krow * 128 + (((2 * i + (q >> 1)) ^ swz_across(krow)) << 4) + (q & 1) * 8));
                }
                f[i] = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                const int row = 16 * i + r16;
                f[i] = *(const LDS_AS bf16x8_t*)(from + row * 128 + (((4 * ks + h) ^ swz_k<64>(row)) << 4));
            }
        }
    }
};

template <int MODE, int MF, int NF, int DEPTH, bool EVEN>
__global__ void __launch_bounds__(kWaves * 64) k_linear_wave(LinearParams<MODE> p, int32_t chunk, int32_t kblocks)
{
    constexpr bool AT = MODE == FUSE_DW, BT = MODE == FUSE_LINEAR || MODE == FUSE_GATED;
    constexpr int FACTORS = fuse_paired(MODE) ? 2 : 1, NB = NF * FACTORS, FR = MF * NB;
    constexpr int A_BYTES = MF * 2048, B_BYTES = NF * 2048;
    constexpr int WAVE_BYTES = std::max(A_BYTES + FACTORS * B_BYTES, FR * 1024);
    __shared__ __attribute__((aligned(1024))) char smem[kWaves * WAVE_BYTES];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups are dealt to the 8 XCDs in turn; each XCD takes a run of tiles, column by
    // column, so that the row tiles of a column tile share its L2.
    const int32_t at_tile = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    if (at_tile >= p.span)
        return;
    const int32_t tn = at_tile / p.tiles_m, tm = at_tile - tn * p.tiles_m;
    const int64_t m0 = (int64_t)tm * (MF * 16), n0 = (int64_t)tn * (NF * 16);
    const int32_t kb_first = blockIdx.y * chunk, kb_end = min(kb_first + chunk, kblocks);
    const WaveOperand<MF, AT, EVEN> oa(p.A, p.lda, m0, p.M, p.K);
    const WaveOperand<NF, !BT, EVEN> ob[2] = {{p.B, p.ldb, n0, p.N, p.K},
                                              {p.B + (FACTORS - 1) * p.N * p.ldb * 2, p.ldb, n0, p.N, p.K}};
    lds_char* own = (lds_char*)smem + w * WAVE_BYTES;

    struct Block {
        u32x4_t a[2 * MF], b[FACTORS][2 * NF];
    };
    Block ahead[DEPTH];
    // Workgroups start at different places along k: with a power-of-two row stride,
    // all of them reading the same columns at once fall on the same few channels.
    const int32_t mine = (kb_end - kb_first - w + kWaves - 1) / kWaves;   // blocks of this wave
    const int32_t rot = mine > 0 ? (int32_t)(blockIdx.x % (unsigned)mine) : 0;
    auto load = [&](Block& v, int32_t t) {
        if (t < mine) {
            const int32_t kb = kb_first + w + (t + rot < mine ? t + rot : t + rot - mine) * kWaves;
#pragma unroll
            for (int h = 0; h < FACTORS; ++h)
                ob[h].load(v.b[h], kb);
            oa.load(v.a, kb);
        }
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load(ahead[d], d);
    f32x4_t acc[MF][NB];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t t0 = 0; t0 < mine; t0 += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (DEPTH > 1 && t0 + d >= mine)
                break;
            oa.stage(own, ahead[d].a);
#pragma unroll
            for (int h = 0; h < FACTORS; ++h)
                ob[h].stage(own + A_BYTES + h * B_BYTES, ahead[d].b[h]);
            load(ahead[d], t0 + d + DEPTH);
            COMPILER_FENCE();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bf16x8_t af[MF], bf[FACTORS][NF];
                oa.fragments(af, own, ks);
#pragma unroll
                for (int h = 0; h < FACTORS; ++h)
                    ob[h].fragments(bf[h], own + A_BYTES + h * B_BYTES, ks);
#pragma unroll
                for (int i = 0; i < MF; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j / NF][j % NF], af[i], acc[i][j], 0, 0, 0);
            }
            COMPILER_FENCE();
        }
    }

#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *(LDS_AS f32x4_t*)(own + (i * NB + j) * 1024 + lane * 16) = acc[i][j];
    __syncthreads();
    // Wave w finishes fragments w, w + 8, ... of one factor with the other's beside
    // them.  Lanes of even g hold columns 8 (g / 2) .. + 3 and get + 4 .. + 7 from the
    // lane 16 further.
    for (int f = w; f < MF * NF; f += kWaves) {
        const int i = f / NF, j = f % NF;
        const int r = i * 16 + r16, cc = j * 16 + g * 4;
        const ChunkAt here{m0 + r, n0 + cc, (g & 1) || m0 + r >= p.e.M ? 0 : left(p.e.N, n0 + cc)};
        EpilogueIn in{};
        if (!p.partial)
            in = epilogue_load<MODE>(p.e, here);
        float v[2][kChunk];
#pragma unroll
        for (int h = 0; h < FACTORS; ++h) {
            const lds_char* from = (lds_char*)smem + (i * NB + h * NF + j) * 1024 + lane * 16;
            f32x4_t s = *(const LDS_AS f32x4_t*)from;
#pragma unroll
            for (int z = 1; z < kWaves; ++z)
                s += *(const LDS_AS f32x4_t*)(from + z * WAVE_BYTES);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[h][q] = s[q];
                v[h][4 + q] = __shfl_xor(s[q], 16);
            }
        }
        if (g & 1)
            continue;
        if (p.partial) {
            const int64_t piece = (int64_t)blockIdx.y * p.span + (tn * p.tiles_m + tm);
            float* to = p.partial + piece * (MF * 16 * NF * 16 * FACTORS) + r * (NF * 16) + cc;
#pragma unroll
            for (int h = 0; h < FACTORS; ++h)
                __builtin_memcpy(to + h * (MF * 16 * NF * 16), v[h], 32);
        } else {
            epilogue_finish<MODE>(p.e, in, epilogue_bias<MODE>(p.e, ChunkAt{0, here.c, here.n}), here, v[0], v[1], [] {});
        }
    }
}

// ---------------------------------------------------------------------------
// Column sums of bf16 X (rows x cols) in fp32: dbias.  A workgroup sums 64 columns of a
// run of rows, `threads` / 8 rows at a time; runs are added in order (ColumnSums).
// Up to kOneRun rows a workgroup of 1024 takes them all: the second launch would take
// longer.  Bound by the bytes, after some 5 us of start and end: 32768 x 1024 in 18 us.
// ---------------------------------------------------------------------------
constexpr int64_t kOneRun = 512;

__global__ void __launch_bounds__(1024) k_column_sums(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld,
                                                      int64_t run, float* to)
{
    __shared__ float sums[128][65];
    const int cl = threadIdx.x & 7, rl = threadIdx.x >> 3, step = blockDim.x >> 3;
    const int64_t c = ((int64_t)blockIdx.x * 8 + cl) * kChunk;
    const int n = left(cols, c);
    const int64_t first = (int64_t)blockIdx.y * run, end = min(first + run, rows);
    float s[kChunk] = {};
#pragma unroll 4
    for (int64_t r = first + rl; r < end; r += step)
        add_chunk(s, load_chunk<false>(x + r * ld + c, n, c));
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
        sums[rl][cl * kChunk + i] = s[i];
    __syncthreads();
    // Halves of the rows' sums, added until one is left.
    for (int half = step / 2; half >= 1; half /= 2) {
        for (int at = threadIdx.x; at < half * 64; at += blockDim.x)
            sums[at >> 6][at & 63] += sums[(at >> 6) + half][at & 63];
        __syncthreads();
    }
    if (threadIdx.x < 64 && (int64_t)blockIdx.x * 64 + threadIdx.x < cols)
        to[blockIdx.y * cols + (int64_t)blockIdx.x * 64 + threadIdx.x] = sums[0][threadIdx.x];
}

// Zero-padded copies of the operands whose rows do not start on 16-byte boundaries
// or end inside a 16-byte chunk, one launch for both.  `lanes` of a workgroup take a
// row together, four chunks each at a time, and a row's last chunk is loaded from its
// last 16 bytes, so that no load waits for another: 24 MB in 9.6 us, 5 TB/s each way.
struct LinearPad {
    const uint16_t* src[2];
    uint16_t* dst[2];
    int64_t rows[2], cols[2], ld[2], dst_ld[2];
    uint32_t blocks[2];
    int32_t lanes[2];        // a power of two, at most 64
};

__global__ void __launch_bounds__(256) k_linear_pad(LinearPad p)
{
    const int o = blockIdx.x >= p.blocks[0];
    const uint32_t block = blockIdx.x - (o ? p.blocks[0] : 0u);
    const int lanes = p.lanes[o], rows = 256 / lanes, lane = threadIdx.x & (lanes - 1), first = threadIdx.x / lanes;
    const int32_t cols = (int32_t)p.cols[o], chunks = (int32_t)(p.dst_ld[o] / kChunk);
    for (int64_t r = (int64_t)block * rows + first; r < p.rows[o]; r += (int64_t)p.blocks[o] * rows) {
        const uint16_t* from = p.src[o] + r * p.ld[o];
        u32x4_t* to = (u32x4_t*)(p.dst[o] + r * p.dst_ld[o]);
        if (cols < kChunk) {
            if (lane == 0)
                *to = load_chunk<false>(from, cols, 0);
            continue;
        }
        for (int32_t c = lane; c < chunks; c += 4 * lanes) {
            u32x4_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_memcpy(&v[i], from + min((c + i * lanes) * kChunk, cols - kChunk), 16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (const int32_t at = c + i * lanes; at < chunks)
                    to[at] = shifted_chunk(v[i], max(at * kChunk - (cols - kChunk), 0));
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// A product C (M x N, N of one factor) over K, as the kernels see it.
struct LinearShape {
    int64_t M, N, K;
    bool bt, at;             // B stored N x K; A stored K x M
    int factors;
    bool a_even, b_even;     // as the tiles read them; else copied for them first

    int64_t a_rows() const { return at ? K : M; }
    int64_t a_cols() const { return at ? M : K; }
    int64_t b_rows() const { return bt ? N * factors : K; }
    int64_t b_cols() const { return bt ? K : N; }
};

// Rows that a workgroup sums the columns of (see k_column_sums).
int64_t column_run(int64_t rows, int64_t cols, int cus)
{
    if (rows <= kOneRun)
        return rows;
    return ceil_div(rows, std::max<int64_t>(1, std::min(4 * (int64_t)cus / ceil_div(cols, 64), rows / 128)));
}

int64_t pad_size(int64_t rows, int64_t cols) { return align256(rows * round8(cols) * 2); }

// A launch holds fewer than 2^32 threads, so many tiles of the waves' kernel, which outputs
// of fewer than 8 columns have to take: 64 rows a tile where there are more than 32.
constexpr int64_t kMaxWaveTiles = (int64_t)1 << 22, kMaxNarrowRows = kMaxWaveTiles * 64;
static_assert((kMaxWaveTiles + 7) * kWaves * 64 < (int64_t)1 << 32, "threads of a launch");

struct LinearPlan {
    int kind;
    int mf, nf;              // TILES_WAVE: fragments
    int bm, bn;              // outputs per workgroup
    int64_t tiles, splits, chunk, grid, workspace;   // chunk: k elements
};

// What a kind of kernel is estimated to take, in us, from the times of some 200 products
// of 1 to 8192 rows and 64 to 8192 columns and k (within 5 to 10 percent of them at the
// root mean square): so much for the call, for each round of tiles over the compute
// units and each k-step of a round; k chunks cost a second launch, and the time that
// their sums take through memory.  What every kind reads and writes alike is left out.
double linear_time(const LinearShape& q, const LinearPlan& pl, int cus)
{
    const int64_t items = pl.tiles * pl.splits;
    const double fill = (double)items / cus, rounds = (double)ceil_div(items, cus);
    const int64_t steps = ceil_div(pl.chunk, 64);
    const double sums = pl.splits > 1 ? 1e-6 * (double)pl.workspace : 0.0, copies =
        1e-6 * (double)((q.a_even ? 0 : pad_size(q.a_rows(), q.a_cols())) + (q.b_even ? 0 : pad_size(q.b_rows(), q.b_cols())));
    if (pl.kind == TILES_WAVE) {
        // Narrow workgroups share a compute unit, and their loads its bandwidth.
        const double k = (double)ceil_div(steps, kWaves) * (copies > 0 ? 1.5 : 1.0);
        const int nb = pl.nf * q.factors;
        double t;
        if (pl.mf == 1)
            t = nb == 1 ? k * (0.27 + 0.28 * fill) : nb == 2 ? k * (0.4 + 0.35 * fill) : k * (0.8 + 1.0 * fill);
        else
            t = rounds * (pl.mf == 2 ? 1.3 * k : 1.6 + 2.35 * k);
        return (pl.mf == 4 ? 1.4 : 3.2) + t + (pl.splits > 1 ? 6.0 + 0.5 * sums : 0.0);
    }
    const double padding = copies > 0 ? 2.5 + copies / 2.2 : 0.0;
    // The weight's gradient reads both operands transposed.
    if (pl.kind == TILES_SMALL)
        return 3.0 + rounds * (4.3 + (q.at ? 0.47 : 0.43) * steps) + (pl.splits > 1 ? 5.3 + 0.2 * sums : 0.0) + padding;
    const double round = pl.kind == TILES_192 ? 7.6 + 0.93 * steps : 9.0 + (q.at ? 1.35 : 1.1) * steps;
    return 1.5 + rounds * round + (pl.splits > 1 ? 5.0 + 0.17 * sums : 0.0) + padding;
}

// The kind, tile and chunks of k (whole 64-wide k-steps, all of them with work) that are
// estimated fastest.
LinearPlan linear_plan(const LinearShape& q, int cus)
{
    LinearPlan best{};
    double least = 0;
    const uint32_t steps = (uint32_t)ceil_div(q.K, 64);
    auto consider = [&](int kind, int mf, int nf) {
        LinearPlan pl{};
        pl.kind = kind;
        pl.mf = mf;
        pl.nf = nf;
        pl.bm = kind == TILES_WAVE ? mf * 16 : kind == TILES_BIG ? 256 : kind == TILES_192 ? 192 : 128;
        pl.bn = kind == TILES_WAVE ? nf * 16 : (kind == TILES_SMALL ? 128 : 256) / q.factors;
        pl.tiles = ceil_div(q.M, pl.bm) * ceil_div(q.N, pl.bn);
        if (kind == TILES_WAVE && pl.tiles > kMaxWaveTiles)
            return;
        for (uint32_t s = 1; s <= std::min<uint32_t>(kMaxSplits, steps) && (s == 1 || pl.tiles * s <= 2 * cus); ++s) {
            const uint32_t per = (steps + s - 1) / s;
            pl.chunk = s == 1 ? q.K : (int64_t)per * 64;
            pl.splits = (steps + per - 1) / per;
            if (pl.splits < s)
                continue;   // the same as for fewer
            pl.grid = kind == TILES_WAVE ? ceil_div(pl.tiles, 8) * 8 : std::min<int64_t>(pl.tiles * s, cus);
            pl.workspace = s > 1 ? pl.tiles * s * pl.bm * pl.bn * q.factors * 4 : 0;
            const double us = linear_time(q, pl, cus);
            if (best.bm == 0 || us < least) {
                least = us;
                best = pl;
            }
        }
    };
    const int mf = q.at || q.M > 32 ? 4 : q.M > 16 ? 2 : 1;
    consider(TILES_WAVE, mf, 4 / q.factors);
    if (mf == 1 && q.bt)
        for (int nf = 2 / q.factors; nf >= 1; nf /= 2)
            consider(TILES_WAVE, mf, nf);
    if (q.N >= kChunk) {   // TileAt's rows
        consider(TILES_SMALL, 0, 0);
        consider(TILES_BIG, 0, 0);
        if (!q.at && q.factors == 1)
            consider(TILES_192, 0, 0);
    }
    return best;
}

// One launch.  `done`, where there is one, becomes this kernel's completion: recorded as a
// marker behind it, it holds up the stream's next kernel 1.3 us longer.
template <class K, class... Args>
int enqueue(K kernel, dim3 grid, dim3 block, hipStream_t s, hipEvent_t done, Args... args)
{
    if (done)
        hipExtLaunchKernelGGL(kernel, grid, block, 0, s, nullptr, done, 0, args...);
    else
        hipLaunchKernelGGL(kernel, grid, block, 0, s, args...);
    return launched();
}

template <class C, int MODE>
int launch_linear(const LinearParams<MODE>& p, int64_t grid, hipStream_t s, hipEvent_t done)
{
    // Masks per lane only where a position may be partial: the k tail inside rows,
    // and columns past N of a K x N B.
    const bool edge = (!C::AT && (p.K % C::BK != 0 || p.K % p.ksplit != 0)) || (!C::BT && p.N % C::BN != 0);
    const bool longk = p.k_steps >= C::LONGK_MIN_KT && p.small_span;
    const dim3 g((unsigned)grid), b(C::THREADS);
    auto run = [&]<bool LONGK, bool EDGE>() {
        if constexpr (C::WIN)
            return enqueue(k_gemm_win<C, LONGK, EDGE, LinearParams<MODE>>, g, b, s, done, p);
        else
            return enqueue(k_gemm<C, LONGK, EDGE, LinearParams<MODE>>, g, b, s, done, p);
    };
    if (longk && !edge)
        return run.template operator()<true, false>();
    if (longk)
        return run.template operator()<true, true>();
    return run.template operator()<false, true>();
}

template <int MODE>
int launch_wave(const LinearParams<MODE>& p, const LinearPlan& pl, bool even, hipStream_t s, hipEvent_t done)
{
    constexpr int F = fuse_paired(MODE) ? 2 : 1;
    constexpr bool BT = MODE == FUSE_LINEAR || F == 2;
    const int32_t kblocks = (int32_t)ceil_div(p.K, 64), chunk = (int32_t)ceil_div(pl.chunk, 64);
    const dim3 g((unsigned)pl.grid, (unsigned)pl.splits), b(kWaves * 64);
    auto run = [&]<int MF, int NF, int DEPTH>() {
        return even ? enqueue(k_linear_wave<MODE, MF, NF, DEPTH, true>, g, b, s, done, p, chunk, kblocks)
                    : enqueue(k_linear_wave<MODE, MF, NF, DEPTH, false>, g, b, s, done, p, chunk, kblocks);
    };
    if constexpr (BT) {
        if (pl.mf == 1 && F == 1 && pl.nf == 1)
            return run.template operator()<1, 1, 4>();
        if (pl.mf == 1 && pl.nf * F == 2)
            return run.template operator()<1, 2 / F, 2>();
    }
    if constexpr (MODE != FUSE_DW) {
        if (pl.mf == 1)
            return run.template operator()<1, 4 / F, 2>();
        if (pl.mf == 2)
            return run.template operator()<2, 4 / F, 1>();
    }
    return run.template operator()<4, 4 / F, 1>();
}

// The product of A and B into epilogue e.  The caller has checked everything but
// the device.
template <int MODE>
int linear_run(LinearShape q, const void* A, int64_t lda, const void* B, int64_t ldb, const Epilogue& e,
               TempMem& tm, int cus, hipStream_t s, float* dbias = nullptr)
{
    constexpr bool PAIR = fuse_paired(MODE), BT = MODE == FUSE_LINEAR || PAIR, AT = MODE == FUSE_DW;
    LinearParams<MODE> p;
    memset((void*)&p, 0, sizeof p);
    p.e = e;
    // Leading dimensions that do not count, a single row's and an absent operand's, may be
    // anything: TileAt's offsets take that of 8 rows, and `far` below all of them.
    auto counted = [&](int64_t& ld, const void* ptr, int64_t width) {
        if (q.M <= 1 || !ptr)
            ld = width;
    };
    const int64_t both = 2 * e.N;
    counted(p.e.ld_in0, e.in0, MODE == FUSE_DGATED ? both : e.N);
    counted(p.e.ld_in1, e.in1, e.N);
    counted(p.e.ld_out0, e.out0, MODE == FUSE_DGATED ? both : e.N);
    counted(p.e.ld_out1, e.out1, MODE == FUSE_GATED ? both : e.N);
    // Operands as the tiles read them: rows on 16-byte boundaries, of whole 16-byte
    // chunks, at most 2^22 elements apart.
    const int64_t a_rows = q.a_rows(), a_cols = q.a_cols(), b_rows = q.b_rows(), b_cols = q.b_cols();
    auto fits = [](const void* ptr, int64_t rows, int64_t cols, int64_t ld) {
        return ((uintptr_t)ptr & 15) == 0 && cols % kChunk == 0 && (rows <= 1 || (ld % kChunk == 0 && ld <= kMaxLd));
    };
    q.a_even = fits(A, a_rows, a_cols, lda);
    q.b_even = fits(B, b_rows, b_cols, ldb);
    const LinearPlan pl = q.K > 0 && q.N > 0 ? linear_plan(q, cus) : LinearPlan{TILES_SMALL, 0, 0, 128, 128 / q.factors, 0, 0, 0, 0, 0};
    p.A = (const char*)A;
    p.B = (const char*)B;
    p.M = q.M;
    p.N = q.N;
    p.K = q.K;
    p.lda = lda;
    p.ldb = ldb;
    p.tiles_m = (int32_t)ceil_div(q.M, pl.bm);
    p.tiles_n = (int32_t)ceil_div(q.N, pl.bn);
    const int64_t tiles = ceil_div(q.M, pl.bm) * ceil_div(q.N, pl.bn);
    const int64_t steps = ceil_div(pl.chunk, 64);
    if (tiles > ((int64_t)1 << 30) || tiles * (pl.splits ? pl.splits : 1) * (steps ? steps : 1) > ((int64_t)1 << 30))
        return GEMM_ERR_UNSUPPORTED_SHAPE;
    p.tiles_mn = p.span = (int32_t)tiles;
    p.splits = (int32_t)pl.splits;
    p.tiles = (int32_t)(tiles * pl.splits);
    p.ksplit = pl.chunk;
    p.k_steps = (int32_t)steps;
    p.group_m = pl.kind == TILES_WAVE ? p.tiles_m : 4;
    p.spin_limit = kSpinLimit;
    p.clock_on = g_clock_on.load(std::memory_order_relaxed) ? 1u : 0u;
    // dbias: sums of A's columns, in runs of rows where there are many.
    ColumnSums sums{};
    int64_t run = a_rows;
    if (dbias) {
        run = column_run(a_rows, a_cols, cus);
        sums = {nullptr, dbias, a_cols, (int32_t)ceil_div(std::max<int64_t>(a_rows, 1), std::max<int64_t>(run, 1)), 0};
    }
    const int64_t runs_bytes = sums.runs > 1 ? align256(sums.runs * a_cols * 4) : 0;
    // The call's temporary memory is free once its last kernel is done.
    void* ws = nullptr;
    hipEvent_t done = nullptr;
    auto finish = [&]() {
        const int64_t units = (int64_t)p.span * pl.bm * pl.bn / (MODE == FUSE_DW && e.fp32 ? 4 : kChunk);
        return enqueue(k_linear_finish<MODE>, dim3(flat_grid(units) + sums.blocks), dim3(256), s, done, p,
                       (int32_t)pl.bm, (int32_t)pl.bn, sums);
    };
    auto start_sums = [&](float* part) {
        const bool one = sums.runs <= 1;
        const unsigned threads = one ? 1024 : 256;
        hipLaunchKernelGGL(k_column_sums, dim3((unsigned)ceil_div(a_cols, 64), (unsigned)sums.runs), dim3(threads), 0, s,
                           (const uint16_t*)A, a_rows, a_cols, lda, run, one ? dbias : part);
        sums.part = part;
        sums.blocks = one ? 0u : (unsigned)ceil_div(a_cols, 16);
        return launched();
    };
    auto join_sums = [&]() {
        return enqueue(k_join_column_sums, dim3(sums.blocks), dim3(256), s, done, sums);
    };
    if (q.K == 0 || q.N == 0) {   // nothing to multiply
        int rc = runs_bytes > 0 ? temp_take_outside_graphs(tm, runs_bytes, s, &ws, &done) : (int)GEMM_OK;
        if (rc == GEMM_OK && dbias)
            rc = start_sums((float*)ws);
        if (rc == GEMM_OK && q.N > 0)
            rc = finish();
        else if (rc == GEMM_OK && sums.blocks > 0)
            rc = join_sums();
        const int frc = temp_give(tm, ws, s, rc == GEMM_OK && done != nullptr);
        return rc != GEMM_OK ? rc : frc;
    }

    const bool wave = pl.kind == TILES_WAVE;
    const bool pad_a = !wave && !q.a_even, pad_b = !wave && !q.b_even;
    const int64_t a_ld = round8(a_cols), b_ld = round8(b_cols);
    const int64_t a_bytes = pad_a ? pad_size(a_rows, a_cols) : 0, b_bytes = pad_b ? pad_size(b_rows, b_cols) : 0;
    // The tiles' epilogue addresses rows by 32-bit offsets; others' sums go through the
    // second launch.
    const bool far = !wave && std::max({p.e.ld_in0, p.e.ld_in1, p.e.ld_out0, p.e.ld_out1}) > kMaxTileLd;
    const int64_t sums_bytes = pl.splits > 1 || !far ? pl.workspace : pl.tiles * pl.bm * pl.bn * q.factors * 4;
    const int64_t bytes = a_bytes + b_bytes + runs_bytes + sums_bytes;
    int rc = GEMM_OK;
    if (bytes > 0 && (rc = temp_take_outside_graphs(tm, bytes, s, &ws, &done)) != GEMM_OK)
        return rc;
    if (dbias)
        rc = start_sums((float*)((char*)ws + a_bytes + b_bytes));
    if (rc == GEMM_OK && (pad_a || pad_b)) {
        LinearPad c{{(const uint16_t*)A, (const uint16_t*)B},
                    {(uint16_t*)ws, (uint16_t*)((char*)ws + a_bytes)},
                    {pad_a ? a_rows : 0, pad_b ? b_rows : 0},
                    {a_cols, b_cols},
                    {lda, ldb},
                    {a_ld, b_ld},
                    {0, 0},
                    {1, 1}};
        for (int o = 0; o < 2; ++o) {
            while (c.lanes[o] < 64 && c.lanes[o] * kChunk < c.cols[o])
                c.lanes[o] *= 2;
            c.blocks[o] = (uint32_t)std::min<int64_t>(ceil_div(c.rows[o] * c.lanes[o], 256), 1 << 20);
        }
        if (pad_a) {
            p.A = (const char*)c.dst[0];
            p.lda = a_ld;
        }
        if (pad_b) {
            p.B = (const char*)c.dst[1];
            p.ldb = b_ld;
        }
        hipLaunchKernelGGL(k_linear_pad, dim3(c.blocks[0] + c.blocks[1]), dim3(256), 0, s, c);
        rc = launched();
    }
    if (sums_bytes > 0)
        p.partial = (float*)((char*)ws + a_bytes + b_bytes + runs_bytes);
    // A single row's stride is never used, but enters sizes and offsets.
    if (a_rows <= 1)
        p.lda = a_ld;
    if (b_rows <= 1)
        p.ldb = b_ld;
    p.small_span = ((a_rows - 1) * p.lda + a_ld) * 2 < (int64_t)kMaxRecords &&
                   ((b_rows / q.factors - 1) * p.ldb + b_ld) * 2 < (int64_t)kMaxRecords;
    const bool second = sums_bytes > 0 || sums.blocks > 0;
    if (rc == GEMM_OK) {
        const hipEvent_t d = second ? nullptr : done;
        if (wave)
            rc = launch_wave<MODE>(p, pl, q.a_even && q.b_even, s, d);
        else if (pl.kind == TILES_SMALL)
            rc = launch_linear<LinearCfg<BT, AT, PAIR, TILES_SMALL>, MODE>(p, pl.grid, s, d);
        else if (pl.kind == TILES_BIG)
            rc = launch_linear<LinearCfg<BT, AT, PAIR, TILES_BIG>, MODE>(p, pl.grid, s, d);
        else if constexpr (!AT && !PAIR)
            rc = launch_linear<LinearCfg<BT, AT, PAIR, TILES_192>, MODE>(p, pl.grid, s, d);
    }
    if (rc == GEMM_OK && second)
        rc = sums_bytes > 0 ? finish() : join_sums();
    const int frc = temp_give(tm, ws, s, rc == GEMM_OK && done != nullptr);
    return rc != GEMM_OK ? rc : frc;
}

// M rows, the other sizes, and which of them is the output's columns.
int linear_sizes(int64_t M, int64_t N, int64_t K, int64_t cols)
{
    if (M < 0 || N < 0 || K < 0)
        return GEMM_ERR_INVALID_VALUE;
    return M > kMaxRows || N > kMaxLd || K > kMaxLd || (cols < kChunk && M > kMaxNarrowRows) ? GEMM_ERR_UNSUPPORTED_SHAPE
                                                                                             : GEMM_OK;
}

bool known_act(int act) { return act >= GEMM_ACT_NONE && act <= GEMM_ACT_SILU; }

// An operand of a call: whether it has to be there, and, of an output, which input's
// very memory it may be (its elements are read before they are written, by the
// lane that writes them).
struct LinearOperand {
    Operand o;
    bool needed;
    const void* in_place;
};

int check_linear(const LinearOperand* ins, int n_ins, const LinearOperand* outs, int n_outs)
{
    for (int i = 0; i < n_ins + n_outs; ++i) {
        const LinearOperand& x = i < n_ins ? ins[i] : outs[i - n_ins];
        if (!x.needed && !x.o.p)
            continue;
        if (const int rc = check_operand(x.o))
            return rc;
    }
    for (int i = 0; i < n_outs; ++i) {
        for (int j = 0; j < n_ins; ++j)
            if (meet(outs[i].o, ins[j].o) && !(outs[i].in_place == ins[j].o.p && ins[j].in_place == ins[j].o.p &&
                                               same_memory(outs[i].o, ins[j].o)))
                return GEMM_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i].o, outs[j].o))
                return GEMM_ERR_ALIAS;
    }
    return GEMM_OK;
}

// The device, then the product, with the caller's workspace or, without one, memory that
// the library keeps.
template <int MODE>
int linear_enqueue(const LinearShape& q, const void* A, int64_t lda, const void* B, int64_t ldb, const Epilogue& e,
                   void* workspace, int64_t workspace_bytes, void* stream, float* dbias = nullptr)
{
    int cus = 0;
    TempMem tm;
    tm.device_done = true;
    if (const int rc = device_info(&cus, &tm.pool, nullptr, &tm.info))
        return rc;
    tm.given(workspace, workspace_bytes);
    return linear_run<MODE>(q, A, lda, B, ldb, e, tm, cus, (hipStream_t)stream, dbias);
}

int check_workspace(const void* workspace, int64_t bytes, const LinearOperand* ins, int n_ins, const LinearOperand* outs,
                    int n_outs)
{
    if (!workspace)
        return GEMM_OK;
    if (bytes < 0)
        return GEMM_ERR_INVALID_VALUE;
    if ((uintptr_t)workspace & 255)
        return GEMM_ERR_MISALIGNED;
    const Operand w{workspace, 1, bytes, bytes, 1};
    for (int i = 0; i < n_ins + n_outs; ++i)
        if (meet(w, (i < n_ins ? ins[i] : outs[i - n_ins]).o))
            return GEMM_ERR_ALIAS;
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_linear_plan_cus(int64_t M, int64_t N, int64_t K, int product, int a_aligned, int b_aligned, int compute_units,
                         gemm_linear_plan_t* out)
{
    if (const int rc = linear_sizes(M, N, K, product == GEMM_LINEAR_BWD_INPUT ? K : product == GEMM_LINEAR_BWD_WEIGHT ? kChunk : N))
        return rc;
    if (!out || compute_units < 1 || product < GEMM_LINEAR || product > GEMM_GATED_LINEAR_BWD_INPUT)
        return GEMM_ERR_INVALID_VALUE;
    LinearShape q{M, N, K, true, false, 1, false, false};
    if (product == GEMM_LINEAR_BWD_INPUT)
        q = {M, K, N, false, false, 1, false, false};
    else if (product == GEMM_LINEAR_BWD_WEIGHT)
        q = {N, K, M, false, true, 1, false, false};
    else if (product == GEMM_GATED_LINEAR)
        q.factors = 2;
    else if (product == GEMM_GATED_LINEAR_BWD_INPUT)
        q = {M, N, K, false, false, 1, false, false};
    q.a_even = a_aligned && q.a_cols() % kChunk == 0;
    q.b_even = b_aligned && q.b_cols() % kChunk == 0;
    memset(out, 0, sizeof *out);
    if (product == GEMM_LINEAR_BWD_WEIGHT && N > 0 && M > kOneRun)
        out->scratch_bytes = align256(ceil_div(M, column_run(M, N, compute_units)) * N * 4);
    if (q.M == 0 || q.N == 0 || q.K == 0)
        return GEMM_OK;
    const LinearPlan pl = linear_plan(q, compute_units);
    out->rows = pl.bm;
    out->cols = pl.bn;
    out->waves_share_k = pl.kind == TILES_WAVE;
    out->threads = pl.kind != TILES_SMALL ? kWaves * 64
                   : q.factors == 2       ? LinearCfg<true, false, true, TILES_SMALL>::THREADS
                                          : LinearCfg<true, false, false, TILES_SMALL>::THREADS;
    out->tiles = pl.tiles;
    out->k_splits = pl.splits;
    out->k_chunk = pl.chunk;
    out->grid = pl.kind == TILES_WAVE ? pl.grid * pl.splits : pl.grid;
    out->workspace_bytes = pl.workspace;
    if (pl.kind != TILES_WAVE)
        out->pad_bytes = (q.a_even ? 0 : pad_size(q.a_rows(), q.a_cols())) + (q.b_even ? 0 : pad_size(q.b_rows(), q.b_cols()));
    out->scratch_bytes += align256(pl.workspace) + out->pad_bytes;
    return GEMM_OK;
}

int gemm_linear(int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W, int64_t ldw,
                const void* bias, int act, const void* residual, int64_t ldr, void* Z, int64_t ldz, void* Y, int64_t ldy,
                void* workspace, int64_t workspace_bytes, void* stream)
{
    if (const int rc = linear_sizes(M, N, K, N))
        return rc;
    if (!known_act(act))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0)
        return GEMM_OK;
    const LinearOperand ins[] = {{{K > 0 ? X : nullptr, M, K, ldx, 2}, K > 0, nullptr},
                                 {{K > 0 ? W : nullptr, N, K, ldw, 2}, K > 0, nullptr},
                                 {{bias, 1, N, N, 2}, false, nullptr},
                                 {{residual, M, N, ldr, 2}, false, residual}};
    const LinearOperand outs[] = {{{Y, M, N, ldy, 2}, true, residual}, {{Z, M, N, ldz, 2}, false, nullptr}};
    if (const int rc = check_linear(ins, 4, outs, 2))
        return rc;
    if (const int rc = check_workspace(workspace, workspace_bytes, ins, 4, outs, 2))
        return rc;
    const Epilogue e{(const uint16_t*)bias, (const uint16_t*)residual, nullptr, Y, (uint16_t*)Z, ldr, 0, ldy, ldz,
                     M, N, act, 0};
    return linear_enqueue<FUSE_LINEAR>({M, N, K, true, false, 1, false, false}, X, ldx, W, ldw, e, workspace, workspace_bytes, stream);
}

int gemm_linear_bwd_input(int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy, const void* W, int64_t ldw,
                          int act, const void* Z, int64_t ldz, const void* dres, int64_t lddr, void* dX, int64_t lddx,
                          void* workspace, int64_t workspace_bytes, void* stream)
{
    if (const int rc = linear_sizes(M, N, K, K))
        return rc;
    if (!known_act(act))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || K == 0)
        return GEMM_OK;
    if (act == GEMM_ACT_NONE)
        Z = nullptr;
    const LinearOperand ins[] = {{{N > 0 ? dY : nullptr, M, N, lddy, 2}, N > 0, nullptr},
                                 {{N > 0 ? W : nullptr, N, K, ldw, 2}, N > 0, nullptr},
                                 {{Z, M, K, ldz, 2}, act != GEMM_ACT_NONE, Z},
                                 {{dres, M, K, lddr, 2}, false, dres}};
    const LinearOperand outs[] = {{{dX, M, K, lddx, 2}, true, dX == Z ? Z : dres}};
    if (const int rc = check_linear(ins, 4, outs, 1))
        return rc;
    if (const int rc = check_workspace(workspace, workspace_bytes, ins, 4, outs, 1))
        return rc;
    const Epilogue e{nullptr, (const uint16_t*)Z, (const uint16_t*)dres, dX, nullptr, ldz, lddr, lddx, 0, M, K, act, 0};
    return linear_enqueue<FUSE_DX>({M, K, N, false, false, 1, false, false}, dY, lddy, W, ldw, e, workspace, workspace_bytes, stream);
}

int gemm_linear_bwd_weight(int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy, const void* X, int64_t ldx,
                           void* dW, int64_t lddw, int dw_type, float* dbias, void* workspace, int64_t workspace_bytes,
                           void* stream)
{
    if (const int rc = linear_sizes(M, N, K, kChunk))
        return rc;
    const bool fp32 = dw_type == GEMM_TYPE_FP32;
    if (!fp32 && dw_type != GEMM_TYPE_BF16)
        return GEMM_ERR_INVALID_VALUE;
    const bool weight = N > 0 && K > 0, bias = dbias && N > 0;
    if (!weight && !bias)
        return GEMM_OK;
    const LinearOperand ins[] = {{{M > 0 ? dY : nullptr, M, N, lddy, 2}, M > 0, nullptr},
                                 {{M > 0 && weight ? X : nullptr, M, K, ldx, 2}, M > 0 && weight, nullptr}};
    const LinearOperand outs[] = {{{weight ? dW : nullptr, N, K, lddw, fp32 ? 4 : 2}, weight, nullptr},
                                  {{dbias, 1, N, N, 4}, false, nullptr}};
    if (const int rc = check_linear(ins, 2, outs, 2))
        return rc;
    if (const int rc = check_workspace(workspace, workspace_bytes, ins, 2, outs, 2))
        return rc;
    const Epilogue e{nullptr, nullptr, nullptr, dW, nullptr, 0, 0, lddw, 0, N, K, GEMM_ACT_NONE, fp32 ? 1 : 0};
    return linear_enqueue<FUSE_DW>({N, K, M, false, true, 1, false, false}, dY, lddy, X, ldx, e, workspace, workspace_bytes,
                                   stream, bias ? dbias : nullptr);
}

int gemm_gated_linear(int64_t M, int64_t F, int64_t K, const void* X, int64_t ldx, const void* W, int64_t ldw,
                      const void* bias, int act, void* GU, int64_t ldgu, void* Y, int64_t ldy, void* workspace,
                      int64_t workspace_bytes, void* stream)
{
    if (const int rc = linear_sizes(M, F, K, F))
        return rc;
    if (!known_act(act))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || F == 0)
        return GEMM_OK;
    const LinearOperand ins[] = {{{K > 0 ? X : nullptr, M, K, ldx, 2}, K > 0, nullptr},
                                 {{K > 0 ? W : nullptr, 2 * F, K, ldw, 2}, K > 0, nullptr},
                                 {{bias, 1, 2 * F, 2 * F, 2}, false, nullptr}};
    const LinearOperand outs[] = {{{Y, M, F, ldy, 2}, true, nullptr}, {{GU, M, 2 * F, ldgu, 2}, false, nullptr}};
    if (const int rc = check_linear(ins, 3, outs, 2))
        return rc;
    if (const int rc = check_workspace(workspace, workspace_bytes, ins, 3, outs, 2))
        return rc;
    const Epilogue e{(const uint16_t*)bias, nullptr, nullptr, Y, (uint16_t*)GU, 0, 0, ldy, ldgu, M, F, act, 0};
    return linear_enqueue<FUSE_GATED>({M, F, K, true, false, 2, false, false}, X, ldx, W, ldw, e, workspace, workspace_bytes, stream);
}

int gemm_gated_linear_bwd_input(int64_t M, int64_t F, int64_t N, const void* dY, int64_t lddy, const void* W, int64_t ldw,
                                int act, const void* GU, int64_t ldgu, void* dGU, int64_t lddgu, void* Y, int64_t ldy,
                                void* workspace, int64_t workspace_bytes, void* stream)
{
    if (const int rc = linear_sizes(M, F, N, F))
        return rc;
    if (!known_act(act))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || F == 0)
        return GEMM_OK;
    const LinearOperand ins[] = {{{N > 0 ? dY : nullptr, M, N, lddy, 2}, N > 0, nullptr},
                                 {{N > 0 ? W : nullptr, N, F, ldw, 2}, N > 0, nullptr},
                                 {{GU, M, 2 * F, ldgu, 2}, true, GU}};
    const LinearOperand outs[] = {{{dGU, M, 2 * F, lddgu, 2}, true, GU}, {{Y, M, F, ldy, 2}, false, nullptr}};
    if (const int rc = check_linear(ins, 3, outs, 2))
        return rc;
    if (const int rc = check_workspace(workspace, workspace_bytes, ins, 3, outs, 2))
        return rc;
    const Epilogue e{nullptr, (const uint16_t*)GU, nullptr, dGU, (uint16_t*)Y, ldgu, 0, lddgu, ldy, M, F, act, 0};
    return linear_enqueue<FUSE_DGATED>({M, F, N, false, false, 1, false, false}, dY, lddy, W, ldw, e, workspace, workspace_bytes, stream);
}

}  // extern "C"
