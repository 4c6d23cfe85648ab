// The product of 8-bit operands with a scale for each block of 128 along k (part
// of library.hip).
//
//   C[i][j] = sum_kb sa[kb][i] * sb[kb][j or j / 128] * sum_{k in kb} A[i][k] * B[j][k]
//
// A block's partial sums start from zero and enter the running sums by one fused
// multiply-add each, times the product of the two scales, which has to be a normal
// number: one scale after the other would take any pair whose result fits, at
// four more products beside each MFMA's four multiply-adds.  The MFMA's rows are
// B's (n) and its columns A's (m): a lane then holds 4 consecutive columns of one
// row of C, so a block's scale product is one value per lane and fragment,
// shared by every fragment of that row against the same 128 columns.
//
// Two ways to contract a block of 128:
//   fast    one v_mfma_f32_16x16x128_f8f6f4, twice the rate of bf16.  It adds
//           each run of 8 consecutive products on a grid of 2^-13 of the run's
//           largest: what a product has below the grid is cut off (measured: beside
//           2^16 a product of 2^3 counts, 1.5 * 2^3 counts as 2^3, and 2^2 is
//           lost; the sums of runs add up as fp32 sums do).  On random operands
//           that is 1.5e-5 of the result's norm, a hundredth of bf16's rounding;
//           where products cancel within a run it is whatever they leave.
//   exact   the bytes converted to bf16, which holds every e4m3 value, and four
//           v_mfma_f32_16x16x32_bf16, whose sums are fp32's (0.7 to 1.1e-7 of the
//           result's norm).  Half the matrix rate, and 16 conversions a fragment.
// A bf16 C takes the fast way unless the caller asks for the exact one, which
// costs 0.4 us at 1 x 8192 x 8192 (13.2), 0.9 at 64 x 8192 x 8192 (19.5), 65 at
// 4096^3 (59) and 590 at 8192^3 (405).  An fp32 C and short sums (bound by C's
// bytes) are computed exactly.
//
// A tile row of 128 bytes is what the bf16 product calls a row of 64 elements:
// the tile configurations, the LDS ring with its swizzle and the raster are the
// bf16 product's, with K, lda and ldb in Params counted in 2-byte units.
#pragma once

namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef LDS_AS float lds_f32;

// What the product needs beside the loader's Params (sizes there in 2-byte
// units along k).
struct Fp8Params {
    const float* sa;
    const float* sb;
    char* c;
    int64_t ldsa, ldsb, ldc;
    int64_t K;               // bytes
    int64_t sb_cols;         // scales per k block of B
    int32_t kblocks;         // ceil(K / 128)
    int32_t sb_shift;        // log2 of B's rows per scale: 7 or 0
    int32_t c_fp32;
};

// One block of 128 of 16 rows of an operand: lane (r16, g) holds 32 bytes of row
// r16, in an order along k that is the same for both operands.
template <bool EXACT>
struct Fp8Frag {
    i32x8_t v;
    __device__ __forceinline__ Fp8Frag() {}
    __device__ __forceinline__ Fp8Frag(u32x4_t lo, u32x4_t hi)
        : v(__builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)))
    {
    }
};

// 8 e4m3 bytes as bf16.
__device__ __forceinline__ bf16x8_t bf16_of(uint32_t w0, uint32_t w1)
{
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <>
struct Fp8Frag<true> {
    bf16x8_t v[4];
    __device__ __forceinline__ Fp8Frag() {}
    __device__ __forceinline__ Fp8Frag(u32x4_t lo, u32x4_t hi)
        : v{bf16_of(lo[0], lo[1]), bf16_of(lo[2], lo[3]), bf16_of(hi[0], hi[1]), bf16_of(hi[2], hi[3])}
    {
    }
};

__device__ __forceinline__ f32x4_t block_sums(const Fp8Frag<false>& b, const Fp8Frag<false>& a)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ f32x4_t block_sums(const Fp8Frag<true>& b, const Fp8Frag<true>& a)
{
    f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[i], a.v[i], d, 0, 0, 0);
    return d;
}

// 4 consecutive values of a row of C at column n (any alignment).
__device__ __forceinline__ void store_c4(const Fp8Params& q, int64_t m, int64_t n, int64_t N, f32x4_t v)
{
    const int64_t at = m * q.ldc + n;
    if (q.c_fp32) {
        float* c = (float*)q.c + at;
        if (n + 4 <= N) {
            __builtin_memcpy(c, &v, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (n + e < N)
                    c[e] = v[e];
        }
    } else {
        uint16_t* c = (uint16_t*)q.c + at;
        const u32x2_t w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if (n + 4 <= N) {
            __builtin_memcpy(c, &w, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (n + e < N)
                    c[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// ---------------------------------------------------------------------------
// Large products: 128-byte k-steps through the two-stage LDS ring.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int MF = 16>
using Fp8Cfg = Cfg<BM, BN, 64, 2, WM, WN, SYNC_BARRIER, true, 0, false, MF>;

// The column of a wave's strip that LDS row `row` of the strip holds.  An MFMA
// leaves a lane 4 consecutive rows of B's fragment at a time (16 x 16: rows 4 g
// .. of each fragment; 32 x 32: rows 8 q + 4 h .. for q = 0 .. 3).  The map
// strings them together, so that a lane ends up with RUN consecutive columns of
// C: 4 of each of the FN fragments, or the 16 of one.
template <class C>
__device__ __forceinline__ int fp8_col(int row)
{
    if constexpr (C::MF == 32)
        return (row & ~31) + ((row >> 2) & 1) * 16 + ((row >> 3) & 3) * 4 + (row & 3);
    else
        return ((row & 15) >> 2) * (4 * C::FN) + (row >> 4) * 4 + (row & 3);
}

// The load stream of one workgroup: positions (output tile, k-step), each an A
// tile, a B tile and, in LDS beside them, the scales of BM rows and BN columns.
//
// As in the bf16 loader, slot s of a 1 KiB load holds tile row s / 8 and the
// 16-byte chunk that the swizzle puts there, and a resource ends at the
// operand's last byte, so rows past the matrix read as zeros; chunks past K are
// masked per lane.  The row of a B slot is fp8_col's, which makes the lanes'
// columns of C consecutive.  A scale load is 4 bytes per lane, one load a wave.
//
// The cursor is free of branches: it steps through a tile's k range with the
// loads' scalar offset, and at a given k-step takes over the next tile's
// origin, which is worked out once per tile.  A resource's byte count is capped
// below 2^31, which no access of a tile reaches (255 rows of at most 2^23
// bytes, and K); a masked lane's offset is past it whatever is added.
template <class C>
struct Fp8Loader {
    static constexpr int SCALE_BYTES = (C::BM + C::BN) * 4;
    static constexpr int AW = C::BM / 64;   // waves that fetch A's scales
    static_assert((C::BM + C::BN) / 64 == C::NCW && C::BK == 64, "one scale load per wave, 128-byte tile rows");

    // A lane's place in the first load of each operand.  Its place in load t is
    // RSTEP tile rows further per load at the same chunk (RSTEP rows are whole
    // periods of the swizzle), a scalar distance for A and, fp8_col being
    // additive in them, for B.
    static constexpr int RSTEP = C::NLW * 8;
    static_assert(RSTEP % C::MF == 0 && (RSTEP % C::TN == 0 || C::TN % RSTEP == 0), "loads of a lane");
    uint32_t voffA, voffB, voffS;
    uint32_t ldaB, ldbB;                    // row strides in bytes
    int32_t kofs;                           // of the lane's chunk within the k-step, bytes
    static constexpr int rows_a(int t) { return t * RSTEP; }
    static constexpr int cols_b(int t)
    {
        return C::MF == 32 || RSTEP % C::TN == 0 ? t * RSTEP : t * RSTEP / C::TN * C::TN + t * RSTEP % C::TN / 16 * 4;
    }
    struct Position {
        const char* a;
        const char* b;
        const char* s;                      // this wave's scales at the position's k block
        uint32_t na, nb, ns;                // bytes left to the end of each operand
        int32_t k, kleft;                   // bytes: offset within the chunk's k range, left of K
    };
    Position cur, nxt;
    int64_t sstep;                          // bytes per k block of this wave's scales

    __device__ __forceinline__ void init(const Params& p, const Fp8Params& q, int w, int lane)
    {
        ldaB = (uint32_t)p.lda * 2u;
        ldbB = (uint32_t)p.ldb * 2u;
        const int row = w * 8 + lane / 8;
        kofs = ((lane % 8) ^ swz_k<64>(row)) * 16;
        voffA = (uint32_t)row * ldaB + (uint32_t)kofs;
        voffB = (uint32_t)(row / C::TN * C::TN + fp8_col<C>(row % C::TN)) * ldbB + (uint32_t)kofs;
        const bool a = w < AW;
        // A's scales in the order a lane reads them: word FM * r + i of a wave's
        // rows holds row MF * i + r.
        const int at = (a ? w : w - AW) * 64 + lane, in = at % C::TM;
        voffS = (uint32_t)(a ? at - in + in % C::FM * C::MF + in / C::FM : at >> q.sb_shift) * 4u;
        sstep = (a ? q.ldsa : q.ldsb) * 4;
    }

    // The first position of the workgroup's work item `ti`; an empty one past
    // the last item.
    __device__ __forceinline__ Position first(const Params& p, const Fp8Params& q, int32_t ti, int32_t n_tiles, int w) const
    {
        int32_t tm, tn, sp, u;
        tile_coords(p, (int32_t)blockIdx.x + min(ti, n_tiles - 1) * (int32_t)gridDim.x, (int32_t)gridDim.x, tm, tn, sp,
                    u);
        const int64_t m0 = (int64_t)tm * C::BM, n0 = (int64_t)tn * C::BN, k0 = (int64_t)sp * p.k_steps * kBlock;
        const bool live = ti < n_tiles, a = w < AW;
        Position r;
        r.a = p.A + m0 * p.lda * 2 + k0;
        r.b = p.B + n0 * p.ldb * 2 + k0;
        r.na = live ? records((uint64_t)(((p.M - 1 - m0) * p.lda * 2) + q.K - k0)) : 0u;
        r.nb = live ? records((uint64_t)(((p.N - 1 - n0) * p.ldb * 2) + q.K - k0)) : 0u;
        r.k = 0;
        r.kleft = (int32_t)(q.K - k0);
        const int64_t n0s = n0 >> q.sb_shift, left = a ? p.M - m0 : q.sb_cols - n0s;
        r.s = (a ? (const char*)(q.sa + m0) : (const char*)(q.sb + n0s)) + (int64_t)sp * p.k_steps * sstep;
        r.ns = live ? (uint32_t)min(left, (int64_t)C::BM + C::BN) * 4u : 0u;
        return r;
    }

    // The next position; `enter` (uniform) takes the next tile's first one.
    // Member by member, which compiles to selects: a branch here would cut the
    // k-step's schedule in two, and the compiler moves sums across the cut.
    __device__ __forceinline__ void step(bool enter)
    {
        cur.a = enter ? nxt.a : cur.a;
        cur.b = enter ? nxt.b : cur.b;
        cur.s = enter ? nxt.s : cur.s + sstep;
        cur.na = enter ? nxt.na : cur.na;
        cur.nb = enter ? nxt.nb : cur.nb;
        cur.ns = enter ? nxt.ns : cur.ns;
        cur.k = enter ? nxt.k : cur.k + kBlock;
        cur.kleft = enter ? nxt.kleft : cur.kleft - kBlock;
    }

    __device__ __forceinline__ void fire(const Position& r, int t, lds_char* stage, int w) const
    {
        const bool ok = kofs < r.kleft;
        const int tb = t - C::A_LOADS;
        if (t < C::A_LOADS)
            lds_dma16(rsrc_n(r.a, r.na), stage + (t * C::NLW + w) * 1024, ok ? voffA : kOOB,
                      (uint32_t)r.k + (uint32_t)rows_a(t) * ldaB);
        else
            lds_dma16(rsrc_n(r.b, r.nb), stage + C::A_BYTES + (tb * C::NLW + w) * 1024, ok ? voffB : kOOB,
                      (uint32_t)r.k + (uint32_t)cols_b(tb) * ldbB);
    }

    // k blocks past K have no scales: they read as zeros.
    __device__ __forceinline__ void fire_scales(const Position& r, lds_char* scales, int w) const
    {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_n(r.s, r.kleft > 0 ? r.ns : 0u), (LDS_AS void*)(scales + w * 256),
                                                 4, voffS, 0, 0, 0);
    }
};

// 16 consecutive columns of a row of C from n on: v(x) is the x-th 4 of them.
template <class V>
__device__ __forceinline__ void store_c16(const Fp8Params& q, int64_t m, int64_t n, int64_t N, V&& v)
{
    if (n + 16 <= N) {
        if (q.c_fp32) {
            float* c = (float*)q.c + m * q.ldc + n;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const f32x4_t y = v(x);
                __builtin_memcpy(c + x * 4, &y, 16);
            }
        } else {
            uint16_t* c = (uint16_t*)q.c + m * q.ldc + n;
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
                const f32x4_t y = v(x), z = v(x + 1);
                const u32x4_t w = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(z[0], z[1]),
                                   pack_bf16x2(z[2], z[3])};
                __builtin_memcpy(c + x * 4, &w, 16);
            }
        }
    } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
            store_c4(q, m, n + x * 4, N, v(x));
    }
}

// The fast way.  Beside an MFMA per pair of fragments and k block, a pair costs
// four fused multiply-adds, and a row of pairs the product of its scales: the
// sums of a block may not stay in the MFMA's accumulator, since the next block's
// scales differ.  Those of a pair are issued three MFMAs later, so that no wave
// waits for its own; each MFMA's slot also carries its share of the k-step's LDS
// reads and loads to LDS, and the k-step holds no branch.
//
// 256 x 256 tiles (8 waves of 128 x 64) read each operand least often and 128 x
// 128 (4 waves of 64 x 64, two workgroups a compute unit) fill the device with
// smaller C.  What bounds 8192^3 (405 to 478 us, 2.3 to 2.7 PFLOP/s; a product
// without block scales reaches 3.0): the matrix cores are busy 0.65 to 0.72 of
// the time, and the clock falls to 1.75 GHz under the load; without its loads
// the kernel reaches 0.78.
template <class C, bool ROWB>
__global__ void __launch_bounds__(C::THREADS, 2) k_gemm_fp8(Params p, Fp8Params q)
{
    using LD = Fp8Loader<C>;
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::RING_BYTES + 2 * LD::SCALE_BYTES];
    lds_char* smem = (lds_char*)smem_raw;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / C::WN, wn = w % C::WN;

    const int32_t G = gridDim.x, b = blockIdx.x;
    const int32_t n_tiles = (b < p.tiles) ? (p.tiles - 1 - b) / G + 1 : 0;
    if (n_tiles == 0)
        return;
    clock_begin(p);
    LD ld;
    ld.init(p, q, w, lane);
    ld.cur = ld.first(p, q, 0, n_tiles, w);
    auto stage_at = [&](int st) { return smem + st * C::STAGE_BYTES; };
    auto scales_at = [&](int st) { return smem + C::RING_BYTES + st * LD::SCALE_BYTES; };

    // Lane (r16, g) reads chunks g and g + 4 of row r16 of each fragment (both
    // operands in the same order, so the order along k does not matter).
    const int swz = swz_k<64>(r16);
    const uint32_t lo = (uint32_t)r16 * 128u + (uint32_t)((g ^ swz) * 16), hi = lo ^ 64u;
    struct Raw {
        u32x4_t lo, hi;
    };
    Raw ar[4], br[C::FN];
    f32x4_t sar[C::FM / 4], sbr[ROWB ? C::FN : 1];
    float sb1 = 0.0f;
    auto read_a = [&](int st, int i) {
        const lds_char* t = stage_at(st) + wm * C::TM * 128 + i * 2048;
        ar[i & 3] = Raw{*(const LDS_AS u32x4_t*)(t + lo), *(const LDS_AS u32x4_t*)(t + hi)};
    };
    auto read_b = [&](int st, int j) {
        const lds_char* t = stage_at(st) + C::A_BYTES + wn * C::TN * 128 + j * 2048;
        br[j] = Raw{*(const LDS_AS u32x4_t*)(t + lo), *(const LDS_AS u32x4_t*)(t + hi)};
    };
    auto read_scales = [&](int st) {
        const lds_char* t = scales_at(st) + (wm * C::TM + r16 * C::FM) * 4;
#pragma unroll
        for (int i = 0; i < C::FM / 4; ++i)
            sar[i] = *(const LDS_AS f32x4_t*)(t + i * 16);
        const lds_char* u = scales_at(st) + (C::BM + wn * C::TN) * 4;
        if constexpr (ROWB) {
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                sbr[j] = *(const LDS_AS f32x4_t*)(u + (g * (4 * C::FN) + j * 4) * 4);
        } else {
            sb1 = *(const lds_f32*)u;
        }
    };

    // Position 0 whole; then what a k-step leaves behind: position 1 under way and
    // the first fragments of position 0 in registers.
    ld.fire_scales(ld.cur, scales_at(0), w);
#pragma unroll
    for (int t = 0; t < C::LOADS; ++t)
        ld.fire(ld.cur, t, stage_at(0), w);
    ld.step(false);
    wait_vmcnt<0>();
    block_barrier();
    read_a(0, 0);
    read_a(0, 1);
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
        read_b(0, j);

    // The MFMAs of a k-step go by pairs of fragment rows, column by column.  So in
    // the last pair a fragment of B has its last use two MFMAs before the next
    // one's, and its successor, the next k-step's, is read in between; it is
    // needed only after as many MFMAs, 2 * FN, whose time covers the read.  A's
    // fragments are read a pair ahead.  The barrier stands before the last pair:
    // by then the wave has read every fragment of the stage, so the stage can be
    // refilled and the next one be read.  The refill's loads go out one every
    // GAP MFMAs, into the next k-step.
    //
    // The partial sums of MFMA n are added to the running sums after MFMA n +
    // LAG, when they are sure to be there; the last LAG of a k-step in the next
    // one, with the scales they belong to (`held`).
    constexpr int NM = C::FM * C::FN, PAIR = 2 * C::FN, TAIL = NM - PAIR, LAG = 3, RING = 4, GAP = 2;
    constexpr auto row_of = [](int n) { return n / PAIR * 2 + n % 2; };
    constexpr auto col_of = [](int n) { return n % PAIR / 2; };
    // The load that goes out at MFMA n, counted from the barrier on; none: -1.
    constexpr auto load_at = [](int n) {
        const int t = n >= TAIL ? n - TAIL : n + PAIR;
        return t % GAP == 0 && t / GAP < C::LOADS ? t / GAP : -1;
    };
    static_assert(NM % RING == 0 && LAG < RING && LAG <= PAIR && C::LOADS * GAP <= NM && C::FM % 4 == 0,
                  "k-step schedule");
    [&]<int... NS>(std::integer_sequence<int, NS...>) {
        ((load_at(TAIL + NS) >= 0 ? ld.fire(ld.cur, load_at(TAIL + NS), stage_at(1), w) : (void)0), ...);
    }(std::make_integer_sequence<int, PAIR>{});
    f32x4_t part[RING];
    Fp8Frag<false> bf[C::FN], af[2];
    int s = 0;
    for (int32_t it = 0; it < n_tiles; ++it) {
        int32_t tm, tn, sp, u;
        tile_coords(p, b + it * G, G, tm, tn, sp, u);
        ld.nxt = ld.first(p, q, it + 1, n_tiles, w);
        f32x4_t acc[C::FM][C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < RING; ++i)
            part[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        float held[2] = {0.0f, 0.0f};
        auto add = [&](int n, float sa, const f32x4_t& sb) {
            f32x4_t& sum = acc[row_of(n)][col_of(n)];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[e] = __builtin_fmaf(part[n % RING][e], ROWB ? sa * sb[e] : sa, sum[e]);
        };
        // Nothing of the scalar loads before may be pending in the loop: scalar
        // and LDS loads share a counter but not an order, and the loop's waits
        // would then be for everything instead of for the fragments they need.
        wait_lgkm0();
        for (int32_t kt = 0; kt < p.k_steps; ++kt) {
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                bf[j] = Fp8Frag<false>(br[j].lo, br[j].hi);
            float sc[C::FM];
            // One slot of the schedule: an MFMA, what is loaded beside it, and
            // the sums of an earlier MFMA.
            auto slot = [&]<int n>() {
                constexpr int i = row_of(n), j = col_of(n), f = load_at(n);
                if constexpr (j == 0)
                    af[i & 1] = Fp8Frag<false>(ar[i & 3].lo, ar[i & 3].hi);
                part[n % RING] = block_sums(bf[j], af[i & 1]);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (j == 0)
                    read_a(n < TAIL ? s : s ^ 1, (i + 2) % C::FM);
                if constexpr (n >= TAIL && n % 2 == 1)
                    read_b(s ^ 1, (n - TAIL) / 2);
                if constexpr (f >= 0)
                    ld.fire(ld.cur, f, stage_at(n < TAIL ? s ^ 1 : s), w);
                // The step's scales: read at its start, needed LAG MFMAs on.
                if constexpr (n == 0)
                    read_scales(s);
                if constexpr (n == TAIL / 2 - 1)
                    ld.fire_scales(ld.cur, scales_at(s ^ 1), w);
                if constexpr (n == LAG) {
#pragma unroll
                    for (int x = 0; x < C::FM; ++x)
                        sc[x] = ROWB ? sar[x / 4][x % 4] : sar[x / 4][x % 4] * sb1;
                }
                if constexpr (n >= LAG)
                    add(n - LAG, sc[row_of(n - LAG)], sbr[ROWB ? col_of(n - LAG) : 0]);
                else if constexpr (!ROWB)
                    add(NM - LAG + n, held[row_of(NM - LAG + n) & 1], f32x4_t{});
                __builtin_amdgcn_sched_barrier(0);
            };
            [&]<int... NS>(std::integer_sequence<int, NS...>) {
                (slot.template operator()<NS>(), ...);
            }(std::make_integer_sequence<int, TAIL>{});
            ld.step(kt == p.k_steps - 2);
            // Every fragment of this stage is in registers and the next
            // position's loads have landed, here and, after the barrier, in
            // every wave: this stage takes the position after next.
            wait_lgkm0();
            wait_vmcnt<0>();
            block_barrier();
            [&]<int... NS>(std::integer_sequence<int, NS...>) {
                (slot.template operator()<TAIL + NS>(), ...);
            }(std::make_integer_sequence<int, PAIR>{});
            if constexpr (ROWB) {
#pragma unroll
                for (int n = NM - LAG; n < NM; ++n)
                    add(n, sc[row_of(n)], sbr[col_of(n)]);
            } else {
                held[0] = sc[C::FM - 2];
                held[1] = sc[C::FM - 1];
            }
            s ^= 1;
        }
        if constexpr (!ROWB) {
#pragma unroll
            for (int n = NM - LAG; n < NM; ++n)
                add(n, held[row_of(n) & 1], f32x4_t{});
        }
        if (p.splits > 1) {
            // Fragments of rows past M are not stored (nor read back).
            float* part = p.partial + (int64_t)(sp * p.span + u) * (C::BM * C::BN);
            const int64_t left = p.M - ((int64_t)tm * C::BM + wm * C::TM);
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
                    if (i * C::MF < left)
                        *(f32x4_t*)(part + (((w * C::FM + i) * C::FN + j) * 64 + lane) * 4) = acc[i][j];
        } else {
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                const int64_t m = (int64_t)tm * C::BM + wm * C::TM + i * 16 + r16;
                if (m < p.M)
                    store_c16(q, m, (int64_t)tn * C::BN + wn * C::TN + g * 16, p.N, [&](int x) { return acc[i][x]; });
            }
        }
    }
    wait_vmcnt<0>();   // the last, empty position's loads still write LDS
    clock_end(p);
}

// The exact way: 128 x 128 tiles, 4 waves of 64 x 64 each, two workgroups on a
// compute unit.  What bounds it is instruction issue: beside its MFMAs, each of
// which takes about 11 clocks of its SIMD's vector issue, a k-step costs a wave
// 128 conversions and 64 or, with row scales, 128 scalings (0.47 MFMA busy at
// 8192^3 with row scales, 0.54 with block scales; the same kernel with a quarter
// of the MFMAs and conversions takes 63% of the time, without its loads 80%).
// One wave's conversions overlap another's MFMAs through the two workgroups,
// which do not wait for each other; spreading them between the MFMAs of 16 x 16
// fragments by hand gave the same time (1040 us against 1060 at 8192^3).  A
// k-step goes in two halves of 64, so that the converted fragments of a half,
// the partial sums and the running sums fit the wave's 256 registers.
template <class C, bool ROWB>
__global__ void __launch_bounds__(C::THREADS, 2) k_gemm_fp8_exact(Params p, Fp8Params q)
{
    using LD = Fp8Loader<C>;
    static_assert(C::MF == 32, "32 x 32 MFMAs");
    __shared__ __attribute__((aligned(1024))) char smem_raw[C::RING_BYTES + 2 * LD::SCALE_BYTES];
    lds_char* smem = (lds_char*)smem_raw;
    const int lane = threadIdx.x & 63, r32 = lane & 31, h = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / C::WN, wn = w % C::WN;

    const int32_t G = gridDim.x, b = blockIdx.x;
    const int32_t n_tiles = (b < p.tiles) ? (p.tiles - 1 - b) / G + 1 : 0;
    if (n_tiles == 0)
        return;
    clock_begin(p);
    LD ld;
    ld.init(p, q, w, lane);
    ld.cur = ld.first(p, q, 0, n_tiles, w);
    auto stage_at = [&](int st) { return smem + st * C::STAGE_BYTES; };
    auto scales_at = [&](int st) { return smem + C::RING_BYTES + st * LD::SCALE_BYTES; };
    auto fire_all = [&](int st) {
        ld.fire_scales(ld.cur, scales_at(st), w);
#pragma unroll
        for (int t = 0; t < C::LOADS; ++t)
            ld.fire(ld.cur, t, stage_at(st), w);
    };

    // Lane (r32, h) reads chunks 4 k + 2 h and the next one of row r32 in half k.
    const int swz = swz_k<64>(r32);
    uint32_t at[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x)
            at[k][x] = (uint32_t)r32 * 128u + (uint32_t)(((4 * k + 2 * h + x) ^ swz) * 16);
    struct Raw {
        u32x4_t lo, hi;
    };
    auto read = [&](const lds_char* t, int k) {
        return Raw{*(const LDS_AS u32x4_t*)(t + at[k][0]), *(const LDS_AS u32x4_t*)(t + at[k][1])};
    };

    fire_all(0);
    int s = 0;
    for (int32_t it = 0; it < n_tiles; ++it) {
        int32_t tm, tn, sp, u;
        tile_coords(p, b + it * G, G, tm, tn, sp, u);
        ld.nxt = ld.first(p, q, it + 1, n_tiles, w);
        f32x16_t acc[C::FM][C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                acc[i][j] = f32x16_t{};
        for (int32_t kt = 0; kt < p.k_steps; ++kt) {
            // As in the fast kernel: this position has landed and the other
            // stage has been read, in every wave.
            wait_vmcnt<0>();
            wait_lgkm0();
            block_barrier();
            ld.step(kt == p.k_steps - 1);
            fire_all(s ^ 1);
            const lds_char* ta = stage_at(s) + wm * C::TM * 128;
            const lds_char* tb = stage_at(s) + C::A_BYTES + wn * C::TN * 128;
            f32x16_t part[C::FM][C::FN];
            Raw ar[C::FM], br[C::FN];
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
                ar[i] = read(ta + i * 4096, 0);
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                br[j] = read(tb + j * 4096, 0);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                Fp8Frag<true> af[C::FM], bf[C::FN];
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
                    af[i] = Fp8Frag<true>(ar[i].lo, ar[i].hi);
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
                    bf[j] = Fp8Frag<true>(br[j].lo, br[j].hi);
                __builtin_amdgcn_sched_barrier(0);
                if (k == 0) {
#pragma unroll
                    for (int i = 0; i < C::FM; ++i)
                        ar[i] = read(ta + i * 4096, 1);
#pragma unroll
                    for (int j = 0; j < C::FN; ++j)
                        br[j] = read(tb + j * 4096, 1);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < C::FM; ++i)
#pragma unroll
                        for (int j = 0; j < C::FN; ++j)
                            part[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                bf[j].v[x], af[i].v[x], k == 0 && x == 0 ? f32x16_t{} : part[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            // A's scales: one for each of the lane's rows.  B's: one, or those of
            // the lane's 16 columns in each fragment.
            const lds_f32* sa = (const lds_f32*)scales_at(s) + wm * C::TM + r32 * C::FM;
            const lds_f32* sb = (const lds_f32*)scales_at(s) + C::BM + wn * C::TN;
            float sai[C::FM];
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
                sai[i] = ROWB ? sa[i] : sa[i] * sb[0];
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                f32x4_t sbj[ROWB ? 4 : 1];
                if constexpr (ROWB) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        sbj[x] = *(const LDS_AS f32x4_t*)(sb + j * 32 + h * 16 + x * 4);
                }
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        acc[i][j][e] = __builtin_fmaf(part[i][j][e], ROWB ? sai[i] * sbj[e / 4][e % 4] : sai[i],
                                                      acc[i][j][e]);
            }
            s ^= 1;
        }
        if (p.splits > 1) {
            float* out = p.partial + (int64_t)(sp * p.span + u) * (C::BM * C::BN);
            const int64_t left = p.M - ((int64_t)tm * C::BM + wm * C::TM);
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (i * C::MF < left)
                            *(f32x4_t*)(out + ((((w * C::FM + i) * C::FN + j) * 4 + x) * 64 + lane) * 4) =
                            f32x4_t{acc[i][j][4 * x], acc[i][j][4 * x + 1], acc[i][j][4 * x + 2], acc[i][j][4 * x + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                const int64_t m = (int64_t)tm * C::BM + wm * C::TM + i * 32 + r32;
                if (m < p.M) {
#pragma unroll
                    for (int j = 0; j < C::FN; ++j)
                        store_c16(q, m, (int64_t)tn * C::BN + wn * C::TN + j * 32 + h * 16, p.N, [&](int x) {
                            return f32x4_t{acc[i][j][4 * x], acc[i][j][4 * x + 1], acc[i][j][4 * x + 2],
                                           acc[i][j][4 * x + 3]};
                        });
                }
            }
        }
    }
    wait_vmcnt<0>();   // the last, empty position's loads still write LDS
    clock_end(p);
}

// Sums the k chunks' partial tiles in chunk order and stores C.  A thread takes
// 4 consecutive columns, in the order the partial tiles are stored in: the
// waves' fragments, for 32 x 32 MFMAs 4 quarters each, then the lanes.
template <class C>
__global__ void __launch_bounds__(256) k_reduce_fp8(Params p, Fp8Params q)
{
    constexpr int QUADS = C::BM * C::BN / 4;
    const int64_t total = (int64_t)p.span * QUADS;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
        const int32_t u = (int32_t)(id / QUADS);
        const int at = (int)(id % QUADS);
        constexpr int QF = C::MF == 32 ? 4 : 1;
        const int lane = at & 63, x = at / 64 % QF, f = at / (64 * QF);
        const int j = f % C::FN, i = f / C::FN % C::FM, w = f / (C::FN * C::FM);
        int32_t tm, tn;
        raster_tile(p, u, tm, tn);
        const int64_t m = (int64_t)tm * C::BM + w / C::WN * C::TM + i * C::MF + lane % C::MF;
        const int64_t n = (int64_t)tn * C::BN + w % C::WN * C::TN +
                          (C::MF == 32 ? j * 32 + (lane >> 5) * 16 + x * 4 : (lane >> 4) * (4 * C::FN) + j * 4);
        if (m >= p.M)
            continue;
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t sp = 0; sp < p.splits; ++sp)
            v += *(const f32x4_t*)(p.partial + (int64_t)(sp * p.span + u) * (C::BM * C::BN) + at * 4);
        store_c4(q, m, n, p.N, v);
    }
}

// ---------------------------------------------------------------------------
// Few rows, or little work: the product is bound by B's bytes and by latency.  A
// workgroup of 8 waves takes MF x NF fragments of C; its waves share out the k
// blocks (wave w takes blocks w, w + 8, ...), stream their fragments from global
// memory straight into registers, DEPTH blocks in use and DEPTH more in flight,
// and add their sums through LDS in wave order.  So every compute unit has loads
// in flight over the whole of k even where C gives few workgroups, with no
// second launch; only a long k against very few columns is split over several
// workgroups, whose sums a second launch adds in order.  Bound by B's bytes where
// there are many columns (1 x 8192 x 8192: 13.0 us, 5.2 TB/s), by the latency of a
// wave's blocks where there are few (300 x 1000 x 4112, 4 blocks a wave: 11.0 us).
//
// ANY takes operands of any alignment and stride and any K >= 16 (otherwise rows
// start on 16-byte boundaries and K is a multiple of 16), by the same 16-byte
// loads at any byte (4 x 4096 x 4096 rows 4100 apart 5.8 us and 4097 apart 7.2; as
// aligned dwords put together, 6.5 and 6.8, with a register more for each load): a
// chunk that reaches past the row's end is read from its last 16 bytes and shifted
// into place, so nothing past the row is read, and rows past the matrix repeat its
// last one, whose sums no one stores.
// ---------------------------------------------------------------------------
struct SkinnyParams {
    const char* a;
    const char* b;
    int64_t M, N, lda, ldb;
    int32_t tiles_m, tiles_n;
    int32_t chunk;           // k blocks per workgroup: all, or a k chunk's (blockIdx.y counts the chunks)
    float* partial;          // with several chunks: M x N sums of each
};

constexpr int kSkinnyWaves = 8;

// 16 bytes without their first `cut` (0 .. 16), zeros after the rest.
__device__ __forceinline__ u32x4_t without_first(u32x4_t v, int cut)
{
    uint64_t x[2];
    __builtin_memcpy(x, &v, 16);
    const int s = (cut & 7) * 8;
    const uint64_t lo = cut >= 8 ? x[1] : x[0], hi = cut >= 8 ? 0u : x[1];
    x[0] = s ? (lo >> s) | (hi << (64 - s)) : lo;
    x[1] = hi >> s;
    if (cut >= 16)
        x[0] = x[1] = 0;
    __builtin_memcpy(&v, x, 16);
    return v;
}

template <int MF, int NF, int DEPTH, bool ROWB, bool EXACT, bool ANY>
__global__ void __launch_bounds__(kSkinnyWaves * 64) k_gemm_fp8_skinny(SkinnyParams p, Fp8Params q)
{
    __shared__ __attribute__((aligned(16))) f32x4_t sums[kSkinnyWaves][MF * NF][64];
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The row tiles of one column tile go to one XCD (workgroups are dealt to the
    // 8 XCDs in turn), which then reads B once.
    const int32_t x = blockIdx.x & 7, y = blockIdx.x >> 3;
    const int32_t tm = y % p.tiles_m, tn = y / p.tiles_m * 8 + x;
    if (tn >= p.tiles_n)
        return;
    const int64_t m0 = (int64_t)tm * (MF * 16), n0 = (int64_t)tn * (NF * 16);
    const int32_t kb_first = blockIdx.y * p.chunk, kb_end = min(kb_first + p.chunk, q.kblocks);
    if (p.partial) {
        q.c = (char*)(p.partial + blockIdx.y * p.M * p.N);
        q.ldc = p.N;
        q.c_fp32 = 1;
    }

    // Rows past the end read as zeros: their offset is past the resource.
    const int64_t a_rows = min(p.M - m0, (int64_t)MF * 16), b_rows = min(p.N - n0, (int64_t)NF * 16);
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + m0 * p.lda, (a_rows - 1) * p.lda + q.K);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.b + n0 * p.ldb, (b_rows - 1) * p.ldb + q.K);
    // Lanes 4 i .. 4 i + 3 read 64 consecutive bytes of a row: the cache takes four
    // such lanes at a time, lanes of four rows one by one.  An MFMA's lane (r16, g)
    // then takes chunk g of row r16 from the lane that read it (64 x 4096 x 4096:
    // 10.5 us read in the MFMA's order, 8.1 so; the exchange is 1.1 of it).
    const int lr = (lane >> 2 & 3) * 4 + (lane >> 4), lc = lane & 3;
    const int from = ((lane & 3) * 16 + (lane & 12) + g) * 4;
    auto mfma_order = [&](u32x4_t v) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v[e]);
        return v;
    };
    uint32_t va[MF] = {}, vb[NF] = {};
    const char *pa[MF] = {}, *pb[NF] = {};
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const int row = i * 16 + lr;
        if constexpr (ANY)
            pa[i] = p.a + (m0 + min(row, (int)a_rows - 1)) * p.lda;
        else
            va[i] = row < a_rows ? (uint32_t)row * (uint32_t)p.lda + lc * 16 : kOOB;
    }
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const int row = j * 16 + lr;
        if constexpr (ANY)
            pb[j] = p.b + (n0 + min(row, (int)b_rows - 1)) * p.ldb;
        else
            vb[j] = row < b_rows ? (uint32_t)row * (uint32_t)p.ldb + lc * 16 : kOOB;
    }

    struct Block {
        u32x4_t a[MF][2], b[NF][2];
        float sa[MF], sb[ROWB ? NF * 4 : 1];
    };
    // ANY: where half h of block kb is read, and how many of its bytes precede it.
    auto place = [&](int32_t kb, int h, int32_t& at) {
        const int32_t k = kb * kBlock + (h * 4 + lc) * 16;
        at = min(k, (int32_t)q.K - 16);
        return min(k - at, 16);
    };
    auto load = [&](Block& v, int32_t kb) {
        // The halves of a line one after the other, while the line is in the L1.
        auto halves = [&](u32x4_t (&to)[2], const char* row, const __amdgpu_buffer_rsrc_t& rsrc, uint32_t voff) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (ANY) {
                    int32_t at;
                    place(kb, h, at);
                    __builtin_memcpy(&to[h], row + at, 16);
                } else {
                    const bool ok = kb * kBlock + (h * 4 + lc) * 16 < (int32_t)q.K;
                    to[h] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                            rsrc, ok ? voff : kOOB, kb * kBlock + h * 64, 0));
                }
            }
        };
#pragma unroll
        for (int j = 0; j < NF; ++j)
            halves(v.b[j], pb[j], rb, vb[j]);
#pragma unroll
        for (int i = 0; i < MF; ++i)
            halves(v.a[i], pa[i], ra, va[i]);
        // The scales, each checked against the end of its array.
        const bool in = kb < kb_end;
        const __amdgpu_buffer_rsrc_t rsa = make_rsrc(q.sa + (in ? kb * q.ldsa : 0) + m0, in ? a_rows * 4 : 0);
#pragma unroll
        for (int i = 0; i < MF; ++i)
            v.sa[i] = as_float(__builtin_amdgcn_raw_buffer_load_b32(rsa, r16 * 4, i * 64, 0));
        const __amdgpu_buffer_rsrc_t rsb =
            make_rsrc(q.sb + (in ? kb * q.ldsb : 0) + (n0 >> q.sb_shift), in ? (ROWB ? b_rows * 4 : 4) : 0);
#pragma unroll
        for (int e = 0; e < (ROWB ? NF * 4 : 1); ++e)
            v.sb[e] = as_float(
                __builtin_amdgcn_raw_buffer_load_b32(rsb, ROWB ? g * 16 + e % 4 * 4 : 0, ROWB ? e / 4 * 64 : 0, 0));
    };

    f32x4_t acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
            acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    auto compute = [&](const Block& v, int32_t kb) {
        const bool tail = ANY && (kb + 1) * kBlock > q.K;
        auto frag = [&](const u32x4_t (&raw)[2]) {
            u32x4_t x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x[h] = raw[h];
                if (tail) {
                    int32_t at;
                    x[h] = without_first(x[h], place(kb, h, at));
                }
                x[h] = mfma_order(x[h]);
            }
            return Fp8Frag<EXACT>(x[0], x[1]);
        };
        Fp8Frag<EXACT> bf[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j)
            bf[j] = frag(v.b[j]);
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const Fp8Frag<EXACT> af = frag(v.a[i]);
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const f32x4_t d = block_sums(bf[j], af);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = __builtin_fmaf(d[e], v.sa[i] * v.sb[ROWB ? j * 4 + e : 0], acc[i][j][e]);
            }
        }
    };

    // A block past the end loads nothing and is not computed (its bytes read as
    // zeros, but a scale may be infinite).
    Block cur[DEPTH], nxt[DEPTH];
    constexpr int STEP = kSkinnyWaves * DEPTH;
    auto load_all = [&](Block (&v)[DEPTH], int32_t kb0) {
        if (kb0 < kb_end) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
                load(v[d], kb0 + d * kSkinnyWaves);
        }
    };
    auto compute_all = [&](const Block (&v)[DEPTH], int32_t kb0) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (kb0 + d * kSkinnyWaves < kb_end)
                compute(v[d], kb0 + d * kSkinnyWaves);
    };
    // Workgroups start at different places along k: with a power-of-two row
    // stride, all of them reading the same columns at once fall on the same few
    // memory channels (8192 x 8192 weight, one token: 18.4 us, and 12.8 so).
    const int32_t rounds = (kb_end - kb_first + STEP - 1) / STEP, rot = (int32_t)(blockIdx.x % (unsigned)rounds);
    auto at = [&](int32_t t) {
        return t < rounds ? kb_first + w + (t + rot < rounds ? t + rot : t + rot - rounds) * STEP : kb_end;
    };
    load_all(cur, at(0));
    for (int32_t t = 0; t < rounds; t += 2) {
        load_all(nxt, at(t + 1));
        compute_all(cur, at(t));
        load_all(cur, at(t + 2));
        compute_all(nxt, at(t + 1));
    }

#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
            sums[w][i * NF + j][lane] = acc[i][j];
    __syncthreads();
    for (int f = w; f < MF * NF; f += kSkinnyWaves) {
        f32x4_t v = sums[0][f][lane];
#pragma unroll
        for (int z = 1; z < kSkinnyWaves; ++z)
            v += sums[z][f][lane];
        const int64_t m = m0 + f / NF * 16 + r16;
        if (m < p.M)
            store_c4(q, m, n0 + f % NF * 16 + g * 4, p.N, v);
    }
}

// Zero-padded copies, dst_cols bytes (a multiple of 16) a row, of the operands
// that do not fit the tiles' loads: those with rows, one launch for both.
struct PadParams {
    const uint8_t* src[2];
    uint8_t* dst[2];
    int64_t rows[2], ld[2];
};

__global__ void __launch_bounds__(256) k_pad_copy8(PadParams p, int64_t src_cols, int64_t dst_cols)
{
    const int64_t per_row = dst_cols / 16, first = p.rows[0] * per_row, total = first + p.rows[1] * per_row;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
        const int o = id >= first;
        const int64_t at = o ? id - first : id, r = at / per_row, c = (at - r * per_row) * 16;
        const uint8_t* s = p.src[o] + r * p.ld[o] + c;
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (c + 16 <= src_cols) {
            __builtin_memcpy(&v, s, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 15; ++e)
                if (c + e < src_cols)
                    v[e >> 2] |= (uint32_t)s[e] << (8 * (e & 3));
        }
        *(u32x4_t*)(p.dst[o] + r * dst_cols + c) = v;
    }
}

__global__ void __launch_bounds__(256) k_zero_c(Fp8Params q, int64_t M, int64_t N)
{
    const int64_t quads = (N + 3) / 4, total = M * quads;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256)
        store_c4(q, id / quads, id % quads * 4, N, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
unsigned flat_grid(int64_t threads)
{
    const int64_t n = (threads + 255) / 256;
    return (unsigned)(n < 65536 ? n : 65536);
}

// C from the k chunks' sums, added in chunk order, 4 columns a thread.
__global__ void __launch_bounds__(256) k_reduce_chunks(SkinnyParams p, Fp8Params q, int32_t chunks)
{
    const int64_t per_row = (p.N + 3) / 4, step = (int64_t)gridDim.x * 256;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < p.M * per_row; t += step) {
        const int64_t m = t / per_row, n = t % per_row * 4;
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t z = 0; z < chunks; ++z) {
            const float* x = p.partial + (z * p.M + m) * p.N + n;
            f32x4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
            if (n + 4 <= p.N) {
                __builtin_memcpy(&y, x, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (n + e < p.N)
                        y[e] = x[e];
            }
            v += y;
        }
        store_c4(q, m, n, p.N, v);
    }
}

template <int MF, int NF, int DEPTH>
int launch_skinny(SkinnyParams p, const Fp8Params& q, const gemm_fp8_plan_t& pl, bool any, TempMem& tm, hipStream_t s)
{
    p.tiles_m = (int32_t)((p.M + MF * 16 - 1) / (MF * 16));
    p.tiles_n = (int32_t)((p.N + NF * 16 - 1) / (NF * 16));
    p.chunk = (int32_t)pl.k_blocks;
    const bool exact = pl.exact;
    const int64_t chunks = pl.k_splits;
    void* ws = nullptr;
    hipEvent_t done = nullptr;
    if (chunks > 1) {
        const int rc = temp_take(tm, pl.workspace_bytes, s, &ws, &done);
        if (rc != GEMM_OK)
            return rc;
    }
    p.partial = (float*)ws;
    const dim3 g((unsigned)(pl.grid / chunks), (unsigned)chunks), b(kSkinnyWaves * 64);
    // Operands of any alignment take 64-bit addresses: less depth leaves them the
    // registers.
    auto run = [&]<bool ROWB, bool EXACT>() {
        if constexpr (MF * NF < 16) {
            if (any) {
                hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fp8_skinny<MF, NF, 1, ROWB, EXACT, true>), g, b, 0, s, p, q);
                return;
            }
        }
        hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fp8_skinny<MF, NF, DEPTH, ROWB, EXACT, false>), g, b, 0, s, p, q);
    };
    const bool rowb = q.sb_shift == 0;
    if constexpr (MF * NF < 16) {
        if (rowb && exact)
            run.template operator()<true, true>();
        else if (rowb)
            run.template operator()<true, false>();
        else if (exact)
            run.template operator()<false, true>();
        else
            run.template operator()<false, false>();
    } else {
        // This form spills 8 registers, the others 65 to 146: they take other shapes.
        run.template operator()<false, false>();
    }
    int rc = launched();
    if (chunks > 1) {
        if (rc == GEMM_OK) {
            hipExtLaunchKernelGGL(k_reduce_chunks, dim3(flat_grid(p.M * ((p.N + 3) / 4))), dim3(256), 0, s, nullptr,
                                  done, 0, p, q, (int32_t)chunks);
            rc = launched();
        }
        const int frc = temp_give(tm, ws, s, rc == GEMM_OK && done != nullptr);
        rc = rc != GEMM_OK ? rc : frc;
    }
    return rc;
}

// Sums of up to this many blocks are computed exactly (see the top).
constexpr int kShortBlocks = 2;

// Estimated times, in ns, by which a call chooses its kernel and its splits;
// what they were read off is measured on an MI355X and noted at each.  Only their
// order matters, and the launch itself is common to all.
struct TileTimes {
    int64_t alone, shared;   // a k-step of a workgroup, of each of two on a compute unit
};
constexpr TileTimes kFast256{1550, 1550 * 2};   // 8192^3: 256 k-steps per compute unit in 0.42 ms
// 1024 x 1024 x 32768 unsplit 182 us for 256 k-steps; 8 splits of 32, two
// workgroups on every compute unit, 54 us with the reduction.
constexpr TileTimes kFast128{700, 1000};
constexpr TileTimes kExact128{1300, 2200};      // the same shape, 80 us with 8 splits
// A split: the reduction's launch, and a partial tile's way to memory and back
// (128 x 4096 x 4096: 20.2 us with 4 splits, 22.2 with 8, 27.9 with none).
constexpr int64_t kSplitLaunch = 6500, kSplitTile = 38;
// Few-rows kernel: bytes a compute unit's workgroup reads per ns, all of them
// reading (64 x 8192 x 8192 in 64 x 32: 20 us; fp32 C converts every byte), in
// fragments of 4 x 4 (256 x 4096 x 4096: 16 us), and what another workgroup in
// turn costs beside its bytes, for each of its fragments (1039 x 1792 x 256 to
// fp32, 4 turns of 8 fragments: 12.5 us, where tiles take 9.7).
constexpr int64_t kSkinnyBytes[2] = {45, 40}, kSkinnyBytes44 = 37, kSkinnyTurn = 190;
constexpr int64_t kChunkBytes = 2000;   // k chunks: bytes per ns of their sums, written and read

// The padded copies of operands that do not fit the tiles' loads, beside their
// bytes: a launch and the memory's event.
constexpr int64_t kPadLaunch = 5000;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t tiles_time(const TileTimes& t, int64_t tile, int per_cu, int64_t M, int64_t N, int64_t kblocks, int64_t splits,
                   int cus)
{
    const int64_t items = ceil_div(M, tile) * ceil_div(N, tile) * splits, steps = ceil_div(kblocks, splits);
    const int64_t run = items <= cus ? steps * t.alone
                        : per_cu == 1 ? ceil_div(items, cus) * steps * t.alone
                                      : ceil_div(items, 2 * (int64_t)cus) * steps * t.shared;
    return run + (splits > 1 ? kSplitLaunch + kSplitTile * items * (M < tile ? M : tile) / tile : 0);
}

// The number of k chunks that is estimated fastest, among those that leave a
// chunk 4 k-steps and fit the card at once.
int64_t choose_fp8_splits(const TileTimes& t, int64_t M, int64_t N, int64_t kblocks, int cus, int64_t* time)
{
    int64_t best = 1;
    *time = tiles_time(t, 128, 2, M, N, kblocks, 1, cus);
    for (int64_t s = 2; s <= kMaxSplits && s * 4 <= kblocks; ++s) {
        if (ceil_div(M, 128) * ceil_div(N, 128) * s > 2 * (int64_t)cus)
            break;
        const int64_t v = tiles_time(t, 128, 2, M, N, kblocks, s, cus);
        if (v < *time) {
            *time = v;
            best = s;
        }
    }
    return best;
}

template <class C>
int launch_tiles(Params p, const Fp8Params& q, const gemm_fp8_plan_t& pl, TempMem& tm, hipStream_t s)
{
    p.tiles_m = (int32_t)((p.M + C::BM - 1) / C::BM);
    p.tiles_n = (int32_t)((p.N + C::BN - 1) / C::BN);
    p.splits = (int32_t)pl.k_splits;
    // The load cursor runs two positions ahead and crosses at most one tile
    // border: a single k-step is followed by one that reads zeros.
    p.k_steps = pl.k_blocks < 2 ? 2 : (int32_t)pl.k_blocks;
    p.ksplit = (int64_t)p.k_steps * (kBlock / 2);
    p.tiles_mn = p.span = (int32_t)pl.tiles;
    p.tile_base = 0;
    p.tiles = p.span * p.splits;
    p.group_m = 4;
    p.partial = nullptr;
    void* ws = nullptr;
    hipEvent_t done = nullptr;
    if (p.splits > 1) {
        const int rc = temp_take(tm, pl.workspace_bytes, s, &ws, &done);
        if (rc != GEMM_OK)
            return rc;
        p.partial = (float*)ws;
    }
    const dim3 grid((unsigned)pl.grid), block(C::THREADS);
    const bool rowb = q.sb_shift == 0;
    if constexpr (C::MF == 32) {
        if (rowb)
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fp8_exact<C, true>), grid, block, 0, s, p, q);
        else
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fp8_exact<C, false>), grid, block, 0, s, p, q);
    } else {
        if (rowb)
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fp8<C, true>), grid, block, 0, s, p, q);
        else
            hipLaunchKernelGGL(HIP_KERNEL_NAME(k_gemm_fp8<C, false>), grid, block, 0, s, p, q);
    }
    int rc = launched();
    if (p.splits > 1) {
        if (rc == GEMM_OK) {
            hipExtLaunchKernelGGL(k_reduce_fp8<C>, dim3(flat_grid(pl.tiles * (C::BM * C::BN / 4))), dim3(256), 0, s,
                                  nullptr, done, 0, p, q);
            rc = launched();
        }
        const int frc = temp_give(tm, ws, s, rc == GEMM_OK && done != nullptr);
        rc = rc != GEMM_OK ? rc : frc;
    }
    return rc;
}

// The product in tiles, on operands whose rows start on 16-byte boundaries, K a
// multiple of 16.
int run_tiles(int64_t M, int64_t N, const char* A, int64_t lda, const char* B, int64_t ldb, const Fp8Params& q,
              const gemm_fp8_plan_t& pl, TempMem& tm, hipStream_t s)
{
    Params p;
    memset(&p, 0, sizeof p);
    p.A = A;
    p.B = B;
    p.M = M;
    p.N = N;
    p.K = q.K / 2;
    p.lda = lda / 2;
    p.ldb = ldb / 2;
    p.clock_on = g_clock_on.load(std::memory_order_relaxed) ? 1u : 0u;
    if (pl.exact)
        return launch_tiles<Fp8Cfg<128, 128, 2, 2, 32>>(p, q, pl, tm, s);
    if (pl.rows == 256)
        return launch_tiles<Fp8Cfg<256, 256, 2, 4>>(p, q, pl, tm, s);
    return launch_tiles<Fp8Cfg<128, 128, 2, 2>>(p, q, pl, tm, s);
}

// The few-rows kernel's shapes: rows in fragments of 16, and as many columns as
// keep the most compute units busy for the fewest bytes.
constexpr struct {
    int mf, nf;
} kShapes[] = {{1, 1}, {1, 2}, {2, 2}, {4, 2}, {4, 4}};

// Workgroups of a k chunk: a multiple of 8 column tiles, each for one of the 8
// XCDs.  A launch's threads have to stay below 2^32, 2^23 workgroups.
int64_t skinny_grid(int64_t M, int64_t N, int64_t rows, int64_t cols)
{
    return ceil_div(M, rows) * ceil_div(ceil_div(N, cols), 8) * 8;
}

// The kernel, k chunks and launch of a product, from its sizes alone: `rowb` for
// row scales of B, a_fits and b_fits for operands whose rows start on 16-byte
// boundaries.  The call runs what stands here.
int plan_fp8(int64_t M, int64_t N, int64_t K, bool rowb, bool exact, bool a_fits, bool b_fits, int cus,
             gemm_fp8_plan_t* out)
{
    const int64_t kblocks = ceil_div(K, kBlock);
    exact = exact || kblocks <= kShortBlocks;
    a_fits = a_fits && K % 16 == 0;
    b_fits = b_fits && K % 16 == 0;
    const TileTimes& t128 = exact ? kExact128 : kFast128;
    int64_t time128 = 0;
    const int64_t splits = choose_fp8_splits(t128, M, N, kblocks, cus, &time128);

    // k chunks where few columns leave compute units idle, each with two blocks or
    // more a wave (32 x 624 x 13056: 17 us, 8.9 with chunks).  Not in the shape of 4
    // x 4 fragments, whose few waves with much each do not keep up with memory (32 x
    // 3264 x 18176: 32 us in 5 chunks, tiles 17.5).
    const bool any = !a_fits || !b_fits;
    int shape = -1;
    int64_t skinny = 0, chunks = 1;
    for (int i = 0; i < (exact || any || rowb ? 4 : 5); ++i) {
        const int64_t rows = kShapes[i].mf * 16, cols = kShapes[i].nf * 16;
        const int64_t groups = ceil_div(M, rows) * ceil_div(N, cols);
        if (skinny_grid(M, N, rows, cols) >= (int64_t)1 << 22)
            continue;   // far from few rows, and past what a launch takes
        for (int64_t c = 1; c <= kMaxSplits; ++c) {
            if (c > 1 && (i == 4 || groups * c > cus || kblocks < c * 2 * kSkinnyWaves))
                break;
            const int64_t turns = ceil_div(groups * c, cus), rate = i == 4 ? kSkinnyBytes44 : kSkinnyBytes[exact];
            const int64_t v = turns * ((M < rows ? M : rows) + cols) * ceil_div(kblocks, c) * kBlock / rate +
                              (turns - 1) * kSkinnyTurn * kShapes[i].mf * kShapes[i].nf +
                              (c > 1 ? kSplitLaunch + c * M * N * 8 / kChunkBytes : 0);
            if (shape < 0 || v < skinny) {
                shape = i;
                skinny = v;
                chunks = c;
            }
        }
    }

    gemm_fp8_plan_t p;
    memset(&p, 0, sizeof p);
    p.exact = exact;
    p.few_rows = shape >= 0 && skinny < time128 + (any ? kPadLaunch : 0) && (!any || K >= 16);
    if (p.few_rows) {
        p.rows = kShapes[shape].mf * 16;
        p.cols = kShapes[shape].nf * 16;
        p.threads = kSkinnyWaves * 64;
        p.k_blocks = ceil_div(kblocks, chunks);
        p.k_splits = ceil_div(kblocks, p.k_blocks);   // no empty chunk
        p.tiles = ceil_div(M, p.rows) * ceil_div(N, p.cols);
        p.grid = skinny_grid(M, N, p.rows, p.cols) * p.k_splits;
        p.workspace_bytes = p.k_splits > 1 ? p.k_splits * M * N * 4 : 0;
        *out = p;
        return GEMM_OK;
    }
    // The exact way takes 128 x 128 tiles at any size: its fragments are twice
    // as large, and beside more running sums they do not fit a wave's registers.
    const bool big = !exact && tiles_time(kFast256, 256, 1, M, N, kblocks, 1, cus) < time128;
    p.rows = p.cols = big ? 256 : 128;
    p.threads = big ? 512 : 256;
    p.k_blocks = ceil_div(kblocks, big ? 1 : splits);
    p.k_splits = ceil_div(kblocks, p.k_blocks);
    p.tiles = ceil_div(M, p.rows) * ceil_div(N, p.cols);
    if (p.tiles * kMaxSplits > INT32_MAX)
        return GEMM_ERR_UNSUPPORTED_SHAPE;
    const int64_t slots = (int64_t)cus * (big ? 1 : 2);
    p.grid = p.tiles * p.k_splits < slots ? p.tiles * p.k_splits : slots;
    p.workspace_bytes = p.k_splits > 1 ? p.tiles * p.k_splits * p.rows * p.cols * 4 : 0;
    const int64_t K16 = (K + 15) & ~(int64_t)15;
    p.pad_bytes = (a_fits ? 0 : align256(M * K16)) + (b_fits ? 0 : align256(N * K16));
    *out = p;
    return GEMM_OK;
}

// The product by its plan.
int run_fp8(int64_t M, int64_t N, const char* A, int64_t lda, bool a_fits, const char* B, int64_t ldb, bool b_fits,
            Fp8Params q, const gemm_fp8_plan_t& pl, TempMem& tm, hipStream_t s)
{
    const bool any = !a_fits || !b_fits;
    if (pl.few_rows) {
        const SkinnyParams p{A, B, M, N, lda, ldb, 0, 0, 0, nullptr};
        switch (pl.rows * 64 + pl.cols) {
        case 16 * 64 + 16: return launch_skinny<1, 1, 2>(p, q, pl, any, tm, s);
        case 16 * 64 + 32: return launch_skinny<1, 2, 2>(p, q, pl, any, tm, s);
        case 32 * 64 + 32: return launch_skinny<2, 2, 2>(p, q, pl, any, tm, s);
        case 64 * 64 + 32: return launch_skinny<4, 2, 1>(p, q, pl, any, tm, s);
        default: return launch_skinny<4, 4, 1>(p, q, pl, any, tm, s);
        }
    }

    void* ws = nullptr;
    int rc = GEMM_OK;
    if (any) {
        const int64_t K16 = (q.K + 15) & ~(int64_t)15;
        const int64_t a_pad = a_fits ? 0 : align256(M * K16);
        rc = temp_take(tm, pl.pad_bytes, s, &ws);
        if (rc != GEMM_OK)
            return rc;
        const PadParams c{{(const uint8_t*)A, (const uint8_t*)B}, {(uint8_t*)ws, (uint8_t*)ws + a_pad},
                          {a_fits ? 0 : M, b_fits ? 0 : N}, {lda, ldb}};
        hipLaunchKernelGGL(k_pad_copy8, dim3(flat_grid((c.rows[0] + c.rows[1]) * (K16 / 16))), dim3(256), 0, s, c, q.K,
                           K16);
        rc = launched();
        if (!a_fits) {
            A = (const char*)c.dst[0];
            lda = K16;
        }
        if (!b_fits) {
            B = (const char*)c.dst[1];
            ldb = K16;
        }
        q.K = K16;   // the copies' zeros extend K to the 16-byte grid
    }
    if (rc == GEMM_OK)
        rc = run_tiles(M, N, A, lda, B, ldb, q, pl, tm, s);
    const int frc = temp_give(tm, ws, s);
    return rc != GEMM_OK ? rc : frc;
}

bool fp8_exact(int c_type) { return (c_type & GEMM_FP8_EXACT) != 0 || c_type == GEMM_TYPE_FP32; }

int fp8_shape(int64_t M, int64_t N, int64_t K, int b_block_rows, int c_type)
{
    const int type = c_type & ~GEMM_FP8_EXACT;
    if (M < 0 || N < 0 || K < 0 || (b_block_rows != 1 && b_block_rows != kBlock) ||
        (type != GEMM_TYPE_BF16 && type != GEMM_TYPE_FP32))
        return GEMM_ERR_INVALID_VALUE;
    return M > kMaxRows || N > kMaxLd || K > kMaxLd ? GEMM_ERR_UNSUPPORTED_SHAPE : GEMM_OK;
}

}  // namespace

extern "C" int gemm_fp8_bt(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const float* SA, int64_t ldsa,
                           const void* B, int64_t ldb, const float* SB, int64_t ldsb, int b_block_rows, void* C,
                           int64_t ldc, int c_type, void* stream)
{
    if (const int rc = fp8_shape(M, N, K, b_block_rows, c_type))
        return rc;
    const bool exact = fp8_exact(c_type);
    c_type &= ~GEMM_FP8_EXACT;
    if (M == 0 || N == 0)
        return GEMM_OK;
    const int64_t kblocks = (K + kBlock - 1) / kBlock, sb_cols = b_block_rows == 1 ? N : (N + kBlock - 1) / kBlock;
    const Operand c{C, M, N, ldc, c_type == GEMM_TYPE_FP32 ? 4 : 2};
    const Operand in[] = {{A, M, K, lda, 1}, {B, N, K, ldb, 1}, {SA, kblocks, M, ldsa, 4}, {SB, kblocks, sb_cols, ldsb, 4}};
    int rc = check_operand(c);
    if (rc == GEMM_OK && K > 0)
        rc = check_operands(in, 4);
    if (rc != GEMM_OK)
        return rc;
    if (K > 0)
        for (const Operand& o : in)
            if (meet(c, o))
                return GEMM_ERR_ALIAS;
    int cus = 0;
    TempMem tm;
    rc = device_info(&cus, &tm.pool, nullptr, &tm.info);
    if (rc != GEMM_OK)
        return rc;
    hipStream_t s = (hipStream_t)stream;
    Fp8Params q{SA, SB, (char*)C, ldsa, ldsb, ldc, K, sb_cols, (int32_t)kblocks, b_block_rows == 1 ? 0 : 7,
                c_type == GEMM_TYPE_FP32};
    if (K == 0) {
        hipLaunchKernelGGL(k_zero_c, dim3(flat_grid(M * ((N + 3) / 4))), dim3(256), 0, s, q, M, N);
        return launched();
    }
    // A single row has no stride: give it one that suits.
    const int64_t K16 = (K + 15) & ~(int64_t)15;
    if (M == 1)
        lda = K16;
    if (N == 1)
        ldb = K16;
    auto fits = [&](const void* ptr, int64_t ld) {
        return K % 16 == 0 && ld % 16 == 0 && ld <= 2 * kMaxLd && ((uintptr_t)ptr & 15) == 0;
    };
    const bool a_fits = fits(A, lda), b_fits = fits(B, ldb);
    gemm_fp8_plan_t pl;
    rc = plan_fp8(M, N, K, b_block_rows == 1, exact, a_fits, b_fits, cus, &pl);
    if (rc != GEMM_OK)
        return rc;
    return run_fp8(M, N, (const char*)A, lda, a_fits, (const char*)B, ldb, b_fits, q, pl, tm, s);
}

extern "C" int gemm_fp8_plan_cus(int64_t M, int64_t N, int64_t K, int b_block_rows, int c_type, int a_aligned,
                                 int b_aligned, int compute_units, gemm_fp8_plan_t* out)
{
    if (!out || compute_units < 1)
        return GEMM_ERR_INVALID_VALUE;
    if (const int rc = fp8_shape(M, N, K, b_block_rows, c_type))
        return rc;
    if (M == 0 || N == 0 || K == 0) {
        memset(out, 0, sizeof *out);
        return GEMM_OK;
    }
    return plan_fp8(M, N, K, b_block_rows == 1, fp8_exact(c_type), a_aligned != 0, b_aligned != 0, compute_units, out);
}
