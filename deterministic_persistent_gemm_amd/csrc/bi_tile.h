// bi_tile.h -- one output tile of C = A . B^T per workgroup, operands streamed
// through an LDS ring: the kernel behind the gated linear layer, the backward
// passes and the 4-bit product.
//
//   C[m, n] = sum_k A(m, k) B(n, k)
//
// Each operand is stored either by rows (an output row's k values are
// contiguous: activations and nn.Linear weights in a forward product) or by
// columns (a memory row holds one k of every output row: the weight in
// dx = dy W, both operands in dw = dy^T x).  Column operands are read from LDS
// with the transposing read, so no operand is ever transposed in memory.
//
// Numerics: one fp32 accumulator per output element, threaded through every
// slice of k in ascending order by one matrix instruction per slice:
// v_mfma_f32_16x16x32_bf16 (32 k), or v_mfma_scale_f32_16x16x128_f8f6f4 on
// 4-bit operands (128 k, one power-of-two scale per operand row and 32 k).
// k past the end of a ragged last slice is zero in both operands.  Nothing in
// that sequence depends on the tile shape, on M or on a row's place in the
// batch.
//
// Layout: the weight fragment is the instruction's first operand, so that lane
// (r = l % 16, g = l / 16) holds four consecutive output columns of row r.  The
// 32 columns of a fragment pair are dealt out so that register q of fragment f
// is column 8 g + 4 f + q: a lane owns eight consecutive columns and stores
// them with one 16-byte (bf16) or two (fp32) stores, without passing the
// output through LDS.
#pragma once

#include "bi_async.h"

namespace bi {

enum TileEpilogue { kEpiLinear = 0, kEpiGated = 1 };
enum TileGate { kGateSilu = 0, kGateGeluTanh = 1 };

struct TileArgs {
    const unsigned char* a;     // A: row operand: row m at a + m lda; column operand: k at a + k lda
    const unsigned char* b;
    int64_t lda, ldb;           // bytes
    const unsigned char* sa;    // 4-bit operands: scale bytes, one row of them per operand row
    const unsigned char* sb;
    int64_t ldsa, ldsb;         // bytes
    const float* bias;          // [N] or nullptr
    void* y;
    int64_t ldy;                // elements
    int y_bf16;
    uint16_t* h;                // gated: pre-activations [M, 2 I] or nullptr
    int64_t ldh;                // elements
    int gate;                   // TileGate
    int M, N;                   // outputs (gated: N = I)
    int64_t K;                  // k values
    int tiles_m, tiles_n;
};

// tanh form of gelu as a sigmoid: 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)).
constexpr float kGeluC2 = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// act(g) = g * gate_sigma(g).  exp overflows to +inf for very negative g,
// where the quotient is 0 as it should be.
__device__ __forceinline__ float gate_sigma(float g, int gate)
{
    const float z = gate == kGateSilu ? g : kGeluC2 * (g + kGeluB * g * g * g);
    return 1.0f / (1.0f + expf(-z));
}

// two fp32 -> packed bf16, round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 v;
    v[0] = (__bf16)lo;
    v[1] = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, v);
}

// Workgroup w runs on XCD w % 8.  Each XCD takes one contiguous eighth of the
// tiles in an order that walks groups of 8 tile rows column by column, so that
// the tiles an XCD works on at one time share rows of A and of B in its L2.
__device__ __forceinline__ int tile_of(int w, int tiles_m, int tiles_n, int& tn)
{
    const int total = tiles_m * tiles_n;
    const int x = w & 7, j = w >> 3;
    const int per = total >> 3, more = total & 7;       // XCD x owns per (+1) tiles
    const int t = x * per + min(x, more) + j;
    constexpr int kGroup = 8;
    const int group = t / (kGroup * tiles_n);
    const int m0 = group * kGroup;
    const int rows = min(kGroup, tiles_m - m0);
    const int in = t - m0 * tiles_n;
    tn = in / rows;
    return m0 + in % rows;
}

// One operand's place in a stage and how its lanes load and read it.
//   ROWS output rows per tile, KB slices per stage, FP4: 128 k per slice.
// Row operands: [slice][row][64 bytes], the row's four 16-byte chunks permuted
// by (row / 2) & 3 (free of bank conflicts for the 16-row fragment reads).
// Column operands: [slice][32 k][ROWS bf16], 32-byte units of a k row permuted
// by a key of the k row, so that the four k rows a transposing read touches
// fall on different banks.  PAIR: the columns of a fragment pair are dealt out
// as described above (the weight side).
template <int ROWS, int KB, bool COL, bool PAIR, bool FP4>
struct TileOperand {
    static_assert(!(COL && FP4), "4-bit operands are stored by rows");
    static constexpr int kSliceBytes = ROWS * 64;
    static constexpr int kBytes = KB * kSliceBytes;
    static constexpr int kLoads = kBytes / 1024;        // 1 KiB wave loads per stage
    static constexpr int kPitch = COL ? ROWS * 2 : 64;
    static constexpr int kUnits = ROWS / 16;            // column operands: 32-byte units per k row

    __device__ __forceinline__ static int col_key(int krow)
    {
        if constexpr (kUnits >= 8)
            return PAIR ? (krow & 3) << 1 : (krow & 3) | ((krow >> 3) & 1) << 2;
        else
            return PAIR ? ((krow >> 1) & 1) << 1 : ((krow >> 1) & 1) | ((krow >> 3) & 1) << 1;
    }

    // The tile row a weight-side LDS row holds: within each 32, fragment f,
    // row i is column 8 (i / 4) + 4 f + i % 4.
    __device__ __forceinline__ static int paired(int p)
    {
        return (p & ~31) + 8 * ((p >> 2) & 3) + 4 * ((p >> 4) & 1) + (p & 3);
    }

    // LDS address of fragment f (16 rows), slice j, for lane (r, g); column
    // operands: the first of two reads, the second 4 kPitch further.
    __device__ __forceinline__ static int frag_at(int f, int r, int g)
    {
        if constexpr (!COL) {
            return f * 1024 + r * 64 + ((g ^ ((r >> 1) & 3)) << 4);
        } else {
            const int krow = 8 * g + (r >> 2), c = r & 3;
            if constexpr (PAIR) {
                const int unit = (f & ~1) + (c >> 1);
                return krow * kPitch + ((unit ^ col_key(krow)) << 5) + ((c & 1) << 4) + ((f & 1) << 3);
            } else {
                return krow * kPitch + ((f ^ col_key(krow)) << 5) + (c << 3);
            }
        }
    }

    __device__ __forceinline__ static u32x4 read(const unsigned char* p)
    {
        if constexpr (!COL) {
            return *reinterpret_cast<const u32x4*>(p);
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 lo = __builtin_bit_cast(u32x2, lds_read_tr(p));
            const u32x2 hi = __builtin_bit_cast(u32x2, lds_read_tr(p + 4 * kPitch));
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
    }
};

// Zero what lies past the end of k: `valid` k values of this lane's eight
// (bf16) or 32 (4-bit) belong to the problem.
template <bool FP4>
__device__ __forceinline__ u32x4 mask_k(u32x4 v, int64_t valid)
{
    if constexpr (FP4) {
        return valid > 0 ? v : u32x4{0u, 0u, 0u, 0u};
    } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = valid >= 2 * i + 2 ? v[i] : valid == 2 * i + 1 ? (v[i] & 0xffffu) : 0u;
        return o;
    }
}

// BM x BN tile on WM x WN waves, KB slices per ring stage, R stages.  CA, CB:
// operand A / B stored by columns.
template <int BM, int BN, int WM, int WN, int KB, int R, bool CA, bool CB, bool FP4, int EPI>
__global__ __launch_bounds__(WM * WN * 64) void k_tile(TileArgs p)
{
    constexpr int NW = WM * WN;
    constexpr int FM = BM / (WM * 16), FN = BN / (WN * 16);
    using A = TileOperand<BM, KB, CA, false, FP4>;
    using B = TileOperand<BN, KB, CB, true, FP4>;
    constexpr int kSliceK = FP4 ? 128 : 32;
    constexpr int kScaleRows = (BM + BN + 63) / 64 * 64;           // A's, then B's; 64 rows per load
    constexpr int kScaleStage = FP4 ? kScaleRows * 4 * KB : 0;     // [slice][row][4 scale bytes]
    constexpr int kStage = A::kBytes + B::kBytes + kScaleStage;
    constexpr int LA = A::kLoads / NW, LB = B::kLoads / NW;
    constexpr int kScaleLoads = FP4 ? kScaleRows / 64 * KB : 0;    // fewer than waves: some load the same twice
    constexpr int LSC = FP4 ? (kScaleLoads + NW - 1) / NW : 0;
    constexpr int LS = LA + LB + LSC;                              // loads per wave and stage
    constexpr int U = KB < 2 ? 2 : KB;                             // slices per loop body
    static_assert(LA * NW == A::kLoads && LB * NW == B::kLoads, "loads split evenly over the waves");
    static_assert(FN % (EPI == kEpiGated ? 4 : 2) == 0, "fragment pairs");
    static_assert(R >= 3 && (R - 2) * LS < 64, "ring depth");
    static_assert(U % 2 == 0 && U % KB == 0, "whole stages per body");
    __shared__ __attribute__((aligned(1024))) unsigned char ring[R * kStage];

    const int lane = threadIdx.x & 63, w = (int)uniform(threadIdx.x >> 6);
    const int wm = w / WN, wn = w % WN;
    const int r = lane & 15, g = lane >> 4;
    int tn;
    const int tm = tile_of((int)blockIdx.x, p.tiles_m, p.tiles_n, tn);
    const int m0 = tm * BM;
    constexpr int kOutN = EPI == kEpiGated ? BN / 2 : BN;          // output columns per tile
    const int n0 = tn * kOutN;
    const int ns = (int)((p.K + kSliceK - 1) / kSliceK);           // slices
    const uint32_t lds0 = lds_byte(ring);

    // ---- loads.  Row operands: load t of a wave covers 16 tile rows of one
    // slice; lane i lands at row i / 4, chunk position i % 4 and fetches the
    // chunk that belongs there.  Rows past the end read the last row, chunks
    // past the end of k the last chunk: neither reaches a stored result.
    // Column operands: a load covers 1024 / pitch k rows of one slice.
    uint32_t voff[LA + LB];                                        // row operands: row offset
    int kch[LA + LB];                                              // row: chunk; column: k row in slice
#pragma unroll
    for (int t = 0; t < LA + LB; ++t) {
        const bool is_a = t < LA;
        const int load = is_a ? w * LA + t : w * LB + (t - LA);
        if (is_a ? CA : CB) {
            const int pitch = is_a ? A::kPitch : B::kPitch;
            const int cpr = pitch / 16;                            // chunks per k row
            const int per = 1024 / pitch;                          // k rows per load
            const int krow = (load * per) % 32 + lane / cpr;
            const int pos = lane % cpr;
            const int key = is_a ? A::col_key(krow) : B::col_key(krow);
            const int chunk = (((pos >> 1) ^ key) << 1) | (pos & 1);
            const int first = is_a ? m0 : n0, total = is_a ? p.M : p.N;
            voff[t] = (uint32_t)(min(first + chunk * 8, total - 8) - first) * 2u;
            kch[t] = krow;
        } else {
            const int rows = is_a ? BM : BN;
            const int row = (load * 16) % rows + (lane >> 2);
            kch[t] = (lane & 3) ^ ((row >> 1) & 3);
            if (is_a) {
                voff[t] = (uint32_t)((int64_t)(min(m0 + row, p.M - 1) - m0) * p.lda);
            } else {
                int q = B::paired(row);
                if constexpr (EPI == kEpiGated) {
                    // 64 LDS rows: 32 gate rows, then the 32 up rows of the same outputs
                    const int out = min(n0 + (q >> 6) * 32 + (q & 31), p.N - 1);
                    q = out - n0 + ((q >> 5) & 1) * p.N;
                } else {
                    q = min(n0 + q, p.N - 1) - n0;
                }
                voff[t] = (uint32_t)((int64_t)q * p.ldb);
            }
        }
    }
    const int kbytes = (int)(FP4 ? p.K / 2 : p.K * 2);             // row operands
    const unsigned char* abase = p.a + (CA ? (int64_t)m0 * 2 : (int64_t)m0 * p.lda);
    const unsigned char* bbase = p.b + (CB ? (int64_t)n0 * 2 : (int64_t)n0 * p.ldb);
    const unsigned char* srow[FP4 ? LSC : 1];                      // this lane's row of scales
    if constexpr (FP4) {
#pragma unroll
        for (int t = 0; t < LSC; ++t) {
            const int row = ((w * LSC + t) % (kScaleRows / 64)) * 64 + lane;
            srow[t] = row < BM ? p.sa + (int64_t)min(m0 + row, p.M - 1) * p.ldsa
                               : p.sb + (int64_t)min(n0 + B::paired(min(row - BM, BN - 1)), p.N - 1) * p.ldsb;
        }
    }

    auto issue_one = [&](int st, int t) __attribute__((always_inline)) {
        const uint32_t base = lds0 + (uint32_t)(st % R) * kStage;
        if (t < LA + LB) {
            const bool is_a = t < LA;
            const int load = is_a ? w * LA + t : w * LB + (t - LA);
            const uint32_t dst = uniform(base + (is_a ? 0 : A::kBytes) + load * 1024);
            if (is_a ? CA : CB) {
                const int pitch = is_a ? A::kPitch : B::kPitch;
                const int slice = st * KB + load / (32 * pitch / 1024);
                const int64_t ld = is_a ? p.lda : p.ldb;
                const int64_t k0 = (int64_t)min(slice, ns - 1) * 32;
                const int krow = (int)min((int64_t)kch[t], p.K - 1 - k0);
                async16(voff[t] + (uint32_t)krow * (uint32_t)ld, (is_a ? abase : bbase) + k0 * ld, dst);
            } else {
                const int slice = st * KB + load / ((is_a ? BM : BN) / 16);
                async16(voff[t] + (uint32_t)min(slice * 64 + kch[t] * 16, kbytes - 16), is_a ? abase : bbase, dst);
            }
        } else if constexpr (FP4) {
            const int load = (w * LSC + (t - LA - LB)) % kScaleLoads;
            const int slice = st * KB + load / (kScaleRows / 64);
            async4(srow[t - LA - LB] + min(slice, ns - 1) * 4, uniform(base + A::kBytes + B::kBytes + load * 256));
        }
    };
    auto issue = [&](int st) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < LS; ++t)
            issue_one(st, t);
    };

    // ---- fragments
    const unsigned char* arow[CA ? FM : 1];
    const unsigned char* brow[CB ? FN : 1];
    if constexpr (CA) {
#pragma unroll
        for (int f = 0; f < FM; ++f)
            arow[f] = ring + A::frag_at(wm * FM + f, r, g);
    } else {
        arow[0] = ring + A::frag_at(wm * FM, r, g);
    }
    if constexpr (CB) {
#pragma unroll
        for (int f = 0; f < FN; ++f)
            brow[f] = ring + A::kBytes + B::frag_at(wn * FN + f, r, g);
    } else {
        brow[0] = ring + A::kBytes + B::frag_at(wn * FN, r, g);
    }
    const unsigned char* sarow = ring + A::kBytes + B::kBytes + (wm * FM * 16 + r) * 4 + g;
    const unsigned char* sbrow = ring + A::kBytes + B::kBytes + (BM + wn * FN * 16 + r) * 4 + g;
    auto at = [&](int s) __attribute__((always_inline)) { return ((s / KB) % R) * kStage; };       // stage of slice s
    auto frag_a = [&](int s, int f) __attribute__((always_inline)) {
        return A::read((CA ? arow[CA ? f : 0] : arow[0] + f * 1024) + at(s) + (s % KB) * A::kSliceBytes);
    };
    auto frag_b = [&](int s, int f) __attribute__((always_inline)) {
        return B::read((CB ? brow[CB ? f : 0] : brow[0] + f * 1024) + at(s) + (s % KB) * B::kSliceBytes);
    };
    auto scale_a = [&](int s, int f) __attribute__((always_inline)) -> int { return sarow[at(s) + (s % KB) * kScaleRows * 4 + f * 64]; };
    auto scale_b = [&](int s, int f) __attribute__((always_inline)) -> int { return sbrow[at(s) + (s % KB) * kScaleRows * 4 + f * 64]; };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
            acc[fm][fn] = f32x4{0.f, 0.f, 0.f, 0.f};

    u32x4 xa[FM], xb[FM], wf[FN];
    int sxa[FP4 ? FM : 1], sxb[FP4 ? FM : 1], swf[FP4 ? FN : 1];
    auto mfma = [&](const u32x4& x, const u32x4& wv, int sx, int sw, f32x4& c) __attribute__((always_inline)) {
        if constexpr (FP4) {
            const i32x8 xv = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
            const i32x8 bv = {(int)wv[0], (int)wv[1], (int)wv[2], (int)wv[3], 0, 0, 0, 0};
            c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv, xv, c, 4, 4, 0, sw, 0, sx);
        } else {
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv), __builtin_bit_cast(bf16x8, x),
                                                        c, 0, 0, 0);
        }
    };

    // ---- prologue: R - 1 stages in flight, the first one landed
#pragma unroll
    for (int st = 0; st < R - 1; ++st)
        issue(st);
    async_wait<(R - 2) * LS>();
    wg_barrier();
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        xa[f] = frag_a(0, f);
        if constexpr (FP4)
            sxa[f] = scale_a(0, f);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        wf[f] = frag_b(0, f);
        if constexpr (FP4)
            swf[f] = scale_b(0, f);
    }

    // Slice s: where it is a stage's last, make the next stage visible (this
    // wave's loads of it waited for, then the barrier, which also tells that
    // every wave is done with the stage before this one, whose slot the loads
    // of this step refill); then the MFMAs of slice s with the reads of slice
    // s + 1's fragments between them, each weight fragment replaced in place
    // once its MFMAs have issued.  Past the last slice, loads and reads touch
    // re-read data that nothing uses.
    auto step = [&](auto tail, int s, int j, u32x4 (&xc)[FM], int (&sxc)[FP4 ? FM : 1], u32x4 (&xn)[FM],
                    int (&sxn)[FP4 ? FM : 1]) __attribute__((always_inline)) {
        const bool stage_end = j % KB == KB - 1;                   // compile-time after unrolling
        if (stage_end) {
            async_wait<(R - 3) * LS>();
            wg_barrier();
        }
        if constexpr (decltype(tail)::value) {
            // this lane's slot: k values s * kSliceK + slot g
            const int64_t valid = p.K - (int64_t)s * kSliceK - g * (kSliceK / 4);
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                xc[f] = mask_k<FP4>(xc[f], valid);
                if constexpr (FP4)
                    sxc[f] = valid > 0 ? sxc[f] : 127;
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                wf[f] = mask_k<FP4>(wf[f], valid);
                if constexpr (FP4)
                    swf[f] = valid > 0 ? swf[f] : 127;
            }
        }
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            xn[f] = frag_a(s + 1, f);
            if constexpr (FP4)
                sxn[f] = scale_a(s + 1, f);
        }
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
                mfma(xc[fm], wf[fn], FP4 ? sxc[FP4 ? fm : 0] : 0, FP4 ? swf[FP4 ? fn : 0] : 0, acc[fm][fn]);
            wf[fn] = frag_b(s + 1, fn);
            if constexpr (FP4)
                swf[fn] = scale_b(s + 1, fn);
            if (stage_end) {
#pragma unroll
                for (int t = fn * LS / FN; t < (fn + 1) * LS / FN; ++t)
                    issue_one(s / KB + R - 1, t);
            }
        }
    };
    auto body = [&](auto tail, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < U; j += 2) {
            step(tail, s + j, j, xa, sxa, xb, sxb);
            step(tail, s + j + 1, j + 1, xb, sxb, xa, sxa);
        }
    };
    const int whole = (int)(p.K / (kSliceK * U)) * U;               // slices of bodies without a ragged end
    for (int s = 0; s < whole; s += U)
        body(std::false_type{}, s);
    if (whole < ns)
        body(std::true_type{}, whole);
    // the loads still in flight land before the workgroup's LDS is given away
    async_wait<0>();

    // ---- epilogue: rows m, eight consecutive columns per fragment pair
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int m = m0 + (wm * FM + fm) * 16 + r;
        if constexpr (EPI == kEpiGated) {
#pragma unroll
            for (int q4 = 0; q4 < FN / 4; ++q4) {
                const int n = n0 + (wn * (FN / 4) + q4) * 32 + 8 * g;
                if (m < p.M && n < p.N) {
                    u32x4 yv, gv, uv;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int f = i >> 1, q = (i & 1) * 2;
                        const float g0 = acc[fm][q4 * 4 + f][q], g1 = acc[fm][q4 * 4 + f][q + 1];
                        const float u0 = acc[fm][q4 * 4 + 2 + f][q], u1 = acc[fm][q4 * 4 + 2 + f][q + 1];
                        yv[i] = pack_bf16(g0 * gate_sigma(g0, p.gate) * u0, g1 * gate_sigma(g1, p.gate) * u1);
                        gv[i] = pack_bf16(g0, g1);
                        uv[i] = pack_bf16(u0, u1);
                    }
                    *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.y) + (int64_t)m * p.ldy + n) = yv;
                    if (p.h) {
                        *reinterpret_cast<u32x4*>(p.h + (int64_t)m * p.ldh + n) = gv;
                        *reinterpret_cast<u32x4*>(p.h + (int64_t)m * p.ldh + p.N + n) = uv;
                    }
                }
            }
        } else {
#pragma unroll
            for (int q2 = 0; q2 < FN / 2; ++q2) {
                const int n = n0 + (wn * (FN / 2) + q2) * 32 + 8 * g;
                if (m < p.M && n < p.N) {
                    f32x4 lo = acc[fm][q2 * 2], hi = acc[fm][q2 * 2 + 1];
                    if (p.bias) {
                        lo += *reinterpret_cast<const f32x4*>(p.bias + n);
                        hi += *reinterpret_cast<const f32x4*>(p.bias + n + 4);
                    }
                    if (p.y_bf16) {
                        const u32x4 v = {pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(hi[0], hi[1]),
                                         pack_bf16(hi[2], hi[3])};
                        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.y) + (int64_t)m * p.ldy + n) = v;
                    } else {
                        float* y = reinterpret_cast<float*>(p.y) + (int64_t)m * p.ldy + n;
                        *reinterpret_cast<f32x4*>(y) = lo;
                        *reinterpret_cast<f32x4*>(y + 4) = hi;
                    }
                }
            }
        }
    }
}

}  // namespace bi
