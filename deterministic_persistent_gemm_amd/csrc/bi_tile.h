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
#include "bi_ffn.h"

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
    float* db;                  // column operand A: [M] sums of its columns over k, or nullptr
    int tiles_m, tiles_n;
};

// tanh form of gelu as a sigmoid: 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)).
constexpr float kGeluC2 = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 2^8 sigma(z(g)), which the callers scale back: act(g) = (g 2^-8) gate_sigma8(g).
// For z of -87.4 and below sigma is subnormal, where the hardware reciprocal gives
// zero, but act = g sigma still a normal number; scaled, it lasts to z = -92.8
// (sigma = 2^-134), below which act is zero: by then |act| < 2^-127.  g 2^-8
// keeps 16 bits of fp32's smallest normal g.  exp overflows to +inf for very
// negative z, where the reciprocal is 0 as it should be.
// The hardware exponential and reciprocal (one ulp each; the argument's roundings
// times its magnitude of at most 93 on top: below 2^-14 relative, far under the
// bf16 rounding of what is stored) in place of expf and a full division, which made
// the epilogue of a 256 x 256 tile 9 us long.
constexpr float kSigmaScale = 0.00390625f;          // 2^-8
__device__ __forceinline__ float gate_sigma8(float g, int gate)
{
    const float z = gate == kGateSilu ? g : kGeluC2 * (g + kGeluB * g * g * g);
    return __builtin_amdgcn_rcpf(kSigmaScale + __builtin_amdgcn_exp2f(__builtin_fmaf(z, -1.4426950408889634f, -8.0f)));
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

// How the weight side's output columns are dealt to fragment rows.  kPairs:
// within each 32, register q of fragment f of lane group g is column
// 8 g + 4 f + q (eight consecutive columns per lane); kSingle: one fragment,
// columns in order.  Gated: kGated4 holds 32 gate rows, dealt as pairs, then the
// 32 up rows of the same outputs; kGated2 16 and 16, kGated1 8 and 8, in order.
enum TileDeal { kPairs, kSingle, kGated4, kGated2, kGated1 };

template <int FN, int EPI> constexpr TileDeal tile_deal()
{
    if (EPI == kEpiGated)
        return FN % 4 == 0 ? kGated4 : FN == 2 ? kGated2 : kGated1;
    return FN % 2 == 0 ? kPairs : kSingle;
}

// The tile output a weight-side LDS row belongs to, and whether it is the up row.
template <TileDeal D> __device__ __forceinline__ int deal_out(int p)
{
    const int pair = 8 * ((p >> 2) & 3) + 4 * ((p >> 4) & 1) + (p & 3);
    return D == kPairs ? (p & ~31) + pair : D == kSingle ? p : D == kGated4 ? (p >> 6) * 32 + pair
         : D == kGated2 ? (p >> 5) * 16 + (p & 15) : (p >> 4) * 8 + (p & 7);
}
template <TileDeal D> __device__ __forceinline__ int deal_up(int p)
{
    return D == kGated4 ? (p >> 5) & 1 : D == kGated2 ? (p >> 4) & 1 : D == kGated1 ? (p >> 3) & 1 : 0;
}

// One operand's place in a stage and how its lanes load and read it.
//   ROWS output rows per tile, KB slices per stage.
// Row operands: WIDE, slices in pairs, so that a load asks for whole 128-byte
// lines: [pair][row][128 bytes], the row's eight 16-byte
// chunks permuted by (row / 2) & 7; else [row][64 bytes], four chunks permuted by
// (row / 2) & 3 (both free of bank conflicts for the 16-row fragment reads).
// Column operands: [slice][32 k][ROWS bf16], 32-byte units of a k row permuted
// by a key of the k row where four k rows span more than the 256 bytes of all
// banks, so that the four k rows a transposing read touches fall on different
// banks.  PAIR: the weight side's columns are dealt as kPairs.
template <int ROWS, int KB, bool COL, bool PAIR, bool WIDE>
struct TileOperand {
    static constexpr int kSliceBytes = ROWS * 64;
    static constexpr int kBytes = KB * kSliceBytes;
    static constexpr int kLoads = kBytes / 1024;        // 1 KiB wave loads per stage
    static constexpr int kSpan = WIDE ? 2 : 1;          // row operands: slices side by side in a row
    static constexpr int kPitch = COL ? ROWS * 2 : 64 * kSpan;
    static constexpr int kChunks = kPitch / 16;
    static constexpr int kLoadRows = 1024 / kPitch;     // rows (column operands: k rows) per load
    static constexpr int kUnits = ROWS / 16;            // column operands: 32-byte units per k row
    static_assert(ROWS % 16 == 0 && (!COL || kUnits == 1 || kUnits == 2 || kUnits == 4 || kUnits % 8 == 0), "tile rows");

    __device__ __forceinline__ static int col_key(int krow)
    {
        if constexpr (kUnits >= 8)
            return PAIR ? (krow & 3) << 1 : (krow & 3) | ((krow >> 3) & 1) << 2;
        else if constexpr (kUnits == 4)
            return PAIR ? ((krow >> 1) & 1) << 1 : ((krow >> 1) & 1) | ((krow >> 3) & 1) << 1;
        else
            return 0;
    }

    __device__ __forceinline__ static int row_key(int row) { return (row >> 1) & (kChunks - 1); }

    // LDS address of fragment f (16 rows), slice 0, for lane (r, g); column
    // operands: the first of two reads, the second 4 kPitch further.
    __device__ __forceinline__ static int frag_at(int f, int r, int g)
    {
        if constexpr (!COL) {
            return (f * 16 + r) * kPitch + ((g ^ row_key(r)) << 4);
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

    // The same in slice j (the second slice of a pair lies four chunks further,
    // under the same permutation).
    __device__ __forceinline__ static int in_slice(int at, int j)
    {
        if constexpr (COL)
            return at + j * kSliceBytes;
        else
            return (j % kSpan == 0 ? at : at ^ 64) + j / kSpan * kSpan * kSliceBytes;
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

// Groups of four slices' scales a ring must hold where stages of kb < 4 slices each
// bring a part of the group after theirs, r stages deep: at the end of stage c the
// loads of stage c + r - 1 overwrite the group that lies a ring behind theirs, while
// the scales of stage c's last slice may still be on their way to registers (the
// barrier there waits for loads, not for LDS reads).
constexpr int scale_ring_groups(int kb, int r)
{
    int most = 0;
    for (int c = 0; c < 4; ++c) {                       // parts repeat every 4 / kb stages
        const int newest = (c + r - 1) / (4 / kb) + 1, oldest = (c * kb + kb - 1) / 4;
        most = newest - oldest + 1 > most ? newest - oldest + 1 : most;
    }
    return most;
}

// A tile: BM x BN outputs (gated: BN weight rows, BN / 2 outputs) on WM x WN
// computing waves, R ring stages of KB slices.  CA, CB: operand A / B stored by
// columns.
template <int BM_, int BN_, int WM_, int WN_, int KB_, int R_, bool CA_, bool CB_, bool FP4_, int EPI_>
struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KB = KB_, R = R_, EPI = EPI_;
    static constexpr bool CA = CA_, CB = CB_, FP4 = FP4_;
    static constexpr int NW = WM * WN;
    static constexpr bool kSums = CA && BM_ < 256;
    static constexpr int FM = BM / (WM * 16), FN = BN / (WN * 16);
    static constexpr TileDeal kDeal = tile_deal<FN, EPI>();
    // 128 bytes of a row at a time: 17 to 32 percent off a 128 x 128 bf16 tile's
    // time, 9 off a 256 x 256 one's.  Short 4-bit streams (16 rows) take 5 percent
    // longer with it and keep 64.
    static constexpr bool kWide = KB % 2 == 0 && !(FP4 && BM < 64);
    using A = TileOperand<BM, KB, CA, false, kWide>;
    using B = TileOperand<BN, KB, CB, kDeal == kPairs || kDeal == kGated4, kWide>;
    static constexpr int kOutN = EPI == kEpiGated ? BN / 2 : BN;       // output columns per tile
    static constexpr int kSliceK = FP4 ? 128 : 32;
    static constexpr int kStage = A::kBytes + B::kBytes;
    // Scales travel in groups of four slices, [row][16 bytes], A's rows then B's:
    // a 4-byte load then takes 16 bytes of each of 16 rows (a load of one slice's
    // four bytes of 64 rows touches 64 cache lines, which cost the 256 x 256
    // tile 30 percent of its time).  A stage of a whole number of groups brings
    // its own; smaller stages each bring a part of the group after theirs, in a
    // ring of as many groups as are in use at a time: four in the 64 x 64 tile,
    // three in the larger ones.
    static constexpr int kGroup = (BM + BN) * 16;
    static constexpr bool kGroupInStage = KB % 4 == 0;
    static constexpr int kGroups = !FP4 ? 0 : kGroupInStage ? R * (KB / 4) : scale_ring_groups(KB < 4 ? KB : 4, R);
    static constexpr int kScaleAt = R * kStage;
    static constexpr int kScaleLoads = !FP4 ? 0 : (BM + BN) / 16 * KB / 4;     // per stage, 16 rows each
    static constexpr int kRing = kScaleAt + kGroups * kGroup;
    static_assert(!FP4 || kGroupInStage || ((BM + BN) / 16 * KB) % 4 == 0, "equal parts of a group per stage");
    static_assert(FM * WM * 16 == BM && FN * WN * 16 == BN, "whole fragments per wave");
    static_assert(!(FP4 && (CA || CB)), "4-bit operands are stored by rows");
    static_assert(EPI != kEpiGated || !CB, "the gated weight is stored by rows");
};

// Shape S (its TileCfg S::C and loading waves S::NL) at index i of its product's list.
template <typename S>
TileInfo tile_info(int i)
{
    using C = typename S::C;
    return {i, S::NL > 0 ? 0 : C::R == 2 ? 2 : 1, C::BM, C::kOutN, C::kSliceK, C::KB, C::R, C::kGroups};
}

// The loads of a stage, spread over NL loading waves (this one is `wl`).
// Row operands: a load covers 16 tile rows of one slice, or 8 rows of a pair;
// the lanes land on a row's chunk positions in turn, each fetching the chunk
// that belongs there.  Rows past the end read the last row, chunks past the end
// of k the last chunk: neither reaches a stored result.  Column operands: a load
// covers 1024 / pitch k rows of one slice, columns past the end read the last
// eight.  Each load is a scalar base and 32 bits of byte offset per lane.
template <typename C, int NL>
struct TileLoads {
    using A = typename C::A;
    using B = typename C::B;
    static constexpr int LA = A::kLoads / NL, LB = B::kLoads / NL;
    static constexpr int LSC = (C::kScaleLoads + NL - 1) / NL;         // past the last: the same loads again
    static constexpr int LS = LA + LB + LSC;                           // loads per wave and stage
    static constexpr int kParts = C::FP4 && !C::kGroupInStage ? 4 / C::KB : 1;  // stages a scale group is spread over
    static constexpr int PA = C::BM / 16 / kParts, PB = C::BN / 16 / kParts;    // loads of a part, by operand
    static_assert(kParts == 1 || (PA * kParts * 16 == C::BM && PB * kParts * 16 == C::BN && PB % 2 == 0), "equal parts");
    static_assert(LA * NL == A::kLoads && LB * NL == B::kLoads, "loads split evenly over the waves");

    uint32_t voff[LA + LB];                                            // this lane's bytes from the slice's first
    int kch[LA + LB];                                                  // row operands: chunk; column: k row in the slice
    // scales, per load: the operand's first row of the tile, its pitch, the lane's
    // row in part 0, rows to the operand's end and per part, the place in a group
    const unsigned char* sbase[LSC > 0 ? LSC : 1];
    uint32_t sld[LSC > 0 ? LSC : 1];
    int srow[LSC > 0 ? LSC : 1], slast[LSC > 0 ? LSC : 1], sstep[LSC > 0 ? LSC : 1], sgroup[LSC > 0 ? LSC : 1];
    uint32_t sdst[LSC > 0 ? LSC : 1];
    const unsigned char *abase, *bbase;
    int64_t lda, ldb, K;
    int ns, kbytes, wl, lane;
    uint32_t lds0;

    __device__ __forceinline__ void init(const TileArgs& p, unsigned char* ring, int wl_, int lane_, int m0, int n0)
    {
        wl = wl_;
        lane = lane_;
        lds0 = lds_byte(ring);
        K = p.K;
        ns = (int)((p.K + C::kSliceK - 1) / C::kSliceK);
        kbytes = (int)(C::FP4 ? p.K / 2 : p.K * 2);                    // row operands
        lda = p.lda;
        ldb = p.ldb;
        abase = p.a + (C::CA ? (int64_t)m0 * 2 : (int64_t)m0 * p.lda);
        bbase = p.b + (C::CB ? (int64_t)n0 * 2 : (int64_t)n0 * p.ldb);
#pragma unroll
        for (int t = 0; t < LA + LB; ++t) {
            const bool is_a = t < LA;
            const int load = is_a ? wl * LA + t : wl * LB + (t - LA);
            if (is_a ? C::CA : C::CB) {
                const int pitch = is_a ? A::kPitch : B::kPitch;
                const int cpr = pitch / 16;                            // chunks per k row
                const int per = 1024 / pitch;                          // k rows per load
                const int krow = (load * per) % 32 + lane / cpr;
                const int pos = lane % cpr;
                const int key = is_a ? A::col_key(krow) : B::col_key(krow);
                const int chunk = (((pos >> 1) ^ key) << 1) | (pos & 1);
                const int first = is_a ? m0 : n0, total = is_a ? p.M : p.N;
                voff[t] = (uint32_t)(min(first + chunk * 8, total - 8) - first) * 2u + (uint32_t)krow * (uint32_t)(is_a ? p.lda : p.ldb);
                kch[t] = krow;
            } else {
                const int chunks = is_a ? A::kChunks : B::kChunks;
                const int row = (load * (is_a ? A::kLoadRows : B::kLoadRows)) % (is_a ? C::BM : C::BN) + lane / chunks;
                kch[t] = (lane % chunks) ^ (is_a ? A::row_key(row) : B::row_key(row));
                if (is_a) {
                    voff[t] = (uint32_t)((int64_t)(min(m0 + row, p.M - 1) - m0) * p.lda) + kch[t] * 16;
                } else {
                    const int out = min(n0 + deal_out<C::kDeal>(row), p.N - 1);
                    voff[t] = (uint32_t)((int64_t)(out - n0 + deal_up<C::kDeal>(row) * p.N) * p.ldb) + kch[t] * 16;
                }
            }
        }
        if constexpr (C::FP4) {
#pragma unroll
            for (int t = 0; t < LSC; ++t) {
                const int load = (wl * LSC + t) % C::kScaleLoads;      // past the last: the same again
                const int j = load % (PA + PB);
                const bool is_a = j < PA;
                const int row = (is_a ? j : j - PA) * 16 + (lane >> 2);
                sbase[t] = is_a ? p.sa + (int64_t)m0 * p.ldsa : p.sb + (int64_t)n0 * p.ldsb;
                sld[t] = (uint32_t)(is_a ? p.ldsa : p.ldsb);
                srow[t] = is_a ? row : deal_out<C::kDeal>(row);
                slast[t] = (is_a ? p.M - m0 : p.N - n0) - 1;
                sstep[t] = (is_a ? PA : PB) * 16;
                sgroup[t] = load / (PA + PB);
                sdst[t] = lds0 + C::kScaleAt + (is_a ? j : C::BM / 16 + j - PA) * 256;
            }
        }
    }

    // Load t of the scales of group `grp` (the first of a stage's groups), part
    // `part` where a group is spread over stages.
    __device__ __forceinline__ void issue_scale(int grp, int part, int t) const
    {
        const int group = grp + sgroup[t];
        const uint32_t off = (uint32_t)min(srow[t] + part * sstep[t], slast[t]) * sld[t];
        async4(off + (uint32_t)min(group * 4 + (lane & 3), ns - 1) * 4u, sbase[t],
               uniform(sdst[t] + (uint32_t)(group % (C::kGroups > 0 ? C::kGroups : 1)) * C::kGroup + part * sstep[t] * 16));
    }

    // The first scale group, where stages bring the group after theirs.
    __device__ __forceinline__ void issue_first_scales() const
    {
        if constexpr (C::FP4 && !C::kGroupInStage) {
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
                for (int t = 0; t < LSC; ++t)
                    issue_scale(0, part, t);
        }
    }

    // Load t of stage st.  WHOLE: every slice of the stage lies inside k, so
    // that only the scalar base moves; otherwise k is clamped.
    template <bool WHOLE>
    __device__ __forceinline__ void issue_one(int st, int t) const
    {
        const uint32_t base = lds0 + (uint32_t)(st % C::R) * C::kStage;
        if (t < LA + LB) {
            const bool is_a = t < LA;
            const int load = is_a ? wl * LA + t : wl * LB + (t - LA);
            const uint32_t dst = uniform(base + (is_a ? 0 : A::kBytes) + load * 1024);
            const unsigned char* from = is_a ? abase : bbase;
            if (is_a ? C::CA : C::CB) {
                const int pitch = is_a ? A::kPitch : B::kPitch;
                const int slice = st * C::KB + load / (32 * pitch / 1024);
                const int64_t ld = is_a ? lda : ldb;
                if constexpr (WHOLE) {
                    async16(voff[t], from + (int64_t)slice * 32 * ld, dst);
                } else {
                    const int64_t k0 = (int64_t)min(slice, ns - 1) * 32;
                    const int past = max(kch[t] - (int)min((int64_t)31, K - 1 - k0), 0);
                    async16(voff[t] - (uint32_t)past * (uint32_t)ld, from + k0 * ld, dst);
                }
            } else {
                const int rows = is_a ? C::BM / A::kLoadRows : C::BN / B::kLoadRows;
                const int slice = st * C::KB + load / rows * A::kSpan;
                if constexpr (WHOLE)
                    async16(voff[t], from + slice * 64, dst);
                else
                    async16(voff[t] + (uint32_t)(min(slice * 64, kbytes - 16 - kch[t] * 16)), from, dst);
            }
        } else if constexpr (C::FP4) {
            if constexpr (C::kGroupInStage)
                issue_scale(st * (C::KB / 4), 0, t - LA - LB);
            else
                issue_scale(st / kParts + 1, st % kParts, t - LA - LB);
        }
    }

    __device__ __forceinline__ void issue(int st) const
    {
        if ((int64_t)(st + 1) * C::KB * C::kSliceK <= K) {
#pragma unroll
            for (int t = 0; t < LS; ++t)
                issue_one<true>(st, t);
        } else {
#pragma unroll
            for (int t = 0; t < LS; ++t)
                issue_one<false>(st, t);
        }
    }
};

// A computing wave's fragment and scale addresses (byte offsets in the ring).
template <typename C>
struct TileFrags {
    const unsigned char* ring;
    int arow[C::CA ? C::FM : 1];
    int brow[C::CB ? C::FN : 1];
    int sarow, sbrow;

    __device__ __forceinline__ void init(const unsigned char* ring_, int wm, int wn, int r, int g)
    {
        ring = ring_;
#pragma unroll
        for (int f = 0; f < (C::CA ? C::FM : 1); ++f)
            arow[f] = C::A::frag_at(wm * C::FM + f, r, g);
#pragma unroll
        for (int f = 0; f < (C::CB ? C::FN : 1); ++f)
            brow[f] = C::A::kBytes + C::B::frag_at(wn * C::FN + f, r, g);
        sarow = C::kScaleAt + (wm * C::FM * 16 + r) * 16 + g;
        sbrow = C::kScaleAt + (C::BM + wn * C::FN * 16 + r) * 16 + g;
    }
    // fragment f of slice j of the stage in slot `at` (a byte offset)
    __device__ __forceinline__ u32x4 a(int at, int j, int f) const
    {
        return C::A::read(ring + C::A::in_slice(arow[C::CA ? f : 0], j) + at + (C::CA ? 0 : f * 16 * C::A::kPitch));
    }
    __device__ __forceinline__ u32x4 b(int at, int j, int f) const
    {
        return C::B::read(ring + C::B::in_slice(brow[C::CB ? f : 0], j) + at + (C::CB ? 0 : f * 16 * C::B::kPitch));
    }
    // scale byte of fragment f in slice s
    __device__ __forceinline__ int sa(int s, int f) const { return C::FP4 ? ring[sarow + group_at(s) + f * 256] : 0; }
    __device__ __forceinline__ int sb(int s, int f) const { return C::FP4 ? ring[sbrow + group_at(s) + f * 256] : 0; }
    __device__ __forceinline__ static int group_at(int s)
    {
        return (s / 4) % (C::kGroups > 0 ? C::kGroups : 1) * C::kGroup + s % 4 * 4;
    }
};

template <bool FP4>
__device__ __forceinline__ void tile_mfma(const u32x4& x, const u32x4& w, int sx, int sw, f32x4& c)
{
    if constexpr (FP4) {
        const i32x8 xv = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
        const i32x8 wv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, c, 4, 4, 0, sw, 0, sx);
    } else {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
    }
}

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

// Sums of A's columns, taken from the fragments on their way to the matrix
// instructions by the first wave column of the first tile column.  Each lane adds
// its k values in ascending order, two per instruction (a bf16 dot product with
// ones, fp32 accumulation; shifts and adds cost 4096 x 1024 x 1024 31.4 -> 34.8
// us); the four lanes of a column are added at the end.  Not in the largest
// tiles: their waves take turns at the barriers, and all wait for the one that
// adds.
template <typename C>
struct TileSums {
    float v[C::kSums ? C::FM : 1] = {};
    bool on;

    __device__ __forceinline__ TileSums(const TileArgs& p, int n0, int wn) : on(C::kSums && p.db && n0 == 0 && wn == 0) {}
    __device__ __forceinline__ void add(const u32x4 (&x)[C::FM])
    {
        if constexpr (C::kSums) {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            const bf16x2 ones = __builtin_bit_cast(bf16x2, 0x3f803f80u);
            if (on) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int f = 0; f < C::FM; ++f) {
                        const uint32_t two = x[f][j];
                        v[f] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), ones, v[f], false);
                    }
            }
        }
    }
    __device__ __forceinline__ void store(const TileArgs& p, int m0, int wm, int r, int g)
    {
        if constexpr (C::kSums) {
            if (on) {
#pragma unroll
                for (int fm = 0; fm < C::FM; ++fm) {
                    float t = v[fm];
                    t += __shfl_xor(t, 16);
                    t += __shfl_xor(t, 32);
                    const int m = m0 + (wm * C::FM + fm) * 16 + r;
                    if (g == 0 && m < p.M)
                        p.db[m] = t;
                }
            }
        }
    }
};

// Stores a wave's outputs: row r of fragment fm, columns as dealt.
template <typename C>
__device__ __forceinline__ void tile_store(const TileArgs& p, const f32x4 (&acc)[C::FM][C::FN], int m0, int n0, int wm, int wn,
                                           int r, int g)
{
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    auto gated = [&](float gv, float uv) __attribute__((always_inline)) { return gv * kSigmaScale * gate_sigma8(gv, p.gate) * uv; };
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
        const int m = m0 + (wm * C::FM + fm) * 16 + r;
        if constexpr (C::kDeal == kGated4) {
#pragma unroll
            for (int q4 = 0; q4 < C::FN / 4; ++q4) {
                const int n = n0 + (wn * (C::FN / 4) + q4) * 32 + 8 * g;
                if (m < p.M && n < p.N) {
                    u32x4 yv, gv, uv;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int f = i >> 1, q = (i & 1) * 2;
                        const float g0 = acc[fm][q4 * 4 + f][q], g1 = acc[fm][q4 * 4 + f][q + 1];
                        const float u0 = acc[fm][q4 * 4 + 2 + f][q], u1 = acc[fm][q4 * 4 + 2 + f][q + 1];
                        yv[i] = pack_bf16(gated(g0, u0), gated(g1, u1));
                        gv[i] = pack_bf16(g0, g1);
                        uv[i] = pack_bf16(u0, u1);
                    }
                    // through the caches, also in large tiles: past them the call alone is up to 3
                    // percent faster, but the down projection that reads y next pays more (both
                    // calls, past / through: M 1000, H 1024, I 2048 33.4 / 29.4 us, M 1000, H 4096,
                    // I 6144 211 / 197, M 4096, H 4096, I 12288 917 / 906)
                    *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.y) + (int64_t)m * p.ldy + n) = yv;
                    if (p.h) {
                        *reinterpret_cast<u32x4*>(p.h + (int64_t)m * p.ldh + n) = gv;
                        *reinterpret_cast<u32x4*>(p.h + (int64_t)m * p.ldh + p.N + n) = uv;
                    }
                }
            }
        } else if constexpr (C::kDeal == kGated2 || C::kDeal == kGated1) {
            // kGated2: gate and up columns 4 g .. 4 g + 3 in the lane's two fragments.
            // kGated1: lane groups 0, 1 hold gate columns 4 g .., groups 2, 3 the
            // up columns of groups 0, 1, which the lanes 32 apart exchange.
            const f32x4 gv = acc[fm][0];
            f32x4 uv = acc[fm][C::FN - 1];
            int n = n0 + wn * 16 + 4 * g;
            bool owner = true, second = false;
            if constexpr (C::kDeal == kGated1) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    uv[q] = __shfl_xor(gv[q], 32);
                n = n0 + wn * 8 + 4 * (g & 1);
                owner = g < 2;
                second = g >= 2;
            }
            if (m < p.M && n < p.N) {
                const u32x2 hv = {pack_bf16(gv[0], gv[1]), pack_bf16(gv[2], gv[3])};
                if (owner) {
                    const u32x2 yv = {pack_bf16(gated(gv[0], uv[0]), gated(gv[1], uv[1])),
                                      pack_bf16(gated(gv[2], uv[2]), gated(gv[3], uv[3]))};
                    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p.y) + (int64_t)m * p.ldy + n) = yv;
                }
                if (p.h) {
                    *reinterpret_cast<u32x2*>(p.h + (int64_t)m * p.ldh + (second ? p.N : 0) + n) = hv;
                    if constexpr (C::kDeal == kGated2)
                        *reinterpret_cast<u32x2*>(p.h + (int64_t)m * p.ldh + p.N + n) =
                            u32x2{pack_bf16(uv[0], uv[1]), pack_bf16(uv[2], uv[3])};
                }
            }
        } else {
            // kPairs: eight columns from two fragments; kSingle: four from one
            constexpr int PF = C::kDeal == kPairs ? 2 : 1;
#pragma unroll
            for (int q2 = 0; q2 < C::FN / PF; ++q2) {
                const int n = n0 + (wn * (C::FN / PF) + q2) * 16 * PF + 4 * PF * g;
                if (m < p.M && n < p.N) {
                    f32x4 v[PF];
#pragma unroll
                    for (int f = 0; f < PF; ++f) {
                        v[f] = acc[fm][q2 * PF + f];
                        if (p.bias)
                            v[f] += *reinterpret_cast<const f32x4*>(p.bias + n + 4 * f);
                    }
                    if (p.y_bf16) {
                        uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + (int64_t)m * p.ldy + n;
                        const u32x2 lo = {pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3])};
                        if constexpr (PF == 2)
                            *reinterpret_cast<u32x4*>(y) =
                                u32x4{lo[0], lo[1], pack_bf16(v[PF - 1][0], v[PF - 1][1]), pack_bf16(v[PF - 1][2], v[PF - 1][3])};
                        else
                            *reinterpret_cast<u32x2*>(y) = lo;
                    } else {
                        float* y = reinterpret_cast<float*>(p.y) + (int64_t)m * p.ldy + n;
#pragma unroll
                        for (int f = 0; f < PF; ++f)
                            *reinterpret_cast<f32x4*>(y + 4 * f) = v[f];
                    }
                }
            }
        }
    }
}

// Middle tiles (64 x 64 to 128 x 128): every wave loads and computes.  A wave
// holds the fragments of two slices: while the MFMAs of slice s issue, the fragments of slice s + 1
// are read -- the A fragments first, then one B fragment after each group of
// MFMAs that used slice s's fragment at that position, which is then free --
// and the loads of a later stage are issued between the groups.  128 x 128 runs
// at 0.96 to 1.0 PFLOP/s in bf16 (4096 x 12288 x 4096), bound by the LDS bytes
// per MFMA (8 KiB of fragments for every 8 MFMAs of a wave); it is taken where
// larger tiles would leave compute units idle.
template <typename C>
__device__ __forceinline__ void tile_body(const TileArgs& p, unsigned char* ring, int block)
{
    constexpr int FM = C::FM, FN = C::FN, KB = C::KB, R = C::R;
    constexpr bool FP4 = C::FP4;
    constexpr int kSliceK = C::kSliceK;
    using Loads = TileLoads<C, C::NW>;
    constexpr int LS = Loads::LS;
    constexpr int U = KB < 2 ? 2 : KB;                             // slices per loop body
    static_assert(R >= 3 && (R - 2) * LS < 64, "ring depth");
    static_assert(U % 2 == 0 && U % KB == 0, "whole stages per body");

    const int lane = threadIdx.x & 63, w = (int)uniform(threadIdx.x >> 6);
    const int wm = w / C::WN, wn = w % C::WN;
    const int r = lane & 15, g = lane >> 4;
    int tn;
    const int tm = tile_of(block, p.tiles_m, p.tiles_n, tn);
    const int m0 = tm * C::BM, n0 = tn * C::kOutN;
    const int ns = (int)((p.K + kSliceK - 1) / kSliceK);           // slices
    Loads loads;
    loads.init(p, ring, w, lane, m0, n0);
    TileFrags<C> frags;
    frags.init(ring, wm, wn, r, g);
    auto at = [&](int s) __attribute__((always_inline)) { return ((s / KB) % R) * C::kStage; };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
            acc[fm][fn] = f32x4{0.f, 0.f, 0.f, 0.f};
    TileSums<C> sums(p, n0, wn);
    u32x4 xa[FM], xb[FM], wf[FN];
    int sxa[FM], sxb[FM], swf[FN];

    // R - 1 stages in flight, the first one landed
    loads.issue_first_scales();
#pragma unroll
    for (int st = 0; st < R - 1; ++st)
        loads.issue(st);
    async_wait<(R - 2) * LS>();
    wg_barrier();
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        xa[f] = frags.a(0, 0, f);
        sxa[f] = frags.sa(0, f);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        wf[f] = frags.b(0, 0, f);
        swf[f] = frags.sb(0, f);
    }

    // Slice s: where it is a stage's last, make the next stage visible (this
    // wave's loads of it waited for, then the barrier, which also tells that
    // every wave is done with the stage before this one, whose slot the loads
    // of this step refill); then the MFMAs of slice s with the reads of slice
    // s + 1's fragments between them.  Past the last slice, loads and reads
    // touch re-read data that nothing uses.
    auto step = [&](auto whole_loads, auto tail, int s, int j, u32x4 (&xc)[FM], int (&sxc)[FM], u32x4 (&xn)[FM], int (&sxn)[FM])
                    __attribute__((always_inline)) {
        const bool stage_end = j % KB == KB - 1;                   // compile-time after unrolling
        if constexpr (decltype(tail)::value) {
            // this lane's slot: k values from s * kSliceK + g * kSliceK / 4 on
            const int64_t valid = p.K - (int64_t)s * kSliceK - g * (kSliceK / 4);
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                xc[f] = mask_k<FP4>(xc[f], valid);
                sxc[f] = valid > 0 ? sxc[f] : 127;
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                wf[f] = mask_k<FP4>(wf[f], valid);
                swf[f] = valid > 0 ? swf[f] : 127;
            }
        }
        if (stage_end) {
            // no MFMA of the slices before may sink past the barrier: having
            // issued, they are the proof that their fragments have been read.  This
            // slice's fragments and scales may still be on their way: the loads
            // below refill the code slot of the stage before, and a scale group
            // that scale_ring_groups keeps clear of this slice's
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (C::kSums) {
                // here, where nothing may be scheduled across anyway: the slice
                // before, still in the registers the next reads will fill, and this one
                static_assert(KB == 2, "two slices per stage");
                sums.add(xn);
                sums.add(xc);
            }
            async_wait<(R - 3) * LS>();
            wg_barrier();
        }
        const int nat = at(s + 1), nj = (j + 1) % KB;
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            xn[f] = frags.a(nat, nj, f);
            sxn[f] = frags.sa(s + 1, f);
        }
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
#pragma unroll
            for (int fm = 0; fm < FM; ++fm)
                tile_mfma<FP4>(xc[fm], wf[fn], sxc[fm], swf[fn], acc[fm][fn]);
            wf[fn] = frags.b(nat, nj, fn);
            swf[fn] = frags.sb(s + 1, fn);
            if (stage_end) {
#pragma unroll
                for (int t = fn * LS / FN; t < (fn + 1) * LS / FN; ++t)
                    loads.template issue_one<decltype(whole_loads)::value>(s / KB + R - 1, t);
            }
        }
    };
    auto body = [&](auto whole_loads, auto tail, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < U; j += 2) {
            step(whole_loads, tail, s + j, j, xa, sxa, xb, sxb);
            step(whole_loads, tail, s + j + 1, j + 1, xb, sxb, xa, sxa);
        }
    };
    const int inside = (int)(p.K / kSliceK);                        // slices without a ragged end
    const int whole = inside / U * U;                               // of bodies of such slices
    const int ahead = (inside / KB - (R - 1)) * KB;                 // bodies up to here load only such slices
    int s = 0;
    for (; s + U <= ahead; s += U)
        body(std::true_type{}, std::false_type{}, s);
    for (; s < whole; s += U)
        body(std::false_type{}, std::false_type{}, s);
    if (whole < ns)
        body(std::false_type{}, std::true_type{}, whole);
    // the loads still in flight land before the workgroup's LDS is given away
    async_wait<0>();
    sums.store(p, m0, wm, r, g);
    tile_store<C>(p, acc, m0, n0, wm, wn, r, g);
}

// The largest tile: two groups of four waves, one wave of each per SIMD, take
// turns.  While one group's MFMAs of a slice run back to back, the other reads
// its fragments of its next slice from LDS; then they swap, one barrier per
// turn.  The matrix unit always has one wave that needs nothing but registers.
//
// Stages of two slices in a ring of two.  Turns of stage S (group 0 computes on
// odd turns, group 1 one turn later):
//   4S      group 0 reads slice 2S         group 1 computes 2S - 1
//   4S + 1  group 0 computes 2S            group 1 reads 2S
//   4S + 2  group 0 reads 2S + 1           group 1 computes 2S
//   4S + 3  group 0 computes 2S + 1        group 1 reads 2S + 1
// The slot of stage S + 1 had its last reader in turn 4S - 1, so its loads are
// issued in turns 4S and 4S + 1 and waited for at the end of turn 4S + 3.
//
// Measured on the gated layer at M = 4096, H = 4096, I = 4096 (two rounds of 256
// tiles): 195 us, 1.41 PFLOP/s, where every wave loading and computing at once
// (as in the middle tiles) took 222.  Timing copies with parts removed: MFMAs
// and barriers alone 135 us (2.03 PFLOP/s, the rate of MFMAs on registers only),
// with the output 153, with the LDS reads 167, with loads that all hit one line
// 180, that hit L2 195 (before the shorter epilogue), with the real ones 207.
// What is left is the delivery of 64 KiB per stage and compute unit.
template <typename C, bool SECOND>
__device__ __forceinline__ void turns_group(const TileArgs& p, unsigned char* ring, const TileLoads<C, C::NW>& loads, int ns,
                                            int wm, int wn, int r, int g, f32x4 (&acc)[C::FM][C::FN])
{
    constexpr int FM = C::FM, FN = C::FN;
    constexpr bool FP4 = C::FP4;
    constexpr int kSliceK = C::kSliceK;
    constexpr int LS = TileLoads<C, C::NW>::LS, kFirst = LS / 2;   // group 0's loads: before and between its MFMAs
    TileFrags<C> frags;
    frags.init(ring, wm, wn, r, g);
    u32x4 xf[FM], wf[FN];
    int sx[FM], sw[FN];

    auto read = [&](int st, int j) __attribute__((always_inline)) {
        const int at = (st % 2) * C::kStage;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            wf[f] = frags.b(at, j, f);
            sw[f] = frags.sb(2 * st + j, f);
        }
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            xf[f] = frags.a(at, j, f);
            sx[f] = frags.sa(2 * st + j, f);
        }
    };
    auto mask = [&](int s) __attribute__((always_inline)) {
        const int64_t valid = p.K - (int64_t)s * kSliceK - g * (kSliceK / 4);
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            xf[f] = mask_k<FP4>(xf[f], valid);
            sx[f] = valid > 0 ? sx[f] : 127;
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            wf[f] = mask_k<FP4>(wf[f], valid);
            sw[f] = valid > 0 ? sw[f] : 127;
        }
    };
    // the MFMAs of a slice with loads t0 .. t1-1 of stage st spread among them
    auto compute = [&](auto whole_loads, int st, auto t0, auto t1) __attribute__((always_inline)) {
        constexpr int kLoads = decltype(t1)::value - decltype(t0)::value;
        constexpr int kEvery = FM * FN / (kLoads > 0 ? kLoads : 1);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < FN * FM; ++i) {
            tile_mfma<FP4>(xf[i % FM], wf[i / FM], sx[i % FM], sw[i / FM], acc[i % FM][i / FM]);
            if (i % kEvery == kEvery / 2 && i / kEvery < kLoads) {
                __builtin_amdgcn_sched_barrier(0);
                loads.template issue_one<decltype(whole_loads)::value>(st, decltype(t0)::value + i / kEvery);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };
    using None = std::integral_constant<int, 0>;
    auto stage = [&](auto whole_loads, auto tail, int st) __attribute__((always_inline)) {
        read(st, 0);
        if constexpr (!SECOND) {
#pragma unroll
            for (int t = 0; t < kFirst; ++t)
                loads.template issue_one<decltype(whole_loads)::value>(st + 1, t);
        }
        wg_barrier_reads_done();
        if constexpr (decltype(tail)::value)
            mask(2 * st);
        if constexpr (!SECOND)
            compute(whole_loads, st + 1, std::integral_constant<int, kFirst>{}, std::integral_constant<int, LS>{});
        else
            compute(whole_loads, st + 2, None{}, None{});
        wg_barrier();
        read(st, 1);
        if constexpr (SECOND)
            async_wait<0>();
        wg_barrier_reads_done();
        if constexpr (decltype(tail)::value)
            mask(2 * st + 1);
        if constexpr (!SECOND) {
            compute(whole_loads, st + 1, None{}, None{});
            async_wait<0>();
        } else {
            compute(whole_loads, st + 2, None{}, std::integral_constant<int, LS>{});
        }
        wg_barrier();
    };
    if constexpr (SECOND) {
        loads.issue(1);
        wg_barrier();
    }
    const int inside = (int)(p.K / (2 * kSliceK)), nst = (ns + 1) / 2;
    constexpr int kAhead = SECOND ? 2 : 1;
    int st = 0;
    for (; st + kAhead < inside; ++st)
        stage(std::true_type{}, std::false_type{}, st);
    for (; st < inside; ++st)
        stage(std::false_type{}, std::false_type{}, st);
    if (st < nst)
        stage(std::false_type{}, std::true_type{}, st);
    if constexpr (!SECOND)
        wg_barrier();
    async_wait<0>();
}

template <typename C>
__device__ __forceinline__ void turns_body(const TileArgs& p, unsigned char* ring, int block)
{
    static_assert(C::KB == 2 && C::R == 2 && C::NW == 8, "eight waves, two stages of two slices");
    const int lane = threadIdx.x & 63, w = (int)uniform(threadIdx.x >> 6);
    const int wm = w / C::WN, wn = w % C::WN;
    const int r = lane & 15, g = lane >> 4;
    int tn;
    const int tm = tile_of(block, p.tiles_m, p.tiles_n, tn);
    const int m0 = tm * C::BM, n0 = tn * C::kOutN;
    const int ns = (int)((p.K + C::kSliceK - 1) / C::kSliceK);
    TileLoads<C, C::NW> loads;
    loads.init(p, ring, w, lane, m0, n0);
    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < C::FN; ++fn)
            acc[fm][fn] = f32x4{0.f, 0.f, 0.f, 0.f};
    loads.issue_first_scales();
    loads.issue(0);
    async_wait<0>();
    wg_barrier();
    if (w < 4)
        turns_group<C, false>(p, ring, loads, ns, wm, wn, r, g, acc);
    else
        turns_group<C, true>(p, ring, loads, ns, wm, wn, r, g, acc);
    tile_store<C>(p, acc, m0, n0, wm, wn, r, g);
}

// Small tiles, where a wave has too few MFMAs per slice to hide the latency of
// its LDS reads and loads behind them: NL waves only load, up to R - 1 stages
// ahead, and the computing waves read all fragments of a stage at once.  One
// barrier per stage hands it over: a loading wave waits for its own loads of
// the stage first, a computing wave for its reads of the stage before, whose
// slot is refilled next.  One token through H = 2048, I = 768 (6.3 MB): 3.4 us
// against 8.1 with 64 x 64 tiles whose waves all load and compute; 16 tokens
// through H = 4096, I = 12288 (203 MB): 36 to 39 us, 5.2 to 5.6 TB/s, the rate of a
// large copy.
template <typename C, int NL>
__device__ __forceinline__ void stream_body(const TileArgs& p, unsigned char* ring, int block)
{
    constexpr int FM = C::FM, FN = C::FN, KB = C::KB, R = C::R;
    constexpr bool FP4 = C::FP4;
    constexpr int kSliceK = C::kSliceK;
    static_assert(!FP4 || C::kGroupInStage, "a stage brings its own scales");
    using Loads = TileLoads<C, NL>;
    constexpr int LS = Loads::LS;
    static_assert(R >= 2 && (R - 2) * LS < 64, "ring depth");

    const int lane = threadIdx.x & 63, w = (int)uniform(threadIdx.x >> 6);
    int tn;
    const int tm = tile_of(block, p.tiles_m, p.tiles_n, tn);
    const int m0 = tm * C::BM, n0 = tn * C::kOutN;
    const int ns = (int)((p.K + kSliceK - 1) / kSliceK);
    const int nst = (ns + KB - 1) / KB;                            // stages

    if (w >= C::NW) {
        Loads loads;
        loads.init(p, ring, w - C::NW, lane, m0, n0);
        for (int st = 0; st < R - 1 && st < nst; ++st)
            loads.issue(st);
        for (int st = 0; st < nst; ++st) {
            async_wait_later<LS, R - 2>(min(R - 2, nst - 1 - st));
            wg_barrier();
            if (st + R - 1 < nst)
                loads.issue(st + R - 1);
        }
        return;
    }

    const int wm = w / C::WN, wn = w % C::WN;
    const int r = lane & 15, g = lane >> 4;
    TileFrags<C> frags;
    frags.init(ring, wm, wn, r, g);
    f32x4 acc[FM][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
            acc[fm][fn] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto stage = [&](auto tail, int st) __attribute__((always_inline)) {
        wg_barrier_reads_done();
        const int at = (st % R) * C::kStage;
        u32x4 x[KB][FM], wf[KB][FN];
        int sx[KB][FM], sw[KB][FN];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
#pragma unroll
            for (int f = 0; f < FM; ++f) {
                x[j][f] = frags.a(at, j, f);
                sx[j][f] = frags.sa(st * KB + j, f);
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                wf[j][f] = frags.b(at, j, f);
                sw[j][f] = frags.sb(st * KB + j, f);
            }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if constexpr (decltype(tail)::value) {
                const int64_t valid = p.K - (int64_t)(st * KB + j) * kSliceK - g * (kSliceK / 4);
#pragma unroll
                for (int f = 0; f < FM; ++f) {
                    x[j][f] = mask_k<FP4>(x[j][f], valid);
                    sx[j][f] = valid > 0 ? sx[j][f] : 127;
                }
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    wf[j][f] = mask_k<FP4>(wf[j][f], valid);
                    sw[j][f] = valid > 0 ? sw[j][f] : 127;
                }
            }
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int fm = 0; fm < FM; ++fm)
                    tile_mfma<FP4>(x[j][fm], wf[j][fn], sx[j][fm], sw[j][fn], acc[fm][fn]);
        }
    };
    const int whole = (int)(p.K / (kSliceK * KB));
    for (int st = 0; st < whole; ++st)
        stage(std::false_type{}, st);
    if (whole < nst)
        stage(std::true_type{}, whole);
    tile_store<C>(p, acc, m0, n0, wm, wn, r, g);
}

template <typename C>
__global__ __launch_bounds__(C::NW * 64) void k_tile(TileArgs p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char ring[C::kRing];
    tile_body<C>(p, ring, (int)blockIdx.x);
}

template <typename C>
__global__ __launch_bounds__(C::NW * 64) void k_turns(TileArgs p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char ring[C::kRing];
    turns_body<C>(p, ring, (int)blockIdx.x);
}

template <typename C, int NL>
__global__ __launch_bounds__((C::NW + NL) * 64) void k_stream(TileArgs p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char ring[C::kRing];
    stream_body<C, NL>(p, ring, (int)blockIdx.x);
}

}  // namespace bi
