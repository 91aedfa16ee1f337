// bi_linear_bwd.hip -- the products of the backward passes in one launch:
// dx = dy W (the weight read by columns), dw = dy^T x (both operands read by
// columns) and the column sums of dy.
#include "bi_ffn.h"
#include "bi_plan.h"
#include "bi_tile.h"
#include "bi_tile_rule.h"

namespace bi {

// What the kernels' 32-bit offsets and tile counts can hold.
static bool in_range(int64_t lddy, int64_t ldx, int64_t ldw, int64_t M, int64_t N, int64_t K)
{
    const int64_t lim = int64_t(1) << 32, grid = int64_t(1) << 29;
    return 255 * lddy * 2 + N * 2 < lim && 32 * lddy * 2 + 512 < lim && 32 * ldw * 2 + 512 < lim &&
           32 * ldx * 2 + 512 < lim && N < (int64_t(1) << 29) && ((M + 31) / 32) * ((K + 31) / 32) < grid &&
           ((N + 63) / 64) * ((K + 63) / 64) < grid;
}

// Column sums of dy where dw's tiles do not take them along (dw not wanted, or in
// its largest tiles, whose matrix instructions leave no room: 221 us against 217
// at 4096 x 4096 x 4096), so db's order of addition follows from the launch: a
// workgroup takes 64 columns and all rows; thread (row
// lane, group of 8 columns) adds its rows in ascending order in fp32, and the 64
// row lanes are added in order.  No split over rows, so nothing is left to fold.
// 4096 x 4096 alone: 11 us, 3.4 TB/s (256 workgroups of 16 columns: the same).
struct SumArgs {
    const uint16_t* dy;
    int64_t lddy;
    float* db;
    int64_t M;
    int N;
};
constexpr int kSumCols = 64, kBwdThreads = 512, kSumLanes = kBwdThreads / 8;

__device__ __forceinline__ void colsum_body(const SumArgs& p, unsigned char* lds, int block)
{
    float(*part)[kSumCols + 1] = reinterpret_cast<float(*)[kSumCols + 1]>(lds);
    const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
    const int c = block * kSumCols + cg * 8;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < p.N) {
#pragma unroll 4
        for (int64_t m = rl; m < p.M; m += kSumLanes) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(p.dy + m * p.lddy + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[2 * j] += __uint_as_float(v[j] << 16);
                acc[2 * j + 1] += __uint_as_float(v[j] & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        part[rl][cg * 8 + j] = acc[j];
    __syncthreads();
    const int col = block * kSumCols + (int)threadIdx.x;
    if (threadIdx.x < kSumCols && col < p.N) {
        float t = part[0][threadIdx.x];
        for (int l = 1; l < kSumLanes; ++l)
            t += part[l][threadIdx.x];
        p.db[col] = t;
    }
}

// Tile shapes of the two products, all on 512 threads so that any two can share
// a launch.  dx's four smallest stream (short batches: few tiles and a long sum
// over N); the others load and compute in every wave.  16 x 32 is for the
// longest sums on the fewest tiles, where a slice's time is the delivery of its
// bytes to one compute unit: dx of 30 rows, N 16928, K 992 takes 45 us instead of
// 56 on 32 x 32 tiles.  On more tiles it is the slower one (119 rows, N 6752, K
// 1792: 35 us against 27), and the rule does not take it there.
template <int SHAPE, bool CA> struct BwdShape;
template <bool CA> struct BwdShape<0, CA> {
    using C = TileCfg<32, 32, 2, 2, 4, 4, CA, true, false, kEpiLinear>;
    static constexpr int NL = 4;
};
template <bool CA> struct BwdShape<1, CA> {
    using C = TileCfg<64, 64, 4, 2, 2, 4, CA, true, false, kEpiLinear>;
    static constexpr int NL = 0;
};
template <> struct BwdShape<1, false> {
    using C = TileCfg<32, 64, 2, 2, 4, 3, false, true, false, kEpiLinear>;
    static constexpr int NL = 4;
};
template <bool CA> struct BwdShape<2, CA> {
    using C = TileCfg<128, 64, 4, 2, 2, 4, CA, true, false, kEpiLinear>;
    static constexpr int NL = 0;
};
template <bool CA> struct BwdShape<3, CA> {
    using C = TileCfg<128, 128, 4, 2, 2, 4, CA, true, false, kEpiLinear>;
    static constexpr int NL = 0;
};
template <> struct BwdShape<5, false> {
    using C = TileCfg<16, 32, 1, 2, 4, 4, false, true, false, kEpiLinear>;
    static constexpr int NL = 4;
};
template <> struct BwdShape<6, false> {
    using C = TileCfg<64, 64, 2, 2, 2, 4, false, true, false, kEpiLinear>;
    static constexpr int NL = 4;
};
template <bool CA> struct BwdShape<4, CA> {
    using C = TileCfg<256, 256, CA ? 4 : 2, CA ? 2 : 4, 2, 2, CA, true, false, kEpiLinear>;
    static constexpr int NL = 0;
};

template <typename S>
__device__ __forceinline__ void bwd_body(const TileArgs& p, unsigned char* ring, int block)
{
    constexpr int kUsed = (S::C::NW + S::NL) * 64;
    static_assert(kUsed == kBwdThreads || (S::NL > 0 && kUsed < kBwdThreads), "one workgroup size");
    if (kUsed < kBwdThreads && (int)threadIdx.x >= kUsed)
        return;                                         // a barrier counts the waves that are left
    if constexpr (S::NL > 0)
        stream_body<typename S::C, S::NL>(p, ring, block);
    else if constexpr (S::C::R == 2)
        turns_body<typename S::C>(p, ring, block);
    else
        tile_body<typename S::C>(p, ring, block);
}

// Workgroups 0 .. ndx-1 tile dx, the next ndw dw, the rest sum columns.
template <int DX, int DW>
__global__ __launch_bounds__(kBwdThreads) void k_bwd(TileArgs dx, TileArgs dw, SumArgs sum, int ndx, int ndw)
{
    using SX = BwdShape<DX, false>;
    using SW = BwdShape<DW, true>;
    constexpr int kRing = SX::C::kRing > SW::C::kRing ? SX::C::kRing : SW::C::kRing;
    static_assert(kRing >= kSumLanes * (kSumCols + 1) * 4, "column sums fit the ring");
    __shared__ __attribute__((aligned(1024))) unsigned char ring[kRing];
    const int b = (int)blockIdx.x;
    if (b < ndx)
        bwd_body<SX>(dx, ring, b);
    else if (b < ndx + ndw)
        bwd_body<SW>(dw, ring, b - ndx);
    else
        colsum_body(sum, ring, b - ndx - ndw);
}

// the costs are explained in bi_tile_rule.h
static constexpr TileShape kDxShapes[] = {{32, 32, 1.17f, 0.054f, 1.13f}, {32, 64, 1.71f, 0.075f, 1.05f}, {128, 64, 1.38f, 0.154f, 0.f},
                                      {128, 128, 1.61f, 0.231f, 0.f}, {256, 256, 3.29f, 0.554f, 0.f}, {16, 32, 1.00f, 0.047f, 1.76f},
                                      {64, 64, 1.20f, 0.095f, 1.28f}};
static constexpr TileShape kDwShapes[] = {{0, 0, 0.f, 0.f, 0.f},          {64, 64, 1.61f, 0.113f, 1.04f}, {128, 64, 2.34f, 0.165f, 0.f},
                                      {128, 128, 2.88f, 0.235f, 0.f}, {256, 256, 6.22f, 0.590f, 0.f}};
constexpr int kNumDxShapes = 7, kNumDwShapes = 4;       // dw: shapes 1 .. 4
// A launch before dw's takes one of dx's first six: the seventh's cost was taken
// beside dw's tiles and is too low for two launches (290 rows, N 16032, K 3296:
// 184 us instead of 157).
constexpr int kNumDxApart = 6;

// The shape pairs that are built; a product alone may use its side of any.
static const int kBwdPairs[][2] = {{0, 1}, {1, 1}, {2, 1}, {0, 2}, {2, 2}, {0, 3}, {2, 3}, {3, 3}, {3, 4}, {4, 4},
                                   {5, 1}, {5, 2}, {5, 3}, {6, 1}, {6, 2}, {6, 3}};
constexpr int kNumBwdPairs = (int)(sizeof(kBwdPairs) / sizeof(kBwdPairs[0]));

// Both products in one launch: all tiles' times spread over the compute units
// plus a part of a last round, but at least the longest tile's time, with some of
// the other's where there is more than one round.  Over 54 problems the launches
// chosen this way took 1.02 times the fastest of the ten pairs without 16 x 32
// tiles and streaming 64 x 64 ones and of all shapes in two launches; with the
// first 98 drawn backward passes took 0.98 of their time, with the second 122 took
// 0.99 of that (0.72 to 0.95 where dx runs on them; 349 rows, N 8032, K 1568 of a
// gated layer 70 -> 50 us).
static float pair_time(const TileShape& a, const TileShape& b, int64_t M, int64_t N, int64_t K, bool dw_f32, int cus)
{
    const float ta = tile_once(a, (N + 31) / 32, false), tb = tile_once(b, (M + 31) / 32, dw_f32);
    const int64_t na = tile_count(a, M, K), nb = tile_count(b, N, K);
    const bool shared = a.share > 0.f && b.share > 0.f, rounds = na + nb > cus;
    const float most = ta > tb ? ta : tb, least = ta > tb ? tb : ta;
    const float all = ((float)na * ta * (shared ? a.share : 1.f) + (float)nb * tb * (shared ? b.share : 1.f)) / (float)cus +
                      (rounds ? (shared ? 0.25f : 0.75f) * least : 0.f);
    const float longest = most + (rounds ? 0.2f * least : 0.f);
    return kTileLaunch + (all > longest ? all : longest);
}

// Beside dw's tiles, workgroups of sums end last: M 4096, N and K 1024 took 38.9
// us with them and takes 31.4 (N 256, K 4096: 42.1, 34.9; M 333: 10.9, 11.2).  So
// dw's tiles sum, all but the largest.
constexpr bool tiles_sum(int dw_shape) { return dw_shape < kNumDwShapes; }

template <int DX, int DW>
static hipError_t bwd_launch(TileArgs dx, TileArgs dw, SumArgs sum, hipStream_t s)
{
    using CX = typename BwdShape<DX, false>::C;
    using CW = typename BwdShape<DW, true>::C;
    static_assert(CX::BM == kDxShapes[DX].bm && CX::BN == kDxShapes[DX].bn && CW::BM == kDwShapes[DW].bm &&
                      CW::BN == kDwShapes[DW].bn && CW::kSums == tiles_sum(DW), "the rule's table");
    dx.tiles_m = (dx.M + CX::BM - 1) / CX::BM;
    dx.tiles_n = (dx.N + CX::BN - 1) / CX::BN;
    dw.tiles_m = (dw.M + CW::BM - 1) / CW::BM;
    dw.tiles_n = (dw.N + CW::BN - 1) / CW::BN;
    const int ndx = dx.y ? dx.tiles_m * dx.tiles_n : 0, ndw = dw.y ? dw.tiles_m * dw.tiles_n : 0;
    if (dw.y && CW::kSums) {
        dw.db = sum.db;
        sum.db = nullptr;
    }
    const int nsum = sum.db ? (sum.N + kSumCols - 1) / kSumCols : 0;
    k_bwd<DX, DW><<<(unsigned)(ndx + ndw + nsum), kBwdThreads, 0, s>>>(dx, dw, sum, ndx, ndw);
    return hipGetLastError();
}

static hipError_t bwd_launch_pair(int pair, const TileArgs& dx, const TileArgs& dw, const SumArgs& sum, hipStream_t s)
{
    switch (pair) {
    case 0: return bwd_launch<0, 1>(dx, dw, sum, s);
    case 1: return bwd_launch<1, 1>(dx, dw, sum, s);
    case 2: return bwd_launch<2, 1>(dx, dw, sum, s);
    case 3: return bwd_launch<0, 2>(dx, dw, sum, s);
    case 4: return bwd_launch<2, 2>(dx, dw, sum, s);
    case 5: return bwd_launch<0, 3>(dx, dw, sum, s);
    case 6: return bwd_launch<2, 3>(dx, dw, sum, s);
    case 7: return bwd_launch<3, 3>(dx, dw, sum, s);
    case 8: return bwd_launch<3, 4>(dx, dw, sum, s);
    case 9: return bwd_launch<4, 4>(dx, dw, sum, s);
    case 10: return bwd_launch<5, 1>(dx, dw, sum, s);
    case 11: return bwd_launch<5, 2>(dx, dw, sum, s);
    case 12: return bwd_launch<5, 3>(dx, dw, sum, s);
    case 13: return bwd_launch<6, 1>(dx, dw, sum, s);
    case 14: return bwd_launch<6, 2>(dx, dw, sum, s);
    default: return bwd_launch<6, 3>(dx, dw, sum, s);
    }
}

// Workgroups of a launch of shape pair `pair` with these outputs.
static int64_t pair_groups(int pair, bool dx, bool dw, bool db, int64_t M, int64_t N, int64_t K)
{
    const int w = kBwdPairs[pair][1];
    return (dx ? tile_count(kDxShapes[kBwdPairs[pair][0]], M, K) : 0) + (dw ? tile_count(kDwShapes[w], N, K) : 0) +
           (db && !(dw && tiles_sum(w)) ? (N + kSumCols - 1) / kSumCols : 0);
}

// The first pair with this shape on its dx (0) or dw (1) side.
static int pair_with(int side, int shape)
{
    for (int i = 0; i < kNumBwdPairs; ++i)
        if (kBwdPairs[i][side] == shape)
            return i;
    return 0;
}

static BwdPlan choose(bool dx, bool dw, int dw_bf16, int64_t M, int64_t N, int64_t K)
{
    const int cus = device_cu_count();
    // each product's own best shape, and the best pair for one launch
    const int bx = pick_tile(kDxShapes, dw ? kNumDxApart : kNumDxShapes, M, K, (N + 31) / 32, false, cus);
    const int bw = 1 + pick_tile(kDwShapes + 1, kNumDwShapes, N, K, (M + 31) / 32, !dw_bf16, cus);
    if (!dw)
        return {pair_with(0, dx ? bx : 1), -1};
    if (!dx)
        return {pair_with(1, bw), -1};
    int best = 0;
    float best_time = 0.f;
    for (int i = 0; i < kNumBwdPairs; ++i) {
        // half of 64 rows idle (M 1, N 3232, K 1856: 14.8 us against 13.0)
        if (kBwdPairs[i][0] == 6 && M <= 32)
            continue;
        const float t = pair_time(kDxShapes[kBwdPairs[i][0]], kDwShapes[kBwdPairs[i][1]], M, N, K, !dw_bf16, cus);
        if (i == 0 || t < best_time) {
            best = i;
            best_time = t;
        }
    }
    const float apart = tile_time(kDxShapes[bx], M, K, (N + 31) / 32, false, cus) +
                        tile_time(kDwShapes[bw], N, K, (M + 31) / 32, !dw_bf16, cus);
    if (best_time <= apart)
        return {best, -1};
    return {pair_with(0, bx), pair_with(1, bw)};
}

bool plan_linear_bwd(bool dx, bool dw, bool db, int dw_bf16, int64_t lddy, int64_t ldx, int64_t ldw, int64_t M, int64_t N,
                     int64_t K, BwdPlan* plan)
{
    if (!in_range(lddy, dw ? ldx : 0, dx ? ldw : 0, M, N, K))
        return false;
    const BwdPlan p = *plan = choose(dx, dw, dw_bf16, M, N, K);
    if (p.second < 0)
        return grid_ok(pair_groups(p.first, dx, dw, db, M, N, K));
    const bool late = tiles_sum(kBwdPairs[p.second][1]);
    return grid_ok(pair_groups(p.first, true, false, db && !late, M, N, K)) &&
           grid_ok(pair_groups(p.second, false, true, db && late, M, N, K));
}

TileInfo linear_bwd_tile_info(int side, int dw_bf16, int64_t M, int64_t N, int64_t K)
{
    const BwdPlan p = choose(true, true, dw_bf16, M, N, K);
    const int i = kBwdPairs[side == 1 && p.second >= 0 ? p.second : p.first][side];
    if (side == 1) {
        switch (i) {
        case 1: return tile_info<BwdShape<1, true>>(i);
        case 2: return tile_info<BwdShape<2, true>>(i);
        case 3: return tile_info<BwdShape<3, true>>(i);
        default: return tile_info<BwdShape<4, true>>(i);
        }
    }
    switch (i) {
    case 0: return tile_info<BwdShape<0, false>>(i);
    case 1: return tile_info<BwdShape<1, false>>(i);
    case 2: return tile_info<BwdShape<2, false>>(i);
    case 3: return tile_info<BwdShape<3, false>>(i);
    case 4: return tile_info<BwdShape<4, false>>(i);
    case 5: return tile_info<BwdShape<5, false>>(i);
    default: return tile_info<BwdShape<6, false>>(i);
    }
}

hipError_t launch_linear_bwd(const BwdPlan& plan, const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx,
                             const uint16_t* w, int64_t ldw, uint16_t* dx, int64_t lddx, void* dw, int dw_bf16, int64_t lddw,
                             float* db, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    TileArgs a{}, b{};
    SumArgs sum{dy, lddy, db, M, (int)N};
    a.a = b.a = reinterpret_cast<const unsigned char*>(dy);
    a.lda = b.lda = lddy * 2;
    a.b = reinterpret_cast<const unsigned char*>(w);
    a.ldb = ldw * 2;
    a.y = dx;
    a.ldy = lddx;
    a.y_bf16 = 1;
    a.M = (int)M;
    a.N = (int)K;
    a.K = N;
    b.b = reinterpret_cast<const unsigned char*>(x);
    b.ldb = ldx * 2;
    b.y = dw;
    b.ldy = lddw;
    b.y_bf16 = dw_bf16;
    b.M = (int)N;
    b.N = (int)K;
    b.K = M;
    if (plan.second < 0)
        return bwd_launch_pair(plan.first, a, b, sum, s);
    TileArgs none{};
    SumArgs nosum{};
    const bool late = tiles_sum(kBwdPairs[plan.second][1]);
    const hipError_t e = bwd_launch_pair(plan.first, a, none, late ? nosum : sum, s);
    return e != hipSuccess ? e : bwd_launch_pair(plan.second, none, b, late ? sum : nosum, s);
}

__global__ __launch_bounds__(256) void k_zero_rows(unsigned char* __restrict__ p, int64_t pitch, int64_t rows, int64_t words)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t i = threadIdx.x; i < words; i += 256)
            reinterpret_cast<uint32_t*>(p + r * pitch)[i] = 0u;
}

hipError_t launch_zero_rows(void* p, int64_t pitch, int64_t rows, int64_t bytes, hipStream_t s)
{
    k_zero_rows<<<(unsigned)(rows < 4096 ? rows : 4096), 256, 0, s>>>(reinterpret_cast<unsigned char*>(p), pitch, rows,
                                                                    bytes / 4);
    return hipGetLastError();
}

}  // namespace bi
