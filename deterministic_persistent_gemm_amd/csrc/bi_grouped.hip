// bi_grouped.hip -- products grouped by expert: rows of x are sorted by expert,
// and expert e's rows, ends[e-1] .. ends[e] - 1, meet its own weight.  Forward
// in bf16 and in 8-bit integers, and the two products of the bf16 backward pass.
//
// The group sizes stay on the device, so the grid holds the most tiles that any
// split of the rows over the experts can need; workgroups find their tile from
// `ends` and those without one end at once.
#include "bi_ffn.h"
#include "bi_plan.h"
#include "bi_tile.h"
#include "bi_tile_rule.h"

namespace bi {

struct GroupArgs {
    const int64_t* ends;        // [E]
    int E;
    int T;                      // rows of x
    int64_t stride_b;           // bytes from expert to expert: the weight (dw: dw itself)
    int64_t stride_sb;          // 8-bit operands: the weight's scales
};

// Inclusive running maximum over the wave's lanes of values that are not negative.
__device__ __forceinline__ int wave_incl_max(int v, int lane)
{
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));   // row_shr:1
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));   // row_shr:2
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));   // row_shr:4
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));   // row_shr:8
    const int r0 = __builtin_amdgcn_readlane(v, 15), r1 = __builtin_amdgcn_readlane(v, 31), r2 = __builtin_amdgcn_readlane(v, 47);
    const int row = lane >> 4;
    return max(max(v, row >= 1 ? r0 : 0), max(row >= 2 ? r1 : 0, row >= 3 ? r2 : 0));
}

// The experts' rows, NE experts in a row to a lane: where the lane's first begins and
// where each of its ends.  All of `ends` is asked for at once: a workgroup has nothing
// to do until it knows its tile.  Ends are held to 0 .. T, and the running maximum makes
// a partition of any values, so that none read or write out of range.
template <int NE>
struct GroupRows {
    int from, end[NE];

    __device__ __forceinline__ GroupRows(const GroupArgs& q, int lane)
    {
        int64_t v[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i)
            v[i] = q.ends[min(lane * NE + i, q.E - 1)];         // past the last expert: no rows
        int top = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            top = max(top, (int)max(min(v[i], (int64_t)q.T), (int64_t)0));
            end[i] = top;
        }
        const int before = __shfl_up(wave_incl_max(top, lane), 1);
        from = lane == 0 ? 0 : before;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            end[i] = max(end[i], from);
    }
    __device__ __forceinline__ int first(int i) const { return i == 0 ? from : end[i - 1]; }
    __device__ __forceinline__ int rows(int i) const { return end[i] - first(i); }
};

// f(NE) of the fewest experts to a lane that hold E in a wave
template <typename F>
__device__ __forceinline__ void with_lanes(int E, F f)
{
    if (E <= 64)
        f(std::integral_constant<int, 1>{});
    else if (E <= 128)
        f(std::integral_constant<int, 2>{});
    else if (E <= 256)
        f(std::integral_constant<int, 4>{});
    else
        f(std::integral_constant<int, kMaxExperts / 64>{});
}

struct GroupTile {
    int e, first, rows;         // expert, its rows
    int tm, tn;                 // tile among the expert's
};

// The tile of workgroup w among all experts' BM-row tiles x tiles_n; false where there
// is none.  Each XCD takes one contiguous eighth of the list, which goes expert by
// expert, four row tiles at a time, column by column: tiles that share rows of A or of
// the weight are then started one after the other, within the few microseconds for
// which a line stays in the L2.  (Eight row tiles of several experts at a time, as
// tile_of has it for one product, 32768 rows of 128 experts, 1536 x 2048: 316 us.)
template <int BM>
__device__ __forceinline__ bool find_tile(const GroupArgs& q, int tiles_n, int w, GroupTile& t)
{
    const int lane = threadIdx.x & 63;
    bool found = false;
    with_lanes(q.E, [&](auto ne) __attribute__((always_inline)) {
        constexpr int NE = decltype(ne)::value;
        const GroupRows<NE> r(q, lane);
        int mine = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            mine += (r.rows(i) + BM - 1) / BM;
        const int incl = (int)wave_incl_scan((uint32_t)mine, lane);
        const int total = __builtin_amdgcn_readlane(incl, 63), tiles = total * tiles_n;
        const int x = w & 7, j = w >> 3;
        const int per = tiles >> 3, more = tiles & 7;
        found = j < per + (x < more ? 1 : 0);
        if (!found)
            return;
        const int at_tile = x * per + min(x, more) + j, tr = at_tile / tiles_n;
        const int l = __builtin_ctzll(__ballot(incl > tr));     // the lane of the tile's expert
        int at = incl - mine, e = 0, first = 0, rows = 0, before = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int n = (r.rows(i) + BM - 1) / BM;
            if (tr >= at && tr < at + n) {
                e = lane * NE + i;
                first = r.first(i);
                rows = r.rows(i);
                before = at;
            }
            at += n;
        }
        t.e = __builtin_amdgcn_readlane(e, l);
        t.first = __builtin_amdgcn_readlane(first, l);
        t.rows = __builtin_amdgcn_readlane(rows, l);
        t.tm = tile_at<4>(at_tile - __builtin_amdgcn_readlane(before, l) * tiles_n, (t.rows + BM - 1) / BM, tiles_n, t.tn);
    });
    return found;
}

// Expert e's rows.
__device__ __forceinline__ void rows_of(const GroupArgs& q, int e, int& first, int& rows)
{
    const int lane = threadIdx.x & 63;
    with_lanes(q.E, [&](auto ne) __attribute__((always_inline)) {
        constexpr int NE = decltype(ne)::value;
        const GroupRows<NE> r(q, lane);
        int f = r.first(0), n = r.rows(0);
#pragma unroll
        for (int i = 1; i < NE; ++i)
            if (e % NE == i) {
                f = r.first(i);
                n = r.rows(i);
            }
        first = __builtin_amdgcn_readlane(f, e / NE);
        rows = __builtin_amdgcn_readlane(n, e / NE);
    });
}

// p at its expert's rows and weight
__device__ __forceinline__ void at_group(TileArgs& p, const GroupArgs& q, const GroupTile& t)
{
    p.a += (int64_t)t.first * p.lda;
    p.b += (int64_t)t.e * q.stride_b;
    p.sa += (int64_t)t.first * 4;
    p.sb += (int64_t)t.e * q.stride_sb;
    p.y = reinterpret_cast<unsigned char*>(p.y) + (int64_t)t.first * p.ldy * (p.y_bf16 ? 2 : 4);
    p.M = t.rows;
}

// Workgroup w of a product over the experts' rows.
template <typename S>
__device__ __forceinline__ void rows_body(TileArgs& p, const GroupArgs& q, unsigned char* ring, int w)
{
    GroupTile t;
    if (!find_tile<S::C::BM>(q, p.tiles_n, w, t))
        return;
    at_group(p, q, t);
    tile_any<S>(p, ring, t.tm, t.tn);
}

// p of expert e's dw, whose sum runs over its rows.
__device__ __forceinline__ void at_expert(TileArgs& p, const GroupArgs& q, int e, int first, int rows)
{
    p.y = reinterpret_cast<unsigned char*>(p.y) + (int64_t)e * q.stride_b;
    p.a += (int64_t)first * p.lda;
    p.b += (int64_t)first * p.ldb;
    p.K = rows;
}

// Zeros for tile (tm, tn): an expert without rows.
template <typename S>
__device__ __forceinline__ void zero_tile(const TileArgs& p, int tm, int tn)
{
    using C = typename S::C;
    const int es = p.y_bf16 ? 2 : 4;
    const int units = C::BN * es / 16, have = (p.N - tn * C::BN) * es / 16;
    for (int i = threadIdx.x; i < C::BM * units; i += (C::NW + S::NL) * 64) {
        const int m = tm * C::BM + i / units, u = i % units;
        if (m < p.M && u < have)
            reinterpret_cast<u32x4*>(reinterpret_cast<unsigned char*>(p.y) + ((int64_t)m * p.ldy + tn * C::BN) * es)[u] =
                u32x4{0u, 0u, 0u, 0u};
    }
}

// Workgroup w of dw, one tile.  An expert's tiles are dealt to all XCDs, as one expert
// may have many times the rows of another; which of them gets one more goes round
// from expert to expert.
template <typename S>
__device__ __forceinline__ void dw_body(TileArgs& p, const GroupArgs& q, unsigned char* ring, int w)
{
    const int tiles = p.tiles_m * p.tiles_n, per = (tiles + 7) >> 3;
    const int j = w >> 3, e = j / per, t = ((w + e) & 7) * per + j - e * per;
    if (t >= tiles)
        return;
    int first, rows, tn;
    rows_of(q, e, first, rows);
    at_expert(p, q, e, first, rows);
    const int tm = tile_at(t, p.tiles_m, p.tiles_n, tn);
    if (rows == 0)
        zero_tile<S>(p, tm, tn);
    else
        tile_any<S>(p, ring, tm, tn);
}

// The largest tiles: a workgroup on every compute unit takes tile after tile.  Each XCD
// has a range of experts of equal cost, and its workgroups take the range's tiles in
// turn, so that an expert's rows are read into one L2 once.  32768 rows of 128 experts,
// 1536 x 2048: 424 us where demand is uneven, 408 where it is not.  (One workgroup a
// tile, an expert's tiles on all XCDs: 441 and 433; an eighth of the experts to each XCD:
// 525 and 428.)
struct GroupTable {
    int first[kMaxExperts + 1];     // where the experts' rows begin
    int cost[kMaxExperts + 1];      // and their costs, in slices a tile
};

// What a tile costs besides its slices: its first loads and its stores; its zeros,
// where there are no rows.
constexpr int kDwTileCost = 6, kDwZeroCost = 3;

// Filled by the first wave.
__device__ __forceinline__ void fill_table(GroupTable& tab, const GroupArgs& q)
{
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        if (lane == 0)
            tab.first[0] = tab.cost[0] = 0;
        with_lanes(q.E, [&](auto ne) __attribute__((always_inline)) {
            constexpr int NE = decltype(ne)::value;
            const GroupRows<NE> r(q, lane);
            int sum[NE], mine = 0;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int rows = r.rows(i);
                mine += lane * NE + i >= q.E ? 0 : rows > 0 ? (rows + 31) / 32 + kDwTileCost : kDwZeroCost;
                sum[i] = mine;
            }
            const int before = (int)wave_incl_scan((uint32_t)mine, lane) - mine;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane * NE + i < q.E) {
                    tab.first[lane * NE + i + 1] = r.end[i];
                    tab.cost[lane * NE + i + 1] = before + sum[i];
                }
        });
    }
    __syncthreads();
}

// The first tile of XCD x's range: costs before it make x eighths of all.
__device__ __forceinline__ int range_start(const GroupTable& tab, int E, int tiles, int x)
{
    if (x == 8)
        return E * tiles;
    const int64_t at = (int64_t)tab.cost[E] * x;
    int e = 0;                                          // the last expert with 8 cost[e] <= at
    for (int step = 512; step > 0; step >>= 1)
        if (e + step < E && 8 * (int64_t)tab.cost[e + step] <= at)
            e += step;
    const int64_t into = at - 8 * (int64_t)tab.cost[e], cost = 8 * (int64_t)(tab.cost[e + 1] - tab.cost[e]);
    return e * tiles + (int)(into * tiles / cost);
}

// A tile's first loads are issued before the tile before it is stored, and need not
// wait for its stores: the counter of both falls in order.
template <typename S>
__device__ __forceinline__ void dw_all(const TileArgs& p, const GroupArgs& q, unsigned char* ring, GroupTable& tab, int w, int groups)
{
    using C = typename S::C;
    static_assert(C::kGrouped && C::R == 2 && S::NL == 0, "no loads are under way at a tile's end");
    fill_table(tab, q);
    const int lane = threadIdx.x & 63, wave = (int)uniform(threadIdx.x >> 6);
    const int tiles = p.tiles_m * p.tiles_n, x = w & 7, step = groups >> 3;
    const int end = (int)uniform((uint32_t)range_start(tab, q.E, tiles, x + 1));
    int t = (int)uniform((uint32_t)range_start(tab, q.E, tiles, x)) + (w >> 3);

    TileArgs now = p, next = p;                         // of the tile at work and of the one that comes
    int m0 = 0, n0 = 0, next_m0 = 0, next_n0 = 0;
    // the next tile with rows from t on, zeros for those without; false at the end
    auto advance = [&]() __attribute__((always_inline)) {
        for (; t < end; t += step) {
            const int e = t / tiles;
            const int first = (int)uniform((uint32_t)tab.first[e]), rows = (int)uniform((uint32_t)tab.first[e + 1]) - first;
            int tn;
            const int tm = tile_at(t - e * tiles, p.tiles_m, p.tiles_n, tn);
            next = p;
            at_expert(next, q, e, first, rows);
            if (rows > 0) {
                next_m0 = tm * C::BM;
                next_n0 = tn * C::BN;
                t += step;
                return true;
            }
            zero_tile<S>(next, tm, tn);
        }
        return false;
    };
    if (!advance())
        return;
    TileLoads<C, C::NW> loads;
    loads.init(next, ring, wave, lane, next_m0, next_n0);
    loads.issue(0);
    constexpr int kStores = C::FM * C::FN / 2;          // of a whole bf16 tile, per wave
    int stores = 0;
    for (bool more = true; more;) {
        now = next;
        m0 = next_m0;
        n0 = next_n0;
        asm volatile("" : : : "memory");                // no store moves down past the wait that counts it
        if (stores == kStores)
            async_wait<kStores>();
        else if (stores == 2 * kStores)
            async_wait<2 * kStores>();
        else
            async_wait<0>();
        wg_barrier();
        f32x4 acc[C::FM][C::FN];
        turns_sums<C>(now, ring, loads, wave, lane, acc);
        // every wave is past its last read of the ring here (turns_group's last barrier)
        more = advance();
        if (more) {
            loads.init(next, ring, wave, lane, next_m0, next_n0);
            loads.issue(0);
        }
        // zeros written on the way are stores ahead of those loads: no harm.  Only a tile
        // without ragged edges has all of its stores issued by every wave
        stores = m0 + C::BM <= p.M && n0 + C::BN <= p.N ? (p.y_bf16 ? kStores : 2 * kStores) : 0;
        tile_store<C>(now, acc, m0, n0, wave / C::WN, wave % C::WN, lane & 15, lane >> 4);
    }
}

// 1536 x 2048, 128 experts, 8 of them a token, bf16.  One token: 11.6 us, the 50 MB of its
// experts' weights at 4.3 TB/s.  4096 tokens: 307 us at 0.67 PFLOP/s.  There the weights of
// all experts are read once for 256 rows each, and a stage's loads hide behind its products
// only in part: copies without stores take 299 us, without products 287, without loads
// 233, loads alone 250, products alone 199.
template <typename S>
__global__ __launch_bounds__((S::C::NW + S::NL) * 64) void k_grouped(TileArgs p, GroupArgs q)
{
    __shared__ __attribute__((aligned(1024))) unsigned char ring[S::C::kRing];
    rows_body<S>(p, q, ring, (int)blockIdx.x);
}

template <typename S> constexpr bool takes_all() { return S::C::BM == 256; }

template <typename S>
__global__ __launch_bounds__((S::C::NW + S::NL) * 64) void k_grouped_dw(TileArgs p, GroupArgs q)
{
    __shared__ __attribute__((aligned(1024))) unsigned char ring[S::C::kRing];
    if constexpr (takes_all<S>()) {
        __shared__ GroupTable tab;
        dw_all<S>(p, q, ring, tab, (int)blockIdx.x, (int)gridDim.x);
    } else {
        dw_body<S>(p, q, ring, (int)blockIdx.x);
    }
}

// Both gradients in one launch (4096 tokens at those sizes: 670 us, two launches 715).  Workgroups 0 .. first - 1 (a multiple of 8) take dx, the rest dw; the
// largest tiles the other way round, so that dx's fill the compute units as dw's
// workgroups end.
constexpr int kBothThreads = 512;

template <typename SX, typename SW>
__global__ __launch_bounds__(kBothThreads) void k_grouped_both(TileArgs dx, GroupArgs qx, TileArgs dw, GroupArgs qw, int first)
{
    constexpr int kX = (SX::C::NW + SX::NL) * 64, kW = (SW::C::NW + SW::NL) * 64;
    static_assert(kX <= kBothThreads && kW <= kBothThreads, "one workgroup size");
    __shared__ __attribute__((aligned(1024))) unsigned char ring[SX::C::kRing > SW::C::kRing ? SX::C::kRing : SW::C::kRing];
    const int b = (int)blockIdx.x;
    if constexpr (takes_all<SW>()) {
        __shared__ GroupTable tab;
        if (b < first)
            dw_all<SW>(dw, qw, ring, tab, b, first);
        else
            rows_body<SX>(dx, qx, ring, b - first);
    } else {
        // waves that a shape does not need leave before its first barrier, which counts those that are left
        if (b < first) {
            if ((int)threadIdx.x < kX)
                rows_body<SX>(dx, qx, ring, b);
        } else if ((int)threadIdx.x < kW) {
            dw_body<SW>(dw, qw, ring, b - first);
        }
    }
}

// --------------------------------------------------------------------- shapes

template <int BM, int BN, int WM, int WN, int KB, int R, int NL_, bool CA, bool CB, TileType TYPE>
struct GroupShape {
    using C = TileCfg<BM, BN, WM, WN, KB, R, CA, CB, TYPE, kEpiLinear, true>;
    static constexpr int NL = NL_;
};

enum GroupOp { kGroupBf16, kGroupInt8, kGroupDx, kGroupDw };

// Costs as in bi_tile_rule.h (a slice is 32 k, in 8 bits 64), fitted to timings of 437
// problems: 320 drawn over 1 to 128 experts, 1 to 32768 rows split evenly or not, widths
// 128 .. 4096 and k 256 .. 4096, and 117 with 8, 64 and 128 experts of 1024 x 1024 to 1536 x
// 2048 at 8 to 32768 rows.  The shapes chosen take 1.005 to 1.019 times the fastest one's
// time on average, 1.25 to 1.49 at worst (costs fitted to one half of the drawn
// problems: 1.018 to 1.032 on the other).  A shape less in its list costs 0.4 to 10
// percent on average and 12 to 150 at worst.
static const TileShape kRowShapes[] = {
    {16, 16, 2.58f, 0.033f, 1.39f}, {16, 32, 1.74f, 0.072f, 0.71f}, {32, 64, 1.73f, 0.092f, 1.33f}, {32, 128, 1.47f, 0.146f, 1.20f},
    {64, 128, 2.11f, 0.163f, 0.f},  {128, 128, 3.19f, 0.460f, 0.71f}, {256, 256, 3.89f, 0.753f, 0.f},
};
static const TileShape kRow8Shapes[] = {
    {16, 16, 3.24f, 0.046f, 1.18f}, {16, 32, 3.09f, 0.079f, 0.69f}, {32, 64, 4.07f, 0.072f, 0.73f}, {32, 128, 2.83f, 0.173f, 1.04f},
    {64, 128, 2.82f, 0.196f, 0.f},  {128, 128, 5.48f, 0.589f, 0.65f}, {256, 256, 10.70f, 1.142f, 0.f},
};
static const TileShape kDxShapes[] = {
    {16, 64, 2.38f, 0.108f, 1.20f}, {32, 32, 2.04f, 0.111f, 1.07f},  {64, 64, 1.96f, 0.144f, 1.04f},
    {64, 128, 2.19f, 0.144f, 0.f},  {128, 128, 4.17f, 0.401f, 0.71f}, {256, 256, 9.32f, 0.509f, 0.f},
};
static const TileShape kDwShapes[] = {
    {64, 64, 3.54f, 0.178f, 0.64f}, {128, 128, 3.59f, 0.622f, 0.60f}, {256, 256, 8.86f, 1.103f, 0.f},
};
constexpr int kNumRowShapes = 7, kNumDxShapes = 6, kNumDwShapes = 3;

// f of the shape at an index of the operator's list
template <GroupOp OP, typename F>
static auto group_shape(int i, F f)
{
    if constexpr (OP == kGroupBf16 || OP == kGroupInt8) {
        constexpr TileType T = OP == kGroupInt8 ? kInt8 : kBf16;
        switch (i) {
        case 0: return f(GroupShape<16, 16, 1, 1, 8, 4, 4, false, false, T>{});
        case 1: return f(GroupShape<16, 32, 1, 1, 4, 4, 4, false, false, T>{});
        case 2: return f(GroupShape<32, 64, 2, 2, 4, 3, 4, false, false, T>{});
        case 3: return f(GroupShape<32, 128, 1, 4, 2, 4, 4, false, false, T>{});
        case 4: return f(GroupShape<64, 128, 2, 2, 2, 3, 4, false, false, T>{});
        case 5: return f(GroupShape<128, 128, 4, 2, 2, 2, 0, false, false, T>{});
        default: return f(GroupShape<256, 256, 4, 2, 2, 2, 0, false, false, T>{});
        }
    } else if constexpr (OP == kGroupDx) {
        switch (i) {
        case 0: return f(GroupShape<16, 64, 1, 2, 4, 4, 4, false, true, kBf16>{});
        case 1: return f(GroupShape<32, 32, 2, 2, 4, 4, 4, false, true, kBf16>{});
        case 2: return f(GroupShape<64, 64, 2, 2, 2, 4, 4, false, true, kBf16>{});
        case 3: return f(GroupShape<64, 128, 2, 2, 2, 3, 4, false, true, kBf16>{});
        case 4: return f(GroupShape<128, 128, 2, 4, 2, 2, 0, false, true, kBf16>{});
        default: return f(GroupShape<256, 256, 2, 4, 2, 2, 0, false, true, kBf16>{});
        }
    } else {
        switch (i) {
        case 0: return f(GroupShape<64, 64, 4, 2, 2, 4, 0, true, true, kBf16>{});
        case 1: return f(GroupShape<128, 128, 2, 2, 1, 4, 0, true, true, kBf16>{});
        default: return f(GroupShape<256, 256, 4, 2, 2, 2, 0, true, true, kBf16>{});
        }
    }
}

// dw's tiles where dx's are beside them in one launch: 128 x 128 on as many waves and
// registers as dx's tiles have, so that two workgroups still share a compute unit.
template <typename F>
static auto both_dw_shape(int i, F f)
{
    if (i == 0)
        return f(GroupShape<64, 64, 4, 2, 2, 4, 0, true, true, kBf16>{});
    if (i == 1)
        return f(GroupShape<128, 128, 4, 2, 1, 4, 0, true, true, kBf16>{});
    return f(GroupShape<256, 256, 4, 2, 2, 2, 0, true, true, kBf16>{});
}

// Row tiles of any split of T rows over E experts, at most.
static int64_t most_row_tiles(int64_t T, int64_t E, int bm)
{
    const int64_t a = E < T ? E : T;
    return (T + a * (bm - 1)) / bm;
}

// What is expected of them: experts with rows if every row took one at random,
// each with half a tile of its last rows missing.
static int64_t likely_row_tiles(int64_t T, int64_t E, int bm)
{
    const float a = (float)E * (1.f - expf(-(float)T / (float)E));
    const float t = (float)T / (float)bm + 0.5f * a;
    return (int64_t)((t > a ? t : a) + 0.5f);
}

// f32_out counts for y alone: dw's stores, the same bytes in any shape, are what all its
// shapes wait for (65 problems in fp32: 1.020 of the fastest, with the wider stores priced
// by the tile 1.026).
static int pick_group(GroupOp op, int64_t T, int64_t E, int64_t N, int64_t K, bool f32_out)
{
    const TileShape* t = op == kGroupDx ? kDxShapes : op == kGroupDw ? kDwShapes : op == kGroupInt8 ? kRow8Shapes : kRowShapes;
    const int n = op == kGroupDx ? kNumDxShapes : op == kGroupDw ? kNumDwShapes : kNumRowShapes, cus = device_cu_count();
    int best = 0;
    float best_time = 0.f;
    for (int i = 0; i < n; ++i) {
        int64_t tiles, slices;
        if (op == kGroupDw) {
            tiles = E * tile_count(t[i], N, K);
            slices = (T / E + 31) / 32;
        } else {
            const int64_t cols = op == kGroupDx ? K : N;
            tiles = likely_row_tiles(T, E, t[i].bm) * ((cols + t[i].bn - 1) / t[i].bn);
            slices = op == kGroupDx ? (N + 31) / 32 : op == kGroupInt8 ? (K + 63) / 64 : (K + 31) / 32;
        }
        const float time = tiles_time(t[i], tiles, slices, f32_out && op != kGroupDw, cus);
        if (i == 0 || time < best_time) {
            best = i;
            best_time = time;
        }
    }
    return best;
}

// The shapes of a backward pass with both gradients, and whether one launch takes them.
// Side by side in one launch small tiles take 0.78 of the time of two launches (55
// problems, 0.62 to 1.00), the largest of both 0.94 (9 problems, 0.90 to 0.98).  Where
// only dw's are the largest, its second largest beside small tiles of dx (0.94), or the
// largest of both (dx's being 64 x 128 or 128 x 128: 0.92); where only dx's are, one
// launch is the slower one (1.12 to 1.39).  Those problems have many rows to an expert.
// The rule does not compare times, and with few rows to an expert one launch loses, bf16
// dw being a write that the other gradient's tiles wait beside, and dx at 256 rows a tile
// serving a handful.  128 experts, 8 for each token, dx alone + dw alone / both, us: 1536
// x 2048, 1 token 150 / 153, 8 223 / 266, 64 345 / 383, 500 415 / 434, 2000 564 / 538, 4096
// 737 / 677; 2048 x 768, 1 token 86 / 81, 8 118 / 137, 64 191 / 226, 500 229 / 254, 2000 317 /
// 298, 4096 415 / 378.
struct GroupBwdPlan {
    int dx, dw;
    bool together;
};

static GroupBwdPlan plan_grouped_bwd(int64_t T, int64_t E, int64_t N, int64_t K)
{
    constexpr int kMostDx = kNumDxShapes - 1, kMostDw = kNumDwShapes - 1;
    const int dx = pick_group(kGroupDx, T, E, N, K, false), dw = pick_group(kGroupDw, T, E, N, K, false);
    if (dw < kMostDw)
        return {dx, dw, dx < kMostDx};
    return dx >= 3 ? GroupBwdPlan{kMostDx, kMostDw, true} : GroupBwdPlan{dx, kMostDw - 1, true};
}

bool grouped_fits(int64_t lda, int64_t ldw, int es, int64_t T, int64_t N, int64_t K, int64_t E)
{
    const int64_t lim = int64_t(1) << 32;
    return 255 * lda * es + K * es < lim && 255 * ldw * es + K * es < lim && N < (int64_t(1) << 29) &&
           (es == 2 || K <= kInt8MaxK) && E <= kMaxExperts;
}

bool grouped_bwd_fits(int64_t lddy, int64_t ldx, int64_t ldw, int64_t T, int64_t N, int64_t K, int64_t E)
{
    const int64_t lim = int64_t(1) << 32;
    return 255 * lddy * 2 + N * 2 < lim && 32 * lddy * 2 + 512 < lim && 32 * ldw * 2 + 512 < lim && 32 * ldx * 2 + 512 < lim &&
           N < (int64_t(1) << 29) && E <= kMaxExperts;
}

// Workgroups of a product over rows, and of dw; both fill in the tile counts.
template <typename C>
static int64_t rows_groups(TileArgs& a, const GroupArgs& q)
{
    a.tiles_n = (a.N + C::BN - 1) / C::BN;
    return most_row_tiles(q.T, q.E, C::BM) * a.tiles_n;
}

template <typename S>
static int64_t dw_groups(TileArgs& a, const GroupArgs& q)
{
    a.tiles_m = (a.M + S::C::BM - 1) / S::C::BM;
    a.tiles_n = (a.N + S::C::BN - 1) / S::C::BN;
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    if (!takes_all<S>())
        return (tiles + 7) / 8 * 8 * q.E;
    // one workgroup for every compute unit, a multiple of 8
    const int cus = device_cu_count();
    return tiles * q.E < (int64_t(1) << 31) ? (cus < 8 ? 8 : cus / 8 * 8) : int64_t(1) << 31;
}

// dry: only whether a launch can hold the grid
template <GroupOp OP>
static hipError_t run_rows(TileArgs a, const GroupArgs& q, int shape, hipStream_t s, bool dry = false)
{
    return group_shape<OP>(shape, [&](auto sh) {
        using S = decltype(sh);
        const int64_t groups = rows_groups<typename S::C>(a, q);
        if (!grid_ok(groups))
            return hipErrorInvalidConfiguration;
        if (dry)
            return hipSuccess;
        k_grouped<S><<<(unsigned)groups, (S::C::NW + S::NL) * 64, 0, s>>>(a, q);
        return hipGetLastError();
    });
}

static hipError_t run_dw(TileArgs a, const GroupArgs& q, int shape, hipStream_t s, bool dry = false)
{
    return group_shape<kGroupDw>(shape, [&](auto sh) {
        using S = decltype(sh);
        const int64_t groups = dw_groups<S>(a, q);
        if (!grid_ok(groups))
            return hipErrorInvalidConfiguration;
        if (dry)
            return hipSuccess;
        k_grouped_dw<S><<<(unsigned)groups, (S::C::NW + S::NL) * 64, 0, s>>>(a, q);
        return hipGetLastError();
    });
}

static hipError_t run_both(TileArgs a, const GroupArgs& qx, int sx, TileArgs b, const GroupArgs& qw, int sw, hipStream_t s)
{
    return group_shape<kGroupDx>(sx, [&](auto x) {
        return both_dw_shape(sw, [&](auto w) {
            using SX = decltype(x);
            using SW = decltype(w);
            if constexpr ((SX::C::BM == 256) == (SW::C::BM == 256)) {
                const int64_t ndx = (rows_groups<typename SX::C>(a, qx) + 7) / 8 * 8, ndw = dw_groups<SW>(b, qw);
                if (!grid_ok(ndx + ndw))
                    return hipErrorInvalidConfiguration;
                k_grouped_both<SX, SW><<<(unsigned)(ndx + ndw), kBothThreads, 0, s>>>(a, qx, b, qw, (int)(takes_all<SW>() ? ndw : ndx));
                return hipGetLastError();
            } else {
                return hipErrorInvalidConfiguration;    // no such kernel; plan_grouped_bwd asks for no such pair
            }
        });
    });
}

hipError_t launch_grouped_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, int64_t stride_w,
                               const int64_t* ends, int64_t E, void* y, int y_bf16, int64_t ldy, int64_t T, int64_t N, int64_t K,
                               hipStream_t s)
{
    TileArgs a{};
    a.a = reinterpret_cast<const unsigned char*>(x);
    a.b = reinterpret_cast<const unsigned char*>(w);
    a.lda = ldx * 2;
    a.ldb = ldw * 2;
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = y_bf16;
    a.N = (int)N;
    a.K = K;
    const GroupArgs q{ends, (int)E, (int)T, stride_w * 2, 0};
    return run_rows<kGroupBf16>(a, q, pick_group(kGroupBf16, T, E, N, K, !y_bf16), s);
}

hipError_t launch_grouped_int8(const int8_t* xq, int64_t ldx, const float* xs, const int8_t* wq, int64_t ldw, int64_t stride_w,
                               const float* ws, int64_t stride_ws, const int64_t* ends, int64_t E, void* y, int y_bf16,
                               int64_t ldy, int64_t T, int64_t N, int64_t K, hipStream_t s)
{
    TileArgs a{};
    a.a = reinterpret_cast<const unsigned char*>(xq);
    a.b = reinterpret_cast<const unsigned char*>(wq);
    a.lda = ldx;
    a.ldb = ldw;
    a.sa = reinterpret_cast<const unsigned char*>(xs);
    a.sb = reinterpret_cast<const unsigned char*>(ws);
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = y_bf16;
    a.N = (int)N;
    a.K = K;
    const GroupArgs q{ends, (int)E, (int)T, stride_w, stride_ws * 4};
    return run_rows<kGroupInt8>(a, q, pick_group(kGroupInt8, T, E, N, K, !y_bf16), s);
}

hipError_t launch_grouped_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
                              int64_t stride_w, const int64_t* ends, int64_t E, uint16_t* dx, int64_t lddx, void* dw, int dw_bf16,
                              int64_t lddw, int64_t stride_dw, int64_t T, int64_t N, int64_t K, hipStream_t s)
{
    TileArgs a{}, b{};
    a.a = b.a = reinterpret_cast<const unsigned char*>(dy);
    a.lda = b.lda = lddy * 2;
    a.b = reinterpret_cast<const unsigned char*>(w);
    a.ldb = ldw * 2;
    a.y = dx;
    a.ldy = lddx;
    a.y_bf16 = 1;
    a.N = (int)K;
    a.K = N;
    b.b = reinterpret_cast<const unsigned char*>(x);
    b.ldb = ldx * 2;
    b.y = dw;
    b.ldy = lddw;
    b.y_bf16 = dw_bf16;
    b.M = (int)N;
    b.N = (int)K;
    const GroupArgs qx{ends, (int)E, (int)T, stride_w * 2, 0};
    const GroupArgs qw{ends, (int)E, (int)T, stride_dw * (dw_bf16 ? 2 : 4), 0};
    const bool do_dx = dx && T > 0;
    if (!do_dx)
        return dw ? run_dw(b, qw, pick_group(kGroupDw, T, E, N, K, false), s) : hipSuccess;
    if (!dw)
        return run_rows<kGroupDx>(a, qx, pick_group(kGroupDx, T, E, N, K, false), s);
    const GroupBwdPlan plan = plan_grouped_bwd(T, E, N, K);
    if (plan.together)
        return run_both(a, qx, plan.dx, b, qw, plan.dw, s);
    // both grids are checked before either launch: a refused call enqueues nothing
    for (const bool dry : {true, false}) {
        hipError_t e = run_rows<kGroupDx>(a, qx, plan.dx, s, dry);
        if (e == hipSuccess)
            e = run_dw(b, qw, plan.dw, s, dry);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

TileInfo grouped_tile_info(int op, int64_t T, int64_t E, int64_t N, int64_t K, int out_bf16)
{
    const auto info = [](int i) { return [i](auto shape) { return tile_info<decltype(shape)>(i); }; };
    const auto alone = [&](GroupOp o) { return pick_group(o, T, E, N, K, !out_bf16 && o != kGroupDx); };
    switch (op) {
    case BI_GROUPED_BF16: return group_shape<kGroupBf16>(alone(kGroupBf16), info(alone(kGroupBf16)));
    case BI_GROUPED_INT8: return group_shape<kGroupInt8>(alone(kGroupInt8), info(alone(kGroupInt8)));
    case BI_GROUPED_DX_ALONE: return group_shape<kGroupDx>(alone(kGroupDx), info(alone(kGroupDx)));
    case BI_GROUPED_DW_ALONE: return group_shape<kGroupDw>(alone(kGroupDw), info(alone(kGroupDw)));
    default: break;
    }
    const GroupBwdPlan plan = plan_grouped_bwd(T, E, N, K);
    if (op == BI_GROUPED_DX)
        return group_shape<kGroupDx>(plan.dx, info(plan.dx));
    return plan.together ? both_dw_shape(plan.dw, info(plan.dw)) : group_shape<kGroupDw>(plan.dw, info(plan.dw));
}

}  // namespace bi
