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

// The end of expert e's rows as given, held to 0 .. T; 0 past the last expert.
__device__ __forceinline__ int group_end(const GroupArgs& q, int e)
{
    if (e >= q.E)
        return 0;
    const int64_t v = q.ends[e];
    return v < 0 ? 0 : v > q.T ? q.T : (int)v;
}

// 64 experts from e0 on, one to a lane: their first row and their number of
// rows.  `from`: where the experts before them ended; moved on.  The running
// maximum makes a partition of any values, so that no ends read or write out of range.
__device__ __forceinline__ void group_rows(const GroupArgs& q, int e0, int lane, int& from, int& first, int& rows)
{
    const int end = max(wave_incl_max(group_end(q, e0 + lane), lane), from);
    const int before = __shfl_up(end, 1);
    first = lane == 0 ? from : before;
    rows = end - first;
    from = __builtin_amdgcn_readlane(end, 63);
}

struct GroupTile {
    int e, first, rows;         // expert, its rows
    int tm, tn;                 // tile among the expert's
};

// The tile of workgroup w among all experts' BM-row tiles x tiles_n, dealt to the
// XCDs as tile_of does; false where there is none.
template <int BM>
__device__ __forceinline__ bool find_tile(const GroupArgs& q, int tiles_n, int w, GroupTile& t)
{
    const int lane = threadIdx.x & 63;
    int from = 0, first, rows, total = 0;
    for (int e0 = 0; e0 < q.E; e0 += 64) {
        group_rows(q, e0, lane, from, first, rows);
        total += __builtin_amdgcn_readlane((int)wave_incl_scan((uint32_t)((rows + BM - 1) / BM), lane), 63);
    }
    const int tiles = total * tiles_n;
    const int x = w & 7, j = w >> 3;
    const int per = tiles >> 3, more = tiles & 7;
    if (j >= per + (x < more ? 1 : 0))
        return false;
    const int tr = tile_at(x * per + min(x, more) + j, total, tiles_n, t.tn);
    int upto = 0;
    from = 0;
    for (int e0 = 0;; e0 += 64) {
        group_rows(q, e0, lane, from, first, rows);
        const int mine = (rows + BM - 1) / BM;
        const int incl = upto + (int)wave_incl_scan((uint32_t)mine, lane);
        const uint64_t past = __ballot(incl > tr);
        if (past) {
            const int l = __builtin_ctzll(past);
            t.e = e0 + l;
            t.first = __builtin_amdgcn_readlane(first, l);
            t.rows = __builtin_amdgcn_readlane(rows, l);
            t.tm = tr - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(mine, l));
            return true;
        }
        upto = __builtin_amdgcn_readlane(incl, 63);
    }
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

template <typename S>
__global__ __launch_bounds__((S::C::NW + S::NL) * 64) void k_grouped(TileArgs p, GroupArgs q)
{
    __shared__ __attribute__((aligned(1024))) unsigned char ring[S::C::kRing];
    GroupTile t;
    if (!find_tile<S::C::BM>(q, p.tiles_n, (int)blockIdx.x, t))
        return;
    at_group(p, q, t);
    tile_any<S>(p, ring, t.tm, t.tn);
}

// dw of one expert per tile: the sum runs over its rows.  An expert without rows
// gets zeros.
template <typename S>
__global__ __launch_bounds__((S::C::NW + S::NL) * 64) void k_grouped_dw(TileArgs p, GroupArgs q)
{
    using C = typename S::C;
    __shared__ __attribute__((aligned(1024))) unsigned char ring[C::kRing];
    int tn;
    const int tr = tile_of((int)blockIdx.x, q.E * p.tiles_m, p.tiles_n, tn);
    const int e = tr / p.tiles_m, tm = tr - e * p.tiles_m;
    const int lane = threadIdx.x & 63;
    int from = 0, first, rows;
    for (int e0 = 0; e0 <= e; e0 += 64)
        group_rows(q, e0, lane, from, first, rows);
    first = __builtin_amdgcn_readlane(first, e & 63);
    rows = __builtin_amdgcn_readlane(rows, e & 63);
    const int es = p.y_bf16 ? 2 : 4;
    p.y = reinterpret_cast<unsigned char*>(p.y) + (int64_t)e * q.stride_b;
    if (rows == 0) {
        const int units = C::BN * es / 16, have = (p.N - tn * C::BN) * es / 16;
        for (int i = threadIdx.x; i < C::BM * units; i += C::NW * 64) {
            const int m = tm * C::BM + i / units, u = i % units;
            if (m < p.M && u < have)
                reinterpret_cast<u32x4*>(reinterpret_cast<unsigned char*>(p.y) + ((int64_t)m * p.ldy + tn * C::BN) * es)[u] =
                    u32x4{0u, 0u, 0u, 0u};
        }
        return;
    }
    p.a += (int64_t)first * p.lda;
    p.b += (int64_t)first * p.ldb;
    p.K = rows;
    tile_any<S>(p, ring, tm, tn);
}

// --------------------------------------------------------------------- shapes

template <int BM, int BN, int WM, int WN, int KB, int R, int NL_, bool CA, bool CB, TileType TYPE>
struct GroupShape {
    using C = TileCfg<BM, BN, WM, WN, KB, R, CA, CB, TYPE, kEpiLinear>;
    static constexpr int NL = NL_;
};

enum GroupOp { kGroupBf16, kGroupInt8, kGroupDx, kGroupDw };

// the costs are explained in bi_tile_rule.h; a slice is 32 k, in 8 bits 64
static const TileShape kRowShapes[] = {
    {16, 16, 0.67f, 0.037f, 1.10f}, {16, 32, 0.29f, 0.063f, 1.10f}, {32, 32, 0.64f, 0.072f, 1.10f}, {64, 32, 0.90f, 0.088f, 0.f},
    {128, 64, 0.65f, 0.204f, 0.f},  {128, 128, 0.72f, 0.277f, 0.f}, {256, 256, 1.87f, 0.688f, 0.f},
};
static const TileShape kDxShapes[] = {
    {16, 32, 1.00f, 0.047f, 1.76f}, {32, 32, 1.17f, 0.054f, 1.13f}, {32, 64, 1.71f, 0.075f, 1.05f},
    {128, 64, 1.38f, 0.154f, 0.f},  {128, 128, 1.61f, 0.231f, 0.f}, {256, 256, 3.29f, 0.554f, 0.f},
};
static const TileShape kDwShapes[] = {
    {64, 64, 1.61f, 0.113f, 1.04f}, {128, 64, 2.34f, 0.165f, 0.f}, {128, 128, 2.88f, 0.235f, 0.f}, {256, 256, 6.22f, 0.590f, 0.f},
};

// f of the shape at an index of the operator's list
template <GroupOp OP, typename F>
static auto group_shape(int i, F f)
{
    if constexpr (OP == kGroupBf16 || OP == kGroupInt8) {
        constexpr TileType T = OP == kGroupInt8 ? kInt8 : kBf16;
        switch (i) {
        case 0: return f(GroupShape<16, 16, 1, 1, 8, 4, 4, false, false, T>{});
        case 1: return f(GroupShape<16, 32, 1, 1, 4, 4, 4, false, false, T>{});
        case 2: return f(GroupShape<32, 32, 2, 1, 4, 4, 4, false, false, T>{});
        case 3: return f(GroupShape<64, 32, 4, 1, 4, 4, 4, false, false, T>{});
        case 4: return f(GroupShape<128, 64, 4, 1, 2, 4, 0, false, false, T>{});
        case 5: return f(GroupShape<128, 128, 4, 2, 2, 4, 0, false, false, T>{});
        default: return f(GroupShape<256, 256, 4, 2, 2, 2, 0, false, false, T>{});
        }
    } else if constexpr (OP == kGroupDx) {
        switch (i) {
        case 0: return f(GroupShape<16, 32, 1, 2, 4, 4, 4, false, true, kBf16>{});
        case 1: return f(GroupShape<32, 32, 2, 2, 4, 4, 4, false, true, kBf16>{});
        case 2: return f(GroupShape<32, 64, 2, 2, 4, 3, 4, false, true, kBf16>{});
        case 3: return f(GroupShape<128, 64, 4, 2, 2, 4, 0, false, true, kBf16>{});
        case 4: return f(GroupShape<128, 128, 4, 2, 2, 4, 0, false, true, kBf16>{});
        default: return f(GroupShape<256, 256, 2, 4, 2, 2, 0, false, true, kBf16>{});
        }
    } else {
        switch (i) {
        case 0: return f(GroupShape<64, 64, 4, 2, 2, 4, 0, true, true, kBf16>{});
        case 1: return f(GroupShape<128, 64, 4, 2, 2, 4, 0, true, true, kBf16>{});
        case 2: return f(GroupShape<128, 128, 4, 2, 2, 4, 0, true, true, kBf16>{});
        default: return f(GroupShape<256, 256, 4, 2, 2, 2, 0, true, true, kBf16>{});
        }
    }
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

static int pick_group(GroupOp op, int64_t T, int64_t E, int64_t N, int64_t K, bool f32_out)
{
    const TileShape* t = op == kGroupDx ? kDxShapes : op == kGroupDw ? kDwShapes : kRowShapes;
    const int n = op == kGroupDx ? 6 : op == kGroupDw ? 4 : 7, cus = device_cu_count();
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
        const float time = tiles_time(t[i], tiles, slices, f32_out, cus);
        if (i == 0 || time < best_time) {
            best = i;
            best_time = time;
        }
    }
    return best;
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

template <GroupOp OP>
static hipError_t run_rows(TileArgs a, const GroupArgs& q, int shape, hipStream_t s, bool dry)
{
    return group_shape<OP>(shape, [&](auto sh) {
        using S = decltype(sh);
        using C = typename S::C;
        a.tiles_n = (a.N + C::BN - 1) / C::BN;
        const int64_t tiles = most_row_tiles(q.T, q.E, C::BM) * a.tiles_n;
        if (!grid_ok(tiles))
            return hipErrorInvalidConfiguration;
        if (dry)
            return hipSuccess;
        k_grouped<S><<<(unsigned)tiles, (C::NW + S::NL) * 64, 0, s>>>(a, q);
        return hipGetLastError();
    });
}

static hipError_t run_dw(TileArgs a, const GroupArgs& q, int shape, hipStream_t s, bool dry)
{
    return group_shape<kGroupDw>(shape, [&](auto sh) {
        using S = decltype(sh);
        using C = typename S::C;
        a.tiles_m = (a.M + C::BM - 1) / C::BM;
        a.tiles_n = (a.N + C::BN - 1) / C::BN;
        const int64_t tiles = (int64_t)q.E * a.tiles_m * a.tiles_n;
        if (!grid_ok(tiles))
            return hipErrorInvalidConfiguration;
        if (dry)
            return hipSuccess;
        k_grouped_dw<S><<<(unsigned)tiles, (C::NW + S::NL) * 64, 0, s>>>(a, q);
        return hipGetLastError();
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
    return run_rows<kGroupBf16>(a, q, pick_group(kGroupBf16, T, E, N, K, !y_bf16), s, false);
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
    return run_rows<kGroupInt8>(a, q, pick_group(kGroupInt8, T, E, N, K, !y_bf16), s, false);
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
    const int sx = pick_group(kGroupDx, T, E, N, K, false), sw = pick_group(kGroupDw, T, E, N, K, !dw_bf16);
    const bool do_dx = dx && T > 0;
    // both grids are checked before either launch: a refused call enqueues nothing
    for (const bool dry : {true, false}) {
        hipError_t e = do_dx ? run_rows<kGroupDx>(a, qx, sx, s, dry) : hipSuccess;
        if (e == hipSuccess && dw)
            e = run_dw(b, qw, sw, s, dry);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

TileInfo grouped_tile_info(int op, int64_t T, int64_t E, int64_t N, int64_t K, int out_bf16)
{
    const auto info = [](int i) { return [i](auto shape) { return tile_info<decltype(shape)>(i); }; };
    const int i = pick_group((GroupOp)op, T, E, N, K, !out_bf16);
    switch (op) {
    case kGroupBf16: return group_shape<kGroupBf16>(i, info(i));
    case kGroupInt8: return group_shape<kGroupInt8>(i, info(i));
    case kGroupDx: return group_shape<kGroupDx>(i, info(i));
    default: return group_shape<kGroupDw>(i, info(i));
    }
}

}  // namespace bi
