// bi_norm.hip -- layer norm and its backward pass.
//
//   m = sum x / H,  v = sum (x - m)^2 / H,  r = 1 / sqrt(v + eps)
//   n = (x - m) r,  y = n w + b
//   g = dy w,  dx = r (g - (sum g + n sum(g n)) / H),  dw = sum_rows dy n,  db = sum_rows dy
//
// A row stays in the registers of its team of T threads, so that it is read once
// and the variance is taken about the mean (no difference of large sums).  T and
// the P chunks of eight values per thread follow from H and the types alone, and
// with them the order of every sum over a row: a thread's chunks one by one, the
// lanes of a wave as a butterfly, then the waves in order.
//
// Both passes are bound by memory as long as a row's loads are on their way while
// the row before is worked on: loads are made by every lane (past the row's end of
// its last chunk, past the last row of that row), since a load under a condition is
// waited for where the condition ends.
#include "bi_ffn.h"
#include "bi_plan.h"
#include "bi_rows.h"

namespace bi {

// w or b of a thread's chunks; `none` where there is no such vector.
template <int T, int P>
__device__ __forceinline__ void load_vector(const float* w, float none, int t, int chunks, float (&v)[P][8])
{
    RowRaw<false, P> raw;
    if (w)
        raw.template load<T>(w, 0, t, chunks);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[i][j] = w ? raw.at(i, j) : none;
}

// Sums of K values over teams of T threads.  Two buffers in turn: a wave that
// writes one again has passed the barrier behind its last readers.
template <int T, int TEAMS, int K>
struct TeamSum {
    static constexpr int W = T / 64;
    float (*buf)[TEAMS][K][W];
    int turn = 0;

    __device__ __forceinline__ void operator()(float (&s)[K])
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
            s[k] = wave_sum(s[k]);
        if constexpr (W > 1) {
            const int team = threadIdx.x / T, wave = threadIdx.x % T / 64;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    buf[turn][team][k][wave] = s[k];
            }
            // no __syncthreads: its fence would wait for the loads of the next row
            wg_barrier_reads_done();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                s[k] = buf[turn][team][k][0];
#pragma unroll
                for (int w = 1; w < W; ++w)
                    s[k] += buf[turn][team][k][w];
            }
            turn ^= 1;
        }
    }
};

// Differences from the mean are held scaled by 2^-7, a power of two that loses
// nothing of differences of 2^-119 and more: their squares then add up to the variance
// times H / 16384, which overflows only where the variance itself does.
constexpr float kDiffScale = 1.0f / 128.0f;
static_assert(kNormMaxH == 128 * 128, "the scale");

struct NormArgs {
    const void* x;
    int64_t ldx;
    const float* w;             // [H] or nullptr: ones
    const float* b;             // [H] or nullptr: zeros
    float eps;
    void* y;
    int64_t ldy;
    float* mean;                // [M] or nullptr
    float* rstd;
    int64_t M;
    int H;
};

// Bound by HBM from a few thousand rows on, by one pass of latency before: 8192 rows of
// 4096, fp32 to bf16 with statistics, 40.7 us (201 MB, 4.95 TB/s; a large copy reaches
// 5.1), bf16 28.2; one row of 4096 3.2 us.
template <bool XB, bool YB, int T, int P, int TEAMS>
__global__ __launch_bounds__(T * TEAMS) void k_layer_norm(NormArgs p)
{
    __shared__ __attribute__((aligned(16))) float buf[2][TEAMS][1][T / 64];
    TeamSum<T, TEAMS, 1> sum{buf};
    const int t = threadIdx.x % T, team = (int)uniform(threadIdx.x / T), chunks = p.H / 8;
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    int64_t m = (int64_t)blockIdx.x * TEAMS + team;
    RowRaw<XB, P> cur, next;
    cur.template load<T>(p.x, min(m, p.M - 1) * p.ldx, t, chunks);
    float w[P][8], b[P][8];
    load_vector<T, P>(p.w, 1.f, t, chunks, w);
    load_vector<T, P>(p.b, 0.f, t, chunks, b);
    const float h = (float)p.H;
    for (int64_t m0 = (int64_t)blockIdx.x * TEAMS; m0 < p.M; m0 += step, m += step) {
        next.template load<T>(p.x, min(m + step, p.M - 1) * p.ldx, t, chunks);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float c = cur.at(i, 0);
#pragma unroll
            for (int j = 1; j < 8; ++j)
                c += cur.at(i, j);
            s[0] += i * T + t < chunks ? c : 0.f;
        }
        sum(s);
        const float mean = s[0] / h, off = -mean * kDiffScale;
        float q[1] = {0.f};
        float d[P][8];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float c = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[i][j] = __builtin_fmaf(cur.at(i, j), kDiffScale, off);
                c = __builtin_fmaf(d[i][j], d[i][j], c);
            }
            q[0] += i * T + t < chunks ? c : 0.f;
        }
        sum(q);
        const float rstd = 1.f / sqrtf(q[0] / (h * (kDiffScale * kDiffScale)) + p.eps), back = rstd * (1.f / kDiffScale);
        RowRaw<YB, P> out;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = __builtin_fmaf(d[i][j] * back, w[i][j], b[i][j]);
            out.set(i, o);
        }
        // the next row is waited for here, before the stores, and not with them
        cur = next;
        __builtin_amdgcn_sched_barrier(0);
        if (m < p.M) {
            out.template store<T>(p.y, m * p.ldy, t, chunks);
            if (t == 0) {
                if (p.mean)
                    p.mean[m] = mean;
                if (p.rstd)
                    p.rstd[m] = rstd;
            }
        }
    }
}

struct NormBwdArgs {
    const void* dy;
    int64_t lddy;
    const void* x;
    int64_t ldx;
    const float* mean;
    const float* rstd;
    const float* w;
    void* dx;                   // or nullptr
    int64_t lddx;
    float* part;                // [workgroup][2][H] sums of dy n and of dy, or nullptr
    float* dw;                  // few rows: [H] or nullptr, summed by columns beside the rows
    float* db;
    int row_groups;             // workgroups that take rows; the others take columns
    int64_t M;
    int H;
};

// dw and db of 64 columns: 8 threads of eight columns by 64 row lanes; a lane adds its
// rows in ascending order, 16 lanes are added in order, then the four sixteens.  The
// statistics are there already, so nothing of this waits for the rows' own sums.
constexpr int kBwdThreads = 512, kSumCols = 64, kSumLanes = kBwdThreads / 8;

template <bool DB, bool XB>
__device__ __forceinline__ void column_sums(const NormBwdArgs& p, int block, float (*part)[2 * kSumCols + 1])
{
    const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3, c = block * kSumCols + cg * 8;
    float dw[8] = {}, db[8] = {};
    if (c < p.H) {
#pragma unroll 4
        for (int64_t m = rl; m < p.M; m += kSumLanes) {
            RowRaw<XB, 1> x;
            RowRaw<DB, 1> d;
            x.template load<0>(p.x, m * p.ldx, c / 8, p.H / 8);
            d.template load<0>(p.dy, m * p.lddy, c / 8, p.H / 8);
            const float mean = p.mean[m], rstd = p.rstd[m];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[j] = __builtin_fmaf(d.at(0, j), (x.at(0, j) - mean) * rstd, dw[j]);
                db[j] += d.at(0, j);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        part[rl][cg * 8 + j] = dw[j];
        part[rl][kSumCols + cg * 8 + j] = db[j];
    }
    __syncthreads();
    const int col = threadIdx.x & (2 * kSumCols - 1), quarter = threadIdx.x / (2 * kSumCols);
    float t = part[quarter * 16][col];
#pragma unroll
    for (int l = 1; l < 16; ++l)
        t += part[quarter * 16 + l][col];
    __syncthreads();
    part[quarter][col] = t;
    __syncthreads();
    const int at = block * kSumCols + (col & (kSumCols - 1));
    float* to = col < kSumCols ? p.dw : p.db;
    if (quarter == 0 && to && at < p.H)
        to[at] = ((part[0][col] + part[1][col]) + part[2][col]) + part[3][col];
}

// One pass over dy and x for all three outputs.  512 threads and one workgroup per compute
// unit: fewer partials of dw and db to write and to add.  8192 rows of 4096 bf16: 43.4 us
// with the fold (218 MB with the partials, 5.0 TB/s), 5.5 of them the second launch; 333
// rows of 2048, columns summed beside the rows, 5.2 us.
template <bool DB, bool XB, int T, int P, int TEAMS>
__global__ __launch_bounds__(T * TEAMS) void k_layer_norm_bwd(NormBwdArgs p)
{
    static_assert(T * TEAMS == kBwdThreads, "one workgroup size");
    __shared__ __attribute__((aligned(16))) float buf[2][TEAMS][2][T / 64];
    __shared__ float fold[TEAMS > 1 && T * 8 * P > kSumLanes * (2 * kSumCols + 1) ? T * 8 * P : kSumLanes * (2 * kSumCols + 1)];
    if ((int)blockIdx.x >= p.row_groups) {
        column_sums<DB, XB>(p, (int)blockIdx.x - p.row_groups, reinterpret_cast<float(*)[2 * kSumCols + 1]>(fold));
        return;
    }
    constexpr bool kAhead = P <= 2;                     // longer rows leave no registers for the next one
    TeamSum<T, TEAMS, 2> sum{buf};
    const int t = threadIdx.x % T, team = (int)uniform(threadIdx.x / T), chunks = p.H / 8;
    const int64_t step = (int64_t)p.row_groups * TEAMS;
    int64_t m = (int64_t)blockIdx.x * TEAMS + team;
    RowRaw<XB, P> x, xn;
    RowRaw<DB, P> d, dn;
    float mean, rstd, meann, rstdn;
    auto load = [&](int64_t row, RowRaw<XB, P>& xr, RowRaw<DB, P>& dr, float& mr, float& rr) __attribute__((always_inline)) {
        row = min(row, p.M - 1);
        xr.template load<T>(p.x, row * p.ldx, t, chunks);
        dr.template load<T>(p.dy, row * p.lddy, t, chunks);
        mr = p.mean[row];
        rr = p.rstd[row];
    };
    if constexpr (kAhead)
        load(m, x, d, mean, rstd);
    float w[P][8], dw[P][8] = {}, db[P][8] = {};
    load_vector<T, P>(p.w, 1.f, t, chunks, w);
    const float h = (float)p.H;
    for (int64_t m0 = (int64_t)blockIdx.x * TEAMS; m0 < p.M; m0 += step, m += step) {
        if constexpr (kAhead)
            load(m + step, xn, dn, meann, rstdn);
        else
            load(m, x, d, mean, rstd);
        // a team without a row works on zeros, which add nothing to dw and db
        const bool live = m < p.M;
        if (!live) {
            x.clear();
            d.clear();
            mean = rstd = 0.f;
        }
        float s[2] = {0.f, 0.f};
        auto norm = [&](int i, int j) __attribute__((always_inline)) { return (x.at(i, j) - mean) * rstd; };
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float c0 = 0.f, c1 = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float dy = d.at(i, j), g = dy * w[i][j], n = norm(i, j);
                c0 += g;
                c1 = __builtin_fmaf(g, n, c1);
                dw[i][j] = __builtin_fmaf(dy, n, dw[i][j]);
                db[i][j] += dy;
            }
            s[0] += i * T + t < chunks ? c0 : 0.f;
            s[1] += i * T + t < chunks ? c1 : 0.f;
        }
        RowRaw<XB, P> out;
        if (p.dx) {
            sum(s);
            const float c0 = s[0] / h, c1 = s[1] / h;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = rstd * (d.at(i, j) * w[i][j] - __builtin_fmaf(norm(i, j), c1, c0));
                out.set(i, o);
            }
        }
        // the next row is waited for here, before the stores, and not with them
        if constexpr (kAhead) {
            x = xn;
            d = dn;
            mean = meann;
            rstd = rstdn;
            __builtin_amdgcn_sched_barrier(0);
        }
        if (p.dx && live)
            out.template store<T>(p.dx, m * p.lddx, t, chunks);
    }
    if (!p.part)
        return;
    // the teams' sums in order, then the workgroup's partial
    auto out = [&](float (&a)[P][8], int which) __attribute__((always_inline)) {
        if constexpr (TEAMS > 1) {
            for (int k = 1; k < TEAMS; ++k) {
                __syncthreads();
                if (team == k) {
#pragma unroll
                    for (int i = 0; i < P; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            fold[(i * 8 + j) * T + t] = a[i][j];
                }
                __syncthreads();
                if (team == 0) {
#pragma unroll
                    for (int i = 0; i < P; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            a[i][j] += fold[(i * 8 + j) * T + t];
                }
            }
        }
        if (team == 0) {
            RowRaw<false, P> sums;
#pragma unroll
            for (int i = 0; i < P; ++i)
                sums.set(i, a[i]);
            sums.template store<T>(p.part, ((int64_t)blockIdx.x * 2 + which) * p.H, t, chunks);
        }
    };
    out(dw, 0);
    out(db, 1);
}

// dw and db from G <= 256 partials: a workgroup takes 32 of the 2 H columns, 8
// threads of four columns by 32 slices of the partials; a slice's partials (all on
// their way at once) are added in order, then the slices.
constexpr int kFoldSlices = 32, kFoldPer = 256 / kFoldSlices;

__global__ __launch_bounds__(256) void k_layer_norm_fold(const float* __restrict__ part, float* __restrict__ dw,
                                                         float* __restrict__ db, int G, int H)
{
    __shared__ f32x4 acc[kFoldSlices][8];
    const int cl = threadIdx.x & 7, sl = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + cl * 4, at = min(c, 2 * H - 4);
    const int per = (G + kFoldSlices - 1) / kFoldSlices, first = sl * per;
    f32x4 v[kFoldPer];
#pragma unroll
    for (int k = 0; k < kFoldPer; ++k)
        v[k] = *reinterpret_cast<const f32x4*>(part + (int64_t)min(first + k, G - 1) * 2 * H + at);
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kFoldPer; ++k)
        if (k < per && first + k < G)
            a += v[k];
    acc[sl][cl] = a;
    __syncthreads();
    if (sl == 0 && c < 2 * H) {
#pragma unroll
        for (int k = 1; k < kFoldSlices; ++k)
            a += acc[k][cl];
        float* to = c < H ? dw : db;
        if (to)
            *reinterpret_cast<f32x4*>(to + (c < H ? c : c - H)) = a;
    }
}

// f(T, P) of a row length
template <typename F>
static void norm_shape(int64_t H, F f)
{
    using std::integral_constant;
    if (H <= 512)
        f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (H <= 1024)
        f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (H <= 2048)
        f(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    else if (H <= 4096)
        f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (H <= 8192)
        f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else
        f(integral_constant<int, 512>{}, integral_constant<int, 4>{});
}

template <typename F>
static void two_types(int a_bf16, int b_bf16, F f)
{
    if (a_bf16)
        b_bf16 ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
    else
        b_bf16 ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

hipError_t launch_layer_norm(const void* x, int x_bf16, int64_t ldx, const float* w, const float* b, float eps, void* y, int y_bf16,
                             int64_t ldy, float* mean, float* rstd, int64_t M, int64_t H, hipStream_t s)
{
    const NormArgs p{x, ldx, w, b, eps, y, ldy, mean, rstd, M, (int)H};
    two_types(x_bf16, y_bf16, [&](auto xb, auto yb) {
        norm_shape(H, [&](auto T, auto P) {
            constexpr int R = T < 256 ? 256 / T : 1;
            const int64_t groups = (M + R - 1) / R, most = (int64_t)device_cu_count() * (1536 / (T * R));
            k_layer_norm<decltype(xb)::value, decltype(yb)::value, T, P, R>
                <<<(unsigned)(groups < most ? groups : most), T * R, 0, s>>>(p);
        });
    });
    return hipGetLastError();
}

// Rows are taken by at most 256 workgroups, one per compute unit.  Over many rows each
// leaves a partial of dw and db, which a second launch adds; up to kColumnRows
// rows, workgroups beside them sum the columns, which reads x and dy twice but needs no
// second launch and no workspace.  Both forms at 1024 rows of bf16, columns / fold, us: H 512
// 6.6 / 8.3, 2048 11.4 / 11.9, 4096 13.3 / 15.3, 8192 18.2 / 19.4, 16384 34.7 / 38.2; at 333
// 5.0 / 8.1, 5.1 / 9.3, 5.9 / 11.8, 9.1 / 16.5, 13.6 / 23.5; at 1536 8.4 / 8.5, 13.9 / 13.3, 17.1 /
// 15.9, 24.8 / 24.6, 50.3 / 48.9; at 2048 16.9 / 8.8 to 63.9 / 58.4.
constexpr int64_t kColumnRows = 1024;

static int64_t bwd_groups(int64_t M, int64_t rows)
{
    const int64_t groups = (M + rows - 1) / rows;
    return groups < 256 ? groups : 256;
}

size_t layer_norm_bwd_ws(int64_t M, int64_t H)
{
    int64_t groups = 0;
    norm_shape(H, [&](auto T, auto) { groups = bwd_groups(M, kBwdThreads / T); });
    return M > kColumnRows ? (size_t)groups * 2 * (size_t)H * 4 : 0;
}

hipError_t launch_layer_norm_bwd(const void* dy, int dy_bf16, int64_t lddy, const void* x, int x_bf16, int64_t ldx,
                                 const float* mean, const float* rstd, const float* w, void* dx, int64_t lddx, float* dw, float* db,
                                 int64_t M, int64_t H, void* ws, hipStream_t s)
{
    NormBwdArgs p{dy, lddy, x, ldx, mean, rstd, w, dx, lddx, nullptr, dw, db, 0, M, (int)H};
    const bool sums = dw || db, columns = sums && M <= kColumnRows, fold = sums && !columns;
    if (fold)
        p.part = reinterpret_cast<float*>(ws);
    two_types(dy_bf16, x_bf16, [&](auto yb, auto xb) {
        norm_shape(H, [&](auto T, auto P) {
            constexpr int R = kBwdThreads / T;
            p.row_groups = dx || fold ? (int)bwd_groups(M, R) : 0;
            const int groups = p.row_groups + (columns ? (int)((H + kSumCols - 1) / kSumCols) : 0);
            k_layer_norm_bwd<decltype(yb)::value, decltype(xb)::value, T, P, R><<<(unsigned)groups, kBwdThreads, 0, s>>>(p);
        });
    });
    if (fold)
        k_layer_norm_fold<<<(unsigned)((2 * H + 31) / 32), 256, 0, s>>>(p.part, dw, db, p.row_groups, (int)H);
    return hipGetLastError();
}

}  // namespace bi
