// bi_norm.hip -- layer norm and its backward pass.
//
//   m = sum x / H,  v = sum (x - m)^2 / H,  r = 1 / sqrt(v + eps)
//   n = (x - m) r,  y = n w + b
//   g = dy w,  dx = r (g - (sum g + n sum(g n)) / H),  dw = sum_rows dy n,  db = sum_rows dy
//
// A row stays in the registers of its team of T threads, so that it is read once
// and the variance is taken about the mean (no difference of large sums).  T and
// the P chunks of eight values per thread follow from H alone, and with them the
// order of every sum over a row: a thread's values in ascending order, then the
// lanes of a wave as a butterfly, then the waves in order.
#include "bi_ffn.h"
#include "bi_plan.h"
#include "bi_tile.h"

namespace bi {

// P chunks of eight values as they lie in memory.
template <bool BF, int P>
struct RowRaw {
    static constexpr int V = BF ? 1 : 2;
    u32x4 v[P * V];

    // thread t of T: chunks t, t + T, ...; zero past the row's end
    template <int T>
    __device__ __forceinline__ void load(const void* x, int64_t at, int t, int chunks)
    {
        const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const unsigned char*>(x) + at * (BF ? 2 : 4));
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i * V + j] = u32x4{0u, 0u, 0u, 0u};
                if (i * T + t < chunks)
                    v[i * V + j] = p[(i * T + t) * V + j];
            }
    }
    __device__ __forceinline__ float at(int i, int j) const     // value j of chunk i
    {
        if constexpr (BF) {
            const uint32_t u = v[i][j >> 1];
            return __uint_as_float(j & 1 ? u & 0xffff0000u : u << 16);
        } else {
            return __uint_as_float(v[2 * i + (j >> 2)][j & 3]);
        }
    }
};

template <bool BF>
__device__ __forceinline__ void store8(void* y, int64_t at, const float (&v)[8])
{
    if constexpr (BF) {
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(y) + at) =
            u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    } else {
        f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(y) + at);
        p[0] = f32x4{v[0], v[1], v[2], v[3]};
        p[1] = f32x4{v[4], v[5], v[6], v[7]};
    }
}

// Sums of K values over teams of T threads.  Two buffers in turn: a wave that
// writes one again has passed the barrier behind its last readers.
template <int T, int TEAMS, int K>
struct TeamSum {
    static constexpr int W = T / 64;
    float (*buf)[TEAMS][W][K];
    int turn = 0;

    __device__ __forceinline__ void operator()(float (&s)[K])
    {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
#pragma unroll
            for (int k = 0; k < K; ++k)
                s[k] += __shfl_xor(s[k], d);
        if constexpr (W > 1) {
            const int team = threadIdx.x / T, wave = threadIdx.x % T / 64;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    buf[turn][team][wave][k] = s[k];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k)
                s[k] = buf[turn][team][0][k];
#pragma unroll
            for (int w = 1; w < W; ++w)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    s[k] += buf[turn][team][w][k];
            turn ^= 1;
        }
    }
};

// Squares are added scaled by 1 / kNormMaxH, a power of two: their sum overflows
// only where the variance itself does.
constexpr float kSquareScale = 1.0f / 16384.0f;
static_assert(kNormMaxH == 16384, "the scale");

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

template <bool XB, bool YB, int T, int P, int TEAMS>
__global__ __launch_bounds__(T * TEAMS) void k_layer_norm(NormArgs p)
{
    __shared__ float buf[2][TEAMS][T / 64][1];
    TeamSum<T, TEAMS, 1> sum{buf};
    const int t = threadIdx.x % T, team = threadIdx.x / T, chunks = p.H / 8;
    float w[P][8], b[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const bool in = i * T + t < chunks;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[i][j] = p.w && in ? p.w[(i * T + t) * 8 + j] : 1.f;
            b[i][j] = p.b && in ? p.b[(i * T + t) * 8 + j] : 0.f;
        }
    }
    const float h = (float)p.H;
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    int64_t m = (int64_t)blockIdx.x * TEAMS + team;
    RowRaw<XB, P> cur, next;
    cur.template load<T>(p.x, min(m, p.M - 1) * p.ldx, t, chunks);
    for (int64_t m0 = (int64_t)blockIdx.x * TEAMS; m0 < p.M; m0 += step, m += step) {
        if (m0 + step < p.M)
            next.template load<T>(p.x, min(m + step, p.M - 1) * p.ldx, t, chunks);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[0] += cur.at(i, j);
        sum(s);
        const float mean = s[0] / h;
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (i * T + t < chunks) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = cur.at(i, j) - mean;
                    q[0] += d * (d * kSquareScale);
                }
            }
        sum(q);
        const float rstd = 1.f / sqrtf(q[0] / (h * kSquareScale) + p.eps);
        if (m < p.M) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (i * T + t < chunks) {
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[j] = (cur.at(i, j) - mean) * rstd * w[i][j] + b[i][j];
                    store8<YB>(p.y, m * p.ldy + (i * T + t) * 8, o);
                }
            if (t == 0) {
                if (p.mean)
                    p.mean[m] = mean;
                if (p.rstd)
                    p.rstd[m] = rstd;
            }
        }
        cur = next;
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
    int64_t M;
    int H;
};

template <bool DB, bool XB, int T, int P, int TEAMS>
__global__ __launch_bounds__(T * TEAMS) void k_layer_norm_bwd(NormBwdArgs p)
{
    __shared__ float buf[2][TEAMS][T / 64][2];
    __shared__ float fold[TEAMS > 1 ? T * 8 * P : 1];
    TeamSum<T, TEAMS, 2> sum{buf};
    const int t = threadIdx.x % T, team = threadIdx.x / T, chunks = p.H / 8;
    float w[P][8], dw[P][8] = {}, db[P][8] = {};
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const bool in = i * T + t < chunks;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[i][j] = p.w && in ? p.w[(i * T + t) * 8 + j] : 1.f;
    }
    const float h = (float)p.H;
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    int64_t m = (int64_t)blockIdx.x * TEAMS + team;
    RowRaw<XB, P> x, xn;
    RowRaw<DB, P> d, dn;
    float mean, rstd, meann, rstdn;
    x.template load<T>(p.x, min(m, p.M - 1) * p.ldx, t, chunks);
    d.template load<T>(p.dy, min(m, p.M - 1) * p.lddy, t, chunks);
    mean = p.mean[min(m, p.M - 1)];
    rstd = p.rstd[min(m, p.M - 1)];
    for (int64_t m0 = (int64_t)blockIdx.x * TEAMS; m0 < p.M; m0 += step, m += step) {
        if (m0 + step < p.M) {
            const int64_t to = min(m + step, p.M - 1);
            xn.template load<T>(p.x, to * p.ldx, t, chunks);
            dn.template load<T>(p.dy, to * p.lddy, t, chunks);
            meann = p.mean[to];
            rstdn = p.rstd[to];
        }
        const bool live = m < p.M;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (i * T + t < chunks) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dy = d.at(i, j), n = (x.at(i, j) - mean) * rstd, g = dy * w[i][j];
                    s[0] += g;
                    s[1] += g * n;
                    if (live) {
                        dw[i][j] += dy * n;
                        db[i][j] += dy;
                    }
                }
            }
        if (p.dx) {
            sum(s);
            const float c0 = s[0] / h, c1 = s[1] / h;
            if (live) {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (i * T + t < chunks) {
                        float o[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float n = (x.at(i, j) - mean) * rstd;
                            o[j] = rstd * (d.at(i, j) * w[i][j] - (c0 + n * c1));
                        }
                        store8<XB>(p.dx, m * p.lddx + (i * T + t) * 8, o);
                    }
            }
        }
        x = xn;
        d = dn;
        mean = meann;
        rstd = rstdn;
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
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (i * T + t < chunks)
                    store8<false>(p.part, ((int64_t)blockIdx.x * 2 + which) * p.H + (i * T + t) * 8, a[i]);
        }
    };
    out(dw, 0);
    out(db, 1);
}

// dw and db from G partials: a workgroup takes 64 of the 2 H columns, 16 threads
// of four columns by 16 slices of the partials; a slice's partials are added in
// order, then the slices.
__global__ __launch_bounds__(256) void k_layer_norm_fold(const float* __restrict__ part, float* __restrict__ dw,
                                                         float* __restrict__ db, int G, int H)
{
    __shared__ f32x4 acc[16][16];
    const int cl = threadIdx.x & 15, sl = threadIdx.x >> 4;
    const int c = blockIdx.x * 64 + cl * 4;
    f32x4 a = {0.f, 0.f, 0.f, 0.f};
    if (c < 2 * H) {
        const int per = (G + 15) / 16, to = min((sl + 1) * per, G);
#pragma unroll 4
        for (int k = sl * per; k < to; ++k)
            a += *reinterpret_cast<const f32x4*>(part + (int64_t)k * 2 * H + c);
    }
    acc[sl][cl] = a;
    __syncthreads();
    if (sl == 0 && c < 2 * H) {
        for (int k = 1; k < 16; ++k)
            a += acc[k][cl];
        float* to = c < H ? dw : db;
        if (to)
            *reinterpret_cast<f32x4*>(to + (c < H ? c : c - H)) = a;
    }
}

// f(T, P, rows per workgroup) of a row length
template <typename F>
static void norm_shape(int64_t H, F f)
{
    using std::integral_constant;
    if (H <= 512)
        f(integral_constant<int, 64>{}, integral_constant<int, 1>{}, integral_constant<int, 4>{});
    else if (H <= 2048)
        f(integral_constant<int, 256>{}, integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (H <= 4096)
        f(integral_constant<int, 256>{}, integral_constant<int, 2>{}, integral_constant<int, 1>{});
    else if (H <= 8192)
        f(integral_constant<int, 512>{}, integral_constant<int, 2>{}, integral_constant<int, 1>{});
    else
        f(integral_constant<int, 1024>{}, integral_constant<int, 2>{}, integral_constant<int, 1>{});
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
        norm_shape(H, [&](auto T, auto P, auto R) {
            const int64_t groups = (M + R - 1) / R, most = (int64_t)device_cu_count() * (2048 / (T * R));
            k_layer_norm<decltype(xb)::value, decltype(yb)::value, T, P, R>
                <<<(unsigned)(groups < most ? groups : most), T * R, 0, s>>>(p);
        });
    });
    return hipGetLastError();
}

// Workgroups of the backward pass, each with a partial of dw and db.
static int64_t bwd_groups(int64_t M, int64_t rows)
{
    const int64_t groups = (M + rows - 1) / rows;
    return groups < 256 ? groups : 256;
}

static int64_t bwd_rows(int64_t H)
{
    return H <= 512 ? 16 : H <= 4096 ? 4 : H <= 8192 ? 2 : 1;
}

size_t layer_norm_bwd_ws(int64_t M, int64_t H) { return (size_t)bwd_groups(M, bwd_rows(H)) * 2 * (size_t)H * 4; }

hipError_t launch_layer_norm_bwd(const void* dy, int dy_bf16, int64_t lddy, const void* x, int x_bf16, int64_t ldx,
                                 const float* mean, const float* rstd, const float* w, void* dx, int64_t lddx, float* dw, float* db,
                                 int64_t M, int64_t H, void* ws, hipStream_t s)
{
    const bool sums = dw || db;
    const NormBwdArgs p{dy, lddy, x, ldx, mean, rstd, w, dx, lddx, sums ? reinterpret_cast<float*>(ws) : nullptr, M, (int)H};
    int64_t groups = 0;
    two_types(dy_bf16, x_bf16, [&](auto yb, auto xb) {
        norm_shape(H, [&](auto T, auto P, auto) {
            constexpr int R = 1024 / T;
            groups = bwd_groups(M, R);
            k_layer_norm_bwd<decltype(yb)::value, decltype(xb)::value, T, P, R><<<(unsigned)groups, 1024, 0, s>>>(p);
        });
    });
    if (sums)
        k_layer_norm_fold<<<(unsigned)((2 * H + 63) / 64), 256, 0, s>>>(p.part, dw, db, (int)groups, (int)H);
    return hipGetLastError();
}

}  // namespace bi
