// bi_int8.hip -- 8-bit integer operands: quantisation of rows and the product of
// two quantised operands.
//
// A row x is kept as codes q, integers in [-127, 127], and one fp32 scale s:
//   s = max(max|x| * (1/127), 2^-126),  q = x / s to the nearest integer, ties to even
// with 1/127 as fp32 holds it.  That is 2^-28 below 1/127, so s is the rounded quotient
// max|x| / 127 or the fp32 number next below (6 of bf16's 128 mantissas); a code differs
// from the quotient's only where x / s lies within 127 * 2^-23 of halfway.
// The product adds code products in 32-bit integers, which rounds nothing, so
// any order of addition gives the same bits.
#include "bi_ffn.h"
#include "bi_plan.h"
#include "bi_rows.h"
#include "bi_tile.h"
#include "bi_tile_rule.h"

namespace bi {

// x / s to the nearest integer, ties to even, for |x / s| < 127.5.  x times the
// reciprocal may round to the wrong side of a halfway point, or onto one; the
// sign of x - (q +- 1/2) s, which a fused multiply-add gives exactly, says where
// x lies.
__device__ __forceinline__ int code_of(float x, float s, float inv)
{
    const float q = rintf(x * inv);
    const int i = (int)q;
    const float above = __builtin_fmaf(-(q + 0.5f), s, x), below = __builtin_fmaf(-(q - 0.5f), s, x);
    const bool odd = i & 1;
    return above > 0.f || (above == 0.f && odd) ? i + 1 : below < 0.f || (below == 0.f && odd) ? i - 1 : i;
}

// The low bytes of a .. d.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    return lo | hi;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The codes of chunk i.  Adding 1.5 * 2^23 to x inv rounds it to the nearest integer,
// which is then in the sum's low bits.  x inv is within 127.5 * 2^-24 of x / s, so that
// integer is the code unless one of the eight lies that near to a halfway point; only
// then (rows of random values: one chunk in 6000) are the sides decided one by one.
template <bool BF, int P>
__device__ __forceinline__ u32x2 codes_of(const RowRaw<BF, P>& r, int i, float s, float inv)
{
    constexpr float kRound = 12582912.0f;
    uint32_t k[8];
    float off = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = r.at(i, j), t = __builtin_fmaf(x, inv, kRound);
        off = fmaxf(off, fabsf(__builtin_fmaf(x, inv, kRound - t)));
        k[j] = __float_as_uint(t);
    }
    if (off > 0.49999f) {
        // tiny rows are scaled up by a power of two, so that no half step is subnormal
        const float up = s < 8.67361738e-19f ? 1.84467441e19f : 1.0f;      // 2^-60, 2^64
        const float s1 = s * up, inv1 = 1.0f / s1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            k[j] = (uint32_t)code_of(r.at(i, j) * up, s1, inv1);
    }
    return u32x2{pack4(k[0], k[1], k[2], k[3]), pack4(k[4], k[5], k[6], k[7])};
}

// The largest magnitude of a thread's values by bit pattern, so that NaN and
// infinity win.
template <bool BF, int P>
__device__ __forceinline__ uint32_t top_of(const RowRaw<BF, P>& r)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, __float_as_uint(r.at(i, j)) & 0x7fffffffu);
    return top;
}

// A team of T threads per row, whose first P chunks of 8 values per thread stay in
// registers between the search for the largest and the codes; longer rows are read
// again.  The next row is on its way meanwhile.  Bound by latency for few rows (3.8 us
// for 16 of 4096); 4096 rows of 4096 bf16 take 16.5 us (50 MB, 3.0 TB/s), since the launch
// gives two rows to each of 2048 workgroups, whose start and end cost as much as memory,
// fp32 19.0 (4.4 TB/s), 4096 rows of 8192 fp32 33.3 (5.0 TB/s).
template <bool BF, int T, int P>
__global__ __launch_bounds__(256) void k_quantize_int8(const void* __restrict__ x, int64_t ldx, uint8_t* __restrict__ q,
                                                       int64_t ldq, float* __restrict__ sc, int64_t rows, int chunks)
{
    constexpr int TEAMS = 256 / T, W = T / 64;
    __shared__ uint32_t tops[2][TEAMS][W];
    const int t = threadIdx.x % T, team = (int)uniform(threadIdx.x / T);
    int turn = 0;
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    int64_t m = (int64_t)blockIdx.x * TEAMS + team;
    RowRaw<BF, P> cur, next;
    cur.template load<T>(x, min(m, rows - 1) * ldx, t, chunks);
    for (int64_t m0 = (int64_t)blockIdx.x * TEAMS; m0 < rows; m0 += step, m += step) {
        next.template load<T>(x, min(m + step, rows - 1) * ldx, t, chunks);
        const int64_t at = min(m, rows - 1);
        uint32_t top = top_of(cur);
        for (int c = P * T + t; c < chunks; c += T) {
            RowRaw<BF, 1> more;
            more.template load<0>(x, at * ldx, c, chunks);
            top = max(top, top_of(more));
        }
        top = wave_max(top);
        if constexpr (W > 1) {
            if ((t & 63) == 0)
                tops[turn][team][t >> 6] = top;
            wg_barrier_reads_done();
#pragma unroll
            for (int w = 0; w < W; ++w)
                top = max(top, tops[turn][team][w]);
            turn ^= 1;
        }
        const bool finite = top < 0x7f800000u;
        const float s = finite ? fmaxf(__uint_as_float(top) * (1.0f / 127.0f), 1.17549435e-38f) : __uint_as_float(0x7fc00000u);
        const float inv = 1.0f / s;
        auto codes = [&](const auto& r, int i) __attribute__((always_inline)) {
            const u32x2 v = codes_of(r, i, s, inv);
            return finite ? v : u32x2{0u, 0u};
        };
        u32x2 out[P];
#pragma unroll
        for (int i = 0; i < P; ++i)
            out[i] = codes(cur, i);
        cur = next;
        __builtin_amdgcn_sched_barrier(0);
        if (m < rows) {
            uint8_t* to = q + m * ldq;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (i * T + t < chunks)
                    *reinterpret_cast<u32x2*>(to + (i * T + t) * 8) = out[i];
            for (int c = P * T + t; c < chunks; c += T) {
                RowRaw<BF, 1> more;
                more.template load<0>(x, m * ldx, c, chunks);
                *reinterpret_cast<u32x2*>(to + (int64_t)c * 8) = codes(more, 0);
            }
            if (t == 0)
                sc[m] = s;
        }
    }
}

template <bool BF, int T, int P>
static void quantize_shape(const void* x, int64_t ldx, uint8_t* q, int64_t ldq, float* sc, int64_t rows, int64_t K, hipStream_t s)
{
    constexpr int R = 256 / T;
    const int64_t groups = (rows + R - 1) / R, most = (int64_t)device_cu_count() * 8;
    k_quantize_int8<BF, T, P><<<(unsigned)(groups < most ? groups : most), 256, 0, s>>>(x, ldx, q, ldq, sc, rows, (int)(K / 8));
}

// A wave to a row while the row leaves most of a workgroup without work: 32768 rows of
// 768 22.0 us (a workgroup 41.3), 8192 of 512 6.0 (11.4); 64 of 2048 5.7 (3.3).
template <bool BF>
static void quantize_rows(const void* x, int64_t ldx, uint8_t* q, int64_t ldq, float* sc, int64_t rows, int64_t K, hipStream_t s)
{
    if (K <= 512)
        quantize_shape<BF, 64, 1>(x, ldx, q, ldq, sc, rows, K, s);
    else if (K <= 1024)
        quantize_shape<BF, 64, 2>(x, ldx, q, ldq, sc, rows, K, s);
    else if (K <= 2048)
        quantize_shape<BF, 256, 1>(x, ldx, q, ldq, sc, rows, K, s);
    else if (K <= 4096)
        quantize_shape<BF, 256, 2>(x, ldx, q, ldq, sc, rows, K, s);
    else
        quantize_shape<BF, 256, 4>(x, ldx, q, ldq, sc, rows, K, s);
}

hipError_t launch_quantize_int8(const void* x, int x_bf16, int64_t ldx, int8_t* q, int64_t ldq, float* sc, int64_t rows,
                                int64_t K, hipStream_t s)
{
    uint8_t* u = reinterpret_cast<uint8_t*>(q);
    if (x_bf16)
        quantize_rows<true>(x, ldx, u, ldq, sc, rows, K, s);
    else
        quantize_rows<false>(x, ldx, u, ldq, sc, rows, K, s);
    return hipGetLastError();
}

// ------------------------------------------------------------------- product

bool int8_fits(int64_t ldx, int64_t ldw, int64_t M, int64_t N, int64_t K)
{
    const int64_t lim = int64_t(1) << 32;
    return 255 * ldx + K < lim && 255 * ldw + K < lim && K <= kInt8MaxK && ((M + 15) / 16) * ((N + 15) / 16) < (int64_t(1) << 31);
}

template <int BM, int BN, int WM, int WN, int KB, int R, int NL_>
struct Int8Shape {
    using C = TileCfg<BM, BN, WM, WN, KB, R, false, false, kInt8, kEpiLinear>;
    static constexpr int NL = NL_;
};

// Costs as in bi_tile_rule.h (a slice is 64 k), fitted to timings of 320 problems drawn
// over M 1 .. 4096, widths 128 .. 12288 and k 256 .. 8192: the shapes chosen take 1.005
// times the fastest one's time on average (fitted to one half of them, 1.013 on the
// other).  Longer k is underpriced (M 256, N 4096, K 12288 on 128 tiles of 64 x 128: 49 us
// taken, 26 estimated).  128 x 128 is there twice: with four stages in its ring, one workgroup to a
// compute unit, and in turns with two, two workgroups.
static const TileShape kInt8Shapes[] = {
    {16, 16, 1.75f, 0.034f, 1.08f}, {16, 32, 1.70f, 0.042f, 1.03f}, {32, 32, 1.71f, 0.047f, 1.38f}, {32, 64, 1.89f, 0.092f, 1.05f},
    {64, 64, 1.90f, 0.102f, 1.14f}, {64, 128, 2.57f, 0.114f, 0.f},  {128, 128, 2.63f, 0.244f, 0.f}, {128, 128, 2.46f, 0.291f, 0.91f},
    {256, 256, 7.18f, 0.670f, 0.f},
};
constexpr int kNumInt8Shapes = 9;

static int int8_pick(int64_t M, int64_t N, int64_t K, int y_bf16)
{
    return pick_tile(kInt8Shapes, kNumInt8Shapes, M, N, (K + 63) / 64, !y_bf16, device_cu_count());
}

// f of the shape at an index of kInt8Shapes
template <typename F>
static auto int8_shape(int i, F f)
{
    switch (i) {
    case 0: return f(Int8Shape<16, 16, 1, 1, 8, 4, 4>{});
    case 1: return f(Int8Shape<16, 32, 1, 1, 4, 4, 4>{});
    case 2: return f(Int8Shape<32, 32, 2, 1, 4, 4, 4>{});
    case 3: return f(Int8Shape<32, 64, 2, 2, 4, 3, 4>{});
    case 4: return f(Int8Shape<64, 64, 2, 2, 2, 4, 4>{});
    case 5: return f(Int8Shape<64, 128, 2, 2, 2, 3, 4>{});
    case 6: return f(Int8Shape<128, 128, 4, 2, 2, 4, 0>{});
    case 7: return f(Int8Shape<128, 128, 4, 2, 2, 2, 0>{});
    default: return f(Int8Shape<256, 256, 4, 2, 2, 2, 0>{});
    }
}

// v_mfma_i32_16x16x64_i8; scales and bias are applied to the sums as y is stored.  16 rows
// through 4096 x 4096 take 6.3 us: the weight's 16.8 MB at the rate that a cold read of
// that length has.  4096 x 12288 x 4096 takes 171 to 174 us on codes of normally distributed
// values (2.4 POP/s), 176 to 178 on codes that are all equally likely, 168 on the same
// operands again and again: a stage of the 256 x 256
// tiles brings the same bytes as in bf16 for twice the products, and three rounds of them
// pay 7 us each for first loads and stores.  (The same tiles one after the other, a
// workgroup to a compute unit for the whole call: 174.6 us where these took 170.7.)
template <typename S>
__global__ __launch_bounds__((S::C::NW + S::NL) * 64) void k_int8(TileArgs p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char ring[S::C::kRing];
    int tn;
    const int tm = tile_of((int)blockIdx.x, p.tiles_m, p.tiles_n, tn);
    tile_any<S>(p, ring, tm, tn);
}

template <typename S>
static hipError_t int8_tile(TileArgs a, hipStream_t s)
{
    using C = typename S::C;
    a.tiles_m = (a.M + C::BM - 1) / C::BM;
    a.tiles_n = (a.N + C::BN - 1) / C::BN;
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    if (!grid_ok(tiles))
        return hipErrorInvalidConfiguration;
    k_int8<S><<<(unsigned)tiles, (C::NW + S::NL) * 64, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_int8_linear(const int8_t* xq, int64_t ldx, const float* xs, const int8_t* wq, int64_t ldw, const float* ws,
                              const float* bias, void* y, int y_bf16, int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    TileArgs a{};
    a.a = reinterpret_cast<const unsigned char*>(xq);
    a.b = reinterpret_cast<const unsigned char*>(wq);
    a.lda = ldx;
    a.ldb = ldw;
    a.sa = reinterpret_cast<const unsigned char*>(xs);
    a.sb = reinterpret_cast<const unsigned char*>(ws);
    a.bias = bias;
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = y_bf16;
    a.M = (int)M;
    a.N = (int)N;
    a.K = K;
    return int8_shape(int8_pick(M, N, K, y_bf16), [&](auto shape) { return int8_tile<decltype(shape)>(a, s); });
}

TileInfo int8_tile_info(int64_t M, int64_t N, int64_t K, int y_bf16)
{
    const int i = int8_pick(M, N, K, y_bf16);
    return int8_shape(i, [i](auto shape) { return tile_info<decltype(shape)>(i); });
}

}  // namespace bi
