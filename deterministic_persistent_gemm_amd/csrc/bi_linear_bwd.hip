// bi_linear_bwd.hip -- the products of the backward passes: dx = dy W (the
// weight read by columns), dw = dy^T x (both operands read by columns) and the
// column sums of dy.
#include "bi_ffn.h"
#include "bi_tile.h"

namespace bi {

bool linear_bwd_fits(int64_t lddy, int64_t ldx, int64_t ldw, int64_t M, int64_t N, int64_t K)
{
    const int64_t lim = int64_t(1) << 32;
    return 255 * lddy * 2 + N * 2 < lim && 32 * lddy * 2 + 512 < lim && 32 * ldw * 2 + 512 < lim &&
           32 * ldx * 2 + 512 < lim && N < (int64_t(1) << 29) && ((M + 15) / 16) * ((K + 15) / 16) < (int64_t(1) << 31) &&
           ((N + 15) / 16) * ((K + 15) / 16) < (int64_t(1) << 31);
}

template <int BM, int BN, int WM, int WN, int KB, int R, bool CA>
static hipError_t bwd_tile(TileArgs a, hipStream_t s)
{
    using C = TileCfg<BM, BN, WM, WN, KB, R, CA, true, false, kEpiLinear>;
    a.tiles_m = (a.M + BM - 1) / BM;
    a.tiles_n = (a.N + BN - 1) / BN;
    k_tile<C><<<(unsigned)(a.tiles_m * a.tiles_n), C::NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_dgrad(const uint16_t* dy, int64_t lddy, const uint16_t* w, int64_t ldw, uint16_t* dx, int64_t lddx,
                        int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    TileArgs a{};
    a.a = reinterpret_cast<const unsigned char*>(dy);
    a.b = reinterpret_cast<const unsigned char*>(w);
    a.lda = lddy * 2;
    a.ldb = ldw * 2;
    a.y = dx;
    a.ldy = lddx;
    a.y_bf16 = 1;
    a.M = (int)M;
    a.N = (int)K;
    a.K = N;
    if (M > 512)
        return bwd_tile<256, 256, 4, 2, 1, 4, false>(a, s);
    return bwd_tile<64, 64, 4, 1, 2, 4, false>(a, s);
}

hipError_t launch_wgrad(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, void* dw, int dw_bf16,
                        int64_t lddw, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    TileArgs a{};
    a.a = reinterpret_cast<const unsigned char*>(dy);
    a.b = reinterpret_cast<const unsigned char*>(x);
    a.lda = lddy * 2;
    a.ldb = ldx * 2;
    a.y = dw;
    a.ldy = lddw;
    a.y_bf16 = dw_bf16;
    a.M = (int)N;
    a.N = (int)K;
    a.K = M;
    if (M > 512)
        return bwd_tile<256, 256, 4, 2, 1, 4, true>(a, s);
    return bwd_tile<64, 64, 4, 1, 2, 4, true>(a, s);
}

// Column sums: a workgroup takes 64 columns and a contiguous part of the rows;
// thread (row lane, column group of 8) adds its rows in ascending order, the 32
// row lanes are added in order, and a second launch adds the parts in order.
// The split follows from (M, N) alone, so the bits repeat.
constexpr int kSumCols = 64, kSumLanes = 32;

static int64_t colsum_parts(int64_t M, int64_t N)
{
    const int64_t groups = (N + kSumCols - 1) / kSumCols;
    int64_t parts = (512 + groups - 1) / groups;
    const int64_t most = (M + 4 * kSumLanes - 1) / (4 * kSumLanes);
    parts = parts < most ? parts : most;
    return parts < 1 ? 1 : parts;
}

size_t colsum_ws_bytes(int64_t M, int64_t N)
{
    const int64_t parts = colsum_parts(M, N);
    return parts > 1 ? (size_t)parts * (size_t)N * 4 : 0;
}

__global__ __launch_bounds__(256) void k_colsum(const uint16_t* __restrict__ dy, int64_t lddy, float* __restrict__ out,
                                                int64_t M, int N, int64_t rows_per)
{
    __shared__ float part[kSumLanes][kSumCols + 1];
    const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
    const int c = blockIdx.x * kSumCols + cg * 8;
    const int64_t lo = (int64_t)blockIdx.y * rows_per;
    const int64_t hi = lo + rows_per < M ? lo + rows_per : M;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < N) {
        for (int64_t m = lo + rl; m < hi; m += kSumLanes) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(dy + m * lddy + c);
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
    const int col = blockIdx.x * kSumCols + threadIdx.x;
    if (threadIdx.x < kSumCols && col < N) {
        float t = part[0][threadIdx.x];
        for (int l = 1; l < kSumLanes; ++l)
            t += part[l][threadIdx.x];
        out[(int64_t)blockIdx.y * N + col] = t;
    }
}

__global__ __launch_bounds__(256) void k_colsum_fold(const float* __restrict__ parts, float* __restrict__ db, int N,
                                                     int nparts)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= N)
        return;
    float t = parts[c];
    for (int i = 1; i < nparts; ++i)
        t += parts[(int64_t)i * N + c];
    db[c] = t;
}

hipError_t launch_colsum(const uint16_t* dy, int64_t lddy, float* db, int64_t M, int64_t N, void* ws, hipStream_t s)
{
    const int64_t parts = colsum_parts(M, N);
    const int64_t rows_per = (M + parts - 1) / parts;
    float* out = parts > 1 ? reinterpret_cast<float*>(ws) : db;
    k_colsum<<<dim3((unsigned)((N + kSumCols - 1) / kSumCols), (unsigned)parts), 256, 0, s>>>(dy, lddy, out, M, (int)N,
                                                                                          rows_per);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1)
        return e;
    k_colsum_fold<<<(unsigned)((N + 255) / 256), 256, 0, s>>>(out, db, (int)N, (int)parts);
    return hipGetLastError();
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
