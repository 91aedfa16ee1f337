// bi_mx.hip -- microscaled 4-bit floating point (OCP MX, MXFP4): quantisation,
// its inverse, and the product of two quantised operands.
//
// A block is 32 consecutive values of a row: 4-bit codes (sign, two exponent
// bits of bias 1, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte
// with the even element in the low half, and one scale byte s standing for
// 2^(s - 127); s = 255 makes the block NaN.
#include "bi_ffn.h"
#include "bi_plan.h"
#include "bi_tile.h"
#include "bi_tile_rule.h"

namespace bi {

// Four lanes share a block, eight values each.  The scale is the power of two
// of the block's largest magnitude over the largest code's (4 <= 6 < 8), so
// x / scale is below 8; it is formed exactly by v_ldexp and rounded to the
// nearest code, ties to even, saturating at 6, by the conversion instruction.
// A block with an infinity or a NaN gets the NaN scale.  Bound by memory: 2 or 4
// bytes read and 0.53 written per value.
template <bool BF16IN>
__global__ __launch_bounds__(256) void k_mx_quantize(const void* __restrict__ x, int64_t ldx, uint8_t* __restrict__ q,
                                                     int64_t ldq, uint8_t* __restrict__ sc, int64_t lds, int64_t total,
                                                     uint32_t cpr)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / cpr;
        const uint32_t c = (uint32_t)(i - m * cpr);
        float v[8];
        if constexpr (BF16IN) {
            const u32x4 u = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + m * ldx + c * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(u[j] << 16);
                v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        } else {
            const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(x) + m * ldx + c * 8);
            const f32x4 a = p[0], b = p[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = a[j];
                v[4 + j] = b[j];
            }
        }
        // the largest magnitude by bit pattern, so that NaN and infinity win
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1, 4));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2, 4));
        const int e = (int)(top >> 23);
        const int s = e == 255 ? 255 : max(e - 2, 0);
        uint32_t code = 0;
        if (s != 255) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = ldexpf(v[j], 127 - s);
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[0], v[1], 1.0f, 0);
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[2], v[3], 1.0f, 1);
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[4], v[5], 1.0f, 2);
            code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[6], v[7], 1.0f, 3);
        }
        *reinterpret_cast<uint32_t*>(q + m * ldq + c * 4) = code;
        if ((c & 3) == 0)
            sc[m * lds + (c >> 2)] = (uint8_t)s;
    }
}

template <bool BF16OUT>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ q, int64_t ldq,
                                                       const uint8_t* __restrict__ sc, int64_t lds, void* __restrict__ y,
                                                       int64_t ldy, int64_t total, uint32_t cpr)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / cpr;
        const uint32_t c = (uint32_t)(i - m * cpr);
        const uint32_t code = *reinterpret_cast<const uint32_t*>(q + m * ldq + c * 4);
        const int s = sc[m * lds + (c >> 2)];
        const f32x2 t[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 2),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 3)};
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = s == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(t[j >> 1][j & 1], s - 127);
        if constexpr (BF16OUT) {
            *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(y) + m * ldy + c * 8) =
                u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        } else {
            f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(y) + m * ldy + c * 8);
            p[0] = f32x4{v[0], v[1], v[2], v[3]};
            p[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
    }
}

static unsigned mx_grid(int64_t total)
{
    const int64_t blocks = (total + 255) / 256;
    return (unsigned)(blocks < 65536 ? blocks : 65536);
}

hipError_t launch_mx_quantize(const void* x, int x_bf16, int64_t ldx, uint8_t* q, int64_t ldq, uint8_t* sc, int64_t lds,
                              int64_t rows, int64_t K, hipStream_t s)
{
    const int64_t total = rows * (K / 8);
    if (x_bf16)
        k_mx_quantize<true><<<mx_grid(total), 256, 0, s>>>(x, ldx, q, ldq, sc, lds, total, (uint32_t)(K / 8));
    else
        k_mx_quantize<false><<<mx_grid(total), 256, 0, s>>>(x, ldx, q, ldq, sc, lds, total, (uint32_t)(K / 8));
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* q, int64_t ldq, const uint8_t* sc, int64_t lds, void* y, int y_bf16,
                                int64_t ldy, int64_t rows, int64_t K, hipStream_t s)
{
    const int64_t total = rows * (K / 8);
    if (y_bf16)
        k_mx_dequantize<true><<<mx_grid(total), 256, 0, s>>>(q, ldq, sc, lds, y, ldy, total, (uint32_t)(K / 8));
    else
        k_mx_dequantize<false><<<mx_grid(total), 256, 0, s>>>(q, ldq, sc, lds, y, ldy, total, (uint32_t)(K / 8));
    return hipGetLastError();
}

// ------------------------------------------------------------------- product

bool mx_fits(int64_t ldx, int64_t ldxs, int64_t ldw, int64_t ldws, int64_t M, int64_t N, int64_t K)
{
    const int64_t lim = int64_t(1) << 32;
    return 255 * ldx + K / 2 < lim && 255 * ldw + K / 2 < lim && 255 * ldxs + K / 32 < lim && 255 * ldws + K / 32 < lim &&
           K < (int64_t(1) << 30) && ((M + 15) / 16) * ((N + 15) / 16) < (int64_t(1) << 31);
}

template <int BM, int BN, int WM, int WN, int KB, int R, int NL_>
struct MxShape {
    using C = TileCfg<BM, BN, WM, WN, KB, R, false, false, true, kEpiLinear>;
    static constexpr int NL = NL_;
};

template <typename S>
static hipError_t mx_tile(TileArgs a, hipStream_t s)
{
    using C = typename S::C;
    a.tiles_m = (a.M + C::BM - 1) / C::BM;
    a.tiles_n = (a.N + C::BN - 1) / C::BN;
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    if (!grid_ok(tiles))
        return hipErrorInvalidConfiguration;
    const unsigned grid = (unsigned)tiles;
    if constexpr (S::NL > 0)
        k_stream<C, S::NL><<<grid, (C::NW + S::NL) * 64, 0, s>>>(a);
    else if constexpr (C::R == 2)
        k_turns<C><<<grid, C::NW * 64, 0, s>>>(a);
    else
        k_tile<C><<<grid, C::NW * 64, 0, s>>>(a);
    return hipGetLastError();
}

// the costs are explained in bi_tile_rule.h; a slice is 128 k
static const TileShape kMxShapes[] = {
    {16, 16, 0.87f, 0.032f, 1.10f}, {16, 32, 0.78f, 0.051f, 0.92f},   {32, 32, 0.97f, 0.068f, 1.10f},
    {64, 64, 1.26f, 0.162f, 1.00f}, {128, 128, 2.25f, 0.393f, 1.10f}, {256, 256, 5.08f, 0.961f, 0.f},
};

static int mx_pick(int64_t M, int64_t N, int64_t K, int y_bf16)
{
    return pick_tile(kMxShapes, 6, M, N, (K + 127) / 128, !y_bf16, device_cu_count());
}

// f of the shape at an index of kMxShapes
template <typename F>
static auto mx_shape(int i, F f)
{
    switch (i) {
    case 0: return f(MxShape<16, 16, 1, 1, 8, 4, 4>{});
    case 1: return f(MxShape<16, 32, 1, 1, 4, 4, 4>{});
    case 2: return f(MxShape<32, 32, 2, 1, 4, 4, 4>{});
    case 3: return f(MxShape<64, 64, 4, 1, 2, 4, 0>{});
    case 4: return f(MxShape<128, 128, 2, 2, 1, 4, 0>{});
    default: return f(MxShape<256, 256, 2, 4, 2, 2, 0>{});
    }
}

hipError_t launch_mx_linear(const uint8_t* xq, int64_t ldx, const uint8_t* xs, int64_t ldxs, const uint8_t* wq,
                            int64_t ldw, const uint8_t* wsc, int64_t ldws, const float* bias, void* y, int y_bf16,
                            int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t s)
{
    TileArgs a{};
    a.a = xq;
    a.b = wq;
    a.lda = ldx;
    a.ldb = ldw;
    a.sa = xs;
    a.sb = wsc;
    a.ldsa = ldxs;
    a.ldsb = ldws;
    a.bias = bias;
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = y_bf16;
    a.M = (int)M;
    a.N = (int)N;
    a.K = K;
    return mx_shape(mx_pick(M, N, K, y_bf16), [&](auto shape) { return mx_tile<decltype(shape)>(a, s); });
}

TileInfo mx_tile_info(int64_t M, int64_t N, int64_t K, int y_bf16)
{
    const int i = mx_pick(M, N, K, y_bf16);
    return mx_shape(i, [i](auto shape) { return tile_info<decltype(shape)>(i); });
}

}  // namespace bi
