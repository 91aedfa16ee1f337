// bi_gated.hip -- the gated linear layer, y = act(x Wg^T) * (x Wu^T), and the
// elementwise part of its backward pass.
#include "bi_ffn.h"
#include "bi_plan.h"
#include "bi_tile.h"
#include "bi_tile_rule.h"

namespace bi {

bool gated_fits(int64_t ldx, int64_t ldw, int64_t M, int64_t I, int64_t H)
{
    // per-lane byte offsets inside a tile's operands are 32 bits wide (the up
    // rows lie I rows behind the gate rows), and the grid is one dimension
    const int64_t lim = int64_t(1) << 32;
    return 255 * ldx * 2 + H * 2 < lim && (I + 255) * ldw * 2 + H * 2 < lim && H < (int64_t(1) << 29) &&
           ((M + 15) / 16) * ((I + 7) / 8) < (int64_t(1) << 31);
}

template <int BM, int BN, int WM, int WN, int KB, int R, int NL_>
struct GatedShape {
    using C = TileCfg<BM, BN, WM, WN, KB, R, false, false, kBf16, kEpiGated>;
    static constexpr int NL = NL_;
};

template <typename S>
static hipError_t gated_tile(TileArgs a, hipStream_t s)
{
    using C = typename S::C;
    a.tiles_m = (a.M + C::BM - 1) / C::BM;
    a.tiles_n = (a.N + C::kOutN - 1) / C::kOutN;
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

// bm x (weight rows / 2); the costs are explained in bi_tile_rule.h
static const TileShape kGatedShapes[] = {
    {16, 8, 0.67f, 0.037f, 1.10f}, {16, 16, 0.29f, 0.063f, 1.10f}, {32, 16, 0.64f, 0.072f, 1.10f}, {64, 16, 0.90f, 0.088f, 0.f},
    {128, 32, 0.65f, 0.204f, 0.f}, {128, 64, 0.72f, 0.277f, 0.f},  {256, 128, 1.87f, 0.688f, 0.f},
};

static int gated_pick(int64_t M, int64_t I, int64_t H)
{
    return pick_tile(kGatedShapes, 7, M, I, (H + 31) / 32, false, device_cu_count());
}

// f of the shape at an index of kGatedShapes
template <typename F>
static auto gated_shape(int i, F f)
{
    switch (i) {
    case 0: return f(GatedShape<16, 16, 1, 1, 8, 4, 4>{});
    case 1: return f(GatedShape<16, 32, 1, 1, 4, 4, 4>{});
    case 2: return f(GatedShape<32, 32, 2, 1, 4, 4, 4>{});
    case 3: return f(GatedShape<64, 32, 4, 1, 4, 4, 4>{});
    case 4: return f(GatedShape<128, 64, 4, 1, 2, 4, 0>{});
    case 5: return f(GatedShape<128, 128, 4, 2, 2, 4, 0>{});
    default: return f(GatedShape<256, 256, 4, 2, 2, 2, 0>{});
    }
}

hipError_t launch_gated(const uint16_t* x, int64_t ldx, const uint16_t* w13, int64_t ldw, int gate, uint16_t* y,
                        int64_t ldy, uint16_t* h, int64_t ldh, int64_t M, int64_t I, int64_t H, hipStream_t s)
{
    TileArgs a{};
    a.a = reinterpret_cast<const unsigned char*>(x);
    a.b = reinterpret_cast<const unsigned char*>(w13);
    a.lda = ldx * 2;
    a.ldb = ldw * 2;
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = 1;
    a.h = h;
    a.ldh = ldh;
    a.gate = gate == BI_GATE_SILU ? kGateSilu : kGateGeluTanh;
    a.M = (int)M;
    a.N = (int)I;
    a.K = H;
    return gated_shape(gated_pick(M, I, H), [&](auto shape) { return gated_tile<decltype(shape)>(a, s); });
}

TileInfo gated_tile_info(int64_t M, int64_t I, int64_t H)
{
    const int i = gated_pick(M, I, H);
    return gated_shape(i, [i](auto shape) { return tile_info<decltype(shape)>(i); });
}

// One thread per eight columns of a row: dy, the gate half and the up half of
// h in, both halves of dh out.  With s = sigma(z(g)), act = g s:
//   silu  act' = s + g s (1 - s)
//   gelu  act' = s + g s (1 - s) z'(g),  z = c (g + b g^3)
// g^2 in z' is held below 1e30: s or 1 - s is exactly 0 long before, and zero
// times an overflowed z' would be NaN.
// dh is rounded to bf16 once: it is the matrix instructions' operand in both
// products that follow, where a wider one would double their work (dx and dw are
// off by 0.0023 of their size instead of the 0.0017 of their own rounding).
__global__ __launch_bounds__(256) void k_gate_bwd(const uint16_t* __restrict__ dy, int64_t lddy,
                                                  const uint16_t* __restrict__ h, int64_t ldh, int gate,
                                                  uint16_t* __restrict__ dh, int64_t lddh, int64_t M, int I)
{
    const uint32_t cpr = (uint32_t)I / 8;
    const int64_t total = M * cpr;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / cpr;
        const int c = (int)(i - m * cpr) * 8;
        const u32x4 dv = *reinterpret_cast<const u32x4*>(dy + m * lddy + c);
        const u32x4 gv = *reinterpret_cast<const u32x4*>(h + m * ldh + c);
        const u32x4 uv = *reinterpret_cast<const u32x4*>(h + m * ldh + I + c);
        u32x4 og, ou;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float rg[2], ru[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float d = __uint_as_float(q ? dv[j] & 0xffff0000u : dv[j] << 16);
                const float gg = __uint_as_float(q ? gv[j] & 0xffff0000u : gv[j] << 16);
                const float uu = __uint_as_float(q ? uv[j] & 0xffff0000u : uv[j] << 16);
                const float s8 = gate_sigma8(gg, gate), sg = s8 * kSigmaScale;
                const float dz = gate == kGateSilu ? 1.0f : kGeluC2 * (1.0f + 3.0f * kGeluB * fminf(gg * gg, 1e30f));
                const float act = gg * kSigmaScale * s8;
                rg[q] = d * uu * (sg + act * (1.0f - sg) * dz);
                ru[q] = d * act;
            }
            og[j] = pack_bf16(rg[0], rg[1]);
            ou[j] = pack_bf16(ru[0], ru[1]);
        }
        *reinterpret_cast<u32x4*>(dh + m * lddh + c) = og;
        *reinterpret_cast<u32x4*>(dh + m * lddh + I + c) = ou;
    }
}

hipError_t launch_gate_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* h, int64_t ldh, int gate, uint16_t* dh,
                           int64_t lddh, int64_t M, int64_t I, hipStream_t s)
{
    const int64_t blocks = (M * (I / 8) + 255) / 256;
    const int64_t grid = blocks < 65536 ? blocks : 65536;
    k_gate_bwd<<<(unsigned)grid, 256, 0, s>>>(dy, lddy, h, ldh, gate == BI_GATE_SILU ? kGateSilu : kGateGeluTanh, dh,
                                              lddh, M, (int)I);
    return hipGetLastError();
}

}  // namespace bi
