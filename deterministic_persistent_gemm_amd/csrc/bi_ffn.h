// bi_ffn.h -- launchers of the feed-forward operators (host side): the gated
// linear layer, the backward passes, 4-bit quantisation and the 4-bit product.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "bi.h"

namespace bi {

// A launch may hold fewer than 2^32 threads, and a workgroup here has at most
// 512: launchers return hipErrorInvalidConfiguration for more workgroups.
inline bool grid_ok(int64_t groups) { return groups < (int64_t(1) << 23); }

// What bi_lab_ffn_tile reports of the tile shape a product takes.
struct TileInfo {
    int32_t shape, kernel, bm, bn, slice_k, stage_slices, ring_stages, scale_groups;
};

// bi_gated.hip
bool gated_fits(int64_t ldx, int64_t ldw, int64_t M, int64_t I, int64_t H);
hipError_t launch_gated(const uint16_t* x, int64_t ldx, const uint16_t* w13, int64_t ldw, int gate, uint16_t* y,
                        int64_t ldy, uint16_t* h, int64_t ldh, int64_t M, int64_t I, int64_t H, hipStream_t s);
TileInfo gated_tile_info(int64_t M, int64_t I, int64_t H);
// dh [M, 2 I] = [dy * h_u * act'(h_g), dy * act(h_g)]
hipError_t launch_gate_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* h, int64_t ldh, int gate, uint16_t* dh,
                           int64_t lddh, int64_t M, int64_t I, hipStream_t s);

// bi_linear_bwd.hip
// The launches of a backward pass: pairs of tile shapes, second -1 where one
// launch takes both products.
struct BwdPlan {
    int first, second;
};
// Plans the pass for the outputs wanted, M >= 1; false where the sizes or a
// launch's grid are out of range.
bool plan_linear_bwd(bool dx, bool dw, bool db, int dw_bf16, int64_t lddy, int64_t ldx, int64_t ldw, int64_t M, int64_t N,
                     int64_t K, BwdPlan* plan);
// dx [M, K] = dy [M, N] . w [N, K], dw [N, K] = dy^T . x [M, K] and db [N] = the
// sum of dy's rows, each where its output is not null
hipError_t launch_linear_bwd(const BwdPlan& plan, const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx,
                             const uint16_t* w, int64_t ldw, uint16_t* dx, int64_t lddx, void* dw, int dw_bf16, int64_t lddw,
                             float* db, int64_t M, int64_t N, int64_t K, hipStream_t s);
// The shape that dx (side 0) or dw (side 1) takes in a pass with both.
TileInfo linear_bwd_tile_info(int side, int dw_bf16, int64_t M, int64_t N, int64_t K);
// rows of `bytes` (a multiple of 4) at a pitch of `pitch` bytes, set to zero
hipError_t launch_zero_rows(void* p, int64_t pitch, int64_t rows, int64_t bytes, hipStream_t s);

// bi_mx.hip
hipError_t launch_mx_quantize(const void* x, int x_bf16, int64_t ldx, uint8_t* q, int64_t ldq, uint8_t* sc, int64_t lds,
                              int64_t rows, int64_t K, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* q, int64_t ldq, const uint8_t* sc, int64_t lds, void* y, int y_bf16,
                                int64_t ldy, int64_t rows, int64_t K, hipStream_t s);
bool mx_fits(int64_t ldx, int64_t ldxs, int64_t ldw, int64_t ldws, int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_linear(const uint8_t* xq, int64_t ldx, const uint8_t* xs, int64_t ldxs, const uint8_t* wq,
                            int64_t ldw, const uint8_t* wsc, int64_t ldws, const float* bias, void* y, int y_bf16,
                            int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t s);
TileInfo mx_tile_info(int64_t M, int64_t N, int64_t K, int y_bf16);

}  // namespace bi
