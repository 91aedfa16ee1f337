// bi_abi.cpp -- the C ABI: argument validation, planning, launch.
//
// Every check happens on the host before anything is enqueued, and a rejected
// call enqueues nothing.  There is no fallback: a shape the recipe table cannot
// serve is an error, never a silent switch to a batch-dependent route (sparse
// MLA page, "Review follow-up" and the fail-closed commit: a batch-dependent
// result is raised, not returned).
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <string.h>

#include "bi.h"
#include "bi_ffn.h"
#include "bi_launch.h"
#include "bi_moe.h"
#include "bi_plan.h"
#include "bi_topk.h"

using namespace bi;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Common validation of a linear call.  elem_x / elem_w: bytes per element.
bi_status_t check_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const float* bias,
                         const void* y, int64_t ldy, int64_t M, int64_t N, int64_t K, int elem_x,
                         int elem_w, int elem_y)
{
    if (M < 0 || N < 0 || K < 0)
        return BI_EINVAL;
    if (M == 0)
        return BI_OK;
    if (!x || !w || !y)
        return BI_EINVAL;
    if (!aligned16(x) || !aligned16(w) || (bias && !aligned16(bias)) || !aligned16(y))
        return BI_EINVAL;
    if (ldx < K || ldw < K || ldy < N)
        return BI_EINVAL;
    if ((ldx * elem_x) % 16 != 0 || (ldw * elem_w) % 16 != 0 || (ldy * elem_y) % 4 != 0)
        return BI_EINVAL;
    if (M > (int64_t(1) << 30))
        return BI_EUNSUPPORTED;
    return BI_OK;
}

bi_status_t run_linear(int xkind, const void* x, int64_t ldx, const void* w, int64_t ldw,
                       const float* bias, void* y, int y_bf16, int64_t ldy, int64_t M, int64_t N,
                       int64_t K, const bi_recipe_t& recipe, int32_t path, void* ws, size_t ws_bytes,
                       hipStream_t stream)
{
    Plan p;
    bi_status_t st = make_plan(recipe, path, M, N, K, &p);
    if (st != BI_OK)
        return st;
    if (p.ws_bytes > 0 && (!ws || ws_bytes < p.ws_bytes || !aligned16(ws)))
        return BI_EWORKSPACE;
    LinearArgs a{x, ldx, w, ldw, bias, y, y_bf16, ldy, (int)M, (int)N, (int)K};
    return launch_linear(xkind, a, p, ws, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

// One matrix of a feed-forward call: `rows` rows of `cols` elements of `elem`
// bytes, 16-byte aligned with a pitch that keeps every row so.
bool matrix_ok(const void* p, int64_t ld, int64_t cols, int elem)
{
    return p && aligned16(p) && ld >= cols && (ld * elem) % 16 == 0 && ld < (int64_t(1) << 40);
}

// Sizes every feed-forward call shares; rows may be 0.
bi_status_t check_sizes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return BI_EINVAL;
    if (N == 0 || K == 0 || N % 16 != 0 || K % 32 != 0)
        return BI_EUNSUPPORTED;
    if (M > (int64_t(1) << 30) || N > (int64_t(1) << 29) || K > (int64_t(1) << 29))
        return BI_EUNSUPPORTED;
    return BI_OK;
}

bool dtype_ok(int32_t d) { return d == BI_F32 || d == BI_BF16; }
int dtype_bytes(int32_t d) { return d == BI_F32 ? 4 : 2; }

// Codes and scales of an MXFP4 operand.
bool mx_ok(const void* q, int64_t ldq, const void* sc, int64_t lds, int64_t K)
{
    return q && sc && aligned16(q) && (reinterpret_cast<uintptr_t>(sc) & 3u) == 0 && ldq >= K / 2 && ldq % 16 == 0 &&
           lds >= K / 32 && lds % 4 == 0 && ldq < (int64_t(1) << 40) && lds < (int64_t(1) << 40);
}

// The status of a feed-forward launch: a grid too large for one is a size that
// is not served.
bi_status_t launch_status(hipError_t e)
{
    return e == hipSuccess ? BI_OK : e == hipErrorInvalidConfiguration ? BI_EUNSUPPORTED : BI_EHIP;
}

size_t dh_bytes(int64_t M, int64_t I) { return (size_t)M * 2 * (size_t)I * 2; }

// The gradients of an empty batch: zero dw and db.
bi_status_t run_empty_bwd(void* dw, int32_t dw_dtype, int64_t lddw, float* db, int64_t N, int64_t K, hipStream_t stream)
{
    const int64_t es = dtype_bytes(dw_dtype);
    if (dw && launch_zero_rows(dw, lddw * es, N, K * es, stream) != hipSuccess)
        return BI_EHIP;
    if (db && launch_zero_rows(db, N * 4, 1, N * 4, stream) != hipSuccess)
        return BI_EHIP;
    return BI_OK;
}

}  // namespace

namespace bi {

bi_status_t linear_f32_checked(const float* x, int64_t ldx, const float* w, int64_t ldw, const float* bias,
                               float* y, int64_t ldy, int64_t M, int64_t N, int64_t K, size_t* ws_needed,
                               bool no_split)
{
    bi_status_t st = check_linear(x, ldx, w, ldw, bias, y, ldy, M, N, K, 4, 4, 4);
    if (st != BI_OK || M == 0) {
        *ws_needed = 0;
        return st;
    }
    bi_recipe_t r;
    if ((st = recipe_for(BI_F32, N, K, &r)) != BI_OK)
        return st;
    Plan p;
    if ((st = make_plan(r, BI_PATH_AUTO | (no_split ? kPathNoSplit : 0), M, N, K, &p)) != BI_OK)
        return st;
    *ws_needed = p.ws_bytes;
    return BI_OK;
}

bi_status_t linear_f32_run(const float* x, int64_t ldx, const float* w, int64_t ldw, const float* bias, float* y,
                           int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                           hipStream_t stream, bool no_split)
{
    bi_status_t st = check_linear(x, ldx, w, ldw, bias, y, ldy, M, N, K, 4, 4, 4);
    if (st != BI_OK || M == 0)
        return st;
    bi_recipe_t r;
    if ((st = recipe_for(BI_F32, N, K, &r)) != BI_OK)
        return st;
    return run_linear(kXF32, x, ldx, w, ldw, bias, y, 0, ldy, M, N, K, r,
                      BI_PATH_AUTO | (no_split ? kPathNoSplit : 0), ws, ws_bytes, stream);
}

}  // namespace bi

extern "C" {

const char* bi_status_str(bi_status_t s)
{
    switch (s) {
    case BI_OK: return "BI_OK";
    case BI_EINVAL: return "BI_EINVAL: invalid argument";
    case BI_EUNSUPPORTED: return "BI_EUNSUPPORTED: (dtype, N, K) not served by the recipe table";
    case BI_EWORKSPACE: return "BI_EWORKSPACE: workspace missing or too small";
    case BI_EHIP: return "BI_EHIP: HIP launch failed";
    }
    return "unknown bi_status_t";
}

bi_status_t bi_describe_recipe(int32_t dtype, int64_t N, int64_t K, bi_recipe_t* out)
{
    return recipe_for(dtype, N, K, out);
}

size_t bi_linear_workspace_size(int32_t dtype, int64_t M, int64_t N, int64_t K)
{
    bi_recipe_t r;
    if (recipe_for(dtype, N, K, &r) != BI_OK || M <= 0)
        return 0;
    Plan p;
    if (make_plan(r, BI_PATH_AUTO, M, N, K, &p) != BI_OK)
        return 0;
    return p.ws_bytes;
}

size_t bi_lab_workspace_size(const bi_recipe_t* recipe, int32_t path, int64_t M, int64_t N, int64_t K)
{
    if (!recipe || M <= 0)
        return 0;
    Plan p;
    if (make_plan(*recipe, path, M, N, K, &p) != BI_OK)
        return 0;
    return p.ws_bytes;
}

bi_status_t bi_linear_f32(const float* x, int64_t ldx, const float* w, int64_t ldw, const float* bias,
                          float* y, int64_t ldy, int64_t M, int64_t N, int64_t K, void* ws,
                          size_t ws_bytes, hipStream_t stream)
{
    return linear_f32_run(x, ldx, w, ldw, bias, y, ldy, M, N, K, ws, ws_bytes, stream);
}

bi_status_t bi_linear_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
                           const float* bias, void* y, int32_t y_dtype, int64_t ldy, int64_t M,
                           int64_t N, int64_t K, void* ws, size_t ws_bytes, hipStream_t stream)
{
    if (y_dtype != BI_F32 && y_dtype != BI_BF16)
        return BI_EINVAL;
    bi_status_t st = check_linear(x, ldx, w, ldw, bias, y, ldy, M, N, K, 2, 2, y_dtype == BI_BF16 ? 2 : 4);
    if (st != BI_OK || M == 0)
        return st;
    bi_recipe_t r;
    if ((st = recipe_for(BI_BF16, N, K, &r)) != BI_OK)
        return st;
    return run_linear(kXBF16, x, ldx, w, ldw, bias, y, y_dtype == BI_BF16, ldy, M, N, K, r, BI_PATH_AUTO,
                      ws, ws_bytes, stream);
}

bi_status_t bi_lab_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const float* bias,
                          void* y, int32_t y_dtype, int64_t ldy, int64_t M, int64_t N, int64_t K,
                          const bi_recipe_t* recipe, int32_t path, void* ws, size_t ws_bytes,
                          hipStream_t stream)
{
    if (!recipe || (y_dtype != BI_F32 && y_dtype != BI_BF16))
        return BI_EINVAL;
    const int ex = recipe->dtype == BI_F32 ? 4 : 2;
    bi_status_t st = check_linear(x, ldx, w, ldw, bias, y, ldy, M, N, K, ex, ex, y_dtype == BI_BF16 ? 2 : 4);
    if (st != BI_OK || M == 0)
        return st;
    return run_linear(recipe->dtype == BI_F32 ? kXF32 : kXBF16, x, ldx, w, ldw, bias, y,
                      y_dtype == BI_BF16, ldy, M, N, K, *recipe, path, ws, ws_bytes, stream);
}

bi_status_t bi_negctl_linear_f32(const float* x, int64_t ldx, const float* w, int64_t ldw,
                                 const float* bias, float* y, int64_t ldy, int64_t M, int64_t N,
                                 int64_t K, void* ws, size_t ws_bytes, hipStream_t stream)
{
    bi_status_t st = check_linear(x, ldx, w, ldw, bias, y, ldy, M, N, K, 4, 4, 4);
    if (st != BI_OK || M == 0)
        return st;
    bi_recipe_t r;
    if ((st = recipe_for(BI_F32, N, K, &r)) != BI_OK)
        return st;
    // the deliberate defect: the k tile width follows the batch size (never
    // wider than the shipped recipe's workspace needs)
    r.block_k = (M < 64) ? 2 * r.block_k : r.block_k;
    if (K % r.block_k != 0)
        return BI_EUNSUPPORTED;
    return run_linear(kXF32, x, ldx, w, ldw, bias, y, 0, ldy, M, N, K, r, BI_PATH_AUTO, ws, ws_bytes,
                      stream);
}

bi_status_t bi_lab_xcc_ids(uint32_t* out, int32_t grid_x, int32_t grid_y, hipStream_t stream)
{
    if (!out || grid_x <= 0 || grid_y <= 0 || (reinterpret_cast<uintptr_t>(out) & 3u) != 0)
        return BI_EINVAL;
    if ((int64_t)grid_x * grid_y > (int64_t(1) << 24) || grid_y > 65535)
        return BI_EUNSUPPORTED;
    return launch_xcc_ids(out, grid_x, grid_y, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

bi_status_t bi_lab_plan(int32_t dtype, int64_t M, int64_t N, int64_t K, int32_t* path)
{
    if (!path || M <= 0)
        return BI_EINVAL;
    bi_recipe_t r;
    bi_status_t st = recipe_for(dtype, N, K, &r);
    if (st != BI_OK)
        return st;
    Plan p;
    if ((st = make_plan(r, BI_PATH_AUTO, M, N, K, &p)) != BI_OK)
        return st;
    *path = p.path;
    return BI_OK;
}

bi_status_t bi_lab_moe_layout(int64_t M, int64_t H, int64_t E, int64_t I, int64_t topk, int64_t* offsets)
{
    return moe_layout_offsets(M, H, E, I, topk, offsets);
}

bi_status_t bi_lab_empty(int32_t grid, int32_t threads, hipStream_t stream)
{
    if (grid <= 0 || threads <= 0 || threads > 1024 || threads % 64 != 0)
        return BI_EINVAL;
    return launch_empty(grid, threads, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

bi_status_t bi_lab_stream_read(const void* src, int64_t bytes, uint32_t* sink, int32_t grid, hipStream_t stream)
{
    if (!src || !sink || bytes <= 0 || bytes % 16 != 0 || grid <= 0 || grid > 65535 ||
        (reinterpret_cast<uintptr_t>(src) & 15u) != 0 || (reinterpret_cast<uintptr_t>(sink) & 3u) != 0)
        return BI_EINVAL;
    return launch_stream_read(src, bytes, sink, grid, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

bi_status_t bi_lab_l2_read(const void* src, int64_t bytes, int32_t iters, uint32_t* sink, int32_t grid,
                           hipStream_t stream)
{
    // a power of two of at least one full round (256 lanes x 8 loads x 16 B)
    // and at most 2 MiB
    if (!src || !sink || bytes < 32768 || bytes > (int64_t(2) << 20) || (bytes & (bytes - 1)) != 0 ||
        iters <= 0 || grid <= 0 || grid > 65535 || (reinterpret_cast<uintptr_t>(src) & 15u) != 0 ||
        (reinterpret_cast<uintptr_t>(sink) & 3u) != 0)
        return BI_EINVAL;
    return launch_l2_read(src, bytes, iters, sink, grid, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

bi_status_t bi_lab_clock(uint64_t* out, int32_t grid, int32_t iters, hipStream_t stream)
{
    if (!out || grid <= 0 || grid > 65535 || iters <= 0 || (reinterpret_cast<uintptr_t>(out) & 7u) != 0)
        return BI_EINVAL;
    return launch_clock(out, grid, iters, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

bi_status_t bi_lab_lds_read(uint64_t* out, int32_t grid, int32_t iters, hipStream_t stream)
{
    if (!out || grid <= 0 || grid > 65535 || iters <= 0 || (reinterpret_cast<uintptr_t>(out) & 7u) != 0)
        return BI_EINVAL;
    return launch_lds_read(out, grid, iters, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

bi_status_t bi_lab_mfma_rate(uint64_t* out, int32_t dtype, int32_t chains, int32_t grid, int32_t iters,
                             hipStream_t stream)
{
    if (!out || (dtype != BI_F32 && dtype != BI_BF16) || (chains != 1 && chains != 2 && chains != 4 && chains != 8) ||
        grid <= 0 || grid > 65535 || iters <= 0 || (reinterpret_cast<uintptr_t>(out) & 7u) != 0)
        return BI_EINVAL;
    return launch_mfma_rate(out, dtype == BI_BF16, chains, grid, iters, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

size_t bi_moe_workspace_size(int64_t M, int64_t H, int64_t E, int64_t I, int64_t topk)
{
    return moe_workspace_size(M, H, E, I, topk);
}

bi_status_t bi_moe_grouped_gemm(const uint16_t* x, const float* w_router, const float* b_router,
                                const uint16_t* w13, const uint16_t* w2, int64_t M, int64_t H,
                                int64_t E, int64_t I, int64_t topk, int32_t* topk_ids,
                                float* topk_probs, float* y, void* ws, size_t ws_bytes,
                                hipStream_t stream)
{
    const bi_moe_options_t opt{BI_ACT_SWIGLU, 1, 0, 1};
    return moe_run(x, w_router, b_router, w13, w2, M, H, E, I, topk, opt, topk_ids, topk_probs, y, ws,
                   ws_bytes, stream);
}

bi_status_t bi_moe_grouped_gemm_ex(const uint16_t* x, const float* w_router, const float* b_router,
                                   const uint16_t* w1, const uint16_t* w2, int64_t M, int64_t H, int64_t E,
                                   int64_t I, int64_t topk, const bi_moe_options_t* options,
                                   int32_t* topk_ids, float* topk_probs, float* y, void* ws, size_t ws_bytes,
                                   hipStream_t stream)
{
    const bi_moe_options_t opt = options ? *options : bi_moe_options_t{BI_ACT_SWIGLU, 1, 0, 1};
    return moe_run(x, w_router, b_router, w1, w2, M, H, E, I, topk, opt, topk_ids, topk_probs, y, ws,
                   ws_bytes, stream);
}

bi_status_t bi_indexer_topk(const float* scores, int64_t ld, int64_t rows, int64_t cols,
                            const int64_t* row_start, const int64_t* row_end, int64_t topk,
                            int32_t* out, int64_t ld_out, hipStream_t stream)
{
    auto al = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    if (rows < 0 || cols < 0 || topk <= 0 || ld < cols || ld_out < topk)
        return BI_EINVAL;
    if (rows == 0)
        return BI_OK;
    if (cols > kTopkMaxCols || rows > (int64_t(1) << 31) - 1 || topk > (int64_t(1) << 30))
        return BI_EUNSUPPORTED;
    if (!out || (cols > 0 && !scores))
        return BI_EINVAL;
    if (!al(scores, 4) || !al(out, 4) || !al(row_start, 8) || !al(row_end, 8))
        return BI_EINVAL;
    return launch_topk_rows(scores, ld, rows, cols, row_start, row_end, topk, out, ld_out, stream) == hipSuccess
               ? BI_OK
               : BI_EHIP;
}

bi_status_t bi_gated_linear_bf16(const uint16_t* x, int64_t ldx, const uint16_t* w13, int64_t ldw, int32_t gate,
                                 uint16_t* y, int64_t ldy, uint16_t* h, int64_t ldh, int64_t M, int64_t I, int64_t H,
                                 hipStream_t stream)
{
    if (gate != BI_GATE_SILU && gate != BI_GATE_GELU_TANH)
        return BI_EINVAL;
    bi_status_t st = check_sizes(M, I, H);
    if (st != BI_OK || M == 0)
        return st;
    if (!matrix_ok(x, ldx, H, 2) || !matrix_ok(w13, ldw, H, 2) || !matrix_ok(y, ldy, I, 2) ||
        (h && !matrix_ok(h, ldh, 2 * I, 2)))
        return BI_EINVAL;
    if (!gated_fits(ldx, ldw, M, I, H))
        return BI_EUNSUPPORTED;
    return launch_status(launch_gated(x, ldx, w13, ldw, gate, y, ldy, h, ldh, M, I, H, stream));
}

size_t bi_gated_linear_bwd_workspace_size(int64_t M, int64_t I)
{
    if (check_sizes(M, I, 32) != BI_OK || M == 0)
        return 0;
    return kDecodeCounterBytes + dh_bytes(M, I);
}

bi_status_t bi_gated_linear_bf16_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx,
                                     const uint16_t* w13, int64_t ldw, const uint16_t* h, int64_t ldh, int32_t gate,
                                     uint16_t* dx, int64_t lddx, void* dw, int32_t dw_dtype, int64_t lddw, int64_t M,
                                     int64_t I, int64_t H, void* ws, size_t ws_bytes, hipStream_t stream)
{
    if ((gate != BI_GATE_SILU && gate != BI_GATE_GELU_TANH) || !dtype_ok(dw_dtype))
        return BI_EINVAL;
    bi_status_t st = check_sizes(M, I, H);
    if (st != BI_OK || (!dx && !dw))
        return st;
    if (dw && !matrix_ok(dw, lddw, H, dtype_bytes(dw_dtype)))
        return BI_EINVAL;
    if (M == 0)
        return run_empty_bwd(dw, dw_dtype, lddw, nullptr, 2 * I, H, stream);
    if (!matrix_ok(dy, lddy, I, 2) || !matrix_ok(h, ldh, 2 * I, 2))
        return BI_EINVAL;
    if (dx && (!matrix_ok(dx, lddx, H, 2) || !matrix_ok(w13, ldw, H, 2)))
        return BI_EINVAL;
    if (dw && !matrix_ok(x, ldx, H, 2))
        return BI_EINVAL;
    BwdPlan plan;
    if (!plan_linear_bwd(dx, dw, false, dw_dtype == BI_BF16, 2 * I, ldx, ldw, M, 2 * I, H, &plan))
        return BI_EUNSUPPORTED;
    if (!ws || ws_bytes < kDecodeCounterBytes + dh_bytes(M, I) || !aligned16(ws))
        return BI_EWORKSPACE;
    uint16_t* dh = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(ws) + kDecodeCounterBytes);
    if (launch_gate_bwd(dy, lddy, h, ldh, gate, dh, 2 * I, M, I, stream) != hipSuccess ||
        launch_linear_bwd(plan, dh, 2 * I, x, ldx, w13, ldw, dx, lddx, dw, dw_dtype == BI_BF16, lddw, nullptr, M, 2 * I, H,
                          stream) != hipSuccess)
        return BI_EHIP;
    return BI_OK;
}

bi_status_t bi_linear_bf16_bwd(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx, const uint16_t* w,
                               int64_t ldw, uint16_t* dx, int64_t lddx, void* dw, int32_t dw_dtype, int64_t lddw,
                               float* db, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    if (!dtype_ok(dw_dtype))
        return BI_EINVAL;
    bi_status_t st = check_sizes(M, N, K);
    if (st != BI_OK || (!dx && !dw && !db))
        return st;
    if ((dw && !matrix_ok(dw, lddw, K, dtype_bytes(dw_dtype))) || (db && !aligned16(db)))
        return BI_EINVAL;
    if (M == 0)
        return run_empty_bwd(dw, dw_dtype, lddw, db, N, K, stream);
    if (!matrix_ok(dy, lddy, N, 2))
        return BI_EINVAL;
    if (dx && (!matrix_ok(dx, lddx, K, 2) || !matrix_ok(w, ldw, K, 2)))
        return BI_EINVAL;
    if (dw && !matrix_ok(x, ldx, K, 2))
        return BI_EINVAL;
    BwdPlan plan;
    if (!plan_linear_bwd(dx, dw, db, dw_dtype == BI_BF16, lddy, ldx, ldw, M, N, K, &plan))
        return BI_EUNSUPPORTED;
    return launch_linear_bwd(plan, dy, lddy, x, ldx, w, ldw, dx, lddx, dw, dw_dtype == BI_BF16, lddw, db, M, N, K, stream) ==
                   hipSuccess
               ? BI_OK
               : BI_EHIP;
}

bi_status_t bi_quantize_mxfp4(const void* x, int32_t x_dtype, int64_t ldx, uint8_t* q, int64_t ldq, uint8_t* sc,
                              int64_t lds, int64_t rows, int64_t K, hipStream_t stream)
{
    if (!dtype_ok(x_dtype))
        return BI_EINVAL;
    bi_status_t st = check_sizes(rows, 16, K);
    if (st != BI_OK || rows == 0)
        return st;
    if (!matrix_ok(x, ldx, K, dtype_bytes(x_dtype)) || !mx_ok(q, ldq, sc, lds, K))
        return BI_EINVAL;
    return launch_mx_quantize(x, x_dtype == BI_BF16, ldx, q, ldq, sc, lds, rows, K, stream) == hipSuccess ? BI_OK : BI_EHIP;
}

bi_status_t bi_dequantize_mxfp4(const uint8_t* q, int64_t ldq, const uint8_t* sc, int64_t lds, void* y, int32_t y_dtype,
                                int64_t ldy, int64_t rows, int64_t K, hipStream_t stream)
{
    if (!dtype_ok(y_dtype))
        return BI_EINVAL;
    bi_status_t st = check_sizes(rows, 16, K);
    if (st != BI_OK || rows == 0)
        return st;
    if (!matrix_ok(y, ldy, K, dtype_bytes(y_dtype)) || !mx_ok(q, ldq, sc, lds, K))
        return BI_EINVAL;
    return launch_mx_dequantize(q, ldq, sc, lds, y, y_dtype == BI_BF16, ldy, rows, K, stream) == hipSuccess ? BI_OK
                                                                                                          : BI_EHIP;
}

bi_status_t bi_linear_mxfp4(const uint8_t* xq, int64_t ldxq, const uint8_t* xs, int64_t ldxs, const uint8_t* wq,
                            int64_t ldwq, const uint8_t* wsc, int64_t ldws, const float* bias, void* y, int32_t y_dtype,
                            int64_t ldy, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    if (!dtype_ok(y_dtype))
        return BI_EINVAL;
    bi_status_t st = check_sizes(M, N, K);
    if (st != BI_OK || M == 0)
        return st;
    if (!mx_ok(xq, ldxq, xs, ldxs, K) || !mx_ok(wq, ldwq, wsc, ldws, K) || (bias && !aligned16(bias)) ||
        !matrix_ok(y, ldy, N, dtype_bytes(y_dtype)))
        return BI_EINVAL;
    if (!mx_fits(ldxq, ldxs, ldwq, ldws, M, N, K))
        return BI_EUNSUPPORTED;
    return launch_status(launch_mx_linear(xq, ldxq, xs, ldxs, wq, ldwq, wsc, ldws, bias, y, y_dtype == BI_BF16, ldy, M, N,
                                          K, stream));
}

bi_status_t bi_lab_ffn_tile(int32_t op, int64_t M, int64_t N, int64_t K, int32_t out_dtype, int32_t* info)
{
    if (op < BI_FFN_GATED || op > BI_FFN_DW || !dtype_ok(out_dtype) || M <= 0 || !info)
        return BI_EINVAL;
    const bi_status_t st = check_sizes(M, N, K);
    if (st != BI_OK)
        return st;
    const int bf16 = out_dtype == BI_BF16;
    const TileInfo t = op == BI_FFN_GATED ? gated_tile_info(M, N, K) : op == BI_FFN_MXFP4 ? mx_tile_info(M, N, K, bf16)
                       : linear_bwd_tile_info(op == BI_FFN_DW, bf16, M, N, K);
    memcpy(info, &t, sizeof t);
    return BI_OK;
}

}  // extern "C"
