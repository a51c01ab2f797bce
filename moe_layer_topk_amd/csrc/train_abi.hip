// C ABI of what stands around the experts (rows in expert order, the norms around
// a block, gradients of the grouped products): host-side validation, before any
// HIP call, and the launches.
#include <math.h>
#include <stdint.h>

#include "moe_fused.h"
#include "moe_launch.h"
#include "moe_train.h"

using namespace moe;

namespace {

bool f32_or_bf16(moe_dtype d) { return d == MOE_F32 || d == MOE_BF16; }

// a workgroup a token and one for 64 rows, 256 threads each, below 2^32 threads
constexpr int64_t kMaxRowTokens = 1 << 23, kMaxRows = 1 << 28;

moe_status check_align_bufs(const moe_align_bufs* al) {
    if (!al || !al->sorted_ids || !al->tile_expert || !al->expert_counts || !al->expert_offsets || !al->active_experts ||
        !al->num_active)
        return MOE_ERR_NULL;
    if (misaligned(al->sorted_ids) || misaligned(al->tile_expert) || misaligned(al->expert_counts) ||
        misaligned(al->expert_offsets))
        return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

// M, topk and H of the row calls (E unknown: pairs are bounded by pair_row).
moe_status check_rows(moe_dtype dtype, int32_t M, int32_t topk, int32_t H) {
    if (!f32_or_bf16(dtype)) return MOE_ERR_UNSUPPORTED;
    if (M < 0 || topk < 1 || H < 1 || H % 8) return MOE_ERR_SHAPE;
    if (topk > kMaxTopk || M > kMaxRowTokens || (int64_t)M * topk > (1 << 24)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status check_nrows(const int32_t* pair_row, int64_t nrows, int32_t M, int32_t topk) {
    if (nrows < 0 || (M > 0 && !pair_row && nrows != (int64_t)M * topk)) return MOE_ERR_SHAPE;
    return nrows > kMaxRows ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_norm(moe_dtype dtype, const void* y, const moe_norm_spec* n, int32_t M, int32_t H) {
    if (!f32_or_bf16(dtype)) return MOE_ERR_UNSUPPORTED;
    if (!n) return MOE_ERR_NULL;
    if (!f32_or_bf16(n->w_dtype)) return MOE_ERR_UNSUPPORTED;
    if (M < 0 || H < 1 || H % 8 || !isfinite(n->scale) || !isfinite(n->eps) || !(n->eps > 0.0f)) return MOE_ERR_SHAPE;
    if (H > kMaxNormH || M >= (1 << 22)) return MOE_ERR_UNSUPPORTED;
    if (M > 0 && !y && (n->post_weight || n->gate)) return MOE_ERR_UNSUPPORTED;  // no block to norm or gate
    if (misaligned(n->post_weight) || misaligned(n->pre_weight) || misaligned(n->gate)) return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

moe_status check_grad(moe_gemm_kind kind, moe_dtype dtype, int32_t M, int32_t topk, int32_t E, int32_t N, int32_t K,
                      int32_t block_m) {
    if ((kind != MOE_GEMM_GATE_UP && kind != MOE_GEMM_DOWN) || dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    moe_status st = check_router(M, E, topk);
    if (st != MOE_OK) return st;
    if (N < 1 || K < 1 || N % 128 || K % 128 || (kind == MOE_GEMM_GATE_UP && N % 256)) return MOE_ERR_SHAPE;
    return moe_align_capacity(M, topk, E, block_m) < 0 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_permute(moe_dtype dtype, const void* x, const float* weights, const int32_t* topk_ids,
                       const moe_align_bufs* al, int32_t M, int32_t topk, int32_t E, int32_t block_m, int32_t H,
                       void* rows, int32_t* pair_row, void* stream) {
    moe_status st = check_rows(dtype, M, topk, H);
    if (st == MOE_OK) st = check_router(M, E, topk);
    if (st != MOE_OK) return st;
    if (!valid_block_m(block_m)) return MOE_ERR_UNSUPPORTED;
    const int64_t cap = moe_align_capacity(M, topk, E, block_m);
    if (cap > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (M == 0) return MOE_OK;
    if (!x || !topk_ids || !rows || !pair_row) return MOE_ERR_NULL;
    if ((st = check_align_bufs(al)) != MOE_OK) return st;
    if (misaligned(x) || misaligned(weights) || misaligned(topk_ids) || misaligned(rows) || misaligned(pair_row))
        return MOE_ERR_ALIGNMENT;
    ScatterRows c{dtype, x, weights, nullptr, cap, nullptr, rows, nullptr, *al, M, topk, E, block_m, H};
    return hip_status(launch_permute(c, topk_ids, pair_row, static_cast<hipStream_t>(stream)));
}

moe_status moe_unpermute(moe_dtype dtype, const void* rows, int64_t nrows, const int32_t* pair_row,
                         const float* weights, int32_t M, int32_t topk, int32_t H, moe_dtype out_dtype, void* out,
                         void* stream) {
    moe_status st = check_rows(dtype, M, topk, H);
    if (st == MOE_OK && !f32_or_bf16(out_dtype)) st = MOE_ERR_UNSUPPORTED;
    if (st == MOE_OK) st = check_nrows(pair_row, nrows, M, topk);
    if (st != MOE_OK || M == 0) return st;
    if (!rows || !out) return MOE_ERR_NULL;
    if (misaligned(rows) || misaligned(pair_row) || misaligned(weights) || misaligned(out)) return MOE_ERR_ALIGNMENT;
    GatherRows c{dtype, out_dtype, rows, nrows, pair_row, weights, nullptr, M, topk, H, out, nullptr};
    return hip_status(launch_gather_rows(c, static_cast<hipStream_t>(stream)));
}

moe_status moe_unpermute_backward(moe_dtype dtype, const void* dout, const void* rows, int64_t nrows,
                                  const int32_t* pair_row, const float* weights, const moe_align_bufs* al, int32_t M,
                                  int32_t topk, int32_t E, int32_t block_m, int32_t H, void* drows, float* dweights,
                                  void* stream) {
    moe_status st = check_rows(dtype, M, topk, H);
    if (st == MOE_OK) st = check_nrows(pair_row, nrows, M, topk);
    if (st == MOE_OK && al) {
        st = check_router(M, E, topk);
        if (st == MOE_OK && !valid_block_m(block_m)) st = MOE_ERR_UNSUPPORTED;
        if (st == MOE_OK && M > 0 && (!pair_row || nrows != moe_align_capacity(M, topk, E, block_m))) st = MOE_ERR_SHAPE;
    }
    if (st != MOE_OK) return st;
    if (!weights && dweights) return MOE_ERR_UNSUPPORTED;
    if (M == 0) return MOE_OK;
    if (!dout || !drows || !rows != !dweights) return MOE_ERR_NULL;
    if (al && (st = check_align_bufs(al)) != MOE_OK) return st;
    if (misaligned(dout) || misaligned(rows) || misaligned(pair_row) || misaligned(weights) || misaligned(drows) ||
        misaligned(dweights))
        return MOE_ERR_ALIGNMENT;
    ScatterRows c{dtype, dout, weights, pair_row, nrows, rows, drows, dweights, al ? *al : moe_align_bufs{}, M, topk, E,
                  block_m, H};
    return hip_status(launch_scatter_rows(c, static_cast<hipStream_t>(stream)));
}

moe_status moe_permute_backward(moe_dtype dtype, const void* drows, int64_t nrows, const int32_t* pair_row,
                                const void* x, const float* weights, int32_t M, int32_t topk, int32_t H, void* dx,
                                float* dweights, void* stream) {
    moe_status st = check_rows(dtype, M, topk, H);
    if (st == MOE_OK) st = check_nrows(pair_row, nrows, M, topk);
    if (st != MOE_OK) return st;
    if (!weights && dweights) return MOE_ERR_UNSUPPORTED;
    if (M == 0) return MOE_OK;
    if (!drows || !dx || !x != !dweights) return MOE_ERR_NULL;
    if (misaligned(drows) || misaligned(pair_row) || misaligned(x) || misaligned(weights) || misaligned(dx) ||
        misaligned(dweights))
        return MOE_ERR_ALIGNMENT;
    GatherRows c{dtype, dtype, drows, nrows, pair_row, weights, x, M, topk, H, dx, dweights};
    return hip_status(launch_gather_rows(c, static_cast<hipStream_t>(stream)));
}

moe_status moe_residual_norm(moe_dtype dtype, const void* h, const void* y, const moe_norm_spec* norm, int32_t M,
                             int32_t H, void* h_out, void* x, void* stream) {
    moe_status st = check_norm(dtype, y, norm, M, H);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    if (!y && h_out) return MOE_ERR_UNSUPPORTED;
    if (!h || (y && !h_out) || !norm->pre_weight != !x || (!y && !x)) return MOE_ERR_NULL;
    if (misaligned(h) || misaligned(y) || misaligned(h_out) || misaligned(x)) return MOE_ERR_ALIGNMENT;
    if (h_out == x) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_residual_norm(NormCall{dtype, h, y, *norm, M, H, h_out, x}, static_cast<hipStream_t>(stream)));
}

size_t moe_residual_norm_workspace_size(int32_t M, int32_t H) {
    if (M <= 0 || H < 1) return 0;
    return (size_t)norm_grad_groups(M, H) * 2 * H * sizeof(float);
}

moe_status moe_residual_norm_backward(moe_dtype dtype, const void* h_out, const void* dh_out, const void* dx,
                                      const void* y, const moe_norm_spec* norm, int32_t M, int32_t H, void* dh, void* dy,
                                      float* dpost_weight, float* dgate, float* dpre_weight, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    moe_status st = check_norm(dtype, y, norm, M, H);
    if (st != MOE_OK) return st;
    if ((dpost_weight && !norm->post_weight) || (dgate && !norm->gate) || (dpre_weight && !norm->pre_weight))
        return MOE_ERR_UNSUPPORTED;
    if (misaligned(dpost_weight) || misaligned(dgate) || misaligned(dpre_weight)) return MOE_ERR_ALIGNMENT;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) {  // sums over no rows
        float* const sums[3] = {dpost_weight, norm->gate_per_token ? nullptr : dgate, dpre_weight};
        for (float* p : sums)
            if (p && launch_zero(p, (size_t)H * sizeof(float), s) != hipSuccess) return MOE_ERR_HIP;
        return MOE_OK;
    }
    if ((norm->pre_weight && !h_out) || !norm->pre_weight != !dx || !y != !dy || !dh || !workspace) return MOE_ERR_NULL;
    if (misaligned(h_out) || misaligned(dh_out) || misaligned(dx) || misaligned(y) || misaligned(dh) || misaligned(dy) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return MOE_ERR_ALIGNMENT;
    if (dh == dy) return MOE_ERR_UNSUPPORTED;
    if (workspace_bytes < moe_residual_norm_workspace_size(M, H)) return MOE_ERR_WORKSPACE;
    return hip_status(launch_residual_norm_backward(
        NormGrad{dtype, h_out, dh_out, dx, y, *norm, M, H, dh, dy, dpost_weight, dgate, dpre_weight,
                 static_cast<float*>(workspace)}, s));
}

moe_status moe_grouped_gemm_dx(moe_gemm_kind kind, moe_dtype dtype, const void* dc, const void* w, const void* z,
                               const moe_align_bufs* al, int32_t M, int32_t topk, int32_t E, int32_t N, int32_t K,
                               int32_t block_m, void* da, void* act, void* stream) {
    moe_status st = check_grad(kind, dtype, M, topk, E, N, K, block_m);
    if (st != MOE_OK) return st;
    if (block_m != 64 && block_m != 128) return MOE_ERR_UNSUPPORTED;
    // (32-bit offsets into an expert's weights: a last column tile reads up to 256 bytes
    // past the last row)
    if ((uint64_t)N * (uint64_t)K * 2 > 0xffff0000ull) return MOE_ERR_UNSUPPORTED;
    if ((kind == MOE_GEMM_GATE_UP && z) || (!z && act)) return MOE_ERR_UNSUPPORTED;
    if (M == 0) return MOE_OK;
    if (!dc || !w || !da) return MOE_ERR_NULL;
    if ((st = check_align_bufs(al)) != MOE_OK) return st;
    if (misaligned(dc) || misaligned(w) || misaligned(z) || misaligned(da) || misaligned(act)) return MOE_ERR_ALIGNMENT;
    GradCall c{dc, nullptr, w, z, *al, M, topk, E, N, K, block_m, false, MOE_BF16, da, act};
    return hip_status(launch_grad_dx(c, static_cast<hipStream_t>(stream)));
}

moe_status moe_grouped_gemm_dw(moe_gemm_kind kind, moe_dtype dtype, const void* dc, const void* a,
                               const moe_align_bufs* al, int32_t M, int32_t topk, int32_t E, int32_t N, int32_t K,
                               int32_t block_m, moe_dtype dw_dtype, void* dw, void* stream) {
    moe_status st = check_grad(kind, dtype, M, topk, E, N, K, block_m);
    if (st != MOE_OK) return st;
    if (!valid_block_m(block_m) || !f32_or_bf16(dw_dtype)) return MOE_ERR_UNSUPPORTED;
    if (!dw) return MOE_ERR_NULL;
    if (misaligned(dw)) return MOE_ERR_ALIGNMENT;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (M == 0) return hip_status(launch_zero(dw, (size_t)E * N * K * (dw_dtype == MOE_F32 ? 4 : 2), s));
    if (!dc || !a) return MOE_ERR_NULL;
    if ((st = check_align_bufs(al)) != MOE_OK) return st;
    if (misaligned(dc) || misaligned(a)) return MOE_ERR_ALIGNMENT;
    GradCall c{dc, a, nullptr, nullptr, *al, M, topk, E, N, K, block_m, kind == MOE_GEMM_GATE_UP, dw_dtype, dw, nullptr};
    return hip_status(launch_grad_dw(c, s));
}

}  // extern "C"
