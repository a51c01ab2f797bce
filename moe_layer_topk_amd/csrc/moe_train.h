// Launchers of what stands around the experts: rows in expert order and back,
// the norms around a block, and the gradients of the grouped products.
// Arguments are validated by the caller (train_abi.hip) before any of these run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe.h"

namespace moe {

// Sum of x over the wavefront, in every lane, in a fixed order: the lane moves of
// wave_max_u32 (no LDS).
__device__ __forceinline__ float wave_sum_f32(float x) {
    auto move = [](float v, auto ctrl, auto rows) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, decltype(rows)::value, 0xF, false));
    };
    x += move(x, std::integral_constant<int, 0xB1>{}, std::integral_constant<int, 0xF>{});
    x += move(x, std::integral_constant<int, 0x4E>{}, std::integral_constant<int, 0xF>{});
    x += move(x, std::integral_constant<int, 0x141>{}, std::integral_constant<int, 0xF>{});
    x += move(x, std::integral_constant<int, 0x140>{}, std::integral_constant<int, 0xF>{});
    x += move(x, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
    x += move(x, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// Rows of tokens in expert order.  weights NULL: 1.  rows_in non-null: also
// dots[p] = <rows_in[row of p], src[p / topk]>.  pair_row NULL: the row of pair p
// is p.  al.sorted_ids non-null: the padding rows of the experts' runs are zeroed.
struct ScatterRows {
    moe_dtype dtype;
    const void* src;       // [M][H]
    const float* weights;  // [M][topk]
    const int32_t* pair_row;
    int64_t nrows;  // rows of rows_in and rows_out
    const void* rows_in;
    void* rows_out;
    float* dots;
    moe_align_bufs al;
    int M, topk, E, block_m, H;
};
hipError_t launch_scatter_rows(const ScatterRows& c, hipStream_t s);

// The same from an alignment (no pair_row yet), which the call writes.
hipError_t launch_permute(const ScatterRows& c, const int32_t* ids, int32_t* pair_row, hipStream_t s);

// out[t] = sum_j w_tj rows[row of (t, j)]; with x: dots[p] = <rows[row of p], x[p / topk]>.
struct GatherRows {
    moe_dtype dtype, out_dtype;
    const void* rows;
    int64_t nrows;
    const int32_t* pair_row;
    const float* weights;
    const void* x;
    int M, topk, H;
    void* out;
    float* dots;
};
hipError_t launch_gather_rows(const GatherRows& c, hipStream_t s);

// One row pass around a block (moe_residual_norm).
struct NormCall {
    moe_dtype dtype;
    const void *h, *y;
    moe_norm_spec n;
    int M, H;
    void *h_out, *x;
};
hipError_t launch_residual_norm(const NormCall& c, hipStream_t s);

constexpr int kMaxNormH = 16384;  // a row is held in the registers of one workgroup

struct NormGrad {
    moe_dtype dtype;
    const void *h_out, *dh_out, *dx, *y;
    moe_norm_spec n;
    int M, H;
    void *dh, *dy;
    float *dpost, *dgate, *dpre;
    float* part;  // [norm_grad_groups(M, H)][2][H]
};
int norm_grad_groups(int M, int H);
hipError_t launch_residual_norm_backward(const NormGrad& c, hipStream_t s);

// The grouped products' gradients, and the plain product of token rows (bfloat16).
struct GradCall {
    const void* dc;  // [P][N] pair order (gate_up: x [M][K])
    const void* a;   // dw: [M][K] (per token) or [P][K]
    const void* w;   // dx: [E][N][K]
    const void* z;   // dx through SiLU-and-mul: [P][2K]
    moe_align_bufs al;
    int M, topk, E, N, K, block_m;
    bool per_token;
    moe_dtype out_dtype;  // dw
    void* out;            // dx: [P][K], or [P][2K] with z; dw: [E][N][K]
    void* act;            // dx with z: [P][K] or NULL
};
hipError_t launch_gate_up(const GradCall& c, hipStream_t s);  // out [P][N]
hipError_t launch_grad_dx(const GradCall& c, hipStream_t s);
hipError_t launch_grad_dw(const GradCall& c, hipStream_t s);

// n bytes of zeros (a multiple of 16).
hipError_t launch_zero(void* p, size_t bytes, hipStream_t s);

}  // namespace moe
