// Grouped router: softmax or sigmoid scores, a bias that only the choice
// sees, groups of experts, top-k, renormalised weights (moe_route_grouped).
#include "moe_route.h"

namespace moe {

// One wavefront per token, tokens in strides over at most 2048 workgroups of
// four (32 wavefronts a CU); the next token's logits load during this one.
template <int V>
__global__ void __launch_bounds__(256) route_grouped_kernel(const void* __restrict__ logits, int bf16, RouteSpec r,
                                                            int M, int E, int topk, int32_t* __restrict__ ids,
                                                            float* __restrict__ weights) {
    const int lane = threadIdx.x & 63;
    int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= M) return;
    const int stride = gridDim.x * 4;
    float l[V];
    load_logits<V>(logits, bf16, (size_t)t, E, l);
    RouteBias<V> rb;
    rb.load(r, E);
    for (;;) {
        const int next = t + stride;
        float ln[V];
        load_logits<V>(logits, bf16, (size_t)(next < M ? next : t), E, ln);
        int sel;
        float w;
        route_grouped_token<V>(r, E, topk, l, rb, &sel, &w);
        if (lane < topk) {
            ids[(size_t)t * topk + lane] = sel;
            weights[(size_t)t * topk + lane] = w;
        }
        if (next >= M) return;
        t = next;
#pragma unroll
        for (int q = 0; q < V; ++q) l[q] = ln[q];
    }
}

hipError_t launch_route_grouped(moe_dtype ldt, const void* logits, const RouteSpec& r, int M, int E, int topk,
                                int32_t* ids, float* weights, hipStream_t s) {
    if (M == 0) return hipSuccess;
    const int blocks = (M + 3) / 4;
    const dim3 grid(blocks < 2048 ? blocks : 2048);
    const int bf16 = ldt == MOE_BF16;
    if (E <= 64) hipLaunchKernelGGL((route_grouped_kernel<1>), grid, dim3(256), 0, s, logits, bf16, r, M, E, topk, ids, weights);
    else if (E <= 128) hipLaunchKernelGGL((route_grouped_kernel<2>), grid, dim3(256), 0, s, logits, bf16, r, M, E, topk, ids, weights);
    else hipLaunchKernelGGL((route_grouped_kernel<4>), grid, dim3(256), 0, s, logits, bf16, r, M, E, topk, ids, weights);
    return hipGetLastError();
}

}  // namespace moe
