// Grouped router: softmax or sigmoid scores, a bias that only the choice
// sees, groups of experts, top-k, renormalised weights (moe_route_grouped).
#include "moe_route.h"

namespace moe {

// One wavefront per token, tokens in strides over at most 2048 workgroups of
// four (32 wavefronts a CU); the next token's logits load during this one.
template <int V, int GM, bool BIASED>
__global__ void __launch_bounds__(256) route_grouped_kernel(const void* __restrict__ logits, int bf16, RouteSpec r,
                                                            int M, int E, int topk, int32_t* __restrict__ ids,
                                                            float* __restrict__ weights) {
    const int lane = threadIdx.x & 63;
    int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= M) return;
    const int stride = gridDim.x * 4;
    float l[V];
    load_logits<V>(logits, bf16, (size_t)t, E, l);
    const RouteWave<V, GM, BIASED> rw(r, E);
    for (;;) {
        const int next = t + stride;
        float ln[V];
        load_logits<V>(logits, bf16, (size_t)(next < M ? next : t), E, ln);
        int sel;
        float w;
        route_grouped_token<V, GM, BIASED>(r, E, topk, l, rw, &sel, &w);
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

template <int V, int GM>
static hipError_t launch_v(const void* logits, int bf16, const RouteSpec& r, int M, int E, int topk, int32_t* ids,
                           float* weights, hipStream_t s) {
    const int blocks = (M + 3) / 4;
    const dim3 grid(blocks < 2048 ? blocks : 2048);
    if (r.bias)
        hipLaunchKernelGGL((route_grouped_kernel<V, GM, true>), grid, dim3(256), 0, s, logits, bf16, r, M, E, topk, ids, weights);
    else
        hipLaunchKernelGGL((route_grouped_kernel<V, GM, false>), grid, dim3(256), 0, s, logits, bf16, r, M, E, topk, ids, weights);
    return hipGetLastError();
}

template <int V>
static hipError_t launch_g(const void* logits, int bf16, const RouteSpec& r, int M, int E, int topk, int32_t* ids,
                           float* weights, hipStream_t s) {
    switch (group_mode(r, E, V)) {
        case kNoGroups: return launch_v<V, kNoGroups>(logits, bf16, r, M, E, topk, ids, weights, s);
        case kLaneGroups: return launch_v<V, kLaneGroups>(logits, bf16, r, M, E, topk, ids, weights, s);
        default: return launch_v<V, kAnyGroups>(logits, bf16, r, M, E, topk, ids, weights, s);
    }
}

hipError_t launch_route_grouped(moe_dtype ldt, const void* logits, const RouteSpec& r, int M, int E, int topk,
                                int32_t* ids, float* weights, hipStream_t s) {
    if (M == 0) return hipSuccess;
    const int bf16 = ldt == MOE_BF16;
    if (E <= 64) return launch_g<1>(logits, bf16, r, M, E, topk, ids, weights, s);
    if (E <= 128) return launch_g<2>(logits, bf16, r, M, E, topk, ids, weights, s);
    return launch_g<4>(logits, bf16, r, M, E, topk, ids, weights, s);
}

}  // namespace moe
