// Grouped router: softmax or sigmoid scores, a bias that only the choice
// sees, groups of experts, top-k, renormalised weights (moe_route_grouped).
#include "moe_block.h"
#include "moe_route.h"

namespace moe {

// One wavefront per token, tokens in strides over at most 2048 workgroups of
// four (32 wavefronts a CU); the next token's logits load during this one.
// Bound by vector ALU work, about 600 instructions a token: 16384 tokens of 256
// experts in 8 groups 22.6 us (17 MB; 46 where float32 settles no choice, see
// moe_route.h), and no faster with more or fewer wavefronts a CU; two tokens a
// wavefront cost as much in sorting as they save.
// Workgroups past `routers` quantise the token rows (qj) the layer needs next.
template <int V, int GM, bool BIASED>
__global__ void __launch_bounds__(256) route_grouped_kernel(const void* __restrict__ logits, int bf16, RouteSpec r,
                                                            int M, int E, int topk, int32_t* __restrict__ ids,
                                                            float* __restrict__ weights, int routers, QuantJob qj) {
    if ((int)blockIdx.x >= routers) {
        quant_rows<MOE_BF16>(qj.x, qj.nblk, qj.q, qj.scale, blockIdx.x - routers, gridDim.x - routers, 256);
        return;
    }
    const int lane = threadIdx.x & 63;
    int t = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= M) return;
    const int stride = routers * 4;
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

struct RouteCall {
    const void* logits;
    int bf16;
    const RouteSpec& r;
    int M, E, topk;
    int32_t* ids;
    float* weights;
    QuantJob qj;
    hipStream_t s;
};

template <int V, int GM, bool BIASED>
static hipError_t launch_vgb(const RouteCall& c) {
    const int blocks = (c.M + 3) / 4, routers = blocks < 2048 ? blocks : 2048;
    const size_t qb = c.qj.q ? (c.qj.nblk + 15) / 16 : 0;
    const int quants = qb < 4096 ? (int)qb : 4096;
    hipLaunchKernelGGL((route_grouped_kernel<V, GM, BIASED>), dim3(routers + quants), dim3(256), 0, c.s, c.logits, c.bf16,
                       c.r, c.M, c.E, c.topk, c.ids, c.weights, routers, c.qj);
    return hipGetLastError();
}

template <int V>
static hipError_t launch_v(const RouteCall& c) {
    switch (group_mode(c.r, c.E, V)) {
        case kNoGroups: return c.r.bias ? launch_vgb<V, kNoGroups, true>(c) : launch_vgb<V, kNoGroups, false>(c);
        case kLaneGroups: return c.r.bias ? launch_vgb<V, kLaneGroups, true>(c) : launch_vgb<V, kLaneGroups, false>(c);
        default: return c.r.bias ? launch_vgb<V, kAnyGroups, true>(c) : launch_vgb<V, kAnyGroups, false>(c);
    }
}

hipError_t launch_route_grouped(moe_dtype ldt, const void* logits, const RouteSpec& r, int M, int E, int topk,
                                int32_t* ids, float* weights, hipStream_t s, const void* x, int H, void* xq, float* xs) {
    if (M == 0) return hipSuccess;
    const RouteCall c{logits, ldt == MOE_BF16, r, M, E, topk, ids, weights,
                      QuantJob{static_cast<const uint16_t*>(x), (size_t)M * (H / 128), static_cast<uint8_t*>(xq), xs}, s};
    if (E <= 64) return launch_v<1>(c);
    if (E <= 128) return launch_v<2>(c);
    return launch_v<4>(c);
}

}  // namespace moe
