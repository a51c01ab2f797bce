// Grouped router: softmax or sigmoid scores, a bias that only the choice
// sees, groups of experts, top-k, renormalised weights (moe_route_grouped).
#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

// One wavefront per token, lane l holding experts l, l + 64, l + 128, l + 192.
__device__ __forceinline__ float logit_at(const void* logits, int dt, size_t i) {
    const float v = dt == MOE_BF16 ? bf2f(reinterpret_cast<const uint16_t*>(logits)[i])
                                   : reinterpret_cast<const float*>(logits)[i];
    return v == v ? v : -__builtin_inff();  // NaN counts as -inf
}

// the larger value, the lower index among equals; index INT_MAX: nothing
__device__ __forceinline__ void wave_argmax(double& v, int& i) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const double ov = __shfl_xor(v, off, 64);
        const int oi = __shfl_xor(i, off, 64);
        if (oi != 0x7fffffff && (i == 0x7fffffff || ov > v || (ov == v && oi < i))) {
            v = ov;
            i = oi;
        }
    }
}

__global__ void __launch_bounds__(256) route_grouped_kernel(const void* __restrict__ logits, int dt, RouteSpec r, int M,
                                                            int E, int topk, int32_t* __restrict__ ids,
                                                            float* __restrict__ weights) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= M) return;
    const float ninf = -__builtin_inff();
    float l[4];
    double s[4], c[4], rank[4];
    bool live[4];
    float m = ninf;
    for (int q = 0; q < 4; ++q) {
        const int e = lane + 64 * q;
        live[q] = e < E;
        l[q] = live[q] ? logit_at(logits, dt, (size_t)t * E + e) : ninf;
        m = fmaxf(m, l[q]);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    double den = 0.0;
    for (int q = 0; q < 4; ++q) {
        if (r.score == MOE_SCORE_SIGMOID)
            s[q] = 1.0 / (1.0 + exp(-(double)l[q]));
        else  // (an infinite maximum: 1 at it, 0 elsewhere; nothing above -inf: all 0)
            s[q] = m == ninf ? 0.0 : l[q] == m ? 1.0 : exp((double)l[q] - (double)m);
        if (!live[q]) s[q] = 0.0;
        den += s[q];
    }
    if (r.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) den += __shfl_xor(den, off, 64);
        for (int q = 0; q < 4; ++q) s[q] = den > 0.0 ? s[q] / den : 0.0;
    }
    for (int q = 0; q < 4; ++q) {
        c[q] = s[q] + ((r.bias && live[q]) ? (double)r.bias[lane + 64 * q] : 0.0);
        if (c[q] != c[q]) c[q] = (double)ninf;
        rank[q] = r.bias ? c[q] : (double)l[q];
    }
    if (r.topk_groups < r.n_groups) {
        const int gs = E / r.n_groups;
        double mine = (double)ninf;  // lane g: the score of group g
        for (int g = 0; g < r.n_groups; ++g) {
            bool left[4];
            for (int q = 0; q < 4; ++q) left[q] = live[q] && (lane + 64 * q) / gs == g;
            double sum = 0.0;
            for (int k = 0; k < r.group_top; ++k) {
                double bv = (double)ninf;
                int bi = 0x7fffffff;
                for (int q = 0; q < 4; ++q)
                    if (left[q] && (bi == 0x7fffffff || c[q] > bv)) {
                        bv = c[q];
                        bi = lane + 64 * q;
                    }
                wave_argmax(bv, bi);
                for (int q = 0; q < 4; ++q)
                    if (lane + 64 * q == bi) left[q] = false;
                sum += bv;
            }
            if (sum != sum) sum = (double)ninf;
            if (lane == g) mine = sum;
        }
        bool open = lane < r.n_groups;
        uint64_t kept = 0;
        for (int k = 0; k < r.topk_groups; ++k) {
            double bv = mine;
            int bi = open ? lane : 0x7fffffff;
            wave_argmax(bv, bi);
            if (lane == bi) open = false;
            kept |= 1ull << bi;
        }
        for (int q = 0; q < 4; ++q) live[q] = live[q] && ((kept >> ((lane + 64 * q) / gs)) & 1);
    }
    double w = 0.0;
    int sel = 0;
    for (int j = 0; j < topk; ++j) {
        double bv = (double)ninf;
        int bi = 0x7fffffff;
        for (int q = 0; q < 4; ++q)
            if (live[q] && (bi == 0x7fffffff || rank[q] > bv)) {
                bv = rank[q];
                bi = lane + 64 * q;
            }
        wave_argmax(bv, bi);
        double sv = 0.0;
        for (int q = 0; q < 4; ++q)
            if (lane + 64 * q == bi) {
                live[q] = false;
                sv = s[q];
            }
        sv = __shfl(sv, bi & 63, 64);
        if (lane == j) {
            w = sv;
            sel = bi;
        }
    }
    if (r.renormalize) {
        double sum = lane < topk ? w : 0.0;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < topk) {
        ids[(size_t)t * topk + lane] = sel;
        weights[(size_t)t * topk + lane] = (float)(w * (double)r.scale);
    }
}

hipError_t launch_route_grouped(moe_dtype ldt, const void* logits, const RouteSpec& r, int M, int E, int topk,
                                int32_t* ids, float* weights, hipStream_t s) {
    if (M == 0) return hipSuccess;
    hipLaunchKernelGGL(route_grouped_kernel, dim3((M + 3) / 4), dim3(256), 0, s, logits, (int)ldt, r, M, E, topk, ids,
                       weights);
    return hipGetLastError();
}

}  // namespace moe
