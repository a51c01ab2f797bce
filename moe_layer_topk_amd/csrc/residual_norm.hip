// The norms around a block with its gate and residual scale, in one pass over the
// rows (moe_residual_norm), and their gradients:
//
//   r1 = (mean y^2 + eps)^-1/2    u = y r1 w_post      (no post norm: u = y)
//   h' = h + s g u                r2 = (mean h'^2 + eps)^-1/2    x = h' r2 w_pre
//
// A workgroup holds a row in registers, so every tensor is read and written once
// and what is in place stays right: all of a row is read before any of it is
// written.  h' goes to the second norm in float32, before its own rounding.
// Bound by memory (16 bytes a lane and tensor).
#include "moe_block.h"
#include "moe_launch.h"
#include "moe_train.h"

namespace moe {

template <int DT>
__device__ __forceinline__ void store8(void* x, size_t i, const float (&v)[8]) {
    if constexpr (DT == MOE_F32) {
        float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(x) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(x) + i) =
            uint4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])};
    }
}

__device__ __forceinline__ void load8w(const void* w, bool bf, size_t i, float (&v)[8]) {
    if (bf)
        load8<MOE_BF16>(w, i, v);
    else
        load8<MOE_F32>(w, i, v);
}

__device__ __forceinline__ float load1w(const void* w, bool bf, size_t i) {
    return bf ? bf2f(static_cast<const uint16_t*>(w)[i]) : static_cast<const float*>(w)[i];
}

// Sums of N values over the workgroup of T threads, in every thread.  `slot`
// alternates between calls, so that one barrier a call is enough.
template <int T, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*lds)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) v[n] += __shfl_xor(v[n], off, 64);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) lds[threadIdx.x >> 6][n] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < T / 64; ++w) s += lds[w][n];
            v[n] = s;
        }
    }
}

// T threads, 8 V columns a thread.
template <int DT, int T, int V>
__global__ void __launch_bounds__(T) residual_norm_kernel(NormCall c) {
    __shared__ float lds[2][T / 64][1];
    const int t = blockIdx.x, tid = threadIdx.x;
    const size_t row = (size_t)t * c.H;
    const bool bf = c.n.w_dtype == MOE_BF16;
    float h[V][8], y[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int col = (i * T + tid) * 8;
        if (col < c.H) {
            load8<DT>(c.h, row + col, h[i]);
            if (c.y) load8<DT>(c.y, row + col, y[i]);
        }
    }
    if (c.y) {
        float r1 = 1.0f;
        if (c.n.post_weight) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((i * T + tid) * 8 < c.H)
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[0] = fmaf(y[i][k], y[i][k], s[0]);
            group_sum<T, 1>(s, lds[0]);
            r1 = 1.0f / sqrtf(s[0] / (float)c.H + c.n.eps);
        }
        float g0 = c.n.scale;
        if (c.n.gate && c.n.gate_per_token) g0 *= load1w(c.n.gate, bf, t);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * 8;
            if (col >= c.H) continue;
            float w[8], g[8];
            if (c.n.post_weight) load8w(c.n.post_weight, bf, col, w);
            if (c.n.gate && !c.n.gate_per_token) load8w(c.n.gate, bf, col, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float u = y[i][k];
                if (c.n.post_weight) u = u * r1 * w[k];
                u *= g0;
                if (c.n.gate && !c.n.gate_per_token) u *= g[k];
                h[i][k] += u;
            }
            store8<DT>(c.h_out, row + col, h[i]);
        }
    }
    if (c.n.pre_weight) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((i * T + tid) * 8 < c.H)
#pragma unroll
                for (int k = 0; k < 8; ++k) s[0] = fmaf(h[i][k], h[i][k], s[0]);
        group_sum<T, 1>(s, lds[1]);
        const float r2 = 1.0f / sqrtf(s[0] / (float)c.H + c.n.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * 8;
            if (col >= c.H) continue;
            float w[8], o[8];
            load8w(c.n.pre_weight, bf, col, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = h[i][k] * r2 * w[k];
            store8<DT>(c.x, row + col, o);
        }
    }
}

// Gradients.  With n = v r the normed row of v and q = d w the gradient at n,
// the gradient of v is r (q - n mean(q n)), and w's is the sum over rows of d n.
// A workgroup takes rows t, t + groups, ... and keeps its part of the three column
// sums in registers; norm_parts_kernel adds the parts in order.
template <int DT, int T, int V>
__global__ void __launch_bounds__(T) residual_norm_backward_kernel(NormGrad c) {
    __shared__ float lds1[2][T / 64][3];
    __shared__ float lds2[2][T / 64][2];
    const int tid = threadIdx.x;
    const bool bf = c.n.w_dtype == MOE_BF16;
    const bool pre = c.n.pre_weight != nullptr, post = c.n.post_weight != nullptr;
    const bool gate_c = c.n.gate && !c.n.gate_per_token, gate_t = c.n.gate && c.n.gate_per_token;
    const float inv_h = 1.0f / (float)c.H;
    float apost[V][8], agate[V][8], apre[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) apost[i][k] = agate[i][k] = apre[i][k] = 0.0f;
    int odd = 0;
    for (int t = blockIdx.x; t < c.M; t += gridDim.x, odd ^= 1) {
        const size_t row = (size_t)t * c.H;
        float y[V][8], h[V][8], dx[V][8], dh[V][8];
        float s[3] = {0.0f, 0.0f, 0.0f};  // y^2, h'^2, dx w_pre h'
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) y[i][k] = h[i][k] = dx[i][k] = dh[i][k] = 0.0f;
            if (col >= c.H) continue;
            if (pre) load8<DT>(c.h_out, row + col, h[i]);
            if (pre) load8<DT>(c.dx, row + col, dx[i]);
            if (c.dh_out) load8<DT>(c.dh_out, row + col, dh[i]);
            if (c.y) load8<DT>(c.y, row + col, y[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * 8;
            float w[8];
            if (pre && col < c.H) load8w(c.n.pre_weight, bf, col, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[0] = fmaf(y[i][k], y[i][k], s[0]);
                if (pre && col < c.H) {
                    s[1] = fmaf(h[i][k], h[i][k], s[1]);
                    s[2] = fmaf(dx[i][k] * w[k], h[i][k], s[2]);
                }
            }
        }
        group_sum<T, 3>(s, lds1[odd]);
        const float r1 = post ? 1.0f / sqrtf(s[0] * inv_h + c.n.eps) : 1.0f;
        if (pre) {
            const float r2 = 1.0f / sqrtf(s[1] * inv_h + c.n.eps);
            const float m = s[2] * r2 * inv_h;  // mean of q n
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int col = (i * T + tid) * 8;
                if (col >= c.H) continue;
                float w[8];
                load8w(c.n.pre_weight, bf, col, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float n = h[i][k] * r2;
                    apre[i][k] = fmaf(dx[i][k], n, apre[i][k]);
                    dh[i][k] += r2 * (dx[i][k] * w[k] - n * m);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * 8;
            if (col < c.H) store8<DT>(c.dh, row + col, dh[i]);
        }
        if (!c.y) continue;
        // du = s g dh'; through the post norm
        float s2[2] = {0.0f, 0.0f};  // du w_post y r1, s dh' u
        const float gt = gate_t ? load1w(c.n.gate, bf, t) : 1.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * 8;
            if (col >= c.H) continue;
            float w[8], g[8];
            if (post) load8w(c.n.post_weight, bf, col, w);
            if (gate_c) load8w(c.n.gate, bf, col, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float n = y[i][k] * r1, u = post ? n * w[k] : n;
                const float d = c.n.scale * dh[i][k];  // at g u
                agate[i][k] = fmaf(d, u, agate[i][k]);
                s2[1] = fmaf(d, u, s2[1]);
                const float du = d * (gate_c ? g[k] : gt);
                apost[i][k] = fmaf(du, n, apost[i][k]);
                const float q = post ? du * w[k] : du;
                s2[0] = fmaf(q, n, s2[0]);
                dh[i][k] = q;
            }
        }
        if (post || gate_t) group_sum<T, 2>(s2, lds2[odd]);
        const float m = post ? s2[0] * inv_h : 0.0f;
        if (gate_t && tid == 0 && c.dgate) c.dgate[t] = s2[1];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * 8;
            if (col >= c.H) continue;
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = post ? r1 * (dh[i][k] - y[i][k] * r1 * m) : dh[i][k];
            store8<DT>(c.dy, row + col, o);
        }
    }
    float* part = c.part + (size_t)blockIdx.x * 3 * c.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int col = (i * T + tid) * 8;
        if (col >= c.H) continue;
        if (c.dpost) store8<MOE_F32>(part, col, apost[i]);
        if (c.dgate && gate_c) store8<MOE_F32>(part, (size_t)c.H + col, agate[i]);
        if (c.dpre) store8<MOE_F32>(part, (size_t)2 * c.H + col, apre[i]);
    }
}

// Sums of the groups' parts: blockIdx.y the vector, a thread a column.
__global__ void __launch_bounds__(64) norm_parts_kernel(const float* __restrict__ part, int groups, int H, float* dpost,
                                                        float* dgate, float* dpre) {
    float* out = blockIdx.y == 0 ? dpost : blockIdx.y == 1 ? dgate : dpre;
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (!out || col >= H) return;
    float s = 0.0f;
    for (int g = 0; g < groups; ++g) s += part[((size_t)g * 3 + blockIdx.y) * H + col];
    out[col] = s;
}

template <int DT, int T, int V>
static hipError_t norm_tv(const NormCall& c, hipStream_t s) {
    hipLaunchKernelGGL((residual_norm_kernel<DT, T, V>), dim3(c.M), dim3(T), 0, s, c);
    return hipGetLastError();
}

template <int DT>
static hipError_t norm_dt(const NormCall& c, hipStream_t s) {
    if (c.H <= 512) return norm_tv<DT, 64, 1>(c, s);
    if (c.H <= 2048) return norm_tv<DT, 256, 1>(c, s);
    if (c.H <= 4096) return norm_tv<DT, 512, 1>(c, s);
    if (c.H <= 8192) return norm_tv<DT, 1024, 1>(c, s);
    return norm_tv<DT, 1024, 2>(c, s);
}

hipError_t launch_residual_norm(const NormCall& c, hipStream_t s) {
    return c.dtype == MOE_BF16 ? norm_dt<MOE_BF16>(c, s) : norm_dt<MOE_F32>(c, s);
}

int norm_grad_groups(int M, int H) { return M < 512 ? M : 512; }

template <int DT, int T, int V>
static hipError_t grad_tv(const NormGrad& c, int groups, hipStream_t s) {
    hipLaunchKernelGGL((residual_norm_backward_kernel<DT, T, V>), dim3(groups), dim3(T), 0, s, c);
    return hipGetLastError();
}

template <int DT>
static hipError_t grad_dt(const NormGrad& c, int groups, hipStream_t s) {
    if (c.H <= 512) return grad_tv<DT, 64, 1>(c, groups, s);
    if (c.H <= 2048) return grad_tv<DT, 256, 1>(c, groups, s);
    if (c.H <= 4096) return grad_tv<DT, 512, 1>(c, groups, s);
    if (c.H <= 8192) return grad_tv<DT, 1024, 1>(c, groups, s);
    return grad_tv<DT, 1024, 2>(c, groups, s);
}

hipError_t launch_residual_norm_backward(const NormGrad& c, hipStream_t s) {
    const int groups = norm_grad_groups(c.M, c.H);
    hipError_t e = c.dtype == MOE_BF16 ? grad_dt<MOE_BF16>(c, groups, s) : grad_dt<MOE_F32>(c, groups, s);
    if (e != hipSuccess) return e;
    float* dgate = c.n.gate_per_token ? nullptr : c.dgate;
    if (!c.dpost && !dgate && !c.dpre) return hipSuccess;
    hipLaunchKernelGGL(norm_parts_kernel, dim3((c.H + 63) / 64, 3), dim3(64), 0, s, c.part, groups, c.H, c.dpost, dgate,
                       c.dpre);
    return hipGetLastError();
}

__global__ void __launch_bounds__(256) zero_kernel(uint4* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = uint4{0, 0, 0, 0};
}

hipError_t launch_zero(void* p, size_t bytes, hipStream_t s) {
    const size_t n = bytes / 16, blocks = (n + 255) / 256;
    if (!n) return hipSuccess;
    hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s, static_cast<uint4*>(p), n);
    return hipGetLastError();
}

}  // namespace moe
