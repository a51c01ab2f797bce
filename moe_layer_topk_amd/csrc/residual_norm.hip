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
#include <algorithm>

#include "moe_block.h"
#include "moe_launch.h"
#include "moe_train.h"

namespace moe {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Rows are stored with the non-temporal hint: 16384 x 4096 bfloat16 rows 111 -> 94
// us, the gradient at 4096 rows 47.8 -> 46.4 (the same hint on the loads: 107, 50).
template <int DT>
__device__ __forceinline__ void store8(void* x, size_t i, const float (&v)[8]) {
    if constexpr (DT == MOE_F32) {
        u32x4* p = reinterpret_cast<u32x4*>(reinterpret_cast<float*>(x) + i);
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, make_float4(v[0], v[1], v[2], v[3])), p);
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, make_float4(v[4], v[5], v[6], v[7])), p + 1);
    } else {
        __builtin_nontemporal_store(u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])},
                                    reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(x) + i));
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

// Sums of N values over the workgroup of T threads, in every thread, in a fixed
// order.  A caller alternates between two `lds`, so that one barrier a call is
// enough.
template <int T, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*lds)[T / 64]) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_sum_f32(v[n]);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) lds[n][threadIdx.x >> 6] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < T / 64; ++w) s += lds[n][w];
            v[n] = s;
        }
    }
}

// T threads, 8 V columns a thread.
template <int DT, int T, int V>
__global__ void __launch_bounds__(T) residual_norm_kernel(NormCall c) {
    __shared__ __attribute__((aligned(16))) float lds[2][1][T / 64];
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

// 16 bytes of a row as loaded: 8 bfloat16 or 4 float32 values.
template <int DT>
struct Raw {
    static constexpr int E = DT == MOE_F32 ? 4 : 8;
    uint4 q;
    __device__ __forceinline__ void load(const void* x, size_t i) {
        q = *reinterpret_cast<const uint4*>(static_cast<const char*>(x) + i * (16 / E));
    }
    __device__ __forceinline__ void zero() { q = uint4{0, 0, 0, 0}; }
    __device__ __forceinline__ float at(int k) const {
        const int n = DT == MOE_F32 ? k : k / 2;
        const uint32_t w = n == 0 ? q.x : n == 1 ? q.y : n == 2 ? q.z : q.w;
        if constexpr (DT == MOE_F32) return __uint_as_float(w);
        return __uint_as_float((k & 1) ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ static void store(void* x, size_t i, const float (&v)[E]) {
        u32x4 o;
        if constexpr (DT == MOE_F32)
            o = __builtin_bit_cast(u32x4, make_float4(v[0], v[1], v[2], v[3]));
        else
            o = u32x4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4 % E], v[5 % E]), pack_bf2(v[6 % E], v[7 % E])};
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(static_cast<char*>(x) + i * (16 / E)));
    }
};

// E (8 or 4) weights.
template <int E>
__device__ __forceinline__ void load_w(const void* w, bool bf, size_t i, float* v) {
#pragma unroll
    for (int k = 0; k < E; k += 4) {
        if (bf) {
            const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + i + k);
            v[k] = __uint_as_float(a.x << 16), v[k + 1] = __uint_as_float(a.x & 0xffff0000u);
            v[k + 2] = __uint_as_float(a.y << 16), v[k + 3] = __uint_as_float(a.y & 0xffff0000u);
        } else {
            const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + i + k);
            v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
        }
    }
}

template <int E>
__device__ __forceinline__ void store_part(float* x, const float (&v)[E]) {
#pragma unroll
    for (int k = 0; k < E; k += 4) *reinterpret_cast<float4*>(x + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
}

// The rows a thread of the gradient kernel reads: its columns of h', dx, dh' and y.
template <int DT, int T, int V, bool FULL>
struct GradRow {
    Raw<DT> h[V], dx[V], dh[V], y[V];
    __device__ __forceinline__ void load(const NormGrad& c, int t, bool pre) {
        const size_t row = (size_t)t * c.H;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + (int)threadIdx.x) * Raw<DT>::E;
            if constexpr (FULL) {
                h[i].load(c.h_out, row + col), dx[i].load(c.dx, row + col);
                dh[i].load(c.dh_out, row + col), y[i].load(c.y, row + col);
                continue;
            }
            const bool in = col < c.H;
            if (in && pre) h[i].load(c.h_out, row + col), dx[i].load(c.dx, row + col);
            else h[i].zero(), dx[i].zero();
            if (in && c.dh_out) dh[i].load(c.dh_out, row + col);
            else dh[i].zero();
            if (in && c.y) y[i].load(c.y, row + col);
            else y[i].zero();
        }
    }
};

// Gradients.  With n = v r the normed row of v and q = d w the gradient at n,
// the gradient of v is r (q - n mean(q n)), and w's is the sum over rows of d n.
// At the block d = s dh' (times the token's gate), q = d g w_post, and one column sum
// S = sum d n gives both dw_post = g S and dg = w_post S (a gate a column).
//
// A workgroup takes rows t, t + groups, ... and keeps its part of the two column sums
// in registers; norm_parts_kernel adds the parts in order.  kHold: the weights stay in
// registers and the next row is on its way while this one waits for its sums (a row
// may be written over one of its inputs, never over another row's).  FULL: everything
// is there (both norms' gradients and the stream's, no gate a token) and a row fills
// the workgroup, so that no load or store hangs on a condition: with one pending, the
// compiler waits for the next row and the stores too.  (The fused multiply-adds are
// spelled out, so that both forms round alike.)
template <int DT, int T, int V, int W, bool kHold, bool FULL>
__global__ void __launch_bounds__(T, W) residual_norm_backward_kernel(NormGrad c) {
    __shared__ __attribute__((aligned(16))) float lds1[2][3][T / 64];
    __shared__ __attribute__((aligned(16))) float lds2[2][2][T / 64];
    constexpr int E = Raw<DT>::E;
    const int tid = threadIdx.x;
    const bool bf = c.n.w_dtype == MOE_BF16;
    const bool pre = FULL || c.n.pre_weight != nullptr, post = c.n.post_weight != nullptr;
    const bool gate_c = c.n.gate && (FULL || !c.n.gate_per_token), gate_t = !FULL && c.n.gate && c.n.gate_per_token;
    const float inv_h = 1.0f / (float)c.H;
    // w_pre, and w_post times the column's gate
    auto load_weights = [&](int col, float* wpre, float* wq) {
        float g[E];
#pragma unroll
        for (int k = 0; k < E; ++k) wpre[k] = wq[k] = g[k] = 1.0f;
        if (pre) load_w<E>(c.n.pre_weight, bf, col, wpre);
        if (post) load_w<E>(c.n.post_weight, bf, col, wq);
        if (gate_c) load_w<E>(c.n.gate, bf, col, g);
#pragma unroll
        for (int k = 0; k < E; ++k) wq[k] *= g[k];
    };
    constexpr int VW = kHold ? V : 1;
    float wpre[VW][E], wq[VW][E];
    if constexpr (kHold) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * E;
#pragma unroll
            for (int k = 0; k < E; ++k) wpre[i][k] = wq[i][k] = 0.0f;
            if (FULL || col < c.H) load_weights(col, wpre[i], wq[i]);
        }
    }
    float apre[V][E], ablk[V][E];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < E; ++k) apre[i][k] = ablk[i][k] = 0.0f;
    GradRow<DT, T, V, FULL> in, next;
    if (kHold && (int)blockIdx.x < c.M) next.load(c, blockIdx.x, pre);
    int odd = 0;
    for (int t = blockIdx.x; t < c.M; t += gridDim.x, odd ^= 1) {
        const size_t row = (size_t)t * c.H;
        if constexpr (kHold) {
            in = next;
            if (t + (int)gridDim.x < c.M) next.load(c, t + gridDim.x, pre);
        } else {
            in.load(c, t, pre);
        }
        float s[3] = {0.0f, 0.0f, 0.0f};  // y^2, h'^2, dx w_pre h'
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * E;
            if (!FULL && col >= c.H) continue;
            if constexpr (!kHold) load_weights(col, wpre[0], wq[0]);
            const float* w = wpre[kHold ? i : 0];
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float y = in.y[i].at(k), h = in.h[i].at(k);
                s[0] = fmaf(y, y, s[0]);
                s[1] = fmaf(h, h, s[1]);
                s[2] = fmaf(in.dx[i].at(k) * w[k], h, s[2]);
            }
        }
        group_sum<T, 3>(s, lds1[odd]);
        const float r1 = post ? 1.0f / sqrtf(fmaf(s[0], inv_h, c.n.eps)) : 1.0f;
        const float r2 = pre ? 1.0f / sqrtf(fmaf(s[1], inv_h, c.n.eps)) : 0.0f;
        const float m2 = s[2] * r2 * inv_h;  // mean of q n at the second norm
        const float gt = c.n.scale * (gate_t ? load1w(c.n.gate, bf, t) : 1.0f);
        float s2[2] = {0.0f, 0.0f};  // q n at the first norm, s dh' u
        float d[V][E];               // q there
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * E;
            if (!FULL && col >= c.H) continue;
            if constexpr (!kHold) load_weights(col, wpre[0], wq[0]);
            const float *w = wpre[kHold ? i : 0], *v = wq[kHold ? i : 0];
            float dh[E];
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float n = in.h[i].at(k) * r2, x = in.dx[i].at(k);  // (no second norm: 0)
                apre[i][k] = fmaf(x, n, apre[i][k]);
                dh[k] = fmaf(r2, fmaf(-n, m2, x * w[k]), in.dh[i].at(k));
            }
            Raw<DT>::store(c.dh, row + col, dh);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float n = in.y[i].at(k) * r1, e = gt * dh[k];
                ablk[i][k] = fmaf(e, n, ablk[i][k]);
                d[i][k] = e * v[k];
                s2[0] = fmaf(d[i][k], n, s2[0]);
                if (gate_t) s2[1] = fmaf(c.n.scale * dh[k] * v[k], n, s2[1]);
            }
        }
        if (!FULL && !c.y) continue;
        if (FULL || post || gate_t) group_sum<T, 2>(s2, lds2[odd]);
        const float m1 = post ? s2[0] * inv_h * r1 : 0.0f;
        if (gate_t && tid == 0 && c.dgate) c.dgate[t] = s2[1];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = (i * T + tid) * E;
            if (!FULL && col >= c.H) continue;
            float o[E];
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = r1 * fmaf(-in.y[i].at(k), m1, d[i][k]);  // (no post norm: r1 = 1, m1 = 0)
            Raw<DT>::store(c.dy, row + col, o);
        }
    }
    float* part = c.part + (size_t)blockIdx.x * 2 * c.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int col = (i * T + tid) * E;
        if (!FULL && col >= c.H) continue;
        if (c.dpre) store_part(part + col, apre[i]);
        if (c.dpost || (c.dgate && gate_c)) store_part(part + c.H + col, ablk[i]);
    }
}

// Sums of the groups' parts: blockIdx.y 0 the second norm's weight, 1 the block's sum,
// times the gate and the first norm's weight.  16 lanes take 64 columns, 64 slices of
// the groups meet in LDS, all in a fixed order.
__global__ void __launch_bounds__(1024) norm_parts_kernel(NormGrad c, int groups) {
    __shared__ float lds[64][64];
    const bool pre = blockIdx.y == 0, bf = c.n.w_dtype == MOE_BF16;
    if (pre ? !c.dpre : !c.dpost && !(c.dgate && !c.n.gate_per_token)) return;
    const int H = c.H, slice = threadIdx.x >> 4, c4 = (threadIdx.x & 15) * 4, col = blockIdx.x * 64 + c4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < H) {
        const float* p = c.part + (size_t)blockIdx.y * H + col;
#pragma unroll 8
        for (int g = slice; g < groups; g += 64) {
            const float4 v = *reinterpret_cast<const float4*>(p + (size_t)g * 2 * H);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    *reinterpret_cast<float4*>(&lds[slice][c4]) = s;
    __syncthreads();
    const int o = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && o < H) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) t += lds[i][threadIdx.x];
        if (pre) {
            c.dpre[o] = t;
        } else {
            const bool gate_c = c.n.gate && !c.n.gate_per_token;
            if (c.dpost) c.dpost[o] = gate_c ? t * load1w(c.n.gate, bf, o) : t;
            if (c.dgate && gate_c) c.dgate[o] = c.n.post_weight ? t * load1w(c.n.post_weight, bf, o) : t;
        }
    }
}

template <int DT, int T, int V>
static hipError_t norm_tv(const NormCall& c, hipStream_t s) {
    hipLaunchKernelGGL((residual_norm_kernel<DT, T, V>), dim3(c.M), dim3(T), 0, s, c);
    return hipGetLastError();
}

template <int DT>
static hipError_t norm_dt(const NormCall& c, hipStream_t s) {
    // Two pieces a thread for bfloat16, one for float32 (64 Mi elements, h and y in,
    // h_out and x out, H = 4096: bfloat16 76 us, one piece 99, four 80; float32 one 195
    // at H = 2048, two 207)
    constexpr int V = DT == MOE_BF16 ? 2 : 1;
    if (c.H <= 512 * V) return norm_tv<DT, 64, V>(c, s);
    if (c.H <= 1024 * V) return norm_tv<DT, 128, V>(c, s);
    if (c.H <= 2048 * V) return norm_tv<DT, 256, V>(c, s);
    if (c.H <= 4096 * V) return norm_tv<DT, 512, V>(c, s);
    if (c.H <= 8192 * V) return norm_tv<DT, 1024, V>(c, s);
    return norm_tv<DT, 1024, 2>(c, s);
}

hipError_t launch_residual_norm(const NormCall& c, hipStream_t s) {
    return c.dtype == MOE_BF16 ? norm_dt<MOE_BF16>(c, s) : norm_dt<MOE_F32>(c, s);
}

// Workgroups of the gradient kernel: two of 512 threads a CU, as many threads of
// smaller ones (at 4096 x 4096, with a third column sum, 512 groups 45 us, 256 49, 768
// 53; now 40), but eight rows each where
// there are rows enough, since every group leaves 8 bytes a column to be added.
int norm_grad_groups(int M, int H) {
    const int most = H > 2048 ? 512 : 1024;
    const int g = M / 8 < 256 ? 256 : M / 8;
    return std::min(M, std::min(g, most));
}

template <int DT, int T, int V, int W, bool kHold>
static hipError_t grad_tv(const NormGrad& c, int groups, hipStream_t s) {
    if constexpr (kHold) {
        if (c.H == T * V * Raw<DT>::E && c.n.pre_weight && c.y && c.dh_out && !(c.n.gate && c.n.gate_per_token)) {
            hipLaunchKernelGGL((residual_norm_backward_kernel<DT, T, V, W, true, true>), dim3(groups), dim3(T), 0, s, c);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((residual_norm_backward_kernel<DT, T, V, W, kHold, false>), dim3(groups), dim3(T), 0, s, c);
    return hipGetLastError();
}

// One 16-byte piece a thread, the weights and the next row in registers (4096 x 4096
// bfloat16 with three column sums: 45 us, without the next row 47, without either 49,
// two pieces a thread 47-97; FULL and two sums: 41 us, 4.9 TB/s, and 47 on inputs that
// change from call to call), until a workgroup has no more threads.
template <int DT>
static hipError_t grad_dt(const NormGrad& c, int groups, hipStream_t s) {
    constexpr int E = Raw<DT>::E;
    if (c.H <= 64 * E) return grad_tv<DT, 64, 1, 4, true>(c, groups, s);
    if (c.H <= 128 * E) return grad_tv<DT, 128, 1, 4, true>(c, groups, s);
    if (c.H <= 256 * E) return grad_tv<DT, 256, 1, 4, true>(c, groups, s);
    if (c.H <= 512 * E) return grad_tv<DT, 512, 1, 4, true>(c, groups, s);
    if (c.H <= 1024 * E) return grad_tv<DT, 1024, 1, 4, true>(c, groups, s);
    // longer rows: pieces in a line, half as many wavefronts with all of the
    // registers (16384 columns, 1024 rows: bfloat16 68 us, float32 147; with a third
    // column sum 102 and 188, on 1024 threads, which spill registers, 147 and 210)
    if (DT == MOE_F32 && c.H <= 2048 * E) return grad_tv<DT, 512, 4, 2, false>(c, groups, s);
    return grad_tv<DT, 512, DT == MOE_F32 ? 8 : 4, 2, false>(c, groups, s);
}

hipError_t launch_residual_norm_backward(const NormGrad& c, hipStream_t s) {
    const int groups = norm_grad_groups(c.M, c.H);
    hipError_t e = c.dtype == MOE_BF16 ? grad_dt<MOE_BF16>(c, groups, s) : grad_dt<MOE_F32>(c, groups, s);
    if (e != hipSuccess) return e;
    const bool block = c.dpost || (c.dgate && !c.n.gate_per_token);
    if (!block && !c.dpre) return hipSuccess;
    hipLaunchKernelGGL(norm_parts_kernel, dim3((c.H + 63) / 64, 2), dim3(1024), 0, s, c, groups);
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
