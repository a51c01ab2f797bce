// Token rows in expert order and back, with the routing weights applied, and
// the gradients (moe_permute, moe_unpermute and their backward calls).
//
//   out of token order:  rows[r(t, j)] = w_tj src[t],  dots[t, j] = <rows_in[r(t, j)], src[t]>
//   back into it:        out[t] = sum_j w_tj rows[r(t, j)],  dots[t, j] = <rows[r(t, j)], x[t]>
//
// r is the place of a pair in the sorted list of the alignment.  The gradient of
// one direction is the other direction plus the dots, so two kernels serve four
// calls.  Both go by tokens: a token's row is read (written) once, whatever topk,
// and its topk expert rows once each, in 16-byte pieces a lane.  Bound by memory.
// (moe_permute of up to 96 MB of rows goes by rows instead: permute_rows_kernel.)
#include "moe_device.h"
#include "moe_launch.h"
#include "moe_train.h"

namespace moe {

// 16 bytes of a row as float32 values: 8 bfloat16 or 4 float32.
template <int DT>
struct Piece {
    static constexpr int N = DT == MOE_BF16 ? 8 : 4;
    float v[N];
    __device__ __forceinline__ static Piece of(const uint4& q) {
        Piece p;
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MOE_BF16) {
                p.v[2 * i] = __uint_as_float(u[i] << 16);
                p.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                p.v[i] = __uint_as_float(u[i]);
            }
        }
        return p;
    }
    __device__ __forceinline__ uint4 pack() const {
        if constexpr (DT == MOE_BF16)
            return uint4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])};
        else
            return uint4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    }
};

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Beyond this many bytes read and written the rows go past the caches (non-temporal
// stores).  Inputs changing from call to call: permute of 4096 x 8 rows of 4 KB 33.5 ->
// 30.5 us, gradient of 4096 x 2 of 8 KB 40.3 -> 37.8; the same inputs again: permute of
// 16384 x 8 of 8 KB 246 -> 218, of 4096 x 8 of 4 KB 26 -> 28.5 (its rows were still cached).
constexpr int64_t kCacheBytes = 96ll << 20;

// Zeroes the padding rows among rows [r0, r0 + 64) of the sorted list: a row
// inside an expert's run (before the padded total) that holds no pair.
__device__ __forceinline__ void zero_padding(const ScatterRows& c, int64_t cap, int64_t r0, int pieces) {
    const int lane = threadIdx.x & 63;
    const int P = c.M * c.topk;
    const int64_t total = min((int64_t)c.al.expert_offsets[c.E], cap);
    const int64_t r = r0 + lane;
    uint64_t pad = __ballot(r < total && (unsigned)c.al.sorted_ids[r] >= (unsigned)P);
    while (pad) {
        const int i = __builtin_ctzll(pad);
        pad &= pad - 1;
        uint4* row = reinterpret_cast<uint4*>(c.rows_out) + (size_t)(r0 + i) * pieces;
        for (int k = threadIdx.x; k < pieces; k += blockDim.x) row[k] = uint4{0, 0, 0, 0};
    }
}

// A workgroup of T threads a token.
template <int DT, int T, bool DOT, bool NT>
__global__ void __launch_bounds__(T) scatter_rows_kernel(ScatterRows c, int pieces, int64_t cap) {
    const int t = blockIdx.x;
    if (t >= c.M) {
        zero_padding(c, cap, (int64_t)(t - c.M) * 64, pieces);
        return;
    }
    __shared__ float part[T / 64][kMaxTopk];
    const int tid = threadIdx.x;
    const uint4* src = reinterpret_cast<const uint4*>(c.src) + (size_t)t * pieces;
    float dot[kMaxTopk];
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j) dot[j] = 0.0f;
    for (int k = tid; k < pieces; k += T) {
        const uint4 q = src[k];
        const auto v = Piece<DT>::of(q);
#pragma unroll
        for (int j = 0; j < kMaxTopk; ++j) {
            if (j >= c.topk) continue;
            const int p = t * c.topk + j;
            const int64_t r = c.pair_row ? c.pair_row[p] : p;
            if (r < 0 || r >= c.nrows) continue;
            const size_t at = (size_t)r * pieces + k;
            if constexpr (DOT) {
                const auto u = Piece<DT>::of(reinterpret_cast<const uint4*>(c.rows_in)[at]);
#pragma unroll
                for (int i = 0; i < Piece<DT>::N; ++i) dot[j] = fmaf(u.v[i], v.v[i], dot[j]);
            }
            uint4 o = q;
            if (c.weights) {
                const float w = c.weights[p];
                auto s = v;
#pragma unroll
                for (int i = 0; i < Piece<DT>::N; ++i) s.v[i] *= w;
                o = s.pack();
            }
            if constexpr (NT)
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o), reinterpret_cast<u32x4*>(c.rows_out) + at);
            else
                reinterpret_cast<uint4*>(c.rows_out)[at] = o;
        }
    }
    if constexpr (DOT) {
#pragma unroll
        for (int j = 0; j < kMaxTopk; ++j) {
            if (j >= c.topk) continue;
            const float s = wave_sum_f32(dot[j]);
            if ((tid & 63) == 0) part[tid >> 6][j] = s;
        }
        __syncthreads();
        if (tid < c.topk) {
            float s = 0.0f;
            for (int w = 0; w < T / 64; ++w) s += part[w][tid];
            c.dots[t * c.topk + tid] = s;
        }
    }
}

template <int DT, int ODT, int T, bool DOT>
__global__ void __launch_bounds__(T) gather_rows_kernel(GatherRows c, int pieces) {
    __shared__ float part[T / 64][kMaxTopk];
    const int t = blockIdx.x, tid = threadIdx.x;
    float dot[kMaxTopk];
#pragma unroll
    for (int j = 0; j < kMaxTopk; ++j) dot[j] = 0.0f;
    for (int k = tid; k < pieces; k += T) {
        Piece<DT> acc, x;
#pragma unroll
        for (int i = 0; i < Piece<DT>::N; ++i) acc.v[i] = 0.0f;
        if constexpr (DOT) x = Piece<DT>::of(reinterpret_cast<const uint4*>(c.x)[(size_t)t * pieces + k]);
#pragma unroll
        for (int j = 0; j < kMaxTopk; ++j) {
            if (j >= c.topk) continue;
            const int p = t * c.topk + j;
            const int64_t r = c.pair_row ? c.pair_row[p] : p;
            if (r < 0 || r >= c.nrows) continue;
            const auto u = Piece<DT>::of(reinterpret_cast<const uint4*>(c.rows)[(size_t)r * pieces + k]);
            const float w = c.weights ? c.weights[p] : 1.0f;
#pragma unroll
            for (int i = 0; i < Piece<DT>::N; ++i) {
                acc.v[i] = fmaf(w, u.v[i], acc.v[i]);
                if constexpr (DOT) dot[j] = fmaf(u.v[i], x.v[i], dot[j]);
            }
        }
        const size_t at = (size_t)t * pieces + k;
        if constexpr (DT == ODT) {
            reinterpret_cast<uint4*>(c.out)[at] = acc.pack();
        } else if constexpr (DT == MOE_BF16) {
            float4* o = reinterpret_cast<float4*>(c.out) + 2 * at;
            o[0] = make_float4(acc.v[0], acc.v[1], acc.v[2], acc.v[3]);
            o[1] = make_float4(acc.v[4], acc.v[5], acc.v[6], acc.v[7]);
        } else {
            reinterpret_cast<uint2*>(c.out)[at] = uint2{pack_bf2(acc.v[0], acc.v[1]), pack_bf2(acc.v[2], acc.v[3])};
        }
    }
    if constexpr (DOT) {
#pragma unroll
        for (int j = 0; j < kMaxTopk; ++j) {
            if (j >= c.topk) continue;
            const float s = wave_sum_f32(dot[j]);
            if ((tid & 63) == 0) part[tid >> 6][j] = s;
        }
        __syncthreads();
        if (tid < c.topk) {
            float s = 0.0f;
            for (int w = 0; w < T / 64; ++w) s += part[w][tid];
            c.dots[t * c.topk + tid] = s;
        }
    }
}

// pair_row from the sorted list: the row of every listed pair, -1 for pairs whose
// id is no expert (they are not listed).  Every entry is written by one thread.
__global__ void __launch_bounds__(256) pair_row_kernel(const int32_t* __restrict__ ids, const int32_t* __restrict__ sorted,
                                                       int P, int E, int64_t cap, int32_t* __restrict__ pair_row) {
    const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (r < P && (unsigned)ids[r] >= (unsigned)E) pair_row[r] = -1;
    if (r < cap) {
        const int p = sorted[r];
        if ((unsigned)p < (unsigned)P) pair_row[p] = (int32_t)r;
    }
}

// The same rows by rows, a workgroup each: one launch, at the price of reading a
// token's row once for each of its pairs.
template <int DT>
__global__ void __launch_bounds__(256) permute_rows_kernel(ScatterRows c, const int32_t* __restrict__ ids,
                                                           int32_t* __restrict__ pair_row, int pieces) {
    const int r = blockIdx.x, P = c.M * c.topk;
    const int p = c.al.sorted_ids[r];
    if (threadIdx.x == 0 && r < P && (unsigned)ids[r] >= (unsigned)c.E) pair_row[r] = -1;
    uint4* row = reinterpret_cast<uint4*>(c.rows_out) + (size_t)r * pieces;
    if ((unsigned)p >= (unsigned)P) {
        if (r < c.al.expert_offsets[c.E])
            for (int k = threadIdx.x; k < pieces; k += 256) row[k] = uint4{0, 0, 0, 0};
        return;
    }
    if (threadIdx.x == 0) pair_row[p] = r;
    const uint4* src = reinterpret_cast<const uint4*>(c.src) + (size_t)(p / c.topk) * pieces;
    const float w = c.weights ? c.weights[p] : 1.0f;
    for (int k = threadIdx.x; k < pieces; k += 256) {
        uint4 q = src[k];
        if (c.weights) {
            auto v = Piece<DT>::of(q);
#pragma unroll
            for (int i = 0; i < Piece<DT>::N; ++i) v.v[i] *= w;
            q = v.pack();
        }
        row[k] = q;
    }
}

static int pieces_of(moe_dtype dt, int H) { return H / (dt == MOE_BF16 ? 8 : 4); }

template <int DT, bool DOT, bool NT>
static hipError_t scatter_t(const ScatterRows& c, hipStream_t s) {
    const int64_t cap = c.al.sorted_ids ? moe_align_capacity(c.M, c.topk, c.E, c.block_m) : 0;
    hipLaunchKernelGGL((scatter_rows_kernel<DT, 256, DOT, NT>), dim3((unsigned)(c.M + (cap + 63) / 64)), dim3(256), 0, s, c,
                       pieces_of(c.dtype, c.H), cap);
    return hipGetLastError();
}

template <int DT>
static hipError_t scatter_dt(const ScatterRows& c, hipStream_t s) {
    const int64_t moved = ((int64_t)c.M + (int64_t)c.M * c.topk * (c.dots ? 2 : 1)) * pieces_of(c.dtype, c.H) * 16;
    const bool nt = moved > kCacheBytes;
    if (c.dots) return nt ? scatter_t<DT, true, true>(c, s) : scatter_t<DT, true, false>(c, s);
    return nt ? scatter_t<DT, false, true>(c, s) : scatter_t<DT, false, false>(c, s);
}

hipError_t launch_scatter_rows(const ScatterRows& c, hipStream_t s) {
    return c.dtype == MOE_BF16 ? scatter_dt<MOE_BF16>(c, s) : scatter_dt<MOE_F32>(c, s);
}

// By rows up to 96 MB of them (1 token 9.3 us against 11.8 by tokens, two launches;
// 1024 x 8 of 4 KB 12.2 against 14.0; 4096 x 2 of 8 KB 20.7 against 25.2), by tokens
// beyond (4096 x 8 of 4 KB 26.3 against 37.5; 16384 x 8 of 8 KB 246 against 338).
template <int DT>
static hipError_t permute_dt(const ScatterRows& c, const int32_t* ids, int32_t* pair_row, hipStream_t s) {
    const int pieces = pieces_of(c.dtype, c.H);
    if (c.nrows * pieces <= (96ll << 20) / 16 && c.nrows < (1 << 24)) {
        hipLaunchKernelGGL((permute_rows_kernel<DT>), dim3((unsigned)c.nrows), dim3(256), 0, s, c, ids, pair_row, pieces);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(pair_row_kernel, dim3((unsigned)((c.nrows + 255) / 256)), dim3(256), 0, s, ids, c.al.sorted_ids,
                       c.M * c.topk, c.E, c.nrows, pair_row);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ScatterRows r = c;
    r.pair_row = pair_row;
    return scatter_dt<DT>(r, s);
}

hipError_t launch_permute(const ScatterRows& c, const int32_t* ids, int32_t* pair_row, hipStream_t s) {
    return c.dtype == MOE_BF16 ? permute_dt<MOE_BF16>(c, ids, pair_row, s) : permute_dt<MOE_F32>(c, ids, pair_row, s);
}

template <int DT, int ODT>
static hipError_t gather_dt(const GatherRows& c, hipStream_t s) {
    const int pieces = pieces_of(c.dtype, c.H);
    if (c.dots)
        hipLaunchKernelGGL((gather_rows_kernel<DT, ODT, 256, true>), dim3(c.M), dim3(256), 0, s, c, pieces);
    else
        hipLaunchKernelGGL((gather_rows_kernel<DT, ODT, 256, false>), dim3(c.M), dim3(256), 0, s, c, pieces);
    return hipGetLastError();
}

hipError_t launch_gather_rows(const GatherRows& c, hipStream_t s) {
    if (c.dtype == MOE_BF16)
        return c.out_dtype == MOE_BF16 ? gather_dt<MOE_BF16, MOE_BF16>(c, s) : gather_dt<MOE_BF16, MOE_F32>(c, s);
    return c.out_dtype == MOE_BF16 ? gather_dt<MOE_F32, MOE_BF16>(c, s) : gather_dt<MOE_F32, MOE_F32>(c, s);
}

}  // namespace moe
