// The grouped router of one token (moe_route_grouped), by one wavefront.
//
// Lane l holds the V = ceil(E / 64) (1, 2 or 4) consecutive experts V l ..
// V l + V - 1, so lanes in order are experts in order and the lowest lane of a
// ballot is the lowest index.  Steps: scores; group scores (the two best
// choices of a group merge across its lanes); every group's rank among the
// groups; a stable sort of the lane's V candidates; topk rounds that take the
// best head of the 64 sorted lists and pop it.
//
// The choice has to be the one of float64 scores.  The float32 pass bounds its
// own error: with eta the bound of one choice, two that differ by more than
// 4 eta are ordered as in float64.  A token with a closer pair at a place that
// matters (neighbours among the taken, the best one left, two groups) is done
// again in float64.  Without a bias experts are ranked by their logits, exactly,
// ties included.
//   One eta serves all comparisons of a token: it is as wide as the largest |bias|
// makes it, and as coarse as 2^-22 beside scores that saturate.  Tokens repeated
// in float64, 256 experts in 8 groups: 0.1% on standard normal logits with biases
// of 0.05, 0.2% (softmax with biases of 0.002: 2%) at a deviation of 6 or 10; at 6
// with biases of 0 97% of the sigmoids' and 20% of the softmaxes', without a bias
// 54% and 14%; with one expert disabled by a bias of -1e4 87 to 100%, of -1e9 or
// -inf all.  A repeated batch takes twice as long (16384 tokens: sigmoid 22 us and
// 46, softmax 27 and 50).
//   sigmoid: 1 / (1 + e), e = exp2(-l log2 e): the argument's rounding costs
//     |l| 2^-24, the exponential 2^-23, and s (1 - s) |l| <= 0.23; with the sum
//     and the reciprocal below 4 x 2^-24, plus the sum's with the bias.
//   softmax: numerators (2 |l - m| + 2) 2^-24, their sum at most
//     (2 ln E + 10) 2^-24 of itself: below 2^-19 of the largest probability.
#pragma once

#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

// ordered integer keys; 0 is left for "nothing here"
template <typename T>
struct RankKey;
template <>
struct RankKey<float> {
    using key = unsigned;
    __device__ static __forceinline__ key of(float v) { return order_key(v); }
    __device__ static __forceinline__ key wave_max(key k) { return wave_max_u32(k); }
    __device__ static __forceinline__ float value(key k) { return key_value(k); }
    __device__ static __forceinline__ key max2(key a, key b) { return a > b ? a : b; }
    __device__ static __forceinline__ key min2(key a, key b) { return a < b ? a : b; }
};
template <>
struct RankKey<double> {
    using key = unsigned long long;
    __device__ static __forceinline__ key of(double v) {
        const key b = (key)__double_as_longlong(v == 0.0 ? 0.0 : v);
        return (b >> 63) ? ~b : (b | (1ull << 63));
    }
    __device__ static __forceinline__ key wave_max(key k) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const key o = (key)__shfl_xor((long long)k, off, 64);
            k = o > k ? o : k;
        }
        return k;
    }
    __device__ static __forceinline__ double value(key k) {
        return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
    }
    __device__ static __forceinline__ key max2(key a, key b) { return a > b ? a : b; }
    __device__ static __forceinline__ key min2(key a, key b) { return a < b ? a : b; }
};

// v of the lane whose number differs in bit `step` from this one's.  Steps 0
// to 3 of float values are lane moves on the vector ALU: quad swaps, and
// mirrors, which are the same thing once every smaller step has been merged.
__device__ __forceinline__ float lane_swap(float v, int step) {
    const int i = __float_as_int(v);
    switch (step) {
        case 0: return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0xB1, 0xF, 0xF, false));
        case 1: return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x4E, 0xF, 0xF, false));
        case 2: return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x141, 0xF, 0xF, false));
        case 3: return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x140, 0xF, 0xF, false));
        default: return __shfl_xor(v, 1 << step, 64);
    }
}
__device__ __forceinline__ unsigned lane_swap(unsigned v, int step) {
    return __float_as_uint(lane_swap(__uint_as_float(v), step));
}
__device__ __forceinline__ double lane_swap(double v, int step) { return __shfl_xor(v, 1 << step, 64); }
__device__ __forceinline__ unsigned long long lane_swap(unsigned long long v, int step) {
    return (unsigned long long)__shfl_xor((long long)v, 1 << step, 64);
}

__device__ __forceinline__ float lane_read(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_read(double v, int lane) {
    const long long b = __double_as_longlong(v);
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)b, lane), hi = (unsigned)__builtin_amdgcn_readlane((int)(b >> 32), lane);
    return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}

__device__ __forceinline__ float wave_max_f32(float v) { return key_value(wave_max_u32(order_key(v))); }

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int step = 0; step < 6; ++step) v += lane_swap(v, step);
    return v;
}

// The V logits of this lane, NaN as -inf, lanes past E -inf.
template <int V>
__device__ __forceinline__ void load_logits(const void* logits, bool bf16, size_t row, int E, float (&l)[V]) {
    const int e0 = V * (int)__lane_id();
    const float ninf = -__builtin_inff();
    if (V > 1 && E % V == 0) {
        // whole vectors: row * E is a multiple of V too
#pragma unroll
        for (int q = 0; q < V; ++q) l[q] = ninf;
        if (e0 < E) {
            if (bf16) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(logits) + row * E + e0;
                if constexpr (V == 4) {
                    const uint2 w = *reinterpret_cast<const uint2*>(p);
                    l[0] = __uint_as_float(w.x << 16);
                    l[1] = __uint_as_float(w.x & 0xffff0000u);
                    l[2] = __uint_as_float(w.y << 16);
                    l[3] = __uint_as_float(w.y & 0xffff0000u);
                } else if constexpr (V == 2) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
                    l[0] = __uint_as_float(w << 16);
                    l[1] = __uint_as_float(w & 0xffff0000u);
                }
            } else {
                const float* p = reinterpret_cast<const float*>(logits) + row * E + e0;
                if constexpr (V == 4) {
                    const float4 w = *reinterpret_cast<const float4*>(p);
                    l[0] = w.x; l[1] = w.y; l[2] = w.z; l[3] = w.w;
                } else if constexpr (V == 2) {
                    const float2 w = *reinterpret_cast<const float2*>(p);
                    l[0] = w.x; l[1] = w.y;
                }
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q) {
            l[q] = ninf;
            if (e0 + q < E)
                l[q] = bf16 ? bf2f(reinterpret_cast<const uint16_t*>(logits)[row * E + e0 + q])
                            : reinterpret_cast<const float*>(logits)[row * E + e0 + q];
        }
    }
#pragma unroll
    for (int q = 0; q < V; ++q) l[q] = l[q] == l[q] ? l[q] : ninf;
}

// Groups of a router: none, whole lanes (a power of two of lanes each, so the
// two best of a group merge by lane swaps), or any size (one masked maximum per
// group and place).
enum { kNoGroups = 0, kLaneGroups = 1, kAnyGroups = 2 };

inline int group_mode(const RouteSpec& r, int E, int V) {
    if (r.topk_groups >= r.n_groups) return kNoGroups;
    const int gs = E / r.n_groups, lanes = gs / V;
    return gs % V == 0 && (lanes & (lanes - 1)) == 0 ? kLaneGroups : kAnyGroups;
}

// What a wavefront keeps over its tokens: the biases of its experts, where its
// group's score lies.
template <int V, int GM, bool BIASED>
struct RouteWave {
    float b[V];
    float top;    // largest |bias|
    int stride;   // lanes from one group's score to the next
    int g0;       // this lane's group (GM kAnyGroups: lane g holds group g)
    int gq[V];    // lane holding the score of the group of candidate q
    __device__ __forceinline__ RouteWave(const RouteSpec& r, int E) {
        const int lane = __lane_id(), e0 = V * lane;
        top = 0.0f;
        if constexpr (BIASED) {
            float m = 0.0f;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                b[q] = e0 + q < E ? r.bias[e0 + q] : 0.0f;
                m = fmaxf(m, fabsf(b[q]));
            }
            top = wave_max_f32(m);
        }
        if constexpr (GM != kNoGroups) {
            const int gs = E / r.n_groups;
            stride = GM == kLaneGroups ? gs / V : 1;
            g0 = lane / stride;
#pragma unroll
            for (int q = 0; q < V; ++q) gq[q] = min((e0 + q) / gs, r.n_groups - 1) * stride;
        }
    }
};

// One pass in T: lane j < topk ends with the j-th expert in sel.  False (float
// only) if a choice was too close to call.
template <typename T, int V, int GM, bool BIASED>
__device__ __forceinline__ bool route_choose(const RouteSpec& r, int E, int topk, const float (&l)[V],
                                             const RouteWave<V, GM, BIASED>& rw, float m, int& sel) {
    using RK = RankKey<T>;
    using key = typename RK::key;
    constexpr bool f32 = sizeof(T) == 4;
    const int lane = __lane_id();
    const int e0 = V * lane;
    const T ninf = -(T)__builtin_inff();

    T c[V];  // choices
    float eta = 0.0f;
    if constexpr (GM != kNoGroups || BIASED) {
        if (r.score == MOE_SCORE_SIGMOID) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if constexpr (f32) c[q] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[q]));
                else c[q] = 1.0 / (1.0 + exp(-(double)l[q]));
            }
            eta = 2.38418579e-07f;  // 2^-22
        } else {
            T den = 0;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                // (an infinite maximum: 1 at it, 0 elsewhere; nothing above -inf: all 0)
                if constexpr (f32) c[q] = l[q] == m ? 1.0f : __expf(l[q] - m);
                else c[q] = l[q] == m ? 1.0 : exp((double)l[q] - (double)m);
                if (m == -__builtin_inff() || e0 + q >= E) c[q] = 0;
                den += c[q];
            }
            den = wave_sum(den);
            const T inv = den > 0 ? 1 / den : 0;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if constexpr (f32) c[q] *= inv;
                else c[q] = den > 0 ? c[q] / den : 0.0;  // rounded once, as a quotient
            }
            eta = 1.90734863e-06f * (float)inv;  // 2^-19 of the largest
        }
        if constexpr (BIASED) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                c[q] += (T)rw.b[q];
                c[q] = c[q] == c[q] ? c[q] : ninf;
            }
            eta += 5.96046448e-08f * (1.0f + rw.top);
        }
    }

    bool close = false;
    uint64_t kept = ~0ull;
    if constexpr (GM != kNoGroups) {
        T mine;  // lane g * stride: the score of group g
        if constexpr (GM == kLaneGroups) {
            key a = 0, b = 0;  // the two best of the lane, then of the group
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const key x = RK::of(c[q]);
                b = RK::max2(b, RK::min2(a, x));
                a = RK::max2(a, x);
            }
            const int lanes = __builtin_amdgcn_readfirstlane(rw.stride);
#pragma unroll
            for (int step = 0; step < 6; ++step) {
                if ((1 << step) >= lanes) break;
                const key oa = lane_swap(a, step), ob = lane_swap(b, step);
                b = RK::max2(RK::min2(a, oa), RK::max2(b, ob));
                a = RK::max2(a, oa);
            }
            // (a lane group of one expert has no second: group_top is 1 then)
            mine = r.group_top == 2 ? RK::value(a) + RK::value(b) : RK::value(a);
        } else {
            mine = ninf;
            const int gs = E / r.n_groups;
            for (int g = 0; g < r.n_groups; ++g) {
                key k[V];
                key best = 0;
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const int e = e0 + q;
                    k[q] = (e >= g * gs && e < (g + 1) * gs) ? RK::of(c[q]) : 0;
                    best = k[q] > best ? k[q] : best;
                }
                const key first = RK::wave_max(best);
                T sum = RK::value(first);
                if (r.group_top == 2) {
                    // the second best: without the lowest lane's lowest candidate that holds the best
                    const int at = (int)__builtin_ctzll(__ballot(best == first));
                    bool gone = lane != at;
                    best = 0;
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        if (!gone && k[q] == first) {
                            gone = true;
                            k[q] = 0;
                        }
                        best = k[q] > best ? k[q] : best;
                    }
                    sum += RK::value(RK::wave_max(best));
                }
                if (lane == g) mine = sum;
            }
        }
        mine = mine == mine ? mine : ninf;
        // rank among the groups; in float32 an equal score counts as too close
        int rank = 0, near = 0;
        const float tol = 8.0f * eta + 4.76837158e-07f * (float)fabs((double)mine);
        const int stride = __builtin_amdgcn_readfirstlane(rw.stride);
#pragma unroll 8
        for (int g = 0; g < r.n_groups; ++g) {
            const T o = lane_read(mine, g * stride);
            if constexpr (f32) {
                rank += o > mine ? 1 : 0;
                near += fabsf(o - mine) > tol ? 0 : 1;  // (itself too)
            } else {
                rank += (o > mine || (o == mine && g < rw.g0)) ? 1 : 0;
            }
        }
        const bool group_lane = lane < r.n_groups * rw.stride;
        close = f32 && group_lane && near > 1;
        kept = __ballot(group_lane && rank < r.topk_groups);
    }

    // the lane's candidates, best first, equal ones in index order (no candidate: key 0)
    key k[V];
    int idx[V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        bool live = e0 + q < E;
        if constexpr (GM != kNoGroups) live = live && ((kept >> rw.gq[q]) & 1);
        const key of = RK::of(BIASED ? c[q] : (T)l[q]);
        k[q] = live ? of : 0;
        idx[q] = e0 + q;
    }
    // neighbours change places only if the later one is larger: stable
#pragma unroll
    for (int pass = 0; pass < V; ++pass)
#pragma unroll
        for (int x = pass & 1; x + 1 < V; x += 2) {
            const bool sw = k[x + 1] > k[x];
            const key hi = RK::max2(k[x], k[x + 1]), lo = RK::min2(k[x], k[x + 1]);
            const int ih = sw ? idx[x + 1] : idx[x], il = sw ? idx[x] : idx[x + 1];
            k[x] = hi;
            k[x + 1] = lo;
            idx[x] = ih;
            idx[x + 1] = il;
        }
    // take the best head of the 64 lists, topk times
    key taken = 0;
    for (int j = 0; j < topk; ++j) {
        const key best = RK::wave_max(k[0]);
        const int at = (int)__builtin_ctzll(__ballot(k[0] == best));
        const int e = __builtin_amdgcn_readlane(idx[0], at);
        const bool slot = lane == j, pop = lane == at;
        sel = slot ? e : sel;
        taken = slot ? best : taken;
        key kn[V];
        int in[V];
#pragma unroll
        for (int q = 0; q + 1 < V; ++q) {
            kn[q] = k[q + 1];
            in[q] = idx[q + 1];
        }
        kn[V - 1] = 0;
        in[V - 1] = idx[V - 1];
#pragma unroll
        for (int q = 0; q < V; ++q) {
            k[q] = pop ? kn[q] : k[q];
            idx[q] = pop ? in[q] : idx[q];
        }
    }
    if constexpr (f32) {
        if constexpr (BIASED) {
            // neighbours among the taken, and the best one left out (none: key 0)
            const key left = RK::wave_max(k[0]);
            key next = (key)__shfl_down((int)taken, 1, 64);
            next = lane == topk - 1 ? left : next;
            const float d = RK::value(taken) - RK::value(next);
            close = close || (lane < topk && next != 0 && !(d > 4.0f * eta));
        }
        return __ballot(close) == 0;
    }
    return true;
}

// Routes the token whose logits are l: lane j < topk ends with expert *sel and
// weight *w.
template <int V, int GM, bool BIASED>
__device__ __forceinline__ void route_grouped_token(const RouteSpec& r, int E, int topk, const float (&l)[V],
                                                    const RouteWave<V, GM, BIASED>& rw, int* sel_out, float* w_out) {
    const int lane = __lane_id();
    const float ninf = -__builtin_inff();
    const bool soft = r.score == MOE_SCORE_SOFTMAX;
    float m = 0.0f;
    if (soft) {
        m = l[0];
#pragma unroll
        for (int q = 1; q < V; ++q) m = fmaxf(m, l[q]);
        m = wave_max_f32(m);
    }
    int sel = 0;
    if (__builtin_expect(!route_choose<float, V, GM, BIASED>(r, E, topk, l, rw, m, sel), 0))
        route_choose<double, V, GM, BIASED>(r, E, topk, l, rw, m, sel);

    // the chosen experts' scores, from their logits: float32 exponentials, sums and
    // quotients (6e-8 of a weight; from float64 it would be its rounding, 3e-8)
    float lj = 0.0f;
#pragma unroll
    for (int q = 0; q < V; ++q) {
        const float v = __shfl(l[q], sel / V, 64);
        lj = sel % V == q ? v : lj;
    }
    const bool mine = lane < topk;
    float s = 0.0f;
    if (mine) s = soft ? (m == ninf ? 0.0f : lj == m ? 1.0f : expf(lj - m)) : 1.0f / (1.0f + expf(-lj));
    float den = 1.0f;
    if (r.renormalize) {
        den = wave_sum(s);
    } else if (soft) {
        den = 0.0f;
#pragma unroll
        for (int q = 0; q < V; ++q)
            den += (V * lane + q < E) ? (l[q] == m ? 1.0f : expf(l[q] - m)) : 0.0f;
        den = wave_sum(den);
    }
    float w = den > 0.0f ? s / den * r.scale : 0.0f;
    if (__ballot(mine && s < 1e-30f && lj > ninf)) {
        // a score that float32 holds badly or not at all: its weight may still be
        // one that it holds (the sum or the factor brings it back)
        double d = 0.0;
        if (mine) d = soft ? (m == ninf ? 0.0 : lj == m ? 1.0 : exp((double)lj - (double)m)) : 1.0 / (1.0 + exp(-(double)lj));
        const double sum = r.renormalize ? wave_sum(d) : (double)den;
        w = sum > 0.0 ? (float)(d / sum * (double)r.scale) : 0.0f;
    }
    *sel_out = sel;
    *w_out = w;
}

}  // namespace moe
