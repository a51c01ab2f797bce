// Block-scaled e4m3 (MOE_FP8_BLOCK): the quantiser of one block of 128 values
// shared by moe_quant_block and the grouped GEMMs.
#pragma once

#include "moe.h"
#include "moe_device.h"
#include "moe_tile.h"

namespace moe {

// Maximum of x over each row of 16 lanes, in every lane of the row (lane moves
// on the vector ALU: quad swaps, then half-row and row mirrors).
__device__ __forceinline__ unsigned row16_max_u32(unsigned x) {
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false));  // row_half_mirror
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, false));  // row_mirror
    return x;
}

// Eight consecutive values of x as float32; i a multiple of 8.
template <int XDT>
__device__ __forceinline__ void load8(const void* x, size_t i, float (&v)[8]) {
    if constexpr (XDT == MOE_F32) {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ unsigned amax8(const float (&v)[8]) {
    unsigned m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    return m;
}

constexpr float kMinBlockScale = 1.17549435e-38f;  // 2^-126

// Quantiser of a block whose largest magnitude has the float32 bits `amax`
// (the maximum of the values' bits without their signs, so a NaN wins over an
// infinity and that over every number): scale = max(amax / 448, 2^-126).
__device__ __forceinline__ float block_scale(unsigned amax) { return fmaxf(__uint_as_float(amax) / 448.0f, kMinBlockScale); }

struct BlockQuant : E4m3Quant {
    float scale;
    bool bad;  // a NaN or an infinity in the block
    __device__ __forceinline__ explicit BlockQuant(unsigned amax) : BlockQuant(block_scale(amax), amax >= 0x7f800000u) {}
    __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) const {
        const uint32_t w = E4m3Quant::pack4(a, b, c, d);
        return bad ? 0x7f7f7f7fu : w;
    }

   private:
    __device__ __forceinline__ BlockQuant(float s0, bool bad0)
        : E4m3Quant(s0), scale(bad0 ? __uint_as_float(0x7fc00000u) : s0), bad(bad0) {}
};

// Rows to quantise beside other work of a launch (q NULL: none).
struct QuantJob {
    const uint16_t* x;  // bfloat16
    size_t nblk;        // blocks of 128 values
    uint8_t* q;
    float* scale;
};

// Blocks of 128 values of x by `nthreads` threads of workgroup `blk` of `nblks`:
// 16 lanes hold a block, 8 values each.
template <int XDT>
__device__ __forceinline__ void quant_rows(const void* x, size_t nblk, uint8_t* q, float* scale, int blk, int nblks,
                                           int nthreads) {
    const int l = threadIdx.x & 15, per = nthreads / 16;
    for (size_t b = (size_t)blk * per + (threadIdx.x >> 4); b < nblk; b += (size_t)nblks * per) {
        float v[8];
        load8<XDT>(x, b * 128 + 8 * l, v);
        const BlockQuant bq(row16_max_u32(amax8(v)));
        *reinterpret_cast<uint2*>(q + b * 128 + 8 * l) =
            uint2{bq.pack4(v[0], v[1], v[2], v[3]), bq.pack4(v[4], v[5], v[6], v[7])};
        if (l == 0) scale[b] = bq.scale;
    }
}

}  // namespace moe
