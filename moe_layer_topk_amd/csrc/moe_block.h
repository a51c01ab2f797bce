// Block-scaled e4m3 (MOE_FP8_BLOCK): the quantiser of one block of 128 values
// shared by moe_quant_block and the grouped GEMMs.
#pragma once

#include "moe_device.h"
#include "moe_tile.h"

namespace moe {

// Maximum of x over each row of 16 lanes, in every lane of the row (lane moves
// on the vector ALU: quad swaps, then half-row and row mirrors).
__device__ __forceinline__ unsigned row16_max_u32(unsigned x) {
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp((int)x, (int)x, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x141, 0xF, 0xF, false));  // row_half_mirror
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x140, 0xF, 0xF, false));  // row_mirror
    return x;
}

constexpr float kMinBlockScale = 1.17549435e-38f;  // 2^-126

// Quantiser of a block whose largest magnitude has the float32 bits `amax`
// (the maximum of the values' bits without their signs, so a NaN wins over an
// infinity and that over every number).  s = max(amax / 448, 2^-126); codes are
// e4m3 of the IEEE float32 quotient x / s, formed from r = 1 / s and two
// remainder corrections as in ActQuant.  Those are exact while no remainder
// falls below what float32 holds, so a block with s < 2^-80 is scaled up by 2^96
// first (s and every x; exact, and the quotients stay the same).
struct BlockQuant {
    float scale, pre, s, r;
    bool bad;
    __device__ __forceinline__ explicit BlockQuant(unsigned amax) {
        bad = amax >= 0x7f800000u;
        scale = fmaxf(__uint_as_float(amax) / 448.0f, kMinBlockScale);
        const bool low = scale < 8.27180613e-25f;                  // 2^-80
        pre = low ? 79228162514264337593543950336.0f : 1.0f;       // 2^96
        s = scale * pre;
        r = 1.0f / s;
        if (bad) scale = __uint_as_float(0x7fc00000u);
    }
    __device__ __forceinline__ float quot(float x) const {
        const float a = x * pre;
        float q = a * r;
        float e = __builtin_fmaf(-q, s, a);
        q = __builtin_fmaf(e, r, q);
        e = __builtin_fmaf(-q, s, a);
        return __builtin_copysignf(__builtin_fmaf(e, r, q), a);
    }
    __device__ __forceinline__ float sat(float x) const { return __builtin_amdgcn_fmed3f(quot(x), -448.0f, 448.0f); }
    __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) const {
        const uint32_t w = pack_fp8x4(sat(a), sat(b), sat(c), sat(d));
        return bad ? 0x7f7f7f7fu : w;
    }
};

}  // namespace moe
