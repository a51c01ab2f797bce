// Device pieces the grouped-GEMM kernels share: the f8f6f4 MFMA, the e4m3
// quantiser, direct-to-LDS copies and the waits that order them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16x16 tile over 128 e4m3 products per lane group: gfx950's f8f6f4 MFMA
// (4x the K of v_mfma_f32_16x16x32_fp8_fp8 per instruction, about 3x its
// throughput).  Each operand is 32 bytes per lane given as two 16-byte
// halves; the same byte positions of A and B meet in the same product, so
// any K order works as long as both operands are loaded alike.  Scale
// operands 0 select the unscaled form.
__device__ __forceinline__ f32x4 mfma_f8_16x16x128(const uint4& a0, const uint4& a1, const uint4& b0,
                                                   const uint4& b1, f32x4 c) {
    const i32x8 a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
    const i32x8 b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// e4m3 codes of the IEEE float32 quotients a / scale (round to nearest even,
// saturated at +-448).  A quotient is formed from r = 1/s (one IEEE division
// per thread) and two remainder corrections by fused multiply-add: with r
// correctly rounded, the first correction leaves the quotient within one
// ulp and the second returns the correctly rounded quotient (Markstein's
// theorem), provided nothing under- or overflows.  A remainder may be as small as
// 2^-34 s (half a step of the smallest quotient a code hangs on), so a scale below
// 2^-80 is raised by multiplying s and every a by 2^64 (exact, and the quotient is
// unchanged; the smallest s, 2^-149, becomes 2^-85; scale <= FLT_MAX/448 keeps r
// normal at the top).  The corrections turn a -0 quotient into +0, so the sign is
// taken from a (s > 0): a zero quotient keeps the sign an IEEE division gives it.  The
// per-value path has no branch.
struct E4m3Quant {
    float pre, s, r;
    __device__ __forceinline__ explicit E4m3Quant(float scale)
        : pre(scale < 8.27180613e-25f ? 18446744073709551616.0f : 1.0f), s(scale * pre), r(1.0f / s) {}  // 2^-80, 2^64
    __device__ __forceinline__ float quot(float a0) const {
        const float a = a0 * pre;
        float q = a * r;
        float e = __builtin_fmaf(-q, s, a);
        q = __builtin_fmaf(e, r, q);
        e = __builtin_fmaf(-q, s, a);
        return __builtin_copysignf(__builtin_fmaf(e, r, q), a);
    }
    __device__ __forceinline__ float sat(float a) const { return __builtin_amdgcn_fmed3f(quot(a), -448.0f, 448.0f); }
    __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) const {
        return pack_fp8x4(sat(a), sat(b), sat(c), sat(d));
    }
};

// Per-tensor quantiser of the float32 intermediate, scale = amax / 448: uniform
// across the wavefront.
struct ActQuant : E4m3Quant {
    using E4m3Quant::E4m3Quant;
    // 16 float32 values (four 16-byte chunks) -> 16 e4m3 codes
    __device__ __forceinline__ uint4 codes16(const uint4& v0, const uint4& v1, const uint4& v2,
                                             const uint4& v3) const {
        return uint4{pack4(v0), pack4(v1), pack4(v2), pack4(v3)};
    }
    __device__ __forceinline__ uint32_t pack4(const uint4& v) const {
        return E4m3Quant::pack4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
};

typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane from global memory straight into LDS: the wave's 64
// lanes fill 1 KB at the wave-uniform LDS byte address in M0 (a 32-bit LDS
// address, so a ring's stage addresses are plain scalar adds).  Issued
// through inline asm so the compiler does not treat every later LDS read as
// dependent on the copy (it would wait for all copies in flight, prefetched
// stages included); the kernels order their rings themselves with explicit
// vmcnt waits and barriers.  "memory" keeps LDS reads and writes of the
// kernel in program order around it.
__device__ __forceinline__ void lds_dma16_at(const void* src, unsigned lds_addr) {
    const unsigned m0 = __builtin_amdgcn_readfirstlane(lds_addr);
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(m0) : "memory", "m0");
}

// The same copy with the non-temporal hint: for data read once (decode
// weights), so the stream does not displace reused lines (token rows) from
// L2; on MI355X it also streams faster (weights of the Mixtral-shaped gate/up
// projection through the decode ring: 5.83 TB/s plain, 6.59 TB/s with nt).
__device__ __forceinline__ void lds_dma16_nt_at(const void* src, unsigned lds_addr) {
    const unsigned m0 = __builtin_amdgcn_readfirstlane(lds_addr);
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(src), "s"(m0) : "memory", "m0");
}

// 4 bytes per lane from global memory into LDS, at consecutive words from the
// wave-uniform LDS byte address.
__device__ __forceinline__ void lds_dma4_at(const void* src, unsigned lds_addr) {
    const unsigned m0 = __builtin_amdgcn_readfirstlane(lds_addr);
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(m0) : "memory", "m0");
}

// Buffer-addressed copies into LDS: a raw (stride 0) buffer resource over
// [base, base + bytes) plus a 32-bit per-lane offset (VGPR) and a wave-uniform
// one (SGPR).  Reads past `bytes` return zeros instead of touching memory.
// The tile kernel's copies take this form rather than 64-bit flat addresses:
// one VGPR per source instead of two, and on MI355X it measured 1-3% faster
// for bf16 prefill (same bytes, less address work per 16-byte copy).  Callers
// keep every offset below 2^32 (the host checks the operand sizes).
typedef int v4i_rsrc __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4i_rsrc buf_rsrc(const void* base, unsigned bytes) {
    const unsigned long long b = (unsigned long long)base;
    v4i_rsrc r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(b & 0xffffffffu));
    r[1] = __builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xffffu));
    r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = 0x00020000;
    return r;
}
__device__ __forceinline__ void lds_dma16_buf(v4i_rsrc rsrc, unsigned voff, unsigned soff, unsigned lds_addr) {
    const unsigned m0 = __builtin_amdgcn_readfirstlane(lds_addr);
    const unsigned so = __builtin_amdgcn_readfirstlane(soff);
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(voff), "s"(rsrc), "s"(m0), "s"(so)
                 : "memory", "m0");
}
__device__ __forceinline__ void lds_dma16_buf_nt(v4i_rsrc rsrc, unsigned voff, unsigned soff, unsigned lds_addr) {
    const unsigned m0 = __builtin_amdgcn_readfirstlane(lds_addr);
    const unsigned so = __builtin_amdgcn_readfirstlane(soff);
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, %3 offen nt lds" ::"v"(voff), "s"(rsrc), "s"(m0), "s"(so)
                 : "memory", "m0");
}

__device__ __forceinline__ unsigned lds_addr_of(const void* p) {
    return (unsigned)(uintptr_t)(const lds_void*)p;
}

// wait until at most n vector-memory operations of this wave are outstanding
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

template <int L>
__device__ __forceinline__ void wait_vm_runtime(int stages_outstanding) {
    switch (stages_outstanding) {
        case 0: wait_vm<0>(); break;
        case 1: wait_vm<L>(); break;
        case 2: wait_vm<2 * L < 64 ? 2 * L : 63>(); break;
        default: wait_vm<3 * L < 64 ? 3 * L : 63>(); break;
    }
}

constexpr int kRingSB = 128;  // bytes of every row per step

// Physical 16-byte chunk of logical chunk c in ring row r.  Rows are 128
// bytes, so rows 2q and 2q+1 share a 256-byte bank window; XOR with q mod 8
// puts 16 consecutive rows read at one logical chunk into 16 distinct
// 16-byte bank groups.
__device__ __forceinline__ int ring_swz(int c, int r) { return c ^ ((r >> 1) & 7); }

// vmcnt wait that is also a compiler memory barrier (LDS reads of the
// stage may not move above it)
template <int N>
__device__ __forceinline__ void ring_wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace moe
