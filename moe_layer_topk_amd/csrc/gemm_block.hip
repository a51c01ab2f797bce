// Grouped expert GEMMs on block-scaled e4m3 (MOE_FP8_BLOCK): codes with one
// float32 scale per 128 k of a token row and per 128 x 128 weight block,
//
//   c[p][n] = sum_b sa[p][b] sw[n/128][b] sum_{k in b} a[p][k] w[n][k].
//
// One block of 128 k is one f8f6f4 MFMA step (two of 64 on the 32-row form):
// its products are summed on the matrix core from zero, and the sum joins the
// float32 accumulator through one fused multiply-add with sa * sw.
#include <type_traits>

#include "moe_block.h"
#include "moe_launch.h"

namespace moe {

struct BlockArgs {
    const void* a;
    const float* a_scale;
    const uint8_t* w;
    const float* w_scale;
    const int32_t* sorted;
    const int32_t* tile_expert;
    const int32_t* counts;
    const int32_t* offsets;
    const int32_t* active;
    const int32_t* num_active;
    int topk, N, K, P, block_m;
    void* c;
    float* c_scale;
    int ksplit;
    float* cpart;
    bool one_tile;  // an expert averages at most 64 rows: weight tiles feed about one row tile
};

// ------------------------------------------------------------ e4m3 act (tiles)
//
// Block tile: 256 weight rows (GATE: 128 gate rows and the matching 128 up
// rows, so one workgroup holds whole 128-column blocks of act and can quantise
// them) x BM sorted token rows x 128 k.  Weights on the MFMA row operand,
// tokens on the column operand: a lane's accumulators all belong to one token,
// so a block's scale sa * sw is one number per 32 x 32 tile.
//
// Operands and the tokens' scales reach LDS by direct copies into an ST-stage
// ring (one stage = 128 bytes of every row), one barrier per stage; 16-byte
// chunks are XOR-swizzled so 16 rows read at one logical chunk fall into
// distinct banks.
//
// Arithmetic.  The f8f6f4 MFMA adds the products of eight consecutive k in a
// window of about 14 bits below the largest one (measured: 448 + 2^-6 loses the
// small term inside a group of eight and keeps it across groups; on normal data
// the sum of a block is off by 1.4e-5 of its size, the bfloat16 MFMA's by
// 1e-8).  DOWN takes it: y is rounded to bfloat16, 150 times coarser.  GATE does
// not: its result decides e4m3 codes and their scales, so it converts the codes
// to bfloat16 (exact) and multiplies those at half the rate with full float32
// sums.

template <int BM_, int WN_, int ST_>
struct BtCfg {
    static constexpr int BM = BM_, BN = 256, ST = ST_;
    static constexpr int WM = 4, WN = WN_, Waves = WM * WN, Threads = 64 * Waves;  // waves: WM along weights, WN along tokens
    static constexpr int TM = BN / WM / 32, TN = BM / WN / 32;                     // 32 x 32 tiles per wave
    static constexpr int ABytes = BM * 128, BBytes = BN * 128, StageBytes = ABytes + BBytes;
    static constexpr int ALoads = BM / 8 / Waves, BLoads = BN / 8 / Waves;         // 1 KB copies per wave and stage
    static constexpr int L = ALoads + BLoads;
    static constexpr int SWaves = BM > 64 ? BM / 64 : 1;                           // waves that also copy scales
    static constexpr int SBuf = 64 * SWaves * 32;                                  // [64 SWaves tokens][8 blocks] float32
    static constexpr int ScaleOff = ST * StageBytes;
    static constexpr int RowOff = ScaleOff + 3 * SBuf;                             // [BM] source row of each token row
    static constexpr int IdOff = RowOff + 64 * SWaves * 4;                         // [BM] pair ids
    static constexpr int AmaxOff = IdOff + BM * 4;                                 // [WM][BM]
    static constexpr int LdsBytes = AmaxOff + WM * BM * 4;
    static constexpr int OutStride = 528;                                          // DOWN: bytes of a staged output row
    static_assert(ALoads * 8 * Waves == BM && BLoads * 8 * Waves == BN, "copy split");
    static_assert(TM == 2 && TN >= 1, "one gate and one up tile per wave");
    static_assert(BM * OutStride <= ScaleOff, "staged output rows");
    static_assert(LdsBytes <= 160 * 1024, "LDS");
};

// e4m3 codes of a 16-byte chunk as two bfloat16 MFMA operands (exact)
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cvt2(uint32_t w, bool hi) {
    const bf16x2_t v = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void cvt16(const uint4& c, uint4 (&o)[2]) {
    o[0] = uint4{cvt2(c.x, false), cvt2(c.x, true), cvt2(c.y, false), cvt2(c.y, true)};
    o[1] = uint4{cvt2(c.z, false), cvt2(c.z, true), cvt2(c.w, false), cvt2(c.w, true)};
}

// the products of two 16-byte chunks of codes on the 16-row bfloat16 MFMA
__device__ __forceinline__ f32x4 mfma_bf16_chunk(const uint4& a, const uint4& b, f32x4 c) {
    uint4 x[2], y[2];
    cvt16(a, x);
    cvt16(b, y);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[h]), __builtin_bit_cast(bf16x8, y[h]), c, 0, 0, 0);
    return c;
}

typedef const float __attribute__((address_space(4))) const_f32;  // uniform loads through the scalar cache

template <bool GATE, class C, bool NTW, bool FAR>
__global__ void __launch_bounds__(C::Threads) block_tile_kernel(BlockArgs g, int m_tiles, int n_tiles, int group_n) {
    extern __shared__ __attribute__((aligned(1024))) char bt_lds[];
    // flat tile order in groups of group_n weight tiles, cut into one
    // contiguous range per XCD
    constexpr int kXcds = 8;
    const int nb = m_tiles * n_tiles;
    const int per = (nb + kXcds - 1) / kXcds;
    const int t = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
    if (t >= nb) return;
    const int ng = t / (group_n * m_tiles);
    const int gw = min(group_n, n_tiles - ng * group_n);
    const int rem = t - ng * group_n * m_tiles;
    const int mtile = rem / gw, ntile = ng * group_n + rem % gw;
    const int e = g.tile_expert[mtile];
    if (e < 0) return;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % C::WM, wn = wave / C::WM;
    const int K = g.K, N = g.N, I = N / 2, P = g.P, nk = K / 128;
    const int n0 = ntile * (GATE ? 128 : 256);
    int* rows_s = reinterpret_cast<int*>(bt_lds + C::RowOff);
    int* ids_s = reinterpret_cast<int*>(bt_lds + C::IdOff);

    // padding rows read the tile's first row (always real); their output is dropped
    const int p0 = g.sorted[mtile * C::BM];
    for (int i = tid; i < 64 * C::SWaves; i += C::Threads) {
        int p = i < C::BM ? g.sorted[mtile * C::BM + i] : P;
        if (i < C::BM) ids_s[i] = p;
        if (p >= P) p = p0;
        rows_s[i] = GATE ? p / g.topk : p;
    }

    // sources of this wave's copies: instruction i fills rows 8 i .. 8 i + 7
    const int lrow = lane >> 3, lphys = lane & 7;
    unsigned asrc[C::ALoads];
    const char* afar[C::ALoads];
#pragma unroll
    for (int j = 0; j < C::ALoads; ++j) {
        const int r = (wave * C::ALoads + j) * 8 + lrow;
        int p = g.sorted[mtile * C::BM + r];
        if (p >= P) p = p0;
        const size_t off = (size_t)(GATE ? p / g.topk : p) * K + ring_swz(lphys, r) * 16;
        asrc[j] = (unsigned)off;
        afar[j] = static_cast<const char*>(g.a) + off;
    }
    const size_t arows = GATE ? (size_t)(P / g.topk) : (size_t)P;
    const v4i_rsrc arsrc = buf_rsrc(g.a, FAR ? 0u : (unsigned)(arows * K));
    const v4i_rsrc brsrc = buf_rsrc(g.w + (size_t)e * N * K, (unsigned)((size_t)N * K));
    unsigned bsrc[C::BLoads];
#pragma unroll
    for (int j = 0; j < C::BLoads; ++j) {
        const int r = (wave * C::BLoads + j) * 8 + lrow;
        int row = GATE ? (r < 128 ? n0 + r : I + n0 + r - 128) : n0 + r;
        if (!GATE && row >= N) row = N - 1;  // N an odd multiple of 128: the last tile's upper half is dropped
        bsrc[j] = (unsigned)row * (unsigned)K + (unsigned)ring_swz(lphys, r) * 16u;
    }
    const unsigned lds0 = lds_addr_of(bt_lds);
    auto issue = [&](int kt) __attribute__((always_inline)) {
        const unsigned st = lds0 + (unsigned)((kt % C::ST) * C::StageBytes);
        const unsigned koff = (unsigned)kt * 128u;
#pragma unroll
        for (int j = 0; j < C::ALoads; ++j) {
            const unsigned d = st + (wave * C::ALoads + j) * 1024;
            if constexpr (FAR) lds_dma16_at(afar[j] + koff, d);
            else lds_dma16_buf(arsrc, asrc[j], koff, d);
        }
#pragma unroll
        for (int j = 0; j < C::BLoads; ++j) {
            const unsigned d = st + C::ABytes + (wave * C::BLoads + j) * 1024;
            if constexpr (NTW) lds_dma16_buf_nt(brsrc, bsrc[j], koff, d);
            else lds_dma16_buf(brsrc, bsrc[j], koff, d);
        }
    };
    // scales of chunk c (blocks 8 c ..): part q of 8 holds tokens 8 (q SWaves + wave) ..
    auto issue_scales = [&](int c, int q) __attribute__((always_inline)) {
        const int i = (q * C::SWaves + wave) * 8;
        const int row = rows_s[i + (lane >> 3)];
        const int kb = min(8 * c + (lane & 7), nk - 1);
        lds_dma4_at(g.a_scale + (size_t)row * nk + kb, lds0 + C::ScaleOff + (c % 3) * C::SBuf + i * 32);
    };
    __syncthreads();
    // this wave's own loads above have to be done before its copies are counted
    wait_vm<0>();
    const bool scaler = wave < C::SWaves;
    if (scaler)
        for (int q = 0; q < 8; ++q) issue_scales(0, q);
    // a stage's copies: its operands, and (scaling waves) one part of the next chunk's scales
    auto issue_all = [&](int kt) __attribute__((always_inline)) {
        issue(kt);
        if (scaler) issue_scales(kt / 8 + 1, kt % 8);
    };
#pragma unroll
    for (int s0 = 0; s0 < C::ST - 1; ++s0)
        if (s0 < nk) issue_all(s0);

    // wave tile: rows of the weights (row operand), tokens (column operand)
    const int l31 = lane & 31, khalf = lane >> 5;
    int wrow[C::TM], trow[C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i) wrow[i] = GATE ? 128 * i + 32 * wm + l31 : 64 * wm + 32 * i + l31;
#pragma unroll
    for (int j = 0; j < C::TN; ++j) trow[j] = (wn * C::TN + j) * 32 + l31;
    const int nreal = min(C::BM, g.offsets[e] + g.counts[e] - mtile * C::BM);
    const int live = __builtin_amdgcn_readfirstlane(min(C::TN, max(0, (nreal - wn * C::TN * 32 + 31) / 32)));
    // weight scales of this wave's rows: GATE a gate and an up block, DOWN one block
    const float* sexp = g.w_scale + (size_t)e * (N / 128) * nk;
    const int nblk = GATE ? n0 / 128 : min((n0 + 64 * wm) / 128, N / 128 - 1);
    const_f32* sw0 = (const_f32*)(uintptr_t)(sexp + (size_t)__builtin_amdgcn_readfirstlane(nblk) * nk);
    const_f32* sw1 = GATE ? sw0 + (size_t)(I / 128) * nk : sw0;

    f32x16 acc[C::TM][C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    auto stage = [&](int kt, auto pf_tag, auto lt_tag) __attribute__((always_inline)) {
        constexpr bool pf = decltype(pf_tag)::value;
        constexpr int LT = decltype(lt_tag)::value;
        // stage kt has landed (and the scales issued with or before it)
        if constexpr (pf) {
            if (scaler) wait_vm<(C::ST - 2) * (C::L + 1)>();
            else wait_vm<(C::ST - 2) * C::L>();
        } else {
            wait_vm<0>();
        }
        __syncthreads();
        if constexpr (pf) issue_all(kt + C::ST - 1);
        if constexpr (LT > 0) {
            const char* sa = bt_lds + (kt % C::ST) * C::StageBytes;
            const char* sb = sa + C::ABytes;
            const float* sc = reinterpret_cast<const float*>(bt_lds + C::ScaleOff + ((kt / 8) % 3) * C::SBuf) + kt % 8;
            const float w0 = sw0[kt], w1 = sw1[kt];
            float s[C::TM][LT];
#pragma unroll
            for (int j = 0; j < LT; ++j) {
                const float tok = sc[trow[j] * 8];
                s[0][j] = tok * w0;
                s[1][j] = tok * w1;
            }
            f32x16 d[C::TM][LT];
#pragma unroll
            for (int i = 0; i < C::TM; ++i)
#pragma unroll
                for (int j = 0; j < LT; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) d[i][j][v] = 0.0f;
            auto chunk = [&](const char* base, int row, int c) {
                return *reinterpret_cast<const uint4*>(base + row * 128 + (ring_swz(c, row) << 4));
            };
            if constexpr (GATE) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 wf[C::TM][2], tf[LT][2];
#pragma unroll
                    for (int i = 0; i < C::TM; ++i) cvt16(chunk(sb, wrow[i], 2 * c + khalf), wf[i]);
#pragma unroll
                    for (int j = 0; j < LT; ++j) cvt16(chunk(sa, trow[j], 2 * c + khalf), tf[j]);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < C::TM; ++i)
#pragma unroll
                            for (int j = 0; j < LT; ++j)
                                d[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, wf[i][h]),
                                                                                  __builtin_bit_cast(bf16x8, tf[j][h]),
                                                                                  d[i][j], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    i32x8 wf[C::TM], tf[LT];
                    auto frag = [&](const char* base, int row) {
                        const uint4 x = chunk(base, row, (2 * c + khalf) * 2), y = chunk(base, row, (2 * c + khalf) * 2 + 1);
                        return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
                    };
#pragma unroll
                    for (int i = 0; i < C::TM; ++i) wf[i] = frag(sb, wrow[i]);
#pragma unroll
                    for (int j = 0; j < LT; ++j) tf[j] = frag(sa, trow[j]);
#pragma unroll
                    for (int i = 0; i < C::TM; ++i)
#pragma unroll
                        for (int j = 0; j < LT; ++j)
                            d[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i], tf[j], d[i][j], 0, 0, 0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < C::TM; ++i)
#pragma unroll
                for (int j = 0; j < LT; ++j)
#pragma unroll
                    for (int v = 0; v < 16; ++v) acc[i][j][v] = __builtin_fmaf(d[i][j][v], s[i][j], acc[i][j][v]);
        }
    };
    const int nmain = max(0, nk - (C::ST - 1));
    auto kloop = [&](auto lt_tag) __attribute__((always_inline)) {
        for (int kt = 0; kt < nmain; ++kt) stage(kt, std::true_type{}, lt_tag);
        for (int kt = nmain; kt < nk; ++kt) stage(kt, std::false_type{}, lt_tag);
    };
    static_assert(C::TN <= 2, "live tile counts 0, 1 and 2");
    if (live == 0) kloop(std::integral_constant<int, 0>{});
    else if (live == C::TN) kloop(std::integral_constant<int, C::TN>{});
    else kloop(std::integral_constant<int, 1>{});

    // epilogue: a lane holds rows 8 (v / 4) + 4 khalf + v % 4 of its tiles' token.
    // The rows go out through LDS, so that every store instruction writes whole
    // lines of a token's row.
    __syncthreads();
    if constexpr (GATE) {
        unsigned* amax_s = reinterpret_cast<unsigned*>(bt_lds + C::AmaxOff);
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
            unsigned m = 0;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                acc[0][j][v] = silu(acc[0][j][v]) * acc[1][j][v];
                m = max(m, __float_as_uint(acc[0][j][v]) & 0x7fffffffu);
            }
            m = max(m, (unsigned)__shfl_xor((int)m, 32, 64));
            if (khalf == 0) amax_s[wm * C::BM + trow[j]] = m;
        }
        __syncthreads();
        constexpr int kStride = 144;
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
            const int r = trow[j];
            const BlockQuant bq(max(max(amax_s[r], amax_s[C::BM + r]), max(amax_s[2 * C::BM + r], amax_s[3 * C::BM + r])));
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint32_t*>(bt_lds + r * kStride + 32 * wm + 8 * q + 4 * khalf) =
                    bq.pack4(acc[0][j][4 * q], acc[0][j][4 * q + 1], acc[0][j][4 * q + 2], acc[0][j][4 * q + 3]);
            const int p = ids_s[r];
            if (wm == 0 && khalf == 0 && p < P) g.c_scale[(size_t)p * (I / 128) + n0 / 128] = bq.scale;
        }
        __syncthreads();
        for (int i = tid; i < C::BM * 8; i += C::Threads) {
            const int r = i >> 3, p = ids_s[r];
            if (p < P)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.c) + (size_t)p * I + n0 + 16 * (i & 7)) =
                    *reinterpret_cast<const uint4*>(bt_lds + r * kStride + 16 * (i & 7));
        }
    } else {
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int j = 0; j < C::TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint2*>(bt_lds + trow[j] * C::OutStride + 2 * (64 * wm + 32 * i + 8 * q + 4 * khalf)) =
                        uint2{pack_bf2(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                              pack_bf2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
        __syncthreads();
        for (int i = tid; i < C::BM * 32; i += C::Threads) {
            const int r = i >> 5, n = n0 + 8 * (i & 31), p = ids_s[r];
            if (p < P && n < N)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.c) + (size_t)p * N + n) =
                    *reinterpret_cast<const uint4*>(bt_lds + r * C::OutStride + 16 * (i & 31));
        }
    }
}

template <bool GATE, class C, bool NTW, bool FAR>
static hipError_t launch_tile(const BlockArgs& a, int64_t cap, hipStream_t s) {
    const int m_tiles = (int)(cap / C::BM), n_tiles = (a.N + 255) / 256;
    const int64_t nb = (int64_t)m_tiles * n_tiles;
    static const hipError_t attr =
        hipFuncSetAttribute(reinterpret_cast<const void*>(&block_tile_kernel<GATE, C, NTW, FAR>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, C::LdsBytes);
    if (attr != hipSuccess) return attr;
    const int group_n = (!GATE || a.one_tile) ? 1 : (n_tiles <= 8 ? n_tiles : 2);
    hipLaunchKernelGGL((block_tile_kernel<GATE, C, NTW, FAR>), dim3((unsigned)((nb + 7) / 8 * 8)), dim3(C::Threads),
                       C::LdsBytes, s, a, m_tiles, n_tiles, group_n);
    return hipGetLastError();
}

template <bool GATE, class C>
static hipError_t launch_tile_c(const BlockArgs& a, int64_t cap, bool far, hipStream_t s) {
    // operands of 4 GiB or more: 64-bit token addresses (rare, one variant)
    if (far) return launch_tile<GATE, C, false, true>(a, cap, s);
    if (a.one_tile) return launch_tile<GATE, C, true, false>(a, cap, s);
    return launch_tile<GATE, C, false, false>(a, cap, s);
}

// ------------------------------------------------------- float32 act (ring)
//
// Few rows per expert: blockIdx.y is an active expert, blockIdx.x a block of
// 64 weight rows (GATE_UP: 32 gate rows and the matching up rows), blockIdx.z
// a K split (DOWN).  The four wavefronts take the blocks of 128 k round robin
// and reduce through LDS at the end; 16 token rows a pass.

template <bool GATE>
__global__ void __launch_bounds__(256) block_rows_kernel(BlockArgs g) {
    const int slot = blockIdx.y;
    if (slot >= *g.num_active) return;
    const int e = g.active[slot];
    const int cnt = g.counts[e], base = g.offsets[e];
    __shared__ f32x4 red[4][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane & 15, lg = lane >> 4;
    const int N = g.N, K = g.K, I = N / 2, nkb = K / 128;
    const int kb0 = (int)((long)blockIdx.z * nkb / g.ksplit), kb1 = (int)((long)(blockIdx.z + 1) * nkb / g.ksplit);
    const int n0 = GATE ? blockIdx.x * 32 : blockIdx.x * 64;
    const uint8_t* wexp = g.w + (size_t)e * N * K;
    const float* sexp = g.w_scale + (size_t)e * (N / 128) * nkb;
    const uint8_t* wrow[4];
    const float* srow[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int row = GATE ? (t < 2 ? n0 + 16 * t : I + n0 + 16 * (t - 2)) : n0 + 16 * t;
        wrow[t] = wexp + (size_t)(row + lr) * K;
        srow[t] = sexp + (size_t)(row / 128) * nkb;
    }
    for (int r0 = 0; r0 < cnt; r0 += 16) {
        const int r = r0 + lr;
        const int p = g.sorted[base + min(r, cnt - 1)];
        const int src = GATE ? p / g.topk : p;
        f32x4 acc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int b = kb0 + wave; b < kb1; b += 4) {
            const int k = 128 * b + 16 * lg;
            uint4 b0, b1;
            float s;
            if constexpr (GATE) {
                const uint8_t* arow = static_cast<const uint8_t*>(g.a) + (size_t)src * K + k;
                b0 = *reinterpret_cast<const uint4*>(arow);
                b1 = *reinterpret_cast<const uint4*>(arow + 64);
                s = g.a_scale[(size_t)src * nkb + b];
            } else {
                const float4* arow = reinterpret_cast<const float4*>(static_cast<const float*>(g.a) + (size_t)src * K + k);
                float4 v[8];
                unsigned m = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    v[u] = arow[u];
                    v[4 + u] = arow[16 + u];
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    m = max(m, max(max(__float_as_uint(v[u].x) & 0x7fffffffu, __float_as_uint(v[u].y) & 0x7fffffffu),
                                   max(__float_as_uint(v[u].z) & 0x7fffffffu, __float_as_uint(v[u].w) & 0x7fffffffu)));
                m = max(m, (unsigned)__shfl_xor((int)m, 16, 64));
                m = max(m, (unsigned)__shfl_xor((int)m, 32, 64));
                const BlockQuant bq(m);
                uint32_t q[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) q[u] = bq.pack4(v[u].x, v[u].y, v[u].z, v[u].w);
                b0 = uint4{q[0], q[1], q[2], q[3]};
                b1 = uint4{q[4], q[5], q[6], q[7]};
                s = bq.scale;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint4 a0 = *reinterpret_cast<const uint4*>(wrow[t] + k), a1 = *reinterpret_cast<const uint4*>(wrow[t] + k + 64);
                f32x4 d = {0.f, 0.f, 0.f, 0.f};
                if constexpr (GATE) {
                    d = mfma_bf16_chunk(a0, b0, d);
                    d = mfma_bf16_chunk(a1, b1, d);
                } else {
                    d = mfma_f8_16x16x128(a0, a1, b0, b1, d);
                }
                const float sc = s * srow[t][b];
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[t][v] = __builtin_fmaf(d[v], sc, acc[t][v]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t) red[wave][t][lane] = acc[t];
        __syncthreads();
        if (r < cnt) {
            auto sum = [&](int t) { return red[0][t][lane] + red[1][t][lane] + red[2][t][lane] + red[3][t][lane]; };
            if constexpr (GATE) {
                if (wave < 2) {
                    const f32x4 gs = sum(wave), us = sum(wave + 2);
                    f32x4 o;
#pragma unroll
                    for (int v = 0; v < 4; ++v) o[v] = silu(gs[v]) * us[v];
                    *reinterpret_cast<f32x4*>(static_cast<float*>(g.c) + (size_t)p * I + n0 + 16 * wave + 4 * lg) = o;
                }
            } else {
                const f32x4 y = sum(wave);
                const int n = n0 + 16 * wave + 4 * lg;
                if (g.cpart)
                    *reinterpret_cast<f32x4*>(g.cpart + ((size_t)blockIdx.z * g.P + p) * N + n) = y;
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.c) + (size_t)p * N + n) =
                        uint2{pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3])};
            }
        }
    }
}

// ------------------------------------------------------------------ dispatch

int block_tile_rows(int M, int E, int topk) {
    const long per_expert = (long)M * topk / E;
    return per_expert > 48 ? 128 : per_expert > 16 ? 64 : 32;
}

bool block_tile_rows_ok(int block_m) { return block_m == 32 || block_m == 64 || block_m == 128; }

bool block_f32_act(int M, int E, int topk, int H, int I) { return M == 1; }

int block_down_ksplit(int M, int topk, int E, int N, int K) {
    const long P = (long)M * topk;
    const long wgs = (long)(N / 64) * (P < E ? P : E);
    if (wgs >= 256) return 1;
    int ks = (int)((256 + wgs - 1) / wgs);
    if (ks > kMaxKsplit) ks = kMaxKsplit;
    if (ks > K / 128 / 6) ks = K / 128 / 6;
    return ks < 1 ? 1 : ks;
}

hipError_t launch_block_gemm(const BlockGemmCall& c, hipStream_t s) {
    if (c.M == 0) return hipSuccess;
    const int P = c.M * c.topk;
    const BlockArgs a{c.a, c.a_scale, static_cast<const uint8_t*>(c.w), c.w_scale, c.al.sorted_ids, c.al.tile_expert,
                      c.al.expert_counts, c.al.expert_offsets, c.al.active_experts, c.al.num_active, c.topk, c.N, c.K,
                      P, c.block_m, c.c, c.c_scale, c.ksplit, c.cpart, P <= 64L * c.E};
    const int slots = P < c.E ? P : c.E;
    const int64_t cap = moe_align_capacity(c.M, c.topk, c.E, c.block_m);
    if (c.kind == MOE_GEMM_GATE_UP_SILU) {
        hipLaunchKernelGGL((block_rows_kernel<true>), dim3(c.N / 64, slots, 1), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    if (c.kind == MOE_GEMM_DOWN) {
        hipLaunchKernelGGL((block_rows_kernel<false>), dim3(c.N / 64, slots, c.ksplit), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const bool gate = c.kind == MOE_GEMM_GATE_UP_SILU_E4M3;
    const bool far = (uint64_t)(gate ? c.M : P) * (uint64_t)c.K > 0xffffffffull;
    using C32 = BtCfg<32, 1, 3>;
    using C64 = BtCfg<64, 2, 3>;
    using C128 = BtCfg<128, 2, 3>;
    if (gate) {
        if (c.block_m == 32) return launch_tile_c<true, C32>(a, cap, far, s);
        if (c.block_m == 64) return launch_tile_c<true, C64>(a, cap, far, s);
        return launch_tile_c<true, C128>(a, cap, far, s);
    }
    if (c.block_m == 32) return launch_tile_c<false, C32>(a, cap, far, s);
    if (c.block_m == 64) return launch_tile_c<false, C64>(a, cap, far, s);
    return launch_tile_c<false, C128>(a, cap, far, s);
}

}  // namespace moe
