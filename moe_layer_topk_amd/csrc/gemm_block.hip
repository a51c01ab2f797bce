// Grouped expert GEMMs on block-scaled e4m3 (MOE_FP8_BLOCK): codes with one
// float32 scale per 128 k of a token row and per 128 x 128 weight block,
//
//   c[p][n] = sum_b sa[p][b] sw[n/128][b] sum_{k in b} a[p][k] w[n][k].
//
// One block of 128 k is one f8f6f4 MFMA step (two of 64 on the 32-row form):
// its products are summed on the matrix core from zero, and the sum joins the
// float32 accumulator through one fused multiply-add with sa * sw.  (gate/up
// multiplies the codes as bfloat16 instead, see below.)
#include <atomic>
#include <type_traits>

#include "moe_block.h"
#include "moe_launch.h"
#include "moe_route.h"

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
    const int32_t* rows_end;  // the last expert's end in the sorted order
    int topk, N, K, P;
    void* c;
    float* c_scale;
    int ksplit;
    float* cpart;
    const int32_t* ids;  // one token: its topk ids, read instead of the alignment
    bool one_tile;  // an expert averages at most 64 rows: weight tiles feed about one row tile
};

// ------------------------------------------------------------ e4m3 act (tiles)
//
// Block tile: BM sorted token rows x 128 k x BN weight rows (DOWN: 128; GATE:
// 256, 128 gate rows and the matching 128 up rows, so one workgroup holds whole
// 128-column blocks of act and can quantise them).  Weights on the MFMA row operand,
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
//
// What bounds it.  gate/up of 8 experts of 4096 x 14336 at 4096 tokens: 1.86 ms,
// 1.03 PFLOP/s.  Of the about 3400 cycles of a stage the products take 1860, and
// a wavefront's conversions, fused multiply-adds and addresses, about 6.6 vector
// instructions a product, do not all fit beside them (without the conversions
// 1.66 ms of then 1.9, without the copies 1.58, without the multiply-adds 1.80).
// Sixteen wavefronts, or four of 64 x 128, are slower (2.26 and 2.5 ms).  down of
// 128 experts of 2048 x 768 at 4096 tokens: 130 us, 0.8 PFLOP/s; 70 of them are
// the copies from L2 (1 GB), 25 the rows' way through LDS, 30 their stores (134
// MB); half the products change nothing.  256 weight rows a tile (139 us), and
// workgroups that stay and fetch the next tile's first stages during the
// epilogue (126 us, gate/up spills) gain nothing.  Few rows: the weight stream,
// 6.3 to 6.5 TB/s.

template <int BM_, int BN_, int WN_, int ST_>
struct BtCfg {
    static constexpr int BM = BM_, BN = BN_, ST = ST_;
    static constexpr int WM = BN / 64, WN = WN_, Waves = WM * WN, Threads = 64 * Waves;  // waves: WM along weights, WN along tokens
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
    static constexpr int OutStride = 2 * BN + 16;                                  // DOWN: bytes of a staged output row
    // wavefronts a SIMD has to hold (bounds the registers): two workgroups of
    // eight wavefronts a CU where the LDS holds them
    static constexpr int MinWaves = Waves == 8 && LdsBytes <= 80 * 1024 ? 4 : 1;
    static_assert(ALoads * 8 * Waves == BM && BLoads * 8 * Waves == BN, "copy split");
    static_assert(TM == 2 && TN >= 1, "one gate and one up tile per wave");
    static_assert(BM * OutStride <= ScaleOff, "staged output rows");
    static_assert(LdsBytes <= 160 * 1024, "LDS");
};

// silu(g) u with the hardware's reciprocal (off by 2^-23 of the value, as far as
// the exponential): a correctly rounded quotient is nine instructions more, of
// the seventeen a value costs.  Below g = -87 the result is 0 or -0.
__device__ __forceinline__ float silu_mul(float g, float u) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u; }

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
typedef const int __attribute__((address_space(4))) const_i32;

template <bool GATE, class C, bool NTW, bool FAR>
__global__ void __launch_bounds__(C::Threads, C::MinWaves) block_tile_kernel(BlockArgs g, int n_tiles, int group_n) {
    static_assert(C::BN == (GATE ? 256 : 128), "whole tiles of N, one block of weight scales for each 128 rows");
    extern __shared__ __attribute__((aligned(1024))) char bt_lds[];
    // flat order of the batch's row tiles x weight tiles in groups of group_n
    // weight tiles, cut into one contiguous range per XCD (of the tiles that
    // exist: with the spare ones of the alignment's capacity counted, a range
    // may hold many more than another)
    constexpr int kXcds = 8;
    const int m_tiles = *(const_i32*)(uintptr_t)g.rows_end / C::BM;
    const int nb = m_tiles * n_tiles;
    const int per = (nb + kXcds - 1) / kXcds;
    const int at = blockIdx.x / kXcds, t = (blockIdx.x % kXcds) * per + at;
    if (at >= per || t >= nb) return;
    const int ng = t / (group_n * m_tiles);
    const int gw = min(group_n, n_tiles - ng * group_n);
    const int rem = t - ng * group_n * m_tiles;
    const int mtile = rem / gw, ntile = ng * group_n + rem % gw;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // everything the tile's addresses need, in as few round trips as they allow
    const int e = ((const_i32*)(uintptr_t)g.tile_expert)[__builtin_amdgcn_readfirstlane(mtile)];
    const int lrow = lane >> 3, lphys = lane & 7;
    int pid = g.sorted[mtile * C::BM + tid % C::BM], pa[C::ALoads];
#pragma unroll
    for (int j = 0; j < C::ALoads; ++j) pa[j] = g.sorted[mtile * C::BM + (wave * C::ALoads + j) * 8 + lrow];
    const int nreal = min(C::BM, ((const_i32*)(uintptr_t)g.offsets)[e] + ((const_i32*)(uintptr_t)g.counts)[e] - mtile * C::BM);
    const int wm = wave % C::WM, wn = wave / C::WM;
    const int K = g.K, N = g.N, I = N / 2, P = g.P, nk = K / 128;
    const int n0 = ntile * 128;
    int* rows_s = reinterpret_cast<int*>(bt_lds + C::RowOff);
    int* ids_s = reinterpret_cast<int*>(bt_lds + C::IdOff);

    // padding rows read the tile's first row (always real); their output is dropped
    const int p0 = ((const_i32*)(uintptr_t)g.sorted)[__builtin_amdgcn_readfirstlane(mtile) * C::BM];
    if (tid < 64 * C::SWaves) {
        if (tid < C::BM) ids_s[tid] = pid;
        if (pid >= P) pid = p0;
        rows_s[tid] = GATE ? pid / g.topk : pid;
    }

    // sources of this wave's copies: instruction i fills rows 8 i .. 8 i + 7
    unsigned asrc[C::ALoads];
    const char* afar[C::ALoads];
#pragma unroll
    for (int j = 0; j < C::ALoads; ++j) {
        const int r = (wave * C::ALoads + j) * 8 + lrow;
        const int p = pa[j] >= P ? p0 : pa[j];
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
        const int row = GATE && r >= 128 ? I + n0 + r - 128 : n0 + r;
        bsrc[j] = (unsigned)row * (unsigned)K + (unsigned)ring_swz(lphys, r) * 16u;
    }
    const unsigned lds0 = lds_addr_of(bt_lds);
    // Stage kt multiplies block (kt + rot) mod nk.  Where the weights come from
    // memory once (NTW), weight tiles start at different blocks: with rows a power
    // of two apart, tiles at one block would all ask the same few channels (16
    // experts of 4096 x 4096 at 64 tokens, gate/up 132 -> 86 us, down 60 -> 49; other
    // sizes within 2%).  Where row tiles share them through L2 it costs 2%.
    const int rot = NTW ? ntile % nk : 0;
    auto block_of = [&](int kt) __attribute__((always_inline)) { return !NTW || kt + rot < nk ? kt + rot : kt + rot - nk; };
    // copy j of stage kt (0 .. L - 1: tokens, then weights)
    auto issue_one = [&](int kt, int j) __attribute__((always_inline)) {
        const unsigned st = lds0 + (unsigned)((kt % C::ST) * C::StageBytes);
        const unsigned koff = (unsigned)block_of(kt) * 128u;
        if (j < C::ALoads) {
            const unsigned d = st + (wave * C::ALoads + j) * 1024;
            if constexpr (FAR) lds_dma16_at(afar[j] + koff, d);
            else lds_dma16_buf(arsrc, asrc[j], koff, d);
        } else {
            const unsigned d = st + C::ABytes + (wave * C::BLoads + j - C::ALoads) * 1024;
            if constexpr (NTW) lds_dma16_buf_nt(brsrc, bsrc[j - C::ALoads], koff, d);
            else lds_dma16_buf(brsrc, bsrc[j - C::ALoads], koff, d);
        }
    };
    // scales of chunk c (stages 8 c ..): part q of 8 holds tokens 8 (q SWaves +
    // wave) ..; further waves repeat the first ones' copy (the same bytes to the
    // same place), so that a stage has no branch and every wave counts alike
    auto scale_copy = [&](int c, int q, int row) __attribute__((always_inline)) {
        const int i = (q * C::SWaves + wave % C::SWaves) * 8;
        const int kb = min(block_of(8 * c + (lane & 7)), nk - 1);
        lds_dma4_at(g.a_scale + (size_t)row * nk + kb, lds0 + C::ScaleOff + (c % 3) * C::SBuf + i * 32);
    };
    auto issue_scales = [&](int c, int q) __attribute__((always_inline)) {
        scale_copy(c, q, rows_s[(q * C::SWaves + wave % C::SWaves) * 8 + (lane >> 3)]);
    };
    __syncthreads();
    // this wave's own loads above have to be done before its copies are counted
    wait_vm<0>();
    // copies [j0, j1) of stage kt; the last is one part of the next chunk's scales
    auto issue = [&](int kt, int j0, int j1) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < C::L; ++j)
            if (j >= j0 && j < j1) issue_one(kt, j);
        if (j0 <= C::L && C::L < j1) issue_scales(kt / 8 + 1, kt % 8);
    };
    issue(0, 0, C::L + 1);
    {
        int row[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) row[q] = rows_s[(q * C::SWaves + wave % C::SWaves) * 8 + (lane >> 3)];
#pragma unroll
        for (int q = 0; q < 8; ++q) scale_copy(0, q, row[q]);
    }
#pragma unroll
    for (int s0 = 1; s0 < C::ST - 1; ++s0)
        if (s0 < nk) issue(s0, 0, C::L + 1);

    // wave tile: rows of the weights (row operand), tokens (column operand)
    const int l31 = lane & 31, khalf = lane >> 5;
    // (GATE: rows 32 wm of the gate half and of the up half, DOWN: rows 64 wm)
    int trow[C::TN];
#pragma unroll
    for (int j = 0; j < C::TN; ++j) trow[j] = (wn * C::TN + j) * 32 + l31;
    const int live = __builtin_amdgcn_readfirstlane(min(C::TN, max(0, (nreal - wn * C::TN * 32 + 31) / 32)));
    // weight scales of the tile: GATE a gate and an up block, DOWN one block
    const float* sexp = g.w_scale + (size_t)e * (N / 128) * nk;
    const_f32* sw0 = (const_f32*)(uintptr_t)(sexp + (size_t)__builtin_amdgcn_readfirstlane(n0 / 128) * nk);
    const_f32* sw1 = GATE ? sw0 + (size_t)(I / 128) * nk : sw0;

    f32x16 acc[C::TM][C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    // LDS offsets of this lane's 16-byte chunks.  The swizzle depends on bits 1-3
    // of the row, which the 32-row tiles share, so a tile is a constant away.
    // GATE: chunk 2 c + khalf of step c (16 k per lane half, two MFMAs);
    // DOWN: chunks 4 c + 2 khalf + h, the two halves of a 64-k MFMA.
    int off[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        off[c] = l31 * 128 + (ring_swz(GATE ? 2 * c + khalf : 4 * (c >> 1) + 2 * khalf + (c & 1), l31) << 4);
    const int tbase = wn * C::TN * 4096, wbase = C::ABytes + (GATE ? wm * 4096 : wm * 8192);
    constexpr int kWStep = GATE ? 128 * 128 : 4096;  // from a wave's first weight tile to its second

    f32x16 d[C::TM][C::TN];  // the block's sums
    float sp[C::TM][C::TN];  // ... and their scales
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j) {
            sp[i][j] = 0.0f;
#pragma unroll
            for (int v = 0; v < 16; ++v) d[i][j][v] = 0.0f;
        }
    auto add_block = [&](auto lt_tag) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
            for (int j = 0; j < decltype(lt_tag)::value; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = __builtin_fmaf(d[i][j][v], sp[i][j], acc[i][j][v]);
    };
    // One stage.  The previous block's scaled sums join the accumulators right
    // after the barrier, while this block's first fragments come from LDS; the
    // next fragments are read (and GATE: converted) and the next stage's copies
    // go out between the products.
    auto stage = [&](int kt, auto pf_tag, auto lt_tag) __attribute__((always_inline)) {
        constexpr bool pf = decltype(pf_tag)::value;
        constexpr int LT = decltype(lt_tag)::value;
        // stage kt has landed (and the scales issued with or before it)
        if constexpr (pf) wait_vm<(C::ST - 2) * (C::L + 1)>();
        else wait_vm<0>();
        __syncthreads();
        if constexpr (LT == 0) {
            if constexpr (pf) issue(kt + C::ST - 1, 0, C::L + 1);
        } else {
            const char* st = bt_lds + (kt % C::ST) * C::StageBytes;
            const float* sc = reinterpret_cast<const float*>(bt_lds + C::ScaleOff + ((kt / 8) % 3) * C::SBuf) + kt % 8;
            uint4 wr[2][C::TM], tr[2][LT];  // codes of two steps
            auto read = [&](int b, int c) __attribute__((always_inline)) {
                const char* p = st + off[c];
#pragma unroll
                for (int i = 0; i < C::TM; ++i) wr[b][i] = *reinterpret_cast<const uint4*>(p + wbase + i * kWStep);
#pragma unroll
                for (int j = 0; j < LT; ++j) tr[b][j] = *reinterpret_cast<const uint4*>(p + tbase + j * 4096);
            };
            read(0, 0);
            read(1, 1);
            const float w0 = sw0[block_of(kt)], w1 = sw1[block_of(kt)];
            float tok[LT];
#pragma unroll
            for (int j = 0; j < LT; ++j) tok[j] = sc[trow[j] * 8];
            __builtin_amdgcn_sched_barrier(0);
            add_block(lt_tag);
            constexpr int kPart = (C::L + 1 + 3) / 4;
            const f32x16 zero = {};
            if constexpr (GATE) {
                uint4 wf[2][C::TM][2], tf[2][LT][2];
                auto cvt = [&](int b) __attribute__((always_inline)) {
#pragma unroll
                    for (int i = 0; i < C::TM; ++i) cvt16(wr[b][i], wf[b][i]);
#pragma unroll
                    for (int j = 0; j < LT; ++j) cvt16(tr[b][j], tf[b][j]);
                };
                cvt(0);
                read(0, 2);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int b = c & 1;
                    if constexpr (pf) issue(kt + C::ST - 1, c * kPart, (c + 1) * kPart);
                    if (c < 3) cvt(b ^ 1);
                    if (c == 0) read(1, 3);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < C::TM; ++i)
#pragma unroll
                            for (int j = 0; j < LT; ++j)
                                d[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                    __builtin_bit_cast(bf16x8, wf[b][i][h]), __builtin_bit_cast(bf16x8, tf[b][j][h]),
                                    c == 0 && h == 0 ? zero : d[i][j], 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < 2 * C::TM * LT; ++q) {
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);  // a product,
                        __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);  // four conversions
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                auto cat = [](const uint4& x, const uint4& y) {
                    return i32x8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
                };
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    i32x8 wf[C::TM], tf[LT];
#pragma unroll
                    for (int i = 0; i < C::TM; ++i) wf[i] = cat(wr[0][i], wr[1][i]);
#pragma unroll
                    for (int j = 0; j < LT; ++j) tf[j] = cat(tr[0][j], tr[1][j]);
                    if (c == 0) {
                        read(0, 2);
                        read(1, 3);
                    }
                    if constexpr (pf) issue(kt + C::ST - 1, c * 2 * kPart, (c + 1) * 2 * kPart);
#pragma unroll
                    for (int i = 0; i < C::TM; ++i)
#pragma unroll
                        for (int j = 0; j < LT; ++j)
                            d[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i], tf[j], c == 0 ? zero : d[i][j], 0,
                                                                                      0, 0, 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int j = 0; j < LT; ++j) {
                sp[0][j] = tok[j] * w0;
                sp[1][j] = tok[j] * w1;
            }
        }
    };
    const int nmain = max(0, nk - (C::ST - 1));
    auto kloop = [&](auto lt_tag) __attribute__((always_inline)) {
        for (int kt = 0; kt < nmain; ++kt) stage(kt, std::true_type{}, lt_tag);
        for (int kt = nmain; kt < nk; ++kt) stage(kt, std::false_type{}, lt_tag);
        add_block(lt_tag);
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
                acc[0][j][v] = silu_mul(acc[0][j][v], acc[1][j][v]);
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
            // (a product with the reciprocal for the IEEE quotient: other codes only
            // within 2^-23 of a tie, nearer than act itself is known; 6 of 8
            // instructions a value.  A NaN scale gives the smallest one here, and
            // its codes are replaced)
            const float inv = 1.0f / fmaxf(bq.scale, kMinBlockScale);
            auto code = [&](float x) { return __builtin_amdgcn_fmed3f(x * inv, -448.0f, 448.0f); };
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t w = pack_fp8x4(code(acc[0][j][4 * q]), code(acc[0][j][4 * q + 1]), code(acc[0][j][4 * q + 2]),
                                              code(acc[0][j][4 * q + 3]));
                *reinterpret_cast<uint32_t*>(bt_lds + r * kStride + 32 * wm + 8 * q + 4 * khalf) = bq.bad ? 0x7f7f7f7fu : w;
            }
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
        constexpr int kVecs = C::BN / 8;  // 16-byte pieces of a row
        for (int i = tid; i < C::BM * kVecs; i += C::Threads) {
            const int r = i / kVecs, v = i % kVecs, n = n0 + 8 * v, p = ids_s[r];
            if (p < P)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.c) + (size_t)p * N + n) =
                    *reinterpret_cast<const uint4*>(bt_lds + r * C::OutStride + 16 * v);
        }
    }
}

template <bool GATE, class C, bool NTW, bool FAR>
static hipError_t launch_tile(const BlockArgs& a, int64_t cap, hipStream_t s) {
    const int m_tiles = (int)(cap / C::BM), n_tiles = a.N / C::BN;
    const int64_t nb = (int64_t)m_tiles * n_tiles;
    if (nb > 0x7fffffffll - 8) return hipErrorInvalidValue;
    // LDS above the default dynamic limit is requested once per kernel and device
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    hipError_t st = hipGetDevice(&dev);
    if (st != hipSuccess) return st;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        st = hipFuncSetAttribute(reinterpret_cast<const void*>(&block_tile_kernel<GATE, C, NTW, FAR>),
                                 hipFuncAttributeMaxDynamicSharedMemorySize, C::LdsBytes);
        if (st != hipSuccess) return st;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    // Weight tiles a row tile meets before the next row tile.  Several row tiles
    // an expert: eight, so that the 32 or 64 workgroups of an XCD share a few of
    // both in its L2 (one / eight / all, us: gate/up of 8 experts of 4096 x 14336
    // at 4096 tokens 1919 / 1865 / 2188, down 736 / 655 / 813; of 128 of 2048 x 768
    // 317 / 253 / 253, 145 / 129 / 134).  One: all, an expert's weights as one
    // stream (down of 64 experts of 4096 x 8192 at 32 tokens 338 / 345 / 304, at 200
    // 379 / 391 / 336; gate/up of 256 of 7168 x 2048 at 1000 1286 / 1219 / 1178).
    const int group_n = a.one_tile || n_tiles < 8 ? n_tiles : 8;
    hipLaunchKernelGGL((block_tile_kernel<GATE, C, NTW, FAR>), dim3((unsigned)((nb + 7) / 8 * 8)), dim3(C::Threads),
                       C::LdsBytes, s, a, n_tiles, group_n);
    return hipGetLastError();
}

template <bool GATE, class C>
static hipError_t launch_tile_c(const BlockArgs& a, int64_t cap, bool far, hipStream_t s) {
    // operands of 4 GiB or more: 64-bit token addresses (rare, one variant)
    if (far) return launch_tile<GATE, C, false, true>(a, cap, s);
    if (a.one_tile) return launch_tile<GATE, C, true, false>(a, cap, s);
    return launch_tile<GATE, C, false, false>(a, cap, s);
}

// ------------------------------------------------------- float32 act (rows)
//
// Few rows per expert.  blockIdx.y is an active expert, blockIdx.x 64 of its
// weight rows (GATE: 32 gate rows and the matching 32 up rows), blockIdx.z a K
// split (DOWN).  The four wavefronts take the blocks of 128 k round robin,
// weights straight from memory into the MFMA operands (16 rows x 64 bytes an
// instruction), and reduce through LDS at the end; 16 token rows a pass.  DOWN
// quantises its float32 rows block by block as moe_quant_block does: a lane
// holds 32 of a row's 128 values, the four lanes of a row share their maximum.
//
// What keeps bytes in flight is workgroups: loading a second block ahead in each
// wavefront costs the occupancy (128 experts of 2048 x 768 at 16 tokens: gate/up
// 40 -> 57 us, down 29 -> 70), and the non-temporal hint makes the two 64-byte
// halves of a line two fetches (40 -> 54, 29 -> 34).

// One block of 128 k of a lane's token row: its values as loaded, then its
// codes (bytes 16 lg .. and 64 + 16 lg .. of the block) and scale.
template <bool F32>
struct TokenBlock {
    static constexpr int kVecs = F32 ? 8 : 2;
    uint4 v[kVecs];
    float s;
    __device__ __forceinline__ void load(const void* a, const float* a_scale, size_t row, int K, int b, int lg) {
        constexpr int kElem = F32 ? 4 : 1;
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(a) + (row * K + 128 * (size_t)b + 16 * lg) * kElem);
#pragma unroll
        for (int u = 0; u < kVecs / 2; ++u) {
            v[u] = p[u];
            v[kVecs / 2 + u] = p[4 * kElem + u];  // 64 values on
        }
        if constexpr (!F32) s = a_scale[row * (K / 128) + b];
    }
    __device__ __forceinline__ void codes(uint4& c0, uint4& c1, float& scale) const {
        if constexpr (!F32) {
            c0 = v[0];
            c1 = v[1];
            scale = s;
        } else {
            unsigned m = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                m = max(m, max(max(v[u].x & 0x7fffffffu, v[u].y & 0x7fffffffu), max(v[u].z & 0x7fffffffu, v[u].w & 0x7fffffffu)));
            m = max(m, (unsigned)__shfl_xor((int)m, 16, 64));
            m = max(m, (unsigned)__shfl_xor((int)m, 32, 64));
            const BlockQuant bq(m);
            auto pack = [&](const uint4& w) {
                return bq.pack4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
            };
            c0 = uint4{pack(v[0]), pack(v[1]), pack(v[2]), pack(v[3])};
            c1 = uint4{pack(v[4]), pack(v[5]), pack(v[6]), pack(v[7])};
            scale = bq.scale;
        }
    }
};

// ONE (GATE): a single token.  Its topk ids give the experts (no alignment is
// read), and a wavefront quantises the blocks of the bfloat16 row that it will
// multiply into its own LDS, 16 blocks at a time, 8 values a lane: what every
// lane group of the MFMA reads is then one broadcast.  Eight
// wavefronts share a workgroup's blocks (one token leaves the chip half empty,
// and a wavefront's blocks run one after another).
//
// ROUTE >= 0 (ONE; 2 * groups mode + biased): the token is routed here too.  Every
// workgroup's first wavefront chooses, while the others quantise their blocks;
// one workgroup writes the ids and weights for the down launch.  Inside it takes
// 3.3 us, as a launch of its own 4.4 and the way to the next one (layer of 256
// experts of 2048 x 512 21.4 -> 18.7 us, of 8 of 4096 x 14336 no change).
struct OneRoute {
    RouteSpec r;
    const float* logits;
    int E;
    int32_t* ids;
    float* wts;
};
struct NoRoute {};

template <bool ONE>
constexpr int kRowsWaves = ONE ? 8 : 4;

template <bool GATE, bool ONE, int ROUTE = -1>
__global__ void __launch_bounds__(64 * kRowsWaves<ONE>, 2)
    block_rows_kernel(BlockArgs g, std::conditional_t<(ROUTE >= 0), OneRoute, NoRoute> route) {
    constexpr int W = kRowsWaves<ONE>;
    static_assert(GATE || !ONE, "one token's down GEMM is block_down_one_kernel");
    static_assert(ONE || ROUTE < 0, "the router of one token");
    constexpr int kChunk = 16;  // blocks a wavefront quantises at a time
    const int slot = blockIdx.y;
    int e = 0, cnt, base;
    if constexpr (ONE) {
        if constexpr (ROUTE < 0) e = g.ids[slot];
        cnt = 1;
        base = 0;
    } else {
        e = g.active[slot];
        if (e < 0) return;
        cnt = g.counts[e];
        base = g.offsets[e];
    }
    __shared__ f32x4 red[W][4][64];
    __shared__ __attribute__((aligned(16))) uint8_t one_q[ONE ? W : 1][ONE ? kChunk * 128 : 16];
    __shared__ float one_s[ONE ? W : 1][kChunk];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int N = g.N, K = g.K, I = N / 2, nkb = K / 128;
    const int kb0 = (int)((long)blockIdx.z * nkb / g.ksplit), kb1 = (int)((long)(blockIdx.z + 1) * nkb / g.ksplit);
    const int n0 = GATE ? blockIdx.x * 32 : blockIdx.x * 64;
    // the wavefront's i-th block is kb0 + wave + W i
    const int mine = kb1 - kb0 > wave ? (kb1 - kb0 - wave + W - 1) / W : 0;
    // (ONE) the token's blocks i0 .. i0 + kChunk - 1 of this wavefront
    auto quantise = [&](int i0) __attribute__((always_inline)) {
        for (int i = i0; i < min(i0 + kChunk, mine); i += 4) {
            const int ib = i + (lane >> 4), l = lane & 15;
            const int b = kb0 + wave + W * min(ib, mine - 1);
            float v[8];
            load8<MOE_BF16>(g.a, 128 * (size_t)b + 8 * l, v);
            const BlockQuant bq(row16_max_u32(amax8(v)));
            const uint2 q = {bq.pack4(v[0], v[1], v[2], v[3]), bq.pack4(v[4], v[5], v[6], v[7])};
            if (ib < mine) {
                *reinterpret_cast<uint2*>(&one_q[wave][(ib - i0) * 128 + 8 * l]) = q;
                if (l == 0) one_s[wave][ib - i0] = bq.scale;
            }
        }
        // (read by this wavefront alone, after its own writes)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    if constexpr (ROUTE >= 0) {
        __shared__ int slot_e;
        if (wave == 0) {
            const RouteWave<4, ROUTE / 2, ROUTE % 2> rw(route.r, route.E);
            float l[4], wt;
            int sel;
            load_logits<4>(route.logits, false, 0, route.E, l);
            route_grouped_token<4, ROUTE / 2, ROUTE % 2>(route.r, route.E, g.topk, l, rw, &sel, &wt);
            if (lane == slot) slot_e = sel;
            if (blockIdx.x == 0 && slot == 0 && lane < g.topk) {
                route.ids[lane] = sel;
                route.wts[lane] = wt;
            }
        }
        quantise(0);
        __syncthreads();
        e = __builtin_amdgcn_readfirstlane(slot_e);
    }
    const uint8_t* wexp = g.w + (size_t)e * N * K + 16 * lg;
    const float* sexp = g.w_scale + (size_t)e * (N / 128) * nkb;
    const uint8_t* wrow[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int row = GATE ? (t < 2 ? n0 + 16 * t : I + n0 + 16 * (t - 2)) : n0 + 16 * t;
        wrow[t] = wexp + (size_t)(row + lr) * K;
    }
    const float* s0 = sexp + (size_t)(n0 / 128) * nkb;
    const float* s1 = GATE ? s0 + (size_t)(I / 128) * nkb : s0;

    for (int r0 = 0; r0 < cnt; r0 += 16) {
        const int r = r0 + lr;
        const int p = ONE ? slot : g.sorted[base + min(r, cnt - 1)];
        const size_t src = GATE ? p / g.topk : p;
        f32x4 acc[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < mine; ++i) {
            const int b = kb0 + wave + W * i;
            uint4 w[4][2], c0, c1;
            TokenBlock<!GATE> x;
            float sx;
            if constexpr (!ONE) x.load(g.a, g.a_scale, src, K, b, lg);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                w[t][0] = *reinterpret_cast<const uint4*>(wrow[t] + 128 * (size_t)b);
                w[t][1] = *reinterpret_cast<const uint4*>(wrow[t] + 128 * (size_t)b + 64);
            }
            const float w0 = s0[b], w1 = s1[b];
            if constexpr (ONE) {
                if (i % kChunk == 0 && (ROUTE < 0 || i > 0)) quantise(i);
                const uint8_t* q = &one_q[wave][(i % kChunk) * 128 + 16 * lg];
                c0 = *reinterpret_cast<const uint4*>(q);
                c1 = *reinterpret_cast<const uint4*>(q + 64);
                sx = one_s[wave][i % kChunk];
            } else {
                x.codes(c0, c1, sx);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f32x4 d = {0.f, 0.f, 0.f, 0.f};
                if constexpr (GATE) {
                    d = mfma_bf16_chunk(w[t][0], c0, d);
                    d = mfma_bf16_chunk(w[t][1], c1, d);
                } else {
                    d = mfma_f8_16x16x128(w[t][0], w[t][1], c0, c1, d);
                }
                const float sc = sx * (t < 2 ? w0 : w1);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[t][v] = __builtin_fmaf(d[v], sc, acc[t][v]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t) red[wave][t][lane] = acc[t];
        __syncthreads();
        if (r < cnt) {
            auto sum = [&](int t) {
                f32x4 v = red[0][t][lane];
#pragma unroll
                for (int u = 1; u < W; ++u) v += red[u][t][lane];
                return v;
            };
            if constexpr (GATE) {
                if (wave < 2) {
                    const f32x4 gs = sum(wave), us = sum(wave + 2);
                    f32x4 o;
#pragma unroll
                    for (int v = 0; v < 4; ++v) o[v] = silu(gs[v]) * us[v];
                    *reinterpret_cast<f32x4*>(static_cast<float*>(g.c) + (size_t)p * I + n0 + 16 * wave + 4 * lg) = o;
                }
            } else if (wave < 4) {
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

// ------------------------------------------------- one token, down + combine
//
// A workgroup owns 16 columns of the output for all of the token's experts, so
// their weighted sum needs no other workgroup and no launch of its own:
// wavefront u takes unit u = (expert slot, K split), the units' columns meet in
// LDS, and out = sum over slots ascending of weight * y, y the sum of its splits
// ascending.  act [topk][K] float32 is quantised by the wavefront that
// multiplies it.  128 experts of 2048 x 768, top 8: 128 workgroups; 8 of 4096 x
// 14336, top 2: 256, four splits each.  12.6 MB of the former in 7.9 us: a
// launch's floor and one chain of loads, products and sums.
constexpr int kOneWaves = 8, kOneUnits = 16;  // units: topk * max(1, 8 / topk) <= 16

__global__ void __launch_bounds__(64 * kOneWaves, 2) block_down_one_kernel(BlockArgs g, const float* __restrict__ wts,
                                                                        uint16_t* __restrict__ out) {
    constexpr int kChunk = 16;
    __shared__ __attribute__((aligned(16))) uint8_t one_q[kOneWaves][kChunk * 128];
    __shared__ float one_s[kOneWaves][kChunk];
    __shared__ float part[kOneUnits][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int N = g.N, K = g.K, nkb = K / 128, n0 = blockIdx.x * 16;
    const int ks = max(1, kOneWaves / g.topk), units = g.topk * ks;
    for (int u = wave; u < units; u += kOneWaves) {
        const int slot = u / ks, z = u - slot * ks;
        const int e = g.ids[slot];
        const int kb0 = (int)((long)z * nkb / ks), nb = (int)((long)(z + 1) * nkb / ks) - kb0;
        const uint8_t* wrow = g.w + ((size_t)e * N + n0 + lr) * K + 128 * (size_t)kb0 + 16 * lg;
        const float* srow = g.w_scale + ((size_t)e * (N / 128) + n0 / 128) * nkb + kb0;
        const float* arow = static_cast<const float*>(g.a) + (size_t)slot * K + 128 * (size_t)kb0;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int c0 = 0; c0 < nb; c0 += kChunk) {
            const int cn = min(kChunk, nb - c0);
            // the first blocks' weights are on their way while act is quantised
            constexpr int U = 4;
            uint4 w[U][2];
            auto load = [&](int i) __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const uint8_t* p = wrow + 128 * (size_t)(c0 + min(i + q, cn - 1));
                    w[q][0] = *reinterpret_cast<const uint4*>(p);
                    w[q][1] = *reinterpret_cast<const uint4*>(p + 64);
                }
            };
            load(0);
            for (int i = 0; i < cn; i += 4) {
                const int ib = i + (lane >> 4), l = lane & 15;
                float v[8];
                load8<MOE_F32>(arow, 128 * (size_t)(c0 + min(ib, cn - 1)) + 8 * l, v);
                const BlockQuant bq(row16_max_u32(amax8(v)));
                if (ib < cn) {
                    *reinterpret_cast<uint2*>(&one_q[wave][ib * 128 + 8 * l]) =
                        uint2{bq.pack4(v[0], v[1], v[2], v[3]), bq.pack4(v[4], v[5], v[6], v[7])};
                    if (l == 0) one_s[wave][ib] = bq.scale;
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            for (int i = 0; i < cn; i += U) {
                if (i > 0) load(i);
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    if (i + q >= cn) break;
                    const uint8_t* t = &one_q[wave][(i + q) * 128 + 16 * lg];
                    const f32x4 d = mfma_f8_16x16x128(w[q][0], w[q][1], *reinterpret_cast<const uint4*>(t),
                                                      *reinterpret_cast<const uint4*>(t + 64), f32x4{0.f, 0.f, 0.f, 0.f});
                    const float sc = one_s[wave][i + q] * srow[c0 + i + q];
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(d[v], sc, acc[v]);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the codes are read before the next chunk's
        }
        if (lr == 0) *reinterpret_cast<f32x4*>(&part[u][4 * lg]) = acc;
    }
    __syncthreads();
    if (threadIdx.x < 16) {
        float o = 0.0f;
        for (int j = 0; j < g.topk; ++j) {
            float y = part[j * ks][threadIdx.x];
            for (int z = 1; z < ks; ++z) y += part[j * ks + z][threadIdx.x];
            o = __builtin_fmaf(wts[j], y, o);
        }
        out[n0 + threadIdx.x] = f2bf(o);
    }
}

hipError_t launch_block_down_one(const BlockGemmCall& c, const float* wts, void* out, hipStream_t s) {
    static_assert(kMaxTopk <= kOneUnits, "a unit for every slot");
    BlockArgs a{};
    a.a = c.a;
    a.w = static_cast<const uint8_t*>(c.w);
    a.w_scale = c.w_scale;
    a.topk = c.topk;
    a.N = c.N;
    a.K = c.K;
    a.ids = c.ids;
    hipLaunchKernelGGL(block_down_one_kernel, dim3(c.N / 16), dim3(64 * kOneWaves), 0, s, a, wts, static_cast<uint16_t*>(out));
    return hipGetLastError();
}

// ------------------------------------------------------------------ dispatch

// Experts that M tokens reach under uniform routing.
static double active_experts(int M, int E, int topk) { return E * (1.0 - __builtin_pow(1.0 - (double)topk / E, (double)M)); }

// Rows per tile (alignment) from the rows per expert.  A tile streams its
// weights once, so the tile should hold an expert's rows; a taller one keeps
// more LDS per workgroup than it fills.  gate/up + down, us, 32 / 64 / 128 rows:
// 8 experts of 4096 x 14336 at 18 rows an expert 231 / 231 / 269, at 24 233 / 234
// / 269, at 40 388 / 260 / 288, at 64 548 / 418 / 336; 128 experts of 2048 x 768 at
// 16 115 / 114 / 123, at 32 152 / 122 / 127, at 48 176 / 151 / 141, at 64 214 / 177
// / 148.
int block_tile_rows(int M, int E, int topk) {
    const long per_expert = (long)M * topk / E;
    return per_expert > 48 ? 128 : per_expert > 18 ? 64 : 32;
}

bool block_tile_rows_ok(int block_m) { return block_m == 32 || block_m == 64 || block_m == 128; }

// Whether a layer passes act in float32 (rows kernels).  They start their
// weight stream at once and spread it over 64-row pieces; the tile kernels pay
// for their ring and for whole 128-column blocks, which more than about two
// rounds of workgroups or more rows per expert repay.  gate/up + down, us,
// rows / tiles: 128 experts of 2048 x 768 at 16 tokens (492 workgroups) 69 / 85,
// at 64 (756) 114 / 113; 8 of 4096 x 1024 at 8 rows an expert 26 / 41, at 16
// 40 / 42; 64 of 4096 x 8192 at one token (512) 154 / 134, at 4 465 / 408.
bool block_f32_act(int M, int E, int topk, int I) {
    return (long)M * topk <= 8L * E && (I / 128) * active_experts(M, E, topk) < 512.0;
}

// K splits of the float32-act down GEMM: about three workgroups a CU, each
// split at least one block for every wavefront (one token of 8 experts of 4096 x
// 14336: 48 us unsplit).
int block_down_ksplit(int M, int topk, int E, int N, int K) {
    const long P = (long)M * topk;
    const long wgs = (long)(N / 64) * (P < E ? P : E);
    int ks = (int)((768 + wgs - 1) / wgs);
    if (ks > kMaxKsplit) ks = kMaxKsplit;
    if (ks > K / 128 / 4) ks = K / 128 / 4;  // a block for every wavefront of a split
    return ks < 1 ? 1 : ks;
}

template <int ROUTE>
static hipError_t launch_gate_one(const BlockArgs& a, const BlockGemmCall& c, hipStream_t s) {
    const OneRoute r{*c.spec, c.logits, c.E, c.ids, c.wts};
    hipLaunchKernelGGL((block_rows_kernel<true, true, ROUTE>), dim3(c.N / 64, c.topk, 1), dim3(64 * kRowsWaves<true>), 0, s, a, r);
    return hipGetLastError();
}

hipError_t launch_block_gemm(const BlockGemmCall& c, hipStream_t s) {
    if (c.M == 0) return hipSuccess;
    const int P = c.M * c.topk;
    const BlockArgs a{c.a, c.a_scale, static_cast<const uint8_t*>(c.w), c.w_scale, c.al.sorted_ids, c.al.tile_expert,
                      c.al.expert_counts, c.al.expert_offsets, c.al.active_experts, c.al.expert_offsets + c.E, c.topk, c.N, c.K,
                      P, c.c, c.c_scale, c.ksplit, c.cpart, c.ids, P <= 64L * c.E};
    const int slots = P < c.E ? P : c.E;
    const int64_t cap = moe_align_capacity(c.M, c.topk, c.E, c.block_m);
    if (c.kind == MOE_GEMM_GATE_UP_SILU) {
        if (c.spec) {
            switch (2 * group_mode(*c.spec, c.E, 4) + (c.spec->bias ? 1 : 0)) {
                case 0: return launch_gate_one<0>(a, c, s);
                case 1: return launch_gate_one<1>(a, c, s);
                case 2: return launch_gate_one<2>(a, c, s);
                case 3: return launch_gate_one<3>(a, c, s);
                case 4: return launch_gate_one<4>(a, c, s);
                default: return launch_gate_one<5>(a, c, s);
            }
        }
        if (c.ids)
            hipLaunchKernelGGL((block_rows_kernel<true, true>), dim3(c.N / 64, slots, 1), dim3(64 * kRowsWaves<true>), 0, s, a,
                               NoRoute{});
        else
            hipLaunchKernelGGL((block_rows_kernel<true, false>), dim3(c.N / 64, slots, 1), dim3(256), 0, s, a, NoRoute{});
        return hipGetLastError();
    }
    if (c.kind == MOE_GEMM_DOWN) {
        hipLaunchKernelGGL((block_rows_kernel<false, false>), dim3(c.N / 64, slots, c.ksplit), dim3(256), 0, s, a, NoRoute{});
        return hipGetLastError();
    }
    const bool gate = c.kind == MOE_GEMM_GATE_UP_SILU_E4M3;
    const bool far = (uint64_t)(gate ? c.M : P) * (uint64_t)c.K > 0xffffffffull;
    // Ring depth.  With about one workgroup a CU, only a deep ring keeps enough
    // bytes in flight; with many, a shallow one lets two or more share a CU and
    // hide each other's starts and ends.  us, deep / shallow: down of 8 experts of
    // 4096 x 14336, 256 workgroups, 73 / 108; of 128 of 2048 x 768, 1300, 36 / 29;
    // gate/up of 8 of 4096 x 1024, 64 workgroups, 30 / 44; of 128 of 2048 x 768, 756,
    // 83 / 72.  (128-row tiles: the LDS holds one shape.)
    const double wgs = active_experts(c.M, c.E, c.topk) * (c.N / (gate ? 256 : 128));
    if (gate) {
        if (c.block_m == 128) return launch_tile_c<true, BtCfg<128, 256, 2, 3>>(a, cap, far, s);
        if (c.block_m == 64) return launch_tile_c<true, BtCfg<64, 256, 2, 3>>(a, cap, far, s);
        if (wgs <= 256.0) return launch_tile_c<true, BtCfg<32, 256, 1, 4>>(a, cap, far, s);
        return launch_tile_c<true, BtCfg<32, 256, 1, 2>>(a, cap, far, s);
    }
    if (c.block_m == 128) return launch_tile_c<false, BtCfg<128, 128, 4, 2>>(a, cap, far, s);
    if (c.block_m == 64) {
        if (wgs <= 512.0) return launch_tile_c<false, BtCfg<64, 128, 2, 4>>(a, cap, far, s);
        return launch_tile_c<false, BtCfg<64, 128, 2, 3>>(a, cap, far, s);
    }
    if (wgs <= 512.0) return launch_tile_c<false, BtCfg<32, 128, 1, 4>>(a, cap, far, s);
    return launch_tile_c<false, BtCfg<32, 128, 1, 3>>(a, cap, far, s);
}

}  // namespace moe
