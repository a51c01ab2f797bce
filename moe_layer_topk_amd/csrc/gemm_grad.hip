// The grouped expert products as a training step needs them, bfloat16 operands,
// float32 sums:
//
//   z:   z[p][n]     = sum_k x[p / topk][k] W[e][n][k]      (MOE_GEMM_GATE_UP)
//   dx:  da[p][k]    = sum_n dc[p][n] W[e][n][k]            (rows of expert e)
//        through SiLU-and-mul, with (g, u) the kept products z[p] and d = da[p]:
//        dg = d u s (1 + g (1 - s)),  du = d g s,  act = g s u,  s = 1 / (1 + exp(-g))
//   dw:  dW[e][n][k] = sum_{p of e} dc[p][n] a[p][k]
//
// The weights are stored with k contiguous, so dx sums over the rows of W and dw
// over the rows of both operands: what a lane of the matrix instruction wants next
// to each other (eight terms of the sum) lies a row apart.  The tiles therefore go
// to LDS as they lie in memory, by direct copies, and are transposed on the way to
// the registers (ds_read_b64_tr_b16: 16 lanes read four rows of 16 columns and each
// gets a column's four values).
#include <type_traits>

#include "moe_device.h"
#include "moe_launch.h"
#include "moe_tile.h"
#include "moe_train.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kXcds = 8;

// What rows and columns outside a matrix read.
__device__ uint4 grad_zeros[64];

// Rows of B columns (a multiple of 128) in LDS.  The 32-byte piece q of row r lies at
// place q ^ 2 (r mod 4): the 32 lanes that read four rows at two neighbouring pieces
// meet every bank once.
__device__ __forceinline__ int tr_place(int q, int r) { return q ^ ((r & 3) << 1); }

// Eight consecutive rows (terms of the sum) of a column, from LDS byte address
// `at` (the lane's, see tr_lane) and four rows on.
template <int B>
__device__ __forceinline__ bf16x8 tr_read8(unsigned at) {
    struct Two {
        s16x4 lo, hi;
    } v;
    v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at);
    v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(at + 4 * 2 * B));
    return __builtin_bit_cast(bf16x8, v);
}

// The lane's address in a tile at 0 for columns col0 .. col0 + 31 (a multiple of
// 32) and rows 0 .. 15: lanes 0-15 and 16-31 take columns 0-15 and 16-31 of rows
// 0-7, lanes 32-63 the same of rows 8-15.
template <int B>
__device__ __forceinline__ unsigned tr_lane(int lane, int col0) {
    const int g = lane >> 4, i = lane & 15;
    const int r = 8 * (g >> 1) + (i >> 2), q = col0 / 16 + (g & 1);
    return (unsigned)(r * 2 * B + tr_place(q, r) * 32 + (i & 3) * 8);
}

// ------------------------------------------------------------------------ dx
//
// Block tile BM rows (of one expert's run) x 256 output columns, 32 terms of the sum
// a stage in a ring of three; four wavefronts of BM/2 x 128.  The weights are the
// matrix instruction's rows, so a lane ends up with four consecutive columns of a
// token.  kZ is the product itself, whose weights need no transposing.
//
// The gradients take 32 terms a stage, so that two workgroups fit a CU: one multiplies
// while the other starts, waits at a barrier or writes out (down product of 8 experts
// of 4096 x 14336, 8192 rows, through SiLU-and-mul: 1100 us against 1285 with 64 terms
// and one workgroup; 128 experts of 1536 x 2048 at 16 rows 83 and 84).  kZ takes 64: its
// weight rows are read 128 bytes at a time, whole lines, instead of 64 (128 experts of
// 1536 x 2048, 16392 rows: 210 us against 233).
//
// What bounds them: at many rows an expert the copies into LDS, 24 KB for the 2.1 MFLOP of
// a stage (dx above: 11.3 GB at 10 TB/s, loads in flight 91% of the time; 1024 us without
// the epilogue, 740 without the copies too), and with them the power that products,
// transposing reads and copies draw together (0.87 PFLOP/s, matrix cores 50% busy at
// 1.4-1.5 GHz; 16% faster on zeros); at 128 rows the same way from L2 to LDS (8.7 TB/s);
// at 16 rows HBM (518 MB, 6.4 TB/s).
enum DxMode { kDx, kDxSilu, kDxSiluNt, kZ };

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return uint4{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7])};
}

// 16 bytes of a row, NT: past the caches.
template <bool NT>
__device__ __forceinline__ uint4 load16(const void* p) {
    if constexpr (NT) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(static_cast<const u32x4*>(p)));
    return *static_cast<const uint4*>(p);
}
template <bool NT>
__device__ __forceinline__ void store16(void* p, uint4 v) {
    if constexpr (NT)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), static_cast<u32x4*>(p));
    else
        *static_cast<uint4*>(p) = v;
}

// Eight columns through SiLU-and-mul's gradient: d the gradient of act, zg and zu the
// products; dg, du their gradients, ac act.
__device__ __forceinline__ void silu_grad8(const float (&d)[8], uint4 zg, uint4 zu, float (&dg)[8], float (&du)[8],
                                           float (&ac)[8]) {
    const uint32_t ug[4] = {zg.x, zg.y, zg.z, zg.w}, uu[4] = {zu.x, zu.y, zu.z, zu.w};
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const float gv = __uint_as_float((x & 1) ? ug[x / 2] & 0xffff0000u : ug[x / 2] << 16);
        const float uv = __uint_as_float((x & 1) ? uu[x / 2] & 0xffff0000u : uu[x / 2] << 16);
        const float s = 1.0f / (1.0f + __expf(-gv));
        const float gs = gv * s;
        du[x] = d[x] * gs;
        ac[x] = gs * uv;
        dg[x] = d[x] * uv * s * (1.0f + gv * (1.0f - s));
    }
}

template <int BM, int NS_>
struct DxCfg {
    static constexpr int ST = 3, Threads = 256, NS = NS_;  // NS: terms of the sum a stage
    static constexpr int Chunks = NS / 8;                  // 16-byte pieces of a row
    static constexpr int ABytes = BM * NS * 2, WBytes = NS * 512, StageBytes = ABytes + WBytes;
    static constexpr int RowsLoad = 64 / Chunks;           // rows a copy
    static constexpr int ALoads = BM / RowsLoad / 4, WLoads = NS / 8, L = ALoads + WLoads;  // copies a wave and stage
    static constexpr int TM = BM / 64, TN = 4;
    static constexpr int IdsOffset = ST * StageBytes, LdsBytes = IdsOffset + BM * 4;
    // place of piece c of row r: rows that share 256 bytes differ
    __device__ static __forceinline__ int swz(int c, int r) { return c ^ ((r / (16 / Chunks)) % Chunks); }
};

template <int BM, int MODE, bool NTW, int NS>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(NS == 32 ? 2 : 1, 2)))
grad_dx_kernel(GradCall g, int m_tiles, int o_tiles, int group) {
    using C = DxCfg<BM, NS>;
    constexpr bool SILU = MODE == kDxSilu || MODE == kDxSiluNt;
    extern __shared__ __attribute__((aligned(1024))) char grad_lds[];
    // the row tiles that exist, cut into one range for each XCD (of those the grid allows
    // for, a batch of few rows an expert leaves a third or more empty, at the end)
    m_tiles = min(m_tiles, g.al.expert_offsets[g.E] / BM);
    const int nb = m_tiles * o_tiles;
    const int per = (nb + kXcds - 1) / kXcds;
    const int l = blockIdx.x / kXcds, t = (blockIdx.x % kXcds) * per + l;
    if (l >= per || t >= nb) return;
    // groups of `group` weight tiles; inside a group the row tiles advance slowest
    const int ng = t / (group * m_tiles);
    const int gw = min(group, o_tiles - ng * group);
    const int rem = t - ng * group * m_tiles;
    const int mtile = rem / gw, otile = ng * group + rem % gw;
    const int e = g.al.tile_expert[mtile];
    if (e < 0) return;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int N = g.N, K = g.K, P = g.M * g.topk;
    const int S = MODE == kZ ? K : N, O = MODE == kZ ? N : K;  // length of the sum, output columns
    const int o0 = otile * 256;
    const int32_t* sorted = g.al.sorted_ids + (size_t)mtile * BM;
    int* ids_s = reinterpret_cast<int*>(grad_lds + C::IdsOffset);
    for (int i = tid; i < BM; i += C::Threads) ids_s[i] = sorted[i];

    // sources of this wave's copies: rows of dc (kZ: of x), and of W 32 rows n (512 of
    // their bytes; kZ: 256 rows, 128 bytes)
    const char* asrc[C::ALoads];
#pragma unroll
    for (int j = 0; j < C::ALoads; ++j) {
        const int r = (wave * C::ALoads + j) * C::RowsLoad + lane / C::Chunks;
        int p = sorted[r];
        if ((unsigned)p >= (unsigned)P) p = sorted[0];  // padding: any row, its results are dropped
        if (MODE == kZ) p /= g.topk;
        asrc[j] = static_cast<const char*>(g.dc) + (size_t)p * S * 2 + C::swz(lane % C::Chunks, r) * 16;
    }
    // (columns past the last read the next row, past the last row zeros; they are dropped)
    const v4i_rsrc wrsrc = buf_rsrc(static_cast<const char*>(g.w) + (size_t)e * N * K * 2, (unsigned)((size_t)N * K * 2));
    unsigned wsrc[C::WLoads];
#pragma unroll
    for (int j = 0; j < C::WLoads; ++j) {
        if constexpr (MODE == kZ) {
            const int r = (wave * C::WLoads + j) * C::RowsLoad + lane / C::Chunks;
            wsrc[j] = (unsigned)((size_t)(o0 + r) * K * 2) + C::swz(lane % C::Chunks, r) * 16;
        } else {
            const int r = (wave * C::WLoads + j) * 2 + (lane >> 5), c = lane & 31;
            wsrc[j] = (unsigned)(((size_t)r * K + o0) * 2) + (tr_place(c >> 1, r) * 2 + (c & 1)) * 16;
        }
    }
    const unsigned wstep = MODE == kZ ? C::NS * 2 : (unsigned)C::NS * 2 * K;  // bytes from a stage to the next
    const unsigned lds0 = lds_addr_of(grad_lds);
    auto issue_part = [&](int kt, int j0, int j1) {
        const unsigned st = lds0 + (unsigned)((kt % C::ST) * C::StageBytes);
#pragma unroll
        for (int j = 0; j < C::L; ++j) {
            if (j < j0 || j >= j1) continue;
            if (j < C::ALoads)
                lds_dma16_at(asrc[j] + (size_t)kt * (C::NS * 2), st + (wave * C::ALoads + j) * 1024);
            else if constexpr (NTW)
                lds_dma16_buf_nt(wrsrc, wsrc[j - C::ALoads], kt * wstep,
                                 st + C::ABytes + (wave * C::WLoads + (j - C::ALoads)) * 1024);
            else
                lds_dma16_buf(wrsrc, wsrc[j - C::ALoads], kt * wstep,
                              st + C::ABytes + (wave * C::WLoads + (j - C::ALoads)) * 1024);
        }
    };

    f32x16 acc[C::TM][C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    int arow[C::TM];
#pragma unroll
    for (int i = 0; i < C::TM; ++i) arow[i] = wm * (BM / 2) + 32 * i + (lane & 31);
    unsigned wlane[C::TN];
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
        wlane[j] = C::ABytes + (MODE == kZ ? (wn * 128 + 32 * j + (lane & 31)) * (C::NS * 2) : tr_lane<256>(lane, wn * 128 + 32 * j));
    // 32-row groups of the tile that hold no pair are left out
    const int nreal = min(BM, g.al.expert_offsets[e] + g.al.expert_counts[e] - mtile * BM);
    const int live = __builtin_amdgcn_readfirstlane(min(C::TM, max(0, (nreal - wm * (BM / 2) + 31) / 32)));

    const int nk = S / C::NS;
#pragma unroll
    for (int s0 = 0; s0 < C::ST - 1; ++s0)
        if (s0 < nk) issue_part(s0, 0, C::L);
    auto stage = [&](int kt, auto pf_tag, auto lt_tag) {
        constexpr bool pf = decltype(pf_tag)::value;
        constexpr int LT = decltype(lt_tag)::value;
        if constexpr (pf)
            wait_vm<(C::ST - 2) * C::L>();
        else
            wait_vm_runtime<C::L>(min(C::ST - 2, nk - 1 - kt));
        __syncthreads();
        const unsigned st = lds0 + (unsigned)((kt % C::ST) * C::StageBytes);
        const char* sa = grad_lds + (kt % C::ST) * C::StageBytes;
        bf16x8 af[2][C::TM], wf[2][C::TN];
        auto read_frags = [&](int buf, int ks) {
            const int c = ks * 2 + (lane >> 5);
#pragma unroll
            for (int i = 0; i < LT; ++i)
                af[buf][i] = *reinterpret_cast<const bf16x8*>(sa + arow[i] * (C::NS * 2) + (C::swz(c, arow[i]) << 4));
#pragma unroll
            for (int j = 0; j < C::TN; ++j)
                if constexpr (LT > 0) {
                    if constexpr (MODE == kZ)
                        wf[buf][j] = *reinterpret_cast<const bf16x8*>(sa + wlane[j] + (C::swz(c, lane & 31) << 4));
                    else
                        wf[buf][j] = tr_read8<256>(st + wlane[j] + ks * 16 * 512);
                }
        };
        read_frags(0, 0);
#pragma unroll
        for (int ks = 0; ks < C::NS / 16; ++ks) {
            const int cur = ks & 1;
            if (ks + 1 < C::NS / 16) read_frags(cur ^ 1, ks + 1);
            // this substep's share of the next copies, between the products
            const int j0 = ks * C::L / (C::NS / 16), j1 = (ks + 1) * C::L / (C::NS / 16);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < C::TM * C::TN; ++q) {
                const int i = q / C::TN, j = q % C::TN;
                if (i < LT) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[cur][j], af[cur][i], acc[i][j], 0, 0, 0);
                if (pf && (q & 1) && j0 + q / 2 < j1) {
                    __builtin_amdgcn_sched_barrier(0);
                    issue_part(kt + C::ST - 1, j0 + q / 2, j0 + q / 2 + 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (pf && C::TM * C::TN / 2 < j1 - j0) issue_part(kt + C::ST - 1, j0 + C::TM * C::TN / 2, j1);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int nmain = nk - (C::ST - 1) > 0 ? nk - (C::ST - 1) : 0;
    auto kloop = [&](auto lt) {
        for (int kt = 0; kt < nmain; ++kt) stage(kt, std::true_type{}, lt);
        for (int kt = nmain; kt < nk; ++kt) stage(kt, std::false_type{}, lt);
    };
    if (live == C::TM)
        kloop(std::integral_constant<int, C::TM>{});
    else if (C::TM > 1 && live == 1)
        kloop(std::integral_constant<int, 1>{});
    else
        kloop(std::integral_constant<int, 0>{});

    // ---- epilogue: 32 rows x 64 columns at a time through the wave's LDS (rows padded by
    // 16 bytes), so that memory sees whole lines
    __syncthreads();
    constexpr int kElem = SILU ? 4 : 2, kRow = 64 * kElem + 16;
    static_assert(4 * 32 * kRow <= C::IdsOffset, "epilogue");
    char* mine = grad_lds + wave * 32 * kRow;
    const int c8 = (lane & 7) * 8;
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
        if (i >= live) break;
        const int r0 = wm * (BM / 2) + 32 * i, rows = min(32, nreal - r0);
#pragma unroll
        for (int jh = 0; jh < 2; ++jh) {
            const int col = o0 + wn * 128 + 64 * jh + c8;
            size_t p[4];
            uint4 zg[4], zu[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = 8 * q + (lane >> 3);
                p[q] = (size_t)ids_s[r0 + min(r, rows - 1)];
                if (SILU && col < O) {
                    const uint16_t* z = static_cast<const uint16_t*>(g.z) + p[q] * 2 * O + col;
                    zg[q] = load16<MODE == kDxSiluNt>(z), zu[q] = load16<MODE == kDxSiluNt>(z + O);
                }
            }
#pragma unroll
            for (int j = 2 * jh; j < 2 * jh + 2; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    char* at = mine + (lane & 31) * kRow + (32 * (j & 1) + 8 * v + 4 * (lane >> 5)) * kElem;
                    const float x0 = acc[i][j][4 * v], x1 = acc[i][j][4 * v + 1], x2 = acc[i][j][4 * v + 2],
                                x3 = acc[i][j][4 * v + 3];
                    if constexpr (SILU)
                        *reinterpret_cast<float4*>(at) = make_float4(x0, x1, x2, x3);
                    else
                        *reinterpret_cast<uint2*>(at) = uint2{pack_bf2(x0, x1), pack_bf2(x2, x3)};
                }
            if (col >= O) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = 8 * q + (lane >> 3);
                if (r >= rows) continue;
                const char* at = mine + r * kRow + c8 * kElem;
                if constexpr (SILU) {
                    const float4 d0 = *reinterpret_cast<const float4*>(at), d1 = *reinterpret_cast<const float4*>(at + 16);
                    const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
                    float dg[8], du[8], ac[8];
                    silu_grad8(d, zg[q], zu[q], dg, du, ac);
                    uint16_t* o = static_cast<uint16_t*>(g.out) + p[q] * 2 * O + col;
                    store16<MODE == kDxSiluNt>(o, pack8(dg));
                    store16<MODE == kDxSiluNt>(o + O, pack8(du));
                    if (g.act)
                        store16<MODE == kDxSiluNt>(static_cast<uint16_t*>(g.act) + p[q] * O + col, pack8(ac));
                } else {
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.out) + p[q] * O + col) = *reinterpret_cast<const uint4*>(at);
                }
            }
        }
    }
}

template <int BM, int MODE, bool NTW, int NS>
static hipError_t launch_dx_t(const GradCall& c, hipStream_t s) {
    using C = DxCfg<BM, NS>;
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&grad_dx_kernel<BM, MODE, NTW, NS>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, C::LdsBytes);
    if (attr != hipSuccess) return attr;
    const int m_tiles = (int)(moe_align_capacity(c.M, c.topk, c.E, BM) / BM), o_tiles = ((MODE == kZ ? c.N : c.K) + 255) / 256;
    const int64_t nb = (int64_t)m_tiles * o_tiles;
    // weight tiles a group: all of few (an XCD reads each row tile once), else two (down
    // product of 4096 x 14336, 4096 tokens: 1, 2, 4, 7, 8, 14 967, 980, 997, 972, 999, 1040
    // us; plain gate/up of 28672 x 4096 1910, 1889, 1922, 1965, 1934, 2097)
    const int group = o_tiles <= 8 ? o_tiles : 2;
    hipLaunchKernelGGL((grad_dx_kernel<BM, MODE, NTW, NS>), dim3((unsigned)((nb + kXcds - 1) / kXcds * kXcds)), dim3(C::Threads),
                       C::LdsBytes, s, c, m_tiles, o_tiles, group);
    return hipGetLastError();
}

// The same products where few workgroups would run: 64 rows x 128 columns a workgroup,
// and of each stage of 128 terms a quarter for each of four groups of four wavefronts
// (2 x 2 of 32 x 64), which have their own part of the ring; their sums are joined
// through LDS, in order.  The time of a stage is its copies' way (0.5 us), whatever their
// size: what helps are fewer stages and more workgroups.  Times below, at dx_few.
struct SplitCfg {
    static constexpr int BM = 64, BN = 128, G = 4, NS = 32, ST = 3, Threads = 256 * G;
    static constexpr int ABytes = BM * NS * 2, WBytes = BN * NS * 2, PartBytes = ABytes + WBytes, StageBytes = G * PartBytes;
    static constexpr int L = 3;                                  // copies a wave and stage
    static constexpr int kRow = BN * 4 + 16, JoinBytes = BM * kRow;  // a group's sums
    static constexpr int IdsOffset = ST * StageBytes, LdsBytes = IdsOffset + BM * 4;
    static_assert(G * JoinBytes <= IdsOffset, "sums");
    __device__ static __forceinline__ int swz(int c, int r) { return c ^ ((r / 4) % 4); }
};

template <int MODE>
__global__ void __launch_bounds__(SplitCfg::Threads) grad_dx_split_kernel(GradCall g, int o_tiles) {
    using C = SplitCfg;
    extern __shared__ __attribute__((aligned(1024))) char grad_lds[];
    // (64-row parts of the list, whatever its block_m)
    const int units = g.al.expert_offsets[g.E] / C::BM, nb = units * o_tiles, per = (nb + kXcds - 1) / kXcds;
    const int l = blockIdx.x / kXcds, t = (blockIdx.x % kXcds) * per + l;
    if (l >= per || t >= nb) return;
    const int unit = t / o_tiles, o0 = (t % o_tiles) * C::BN;
    const int e = g.al.tile_expert[unit * C::BM / g.block_m];
    if (e < 0) return;
    const int nreal = min(C::BM, g.al.expert_offsets[e] + g.al.expert_counts[e] - unit * C::BM);
    if (nreal <= 0) return;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int grp = wave >> 2, wv = wave & 3, wm = wv >> 1, wn = wv & 1;
    const int N = g.N, K = g.K, P = g.M * g.topk;
    const int S = MODE == kZ ? K : N, O = MODE == kZ ? N : K;
    const int32_t* sorted = g.al.sorted_ids + (size_t)unit * C::BM;
    int* ids_s = reinterpret_cast<int*>(grad_lds + C::IdsOffset);
    if (tid < C::BM) ids_s[tid] = sorted[tid];

    // one copy of 16 rows of dc (kZ: of x) and two of W a wavefront and stage
    const int ar = wv * 16 + (lane >> 2);
    int ap = sorted[ar];
    if ((unsigned)ap >= (unsigned)P) ap = sorted[0];
    if (MODE == kZ) ap /= g.topk;
    const char* asrc = static_cast<const char*>(g.dc) + (size_t)ap * S * 2 + grp * (C::NS * 2) + C::swz(lane & 3, ar) * 16;
    const v4i_rsrc wrsrc = buf_rsrc(static_cast<const char*>(g.w) + (size_t)e * N * K * 2, (unsigned)((size_t)N * K * 2));
    unsigned wsrc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (MODE == kZ) {
            const int r = (wv * 2 + j) * 16 + (lane >> 2);
            wsrc[j] = (unsigned)((size_t)(o0 + r) * K * 2) + grp * (C::NS * 2) + C::swz(lane & 3, r) * 16;
        } else {
            const int r = (wv * 2 + j) * 4 + (lane >> 4), c = lane & 15;
            wsrc[j] = (unsigned)(((size_t)(grp * C::NS + r) * K + o0) * 2) + (tr_place(c >> 1, r) * 2 + (c & 1)) * 16;
        }
    }
    const unsigned astep = C::G * C::NS * 2, wstep = MODE == kZ ? astep : astep * (unsigned)K;
    const unsigned lds0 = lds_addr_of(grad_lds) + grp * C::PartBytes;
    auto issue = [&](int kt) {
        const unsigned st = lds0 + (unsigned)((kt % C::ST) * C::StageBytes);
        lds_dma16_at(asrc + (size_t)kt * astep, st + wv * 1024);
#pragma unroll
        for (int j = 0; j < 2; ++j) lds_dma16_buf(wrsrc, wsrc[j], kt * wstep, st + C::ABytes + (wv * 2 + j) * 1024);
    };

    f32x16 acc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][v] = 0.0f;
    const int arow = wm * 32 + (lane & 31);
    unsigned wlane[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        wlane[j] = C::ABytes + (MODE == kZ ? (wn * 64 + 32 * j + (lane & 31)) * (C::NS * 2) : tr_lane<C::BN>(lane, wn * 64 + 32 * j));
    const bool live = nreal > wm * 32;

    const int nk = S / (C::G * C::NS);
#pragma unroll
    for (int s0 = 0; s0 < C::ST - 1; ++s0)
        if (s0 < nk) issue(s0);
    for (int kt = 0; kt < nk; ++kt) {
        if (kt + C::ST - 1 < nk)
            wait_vm<(C::ST - 2) * C::L>();
        else
            wait_vm_runtime<C::L>(min(C::ST - 2, nk - 1 - kt));
        __syncthreads();
        if (kt + C::ST - 1 < nk) issue(kt + C::ST - 1);
        if (live) {
            const unsigned off = (unsigned)((kt % C::ST) * C::StageBytes);
            const char* sa = grad_lds + grp * C::PartBytes + off;
#pragma unroll
            for (int ks = 0; ks < C::NS / 16; ++ks) {
                const int c = ks * 2 + (lane >> 5);
                const bf16x8 af = *reinterpret_cast<const bf16x8*>(sa + arow * (C::NS * 2) + (C::swz(c, arow) << 4));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    bf16x8 wf;
                    if constexpr (MODE == kZ)
                        wf = *reinterpret_cast<const bf16x8*>(sa + wlane[j] + (C::swz(c, lane & 31) << 4));
                    else
                        wf = tr_read8<C::BN>(lds0 + off + wlane[j] + ks * 16 * (2 * C::BN));
                    acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf, af, acc[j], 0, 0, 0);
                }
            }
        }
    }

    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            *reinterpret_cast<float4*>(grad_lds + grp * C::JoinBytes + arow * C::kRow +
                                       (wn * 64 + 32 * j + 8 * v + 4 * (lane >> 5)) * 4) =
                make_float4(acc[j][4 * v], acc[j][4 * v + 1], acc[j][4 * v + 2], acc[j][4 * v + 3]);
    __syncthreads();
    const int r = tid >> 4, c8 = (tid & 15) * 8;  // eight columns a thread
    if (r >= nreal) return;
    const size_t p = (size_t)ids_s[r];
    float d[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const char* at = grad_lds + r * C::kRow + (c8 + 4 * h) * 4;
        float4 sum = *reinterpret_cast<const float4*>(at);
#pragma unroll
        for (int q = 1; q < C::G; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(at + q * C::JoinBytes);
            sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
        }
        d[4 * h] = sum.x, d[4 * h + 1] = sum.y, d[4 * h + 2] = sum.z, d[4 * h + 3] = sum.w;
    }
    const int col = o0 + c8;
    uint16_t* out = static_cast<uint16_t*>(g.out);
    if constexpr (MODE == kDxSilu) {
        const uint16_t* z = static_cast<const uint16_t*>(g.z) + p * 2 * O + col;
        float dg[8], du[8], ac[8];
        silu_grad8(d, load16<false>(z), load16<false>(z + O), dg, du, ac);
        uint16_t* o = out + p * 2 * O + col;
        store16<false>(o, pack8(dg));
        store16<false>(o + O, pack8(du));
        if (g.act) store16<false>(static_cast<uint16_t*>(g.act) + p * O + col, pack8(ac));
    } else {
        store16<false>(out + p * O + col, pack8(d));
    }
}

// Up to 300 workgroups of it (of a guess: every expert hit, the last part of each half
// full).  Regular against split, us, with its workgroups, on the same inputs again and
// again (on inputs that change from call to call the first of them 168 and 83, the one of
// 5888 terms 73 and 31, the one of 2560 terms 31 and 19): dx of 8 experts, 2112 rows, 11008
// terms, 168: 147 and 64; 128 experts of 1536 x 2048, 8 rows, 128: 22 and 12; 4096 terms,
// 288: 59 and 51; 1536 terms, 464: 29 and 32; through SiLU, 5888 terms, 39: 71 and 30;
// 1024 terms, 576: 31 and 37; gate/up of 2560 terms, 32: 30 and 14; 2432 terms, 260: 34
// and 21; 2048 terms, 348: 32 and 34; 1024 terms, 384: 18 and 23.
static bool dx_few(const GradCall& c, int O) {
    const int64_t P = (int64_t)c.M * c.topk, hit = P < c.E ? P : c.E, full = P / SplitCfg::BM + hit / 2;
    return (hit > full ? hit : full) * (O / SplitCfg::BN) <= 300;
}

template <int MODE>
static hipError_t launch_dx_split(const GradCall& c, hipStream_t s) {
    using C = SplitCfg;
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&grad_dx_split_kernel<MODE>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, C::LdsBytes);
    if (attr != hipSuccess) return attr;
    const int o_tiles = (MODE == kZ ? c.N : c.K) / C::BN;
    const int64_t nb = moe_align_capacity(c.M, c.topk, c.E, c.block_m) / C::BM * o_tiles;
    hipLaunchKernelGGL((grad_dx_split_kernel<MODE>), dim3((unsigned)((nb + kXcds - 1) / kXcds * kXcds)), dim3(C::Threads),
                       C::LdsBytes, s, c, o_tiles);
    return hipGetLastError();
}

// Weights go past the caches (non-temporal) while an expert's rows mostly fit one row
// tile: dx of 128 experts of 1536 x 2048 at 16 rows each 136 -> 123 us, at 96 167 -> 153,
// at 128 203 against 224; gate/up of 8 of 28672 x 4096 at 16 320 -> 293, at 96 355 -> 333,
// at 128 408 against 491.
template <int BM, int MODE>
static hipError_t launch_dx_w(const GradCall& c, hipStream_t s) {
    constexpr int NS = MODE == kZ ? 64 : 32;
    return (int64_t)c.M * c.topk <= 96ll * c.E ? launch_dx_t<BM, MODE, true, NS>(c, s) : launch_dx_t<BM, MODE, false, NS>(c, s);
}

template <int MODE>
static hipError_t launch_dx_m(const GradCall& c, hipStream_t s) {
    if (dx_few(c, MODE == kZ ? c.N : c.K)) return launch_dx_split<MODE == kDxSiluNt ? kDxSilu : MODE>(c, s);
    return c.block_m == 128 ? launch_dx_w<128, MODE>(c, s) : launch_dx_w<64, MODE>(c, s);
}

// Past 96 MB of z, its gradients and activations they go past the caches (128 experts of
// 2048 x 768, 16384 rows, 126 MB: 165 -> 148 us; 8 of 4096 x 14336, 8192 rows: 1145 ->
// 1119; at 4096 rows of 128 experts, 31 MB, a tie).
hipError_t launch_grad_dx(const GradCall& c, hipStream_t s) {
    if (c.z && (int64_t)c.M * c.topk * c.K * 10 > (96ll << 20)) return launch_dx_m<kDxSiluNt>(c, s);
    return c.z ? launch_dx_m<kDxSilu>(c, s) : launch_dx_m<kDx>(c, s);
}

hipError_t launch_gate_up(const GradCall& c, hipStream_t s) { return launch_dx_m<kZ>(c, s); }

// ------------------------------------------------------------------------ dw
//
// Block tile B x B of one expert's matrix, 32 pair rows a stage in a ring; wavefronts
// of 64 n x B/2 k.  Both operands are transposed on the way to the registers.  Rows
// past the expert's last and columns past the matrix read zeros.  Every XCD takes an
// eighth of each expert's tiles: experts with many rows are shared by all of the chip.
//
// B = 256: eight wavefronts, two a SIMD, a workgroup a CU; bound by the power that
// products, LDS reads and copies draw together (the clock falls to 1.7 GHz).  B = 128:
// four wavefronts and a third of the LDS, three workgroups a CU, so that one begins
// while another is stored: for experts of few rows, whose results' stores are the work, and
// where few workgroups of the larger tile would run.

template <int B>
struct DwCfg {
    static constexpr int ST = B == 256 ? 4 : 3, RP = 32;
    static constexpr int WN = B / 64, Waves = 2 * WN, Threads = 64 * Waves, TN = B / 64;  // TN: 32-column tiles k of a wavefront
    static constexpr int RowBytes = 2 * B, HalfBytes = RP * RowBytes, StageBytes = 2 * HalfBytes;
    static constexpr int RowLanes = RowBytes / 16, CopyRows = 64 / RowLanes;  // lanes of a row, rows of a copy
    static constexpr int Ids = B == 256 ? 2048 : 512;  // rows between refills of the row lists
    static constexpr int IdsOffset = ST * StageBytes, LdsBytes = IdsOffset + Ids * 8;
    static constexpr int L = 4;  // copies a wave and stage: two of dc's rows, two of a's
    static_assert(RP == 2 * CopyRows * Waves, "copies");
};

template <int ODT, int B>
__global__ void __launch_bounds__(DwCfg<B>::Threads) __attribute__((amdgpu_waves_per_eu(B == 256 ? 2 : 3, B == 256 ? 2 : 3)))
grad_dw_kernel(GradCall g, int n_tiles, int k_tiles, int per_xcd) {
    using C = DwCfg<B>;
    extern __shared__ __attribute__((aligned(1024))) char grad_lds[];
    const int xcd = blockIdx.x % kXcds, l = blockIdx.x / kXcds;
    const int e = l / per_xcd, t = xcd * per_xcd + l % per_xcd;
    if (t >= n_tiles * k_tiles) return;
    // groups of four k tiles, n tiles in order: what runs together on an XCD covers
    // a few of each
    const int gk = t / (n_tiles * 4), gw = min(4, k_tiles - gk * 4), rem = t - gk * n_tiles * 4;
    const int n0 = (rem / gw) * B, k0 = (gk * 4 + rem % gw) * B;
    const int N = g.N, K = g.K;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave >> 1, wk = wave & 1;
    const int count = g.al.expert_counts[e];
    const int32_t* sorted = g.al.sorted_ids + g.al.expert_offsets[e];
    int2* ids_s = reinterpret_cast<int2*>(grad_lds + C::IdsOffset);  // rows of dc and of a, -1: zeros

    // copy j of the wave: rows lrow + j CopyRows of a stage (a row: RowLanes lanes).  A lane
    // whose columns lie past the matrix reads zeros.
    const int c = lane % C::RowLanes, lrow = 2 * C::CopyRows * wave + lane / C::RowLanes;
    const char* zeros = reinterpret_cast<const char*>(grad_zeros) + c * 16;
    const char *abase[2], *bbase[2];
    unsigned ald[2], bld[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int lc = (tr_place(c >> 1, lrow + C::CopyRows * j) * 2 + (c & 1)) * 8;
        abase[j] = n0 + lc < N ? static_cast<const char*>(g.dc) + (size_t)(n0 + lc) * 2 : zeros;
        bbase[j] = k0 + lc < K ? static_cast<const char*>(g.a) + (size_t)(k0 + lc) * 2 : zeros;
        ald[j] = n0 + lc < N ? (unsigned)N * 2 : 0;
        bld[j] = k0 + lc < K ? (unsigned)K * 2 : 0;
    }
    const unsigned lds0 = lds_addr_of(grad_lds);
    f32x16 acc[2][C::TN];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    unsigned nlane[2], klane[C::TN];
#pragma unroll
    for (int i = 0; i < 2; ++i) nlane[i] = tr_lane<B>(lane, wn * 64 + 32 * i);
#pragma unroll
    for (int j = 0; j < C::TN; ++j) klane[j] = C::HalfBytes + tr_lane<B>(lane, wk * (B / 2) + 32 * j);

    for (int base = 0; base < count; base += C::Ids) {
        const int n = min(C::Ids, count - base), nst = (n + C::RP - 1) / C::RP;
        __syncthreads();
        for (int i = tid; i < nst * C::RP; i += C::Threads) {
            const int p = i < n ? sorted[base + i] : -1;
            ids_s[i] = int2{p, g.per_token && p >= 0 ? p / g.topk : p};
        }
        __syncthreads();
        int2 id[2];  // of the next stage to be copied
        auto fetch_ids = [&](int kt) {
            id[0] = ids_s[kt * C::RP + lrow];
            id[1] = ids_s[kt * C::RP + lrow + C::CopyRows];
        };
        auto issue = [&](int kt, int j) {
            const char* pa = abase[j] + (size_t)(unsigned)id[j].x * ald[j];
            const char* pb = bbase[j] + (size_t)(unsigned)id[j].y * bld[j];
            pa = id[j].x < 0 ? zeros : pa;
            pb = id[j].x < 0 ? zeros : pb;
            const unsigned at = lds0 + (unsigned)((kt % C::ST) * C::StageBytes) + (2 * wave + j) * 1024;
            lds_dma16_at(pa, at);
            lds_dma16_at(pb, at + C::HalfBytes);
        };
        for (int s0 = 0; s0 < C::ST - 1; ++s0)
            if (s0 < nst) {
                fetch_ids(s0);
                issue(s0, 0);
                issue(s0, 1);
            }
        if (C::ST - 1 < nst) fetch_ids(C::ST - 1);
        auto stage = [&](int kt, auto pf_tag) {
            constexpr bool pf = decltype(pf_tag)::value;
            if constexpr (pf)
                wait_vm<(C::ST - 2) * C::L>();
            else
                wait_vm_runtime<C::L>(min(C::ST - 2, nst - 1 - kt));
            __syncthreads();
            const unsigned st = lds0 + (unsigned)((kt % C::ST) * C::StageBytes);
            // the first half's fragments, then its products with the second half's reads and
            // the copies between them: a wavefront that read both halves first kept the
            // others' first reads waiting (3.88 -> 3.66 million cycles, 2060 -> 2022 us)
            bf16x8 nf[2][2], kf[2][C::TN];
            auto read = [&](int ks, int m) {  // the order they are used in
                if (m == 0 || m == C::TN + 1)
                    nf[ks][m ? 1 : 0] = tr_read8<B>(st + nlane[m ? 1 : 0] + ks * 16 * C::RowBytes);
                else
                    kf[ks][m - 1] = tr_read8<B>(st + klane[m - 1] + ks * 16 * C::RowBytes);
            };
#pragma unroll
            for (int m = 0; m < C::TN + 2; ++m) read(0, m);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < 4 * C::TN; ++q) {
                const int ks = q / (2 * C::TN), i = q / C::TN % 2, j = q % C::TN;
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[ks][j], nf[ks][i], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (q < C::TN + 2) read(1, q);
                if (pf && q == 1) issue(kt + C::ST - 1, 0);
                if (pf && q == C::TN + 1) issue(kt + C::ST - 1, 1);
                if (pf && q == 3 * C::TN && kt + C::ST < nst) fetch_ids(kt + C::ST);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        const int nmain = max(0, nst - (C::ST - 1));
        for (int kt = 0; kt < nmain; ++kt) stage(kt, std::true_type{});
        for (int kt = nmain; kt < nst; ++kt) stage(kt, std::false_type{});
    }

    // ---- epilogue: 32 n rows of the wave's tile at a time through LDS.  In float32 they
    // reach past the ring into the row lists, which nothing reads any more: a workgroup
    // has this one tile (one that went on to another would fetch wild rows).
    __syncthreads();
    constexpr int kElem = ODT == MOE_F32 ? 4 : 2, kRow = 32 * C::TN * kElem + 16;
    static_assert(C::Waves * 32 * kRow <= C::LdsBytes, "epilogue");
    char* mine = grad_lds + wave * 32 * kRow;
    char* out = static_cast<char*>(g.out) + (size_t)e * N * K * kElem;
    constexpr int kLanes = 32 * C::TN * kElem / 16;  // of a row
    const int col = k0 + wk * (B / 2) + (lane % kLanes) * (16 / kElem);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                char* at = mine + (lane & 31) * kRow + (32 * j + 8 * v + 4 * (lane >> 5)) * kElem;
                const float x0 = acc[i][j][4 * v], x1 = acc[i][j][4 * v + 1], x2 = acc[i][j][4 * v + 2],
                            x3 = acc[i][j][4 * v + 3];
                if constexpr (ODT == MOE_F32)
                    *reinterpret_cast<float4*>(at) = make_float4(x0, x1, x2, x3);
                else
                    *reinterpret_cast<uint2*>(at) = uint2{pack_bf2(x0, x1), pack_bf2(x2, x3)};
            }
#pragma unroll
        for (int q = 0; q < 32 * kLanes / 64; ++q) {
            const int r = q * (64 / kLanes) + lane / kLanes, n = n0 + wn * 64 + 32 * i + r;
            const uint4 v = *reinterpret_cast<const uint4*>(mine + r * kRow + (lane % kLanes) * 16);
            // (non-temporal: 128 experts of 2048 x 768 in float32 175 -> 150 us)
            if (n < N && col < K)
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(out + ((size_t)n * K + col) * kElem));
        }
    }
}

template <int ODT, int B>
static hipError_t launch_dw_t(const GradCall& c, hipStream_t s) {
    using C = DwCfg<B>;
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&grad_dw_kernel<ODT, B>),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, C::LdsBytes);
    if (attr != hipSuccess) return attr;
    const int n_tiles = (c.N + B - 1) / B, k_tiles = (c.K + B - 1) / B;
    const int per_xcd = (n_tiles * k_tiles + kXcds - 1) / kXcds;
    hipLaunchKernelGGL((grad_dw_kernel<ODT, B>), dim3((unsigned)(kXcds * c.E * per_xcd)), dim3(C::Threads), C::LdsBytes, s, c,
                       n_tiles, k_tiles, per_xcd);
    return hipGetLastError();
}

template <int ODT>
static hipError_t launch_dw_o(const GradCall& c, hipStream_t s) {
    // B = 128 for experts of up to 8 M weights and 192 rows on average: 128 experts of 2048
    // x 768 at 64 rows each float32 146 -> 141 us, bfloat16 97 -> 84, at 192 rows 192 ->
    // 173 and 150 -> 140, at 512 rows 349 against 387 and 288 against 311; of 1536 x 2048
    // at 64 rows 279 -> 264 and 180 -> 169.  Matrices of 4096 x 14336 at 64 rows: float32
    // 353 against 386, bfloat16 212 and 202.
    // Also where 256 x 256 tiles are up to 160 workgroups, with any rows: 4 of 512 x 512 at
    // 1024 rows each 27 -> 16 us, 8 of 1024 x 1024 at 512 rows (128 workgroups) 19 -> 16, at
    // 1024 rows 29 -> 28; of 2048 x 1024 at 1024 rows (256) 38 against 45.
    const int64_t large = (int64_t)c.E * ((c.N + 255) / 256) * ((c.K + 255) / 256);
    const bool small = large <= 160 || ((int64_t)c.N * c.K <= (8 << 20) && (int64_t)c.M * c.topk <= 192ll * c.E);
    return small ? launch_dw_t<ODT, 128>(c, s) : launch_dw_t<ODT, 256>(c, s);
}

hipError_t launch_grad_dw(const GradCall& c, hipStream_t s) {
    return c.out_dtype == MOE_F32 ? launch_dw_o<MOE_F32>(c, s) : launch_dw_o<MOE_BF16>(c, s);
}

}  // namespace moe
