// Block-scaled e4m3 quantisation (moe_quant_block): per block of rows x 128
// values s = max(amax / 448, 2^-126) and codes e4m3(x / s).
#include "moe_block.h"
#include "moe_launch.h"

namespace moe {

// One scale per 128 values of a row: 16 lanes hold a block, 8 values each, so
// that a maximum is four lane moves and a row is read and written once, in whole
// lines.  Bound by memory: 4096 x 14336 float32 49.6 us, 5.9 TB/s.
template <int XDT>
__global__ void __launch_bounds__(256) quant_rows_kernel(const void* __restrict__ x, size_t nblk,
                                                         uint8_t* __restrict__ q, float* __restrict__ scale) {
    quant_rows<XDT>(x, nblk, q, scale, blockIdx.x, gridDim.x, 256);
}

// One scale per 128 x 128 block: a workgroup per block, thread (r, l) holds 8
// values of rows r, r + 16, ..., r + 112, kept in registers from the maximum to
// the codes.  Bound by memory: 16384 x 8192 bfloat16 79 us, 5.1 TB/s.
template <int XDT>
__global__ void __launch_bounds__(256) quant_tile_kernel(const void* __restrict__ x, int rows, int K,
                                                         uint8_t* __restrict__ q, float* __restrict__ scale) {
    __shared__ unsigned wmax[4];
    const int nkb = K / 128;
    const int r0 = (int)(blockIdx.x / nkb) * 128, l = threadIdx.x & 15, rr = threadIdx.x >> 4;
    const size_t col = (size_t)(blockIdx.x % nkb) * 128 + 8 * l;
    float v[8][8];
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + rr + 16 * i;
        if (r < rows) {
            load8<XDT>(x, (size_t)r * K + col, v[i]);
            m = max(m, amax8(v[i]));
        }
    }
    m = wave_max_u32(m);
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
    __syncthreads();
    const BlockQuant bq(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + rr + 16 * i;
        if (r < rows)
            *reinterpret_cast<uint2*>(q + (size_t)r * K + col) =
                uint2{bq.pack4(v[i][0], v[i][1], v[i][2], v[i][3]), bq.pack4(v[i][4], v[i][5], v[i][6], v[i][7])};
    }
    if (threadIdx.x == 0) scale[blockIdx.x] = bq.scale;
}

template <int XDT>
static hipError_t launch_x(const void* x, int rows, int K, int block_rows, void* q, float* scale, hipStream_t s) {
    if (block_rows == 1) {
        const size_t nblk = (size_t)rows * (K / 128);
        const size_t blocks = (nblk + 15) / 16;
        hipLaunchKernelGGL((quant_rows_kernel<XDT>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, x, nblk,
                           static_cast<uint8_t*>(q), scale);
    } else {
        hipLaunchKernelGGL((quant_tile_kernel<XDT>), dim3((unsigned)((size_t)(K / 128) * (((size_t)rows + 127) / 128))), dim3(256), 0, s, x, rows, K,
                           static_cast<uint8_t*>(q), scale);
    }
    return hipGetLastError();
}

hipError_t launch_quant_block(moe_dtype xdt, const void* x, int rows, int K, int block_rows, void* q, float* scale,
                              hipStream_t s) {
    if (rows == 0) return hipSuccess;
    if (xdt == MOE_F32) return launch_x<MOE_F32>(x, rows, K, block_rows, q, scale, s);
    return launch_x<MOE_BF16>(x, rows, K, block_rows, q, scale, s);
}

}  // namespace moe
