// hl_fp8_quant.cu -- headloss_fp8_quantize (include/headloss_fp8.h): a matrix and / or its
// transpose in 8-bit floating point with a scale for each block of 128.
//
// One CTA a 128 x 128 tile, which holds whole blocks of every kind.  A thread has 8 rows x 8
// columns in registers: the row maxima join over the 16 lanes of a row, the column maxima over
// the 16 row groups through shared memory.  The transpose's codes are turned 8 x 8 in registers
// and leave through a 16 KB tile in shared memory whose 8-byte units are placed by XOR, so that
// both its writes and its reads touch every bank once and global stores are whole 128-byte rows.
// HBM bound: each input element is read once, each code written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "headloss.h"
#include "headloss_fp8.h"

namespace hl_fp8 {

constexpr int QT = 128;        // tile edge
constexpr int QTHREADS = 256;
constexpr float LEAST = 1.17549435e-38f;  // 2^-126: 1 / s stays finite

struct QuantArgs {
    const void* x;
    int64_t rows, cols, ld;
    int vec;     // rows start on 16-byte boundaries
    int e5m2;
    float inv_top;
    unsigned char* q;
    int64_t ldq;
    float* scales;
    int block;
    unsigned char* qt;
    int64_t ldqt;
    float* scales_t;
    int block_t;
    int col_tiles, row_tiles;
};

__device__ __forceinline__ float scale_of(uint32_t amax_bits, float inv_top) {
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return fmaxf(__fmul_rn(__uint_as_float(amax_bits), inv_top), LEAST);
}
__device__ __forceinline__ uint32_t code2(float a, float b, int e5m2) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, e5m2 ? __NV_E5M2 : __NV_E4M3);
}
__device__ __forceinline__ uint2 code8(const float (&v)[8], int e5m2) {
    return make_uint2(code2(v[0], v[1], e5m2) | code2(v[2], v[3], e5m2) << 16,
                      code2(v[4], v[5], e5m2) | code2(v[6], v[7], e5m2) << 16);
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if (DT == HEADLOSS_FP32) return static_cast<const float*>(p)[i];
    if (DT == HEADLOSS_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if (DT == HEADLOSS_FP32) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = f[0], b = f[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = DT == HEADLOSS_BF16
                                 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[k]))
                                 : __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(QTHREADS) quantize_kernel(const QuantArgs a) {
    __shared__ uint32_t wmax[8][QT];            // column maxima of each warp, or the warps' maxima
    __shared__ float cscale[QT];
    __shared__ __align__(16) uint2 turned[QT][16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = tid >> 4, c = tid & 15;       // row group, column group
    const int ct = blockIdx.x % a.col_tiles, rt = blockIdx.x / a.col_tiles;
    const int64_t r0 = int64_t(rt) * QT, c0 = int64_t(ct) * QT;
    const int64_t row = r0 + g * 8, col = c0 + c * 8;

    float v[8][8];
    const bool whole = a.vec && col + 8 <= a.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (whole && row + i < a.rows) {
            load8<DT>(a.x, (row + i) * a.ld + col, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i][j] = row + i < a.rows && col + j < a.cols ? load1<DT>(a.x, (row + i) * a.ld + col + j) : 0.f;
        }
    }
    // magnitudes compare as integers, NaN above infinity above the rest
    uint32_t rm[8] = {}, cm[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = __float_as_uint(v[i][j]) & 0x7fffffffu;
            rm[i] = max(rm[i], m);
            cm[j] = max(cm[j], m);
        }
    const bool whole_block = (a.q && a.block == QT) || (a.qt && a.block_t == QT);
    const bool by_column = a.qt && a.block_t == 1;
    float ts = 0.f;  // the tile's scale
    if (whole_block) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) wmax[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, wmax[w][0]);
        ts = scale_of(m, a.inv_top);
        __syncthreads();
    }
    if (by_column) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = max(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
            if (lane < 16) wmax[warp][c * 8 + j] = m;
        }
        __syncthreads();
        if (tid < QT) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) m = max(m, wmax[w][tid]);
            cscale[tid] = scale_of(m, a.inv_top);
            if (c0 + tid < a.cols) a.scales_t[int64_t(rt) * a.cols + c0 + tid] = cscale[tid];
        }
        __syncthreads();
    }
    if (a.q) {
        if (a.block == QT && tid == 0) a.scales[int64_t(rt) * a.col_tiles + ct] = ts;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = ts;
            if (a.block == 1) {
                uint32_t m = rm[i];
#pragma unroll
                for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                s = scale_of(m, a.inv_top);
                if (c == 0 && row + i < a.rows) a.scales[int64_t(ct) * a.rows + row + i] = s;
            }
            const float inv = __frcp_rn(s);
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(v[i][j], inv);
            if (row + i < a.rows && col < a.cols)
                *reinterpret_cast<uint2*>(a.q + (row + i) * a.ldq + col) = code8(y, a.e5m2);
        }
    }
    if (a.qt) {
        if (a.block_t == QT && tid == 0) a.scales_t[int64_t(ct) * a.row_tiles + rt] = ts;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float inv = __frcp_rn(by_column ? cscale[c * 8 + j] : ts);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(v[i][j], inv);
            turned[c * 8 + j][g ^ c] = code8(y, a.e5m2);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int cc = k * 16 + g;  // a column of x: 16 threads write its 128 rows
            if (c0 + cc < a.cols && r0 + c * 8 < a.rows)
                *reinterpret_cast<uint2*>(a.qt + (c0 + cc) * a.ldqt + r0 + c * 8) = turned[cc][c ^ (cc >> 3)];
        }
    }
}

}  // namespace hl_fp8

extern "C" int headloss_fp8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int dtype,
                                     int type, void* q, int64_t ldq, float* scales, int block, void* qt,
                                     int64_t ldqt, float* scales_t, int block_t, void* stream) {
    using namespace hl_fp8;
    const int64_t most = (int64_t(1) << 31) - QT;
    if (rows < 0 || cols < 0 || rows >= most || cols >= most || ld < cols) return HEADLOSS_ERR_ARG;
    if (type != HEADLOSS_E4M3 && type != HEADLOSS_E5M2) return HEADLOSS_ERR_ARG;
    if (dtype != HEADLOSS_FP32 && dtype != HEADLOSS_BF16 && dtype != HEADLOSS_FP16) return HEADLOSS_ERR_DTYPE;
    if (!q && !qt) return HEADLOSS_ERR_ARG;
    if (q && (!scales || ldq < cols || (block != 1 && block != QT))) return HEADLOSS_ERR_ARG;
    if (qt && (!scales_t || ldqt < rows || (block_t != 1 && block_t != QT))) return HEADLOSS_ERR_ARG;
    auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    if ((q && ((bits(q) & 15) || (ldq & 15) || (bits(scales) & 3))) ||
        (qt && ((bits(qt) & 15) || (ldqt & 15) || (bits(scales_t) & 3))))
        return HEADLOSS_ERR_ALIGN;
    if (rows == 0 || cols == 0) return HEADLOSS_OK;
    if (!x) return HEADLOSS_ERR_ARG;
    const int size = dtype == HEADLOSS_FP32 ? 4 : 2;
    if (bits(x) & (size - 1)) return HEADLOSS_ERR_ALIGN;
    QuantArgs a = {};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.vec = !(bits(x) & 15) && (rows == 1 || !((ld * size) & 15));
    a.e5m2 = type == HEADLOSS_E5M2;
    a.inv_top = a.e5m2 ? float(1.0 / 57344.0) : float(1.0 / 448.0);
    a.q = static_cast<unsigned char*>(q);
    a.ldq = ldq;
    a.scales = scales;
    a.block = block;
    a.qt = static_cast<unsigned char*>(qt);
    a.ldqt = ldqt;
    a.scales_t = scales_t;
    a.block_t = block_t;
    a.col_tiles = int((cols + QT - 1) / QT);
    a.row_tiles = int((rows + QT - 1) / QT);
    const int64_t tiles = int64_t(a.col_tiles) * a.row_tiles;
    if (tiles > INT32_MAX) return HEADLOSS_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == HEADLOSS_FP32) quantize_kernel<HEADLOSS_FP32><<<unsigned(tiles), QTHREADS, 0, s>>>(a);
    else if (dtype == HEADLOSS_BF16) quantize_kernel<HEADLOSS_BF16><<<unsigned(tiles), QTHREADS, 0, s>>>(a);
    else quantize_kernel<HEADLOSS_FP16><<<unsigned(tiles), QTHREADS, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
}
