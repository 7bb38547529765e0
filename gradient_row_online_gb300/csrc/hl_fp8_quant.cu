// hl_fp8_quant.cu -- headloss_fp8_quantize (include/headloss_fp8.h): a matrix and / or its
// transpose in 8-bit floating point with a scale for each block of 128.
//
// One CTA a 128 x 128 tile, which holds whole blocks of every kind.  A thread has 8 rows x 8
// columns in registers, 16-bit inputs as they came. Magnitudes compare as integers or packed pairs,
// with a NaN above all. The row maxima join over the 16 lanes of a row by halving exchanges, which
// leave each lane one row's maximum: a lane computes one scale, not eight. The column maxima join
// over the 16 row groups through shared memory. Where both outputs have 128 x 128 blocks the codes are
// the same: they are made once and turned 8 x 8 by byte permutes. The transpose's codes leave through
// a 16 KB tile in shared memory whose 8-byte units are placed by XOR, so that both its writes and its
// reads touch every bank once and global stores are whole 128-byte rows.
// HBM bound: each input element is read once, each code written once. Measured, both outputs, bf16: 4096 x 128256 in
// blocks of 1 and 1 359 us, 5.9 TB/s; 128256 x 4096 in blocks of 128 and 128 308 us, 6.8 TB/s.
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
    int leads;   // the kernel launched next waits for this one itself
};

__device__ __forceinline__ float scale_of(uint32_t amax_bits, float inv_top) {
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return fmaxf(__fmul_rn(__uint_as_float(amax_bits), inv_top), LEAST);
}
template <int TYPE>
__device__ __forceinline__ uint32_t code2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, TYPE == HEADLOSS_E5M2 ? __NV_E5M2 : __NV_E4M3);
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
// The transpose of 4 x 4 bytes.
__device__ __forceinline__ void turn4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&t)[4]) {
    const uint32_t ab0 = prmt(a, b, 0x5140), ab1 = prmt(a, b, 0x7362);
    const uint32_t cd0 = prmt(c, d, 0x5140), cd1 = prmt(c, d, 0x7362);
    t[0] = prmt(ab0, cd0, 0x5410);
    t[1] = prmt(ab0, cd0, 0x7632);
    t[2] = prmt(ab1, cd1, 0x5410);
    t[3] = prmt(ab1, cd1, 0x7632);
}

// Eight rows x eight columns of a thread.
template <int DT>
struct Tile {
    uint32_t w[8][4];  // pairs of 16-bit values
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {  // of the magnitudes; the signs are lost
        uint32_t r;
        if (DT == HEADLOSS_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float2 pair(uint32_t u) {
        if (DT == HEADLOSS_BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
    __device__ __forceinline__ void load(int i, const void* x, int64_t at) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
        w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
    }
    __device__ __forceinline__ void load_some(int i, const void* x, int64_t at, int n) {
        const uint16_t* p = static_cast<const uint16_t*>(x) + at;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[i][k] = (2 * k < n ? uint32_t(p[2 * k]) : 0u) | (2 * k + 1 < n ? uint32_t(p[2 * k + 1]) << 16 : 0u);
    }
    __device__ __forceinline__ void values(int i, int k, float& lo, float& hi) const {
        const float2 f = pair(w[i][k]);
        lo = f.x;
        hi = f.y;
    }
    // the bits of the largest magnitude as fp32
    __device__ __forceinline__ uint32_t row_top(int i) const {
        const float2 f = pair(larger(larger(w[i][0], w[i][1]), larger(w[i][2], w[i][3])));
        return max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu);
    }
    __device__ __forceinline__ void col_tops(uint32_t (&m)[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t t = w[0][k];
#pragma unroll
            for (int i = 1; i < 8; ++i) t = larger(t, w[i][k]);
            const float2 f = pair(t);
            m[2 * k] = __float_as_uint(f.x) & 0x7fffffffu;
            m[2 * k + 1] = __float_as_uint(f.y) & 0x7fffffffu;
        }
    }
};
template <>
struct Tile<HEADLOSS_FP32> {
    float v[8][8];
    __device__ __forceinline__ void load(int i, const void* x, int64_t at) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
        const float4 a = __ldg(f), b = __ldg(f + 1);
        v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
        v[i][4] = b.x, v[i][5] = b.y, v[i][6] = b.z, v[i][7] = b.w;
    }
    __device__ __forceinline__ void load_some(int i, const void* x, int64_t at, int n) {
        const float* p = static_cast<const float*>(x) + at;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = j < n ? p[j] : 0.f;
    }
    __device__ __forceinline__ void values(int i, int k, float& lo, float& hi) const {
        lo = v[i][2 * k];
        hi = v[i][2 * k + 1];
    }
    __device__ __forceinline__ uint32_t row_top(int i) const {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void col_tops(uint32_t (&m)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m[j] = max(m[j], __float_as_uint(v[i][j]) & 0x7fffffffu);
        }
    }
};

template <int DT, int TYPE>
__global__ void __launch_bounds__(QTHREADS) quantize_kernel(const __grid_constant__ QuantArgs a) {
    __shared__ uint32_t wmax[8][QT];            // column maxima of each warp, or the warps' maxima
    __shared__ __align__(16) float cinv[QT];    // inverse scales of the columns
    __shared__ __align__(16) uint2 turned[QT][16];
    if (a.leads) asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = tid >> 4, c = tid & 15;       // row group, column group
    const int rt = int(blockIdx.x / unsigned(a.col_tiles)), ct = int(blockIdx.x) - rt * a.col_tiles;
    const int64_t r0 = int64_t(rt) * QT, c0 = int64_t(ct) * QT;
    const int64_t row = r0 + g * 8, col = c0 + c * 8;
    const int rows = int(max(int64_t(0), min(int64_t(8), a.rows - row))), cols = int(max(int64_t(0), min(int64_t(8), a.cols - col)));

    Tile<DT> t;
    const bool whole = a.vec && cols == 8;
    const int64_t at = row * a.ld + col;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (whole && i < rows) t.load(i, a.x, at + i * a.ld);
        else t.load_some(i, a.x, at + i * a.ld, i < rows ? cols : 0);
    }
    const bool same = a.q && a.qt && a.block == QT && a.block_t == QT;  // one set of codes
    const bool by_row = a.q && a.block == 1, by_column = a.qt && a.block_t == 1;
    float ts = 0.f, tinv = 0.f;  // the tile's scale
    if ((a.q && !by_row) || (a.qt && !by_column)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, t.row_top(i));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) wmax[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, wmax[w][0]);
        ts = scale_of(m, a.inv_top);
        tinv = __frcp_rn(ts);
        if (tid == 0 && a.q && !by_row) a.scales[int64_t(rt) * a.col_tiles + ct] = ts;
        if (tid == 0 && a.qt && !by_column) a.scales_t[int64_t(ct) * a.row_tiles + rt] = ts;
        if (by_column) __syncthreads();
    }
    if (by_column) {
        uint32_t cm[8];
        t.col_tops(cm);
#pragma unroll
        for (int j = 0; j < 8; ++j) cm[j] = max(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
        if (lane < 16) {
            *reinterpret_cast<uint4*>(&wmax[warp][c * 8]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
            *reinterpret_cast<uint4*>(&wmax[warp][c * 8 + 4]) = make_uint4(cm[4], cm[5], cm[6], cm[7]);
        }
        __syncthreads();
        if (tid < QT) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) m = max(m, wmax[w][tid]);
            const float s = scale_of(m, a.inv_top);
            cinv[tid] = __frcp_rn(s);
            if (c0 + tid < a.cols) a.scales_t[int64_t(rt) * a.cols + c0 + tid] = s;
        }
        __syncthreads();
    }
    if (a.q) {
        float mine = tinv;  // by rows: the inverse scale of row 4 (c & 8) + 2 (c & 4) + (c & 2) of the eight
        if (by_row) {
            uint32_t m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = t.row_top(i);
#pragma unroll
            for (int n = 4, o = 8; n; n >>= 1, o >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const bool high = c & o;
                    const uint32_t give = high ? m[i] : m[i + n], keep = high ? m[i + n] : m[i];
                    m[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, o));
                }
            m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
            const float s = scale_of(m[0], a.inv_top);
            const int i = (c & 8) / 2 + (c & 4) / 2 + (c & 2) / 2;
            if (!(c & 1) && i < rows) a.scales[int64_t(ct) * a.rows + row + i] = s;
            mine = __frcp_rn(s);
        }
        uint2 codes[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float inv = by_row ? __shfl_sync(0xffffffffu, mine, (lane & 16) | (i & 4) * 2 | (i & 2) * 2 | (i & 1) * 2) : tinv;
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                t.values(i, k, lo, hi);
                h[k] = code2<TYPE>(__fmul_rn(lo, inv), __fmul_rn(hi, inv));
            }
            codes[i] = make_uint2(prmt(h[0], h[1], 0x5410), prmt(h[2], h[3], 0x5410));
            if (i < rows && cols > 0) *reinterpret_cast<uint2*>(a.q + (row + i) * a.ldq + col) = codes[i];
        }
        if (same) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t lo[4], hi[4];
                turn4(h ? codes[0].y : codes[0].x, h ? codes[1].y : codes[1].x, h ? codes[2].y : codes[2].x,
                      h ? codes[3].y : codes[3].x, lo);
                turn4(h ? codes[4].y : codes[4].x, h ? codes[5].y : codes[5].x, h ? codes[6].y : codes[6].x,
                      h ? codes[7].y : codes[7].x, hi);
#pragma unroll
                for (int j = 0; j < 4; ++j) turned[c * 8 + 4 * h + j][g ^ c] = make_uint2(lo[j], hi[j]);
            }
        }
    }
    if (a.qt) {
        if (!same) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 inv = by_column ? *reinterpret_cast<const float2*>(&cinv[c * 8 + 2 * k]) : make_float2(tinv, tinv);
                uint32_t h0[4], h1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a0, a1, b0, b1;
                    t.values(2 * i, k, a0, a1);
                    t.values(2 * i + 1, k, b0, b1);
                    h0[i] = code2<TYPE>(__fmul_rn(a0, inv.x), __fmul_rn(b0, inv.x));
                    h1[i] = code2<TYPE>(__fmul_rn(a1, inv.y), __fmul_rn(b1, inv.y));
                }
                turned[c * 8 + 2 * k][g ^ c] = make_uint2(prmt(h0[0], h0[1], 0x5410), prmt(h0[2], h0[3], 0x5410));
                turned[c * 8 + 2 * k + 1][g ^ c] = make_uint2(prmt(h1[0], h1[1], 0x5410), prmt(h1[2], h1[3], 0x5410));
            }
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

template <int DT>
void launch_quantize(const QuantArgs& a, int type, unsigned tiles, cudaStream_t s) {
    if (type == HEADLOSS_E4M3) quantize_kernel<DT, HEADLOSS_E4M3><<<tiles, QTHREADS, 0, s>>>(a);
    else quantize_kernel<DT, HEADLOSS_E5M2><<<tiles, QTHREADS, 0, s>>>(a);
}

int quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int dtype, int type, void* q, int64_t ldq,
             float* scales, int block, void* qt, int64_t ldqt, float* scales_t, int block_t, bool leads,
             cudaStream_t s) {
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
    a.inv_top = type == HEADLOSS_E5M2 ? float(1.0 / 57344.0) : float(1.0 / 448.0);
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
    a.leads = leads;
    if (dtype == HEADLOSS_FP32) launch_quantize<HEADLOSS_FP32>(a, type, unsigned(tiles), s);
    else if (dtype == HEADLOSS_BF16) launch_quantize<HEADLOSS_BF16>(a, type, unsigned(tiles), s);
    else launch_quantize<HEADLOSS_FP16>(a, type, unsigned(tiles), s);
    return cudaGetLastError() == cudaSuccess ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
}

}  // namespace hl_fp8

extern "C" int headloss_fp8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int dtype,
                                     int type, void* q, int64_t ldq, float* scales, int block, void* qt,
                                     int64_t ldqt, float* scales_t, int block_t, void* stream) {
    return hl_fp8::quantize(x, rows, cols, ld, dtype, type, q, ldq, scales, block, qt, ldqt, scales_t, block_t,
                            false, static_cast<cudaStream_t>(stream));
}
