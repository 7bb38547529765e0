// hl_fp8_gemm.cu -- headloss_fp8_matmul (include/headloss_fp8.h): out = a . b^T of 8-bit
// matrices, a's scales for each row and 128 columns, b's for each 128 x 128.
//
// The tensor cores sum a K block of 128 (four tcgen05.mma kind::f8f6f4, K = 32 each) into one of
// two TMEM accumulators; the epilogue warps read it back and add it, times its scales, to fp32
// sums in registers while the next block's MMAs fill the other accumulator.  So each block's
// scale is applied exactly once, in fp32, and a sum over K never lives in the accumulator for more
// than 128 products.
//
// One CTA an SM walks the 128 x 256 tiles of out. Few rows of a take the same way: a's tile is then
// 64 rows of copies, the MMAs' other rows are whatever follows and their sums never read, and b, 256 rows
// at a time, streams through at HBM's rate. (b as the MMA's 128 rows and a as its 16 to 64 columns is
// slower: such an MMA takes the time of 128 columns and more, and moves half the bytes of b: 48 x 128256 took 115
// us.) The tiles of the last round, which are fewer than SMs, have their K split where that takes less time; the
// parts go to the workspace in fp32 and a second kernel adds them in order.
//
// What bounds it, at many rows: shared memory moves 96 KB a block of K (48 written by the copies, 48 read by the
// MMAs), 768 cycles at 128 bytes a cycle, and reading the accumulator back takes another 256 of TMEM's: 1024 one after
// the other, of which the MMAs' own 512 are half. Measured some 1000 cycles, 2.3 PFLOP/s (8192 x 32000 x 4096 0.90 to 0.94 ms); with K
// summed in TMEM throughout, which the scales do not allow, 0.74 ms. Tiles of 256 x 256 on pairs of CTAs
// (cta_group::2) move 64 KB a block, but with two accumulators the way over to the other CTA and back is not
// hidden (840 cycles from an accumulator's release to the next MMAs on it): 1.30 ms.
// Every wait is bounded; one that gives up sets bit 0 of *err, and the kernel drains what it issued.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "headloss.h"
#include "headloss_fp8.h"
#include "hl_tc.cuh"

namespace hl_fp8 {

using namespace hl_tc;

constexpr int BK = 128;              // one scale block, one swizzle row of bytes
constexpr uint32_t IDESC_FIXED = 1u << 4;  // D is fp32; A and B K-major

__host__ __device__ constexpr uint32_t idesc_of(int m, int n, int a_type, int b_type) {
    return IDESC_FIXED | uint32_t(a_type) << 7 | uint32_t(b_type) << 10 | uint32_t(n >> 3) << 17 |
           uint32_t(m >> 4) << 24;
}

template <int OT>
__device__ __forceinline__ uint32_t round2(float a, float b) {  // two 16-bit outputs
    if (OT == HEADLOSS_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <int OT>
__device__ __forceinline__ void store1(void* out, int64_t i, float v) {
    if (OT == HEADLOSS_FP32) static_cast<float*>(out)[i] = v;
    else if (OT == HEADLOSS_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

// ------------------------------------------------------------------ wide ----

constexpr int WM = 128, WN = 256;
constexpr int WB_BYTES = WN * BK;                           // 32 KB
constexpr int W_EPI_WARPS = 8;                              // 2 for each TMEM lane quadrant
constexpr int W_THREADS = 128 + 32 * W_EPI_WARPS;
// Launched with 168 registers a thread (64512 a CTA); the warpgroup of the copies and MMAs
// gives up its share to the two that hold the sums: 128 * 40 + 256 * 224 = 62464.
constexpr int W_LAUNCH_REGS = 168, W_FEW_REGS = 40, W_SUM_REGS = 224;
static_assert(128 * W_FEW_REGS + 32 * W_EPI_WARPS * W_SUM_REGS <= W_THREADS * W_LAUNCH_REGS, "registers");
constexpr int W_OUT_BYTES = 32 * 128;                       // 32 rows x 128 bytes of one warp
// By the rows of a's copies. Up to 64 rows leave shared memory for five stages, that is for 160 KB of b in flight,
// and fewer warps have rows to write out (16 x 128256: 119 us with copies of 128 rows, 92 with 64, 94 with 32).
template <int A_ROWS>
struct Wide {
    static constexpr int STAGES = A_ROWS == 64 ? 5 : 4;
    static constexpr int A_BYTES = A_ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + WB_BYTES;
    static constexpr int OUT_OFF = STAGES * STAGE_BYTES;
    static constexpr int OUT_WARPS = 2 * A_ROWS / 32;
    static constexpr int BAR_OFF = OUT_OFF + OUT_WARPS * W_OUT_BYTES;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
    static_assert(SMEM <= 232448 && STAGE_BYTES >= WM * BK, "shared memory; the MMAs read 128 rows from a's first");
};
constexpr int GN = 16;                                      // column tiles a group of the tile order

struct WideArgs {
    const float* a_scales;  // [KB][M]
    const float* b_scales;  // [NB][KB]
    int64_t M, N;
    int KB, NB, MT, NT;
    uint32_t whole;         // tiles that one CTA sums over all of K; the others, fewer than SMs,
    int splits;             // in as many parts of K
    float* parts;           // [part][column half][32 rows][128 columns][row]
    void* out;
    int64_t ldo;
    int early;              // b was in place before the launch in front of this one began
    int tma_out;            // rows of out start on 16-byte boundaries
    int n_even;             // and end on them
    uint32_t idesc;
    int* err;
};

// Position i of the tile order: GN column tiles at a time, every row tile within a group.
__device__ __forceinline__ void tile_at(uint32_t i, uint32_t MT, uint32_t NT, int& m, int& n) {
    const uint32_t per = MT * GN, g = i / per;
    const uint32_t w = i - g * per, wide = min(NT - g * GN, uint32_t(GN));
    m = int(w / wide);
    n = int(g * GN + w % wide);
}

// Piece i of the work: a tile, blocks k0 .. k1 - 1 of K, and the part that it is (-1: the whole sum).
struct Piece {
    uint32_t tile;
    int k0, k1, part;
};
__device__ __forceinline__ Piece piece_at(const WideArgs& p, uint32_t i) {
    if (i < p.whole) return {i, 0, p.KB, -1};
    const uint32_t j = i - p.whole, t = j / uint32_t(p.splits), sp = j - t * uint32_t(p.splits);
    return {p.whole + t, int(uint64_t(p.KB) * sp / uint32_t(p.splits)), int(uint64_t(p.KB) * (sp + 1) / uint32_t(p.splits)),
            p.splits > 1 ? int(j) : -1};
}
__device__ __forceinline__ uint32_t pieces(const WideArgs& p) {
    return p.whole + (uint32_t(p.MT) * p.NT - p.whole) * uint32_t(p.splits);
}

// 32 staged rows (128 bytes each, 128-byte swizzle) to rows of out that start anywhere: the first `cols` elements.
// What costs is the sectors that a store instruction writes in part. So fp32 rows go an element a lane, 128
// bytes in a row (4096 x 100001 x 512: 675 us, the other way 114 more; 410 where rows start on 16 bytes and TMA stores
// them), and 16-bit rows, eight lanes each, in 16-byte units of out, each put together from two of the staged ones, with
// the elements before and behind them (508 us, an element a lane 112 more; 284 on 16 bytes).
template <int OT>
__device__ __forceinline__ void store_rows(const unsigned char* stage, const WideArgs& p, int64_t r0, int64_t c0, int cols,
                                           int lane) {
    constexpr int SIZE = OT == HEADLOSS_FP32 ? 4 : 2, PER = 16 / SIZE;
    if (cols <= 0) return;
    if (OT == HEADLOSS_FP32) {
        for (int r = 0; r < 32 && r0 + r < p.M; ++r)
            if (lane < cols)
                static_cast<float*>(p.out)[(r0 + r) * p.ldo + c0 + lane] =
                    *reinterpret_cast<const float*>(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
        return;
    }
    const int j = lane & 7;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3);
        if (r0 + r >= p.M) break;
        char* out = static_cast<char*>(p.out) + ((r0 + r) * p.ldo + c0) * SIZE;
        const unsigned char* row = stage + r * 128;
        const int ahead = int(-reinterpret_cast<uintptr_t>(out) & 15);  // bytes before the first whole unit
        const int o = ahead + 16 * j, u = o >> 4, shift = o & 15;
        if (o + 16 <= cols * SIZE) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + ((u ^ (r & 7)) << 4));
            const uint4 y = *reinterpret_cast<const uint4*>(row + (((u + (shift != 0)) ^ (r & 7)) << 4));
            uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 6; ++k) w[k] = shift & 8 ? w[k + 2] : w[k];
#pragma unroll
            for (int k = 0; k < 5; ++k) w[k] = shift & 4 ? w[k + 1] : w[k];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], (shift & 3) * 8);
            *reinterpret_cast<uint4*>(out + o) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const int head = ahead / SIZE, tail = head + (cols > head ? (cols - head) / PER * PER : 0);
        auto element = [&](int e) {
            const int byte = e * SIZE;
            *reinterpret_cast<uint16_t*>(out + byte) =
                *reinterpret_cast<const uint16_t*>(row + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15));
        };
        if (j < head && j < cols) element(j);
        if (tail + j < cols) element(tail + j);
    }
}

#ifdef HL_FAULT_INJECT  // test builds alone: the first CTA leaves out a's copy of this block
static __device__ int injected_drop = -1;
#endif

template <int OT, int A_ROWS>
__global__ void __launch_bounds__(W_THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_o, const WideArgs p) {
    using L = Wide<A_ROWS>;
    constexpr int STAGES = L::STAGES;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // full: a stage has its tiles, and the accumulator its block goes to was read (an arrival a warp);
    // empty: the block's MMAs are done, so its stage is free and its sums can be read. One wait and one
    // commit a block: each costs the issuing warp some hundred cycles of the block's 768.
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* empty = full + STAGES;
    uint64_t* mma_done = empty + STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t items = pieces(p);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(su32(&full[s]), 1 + W_EPI_WARPS);
            mbar_init(su32(&empty[s]), 1);
        }
        mbar_init(su32(mma_done), 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(su32(tmem_slot), 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp != 2) grid_wait();

    if (warp < 4) {
        give_registers<W_FEW_REGS>();
        if (warp == 0) {  // copies
            const Piece w0 = piece_at(p, blockIdx.x);
            const uint32_t ahead = p.early ? uint32_t(min(w0.k1 - w0.k0, STAGES)) : 0;
            uint32_t it = 0;
            bool go = true;
            for (uint32_t i = blockIdx.x; go && i < items; i += gridDim.x) {
                const Piece w = piece_at(p, i);
                int m, n;
                tile_at(w.tile, p.MT, p.NT, m, n);
                for (int kb = w.k0; kb < w.k1; ++kb, ++it) {
                    const int s = int(it % STAGES);
                    const uint32_t a = su32(smem + s * L::STAGE_BYTES), bar = su32(&full[s]);
                    if (it >= ahead) {
                        if (!warp_wait(su32(&empty[s]), ((it / STAGES) & 1u) ^ 1u, abort, p.err)) {
                            go = false;
                            break;
                        }
                        warp_expect_tx(bar, L::STAGE_BYTES);
                        warp_tma_load_2d(a + L::A_BYTES, &map_b, kb * BK, n * WN, bar);
                    }
#ifdef HL_FAULT_INJECT
                    if (blockIdx.x == 0 && int(it) == injected_drop) continue;
#endif
                    warp_tma_load_2d(a, &map_a, kb * BK, m * WM, bar);
                }
            }
            for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; ++j)  // what was issued has landed
                drain_phase(su32(&full[j % STAGES]), (j / STAGES) & 1u, p.err);
        } else if (warp == 1) {  // MMAs
            uint32_t it = 0;
            bool go = true;
            for (uint32_t i = blockIdx.x; go && i < items; i += gridDim.x) {
                const Piece w = piece_at(p, i);
                for (int kb = w.k0; kb < w.k1; ++kb, ++it) {
                    const int s = int(it % STAGES);
                    const uint32_t acc = it & 1u;
                    const uint32_t a = su32(smem + s * L::STAGE_BYTES);
                    const uint64_t da = smem_desc(a), db = smem_desc(a + L::A_BYTES);
                    if (!warp_wait(su32(&full[s]), (it / STAGES) & 1u, abort, p.err)) {
                        go = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)  // 32 bytes of K each: two units of the descriptor's address
                        warp_mma_f8(tmem + acc * WN, da + 2 * k, db + 2 * k, p.idesc, k != 0);
                    warp_mma_commit(su32(&empty[s]));
                }
            }
            if (it) {  // what was issued is done before TMEM is freed
                warp_mma_commit(su32(mma_done));
                drain_phase(su32(mma_done), 0u, p.err);
            }
        }
        else if (warp == 2 && p.early) {  // the first stages' rows of b, before a's quantisation is done
            const Piece w = piece_at(p, blockIdx.x);
            int m, n;
            tile_at(w.tile, p.MT, p.NT, m, n);
            const uint32_t ahead = uint32_t(min(w.k1 - w.k0, STAGES));
            for (uint32_t s = 0; s < ahead; ++s) {
                warp_expect_tx(su32(&full[s]), L::STAGE_BYTES);
                warp_tma_load_2d(su32(smem + s * L::STAGE_BYTES) + L::A_BYTES, &map_b, (w.k0 + int(s)) * BK, n * WN, su32(&full[s]));
            }
            grid_wait();
        }
        __syncwarp();
    } else {  // scaled sums: warp w has TMEM lanes 32 (w % 4) .., columns 128 h ..
        take_registers<W_SUM_REGS>();
        const int q = warp & 3, h = (warp - 4) >> 2;
        // (a warp without rows has no place to stage them, and writes none)
        unsigned char* stage = smem + L::OUT_OFF + (h * (A_ROWS / 32) + q) * W_OUT_BYTES;
        uint32_t it = 0;
        bool go = true;
        if (lane == 0) {  // both accumulators are free
            mbar_arrive(su32(&full[0]));
            mbar_arrive(su32(&full[1]));
        }
        for (uint32_t i = blockIdx.x; go && i < items; i += gridDim.x) {
            const Piece w = piece_at(p, i);
            const int k0 = w.k0, k1 = w.k1;
            int m, n;
            tile_at(w.tile, p.MT, p.NT, m, n);
            const int64_t row = int64_t(m) * WM + 32 * q + lane;
            const int nb = min(2 * n + h, p.NB - 1);
            const bool in = row < p.M;
            if (int64_t(m) * WM + 32 * q >= p.M) {  // this warp has no rows of out
                for (int kb = k0; go && kb < k1; ++kb, ++it) {
                    go = warp_wait(su32(&empty[it % STAGES]), (it / STAGES) & 1u, abort, p.err);
                    if (go && lane == 0) mbar_arrive(su32(&full[(it + 2) % STAGES]));
                }
                continue;
            }
            const float* sa = p.a_scales + (in ? row : 0);
            const float* sb = p.b_scales + int64_t(nb) * p.KB;
            float sum[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) sum[j] = 0.f;
            // scales four blocks ahead: a load takes about as long as a block
            float fa[4], fb[4];
            auto fetch = [&](int kb, float& x, float& y) {
                x = in && kb < k1 ? __ldg(sa + int64_t(kb) * p.M) : 0.f;
                y = kb < k1 ? __ldg(sb + kb) : 0.f;
            };
#pragma unroll
            for (int j = 0; j < 4; ++j) fetch(k0 + j, fa[j], fb[j]);
            for (int kb = k0; kb < k1; ++kb, ++it) {
                const float s = fa[0] * fb[0];
#pragma unroll
                for (int j = 0; j < 3; ++j) fa[j] = fa[j + 1], fb[j] = fb[j + 1];
                fetch(kb + 4, fa[3], fb[3]);
                const int acc = int(it & 1u);
                // Lanes may answer differently where the limit runs out as the phase completes. They go on together
                // all the same, and ask one another where they meet: a vote here delays every block (8192 x
                // 32000 x 4096 in 987 us, and 900).
                const bool there = wait_phase(su32(&empty[it % STAGES]), (it / STAGES) & 1u, abort, p.err);
                __syncwarp();
                tc_fence_after();
                const uint32_t t = tmem + (uint32_t(32 * q) << 16) + uint32_t(acc * WN + 128 * h);
                // the next 32 columns are on their way while these are added
                uint32_t v[2][32];
                tmem_ld32(t, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_wait32(v[c & 1]);
                    if (c < 3) {
                        tmem_ld32(t + 32 * (c + 1), v[(c + 1) & 1]);
                    } else {  // all is read: the accumulator is free for the block after the next
                        tc_fence_before();
                        go = __all_sync(0xffffffffu, there);
                        if (go && lane == 0) mbar_arrive(su32(&full[(it + 2) % STAGES]));
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[32 * c + j] = fmaf(__uint_as_float(v[c & 1][j]), s, sum[32 * c + j]);
                }
                if (!go) break;
            }
            if (!go) break;
            if (w.part >= 0) {
                float* to = p.parts + ((int64_t(w.part) * 2 + h) * 4 + q) * 4096 + lane;
#pragma unroll
                for (int j = 0; j < 128; ++j) to[j * 32] = sum[j];
                continue;
            }
            // 128 bytes of 32 rows at a time through shared memory (128-byte swizzle)
            constexpr int COLS = OT == HEADLOSS_FP32 ? 32 : 64;
            const int64_t r0 = int64_t(m) * WM + 32 * q, n0 = int64_t(n) * WN + 128 * h;
#pragma unroll
            for (int g = 0; g < 128 / COLS; ++g) {
                if (lane == 0) bulk_wait_read0();
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint4 u;
                    if (OT == HEADLOSS_FP32) {
                        const float* f = sum + 32 * g + 4 * c;
                        u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                       __float_as_uint(f[3]));
                    } else {
                        const float* f = sum + 64 * g + 8 * c;
                        u = make_uint4(round2<OT>(f[0], f[1]), round2<OT>(f[2], f[3]), round2<OT>(f[4], f[5]),
                                       round2<OT>(f[6], f[7]));
                    }
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) * 16)) = u;
                }
                const int64_t c0 = n0 + g * COLS;
                // a store that TMA clips at N would still write whole 16-byte units
                if (p.tma_out && (p.n_even || c0 + COLS <= p.N)) {
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && r0 < p.M && c0 < p.N) {
                        tma_store_2d(&map_o, int(c0), int(r0), su32(stage));
                        bulk_commit();
                    }
                } else {
                    __syncwarp();
                    store_rows<OT>(stage, p, r0, c0, int(min(int64_t(COLS), p.N - c0)), lane);
                    __syncwarp();
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of the tiles whose K was split, added in their order: a CTA 32 rows x 32 columns.
template <int OT>
__global__ void __launch_bounds__(256) join_kernel(const WideArgs p) {
    __shared__ float sums[32][33];
    const int piece = blockIdx.x & 31, q = piece & 3, h = piece >> 2 & 1, j0 = (piece >> 3) * 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t t = blockIdx.x >> 5;
    int m, n;
    tile_at(p.whole + t, p.MT, p.NT, m, n);
    const int64_t r0 = int64_t(m) * WM + 32 * q, c0 = int64_t(n) * WN + 128 * h + j0;
    if (r0 >= p.M || c0 >= p.N) return;
    const float* from = p.parts + ((int64_t(t) * p.splits * 2 + h) * 4 + q) * 4096 + (j0 + warp * 4) * 32 + lane;
    float x[4] = {};
#pragma unroll 8
    for (int sp = 0; sp < p.splits; ++sp)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += from[int64_t(sp) * 8 * 4096 + j * 32];
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[lane][warp * 4 + j] = x[j];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t row = r0 + warp * 4 + r;
        if (row < p.M && c0 + lane < p.N) store1<OT>(p.out, row * p.ldo + c0 + lane, sums[warp * 4 + r][lane]);
    }
}

// ------------------------------------------------------------------ host ----

int quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, int dtype, int type, void* q, int64_t ldq,
             float* scales, int block, void* qt, int64_t ldqt, float* scales_t, int block_t, bool leads,
             cudaStream_t s);  // hl_fp8_quant.cu

// a quantised x of M x K within a workspace: its codes, its scales
int64_t codes_bytes(int64_t M, int64_t K) { return M * ((K + 15) / 16 * 16); }
int64_t scales_bytes(int64_t M, int64_t K) { return (M * ((K + 127) / 128) * 4 + 15) / 16 * 16; }

int make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t rows, int64_t cols,
             int64_t pitch_bytes, int box_rows, int box_cols) {
    auto fn = encode_tiled();
    if (!fn) return 1;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(pitch_bytes)};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS;
}

struct Plan {
    int64_t whole;
    int splits;
    int64_t bytes;
};

// The tiles go over the SMs in rounds; those of the last, incomplete round have their K in as many parts as take
// the least time: a block of K counts 0.58 us (0.53 measured in full rounds), with few rows what its 32 KB of b take (0.4 us alone, HBM's rate
// together), and for parts a second launch (4 us) and their sums written and read (5 bytes a picosecond). Measured,
// whole and in parts: 4096 x 4096 x 128256 2020 and 1830 us, 512 x 4096 x 128256 502 and 287, 1 x 4096 x 32000 117
// and 35, 200 x 1000 x 5003 29 and 15.
Plan plan_of(int64_t M, int64_t N, int64_t K, int sms) {
    const int64_t KB = (K + BK - 1) / BK, tiles = ((M + WM - 1) / WM) * ((N + WN - 1) / WN), rest = tiles % sms;
    Plan r = {tiles - rest, 1, 0};
    double least = 0;
    for (int64_t s = 1; rest && s <= 16 && (s == 1 || s <= KB / 4); ++s) {
        const int64_t at_once = rest * s < sms ? rest * s : sms, rounds = (rest * s + sms - 1) / sms;
        const double together = double(at_once) * WN * BK / 6.5e6;
        const double block = M > 64 ? 0.58 : together > 0.4 ? together : 0.4;
        const double t = block * double(rounds) * double((KB + s - 1) / s) +
                         (s > 1 ? 4.0 + double(rest * s * (M < WM ? M : WM) * WN) * 8 / 5e6 : 0.0);
        if (s == 1 || t < least) {
            least = t;
            r.splits = int(s);
        }
    }
    if (r.splits > 1) r.bytes = rest * r.splits * int64_t(WM) * WN * 4;
    else r.whole = tiles;
    return r;
}

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    const int64_t most = (int64_t(1) << 31) - 256;
    if (M < 0 || N < 0 || K < 1 || M >= most || N >= most || K >= most) return false;
    return ((M + WM - 1) / WM) * ((N + WN - 1) / WN) <= INT32_MAX;
}

int sm_count(int* sms) {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess &&
           cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

template <int OT, int A_ROWS>
int launch_rows(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo, const WideArgs& a, int sms,
                cudaStream_t s) {
    const auto fn = wide_kernel<OT, A_ROWS>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide<A_ROWS>::SMEM) != cudaSuccess)
        return HEADLOSS_ERR_CUDA;
    const int64_t rest = int64_t(a.MT) * a.NT - a.whole, items = a.whole + rest * a.splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(items < sms ? items : sms));
    cfg.blockDim = dim3(W_THREADS);
    cfg.dynamicSmemBytes = Wide<A_ROWS>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.early ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, fn, ma, mb, mo, a) != cudaSuccess) return HEADLOSS_ERR_CUDA;
    if (a.splits > 1) {
        join_kernel<OT><<<unsigned(rest * 32), 256, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return HEADLOSS_ERR_CUDA;
    }
    return HEADLOSS_OK;
}
int rows_of_copies(int64_t M) { return M <= 64 ? 64 : WM; }
template <int OT>
int launch_wide(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo, const WideArgs& a, int sms,
                cudaStream_t s) {
    return rows_of_copies(a.M) == 64 ? launch_rows<OT, 64>(ma, mb, mo, a, sms, s)
                                     : launch_rows<OT, WM>(ma, mb, mo, a, sms, s);
}

}  // namespace hl_fp8

#ifdef HL_FAULT_INJECT
// Test builds alone: the products that follow lose a copy of block `drop` (-1: none), and their waits
// give up after `wait_ns` (0: the usual limit).
extern "C" int headloss_fp8_test_inject(int drop, unsigned long long wait_ns) {
    if (!wait_ns) wait_ns = hl_tc::WAIT_NS;
    return cudaMemcpyToSymbol(hl_fp8::injected_drop, &drop, sizeof drop) != cudaSuccess ||
           cudaMemcpyToSymbol(hl_tc::injected_wait_ns, &wait_ns, sizeof wait_ns) != cudaSuccess;
}
#endif

extern "C" int64_t headloss_fp8_workspace(int64_t M, int64_t N, int64_t K) {
    using namespace hl_fp8;
    int sms = 0;
    if (!sizes_ok(M, N, K) || !sm_count(&sms)) return -1;
    return M && N ? plan_of(M, N, K, sms).bytes : 0;
}

namespace hl_fp8 {

// The product; early: the kernel in front of it in the stream is a's quantisation, which leads.
int matmul(const void* a, int64_t lda, const float* a_scales, int a_type, const void* b, int64_t ldb,
           const float* b_scales, int b_type, int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
           int out_dtype, void* workspace, int64_t workspace_bytes, int* err, bool early, bool check_only,
           cudaStream_t s) {
    if (!sizes_ok(M, N, K) || lda < K || ldb < K || ldo < N) return HEADLOSS_ERR_ARG;
    auto known = [](int t) { return t == HEADLOSS_E4M3 || t == HEADLOSS_E5M2; };
    if (!known(a_type) || !known(b_type)) return HEADLOSS_ERR_ARG;
    if (out_dtype != HEADLOSS_FP32 && out_dtype != HEADLOSS_BF16 && out_dtype != HEADLOSS_FP16)
        return HEADLOSS_ERR_DTYPE;
    if (M == 0 || N == 0) return HEADLOSS_OK;
    if (!a || !b || !a_scales || !b_scales || !out || !err) return HEADLOSS_ERR_ARG;
    const int size = out_dtype == HEADLOSS_FP32 ? 4 : 2;
    auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    if (((bits(a) | bits(b) | bits(workspace)) & 15) || ((lda | ldb) & 15) ||
        ((bits(a_scales) | bits(b_scales) | bits(err)) & 3) || (bits(out) & (size - 1)))
        return HEADLOSS_ERR_ALIGN;
    int sms = 0;
    if (!sm_count(&sms)) return HEADLOSS_ERR_CUDA;
    const Plan plan = plan_of(M, N, K, sms);
    if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes)) return HEADLOSS_ERR_ARG;
    if (check_only) return HEADLOSS_OK;
    const int KB = int((K + BK - 1) / BK);
    CUtensorMap ma, mb, mo;
    const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    WideArgs w = {};
    w.a_scales = a_scales;
    w.b_scales = b_scales;
    w.M = M;
    w.N = N;
    w.KB = KB;
    w.NB = int((N + 127) / 128);
    w.MT = int((M + WM - 1) / WM);
    w.NT = int((N + WN - 1) / WN);
    w.whole = uint32_t(plan.whole);
    w.splits = plan.splits;
    w.parts = static_cast<float*>(workspace);
    w.out = out;
    w.ldo = ldo;
    w.tma_out = !(bits(out) & 15) && !((ldo * size) & 15);
    w.n_even = !((N * size) & 15);
    w.early = early;
    w.idesc = idesc_of(WM, WN, a_type, b_type);
    w.err = err;
    if (make_map(&ma, U8, a, M, K, lda, rows_of_copies(M), BK) || make_map(&mb, U8, b, N, K, ldb, WN, BK))
        return HEADLOSS_ERR_CUDA;
    if (w.tma_out) {
        const auto type = out_dtype == HEADLOSS_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                          : out_dtype == HEADLOSS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if (make_map(&mo, type, out, M, N, ldo * size, 32, 128 / size)) return HEADLOSS_ERR_CUDA;
    } else {
        mo = ma;  // not used
    }
    return out_dtype == HEADLOSS_FP32   ? launch_wide<HEADLOSS_FP32>(ma, mb, mo, w, sms, s)
           : out_dtype == HEADLOSS_BF16 ? launch_wide<HEADLOSS_BF16>(ma, mb, mo, w, sms, s)
                                        : launch_wide<HEADLOSS_FP16>(ma, mb, mo, w, sms, s);
}

}  // namespace hl_fp8

extern "C" int headloss_fp8_matmul(const void* a, int64_t lda, const float* a_scales, int a_type,
                                   const void* b, int64_t ldb, const float* b_scales, int b_type, int64_t M,
                                   int64_t N, int64_t K, void* out, int64_t ldo, int out_dtype,
                                   void* workspace, int64_t workspace_bytes, int* err, void* stream) {
    return hl_fp8::matmul(a, lda, a_scales, a_type, b, ldb, b_scales, b_type, M, N, K, out, ldo, out_dtype,
                          workspace, workspace_bytes, err, false, false, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t headloss_fp8_linear_workspace(int64_t M, int64_t N, int64_t K) {
    const int64_t need = headloss_fp8_workspace(M, N, K);
    return need < 0 ? -1 : hl_fp8::codes_bytes(M, K) + hl_fp8::scales_bytes(M, K) + need;
}

extern "C" int headloss_fp8_linear(const void* x, int64_t ldx, int dtype, const void* b, int64_t ldb,
                                   const float* b_scales, int b_type, int64_t M, int64_t N, int64_t K,
                                   void* out, int64_t ldo, int out_dtype, void* workspace,
                                   int64_t workspace_bytes, int* err, void* stream) {
    using namespace hl_fp8;
    if (!sizes_ok(M, N, K)) return HEADLOSS_ERR_ARG;
    const int64_t pitch = (K + 15) / 16 * 16, codes = codes_bytes(M, K), scales = scales_bytes(M, K);
    char* at = static_cast<char*>(workspace);
    if (M && N && (!at || workspace_bytes < codes + scales)) return HEADLOSS_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto product = [&](bool check_only) {
        return matmul(at, pitch, reinterpret_cast<float*>(at + codes), HEADLOSS_E4M3, b, ldb, b_scales, b_type, M, N,
                      K, out, ldo, out_dtype, at + codes + scales, workspace_bytes - codes - scales, err, true,
                      check_only, s);
    };
    int rc = product(true);
    if (rc != HEADLOSS_OK || M == 0 || N == 0) return rc;
    rc = quantize(x, M, K, ldx, dtype, HEADLOSS_E4M3, at, pitch, reinterpret_cast<float*>(at + codes), 1, nullptr, 0,
                  nullptr, 0, true, s);
    return rc == HEADLOSS_OK ? product(false) : rc;
}
