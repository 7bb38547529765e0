// hl_clip.cu -- the global gradient norm over many tensors, and clipping
// (headloss_clip_grads in include/headloss_clip.h).
//
// One cooperative kernel.  The list is cut into tiles of 256 16-byte words, none
// across two tensors; a CTA takes a contiguous run of tiles, its warps in turn, eight words a
// lane in flight.
//   phase 1   squares, in fp32 over a lane's share of one tile (at most 64), in
//             fp64 from there on, in an order that the sizes, the addresses modulo 16 and the
//             grid fix;
//   barrier   over the grid (bounded); the last CTA to arrive joins the CTAs' sums in
//             their order and publishes the factor.  A CTA that waits too long publishes a
//             failure instead; whichever comes first holds for all, and after a failure none
//             goes on to phase 2.  Up to eight CTAs are one cluster, whose
//             CTAs send one another their sums and join them each;
//   phase 2   the run again, backwards: the last tile is still in registers, the ones before it
//             still in L2.  In place with factor 1 it is left out.
// The factor needs the whole norm first, so gradients beyond what the chip holds are read
// twice: 3 n bytes where the operator's own floor is 2 n.  Measured on 4.23 GB of fp32 in 353 tensors:
// 1,890 us, the measured copy bandwidth on 3 n; on 59 MB of bf16 in 448, whose second read is from L2:
// 30.7 us (28.6 on the GPU alone) against 17.5 at 2 n, the barrier and the short phases' starts being
// the difference.  In place without clipping the second phase is left out: 288 tensors of 1.06 G
// fp32 640 us, one read at the copy bandwidth.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <new>

#include "headloss.h"
#include "headloss_clip.h"

namespace hl_clip {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int LANE_WORDS = 8;
constexpr int TILE = 32 * LANE_WORDS;  // words a tile
constexpr int MAX_GRID = 512;
constexpr int CLUSTER = 8;              // CTAs that are one cluster at most
constexpr int BATCH = 512;             // list entries a launch of list_kernel carries
constexpr unsigned FULL = 0xffffffffu;
constexpr unsigned long long WAIT_NS = 2000000000ull;
constexpr unsigned FAILED = 0x7fffffffu;  // a factor's bits (NaN): a CTA gave up at the barrier

struct Entry {
    const void* grad;
    void* out;
    int64_t n;
    uint32_t first;  // index of the tensor's first tile
    int dtype;
};

// A list in kernel arguments, with the entry each CTA's run starts in (N = 0: the list is in
// the workspace).
template <int N>
struct List {
    Entry e[N];
    uint16_t start[MAX_GRID];
};
template <>
struct List<0> {
    const Entry* e;
};
struct Batch {
    Entry e[BATCH];
};

// The barrier's words on lines of their own: the waiting CTAs' polls would hold up the arrivals.
// The generation counts the handle's launches with a barrier: an arrival tells a CTA its own,
// whenever it comes, and the answer of generation g carries g + 1.
struct Sync {
    alignas(128) unsigned long long arrived;  // generation << 32 | arrivals
    alignas(128) unsigned long long answer;   // generation + 1 << 32 | the factor's bits
    alignas(128) double parts[MAX_GRID];
};

struct Call {
    int n;            // entries
    uint32_t tiles;
    float max_norm, inv_scale;
    float* stats;
    Sync* sync;
    bool cluster;     // the grid is one cluster
#ifdef HL_FAULT_INJECT
    int late;         // a CTA that comes late to the barrier (-1: none), by late_ns
    unsigned long long late_ns, wait_ns;
#endif
};

__global__ void list_kernel(const __grid_constant__ Batch b, Entry* list, int at, int n) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) list[at + i] = b.e[i];
}

// ---------------------------------------------------------------- elements ----

template <int DTYPE>
struct Type;
template <>
struct Type<HEADLOSS_FP32> {
    using T = float;
    static constexpr int EPW = 4;
    __device__ static void unpack(const uint4& w, float* v) {
        v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
    }
    __device__ static uint4 pack(const float* v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
    __device__ static float up(float x) { return x; }
    __device__ static float down(float v) { return v; }
};
template <>
struct Type<HEADLOSS_BF16> {
    using T = __nv_bfloat16;
    static constexpr int EPW = 8;
    __device__ static void unpack(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 pack(const float* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ static float up(T x) { return __bfloat162float(x); }
    __device__ static T down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Type<HEADLOSS_FP16> {
    using T = __half;
    static constexpr int EPW = 8;
    __device__ static void unpack(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    __device__ static uint4 pack(const float* v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ static float up(T x) { return __half2float(x); }
    __device__ static T down(float v) { return __float2half_rn(v); }
};

// -------------------------------------------------------------------- tiles ----

// A lane's part of a tile.  Word w of the tensor starts at its address rounded down to 16
// bytes + 16 w; the words inside the tensor are the tile's [k0, k1), and of the two that may reach
// outside it (the tensor's first and last) a lane has one element at most.
struct Part {
    const uint4* words;  // the tile's first word
    int k0, k1;
    int64_t at;          // element of the tensor at the tile's first word
    int64_t edge;        // the lane's element of a word at an end, or -1
};

template <int D>
__device__ __forceinline__ Part part_of(const Entry& t, uint32_t tile, int lane) {
    constexpr int EPW = Type<D>::EPW, ES = 16 / EPW;
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.grad);
    const int head = int(at & 15) / ES;
    const int64_t w0 = int64_t(tile - t.first) * TILE;
    Part p;
    p.words = reinterpret_cast<const uint4*>(at & ~uintptr_t(15)) + w0;
    p.at = w0 * EPW - head;
    const int64_t left = t.n - p.at;  // elements from the tile's first word on
    p.k0 = p.at < 0 ? 1 : 0;
    p.k1 = left < int64_t(TILE) * EPW ? int(left) / EPW : TILE;
    p.edge = -1;
    if (p.k0) {  // the word before [k0, k1)
        if (lane < EPW && lane >= head && lane - head < t.n) p.edge = lane - head;
    }
    if (left < int64_t(TILE) * EPW && left % EPW && p.k1 >= p.k0) {  // the word after it
        const int e = lane - 16;
        if (e >= 0 && e < int(left % EPW)) p.edge = p.at + int64_t(p.k1) * EPW + e;
    }
    return p;
}

// Any tile word by word: a lane's sum of squares of values times `by`, or the values times `by` to
// out.  For sums that left fp32's range and outputs off the gradient's 16-byte grid.
template <int D>
__device__ __noinline__ float any_tile(const Entry& t, uint32_t tile, int lane, float by, bool store) {
    constexpr int EPW = Type<D>::EPW;
    using T = typename Type<D>::T;
    const Part p = part_of<D>(t, tile, lane);
    T* y = static_cast<T*>(t.out);
    float s = 0.f;
    if (p.edge >= 0) {
        const float v = Type<D>::up(static_cast<const T*>(t.grad)[p.edge]) * by;
        s = v * v;
        if (store) y[p.edge] = Type<D>::down(v);
    }
    for (int k = lane; k < p.k1; k += 32) {  // (the lane's words, as in sum_tile)
        if (k < p.k0) continue;
        float v[EPW];
        Type<D>::unpack(p.words[k], v);
#pragma unroll
        for (int e = 0; e < EPW; ++e) {
            v[e] *= by;
            s = fmaf(v[e], v[e], s);
            if (store) y[p.at + int64_t(k) * EPW + e] = Type<D>::down(v[e]);
        }
    }
    return s;
}

// A lane's words and element of a tile (0 where it has none) to d and `edge`, and its sum of
// squares in fp64: fp32 over the tile's share, from scaled values where that left fp32's range
// or came near its lower end.
template <int D>
__device__ __forceinline__ double sum_tile(const Entry& t, uint32_t tile, int lane, uint4* d,
                                           float* edge) {
    constexpr int EPW = Type<D>::EPW;
    const Part p = part_of<D>(t, tile, lane);
#pragma unroll
    for (int i = 0; i < LANE_WORDS; ++i) {
        const int k = i * 32 + lane;
        d[i] = make_uint4(0, 0, 0, 0);
        if (k >= p.k0 && k < p.k1) d[i] = p.words[k];
    }
    *edge = p.edge >= 0 ? Type<D>::up(static_cast<const typename Type<D>::T*>(t.grad)[p.edge]) : 0.f;
    float s[4] = {*edge * *edge, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < LANE_WORDS; ++i) {
        float v[EPW];
        Type<D>::unpack(d[i], v);
#pragma unroll
        for (int e = 0; e < EPW; ++e) s[e & 3] = fmaf(v[e], v[e], s[e & 3]);
    }
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (sum >= 1e-24f && sum <= 1e36f) return double(sum);
    // (2^100: a sum below 1e-24 comes to 1.6e36 at most, the least subnormal's square to 2^-98)
    const bool low = sum < 1e-24f;
    return double(any_tile<D>(t, tile, lane, low ? 0x1p+100f : 0x1p-70f, false)) *
           (low ? 0x1p-200 : 0x1p+140);
}

// The clipped tile; `here`: the lane's part is in d and `edge`.
template <int D>
__device__ __forceinline__ void clip_tile(const Entry& t, uint32_t tile, int lane, uint4* d,
                                          float edge, bool here, float factor) {
    constexpr int EPW = Type<D>::EPW;
    using T = typename Type<D>::T;
    const Part p = part_of<D>(t, tile, lane);
    T* y = static_cast<T*>(t.out);
    if (reinterpret_cast<uintptr_t>(y + p.at) & 15) {
        any_tile<D>(t, tile, lane, factor, true);
        return;
    }
    if (!here) {
#pragma unroll
        for (int i = 0; i < LANE_WORDS; ++i) {
            const int k = i * 32 + lane;
            if (k >= p.k0 && k < p.k1) d[i] = p.words[k];
        }
        if (p.edge >= 0) edge = Type<D>::up(static_cast<const T*>(t.grad)[p.edge]);
    }
    uint4* out = reinterpret_cast<uint4*>(y + p.at);
#pragma unroll
    for (int i = 0; i < LANE_WORDS; ++i) {
        const int k = i * 32 + lane;
        float v[EPW];
        Type<D>::unpack(d[i], v);
#pragma unroll
        for (int e = 0; e < EPW; ++e) v[e] *= factor;
        if (k >= p.k0 && k < p.k1) __stcs(out + k, Type<D>::pack(v));
    }
    if (p.edge >= 0) y[p.edge] = Type<D>::down(edge * factor);
}

// ------------------------------------------------------------------- kernel ----

// The barrier's words.  An arrival releases the CTA's sum and acquires the others'; the answer
// carries all that the waiting CTAs need in one word, so it needs no fence.
__device__ __forceinline__ unsigned long long arrive(unsigned long long* p) {
    unsigned long long v;
    asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long load_answer(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
// Publishes `v` where the answer still is `seen`, an earlier generation's; the answer that holds.
__device__ __forceinline__ unsigned long long publish(unsigned long long* p, unsigned long long seen,
                                                      unsigned long long v) {
    unsigned long long old;
    asm volatile("atom.cas.relaxed.gpu.global.b64 %0, [%1], %2, %3;"
                 : "=l"(old) : "l"(p), "l"(seen), "l"(v) : "memory");
    return old == seen ? v : old;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// The block's sum, in thread 0 (a fixed order).
__device__ double block_sum(double v) {
    __shared__ double red[WARPS];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < WARPS; ++i) v += red[i];
    return v;
}

template <int N>
__global__ void __launch_bounds__(THREADS, 2) clip_kernel(const __grid_constant__ List<N> list,
                                                          const __grid_constant__ Call c) {
    __shared__ bool s_last;
    __shared__ float s_factor;
    __shared__ double s_parts[CLUSTER];
    if (c.cluster)  // every CTA has started before one writes to another
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t t0 = uint32_t(uint64_t(c.tiles) * blockIdx.x / gridDim.x);
    const uint32_t t1 = uint32_t(uint64_t(c.tiles) * (blockIdx.x + 1) / gridDim.x);
    int at;
    if constexpr (N > 0) {
        at = list.start[blockIdx.x];
    } else {
        int lo = 0, hi = c.n;  // the last entry whose first tile is not after t0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (list.e[mid].first <= t0) lo = mid;
            else hi = mid;
        }
        at = lo;
    }

    uint4 d[LANE_WORDS];
    double mine = 0.0;
    uint32_t last = 0xffffffffu;  // the warp's last tile, in d and edge
    float edge = 0.f;
    for (uint32_t t = t0 + warp; t < t1; t += WARPS) {
        while (at + 1 < c.n && list.e[at + 1].first <= t) ++at;
        const Entry& e = list.e[at];
        if (e.dtype == HEADLOSS_BF16) mine += sum_tile<HEADLOSS_BF16>(e, t, lane, d, &edge);
        else if (e.dtype == HEADLOSS_FP32) mine += sum_tile<HEADLOSS_FP32>(e, t, lane, d, &edge);
        else mine += sum_tile<HEADLOSS_FP16>(e, t, lane, d, &edge);
        last = t;
    }
    mine = block_sum(mine);

    Sync* s = c.sync;
    unsigned long long before = 0;
    unsigned tag = 0;  // of this launch's answer
    const bool alone = gridDim.x == 1 || c.cluster;  // the CTA forms the factor by itself
    if (c.cluster) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (threadIdx.x == 0) {
            const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&s_parts[blockIdx.x]));
            for (unsigned r = 0; r < gridDim.x; ++r) {
                uint32_t to;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(r));
                asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(mine) : "memory");
            }
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (threadIdx.x == 0) {
            mine = 0.0;
            for (unsigned r = 0; r < gridDim.x; ++r) mine += s_parts[r];
        }
    }
    if (threadIdx.x == 0) {
        s_last = alone;
        if (!alone) {
#ifdef HL_FAULT_INJECT
            if (int(blockIdx.x) == c.late)
                for (const unsigned long long from = now_ns(); now_ns() - from < c.late_ns;) __nanosleep(1000);
            const unsigned long long limit = c.wait_ns ? c.wait_ns : WAIT_NS;
#else
            constexpr unsigned long long limit = WAIT_NS;
#endif
            s->parts[blockIdx.x] = mine;
            before = load_answer(&s->answer);
            const unsigned long long n = arrive(&s->arrived);
            tag = unsigned(n >> 32) + 1;
            s_last = unsigned(n) == gridDim.x - 1;
            if (!s_last) {
                const unsigned long long began = now_ns();
                unsigned long long got;
                while (unsigned((got = load_answer(&s->answer)) >> 32) != tag) {
                    __nanosleep(64);
                    if (now_ns() - began > limit) {
                        got = publish(&s->answer, got, uint64_t(tag) << 32 | FAILED);
                        break;
                    }
                }
                s_factor = __uint_as_float(unsigned(got));
            }
        }
    }
    __syncthreads();
    if (s_last) {
        double v = mine;
        if (!alone) {
            v = 0.0;
            for (int i = threadIdx.x; i < int(gridDim.x); i += THREADS)
                v += reinterpret_cast<volatile double*>(s->parts)[i];
            v = block_sum(v);
        }
        if (threadIdx.x == 0) {
            float norm, factor = c.inv_scale;
            if (v >= 1e-30 && v <= 1e36) {  // (fp64's root and division take long here)
                norm = c.inv_scale * sqrtf(float(v));
                if (norm > c.max_norm && isfinite(norm)) factor *= c.max_norm / norm;
            } else {
                const double wide = double(c.inv_scale) * sqrt(v);
                norm = float(wide);
                if (wide > double(c.max_norm) && isfinite(norm))
                    factor = float(double(c.inv_scale) * (double(c.max_norm) / wide));
            }
            if (!alone) {
                unsigned long long got = before;
                if (unsigned(before >> 32) != tag)  // (else one gave up before this CTA came)
                    got = publish(&s->answer, before, uint64_t(tag) << 32 | __float_as_uint(factor));
                s->arrived = uint64_t(tag) << 32;  // (no one arrives any more in this launch)
                factor = __uint_as_float(unsigned(got));
                if (isnan(factor)) norm = factor;
            }
            if (!alone || blockIdx.x == 0) c.stats[0] = norm, c.stats[1] = factor;
            s_factor = factor;
        }
    }
    __syncthreads();
    const float factor = s_factor;

    if (last == 0xffffffffu || isnan(factor)) return;
    bool here = true;
    for (uint32_t t = last;; t -= WARPS) {
        while (list.e[at].first > t) --at;
        const Entry& e = list.e[at];
        if (factor != 1.f || e.grad != e.out) {
            if (e.dtype == HEADLOSS_BF16) clip_tile<HEADLOSS_BF16>(e, t, lane, d, edge, here, factor);
            else if (e.dtype == HEADLOSS_FP32) clip_tile<HEADLOSS_FP32>(e, t, lane, d, edge, here, factor);
            else clip_tile<HEADLOSS_FP16>(e, t, lane, d, edge, here, factor);
        }
        here = false;
        if (t < t0 + WARPS) break;
    }
}

template <int N>
int launch(const List<N>& list, const Call& call, int grid, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (call.cluster) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {unsigned(grid), 1, 1};
    } else {
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = grid > 1;
    void* args[] = {const_cast<List<N>*>(&list), const_cast<Call*>(&call)};
    if (cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&clip_kernel<N>), args) !=
        cudaSuccess) {
        cudaGetLastError();
        return HEADLOSS_ERR_CUDA;
    }
    return HEADLOSS_OK;
}

// The list of a call, put together on the host.
struct Builder {
    const headloss_gradient* g;
    int n, used = 0;
    uint64_t tiles = 0;
    static uint64_t tiles_of(const headloss_gradient& t) {
        const int es = t.dtype == HEADLOSS_FP32 ? 4 : 2, epw = 16 / es;
        const int64_t head = int64_t(reinterpret_cast<uintptr_t>(t.grad) & 15) / es;
        const uint64_t words = uint64_t(head + t.n + epw - 1) / epw;
        return (words + TILE - 1) / TILE;
    }
    void count() {
        for (int i = 0; i < n; ++i)
            if (g[i].n) ++used, tiles += tiles_of(g[i]);
    }
    // calls f(entry) for every tensor that has elements
    template <typename F>
    void each(F f) const {
        uint64_t at = 0;
        for (int i = 0; i < n; ++i) {
            if (!g[i].n) continue;
            f(Entry{g[i].grad, g[i].out, g[i].n, uint32_t(at), g[i].dtype});
            at += tiles_of(g[i]);
        }
    }
};

template <int N>
int launch_list(const Builder& b, const Call& call, int grid, cudaStream_t s) {
    static_assert(sizeof(List<N>) + sizeof(Call) <= 32764, "kernel arguments");
    List<N> list;
    int i = 0;
    b.each([&](const Entry& e) { list.e[i++] = e; });
    int at = 0;
    for (int cta = 0; cta < grid; ++cta) {
        const uint32_t t0 = uint32_t(b.tiles * cta / grid);
        while (at + 1 < b.used && list.e[at + 1].first <= t0) ++at;
        list.start[cta] = uint16_t(at);
    }
    return launch<N>(list, call, grid, s);
}

}  // namespace hl_clip

struct headloss_clip {
    int max_grads = 0;
    int grid = 0;  // CTAs that are resident at once
    void* ws = nullptr;
    hl_clip::Sync* sync = nullptr;
    hl_clip::Entry* list = nullptr;
#ifdef HL_FAULT_INJECT
    int late = -1;
    unsigned long long late_ns = 0, wait_ns = 0;
#endif
};

extern "C" {

int headloss_clip_create(int max_grads, headloss_clip_t* out) {
    using namespace hl_clip;
    if (!out) return HEADLOSS_ERR_ARG;
    *out = nullptr;
    if (max_grads < 1 || max_grads > (1 << 24)) return HEADLOSS_ERR_ARG;
    int device = 0, sms = 0, ctas = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, clip_kernel<1>, THREADS, 0) !=
            cudaSuccess ||
        ctas < 1)
        return HEADLOSS_ERR_CUDA;
    headloss_clip* h = new (std::nothrow) headloss_clip();
    if (!h) return HEADLOSS_ERR_ARG;
    h->max_grads = max_grads;
    h->grid = sms * (ctas < 2 ? ctas : 2);
    if (h->grid > MAX_GRID) h->grid = MAX_GRID;
    if (cudaMalloc(&h->ws, sizeof(Sync) + size_t(max_grads) * sizeof(Entry)) != cudaSuccess ||
        cudaMemset(h->ws, 0, sizeof(Sync)) != cudaSuccess ||
        cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(h->ws);
        delete h;
        return HEADLOSS_ERR_CUDA;
    }
    h->sync = static_cast<Sync*>(h->ws);
    h->list = reinterpret_cast<Entry*>(h->sync + 1);
    *out = h;
    return HEADLOSS_OK;
}

void headloss_clip_destroy(headloss_clip_t h) {
    if (!h) return;
    cudaFree(h->ws);
    delete h;
}

#ifdef HL_FAULT_INJECT
// Test builds alone: CTA `late` (-1: none) comes `late_ns` late to the grid's barrier, where the
// others give up after `wait_ns` (0: the usual limit).
void headloss_clip_test_inject(headloss_clip_t h, int late, unsigned long long late_ns,
                               unsigned long long wait_ns) {
    h->late = late, h->late_ns = late_ns, h->wait_ns = wait_ns;
}
#endif

int headloss_clip_grads(headloss_clip_t h, const headloss_gradient* grads, int n_grads,
                        float max_norm, float inv_scale, float* stats_out, void* stream) {
    using namespace hl_clip;
    if (!h || n_grads < 0 || n_grads > h->max_grads || (n_grads > 0 && !grads) || !stats_out)
        return HEADLOSS_ERR_ARG;
    if (!(max_norm > 0.f) || !(inv_scale > 0.f) || !isfinite(inv_scale)) return HEADLOSS_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(stats_out) & 3u) return HEADLOSS_ERR_ALIGN;
    for (int i = 0; i < n_grads; ++i) {
        const headloss_gradient& g = grads[i];
        if (g.n < 0 || (g.n > 0 && (!g.grad || !g.out))) return HEADLOSS_ERR_ARG;
        if (g.dtype != HEADLOSS_FP32 && g.dtype != HEADLOSS_BF16 && g.dtype != HEADLOSS_FP16)
            return HEADLOSS_ERR_DTYPE;
        if (g.n > 0 && ((reinterpret_cast<uintptr_t>(g.grad) | reinterpret_cast<uintptr_t>(g.out)) &
                        (g.dtype == HEADLOSS_FP32 ? 3u : 1u)))
            return HEADLOSS_ERR_ALIGN;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Builder b{grads, n_grads};
    b.count();
    if (b.tiles >= (uint64_t(1) << 32) - MAX_GRID * WARPS) return HEADLOSS_ERR_ARG;
    Call call = {};
    call.n = b.used;
    call.tiles = uint32_t(b.tiles);
    call.max_norm = max_norm;
    call.inv_scale = inv_scale;
    call.stats = stats_out;
    call.sync = h->sync;
    // a warp a tile as far as the grid goes; a cluster's warps take up to two, which costs less
    // than the grid's barrier
    int64_t want = (int64_t(b.tiles) + WARPS - 1) / WARPS;
    if (want <= 2 * CLUSTER) want = want < CLUSTER ? want : CLUSTER;
    const int grid = int(want < 1 ? 1 : want < h->grid ? want : h->grid);
    call.cluster = grid > 1 && grid <= CLUSTER;
#ifdef HL_FAULT_INJECT
    call.late = h->late, call.late_ns = h->late_ns, call.wait_ns = h->wait_ns;
#endif
    if (b.used <= 1) return launch_list<1>(b, call, grid, s);
    if (b.used <= 16) return launch_list<16>(b, call, grid, s);
    if (b.used <= 64) return launch_list<64>(b, call, grid, s);
    if (b.used <= 160) return launch_list<160>(b, call, grid, s);
    if (b.used <= 320) return launch_list<320>(b, call, grid, s);
    if (b.used <= 512) return launch_list<512>(b, call, grid, s);
    if (b.used <= 960) return launch_list<960>(b, call, grid, s);
    Batch batch;
    int in_batch = 0, at = 0;
    bool ok = true;
    auto flush = [&]() {
        if (in_batch) list_kernel<<<1, 256, 0, s>>>(batch, h->list, at, in_batch);
        ok &= cudaGetLastError() == cudaSuccess;
        at += in_batch;
        in_batch = 0;
    };
    b.each([&](const Entry& e) {
        batch.e[in_batch++] = e;
        if (in_batch == BATCH) flush();
    });
    flush();
    if (!ok) return HEADLOSS_ERR_CUDA;
    return launch<0>(List<0>{h->list}, call, grid, s);
}

}  // extern "C"
