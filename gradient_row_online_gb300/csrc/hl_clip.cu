// hl_clip.cu -- the global gradient norm over many tensors, and clipping
// (headloss_clip_grads in include/headloss_clip.h).
//
// The list is cut into chunks of at most CHUNK elements, none across two
// tensors.  One kernel sums the squares of a chunk (fp32 a thread over
// CHUNK / THREADS elements, fp64 from there on), a second joins the chunks in
// a fixed order and scales.  The list goes to the workspace in kernel
// arguments, a few hundred entries a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <math.h>
#include <stdint.h>

#include <new>

#include "headloss.h"
#include "headloss_clip.h"

namespace hl_clip {

constexpr int THREADS = 256;
constexpr int CHUNK = 16384;
constexpr int GRID = 152 * 8;
constexpr int BATCH = 120;  // list entries a launch of list_kernel carries

struct Entry {
    const void* grad;
    void* out;
    int64_t n;
    int64_t first;  // index of the tensor's first chunk
    int dtype;
};
struct Batch {
    Entry e[BATCH];
};

__global__ void list_kernel(const __grid_constant__ Batch b, Entry* list, int at, int n) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) list[at + i] = b.e[i];
}

__device__ __forceinline__ float load(const void* p, int64_t i, int dtype) {
    if (dtype == HEADLOSS_FP32) return static_cast<const float*>(p)[i];
    if (dtype == HEADLOSS_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store(void* p, int64_t i, int dtype, float v) {
    if (dtype == HEADLOSS_FP32) static_cast<float*>(p)[i] = v;
    else if (dtype == HEADLOSS_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// The entry of a chunk: the last one whose first chunk is not after it.
__device__ int entry_of(const Entry* list, int n, int64_t chunk) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (list[mid].first <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ double block_sum(double v) {
    __shared__ double red[THREADS / 32];
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < THREADS / 32; ++i) v += red[i];
    return v;
}

// The sum of a thread's squares, again from scaled values where the plain sum left
// fp32's range (or came too near its lower end).
constexpr float LOW = 1e-24f, HIGH = 1e36f;

__global__ void __launch_bounds__(THREADS) norm_kernel(const Entry* list, int n, int64_t chunks,
                                                       double* parts) {
    double mine = 0.0;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Entry& t = list[entry_of(list, n, c)];
        const int64_t a = (c - t.first) * CHUNK, b = min(t.n, a + CHUNK);
        const int dtype = t.dtype;
        float s = 0.f;
        for (int64_t i = a + threadIdx.x; i < b; i += THREADS) {
            const float v = load(t.grad, i, dtype);
            s = fmaf(v, v, s);
        }
        if (s >= LOW && s <= HIGH) {
            mine += double(s);
        } else {
            const float up = s < LOW ? 0x1p+60f : 0x1p-70f;
            s = 0.f;
            for (int64_t i = a + threadIdx.x; i < b; i += THREADS) {
                const float v = load(t.grad, i, dtype) * up;
                s = fmaf(v, v, s);
            }
            mine += double(s) / (double(up) * double(up));
        }
    }
    mine = block_sum(mine);
    if (threadIdx.x == 0) parts[blockIdx.x] = mine;
}

__global__ void __launch_bounds__(THREADS) scale_kernel(const Entry* list, int n, int64_t chunks,
                                                        const double* parts, float max_norm,
                                                        float inv_scale, float* stats) {
    double total = 0.0;
    for (int i = threadIdx.x; i < GRID; i += THREADS) total += parts[i];
    total = block_sum(total);
    const double norm = double(inv_scale) * sqrt(total);
    const float factor = norm > double(max_norm) && isfinite(float(norm))
                             ? float(double(inv_scale) * (double(max_norm) / norm))
                             : inv_scale;
    if (blockIdx.x == 0 && threadIdx.x == 0) stats[0] = float(norm), stats[1] = factor;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Entry& t = list[entry_of(list, n, c)];
        if (factor == 1.f && t.grad == t.out) continue;
        const int64_t a = (c - t.first) * CHUNK, b = min(t.n, a + CHUNK);
        const int dtype = t.dtype;
        for (int64_t i = a + threadIdx.x; i < b; i += THREADS)
            store(t.out, i, dtype, load(t.grad, i, dtype) * factor);
    }
}

}  // namespace hl_clip

struct headloss_clip {
    int max_grads = 0;
    void* ws = nullptr;
    double* parts = nullptr;
    hl_clip::Entry* list = nullptr;
};

extern "C" {

int headloss_clip_create(int max_grads, headloss_clip_t* out) {
    using namespace hl_clip;
    if (!out) return HEADLOSS_ERR_ARG;
    *out = nullptr;
    if (max_grads < 1 || max_grads > (1 << 24)) return HEADLOSS_ERR_ARG;
    headloss_clip* h = new (std::nothrow) headloss_clip();
    if (!h) return HEADLOSS_ERR_ARG;
    h->max_grads = max_grads;
    if (cudaMalloc(&h->ws, GRID * sizeof(double) + size_t(max_grads) * sizeof(Entry)) !=
        cudaSuccess) {
        cudaGetLastError();
        delete h;
        return HEADLOSS_ERR_CUDA;
    }
    h->parts = static_cast<double*>(h->ws);
    h->list = reinterpret_cast<Entry*>(h->parts + GRID);
    *out = h;
    return HEADLOSS_OK;
}

void headloss_clip_destroy(headloss_clip_t h) {
    if (!h) return;
    cudaFree(h->ws);
    delete h;
}

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
    int64_t chunks = 0;
    int used = 0;
    Batch b;
    int in_batch = 0;
    auto flush = [&]() {
        if (in_batch) list_kernel<<<1, 128, 0, s>>>(b, h->list, used - in_batch, in_batch);
        in_batch = 0;
    };
    for (int i = 0; i < n_grads; ++i) {
        if (grads[i].n == 0) continue;
        b.e[in_batch++] = Entry{grads[i].grad, grads[i].out, grads[i].n, chunks, grads[i].dtype};
        chunks += (grads[i].n + CHUNK - 1) / CHUNK;
        ++used;
        if (in_batch == BATCH) flush();
    }
    flush();
    norm_kernel<<<GRID, THREADS, 0, s>>>(h->list, used, chunks, h->parts);
    scale_kernel<<<GRID, THREADS, 0, s>>>(h->list, used, chunks, h->parts, max_norm, inv_scale,
                                          stats_out);
    return cudaGetLastError() == cudaSuccess ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
}

}  // extern "C"
