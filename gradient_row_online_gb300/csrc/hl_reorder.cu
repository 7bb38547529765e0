// hl_reorder.cu -- headloss_reorder (include/headloss_beam.h): a request's beams take their
// parents' states.
//
// A thread has one word (16 bytes where the layout allows) at the same place of all beams of a
// request: it reads the parents' before it writes, so that any map of parents is right in place
// without a copy or a barrier, and a row that is its own parent costs nothing there. The words of
// all beams are in flight together. HBM bound: a parent that several beams share is read from
// HBM once.
#include <cuda_runtime.h>
#include <stdint.h>

#include <new>

#include "headloss.h"
#include "headloss_beam.h"

namespace hl_reorder {

constexpr int CHUNK = 1024;     // words of a unit of work
constexpr int MAX_BEAMS = 64;

struct Item {
    const char* src;
    char* dst;
    int64_t row_stride, outer_stride, position_stride;
    int64_t run_words;    // words of a position
    int64_t outer, positions;
    int64_t chunks;       // units of a line (request, outer)
    int word;             // bytes
    int linear;           // positions follow one another without a gap
};

struct Args {
    const Item* items;
    const int64_t* lines;  // [n + 1] units of one request before state i
    int n, beams;
    int64_t requests, units;
    const int32_t *parents, *begin, *end;
};

template <typename W, int BT, int T>
__device__ __forceinline__ void move(const Item& it, const char* src, char* dst, const int32_t* __restrict__ par,
                                     int B, int64_t k0, int64_t k1, int64_t first, W* column) {
    const bool inplace = it.src == it.dst;
    for (int64_t k = k0 + threadIdx.x; k < k1; k += T) {
        int64_t at;
        if (it.linear) {
            at = (first * it.run_words + k) * int64_t(sizeof(W));
        } else {
            const int64_t p = k / it.run_words;
            at = (first + p) * it.position_stride + (k - p * it.run_words) * int64_t(sizeof(W));
        }
        if (BT > 0) {
            W v[BT > 0 ? BT : 1];
#pragma unroll
            for (int b = 0; b < BT; ++b)
                if (b < B && !(inplace && par[b] == b))
                    v[b] = *reinterpret_cast<const W*>(src + par[b] * it.row_stride + at);
#pragma unroll
            for (int b = 0; b < BT; ++b)
                if (b < B && !(inplace && par[b] == b)) *reinterpret_cast<W*>(dst + b * it.row_stride + at) = v[b];
        } else {  // more beams than registers: through a column of shared memory of the thread's own
            for (int b = 0; b < B; ++b)
                if (!(inplace && par[b] == b))
                    column[b * T + threadIdx.x] = *reinterpret_cast<const W*>(src + par[b] * it.row_stride + at);
            for (int b = 0; b < B; ++b)
                if (!(inplace && par[b] == b))
                    *reinterpret_cast<W*>(dst + b * it.row_stride + at) = column[b * T + threadIdx.x];
        }
    }
}

template <int BT, int T>
__global__ void __launch_bounds__(T) reorder_kernel(const Args a) {
    extern __shared__ __align__(16) unsigned char columns[];
    __shared__ int32_t par[MAX_BEAMS];
    for (int64_t u = blockIdx.x; u < a.units; u += gridDim.x) {
        const int64_t r = u % a.requests, line = u / a.requests;
        int lo = 0, hi = a.n - 1;  // the state: the last one whose units begin at or before `line`
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (a.lines[mid] <= line) lo = mid;
            else hi = mid - 1;
        }
        const Item& it = a.items[lo];
        const int64_t in = line - a.lines[lo], o = in / it.chunks, c = in - o * it.chunks;
        int64_t first = 0, last = it.positions;
        if (a.begin) {
            first = max(int64_t(a.begin[r]), int64_t(0));
            last = min(int64_t(a.end[r]), it.positions);
        }
        const int64_t words = (last - first) * it.run_words, k0 = c * CHUNK, k1 = min(words, k0 + CHUNK);
        if (k0 >= k1) continue;
        __syncthreads();
        if (threadIdx.x < a.beams) {
            const int p = a.parents[r * a.beams + threadIdx.x];
            par[threadIdx.x] = p >= 0 && p < a.beams ? p : int(threadIdx.x);
        }
        __syncthreads();
        const int64_t at = r * a.beams * it.row_stride + o * it.outer_stride;
        const char* src = it.src + at;
        char* dst = it.dst + at;
        switch (it.word) {
            case 16: move<uint4, BT, T>(it, src, dst, par, a.beams, k0, k1, first, reinterpret_cast<uint4*>(columns)); break;
            case 4: move<uint32_t, BT, T>(it, src, dst, par, a.beams, k0, k1, first, reinterpret_cast<uint32_t*>(columns)); break;
            case 2: move<uint16_t, BT, T>(it, src, dst, par, a.beams, k0, k1, first, reinterpret_cast<uint16_t*>(columns)); break;
            default: move<uint8_t, BT, T>(it, src, dst, par, a.beams, k0, k1, first, columns); break;
        }
    }
}

}  // namespace hl_reorder

struct headloss_reorder_s {
    hl_reorder::Item* items;
    int64_t* lines;
    int n, beams, sms;
    int64_t units;  // of one request
};

extern "C" int headloss_reorder_create(const headloss_state* states, int n, int beams, headloss_reorder_t* out) {
    using namespace hl_reorder;
    if (!states || !out || n < 1 || n > (1 << 20) || beams < 1 || beams > MAX_BEAMS) return HEADLOSS_ERR_ARG;
    Item* items = new (std::nothrow) Item[n];
    int64_t* lines = new (std::nothrow) int64_t[n + 1];
    headloss_reorder_s* h = new (std::nothrow) headloss_reorder_s();
    int rc = items && lines && h ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
    int64_t units = 0;
    for (int i = 0; rc == HEADLOSS_OK && i < n; ++i) {
        const headloss_state& s = states[i];
        if (!s.state || !s.out || s.outer < 0 || s.positions < 0 || s.run_bytes < 0 || s.row_stride < 0 ||
            s.outer_stride < 0 || s.position_stride < 0) {
            rc = HEADLOSS_ERR_ARG;
            break;
        }
        Item& it = items[i];
        it.src = static_cast<const char*>(s.state);
        it.dst = static_cast<char*>(s.out);
        it.row_stride = s.row_stride;
        it.outer_stride = s.outer > 1 ? s.outer_stride : 0;
        it.position_stride = s.positions > 1 ? s.position_stride : s.run_bytes;
        const uint64_t bits = uint64_t(reinterpret_cast<uintptr_t>(s.state) | reinterpret_cast<uintptr_t>(s.out)) |
                              uint64_t(it.row_stride | it.outer_stride | it.position_stride | s.run_bytes);
        it.word = bits & 1 ? 1 : bits & 2 ? 2 : bits & 12 ? 4 : 16;
        it.run_words = s.run_bytes / it.word;
        it.outer = s.outer;
        it.positions = s.positions;
        it.linear = it.position_stride == s.run_bytes;
        const int64_t words = it.positions * it.run_words;
        it.chunks = words ? (words + CHUNK - 1) / CHUNK : 0;
        lines[i] = units;
        units += it.outer * it.chunks;
    }
    if (rc == HEADLOSS_OK) {
        lines[n] = units;
        h->n = n;
        h->beams = beams;
        h->units = units;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaMalloc(&h->items, n * sizeof(Item)) != cudaSuccess ||
            cudaMalloc(&h->lines, (n + 1) * sizeof(int64_t)) != cudaSuccess ||
            cudaMemcpy(h->items, items, n * sizeof(Item), cudaMemcpyHostToDevice) != cudaSuccess ||
            cudaMemcpy(h->lines, lines, (n + 1) * sizeof(int64_t), cudaMemcpyHostToDevice) != cudaSuccess)
            rc = HEADLOSS_ERR_CUDA;
    }
    delete[] items;
    delete[] lines;
    if (rc != HEADLOSS_OK) {
        headloss_reorder_destroy(h);
        return rc;
    }
    *out = h;
    return HEADLOSS_OK;
}

extern "C" int headloss_reorder(headloss_reorder_t h, const int32_t* parents, int64_t requests,
                                const int32_t* begin, const int32_t* end, void* stream) {
    using namespace hl_reorder;
    if (!h || requests < 0 || requests > INT32_MAX || requests * h->beams > INT32_MAX) return HEADLOSS_ERR_ARG;
    if (requests == 0) return HEADLOSS_OK;
    if (!parents || !begin != !end) return HEADLOSS_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(parents) | reinterpret_cast<uintptr_t>(begin) | reinterpret_cast<uintptr_t>(end)) & 3)
        return HEADLOSS_ERR_ALIGN;
    Args a = {};
    a.items = h->items;
    a.lines = h->lines;
    a.n = h->n;
    a.beams = h->beams;
    a.requests = requests;
    a.units = h->units * requests;
    a.parents = parents;
    a.begin = begin;
    a.end = end;
    if (a.units == 0) return HEADLOSS_OK;
    const int64_t most = int64_t(h->sms) * 8;
    const unsigned grid = unsigned(a.units < most ? a.units : most);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (h->beams <= 4) reorder_kernel<4, 256><<<grid, 256, 0, s>>>(a);
    else if (h->beams <= 8) reorder_kernel<8, 256><<<grid, 256, 0, s>>>(a);
    else if (h->beams <= 16) reorder_kernel<16, 256><<<grid, 256, 0, s>>>(a);
    else {
        const int bytes = h->beams * 128 * 16;
        if (cudaFuncSetAttribute(reorder_kernel<0, 128>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return HEADLOSS_ERR_CUDA;
        reorder_kernel<0, 128><<<grid, 128, bytes, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
}

extern "C" void headloss_reorder_destroy(headloss_reorder_t h) {
    if (!h) return;
    if (h->items) cudaFree(h->items);
    if (h->lines) cudaFree(h->lines);
    delete h;
}
