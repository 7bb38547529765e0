// hl_reorder.cu -- headloss_reorder (include/headloss_beam.h): a request's beams take their
// parents' states.
//
// A thread has words (16 bytes where the layout allows) at the same place of all beams of a
// request: it reads the parents' before it writes, so that any map of parents is right in place
// without a copy or a barrier, and a row that is its own parent costs nothing there. The words of
// all beams, and of several places, are in flight together. HBM bound: a parent that several
// beams share is read from HBM once. Measured, GPU time, means over twelve draws of parents and ranges: 16 caches
// of 16 x 4 beams x 8 x 2048 x 128 bf16 in place, up to a quarter of the positions, 64 us, 71% of the measured copy
// rate over the bytes that move (64 to 80% in single draws: a third of the beams move, so most of a thread's
// places have no load in flight); 32 caches of one request 8.5 us, of which a launch that moves nothing
// takes 6.2.
//
// A unit of work is a line (a state, an outer index, a request) or one of C interleaved shares of it;
// its CTA finds the positions to take from begin and end, so that a short range of a long cache costs
// no empty units.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <new>

#include "headloss.h"
#include "headloss_beam.h"
#include "hl_reorder_plan.h"

namespace hl_reorder {

constexpr int MAX_BEAMS = 64;

struct Item {
    const char* src;
    char* dst;
    int64_t row_stride, outer_stride, position_stride;
    int64_t run_words;    // words of a position
    int64_t positions;
    int64_t linear;       // positions follow one another without a gap
};

struct Args {
    const Item* items;
    const uint32_t* lines;  // [n] lines of one request before state i
    int n, beams;
    uint32_t requests, units, shares;
    uint32_t outer;         // lines of every state where they have the same number, else 0
    const int32_t *parents, *begin, *end;
};

// U16 places of 16-byte words at once, and of smaller ones as many as make 16 words.
template <typename W, int BT, int U16>
__host__ __device__ constexpr int places() {
    return sizeof(W) == 16 || BT == 0 ? U16 : 16 / (BT > 0 ? BT : 1);
}
template <typename W, int BT, int U16, int T>
__device__ __forceinline__ void move(const Item& it, const char* src, char* dst, const int32_t* __restrict__ parents,
                                     int B, uint32_t share, uint32_t shares, int64_t words, int64_t first, W* column) {
    constexpr int U = places<W, BT, U16>();
    const int64_t k0 = int64_t(share) * (BT > 0 ? U * T : T), step = int64_t(shares) * (BT > 0 ? U * T : T);
    if (k0 >= words) return;
    const bool inplace = it.src == it.dst;
    auto parent = [&](int b) {
        const int p = __ldg(parents + b);
        return p >= 0 && p < B ? p : b;
    };
    auto place = [&](int64_t k) {
        if (it.linear) return (first * it.run_words + k) * int64_t(sizeof(W));
        const int64_t p = k / it.run_words;
        return (first + p) * it.position_stride + (k - p * it.run_words) * int64_t(sizeof(W));
    };
    if (BT > 0) {
        int64_t from[BT > 0 ? BT : 1];
        uint32_t moves = 0;
#pragma unroll
        for (int b = 0; b < BT; ++b) {
            const int p = b < B ? parent(b) : b;
            from[b] = p * it.row_stride;
            if (b < B && !(inplace && p == b)) moves |= 1u << b;
        }
        if (!moves) return;
#pragma unroll 1
        for (int64_t k = k0 + threadIdx.x; k < words; k += step) {
            W v[U][BT > 0 ? BT : 1];
            int64_t at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                at[u] = place(k + u * T);
#pragma unroll
                for (int b = 0; b < BT; ++b)
                    if ((moves >> b & 1) && k + u * T < words) v[u][b] = *reinterpret_cast<const W*>(src + from[b] + at[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int b = 0; b < BT; ++b)
                    if ((moves >> b & 1) && k + u * T < words) *reinterpret_cast<W*>(dst + b * it.row_stride + at[u]) = v[u][b];
        }
    } else {  // more beams than registers: through a column of shared memory of the thread's own
        for (int64_t k = k0 + threadIdx.x; k < words; k += step) {
            const int64_t at = place(k);
            for (int b = 0; b < B; ++b) {
                const int p = parent(b);
                if (!(inplace && p == b)) column[b * T + threadIdx.x] = *reinterpret_cast<const W*>(src + p * it.row_stride + at);
            }
            for (int b = 0; b < B; ++b)
                if (!(inplace && parent(b) == b))
                    *reinterpret_cast<W*>(dst + b * it.row_stride + at) = column[b * T + threadIdx.x];
        }
    }
}

template <typename W, int BT, int U, int T>
__global__ void __launch_bounds__(T, 512 / T) reorder_kernel(const Args a) {
    extern __shared__ __align__(16) unsigned char columns[];
    for (uint32_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        const uint32_t share = unit % a.shares, line = unit / a.shares;
        const uint32_t q = line / a.requests, r = line - q * a.requests;
        // the state: the last one whose lines begin at or before q
        int lo = a.outer ? int(q / a.outer) : 0, hi = a.outer ? lo : a.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (__ldg(a.lines + mid) <= q) lo = mid;
            else hi = mid - 1;
        }
        const Item it = a.items[lo];
        int64_t first = 0, last = it.positions;
        if (a.begin) {
            first = max(__ldg(a.begin + r), 0);
            last = min(int64_t(__ldg(a.end + r)), it.positions);
        }
        const int64_t words = (last - first) * it.run_words;
        if (words <= 0) continue;
        const int64_t at = int64_t(r) * a.beams * it.row_stride +
                           int64_t(q - (a.outer ? uint32_t(lo) * a.outer : __ldg(a.lines + lo))) * it.outer_stride;
        move<W, BT, U, T>(it, it.src + at, it.dst + at, a.parents + int64_t(r) * a.beams, a.beams, share, a.shares,
                          words, first, reinterpret_cast<W*>(columns));
    }
}

inline int64_t gcd(int64_t a, int64_t b) {
    while (b) {
        const int64_t t = a % b;
        a = b;
        b = t;
    }
    return a;
}

// The states whose words have one size.
struct Group {
    const Item* items;
    const uint32_t* lines;
    int n;
    int64_t total;   // lines of one request
    int64_t most;    // words of the longest
    int64_t outer;   // lines of every state where they have the same number, else -1
};

template <typename W, int BT, int U, int T>
int launch(Args a, const Group& g, int sms, int smem, cudaStream_t s) {
    constexpr int chunk = places<W, BT, U>() * T;
    const int64_t chunks = (g.most + chunk - 1) / chunk, lines = g.total * a.requests;
    // The CTAs that are resident at once: a second wave of fewer ends later (the mean of 16 caches of 16 x 4 beams
    // over twelve draws of parents and ranges 69 us, and 64; through shared memory, where twice as many
    // fit, the other way round: 216 us of 32 beams, and 198).
    const int64_t grid = int64_t(sms) * ((BT ? 512 : 1024) / T);
    const int64_t shares = shares_of(lines, g.most, chunks, grid);
    a.shares = uint32_t(shares);
    a.units = uint32_t(lines * shares);
    // Requests differ in their moves and ranges, and follow one another in the units: with a grid that shares
    // no divisor with their number every CTA meets all of them.
    int64_t ctas = a.units < grid ? a.units : grid;
    while (ctas < a.units && gcd(ctas, a.requests * shares) > 1) --ctas;
    if (smem && cudaFuncSetAttribute(reorder_kernel<W, BT, U, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return HEADLOSS_ERR_CUDA;
    reorder_kernel<W, BT, U, T><<<unsigned(ctas), T, smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
}

// Twelve to sixteen words of a thread in flight, in 128 registers: three places of four beams' 16-byte words (a fourth
// spills; two places of five to eight beams spill 88 bytes, the smaller words of up to four beams 20), fewer places
// where a line has too few words for that on every SM; more than 16 beams go through shared memory.
template <typename W>
int launch_words(const Args& a, const Group& g, int sms, cudaStream_t s) {
    constexpr int FULL = sizeof(W) == 16 ? 3 : 1;  // (of smaller words `places` takes as many as make 16)
    if (a.beams > 16) return launch<W, 0, 1, 128>(a, g, sms, a.beams * 128 * int(sizeof(W)), s);
    if (a.beams > 8) return launch<W, 16, 1, 256>(a, g, sms, 0, s);
    const bool few = g.total * a.requests * ((g.most + 1023) / 1024) < 4 * sms;
    if (a.beams > 4) return few ? launch<W, 8, 1, 128>(a, g, sms, 0, s) : launch<W, 8, 2, 256>(a, g, sms, 0, s);
    return few ? launch<W, 4, 1, 256>(a, g, sms, 0, s) : launch<W, 4, FULL, 256>(a, g, sms, 0, s);
}

}  // namespace hl_reorder

struct headloss_reorder_s {
    hl_reorder::Item* items;
    uint32_t* lines;
    int beams, sms;
    hl_reorder::Group groups[4];  // words of 16, 4, 2 and 1 bytes
    headloss_state* states;       // on the host
    int n;
    std::atomic<int64_t> apart;   // so many rows are known to share no memory
};

extern "C" int headloss_reorder_create(const headloss_state* states, int n, int beams, headloss_reorder_t* out) {
    using namespace hl_reorder;
    if (!states || !out || n < 1 || n > (1 << 20) || beams < 1 || beams > MAX_BEAMS) return HEADLOSS_ERR_ARG;
    int live = 0;  // states that hold anything
    for (int i = 0; i < n; ++i) {
        const headloss_state& s = states[i];
        if (!s.state || !s.out || s.outer < 0 || s.positions < 0 || s.run_bytes < 0 || s.row_stride < 0 ||
            s.outer_stride < 0 || s.position_stride < 0)
            return HEADLOSS_ERR_ARG;
        if (!s.outer || !s.positions || !s.run_bytes) continue;
        if (s.outer > INT32_MAX || s.positions > INT64_MAX / s.run_bytes) return HEADLOSS_ERR_ARG;
        ++live;
    }
    Item* items = new (std::nothrow) Item[n];
    uint32_t* lines = new (std::nothrow) uint32_t[n];
    headloss_reorder_s* h = new (std::nothrow) headloss_reorder_s();
    headloss_state* held = new (std::nothrow) headloss_state[live > 0 ? live : 1];
    if (h) h->states = new (std::nothrow) headloss_state[live > 0 ? live : 1];
    int rc = items && lines && h && held && h->states ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
    if (rc == HEADLOSS_OK) {
        live = 0;
        for (int i = 0; i < n; ++i)
            if (states[i].outer && states[i].positions && states[i].run_bytes) held[live++] = states[i];
        h->n = without_repeats(held, live, h->states);
        if (h->n < 0) rc = HEADLOSS_ERR_CUDA;
    }
    int used = 0;
    const int sizes[4] = {16, 4, 2, 1};
    for (int t = 0; t < 4 && rc == HEADLOSS_OK; ++t) {
        const int from = used;
        Group group = {};
        for (int i = 0; i < h->n; ++i) {
            const headloss_state& s = h->states[i];
            const int64_t outer_stride = s.outer > 1 ? s.outer_stride : 0;
            const int64_t position_stride = s.positions > 1 ? s.position_stride : s.run_bytes;
            const uint64_t bits = uint64_t(reinterpret_cast<uintptr_t>(s.state) | reinterpret_cast<uintptr_t>(s.out)) |
                                  uint64_t(s.row_stride | outer_stride | position_stride | s.run_bytes);
            if ((bits & 1 ? 1 : bits & 2 ? 2 : bits & 12 ? 4 : 16) != sizes[t]) continue;
            Item& it = items[used];
            it.src = static_cast<const char*>(s.state);
            it.dst = static_cast<char*>(s.out);
            it.row_stride = s.row_stride;
            it.outer_stride = outer_stride;
            it.position_stride = position_stride;
            it.run_words = s.run_bytes / sizes[t];
            it.positions = s.positions;
            it.linear = position_stride == s.run_bytes;
            lines[used] = uint32_t(group.total);
            group.outer = used == from || group.outer == s.outer ? s.outer : -1;
            ++used;
            group.total += s.outer;
            if (group.total > INT32_MAX) {
                rc = HEADLOSS_ERR_ARG;
                break;
            }
            if (it.positions * it.run_words > group.most) group.most = it.positions * it.run_words;
        }
        group.n = used - from;
        h->groups[t] = group;
    }
    if (rc == HEADLOSS_OK) {
        h->beams = beams;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaMalloc(&h->items, n * sizeof(Item)) != cudaSuccess ||
            cudaMalloc(&h->lines, n * sizeof(uint32_t)) != cudaSuccess ||
            cudaMemcpy(h->items, items, used * sizeof(Item), cudaMemcpyHostToDevice) != cudaSuccess ||
            cudaMemcpy(h->lines, lines, used * sizeof(uint32_t), cudaMemcpyHostToDevice) != cudaSuccess) {
            cudaGetLastError();
            rc = HEADLOSS_ERR_CUDA;
        }
        int from = 0;
        for (int t = 0; t < 4; ++t) {
            h->groups[t].items = h->items + from;
            h->groups[t].lines = h->lines + from;
            from += h->groups[t].n;
        }
    }
    delete[] items;
    delete[] lines;
    delete[] held;
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
    for (const Group& g : h->groups)
        if (g.total * requests > INT32_MAX) return HEADLOSS_ERR_ARG;
    const int64_t rows = requests * h->beams;
    if (rows > h->apart.load(std::memory_order_relaxed)) {
        if (conflict(h->states, h->n, rows)) return HEADLOSS_ERR_ARG;
        h->apart.store(rows, std::memory_order_relaxed);  // (another call's smaller number is right, too)
    }
    Args a = {};
    a.beams = h->beams;
    a.requests = uint32_t(requests);
    a.parents = parents;
    a.begin = begin;
    a.end = end;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int t = 0; t < 4; ++t) {
        const Group& g = h->groups[t];
        if (!g.n) continue;
        a.items = g.items;
        a.lines = g.lines;
        a.n = g.n;
        a.outer = g.outer > 0 ? uint32_t(g.outer) : 0;
        const int rc = t == 0   ? launch_words<uint4>(a, g, h->sms, s)
                       : t == 1 ? launch_words<uint32_t>(a, g, h->sms, s)
                       : t == 2 ? launch_words<uint16_t>(a, g, h->sms, s)
                                : launch_words<uint8_t>(a, g, h->sms, s);
        if (rc != HEADLOSS_OK) return rc;
    }
    return HEADLOSS_OK;
}

extern "C" void headloss_reorder_destroy(headloss_reorder_t h) {
    if (!h) return;
    if (h->items) cudaFree(h->items);
    if (h->lines) cudaFree(h->lines);
    delete[] h->states;
    delete h;
}
