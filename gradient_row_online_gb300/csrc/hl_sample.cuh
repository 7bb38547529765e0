// hl_sample.cuh -- the sampling kernel (headloss_sample in
// include/headloss_sample.h, where the definition stands).
//
// One thread-block cluster a row, each CTA a contiguous run of the row's 16-byte
// words in its shared memory, each warp a contiguous segment of that, copied by
// the warp's own cp.async.bulk.  A logit is read from HBM once; every later pass
// is over shared memory.  (Rows too long for eight CTAs' shared memory are read from
// global memory in every pass: RES = false.)
//
// All three filters keep a prefix of the order (x descending, index ascending), so a
// row's kept set is a cut in that order, and min-p's comparison.  Masses are integers
// (2^30 the largest logit's): exact sums in any order, so atomics, splits and cluster
// sizes never change a token.  A row goes one of three ways:
//
//   no top-k, no top-p   one pass sums the masses by warp segment.
//   a small top-k        the k-th largest of the CTA's thread maxima bounds the cut from
//                        below (at least k tokens lie at or above it); the few
//                        tokens at or above the largest CTA's bound go to the leader CTA,
//                        which ranks them and finishes the row alone.
//   else                 `resolve`: a histogram of the order (1/32 octave of mass a bin) with
//                        exact integer masses finds the bin of the cut, whose few tokens go to
//                        the leader to be ranked; a bin with too many (ties, dense rows) is
//                        cut into bins of keys again.  Then the segment masses of what is kept.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>

#include "headloss.h"
#include "hl_rows.cuh"

namespace hl_sample {

using hl::bulk_g2s;
using hl::cluster_ctarank;
using hl::map_peer;
using hl::smem_addr;

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAXC = 8;       // CTAs a cluster at most
constexpr int BINS = 2 * THREADS;
constexpr int CAP = 2048;     // tokens the leader can rank
constexpr int RANKED = 512;   // ranked by comparison with all; more are sorted
constexpr int MAX_TOPK = 256; // longest top-k that takes the thread-maxima bound
constexpr float UNIT = 1073741824.f;  // 2^30, the weight of the largest logit
constexpr float MODEL_UNIT = 1099511627776.f;  // 2^40
constexpr float LN2 = 0.69314718055994531f;
constexpr unsigned FULL = 0xffffffffu;
constexpr unsigned long long WAIT_NS = 2000000000ull;

struct Args {
    const void* logits;
    int64_t ld;
    int64_t row0;  // first row of this launch
    int V;
    const double* uniforms;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    float cap, inv_cap, K;
    int64_t* tokens;
    float* logprobs;
    float* draw_logprobs;
    int32_t* n_kept;
    int* err;
};

typedef unsigned long long u64;

struct Shared {
    u64 bar[WARPS];
    u64 list[CAP];       // (key << 32 | ~index) of the tokens to rank, a run a CTA (leader)
    u64 sorted[RANKED];
    u64 scratch[BINS];   // the list put together; the histogram's masses (hi, lo halves)
    uint32_t cnt[BINS];
    u64 xch[2][MAXC][4];
    u64 red[WARPS];
    u64 seg[WARPS];
    u64 ored[WARPS];
    float fred[WARPS];
    uint32_t list_n[MAXC];
    u64 list_own[MAXC];
    uint32_t n_local;
    uint32_t pick_bin, pick_n, pick_most;
    u64 pick_before;
    uint32_t cut_key;
    int cut_idx;
};

// A cut of the order: tokens above the key stay, and at the key those up to an index.
struct Cut {
    uint32_t key;
    int idx;
};
constexpr Cut NO_CUT{0u, 0x7fffffff};

// A key whose unsigned order is the order of the floats; -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t KEY_NONE = 0x007fffffu;  // -inf

__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// rint(2^30 e); a NaN gives 0
__device__ __forceinline__ uint32_t weight_of(float e) {
    return __float2uint_rn(__fmul_rn(e, UNIT));
}

// ---------------------------------------------------------------- elements ----

template <typename DT>
struct Elem;

template <>
struct Elem<__nv_bfloat16> {
    static constexpr int EPW = 8;
    static constexpr uint32_t LOWEST = 0xff80ff80u;  // -inf twice
    __device__ static void unpack(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ static uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // largest of the running pair
    __device__ static float top(uint32_t m) {
        const float a = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        return a == a ? a : -CUDART_INF_F;
    }
    __device__ static uint32_t word_max(const uint4& w) {
        return max2(max2(w.x, w.y), max2(w.z, w.w));
    }
    __device__ static float load(const void* p, int64_t i) {
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    }
};

template <>
struct Elem<__half> {
    static constexpr int EPW = 8;
    static constexpr uint32_t LOWEST = 0xfc00fc00u;
    __device__ static void unpack(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    __device__ static uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    __device__ static float top(uint32_t m) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
        const float a = fmaxf(f.x, f.y);
        return a == a ? a : -CUDART_INF_F;
    }
    __device__ static uint32_t word_max(const uint4& w) {
        return max2(max2(w.x, w.y), max2(w.z, w.w));
    }
    __device__ static float load(const void* p, int64_t i) {
        return __half2float(static_cast<const __half*>(p)[i]);
    }
};

template <>
struct Elem<float> {
    static constexpr int EPW = 4;
    static constexpr uint32_t LOWEST = 0xff800000u;
    __device__ static void unpack(const uint4& w, float* v) {
        v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
    }
    __device__ static uint32_t max2(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    __device__ static float top(uint32_t m) {
        const float a = __uint_as_float(m);
        return a == a ? a : -CUDART_INF_F;
    }
    __device__ static uint32_t word_max(const uint4& w) {
        return max2(max2(w.x, w.y), max2(w.z, w.w));
    }
    __device__ static float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
};

// ------------------------------------------------------------ block helpers ----

__device__ __forceinline__ u64 warp_add(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 n = __shfl_up_sync(FULL, v, o);
        if (lane >= o) v += n;
    }
    return v;
}
// Exclusive prefix over the block's threads, and the block's total.
__device__ __forceinline__ u64 block_scan(u64 v, u64* red, u64* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 inc = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    const u64 mine = warp_scan(lane < WARPS ? red[lane] : 0, lane);
    *total = __shfl_sync(FULL, mine, WARPS - 1);
    const u64 before = __shfl_sync(FULL, mine, warp ? warp - 1 : 0);
    return inc - v + (warp ? before : 0);
}

__device__ __forceinline__ void st_peer64(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_peer32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_peer32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    hl::cluster_barrier();
}

// -------------------------------------------------------------------- a row ----

template <typename DT, bool CAPPED, bool RES>
struct Row {
    using E = Elem<DT>;
    static constexpr int EPW = E::EPW;

    const Args& a;
    Shared& s;
    uint4* words;        // this CTA's words (RES)
    const uint4* gwords; // the row's first word in global memory (16-byte aligned)
    int64_t row;
    int head;            // elements of the first word before the row
    int C, rank, lane, warp;
    int w0, s0, s1;      // the CTA's first word of the row; the warp's segment of its words
    int nw;              // words of the row
    int par = 0;
    bool inf_row = false;
    float top, zm, c;

    __device__ Row(const Args& a_, Shared& s_) : a(a_), s(s_) {}

    // index of element e of the CTA's word i
    __device__ int index(int i, int e) const { return (w0 + i) * EPW + e - head; }

    // A word of the row in global memory; elements outside the row are -inf.
    __device__ uint4 global_word(int w) const {
        const int first = w * EPW - head;
        if (first >= 0 && first + EPW <= a.V) return __ldg(gwords + w);
        union {
            uint4 q;
            DT d[EPW];
        } u;
        u.q = make_uint4(E::LOWEST, E::LOWEST, E::LOWEST, E::LOWEST);
        const DT* x = reinterpret_cast<const DT*>(gwords);
        for (int e = 0; e < EPW; ++e)
            if (first + e >= 0 && first + e < a.V) u.d[e] = x[w * EPW + e];
        return u.q;
    }
    __device__ __forceinline__ uint4 word(int i) const {
        if constexpr (RES) return words[i];
        else return global_word(w0 + i);
    }
    __device__ __forceinline__ void values(int i, float* v) const {
        E::unpack(word(i), v);
        if constexpr (!RES) {
            if (inf_row)
                for (int e = 0; e < EPW; ++e) v[e] = v[e] == CUDART_INF_F ? 0.f : -CUDART_INF_F;
        }
    }

    __device__ __forceinline__ float z(float v) const {
        if constexpr (CAPPED) return __fmul_rn(tanhf(__fmul_rn(v, a.inv_cap)), a.cap);
        else return v;
    }
    // Exponent and mass share of a logit.  Without a softcap -inf and NaN give 0 mass by
    // themselves.
    __device__ __forceinline__ float share(float v) const {
        const float e = ex2f(__fmul_rn(__fsub_rn(z(v), zm), c));
        if constexpr (CAPPED) return v > -CUDART_INF_F ? e : 0.f;
        else return e;
    }
    // The same where +inf may stand (ranked tokens of a row that was not rewritten).
    __device__ __forceinline__ float exponent(float v) const {
        const float zz = z(v);
        return zz == zm ? 0.f : __fmul_rn(__fsub_rn(zz, zm), c);
    }
    __device__ __forceinline__ float model_share(float v) const {
        const float e = ex2f(__fmul_rn(__fsub_rn(z(v), zm), a.K));
        if constexpr (CAPPED) return v > -CUDART_INF_F ? e : 0.f;
        else return e;
    }
    // Mass of the whole softmax at T = 1: a word's shares summed in fp32 in one order, the words
    // in fixed point (2^-40 of the largest logit's), so that it too is the same
    // however the row is split.
    struct Model {
        u64 sum = 0;
        bool odd = false;  // a word with a NaN (or +inf)
        __device__ __forceinline__ void add(const float* sh) {
            float t;
            if constexpr (EPW == 8)
                t = ((sh[0] + sh[1]) + (sh[2] + sh[3])) + ((sh[4] + sh[5]) + (sh[6] + sh[7]));
            else t = (sh[0] + sh[1]) + (sh[2] + sh[3]);
            odd |= !(t < 16.f);
            sum += __float2ull_rn(__fmul_rn(t, MODEL_UNIT));
        }
    };
    __device__ __forceinline__ void add_model(Model& m, const float* v) const {
        float sh[EPW];
#pragma unroll
        for (int e = 0; e < EPW; ++e) sh[e] = model_share(v[e]);
        m.add(sh);
    }
    // The warp's sum; words with a NaN or +inf are gone over again with care.
    __device__ u64 model_sum(Model m) const {
        if (__any_sync(FULL, m.odd)) {
            m = Model();
            for (int i = s0 + lane; i < s1; i += 32) {
                float v[EPW];
                values(i, v);
                for (int e = 0; e < EPW; ++e) {
                    const float zz = z(v[e]);
                    v[e] = !(v[e] > -CUDART_INF_F) ? 0.f
                           : zz == zm              ? 1.f
                                      : ex2f(__fmul_rn(__fsub_rn(zz, zm), a.K));
                }
                m.add(v);
            }
        }
        return warp_add(m.sum);
    }

    // Bin of the order: 1/32 octave of mass a bin without a softcap (with one, of the raw
    // logit's distance); the last takes what is further off.
    __device__ __forceinline__ uint32_t bin_of(float v) const {
        return min(uint32_t(BINS - 1),
                   __float2uint_rz(__fmul_rn(__fmul_rn(__fsub_rn(top, v), c), 32.f)));
    }
    __device__ __forceinline__ bool inside(float v, int idx, const Cut& k, float kv) const {
        return v > kv || (v == kv && idx <= k.idx);
    }

    // Every CTA's NV values (in warp 0's lanes, all alike) at every CTA.
    template <int NV>
    __device__ const u64 (*exchange(const u64 (&v)[NV]))[4] {
        if (warp == 0 && lane < C) {
            const uint32_t at = map_peer(smem_addr(&s.xch[par][rank][0]), lane);
#pragma unroll
            for (int i = 0; i < NV; ++i) st_peer64(at + 8 * i, v[i]);
        }
        cluster_barrier();
        const u64(*got)[4] = s.xch[par];
        par ^= 1;
        return got;
    }

    __device__ void no_token() const {
        a.tokens[row] = -1;
        if (a.logprobs) a.logprobs[row] = 0.f;
        if (a.draw_logprobs) a.draw_logprobs[row] = 0.f;
        if (a.n_kept) a.n_kept[row] = 0;
    }
    __device__ void answer(float v, int idx, u64 W, u64 own, int kept) const {
        a.tokens[row] = idx;
        const float zz = z(v);
        if (a.logprobs)
            a.logprobs[row] = (zz == zm ? 0.f : __fsub_rn(zz, zm) * a.K * LN2) -
                              logf(float(double(own) * (1.0 / MODEL_UNIT)));
        if (a.draw_logprobs)
            a.draw_logprobs[row] = exponent(v) * LN2 - logf(float(double(W) * (1.0 / UNIT)));
        if (a.n_kept) a.n_kept[row] = kept;
    }
    __device__ static u64 target_of(double u, u64 W) {
        const u64 t = u64(u * double(W));
        return t < W ? t : W - 1;
    }

    // ------------------------------------------------------ lists to rank ----

    // Appends a token to this CTA's run of the leader's list.
    __device__ __forceinline__ void append(float v, int idx) {
        const uint32_t at = atomicAdd(&s.n_local, 1u);
        if (at < uint32_t(CAP / C))
            st_peer64(map_peer(smem_addr(&s.list[rank * (CAP / C) + at]), 0),
                      (u64(key_of(v)) << 32) | uint32_t(~idx));
    }
    // After the appends and a block barrier: the CTA's count (and model mass) to the leader.
    __device__ void send_counts(u64 own) {
        if (threadIdx.x == 0) {
            st_peer32(map_peer(smem_addr(&s.list_n[rank]), 0), s.n_local);
            st_peer64(map_peer(smem_addr(&s.list_own[rank]), 0), own);
        }
    }
    // Leader: the runs in order, descending; false where a run overflowed.
    __device__ const u64* rank_list(int* n_out) {
        const int run = CAP / C;
        int n = 0;
        for (int r = 0; r < C; ++r) n += int(s.list_n[r]);
        *n_out = n;
        auto at = [&](int i) -> u64 {
            int r = 0;
            while (i >= int(s.list_n[r])) i -= int(s.list_n[r++]);
            return s.list[r * run + i];
        };
        if (n <= RANKED) {
            const u64 mine = int(threadIdx.x) < n ? at(threadIdx.x) : 0;
            if (int(threadIdx.x) < n) s.scratch[threadIdx.x] = mine;
            __syncthreads();
            if (int(threadIdx.x) < n) {
                int better = 0;
                for (int j = 0; j < n; ++j) better += s.scratch[j] > mine;
                s.sorted[better] = mine;
            }
            __syncthreads();
            return s.sorted;
        }
        u64 v[CAP / THREADS];
#pragma unroll
        for (int q = 0; q < CAP / THREADS; ++q) {
            const int i = q * THREADS + threadIdx.x;
            v[q] = i < n ? at(i) : 0;
        }
        __syncthreads();
        int m = 2 * RANKED;
        while (m < n) m <<= 1;
#pragma unroll
        for (int q = 0; q < CAP / THREADS; ++q) s.list[q * THREADS + threadIdx.x] = v[q];
        __syncthreads();
        for (int size = 2; size <= m; size <<= 1)
            for (int step = size >> 1; step; step >>= 1) {
                for (int i = threadIdx.x; i < m / 2; i += THREADS) {
                    const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
                    const u64 x = s.list[lo], y = s.list[hi];
                    if ((x < y) == ((lo & size) == 0)) s.list[lo] = y, s.list[hi] = x;
                }
                __syncthreads();
            }
        return s.list;
    }

    // -------------------------------------------------------- small top-k ----

    // Top-16 bits of the k-th largest thread maximum's key: at least k of the CTA's
    // tokens are at or above it.
    __device__ uint32_t bound_of(float mine, int k) const {
        const uint32_t key = key_of(mine);
        uint32_t at = 0;
        for (int b = 31; b >= 16; --b) {
            const uint32_t next = at | (1u << b);
            if (__syncthreads_count(key >= next) >= k) at = next;
        }
        return at;
    }

    // The tokens at or above `bound` to the leader, and the row finished there.  False (in
    // every CTA) where they are too many.
    __device__ bool few(uint32_t bound, int k, float p, float least, double u) {
        const float from = bound > KEY_NONE ? of_key(bound) : -CUDART_INF_F;
        if (threadIdx.x == 0) s.n_local = 0;
        __syncthreads();
        Model model;
        const bool want = a.logprobs != nullptr;
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint4 w = word(i);
            if (want || E::top(E::word_max(w)) >= from) {
                float v[EPW];
                E::unpack(w, v);
                if (want) add_model(model, v);
                if (E::top(E::word_max(w)) >= from)
                    for (int e = 0; e < EPW; ++e)
                        if (v[e] >= from && v[e] > -CUDART_INF_F) append(v[e], index(i, e));
            }
        }
        u64 own = want ? model_sum(model) : 0;
        if (lane == 0) s.ored[warp] = own;
        __syncthreads();
        own = 0;
        for (int i = 0; i < WARPS; ++i) own += s.ored[i];
        send_counts(own);
        const u64 count[1] = {s.n_local};
        const u64(*all)[4] = exchange(count);
        for (int r = 0; r < C; ++r)
            if (all[r][0] > u64(CAP / C)) return false;
        if (rank) return true;

        int n;
        const u64* sorted = rank_list(&n);
        k = min(k, n);
        const int t = threadIdx.x;
        const u64 mine = t < k ? sorted[t] : 0;
        const float v = of_key(uint32_t(mine >> 32));
        const int idx = int(~uint32_t(mine));
        const float e = t < k ? ex2f(exponent(v)) : 0.f;
        uint32_t w = t < k ? weight_of(e) : 0u;
        u64 W;
        const u64 before = block_scan(w, s.red, &W);
        if (p < 1.f && t > 0 && !(double(before) < double(p) * double(W))) w = 0;
        if (!(e >= least)) w = 0;
        // the kept masses by index
        block_scan((u64(w > 0) << 48) + w, s.seg, &W);
        const int kept = int(W >> 48);
        W &= (u64(1) << 48) - 1;
        if (t < k) s.scratch[t] = (u64(uint32_t(idx)) << 32) | w;
        __syncthreads();
        if (w) {
            u64 lower = 0;
            for (int j = 0; j < k; ++j) {
                const u64 o = s.scratch[j];
                if (int(o >> 32) < idx) lower += uint32_t(o);
            }
            const u64 at = target_of(u, W);
            if (at >= lower && at < lower + w) {
                u64 all_own = 0;
                for (int r = 0; r < C; ++r) all_own += s.list_own[r];
                answer(v, idx, W, all_own, kept);
            }
        }
        return true;
    }

    // ------------------------------------------------------------ the cut ----

    // The cut after the first tokens of the order, among those inside `within`, before which
    // the count is below k (by_mass = false) or the mass below p times theirs.  The histograms
    // hold the tokens with a mass alone: one without is never drawn.
    // Collective over the cluster.  Model mass is summed on the way where own is given.
    __device__ Cut resolve(bool by_mass, int64_t k, float p, const Cut& within, u64* own) {
        const float wv = of_key(within.key);
        const bool all = within.key == 0u;
        uint32_t* hi = reinterpret_cast<uint32_t*>(s.scratch);
        uint32_t* lo = hi + BINS;
        u64 before = 0;
        double target = 0.0;
        uint32_t bin = 0, k0 = 0, k1 = 0;  // after level 0: keys k0 <= key <= k1
        int shift = 0;
        bool ties = false;
        for (int level = 0;; ++level) {
            for (int i = threadIdx.x; i < BINS; i += THREADS) s.cnt[i] = 0, hi[i] = 0, lo[i] = 0;
            __syncthreads();
            Model model;
            for (int i = s0 + lane; i < s1; i += 32) {
                float v[EPW], sh[EPW];
                values(i, v);
#pragma unroll
                for (int e = 0; e < EPW; ++e) sh[e] = share(v[e]);
                if (level == 0 && own) {
                    if (c == a.K) model.add(sh);
                    else add_model(model, v);
                }
#pragma unroll
                for (int e = 0; e < EPW; ++e) {
                    const uint32_t w = weight_of(sh[e]);
                    if (!w || !(all || inside(v[e], index(i, e), within, wv))) continue;
                    uint32_t b;
                    if (level == 0) {
                        b = bin_of(v[e]);
                    } else {
                        const uint32_t key = key_of(v[e]);
                        if (key < k0 || key > k1) continue;
                        b = (k1 - key) >> shift;
                    }
                    atomicAdd(&s.cnt[b], 1u);
                    if (by_mass) {
                        atomicAdd(&hi[b], w >> 16);
                        atomicAdd(&lo[b], w & 0xffffu);
                    }
                }
            }
            if (level == 0 && own) *own = model_sum(model);
            cluster_barrier();
            // every CTA joins all histograms, two bins a thread
            u64 m[2] = {0, 0};
            uint32_t n[2] = {0, 0}, most[2] = {0, 0};
            for (int r = 0; r < C; ++r) {
                const uint32_t pc = map_peer(smem_addr(&s.cnt[2 * threadIdx.x]), r);
                const uint32_t ph = map_peer(smem_addr(&hi[2 * threadIdx.x]), r);
                const uint32_t pl = map_peer(smem_addr(&lo[2 * threadIdx.x]), r);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t x = ld_peer32(pc + 4 * q);
                    n[q] += x;
                    most[q] = max(most[q], x);
                    if (by_mass)
                        m[q] += (u64(ld_peer32(ph + 4 * q)) << 16) + ld_peer32(pl + 4 * q);
                }
            }
            if (!by_mass) m[0] = n[0], m[1] = n[1];
            u64 total;
            u64 at = before + block_scan(m[0] + m[1], s.red, &total);
            if (level == 0) target = by_mass ? double(p) * double(total) : double(k);
            if (threadIdx.x == 0) s.pick_bin = BINS;
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                // the first bin with a token that the target does not pass
                const bool starts = double(at) < target || (at == before && n[q] && before == 0);
                if (n[q] && starts && double(at + m[q]) >= target) {
                    s.pick_bin = 2 * threadIdx.x + q;
                    s.pick_n = n[q];
                    s.pick_most = most[q];
                    s.pick_before = at;
                }
                at += m[q];
            }
            __syncthreads();
            bin = s.pick_bin;
            if (bin == BINS) {  // the target is past all of them
                cluster_barrier();
                return within;
            }
            const uint32_t some = s.pick_most;
            before = s.pick_before;
            if (level == 0) {
                if (some <= uint32_t(CAP / C)) break;
                // the bin's range of keys
                uint32_t least = 0xffffffffu, largest = 0;
                for (int i = s0 + lane; i < s1; i += 32) {
                    float v[EPW];
                    values(i, v);
                    for (int e = 0; e < EPW; ++e) {
                        if (!weight_of(share(v[e])) || bin_of(v[e]) != bin ||
                            !(all || inside(v[e], index(i, e), within, wv)))
                            continue;
                        const uint32_t key = key_of(v[e]);
                        least = min(least, key), largest = max(largest, key);
                    }
                }
                least = __reduce_min_sync(FULL, least), largest = __reduce_max_sync(FULL, largest);
                if (lane == 0) s.red[warp] = (u64(~least) << 32) | largest;
                __syncthreads();
                for (int i = 0; i < WARPS; ++i)
                    least = min(least, ~uint32_t(s.red[i] >> 32)),
                    largest = max(largest, uint32_t(s.red[i]));
                const u64 mine[1] = {(u64(~least) << 32) | largest};
                const u64(*got)[4] = exchange(mine);
                for (int r = 0; r < C; ++r)
                    least = min(least, ~uint32_t(got[r][0] >> 32)),
                    largest = max(largest, uint32_t(got[r][0]));
                k0 = least, k1 = largest;
            } else {
                k1 = k1 - (bin << shift);
                const uint32_t span = (1u << shift) - 1;
                k0 = k1 - k0 > span ? k1 - span : k0;
                if (some <= uint32_t(CAP / C)) break;
                cluster_barrier();
            }
            if (k0 == k1) {
                ties = true;
                break;
            }
            shift = 0;
            while (((k1 - k0) >> shift) >= uint32_t(BINS)) ++shift;
        }
        const bool by_bin = k1 == 0;

        if (!ties) {
            if (threadIdx.x == 0) s.n_local = 0;
            __syncthreads();
            for (int i = s0 + lane; i < s1; i += 32) {
                float v[EPW];
                values(i, v);
#pragma unroll
                for (int e = 0; e < EPW; ++e) {
                    bool in;
                    if (by_bin) in = bin_of(v[e]) == bin;
                    else in = key_of(v[e]) >= k0 && key_of(v[e]) <= k1;
                    if (in && weight_of(share(v[e])) &&
                        (all || inside(v[e], index(i, e), within, wv)))
                        append(v[e], index(i, e));
                }
            }
            __syncthreads();
            send_counts(0);
            cluster_barrier();
            if (rank == 0) {
                int n;
                const u64* sorted = rank_list(&n);
                u64 w[CAP / THREADS], mine = 0;
                const int i0 = threadIdx.x * (CAP / THREADS);
#pragma unroll
                for (int q = 0; q < CAP / THREADS; ++q) {
                    w[q] = i0 + q < n ? (by_mass ? weight_of(share(of_key(uint32_t(sorted[i0 + q] >> 32)))) : 1u) : 0u;
                    mine += w[q];
                }
                u64 total;
                u64 at = before + block_scan(mine, s.red, &total);
                u64 stay = 0;
#pragma unroll
                for (int q = 0; q < CAP / THREADS; ++q) {
                    stay += i0 + q < n && (double(at) < target || (at == 0 && i0 + q == 0));
                    at += w[q];
                }
                block_scan(stay, s.red, &total);
                const u64 last = sorted[total - 1];
                if (warp == 0 && lane < C) {
                    st_peer32(map_peer(smem_addr(&s.cut_key), lane), uint32_t(last >> 32));
                    st_peer32(map_peer(smem_addr(&s.cut_idx), lane), ~uint32_t(last));
                }
            }
            cluster_barrier();
            return Cut{s.cut_key, s.cut_idx};
        }

        // all at one key: how many stay, and the index of the last of them
        u64 stay;
        if (by_mass) {
            const u64 w = weight_of(share(of_key(k0)));
            stay = 0;
            if (target > double(before)) {
                stay = u64((target - double(before)) / double(w));
                while (stay && double(before + (stay - 1) * w) >= target) --stay;
                while (double(before + stay * w) < target) ++stay;
            }
            if (!stay) stay = 1;
        } else {
            stay = u64(k) - before;
        }
        const float kv = of_key(k0);
        uint32_t mine = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            float v[EPW];
            values(i, v);
            for (int e = 0; e < EPW; ++e)
                mine += v[e] == kv && (all || inside(v[e], index(i, e), within, wv));
        }
        mine = __reduce_add_sync(FULL, mine);
        __syncthreads();
        if (lane == 0) s.seg[warp] = mine;
        __syncthreads();
        u64 lower = 0, count[1] = {0};
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) lower += s.seg[i];
            count[0] += s.seg[i];
        }
        const u64(*got)[4] = exchange(count);
        for (int r = 0; r < rank; ++r) lower += got[r][0];
        if (stay > lower && stay <= lower + mine) {
            for (int i = s0; i < s1; i += 32) {
                float v[EPW];
                uint32_t here = 0;
                if (i + lane < s1) {
                    values(i + lane, v);
                    for (int e = 0; e < EPW; ++e)
                        here += v[e] == kv && (all || inside(v[e], index(i + lane, e), within, wv));
                }
                const u64 inc = warp_scan(here, lane);
                if (stay > lower + inc - here && stay <= lower + inc) {
                    u64 at = lower + inc - here;
                    for (int e = 0; e < EPW; ++e) {
                        if (!(v[e] == kv && (all || inside(v[e], index(i + lane, e), within, wv))))
                            continue;
                        if (++at == stay)
                            for (int r = 0; r < C; ++r)
                                st_peer32(map_peer(smem_addr(&s.cut_idx), r),
                                          uint32_t(index(i + lane, e)));
                    }
                }
                lower += __shfl_sync(FULL, inc, 31);
            }
        }
        cluster_barrier();
        return Cut{k0, s.cut_idx};
    }

    // ----------------------------------------------------------- the draw ----

    // Mass of the logit as the cut and min-p leave it.
    template <bool CUTS>
    __device__ __forceinline__ uint32_t kept_mass(float v, float sh, int idx, const Cut& cut,
                                                  float kv, float least) const {
        uint32_t w = weight_of(sh);
        if constexpr (CUTS) {
            if (!(sh >= least && inside(v, idx, cut, kv))) w = 0;
        }
        return w;
    }

    // Masses by segment, the target's segment, the token.  OWN: the model's mass is summed on
    // the way (else own is the warp's already).
    template <bool CUTS>
    __device__ void draw(const Cut& cut, float least, double u, u64 own, bool sum_own) {
        const float kv = of_key(cut.key);
        const float kvc = cut.key ? kv : -CUDART_INF_F;
        u64 mass = 0;
        uint32_t kept = 0;
        Model model;
        const bool same = c == a.K;
        for (int i = s0 + lane; i < s1; i += 32) {
            float v[EPW], sh[EPW];
            values(i, v);
#pragma unroll
            for (int e = 0; e < EPW; ++e) sh[e] = share(v[e]);
            if (sum_own) {
                if (same) model.add(sh);
                else add_model(model, v);
            }
#pragma unroll
            for (int e = 0; e < EPW; e += 2) {
                const uint32_t wa = kept_mass<CUTS>(v[e], sh[e], index(i, e), cut, kvc, least);
                const uint32_t wb =
                    kept_mass<CUTS>(v[e + 1], sh[e + 1], index(i, e + 1), cut, kvc, least);
                mass += wa + wb;  // at most 2^31 and a little
                kept += (wa != 0) + (wb != 0);
            }
        }
        mass = warp_add(mass);
        kept = __reduce_add_sync(FULL, kept);
        if (sum_own) own = model_sum(model);
        __syncthreads();
        if (lane == 0) s.seg[warp] = mass, s.red[warp] = kept, s.ored[warp] = own;
        __syncthreads();
        u64 lower = 0, cta[3] = {0, 0, 0};
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) lower += s.seg[i];
            cta[0] += s.seg[i], cta[1] += s.red[i], cta[2] += s.ored[i];
        }
        const u64(*got)[4] = exchange(cta);
        u64 W = 0, all_own = 0;
        int all_kept = 0;
        for (int r = 0; r < C; ++r) {
            if (r < rank) lower += got[r][0];
            W += got[r][0], all_kept += int(got[r][1]);
            all_own += got[r][2];
        }
        const u64 t = target_of(u, W);
        if (t < lower || t >= lower + mass) return;
        for (int i = s0; i < s1; i += 32) {
            float v[EPW];
            uint32_t w[EPW];
            u64 here = 0;
            if (i + lane < s1) {
                values(i + lane, v);
#pragma unroll
                for (int e = 0; e < EPW; ++e) {
                    w[e] = kept_mass<CUTS>(v[e], share(v[e]), index(i + lane, e), cut, kvc, least);
                    here += w[e];
                }
            }
            const u64 inc = warp_scan(here, lane);
            const u64 from = lower + inc - here;
            if (t >= from && t < from + here) {
                u64 at = from;
#pragma unroll
                for (int e = 0; e < EPW; ++e) {
                    if (t >= at && t < at + w[e]) answer(v[e], index(i + lane, e), W, all_own, all_kept);
                    at += w[e];
                }
            }
            lower += __shfl_sync(FULL, inc, 31);
            if (t < lower) return;
        }
    }
};

template <typename DT, bool CAPPED, bool RES>
__global__ void __launch_bounds__(THREADS, 2) sample_kernel(const __grid_constant__ Args a) {
    __shared__ Shared s;
    extern __shared__ __align__(16) uint4 words[];
    using R = Row<DT, CAPPED, RES>;
    constexpr int EPW = R::EPW;
    R r(a, s);
    cluster_arrive();  // before the first write to a peer: every CTA has started
    uint32_t C;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
    r.C = int(C);
    r.rank = int(cluster_ctarank());
    r.lane = threadIdx.x & 31, r.warp = threadIdx.x >> 5;
    r.row = a.row0 + blockIdx.x / C;
    r.words = words;
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.logits) + uint64_t(r.row * a.ld) * sizeof(DT);
    r.gwords = reinterpret_cast<const uint4*>(base & ~uintptr_t(15));
    r.head = int((base & 15) / sizeof(DT));
    r.nw = (r.head + a.V + EPW - 1) / EPW;
    const int per = (r.nw + r.C - 1) / r.C;
    r.w0 = min(r.nw, r.rank * per);
    const int mine = min(r.nw, r.w0 + per) - r.w0, seg = (mine + WARPS - 1) / WARPS;
    r.s0 = min(mine, r.warp * seg), r.s1 = min(mine, r.s0 + seg);
    const int lane = r.lane, warp = r.warp;

    // the warp's words: whole ones by a bulk copy, those that reach outside the row by element
    bool lost = false;
    if constexpr (RES) {
        const int f0 = r.w0 == 0 && r.s0 == 0 && r.head ? 1 : r.s0;  // first whole word
        const bool ragged = (r.head + a.V) % EPW != 0;
        const int f1 = ragged && r.w0 + r.s1 == r.nw && r.s1 > r.s0 ? r.s1 - 1 : r.s1;
        const uint32_t bar = smem_addr(&s.bar[warp]);
        if (lane == 0) {
            hl::mbar_init(bar, 1);
            hl::fence_mbar_init();
            hl::fence_proxy_async();
            if (f1 > f0) {
                hl::mbar_arrive_expect_tx(bar, uint32_t(f1 - f0) * 16);
                bulk_g2s(smem_addr(words + f0), r.gwords + r.w0 + f0, uint32_t(f1 - f0) * 16, bar);
            }
        }
        __syncwarp();
        if (lane == 1 && r.s0 < r.s1 && f0 > r.s0) words[r.s0] = r.global_word(r.w0 + r.s0);
        if (lane == 2 && f1 < r.s1 && f1 >= f0) words[f1] = r.global_word(r.w0 + f1);
        if (f1 > f0 && !hl::mbar_wait_bounded(bar, 0, WAIT_NS)) {
            lost = true;
            hl::mbar_wait_bounded(bar, 0, WAIT_NS);  // so that the copy does not land later
        }
        __syncwarp();
    }

    // settings, the largest logit
    const float temp = a.temperature ? a.temperature[r.row] : 1.f;
    const double u = a.uniforms[r.row];
    const int want_k = a.top_k ? a.top_k[r.row] : 0;
    const float p = a.top_p ? a.top_p[r.row] : 1.f;
    const float least = a.min_p ? a.min_p[r.row] : 0.f;
    const bool bad = !(temp >= 0.f && temp < CUDART_INF_F) || !(u >= 0.0 && u < 1.0) ||
                     !(p >= 0.f) || !(least >= 0.f && least <= 1.f);
    r.c = __fdiv_rn(a.K, temp);
    const bool greedy = !(r.c < CUDART_INF_F);
    if (greedy) r.c = a.K;
    const int k = greedy ? 1 : want_k <= 0 || want_k > a.V ? a.V : want_k;
    const bool small_k = k < a.V && k <= MAX_TOPK;

    uint32_t m2 = R::E::LOWEST;
    for (int i = r.s0 + lane; i < r.s1; i += 32) m2 = R::E::max2(m2, R::E::word_max(r.word(i)));
    const float mine_top = R::E::top(m2);
    float top = mine_top;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
    if (lane == 0) s.fred[warp] = top;
    const bool any_lost = __syncthreads_or(lost);
    for (int i = 0; i < WARPS; ++i) top = fmaxf(top, s.fred[i]);
    uint32_t bound = 0;
    if (small_k && !bad) bound = k == 1 ? key_of(top) : r.bound_of(mine_top, k);
    cluster_wait();
    const u64 own_max[2] = {(u64(any_lost) << 32) | key_of(top), bound};
    const u64(*got)[4] = r.exchange(own_max);
    uint32_t topkey = 0;
    bool given_up = false;
    for (int i = 0; i < r.C; ++i) {
        topkey = max(topkey, uint32_t(got[i][0]));
        bound = max(bound, uint32_t(got[i][1]));
        given_up |= (got[i][0] >> 32) != 0;
    }
    r.top = of_key(topkey);
    if (bad || given_up || topkey == KEY_NONE) {
        if (r.rank == 0 && threadIdx.x == 0) {
            r.no_token();
            if (bad || given_up) atomicOr(a.err, bad ? 1 : 2);
        }
        return;
    }
    r.zm = r.z(r.top);

    if (small_k && r.few(bound, k, p, least, u)) return;

    // +inf without a softcap: the tokens at +inf share the mass alike, all others have none
    if (!CAPPED && r.top == CUDART_INF_F) {
        if constexpr (RES) {
            DT* x = reinterpret_cast<DT*>(words);
            for (int i = r.s0 + lane; i < r.s1; i += 32)
                for (int e = 0; e < EPW; ++e) {
                    const float v = R::E::load(x, i * EPW + e);
                    x[i * EPW + e] = DT(v == CUDART_INF_F ? 0.f : -CUDART_INF_F);
                }
            __syncwarp();
        }
        r.inf_row = true;
        r.top = r.zm = 0.f;
    }
    const bool want = a.logprobs != nullptr;
    u64 own = 0;
    bool have = !want;
    Cut cut = NO_CUT;
    if (k < a.V) cut = r.resolve(false, k, 1.f, cut, have ? nullptr : &own), have = true;
    if (p < 1.f) cut = r.resolve(true, 0, p, cut, have ? nullptr : &own), have = true;
    if (cut.key == 0u && least == 0.f) r.template draw<false>(cut, 0.f, u, own, !have);
    else r.template draw<true>(cut, least, u, own, !have);
}

// -------------------------------------------------------------------- launch ----

// Shared memory of a CTA's words at most: two CTAs an SM beside the fixed part.
constexpr int SLICE = 72 * 1024;
constexpr int SLICE_MOST = 160 * 1024;

template <typename DT, bool CAPPED>
int launch(Args a, int64_t N, int device, int sms, cudaStream_t st) {
    const int64_t words = (int64_t(a.V) * sizeof(DT) + 30) / 16;  // at most, wherever rows start
    auto slice = [&](int c) { return (words + c - 1) / c * 16; };
    int C = 1;
    while (C < MAXC && slice(C) > SLICE) ++C;
    // few rows: more CTAs a row, while each warp has a few words a lane
    while (C < MAXC && N * (C + 1) <= sms && slice(C) > 16 * 1024) ++C;
    const bool resident = slice(C) <= SLICE_MOST;
    const void* kernel = resident ? reinterpret_cast<const void*>(&sample_kernel<DT, CAPPED, true>)
                                  : reinterpret_cast<const void*>(&sample_kernel<DT, CAPPED, false>);
    const int smem = resident ? int(slice(C)) : 0;
    if (resident) {
        static std::atomic<uint64_t> done{0};  // devices whose limit is raised
        const uint64_t bit = uint64_t(1) << (device & 63);
        if (!(done.load() & bit) || device > 63) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     SLICE_MOST) != cudaSuccess) {
                cudaGetLastError();
                return HEADLOSS_ERR_CUDA;
            }
            done.fetch_or(bit);
        }
    }
    constexpr int64_t ROWS = int64_t(1) << 27;  // a launch's rows at most
    for (int64_t at = 0; at < N; at += ROWS) {
        a.row0 = at;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned((N - at < ROWS ? N - at : ROWS) * C));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = size_t(smem);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {unsigned(C), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        void* args[] = {&a};
        if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
            cudaGetLastError();
            return HEADLOSS_ERR_CUDA;
        }
    }
    return HEADLOSS_OK;
}

int launch_fp32(const Args& a, int64_t N, int device, int sms, cudaStream_t st);
int launch_bf16(const Args& a, int64_t N, int device, int sms, cudaStream_t st);
int launch_fp16(const Args& a, int64_t N, int device, int sms, cudaStream_t st);

}  // namespace hl_sample
