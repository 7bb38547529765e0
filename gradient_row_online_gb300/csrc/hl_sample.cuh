// hl_sample.cuh -- the sampling kernel (headloss_sample in
// include/headloss_sample.h, where the definition stands).
//
// One thread-block cluster a row, each CTA a contiguous run of the row's 16-byte
// words in its shared memory, each warp a contiguous segment of that, copied by
// the warp's own cp.async.bulk.  A logit is read from HBM once; every pass is over
// shared memory.  (Rows too long for eight CTAs' shared memory are read from
// global memory in every pass: RES = false.)
//
// All three filters keep a prefix of the order (x descending, index ascending), so a
// row's kept set is a cut in that order, and min-p's comparison.  Masses are integers
// (2^30 the largest logit's): exact sums in any order, so atomics, splits and cluster
// sizes never change a token.  After the exchange of the largest logit a row goes one of
// these ways, each ending in the leader CTA while the others have left:
//
//   no top-k, no top-p   every warp sums its segment's masses.
//   a small top-k        histograms of the CTAs' thread maxima bound the cut from below (as many
//                        tokens as maxima lie above it; the bounds go along with the largest
//                        logit); the few tokens above the bound are ranked by the leader,
//                        which finishes the row alone.
//   top-p                a histogram of the order (1/32 octave of mass a bin) with exact masses
//                        finds the bin of the cut; the next pass sums the segments' masses in the
//                        bins above it and sends the bin's few tokens to be ranked.
//   else                 `resolve`: the same by count or mass within another cut, where a bin with
//                        too many tokens (ties, dense rows) is cut into bins of keys again.
//
// The leader then knows the segment that holds the drawn target and goes over it once more
// (from L2) for the token.
//
// What bounds it: barriers and the leader's last step, two to four a row, each a microsecond
// or two, at 56-62% of the issue slots; every logit comes from HBM once.  Measured (logits' bytes
// over the time): 1024 x 151936 bf16 unfiltered 118 us, 2.6 TB/s; 1024 x 128256 top-p 248 us,
// 1.1 TB/s; 8192 x 32000 top-k and top-p 264 us, 2.0 TB/s; 512 x 128256 fp16 capped 86 us, 1.5 TB/s;
// one row of 32000 8.3 us.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "headloss.h"
#include "hl_pack.cuh"
#include "hl_rows.cuh"
#include "hl_tanh_poly.h"

namespace hl_sample {

using hl::bulk_g2s;
using hl::cluster_ctarank;
using hl::map_peer;
using hl::smem_addr;

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int MAXC = 8;       // CTAs a cluster at most
constexpr int BINS = 4 * THREADS;
constexpr int CAP = 832;      // tokens the leader can rank
constexpr int RANKED = 256;   // ranked by comparison with all; more are sorted
constexpr int MAX_TOPK = 128; // longest top-k that takes the thread-maxima bound
constexpr int SEGS = MAXC * WARPS;
constexpr int QUEUE = 512;
constexpr float PER_OCTAVE = 32.f;  // bins an octave of mass
constexpr int TOPS = 128;           // bins of the thread maxima,
constexpr float TOPS_PER_OCTAVE = 4.f;
constexpr int SPLIT = 15;  // a mass is added as its bits above and below this one: either sum
                           // stays below 2^32 for up to 2^17 tokens a CTA
constexpr float UNIT = 1073741824.f;  // 2^30, the weight of the largest logit
constexpr float LN2 = 0.69314718055994531f;
constexpr unsigned FULL = 0xffffffffu;
constexpr unsigned long long WAIT_NS = 2000000000ull;

struct Args {
    const void* logits;
    int64_t ld;
    int64_t row0;  // first row of this launch
    int per;       // 16-byte words a CTA
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
#ifdef HL_FAULT_INJECT
    int64_t drop_row;  // its copies are left out (-1: none)
    unsigned long long wait_ns;
#endif
};

typedef unsigned long long u64;

struct Shared {
    u64 bar[WARPS];
    union {  // (aligned: cnt, and hi, lo, tops and rank below, are also read 16 bytes at a time)
        alignas(16) u64 list[CAP];  // (key << 32 | ~index) of the tokens to rank, a run a CTA (leader)
        uint32_t cnt[BINS];  // histogram of counts
    };
    union {
        u64 groups[MAXC][32];  // the CTAs' histograms by groups of 32 bins
        int queue[QUEUE];      // words with tokens to list
    };
    union {
        struct {
            alignas(16) uint32_t hi[BINS];  // histogram of masses, above and below bit SPLIT
            uint32_t lo[BINS];
        };
        uint32_t tops[TOPS];  // histogram of the thread maxima
        u64 rank[BINS];       // where lists are ranked
    };
    u64 xch[2][MAXC][2];   // exchanges of two values a CTA
    u64 seg_mass[SEGS];    // the segments' kept masses, the model's, and counts (leader)
    u64 seg_model[SEGS];
    uint32_t seg_kept[SEGS];
    u64 my_mass[WARPS];    // the CTA's own segments
    u64 my_model[WARPS];
    uint32_t my_kept[WARPS];
    double target;
    uint32_t list_n[MAXC];
    u64 red[WARPS];
    uint32_t ired[WARPS];
    uint32_t n_local, queued;
    uint32_t pick_bin, pick_most;
    u64 pick_before;
    uint32_t cut_key;
    int cut_idx;
    u64 fin[3];
    uint32_t fin_seg;
};
static_assert(alignof(Shared) >= 16 && offsetof(Shared, list) % 16 == 0 && offsetof(Shared, hi) % 16 == 0,
              "words of 16 bytes");

// A cut of the order: tokens above the key stay, and at the key those up to an index.
struct Cut {
    uint32_t key;
    int idx;
};

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

// Arrival of a warp that wrote nothing another CTA reads (no fence).
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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
    static constexpr int PAIRS = EPW / 2;

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
    float zt;            // the largest logit's z in the model's log-prob (CAPPED)

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
    // Of a row whose largest logit is +inf (no softcap): the tokens at +inf share the mass
    // alike, all others have none.
    __device__ __forceinline__ void unpack(const uint4& w, float* v, bool mapped) const {
        E::unpack(w, v);
        if (mapped && inf_row)
            for (int e = 0; e < EPW; ++e) v[e] = v[e] == CUDART_INF_F ? 0.f : -CUDART_INF_F;
    }
    __device__ __forceinline__ void values(int i, float* v) const { unpack(word(i), v, !RES); }

    __device__ __forceinline__ float z(float v) const {
        if constexpr (CAPPED) return __fmul_rn(tanhf(__fmul_rn(v, a.inv_cap)), a.cap);
        else return v;
    }
    // Exponents of a word's logits, and their mass shares; -inf and NaN have none.  A NaN's share
    // is NaN without a softcap, which makes the weight 0.
    __device__ __forceinline__ void shares(const float* v, hl::f2* d, float* sh) const {
        const hl::f2 nz = hl::pk1(-zm), cc = hl::pk1(c);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            d[i] = hl::mul2(hl::add2(hl::pk(z(v[2 * i]), z(v[2 * i + 1])), nz), cc);
            float x, y;
            hl::upk(d[i], x, y);
            sh[2 * i] = ex2f(x), sh[2 * i + 1] = ex2f(y);
            if constexpr (CAPPED) {
                if (!(v[2 * i] > -CUDART_INF_F)) sh[2 * i] = 0.f;
                if (!(v[2 * i + 1] > -CUDART_INF_F)) sh[2 * i + 1] = 0.f;
            }
        }
    }
    __device__ __forceinline__ void weights(const float* sh, uint32_t* w) const {
        const hl::f2 unit = hl::pk1(UNIT);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float x, y;
            hl::upk(hl::mul2(hl::pk(sh[2 * i], sh[2 * i + 1]), unit), x, y);
            w[2 * i] = __float2uint_rn(x), w[2 * i + 1] = __float2uint_rn(y);
        }
    }
    __device__ __forceinline__ float share(float v) const {
        const float e = ex2f(__fmul_rn(__fsub_rn(z(v), zm), c));
        if constexpr (CAPPED) return v > -CUDART_INF_F ? e : 0.f;
        else return e;
    }
    // The exponent where +inf may stand.
    __device__ __forceinline__ float exponent(float v) const {
        const float zz = z(v);
        return zz == zm ? 0.f : __fmul_rn(__fsub_rn(zz, zm), c);
    }

    // Mass of the whole softmax at T = 1: a word's shares summed in fp32 in one order, the words
    // in fixed point, so that it too is the same however the row is split.  A word's sum t < 16 is
    // taken apart by adding and subtracting 1.5 * 2^23 units: H units of 2^-13, and the
    // exact remainder in units of 2^-36; the integers are the low bits of the sums.
    struct Model {
        std::conditional_t<RES, int, int64_t> high = 0, low = 0;
        bool odd = false;  // a word with a NaN (or +inf)
        __device__ __forceinline__ void add(const float* sh) {
            constexpr float HIGH = 12582912.f * 0x1p-13f, LOW = 12582912.f;
            float t;
            if constexpr (EPW == 8)
                t = ((sh[0] + sh[1]) + (sh[2] + sh[3])) + ((sh[4] + sh[5]) + (sh[6] + sh[7]));
            else t = (sh[0] + sh[1]) + (sh[2] + sh[3]);
            odd |= !(t < 15.f);
            const float h = __fadd_rn(t, HIGH);
            const float l = __fmaf_rn(__fsub_rn(t, __fsub_rn(h, HIGH)), 0x1p+36f, LOW);
            high += __float_as_int(h) - 0x44c00000;
            low += __float_as_int(l) - 0x4b400000;
        }
        // in units of 2^-36
        __device__ __forceinline__ u64 sum() const {
            return u64(int64_t(high) * (1 << 23) + int64_t(low));
        }
    };
    // z of the model's log-prob: with a softcap by the loss's degree-5 fit of tanh (5.8e-8
    // relative on |x / c| <= 0.8) where a logit allows it, two logits an instruction; the
    // library's tanhf, which the draw's integer weights take, would be most of the pass
    // (38 instructions a token instead of 26 on capped rows).  Fit and tanhf differ by up to 8e-6 at
    // c = 50, so which of them a logit takes depends on that logit alone, in the sum, for the
    // largest and for the drawn token: a row's one dominant token has log p = 0.
    __device__ __forceinline__ hl::f2 fit_z(hl::f2 x) const {
        const hl::f2 y = hl::mul2(x, hl::pk1(a.inv_cap)), y2 = hl::mul2(y, y);
        hl::f2 p = hl::fma2(hl::pk1(HL_TANH_B_C5), y2, hl::pk1(HL_TANH_B_C4));
        p = hl::fma2(p, y2, hl::pk1(HL_TANH_B_C3));
        p = hl::fma2(p, y2, hl::pk1(HL_TANH_B_C2));
        p = hl::fma2(p, y2, hl::pk1(HL_TANH_B_C1));
        p = hl::fma2(p, y2, hl::pk1(HL_TANH_B_C0));
        return hl::mul2(x, p);  // c tanh(x / c) = x P((x / c)^2)
    }
    __device__ __forceinline__ bool fits(float v) const {  // (a NaN, which has no mass, either way)
        return __fmul_rn(fabsf(v), a.inv_cap) <= HL_TANH_B_Y0;
    }
    __device__ __forceinline__ float model_z(float v) const {
        if constexpr (CAPPED) return fits(v) ? hl::lo_of(fit_z(hl::pk1(v))) : z(v);
        else return v;
    }
    __device__ __forceinline__ float model_top() const {
        if constexpr (CAPPED) return zt;
        else return zm;
    }
    __device__ __forceinline__ void model_z(const float* v, hl::f2* zz) const {
        if constexpr (CAPPED) {
            float far = 0.f;
#pragma unroll
            for (int e = 0; e < EPW; ++e) far = fmaxf(far, fabsf(v[e]));
            if (fits(far)) {
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) zz[i] = fit_z(hl::pk(v[2 * i], v[2 * i + 1]));
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) zz[i] = hl::pk(model_z(v[2 * i]), model_z(v[2 * i + 1]));
    }
    __device__ __forceinline__ void add_model(Model& m, const float* v) const {
        const hl::f2 nz = hl::pk1(-model_top()), kk = hl::pk1(a.K);
        float sh[EPW];
        hl::f2 zz[PAIRS];
        model_z(v, zz);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float x, y;
            hl::upk(hl::mul2(hl::add2(zz[i], nz), kk), x, y);
            sh[2 * i] = ex2f(x), sh[2 * i + 1] = ex2f(y);
            if constexpr (CAPPED) {
                if (!(v[2 * i] > -CUDART_INF_F)) sh[2 * i] = 0.f;
                if (!(v[2 * i + 1] > -CUDART_INF_F)) sh[2 * i + 1] = 0.f;
            }
        }
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
                    const float zz = model_z(v[e]), zt = model_top();
                    v[e] = !(v[e] > -CUDART_INF_F) ? 0.f
                           : zz == zt              ? 1.f
                                      : ex2f(__fmul_rn(__fsub_rn(zz, zt), a.K));
                }
                m.add(v);
            }
        }
        // (a segment of the longest row holds 2^25 tokens, their sum 2^61 units; 64 segments of
        // rows that are not resident are added in units of 2^-32, up to 2^63)
        const u64 sum = warp_add(m.sum());
        return RES ? sum : (sum + 8) >> 4;
    }

    // Bin of the order: 1/32 octave of mass a bin without a softcap (with one, of the raw
    // logit's distance); the last takes what is further off.
    __device__ __forceinline__ uint32_t bin_of(float v) const {
        return min(uint32_t(BINS - 1),
                   __float2uint_rn(__fmul_rn(__fmul_rn(__fsub_rn(top, v), c), PER_OCTAVE)));
    }
    // Below every logit of a bin (of `per` an octave): distances lie below (bin + 1/2) / (per c),
    // and a little more for the roundings.  -inf where c is so small that a bin has no end (c = 0:
    // all logits are in bin 0, whatever the largest is).
    __device__ float lower_edge(float top, float bin, float per) const {
        const float far = __fmul_ru(__fdiv_ru(bin + 0.5f, __fmul_rd(c, per)), 1.00001f);
        return far < CUDART_INF_F ? __fsub_rd(top, far) : -CUDART_INF_F;
    }
    __device__ __forceinline__ bool inside(float v, int idx, const Cut& k, float kv) const {
        return v > kv || (v == kv && idx <= k.idx);
    }

    // Every CTA's two values (of warp 0's lanes, all alike) at every CTA.  ALONE: the other
    // warps wrote nothing that another CTA reads after it.
    template <bool ALONE>
    __device__ const u64 (*exchange(u64 v0, u64 v1 = 0))[2] {
        __syncwarp();
        if (warp == 0) {
            if (lane < C) {
                const uint32_t at = map_peer(smem_addr(&s.xch[par][rank][0]), lane);
                st_peer64(at, v0);
                st_peer64(at + 8, v1);
            }
            __syncwarp();
            cluster_arrive();
        } else if constexpr (ALONE) {
            cluster_arrive_relaxed();
        } else {
            cluster_arrive();
        }
        cluster_wait();
        const u64(*got)[2] = s.xch[par];
        par ^= 1;
        return got;
    }

    __device__ void no_token() const {
        a.tokens[row] = -1;
        if (a.logprobs) a.logprobs[row] = 0.f;
        if (a.draw_logprobs) a.draw_logprobs[row] = 0.f;
        if (a.n_kept) a.n_kept[row] = 0;
    }
    __device__ void answer(float v, int idx, u64 W, u64 model, int kept) const {
        a.tokens[row] = idx;
        const float zz = model_z(v), zt = model_top();
        if (a.logprobs)
            a.logprobs[row] = (zz == zt ? 0.f : __fsub_rn(zz, zt) * a.K * LN2) -
                              logf(float(model) * (RES ? 0x1p-36f : 0x1p-32f));
        if (a.draw_logprobs)
            a.draw_logprobs[row] = exponent(v) * LN2 - logf(float(W) * 0x1p-30f);
        if (a.n_kept) a.n_kept[row] = kept;
    }
    __device__ static u64 target_of(double u, u64 W) {
        const u64 t = u64(u * double(W));
        return t < W ? t : W - 1;
    }

    // ------------------------------------------------------ lists to rank ----

    // Words with tokens to list are queued as a pass finds them (their lanes would hold up the
    // others), and gone through a thread a word after a block barrier.
    __device__ __forceinline__ void enqueue(int i) {
        const uint32_t n = atomicAdd(&s.queued, 1u);
        if (n < QUEUE) s.queue[n] = i;
    }
    // How many are queued; with too many the CTA's count shows an overflow.
    __device__ uint32_t queued() {
        const uint32_t n = s.queued;
        if (n > QUEUE && threadIdx.x == 0) s.n_local = CAP + 1;
        return n > QUEUE ? 0u : n;
    }
    // Appends tokens of a word (the bits of `which`) to this CTA's run of the leader's list.
    __device__ __forceinline__ void append(const float* v, uint32_t which, int i) {
        if (!which) return;
        uint32_t at = atomicAdd(&s.n_local, uint32_t(__popc(which)));
        const uint32_t run = uint32_t(CAP / C), to = map_peer(smem_addr(&s.list[rank * run]), 0);
#pragma unroll
        for (int e = 0; e < EPW; ++e) {
            if (!(which >> e & 1)) continue;
            if (at < run) st_peer64(to + 8 * at, (u64(key_of(v[e])) << 32) | uint32_t(~index(i, e)));
            ++at;
        }
    }
    // After the appends and a block barrier: the CTA's count to the leader.
    __device__ void send_count() {
        if (threadIdx.x == 0) st_peer32(map_peer(smem_addr(&s.list_n[rank]), 0), s.n_local);
    }
    // Leader: how many tokens are listed, and the i-th over the runs.
    __device__ int count_listed() const {
        int n = 0;
        for (int r = 0; r < C; ++r) n += int(s.list_n[r]);
        return n;
    }
    __device__ u64 listed(int i) const {
        int r = 0;
        while (i >= int(s.list_n[r])) i -= int(s.list_n[r++]);
        return s.list[r * (CAP / C) + i];
    }
    // Leader: the runs put together, descending.
    __device__ const u64* rank_list(int* n_out) {
        const int n = count_listed();
        *n_out = n;
        auto at = [&](int i) -> u64 { return listed(i); };
        if (n <= RANKED) {
            // by comparison with all; up to half as many, two threads a token, each with half of the others
            u64* sorted = s.rank + RANKED;
            uint32_t* part = reinterpret_cast<uint32_t*>(sorted + RANKED);
            const bool halves = n <= RANKED / 2;
            const int i = halves ? threadIdx.x & (RANKED / 2 - 1) : threadIdx.x;
            const u64 mine = i < n ? at(i) : 0;
            if (i < n) s.rank[i] = mine;
            if (threadIdx.x == 0 && (n & 1)) s.rank[n] = 0;
            __syncthreads();
            const int pairs = (n + 1) / 2, mid = halves ? (pairs + 1) / 2 : pairs;
            const bool second = halves && threadIdx.x >= RANKED / 2;
            int better = 0;
            if (i < n) {
                const ulonglong2* two = reinterpret_cast<const ulonglong2*>(s.rank);
#pragma unroll 4
                for (int j = second ? mid : 0; j < (second ? pairs : mid); ++j) {
                    const ulonglong2 o = two[j];
                    better += (o.x > mine) + (o.y > mine);
                }
                if (second) part[i] = uint32_t(better);
            }
            if (halves) __syncthreads();
            if (i < n && !second) sorted[better + (halves ? int(part[i]) : 0)] = mine;
            __syncthreads();
            return sorted;
        }
        static_assert(CAP <= BINS, "a list fits the histograms' place");
        int m = 2 * RANKED;
        while (m < n) m <<= 1;
        for (int i = threadIdx.x; i < m; i += THREADS) s.rank[i] = i < n ? at(i) : 0;
        __syncthreads();
        for (int size = 2; size <= m; size <<= 1)
            for (int step = size >> 1; step; step >>= 1) {
                for (int i = threadIdx.x; i < m / 2; i += THREADS) {
                    const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
                    const u64 x = s.rank[lo], y = s.rank[hi];
                    if ((x < y) == ((lo & size) == 0)) s.rank[lo] = y, s.rank[hi] = x;
                }
                __syncthreads();
            }
        return s.rank;
    }

    // A bin's mass from its two sums.
    __device__ __forceinline__ static u64 joined(uint32_t hi, uint32_t lo) {
        return (u64(hi) << (RES ? SPLIT : 32)) + lo;
    }
    // The bin of the cluster's histograms that the target (a count k, or p times the total, formed
    // where `first`) falls in: s.pick_bin (BINS where the target is past them all), what lies
    // before it over `before`, and the largest count of a CTA in it (COUNTS: where the
    // counts were taken).  Every CTA tells the others its sums over groups of 32 bins and then
    // reads the bins of one group from them: the histograms themselves would be
    // twice the slice's bytes.  Collective; the peers' bins are read until the next barrier.
    template <bool MASS, bool COUNTS>
    __device__ void locate(double p, bool first, u64 before) {
        __syncthreads();
        const int t = threadIdx.x;
        u64 sum;
        if constexpr (MASS) {
            const uint4 x = reinterpret_cast<const uint4*>(s.hi)[t], y = reinterpret_cast<const uint4*>(s.lo)[t];
            sum = joined(x.x, y.x) + joined(x.y, y.y) + joined(x.z, y.z) + joined(x.w, y.w);
        } else {
            const uint4 x = reinterpret_cast<const uint4*>(s.cnt)[t];
            sum = u64(x.x) + x.y + x.z + x.w;
        }
        static_assert(BINS == 4 * THREADS && BINS == 32 * 32 && MAXC == 8, "eight threads a group");
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(FULL, sum, o);
        if ((lane & 7) < C) st_peer64(map_peer(smem_addr(&s.groups[rank][t >> 3]), lane & 7), sum);
        cluster_barrier();
        if (warp == 0) {
            u64 g = 0;
            for (int r = 0; r < C; ++r) g += s.groups[r][lane];
            u64 inc = warp_scan(g, lane);
            const double target = !first ? s.target : MASS ? p * double(__shfl_sync(FULL, inc, 31)) : p;
            if (lane == 0) s.pick_bin = BINS, s.target = target;
            // a target of 0 keeps the first token all the same
            auto holds = [&](u64 at, u64 m) {
                return m && (double(at) < target || at == 0) && double(at + m) >= target;
            };
            u64 at = before + inc - g;
            const unsigned hit = __ballot_sync(FULL, holds(at, g));
            if (hit) {
                const int group = __ffs(hit) - 1, bin = group * 32 + lane;
                at = __shfl_sync(FULL, at, group);
                uint32_t n[MAXC], hi[MAXC], lo[MAXC];  // all peers' at once
#pragma unroll
                for (int r = 0; r < MAXC; ++r) {
                    n[r] = hi[r] = lo[r] = 0;
                    if (r < C) {
                        if constexpr (!MASS || COUNTS) n[r] = ld_peer32(map_peer(smem_addr(&s.cnt[bin]), r));
                        if constexpr (MASS) {
                            hi[r] = ld_peer32(map_peer(smem_addr(&s.hi[bin]), r));
                            lo[r] = ld_peer32(map_peer(smem_addr(&s.lo[bin]), r));
                        }
                    }
                }
                u64 m = 0;
                uint32_t most = 0;
#pragma unroll
                for (int r = 0; r < MAXC; ++r) {
                    most = max(most, n[r]);
                    m += MASS ? joined(hi[r], lo[r]) : u64(n[r]);
                }
                inc = warp_scan(m, lane);
                at += inc - m;
                if (holds(at, m)) s.pick_bin = uint32_t(bin), s.pick_most = most, s.pick_before = at;
            }
        }
        __syncthreads();
    }

    // -------------------------------------------------------- small top-k ----

    // Bounds from below of the k-th and of the ceil(k / C)-th largest logit of the CTA, as keys: the
    // lower edges of the bins where the histogram of its thread maxima (from its own
    // largest) reaches so many.  At least k tokens lie at or above the largest of the first over the CTAs,
    // and at or above the least of the second.  In warp 0.
    __device__ u64 bounds_of(float mine, float cta_top, int k) {
        if (mine > -CUDART_INF_F)
            atomicAdd(&s.tops[min(uint32_t(TOPS - 1), __float2uint_rn(__fmul_rn(
                                                          __fmul_rn(__fsub_rn(cta_top, mine), c),
                                                          TOPS_PER_OCTAVE)))],
                      1u);
        __syncthreads();
        if (warp) return 0;
        static_assert(TOPS == 128, "four bins a lane");
        const uint4 n = reinterpret_cast<const uint4*>(s.tops)[lane];
        const uint32_t sum = n.x + n.y + n.z + n.w;
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t m = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += m;
        }
        auto bound = [&](uint32_t want) -> uint32_t {
            const unsigned past = __ballot_sync(FULL, inc >= want);
            if (!past) return KEY_NONE;
            const int at = __ffs(past) - 1;
            uint32_t have = inc - sum + n.x;  // (only lane `at`'s is used)
            int bin = 4 * lane;
            if (have < want) ++bin, have += n.y;
            if (have < want) ++bin, have += n.z;
            if (have < want) ++bin;
            bin = __shfl_sync(FULL, bin, at);
            const float edge = lower_edge(cta_top, float(bin), TOPS_PER_OCTAVE);
            return bin < TOPS - 1 ? key_of(edge) : KEY_NONE;
        };
        return (u64(bound(uint32_t(k))) << 32) | bound(uint32_t((k + C - 1) / C));
    }

    // The tokens at or above `from` to the leader, and the row finished there.  False (in
    // every CTA) where they are too many.
    __device__ bool few(float from, int k, float p, float least, double u) {
        const bool want = a.logprobs != nullptr;
        Model model;
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint4 w = word(i);
            if (want) {
                float v[EPW];
                E::unpack(w, v);
                add_model(model, v);
            }
            if (E::top(E::word_max(w)) >= from) enqueue(i);
        }
        if (want) {
            const u64 m = model_sum(model);
            if (lane == 0) s.my_model[warp] = m;
        }
        __syncthreads();
        for (uint32_t j = threadIdx.x; j < queued(); j += THREADS) {
            const int i = s.queue[j];
            float v[EPW];
            E::unpack(word(i), v);
            uint32_t which = 0;
#pragma unroll
            for (int e = 0; e < EPW; ++e) which |= v[e] >= from && v[e] > -CUDART_INF_F ? 1u << e : 0u;
            append(v, which, i);
        }
        __syncthreads();
        if (warp == 0) {
            if (want && lane < WARPS)
                st_peer64(map_peer(smem_addr(&s.seg_model[rank * WARPS + lane]), 0), s.my_model[lane]);
            if (lane == 0) st_peer32(map_peer(smem_addr(&s.list_n[rank]), 0), s.n_local);
        }
        const u64(*all)[2] = exchange<false>(s.n_local);
        if (__any_sync(FULL, lane < C && all[lane][0] > u64(CAP / C))) return false;
        if (rank) return true;

        int n;
        const u64* sorted = rank_list(&n);
        k = min(k, n);
        const int t = threadIdx.x;
        if (t >= MAX_TOPK) return true;  // (warps beyond: nothing left to rank)
        const u64 mine = t < k ? sorted[t] : 0;
        const float v = of_key(uint32_t(mine >> 32));
        const int idx = int(~uint32_t(mine));
        const float e = t < k ? ex2f(exponent(v)) : 0.f;
        uint32_t w = t < k ? weight_of(e) : 0u;
        // mass before it in the order, over the first warps
        constexpr int RW = MAX_TOPK / 32;
        u64 before = warp_scan(w, lane), W = 0;
        if (lane == 31) s.red[warp] = before;
        named_barrier();
        before -= w;
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            if (i < warp) before += s.red[i];
            W += s.red[i];
        }
        // (before < p W as integers: before < ceil(p W))
        if (p < 1.f && t > 0 && before >= u64(__double2ull_ru(double(p) * double(W)))) w = 0;
        if (!(e >= least)) w = 0;
        // the kept masses by index
        u64* by_index = s.rank;  // (the ranked list was read before the barrier)
        if (t < k) by_index[t] = (u64(uint32_t(idx)) << 32) | w;
        const u64 part = warp_add((u64(w > 0) << 48) + w);
        if (lane == 0) s.seg_mass[warp] = part;
        named_barrier();
        W = 0;
#pragma unroll
        for (int i = 0; i < RW; ++i) W += s.seg_mass[i];
        const int kept = int(W >> 48);
        W &= (u64(1) << 48) - 1;
        if (!__any_sync(FULL, w > 0)) return true;
        const u64 at = target_of(u, W);
        u64 lower = 0;
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const u64 o = by_index[j];
            if (int(o >> 32) < idx) lower += uint32_t(o);
        }
        const bool it = w && at >= lower && at < lower + w;
        if (__any_sync(FULL, it)) {
            u64 all_model = 0;
            for (int i = lane; i < C * WARPS; i += 32) all_model += s.seg_model[i];
            all_model = warp_add(all_model);
            if (it) answer(v, idx, W, all_model, kept);
        }
        return true;
    }
    __device__ static void named_barrier() {
        asm volatile("bar.sync 1, %0;" ::"n"(MAX_TOPK) : "memory");
    }

    // ------------------------------------------------------------ the cut ----

    __device__ void clear_histogram() {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(s.hi)[threadIdx.x] = zero;
        reinterpret_cast<uint4*>(s.lo)[threadIdx.x] = zero;
    }
    // Adds a mass to a bin; `at` is the bin's place, a shared-memory address of its upper sum.
    __device__ __forceinline__ void add_at(uint32_t at, uint32_t w) {
        asm volatile("red.shared.add.u32 [%0 + %3], %1;\n\tred.shared.add.u32 [%0], %2;" ::"r"(at),
                     "r"(w & ((1u << SPLIT) - 1)), "r"(w >> SPLIT), "n"(4 * BINS)
                     : "memory");
    }
    __device__ __forceinline__ void add_bin(uint32_t b, uint32_t w) {
        if constexpr (RES) {
            if (w) add_at(smem_addr(s.hi) + 4 * b, w);
        } else if (w) {  // any number of tokens a CTA: 64 bits, the carry by hand
            const uint32_t old = atomicAdd(&s.lo[b], w);
            if (old + w < old) atomicAdd(&s.hi[b], 1u);
        }
    }

    // How a pass sums the model's mass: not at all, from the row's own shares (T = 1), or from
    // its own exponentials.
    enum { NO_MODEL, SAME, APART };
    template <int MODEL>
    __device__ __forceinline__ void model_of(Model& m, const float* v, const float* sh) const {
        if constexpr (MODEL == SAME) m.add(sh);
        if constexpr (MODEL == APART) add_model(m, v);
    }

    // The histogram of masses of all tokens.  Without a softcap the bin comes from the
    // exponent: 2^23 - 32 d rounds to it.
    template <int MODEL>
    __device__ u64 histogram() {
        const hl::f2 slope = hl::pk1(-PER_OCTAVE), magic = hl::pk1(8388608.f);
        const uint32_t origin = smem_addr(s.hi) - 4 * 0x4b000000u;
        // tokens without a mass (31 octaves down, -inf, NaN) add their 0 to a bin past all others, one a
        // lane: predicated adds compiled to branches, three more instructions an add
        const float none = 8388608.f + float(BINS - 32 + lane);
        Model m;
        for (int i = s0 + lane; i < s1; i += 32) {
            float v[EPW], sh[EPW];
            hl::f2 d[PAIRS];
            uint32_t w[EPW];
            values(i, v);
            shares(v, d, sh);
            model_of<MODEL>(m, v, sh);
            weights(sh, w);
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                if constexpr (CAPPED || !RES) {
                    add_bin(bin_of(v[2 * j]), w[2 * j]);
                    add_bin(bin_of(v[2 * j + 1]), w[2 * j + 1]);
                } else {
                    float x, y;
                    hl::upk(hl::fma2(d[j], slope, magic), x, y);
                    add_at(__float_as_uint(fminf(x, none)) * 4 + origin, w[2 * j]);
                    add_at(__float_as_uint(fminf(y, none)) * 4 + origin, w[2 * j + 1]);
                }
            }
        }
        return MODEL == NO_MODEL ? 0 : model_sum(m);
    }

    // The cut after the first tokens of the order, among those inside `within`, before which
    // the count is below k (by_mass = false) or the mass below p times theirs.  Tokens
    // without a mass are left out: they are never drawn.  Collective over the cluster.
    __device__ Cut resolve(bool by_mass, int k, float p, const Cut& within) {
        const float wv = of_key(within.key);
        const bool all = within.key == 0u;
        u64 before = 0;
        double target = 0.0;
        uint32_t bin = 0, k0 = 0, k1 = 0;  // after level 0: keys k0 <= key <= k1
        int shift = 0;
        bool ties = false;
        for (int level = 0;; ++level) {
            cluster_barrier();  // the last histogram's readers are done
            clear_histogram();
            reinterpret_cast<uint4*>(s.cnt)[threadIdx.x] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            for (int i = s0 + lane; i < s1; i += 32) {
                float v[EPW];
                values(i, v);
                for (int e = 0; e < EPW; ++e) {
                    const uint32_t w = weight_of(share(v[e]));
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
                    if (by_mass) add_bin(b, w);
                }
            }
            if (by_mass) locate<true, true>(double(p), level == 0, before);
            else locate<false, true>(double(k), level == 0, before);
            cluster_barrier();  // the counts were read: the list's place is free
            target = s.target;
            bin = s.pick_bin;
            if (bin == BINS) return within;  // the target is past all of them
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
                __syncthreads();
                if (lane == 0) s.red[warp] = (u64(~least) << 32) | largest;
                __syncthreads();
                for (int i = 0; i < WARPS; ++i)
                    least = min(least, ~uint32_t(s.red[i] >> 32)),
                    largest = max(largest, uint32_t(s.red[i]));
                const u64(*got)[2] = exchange<true>((u64(~least) << 32) | largest);
                for (int r = 0; r < C; ++r)
                    least = min(least, ~uint32_t(got[r][0] >> 32)),
                    largest = max(largest, uint32_t(got[r][0]));
                k0 = least, k1 = largest;
            } else {
                k1 = k1 - (bin << shift);
                const uint32_t span = (1u << shift) - 1;
                k0 = k1 - k0 > span ? k1 - span : k0;
                if (some <= uint32_t(CAP / C)) break;
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
            __syncthreads();
            if (threadIdx.x == 0) s.n_local = 0;
            __syncthreads();
            for (int i = s0 + lane; i < s1; i += 32) {
                float v[EPW];
                values(i, v);
                uint32_t which = 0;
#pragma unroll
                for (int e = 0; e < EPW; ++e) {
                    bool in;
                    if (by_bin) in = bin_of(v[e]) == bin;
                    else in = key_of(v[e]) >= k0 && key_of(v[e]) <= k1;
                    if (in && weight_of(share(v[e])) &&
                        (all || inside(v[e], index(i, e), within, wv)))
                        which |= 1u << e;
                }
                append(v, which, i);
            }
            __syncthreads();
            send_count();
            cluster_barrier();
            if (rank == 0) {
                int n;
                const u64* sorted = rank_list(&n);
                const Cut cut = cut_of(sorted, n, by_mass, before, target);
                if (warp == 0 && lane < C) {
                    st_peer32(map_peer(smem_addr(&s.cut_key), lane), cut.key);
                    st_peer32(map_peer(smem_addr(&s.cut_idx), lane), uint32_t(cut.idx));
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
        if (lane == 0) s.red[warp] = mine;
        __syncthreads();
        u64 lower = 0, count = 0;
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) lower += s.red[i];
            count += s.red[i];
        }
        const u64(*got)[2] = exchange<true>(count);
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

    // Leader: the last of a ranked list's tokens that stay (whole block).
    __device__ Cut cut_of(const u64* sorted, int n, bool by_mass, u64 before, double target) {
        constexpr int Q = (CAP + THREADS - 1) / THREADS;
        u64 w[Q], mine = 0;
        const int i0 = threadIdx.x * Q;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            w[q] = 0;
            if (i0 + q < n)
                w[q] = by_mass ? weight_of(share(of_key(uint32_t(sorted[i0 + q] >> 32)))) : 1u;
            mine += w[q];
        }
        u64 total;
        u64 at = before + block_scan(mine, s.red, &total);
        u64 stay = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            stay += i0 + q < n && (double(at) < target || (at == 0 && i0 + q == 0));
            at += w[q];
        }
        block_scan(stay, s.red, &total);
        const u64 last = sorted[total - 1];
        return Cut{uint32_t(last >> 32), int(~uint32_t(last))};
    }

    // ----------------------------------------------------------- the draw ----

    // A segment's sums; then, after a block barrier, the CTA's to the leader (warp 0).
    __device__ void keep_segment(u64 mass, uint32_t kept, u64 model) {
        mass = warp_add(mass);
        kept = __reduce_add_sync(FULL, kept);
        if (lane == 0) s.my_mass[warp] = mass, s.my_kept[warp] = kept, s.my_model[warp] = model;
    }
    __device__ void send_segments() {
        if (lane < WARPS) {
            const int g = rank * WARPS + lane;
            st_peer64(map_peer(smem_addr(&s.seg_mass[g]), 0), s.my_mass[lane]);
            st_peer32(map_peer(smem_addr(&s.seg_kept[g]), 0), s.my_kept[lane]);
            st_peer64(map_peer(smem_addr(&s.seg_model[g]), 0), s.my_model[lane]);
        }
        __syncwarp();
    }
    // The last step of a row: the sums to the leader, which waits for all; the others leave
    // (their shared memory is read by no one after the barrier before).
    __device__ bool leave() {
        __syncthreads();
        if (warp == 0) {
            send_segments();
            cluster_arrive();
        } else {
            if (rank) return true;
            cluster_arrive_relaxed();
        }
        if (rank) return true;
        cluster_wait();
        return false;
    }

    // No filter: the masses of everything.
    template <int MODEL>
    __device__ void sum_all() {
        Model m;
        u64 mass = 0;
        uint32_t kept = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            float v[EPW], sh[EPW];
            hl::f2 d[PAIRS];
            uint32_t w[EPW];
            values(i, v);
            shares(v, d, sh);
            model_of<MODEL>(m, v, sh);
            weights(sh, w);
#pragma unroll
            for (int j = 0; j < EPW; j += 2) {
                mass += w[j] + w[j + 1];  // at most 2^31 and a little
                kept += min(w[j], 1u) + min(w[j + 1], 1u);
            }
        }
        keep_segment(mass, kept, MODEL == NO_MODEL ? 0 : model_sum(m));
    }

    // The masses of what the cut and min-p leave.
    __device__ void sum_kept(const Cut& cut, float least, bool want, u64 model) {
        const float kv = cut.key ? of_key(cut.key) : -CUDART_INF_F;
        const bool same = !CAPPED && c == a.K;
        Model m;
        u64 mass = 0;
        uint32_t kept = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            float v[EPW], sh[EPW];
            hl::f2 d[PAIRS];
            uint32_t w[EPW];
            values(i, v);
            shares(v, d, sh);
            if (want) {
                if (same) m.add(sh);
                else add_model(m, v);
            }
            weights(sh, w);
#pragma unroll
            for (int e = 0; e < EPW; ++e) {
                const bool in = sh[e] >= least && inside(v[e], index(i, e), cut, kv) && w[e];
                mass += in ? w[e] : 0u;
                kept += in;
            }
        }
        keep_segment(mass, kept, want ? model_sum(m) : model);
    }

    // The masses of the bins above `bin` (and of min-p), the bin's tokens to the leader.  Words
    // with nothing at or above the bin's lower edge are passed over.
    template <bool LEAST>
    __device__ void sum_above(uint32_t bin, float least, u64 model) {
        const hl::f2 slope = hl::pk1(-PER_OCTAVE), magic = hl::pk1(8388608.f);
        const float edge = 8388608.f + float(bin);
        const float from = lower_edge(top, float(bin), PER_OCTAVE);
        u64 mass = 0;
        uint32_t kept = 0;
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const int i = i0 + lane;
            const uint4 q4 = i < s1 ? word(i) : make_uint4(E::LOWEST, E::LOWEST, E::LOWEST, E::LOWEST);
            if (!__any_sync(FULL, E::top(E::word_max(q4)) >= from)) continue;
            float v[EPW], sh[EPW], at[EPW];
            hl::f2 d[PAIRS];
            uint32_t w[EPW];
            unpack(q4, v, !RES);
            shares(v, d, sh);
            weights(sh, w);
            bool on_edge = false;
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                if constexpr (CAPPED) {
                    at[2 * j] = 8388608.f + float(bin_of(v[2 * j]));
                    at[2 * j + 1] = 8388608.f + float(bin_of(v[2 * j + 1]));
                } else {
                    hl::upk(hl::fma2(d[j], slope, magic), at[2 * j], at[2 * j + 1]);
                }
                uint32_t both = 0;
#pragma unroll
                for (int e = 2 * j; e < 2 * j + 2; ++e) {
                    bool in = at[e] < edge;
                    if constexpr (LEAST) in = in && sh[e] >= least;
                    if constexpr (CAPPED) in = in && w[e];
                    if (in) both += w[e], ++kept;
                    on_edge |= at[e] == edge;
                }
                mass += both;
            }
            if (on_edge && i < s1) enqueue(i);  // (at c = 0 a lane past the segment sees -inf in bin 0)
        }
        keep_segment(mass, kept, model);
        __syncthreads();
        for (uint32_t j = threadIdx.x; j < queued(); j += THREADS) {
            const int i = s.queue[j];
            float v[EPW];
            values(i, v);
            uint32_t which = 0;
#pragma unroll
            for (int e = 0; e < EPW; ++e) {
                const float x = CAPPED ? 8388608.f + float(bin_of(v[e]))
                                       : __fmaf_rn(__fmul_rn(__fsub_rn(v[e], zm), c), -PER_OCTAVE, 8388608.f);
                which |= x == edge && weight_of(share(v[e])) ? 1u << e : 0u;
            }
            append(v, which, i);
        }
    }

    // Leader, whole block: the same once the bin of the cut is listed, with `before` the mass
    // above it: the listed tokens inside the cut join their segments.
    __device__ void finish_bin(u64 before, float least, double u) {
        const int n = count_listed();
        // before a mass of p W: as integers, before its ceiling
        const u64 limit = u64(__double2ull_ru(s.target));
        if (n > RANKED) {
            int count;
            const u64* sorted = rank_list(&count);
            const Cut cut = cut_of(sorted, count, true, before, s.target);
            const float kv = of_key(cut.key);
            for (int i = threadIdx.x; i < count; i += THREADS) {
                const float v = of_key(uint32_t(sorted[i] >> 32));
                const int idx = int(~uint32_t(sorted[i]));
                if (inside(v, idx, cut, kv)) join_segment(v, idx, least);
            }
            __syncthreads();
            finish(cut, least, u);
            return;
        }
        // a token's mass before it by comparison with all; the last that stays is the cut
        const int t = threadIdx.x;
        const u64 mine = t < n ? listed(t) : 0;
        const float v = of_key(uint32_t(mine >> 32));
        ulonglong2* all = reinterpret_cast<ulonglong2*>(s.rank);
        if (t < n) all[t] = make_ulonglong2(mine, weight_of(share(v)));
        __syncthreads();
        u64 last = ~u64(0);
        if (t < n) {
            u64 at = before;
#pragma unroll 4
            for (int j = 0; j < n; ++j) {
                const ulonglong2 o = all[j];
                at += o.x > mine ? o.y : 0;
            }
            if (at < limit || at == 0) {
                last = mine;
                join_segment(v, int(~uint32_t(mine)), least);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const u64 other = __shfl_xor_sync(FULL, last, o);
            last = other < last ? other : last;
        }
        if (lane == 0) s.red[warp] = last;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WARPS; ++i) last = s.red[i] < last ? s.red[i] : last;
        finish(Cut{uint32_t(last >> 32), int(~uint32_t(last))}, least, u);
    }
    // A listed token that stays joins its segment.
    __device__ void join_segment(float v, int idx, float least) {
        const float sh = share(v);
        if (!(sh >= least)) return;
        const int w = (idx + head) / EPW, cta = w / a.per;
        const int have = min(nw, (cta + 1) * a.per) - cta * a.per;
        const int g = cta * WARPS + (w - cta * a.per) / ((have + WARPS - 1) / WARPS);
        atomicAdd(&s.seg_mass[g], u64(weight_of(sh)));
        atomicAdd(&s.seg_kept[g], 1u);
    }

    // Leader, whole block: the target's segment from the segments' masses, and the token by going
    // over the segment again.
    __device__ void finish(const Cut& cut, float least, double u) {
        if (warp == 0) {
            static_assert(SEGS == 64, "two segments a lane");
            const int n = C * WARPS, g = 2 * lane;
            const u64 m0 = g < n ? s.seg_mass[g] : 0, m1 = g + 1 < n ? s.seg_mass[g + 1] : 0;
            const uint32_t kept = __reduce_add_sync(
                FULL, (g < n ? s.seg_kept[g] : 0) + (g + 1 < n ? s.seg_kept[g + 1] : 0));
            const u64 model = warp_add((g < n ? s.seg_model[g] : 0) + (g + 1 < n ? s.seg_model[g + 1] : 0));
            const u64 inc = warp_scan(m0 + m1, lane), W = __shfl_sync(FULL, inc, 31);
            const u64 t = target_of(u, W), from = inc - m0 - m1;
            if (t >= from && t < inc) {
                const bool second = t >= from + m0;
                s.fin[0] = t - from - (second ? m0 : 0);
                s.fin_seg = uint32_t(g) + (second ? 1u : 0u);
            }
            if (lane == 0) s.fin[1] = W, s.fin[2] = model, s.pick_most = kept;
        }
        __syncthreads();
        const u64 t = s.fin[0], W = s.fin[1], model = s.fin[2];
        const int kept = int(s.pick_most);
        // the segment's words of the row, as the kernel cut them
        const int cta = int(s.fin_seg / WARPS), part = int(s.fin_seg % WARPS);
        const int from = min(nw, cta * a.per), mine = min(nw, from + a.per) - from;
        const int seg = (mine + WARPS - 1) / WARPS;
        const int b0 = from + min(mine, part * seg), b1 = from + min(mine, (part + 1) * seg);
        const float kv = cut.key ? of_key(cut.key) : -CUDART_INF_F;
        u64 lower = 0;
        for (int b = b0; b < b1; b += THREADS) {
            const int i = b + threadIdx.x;
            float v[EPW];
            uint32_t w[EPW];
            u64 here = 0;
            if (i < b1) {
                unpack(global_word(i), v, true);
#pragma unroll
                for (int e = 0; e < EPW; ++e) {
                    const float sh = share(v[e]);
                    w[e] = sh >= least && inside(v[e], i * EPW + e - head, cut, kv) ? weight_of(sh) : 0u;
                    here += w[e];
                }
            }
            u64 total;
            u64 at = lower + block_scan(here, s.red, &total);
            if (t >= at && t < at + here) {
#pragma unroll
                for (int e = 0; e < EPW; ++e) {
                    if (t >= at && t < at + w[e]) answer(v[e], i * EPW + e - head, W, model, kept);
                    at += w[e];
                }
            }
            lower += total;
            if (t < lower) return;
        }
    }
};

template <typename DT, bool CAPPED, bool RES>
__global__ void __launch_bounds__(THREADS, 4) sample_kernel(const __grid_constant__ Args a) {
    __shared__ Shared s;
    extern __shared__ __align__(16) uint4 words[];
    using R = Row<DT, CAPPED, RES>;
    constexpr int EPW = R::EPW;
    R r(a, s);
    cluster_arrive_relaxed();  // waited for before the first write to a peer: every CTA has started
    uint32_t C;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
    r.C = int(C);
    r.rank = int(cluster_ctarank());
    r.lane = threadIdx.x & 31, r.warp = threadIdx.x >> 5;
    r.row = a.row0 + hl::cluster_id_x();
    r.words = words;
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.logits) + uint64_t(r.row * a.ld) * sizeof(DT);
    r.gwords = reinterpret_cast<const uint4*>(base & ~uintptr_t(15));
    r.head = int((base & 15) / sizeof(DT));
    r.nw = (r.head + a.V + EPW - 1) / EPW;
    r.w0 = min(r.nw, r.rank * a.per);
    const int mine = min(r.nw, r.w0 + a.per) - r.w0, seg = (mine + WARPS - 1) / WARPS;
    r.s0 = min(mine, r.warp * seg), r.s1 = min(mine, r.s0 + seg);
    const int lane = r.lane, warp = r.warp;

    // the warp's words: whole ones by a bulk copy, those that reach outside the row by element
    bool lost = false;
    int f0 = 0, f1 = 0;
    const uint32_t bar = smem_addr(&s.bar[warp]);
    if constexpr (RES) {
        f0 = r.w0 == 0 && r.s0 == 0 && r.head ? 1 : r.s0;  // first whole word
        const bool ragged = (r.head + a.V) % EPW != 0;
        f1 = ragged && r.w0 + r.s1 == r.nw && r.s1 > r.s0 ? r.s1 - 1 : r.s1;
        if (lane == 0) {
            hl::mbar_init(bar, 1);
            hl::fence_mbar_init();
            hl::fence_proxy_async();
            if (f1 > f0) {
                hl::mbar_arrive_expect_tx(bar, uint32_t(f1 - f0) * 16);
#ifdef HL_FAULT_INJECT
                if (r.row != a.drop_row)
#endif
                bulk_g2s(smem_addr(words + f0), r.gwords + r.w0 + f0, uint32_t(f1 - f0) * 16, bar);
            }
        }
        __syncwarp();
        if (lane == 1 && r.s0 < r.s1 && f0 > r.s0) words[r.s0] = r.global_word(r.w0 + r.s0);
        if (lane == 2 && f1 < r.s1 && f1 >= f0) words[f1] = r.global_word(r.w0 + f1);
    }
    // meanwhile: the settings, an empty histogram
    const float temp = a.temperature ? a.temperature[r.row] : 1.f;
    const double u = a.uniforms[r.row];
    const int want_k = a.top_k ? a.top_k[r.row] : 0;
    const float p = a.top_p ? a.top_p[r.row] : 1.f;
    const float least = a.min_p ? a.min_p[r.row] : 0.f;
    if (threadIdx.x == 0) s.n_local = s.queued = 0;
    const u64 ubits = u64(__double_as_longlong(u));  // in [0, 1): below 1.0's bits (or -0)
    const bool bad = !(temp >= 0.f && temp < CUDART_INF_F) ||
                     !(ubits < 0x3ff0000000000000ull || ubits == 0x8000000000000000ull) ||
                     !(p >= 0.f) || !(least >= 0.f && least <= 1.f);
    r.c = __fdiv_rn(a.K, fabsf(temp));  // (of -0 too: a negative c would send the bins out of range)
    const bool greedy = !(r.c < CUDART_INF_F);
    if (greedy) r.c = a.K;
    const int k = greedy ? 1 : want_k <= 0 || want_k > a.V ? a.V : want_k;
    const bool small_k = k < a.V && k <= MAX_TOPK;
    if (small_k) {
        if (threadIdx.x < TOPS) s.tops[threadIdx.x] = 0;
    } else if (p < 1.f) {
        r.clear_histogram();
    }
    if constexpr (RES) {
#ifdef HL_FAULT_INJECT
        const unsigned long long limit = a.wait_ns;
#else
        constexpr unsigned long long limit = WAIT_NS;
#endif
        if (f1 > f0 && !hl::mbar_wait_bounded(bar, 0, limit)) {
            lost = true;
            hl::mbar_wait_bounded(bar, 0, limit);  // so that the copy does not land later
        }
        __syncwarp();
    }

    // the largest logit
    uint32_t m2 = R::E::LOWEST;
#pragma unroll 4
    for (int i = r.s0 + lane; i < r.s1; i += 32) m2 = R::E::max2(m2, R::E::word_max(r.word(i)));
    const float mine_top = R::E::top(m2);
    const uint32_t warp_top = __reduce_max_sync(FULL, key_of(mine_top));
    if (lane == 0) s.ired[warp] = warp_top;
    const bool any_lost = __syncthreads_or(lost);
    const uint32_t cta_top = __reduce_max_sync(FULL, s.ired[lane % WARPS]);
    cluster_wait();
    const u64 bounds = small_k && k > 1 ? r.bounds_of(mine_top, of_key(cta_top), k) : 0;
    const u64(*got)[2] = r.template exchange<true>((u64(any_lost) << 32) | cta_top, bounds);
    const u64 other = got[lane < r.C ? lane : 0][0], edges = got[lane < r.C ? lane : 0][1];
    const uint32_t topkey = __reduce_max_sync(FULL, uint32_t(other));
    const bool given_up = __any_sync(FULL, (other >> 32) != 0);
    r.top = of_key(topkey);
    if (bad || given_up || topkey == KEY_NONE) {
        if (r.rank == 0 && threadIdx.x == 0) {
            r.no_token();
            if (bad || given_up) atomicOr(a.err, bad ? 1 : 2);
        }
        return;
    }
    r.zm = r.z(r.top);
    if constexpr (CAPPED) r.zt = r.model_z(r.top);

    if (small_k) {
        const uint32_t edge = max(__reduce_max_sync(FULL, uint32_t(edges >> 32)),
                                  __reduce_min_sync(FULL, uint32_t(edges)));
        const float from = k == 1 ? r.top : edge > KEY_NONE ? of_key(edge) : -CUDART_INF_F;
        if (r.few(from, k, p, least, u)) return;
    }

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
    const Cut none{0u, 0x7fffffff};
    const bool want = a.logprobs != nullptr;
    if (k == a.V && !(p < 1.f)) {
        if (least != 0.f) r.sum_kept(none, least, want, 0);
        else if (!want) r.template sum_all<R::NO_MODEL>();
        else if (!CAPPED && r.c == a.K) r.template sum_all<R::SAME>();
        else r.template sum_all<R::APART>();
        if (!r.leave()) r.finish(none, least, u);
        return;
    }
    if (k == a.V) {
        const u64 model = !want           ? r.template histogram<R::NO_MODEL>()
                          : !CAPPED && r.c == a.K ? r.template histogram<R::SAME>()
                                       : r.template histogram<R::APART>();
        r.template locate<true, false>(double(p), true, 0);
        const uint32_t bin = s.pick_bin;
        const u64 before = s.pick_before;
        if (bin < BINS - 1) {
            if (least == 0.f) r.template sum_above<false>(bin, least, model);
            else r.template sum_above<true>(bin, least, model);
            __syncthreads();
            if (warp == 0) {
                r.send_segments();
                if (lane == 0) st_peer32(map_peer(smem_addr(&s.list_n[r.rank]), 0), s.n_local);
            }
            const u64(*all)[2] = r.template exchange<false>(s.n_local);
            if (!__any_sync(FULL, lane < r.C && all[lane][0] > u64(CAP / r.C))) {
                if (r.rank == 0) r.finish_bin(before, least, u);
                return;
            }
        }
        const Cut cut = r.resolve(true, 0, p, none);
        r.sum_kept(cut, least, false, model);
        if (!r.leave()) r.finish(cut, least, u);
        return;
    }
    Cut cut = r.resolve(false, k, 1.f, none);
    if (p < 1.f) cut = r.resolve(true, 0, p, cut);
    r.sum_kept(cut, least, want, 0);
    if (!r.leave()) r.finish(cut, least, u);
}

// -------------------------------------------------------------------- launch ----

// Shared memory of a CTA's words: four CTAs an SM beside the fixed part (three for calls without
// top-k and top-p, whose rows have fewer steps to wait for), and the most.  Measured, us, at 24 / 38 /
// 50 / 66 KB: 1024 rows of 151936 unfiltered 124 / 124 / 119 / 140, 1024 x 128256 top-p
// 263 / 250 / 275 / 292, 8192 x 32000 top-k 385 / 302 / 303 / 315.
constexpr int SLICE = 38 * 1024;
constexpr int SLICE_UNFILTERED = 50 * 1024;
constexpr int SLICE_MOST = 192 * 1024;

// (static, so that `done` is this library's own where a process holds two copies of it)
template <typename DT, bool CAPPED>
static int launch(Args a, int64_t N, int device, int sms, cudaStream_t st) {
    const int64_t words = (int64_t(a.V) * sizeof(DT) + 30) / 16;  // at most, wherever rows start
    auto slice = [&](int c) { return (words + c - 1) / c * 16; };
    int C = 1;
    const int most = a.top_k || a.top_p ? SLICE : SLICE_UNFILTERED;
    while (C < MAXC && slice(C) > most) ++C;
    // few rows: more CTAs a row, while each warp has a few words a lane
    while (C < MAXC && N * (C + 1) <= 2 * sms && slice(C) > 8 * 1024) ++C;
    const bool resident = slice(C) <= SLICE_MOST;
    const void* kernel = resident ? reinterpret_cast<const void*>(&sample_kernel<DT, CAPPED, true>)
                                  : reinterpret_cast<const void*>(&sample_kernel<DT, CAPPED, false>);
    a.per = int(slice(C) / 16);
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
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {unsigned(C), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (C <= 4) {  // small clusters where there is room: 8192 x 32000 294 -> 262 us; at eight
                       // CTAs a cluster the default spread is 2% better
            attr[1].id = cudaLaunchAttributeClusterSchedulingPolicyPreference;
            attr[1].val.clusterSchedulingPolicyPreference = cudaClusterSchedulingPolicyLoadBalancing;
            cfg.numAttrs = 2;
        }
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
