// hl_beam.cu -- headloss_beam_select (include/headloss_beam.h).
//
// slice_kernel: a row is split into slices, a CTA each, as far as the rows alone do not fill the GPU. A
// slice goes in batches of 2048 16-byte words through a ring of two in shared memory (cp.async; each thread
// copies and reads its own eight words, so it waits for nobody): one read of the logits. A bound for its candidates comes from the first batch's maxima of groups of
// threads: the keep-th largest of them has at least `keep` logits at or above it, and hardly more.
// The words at the bound and above are listed, and the list raises the bound as it grows; the
// exponentials are added in fp32 on the way. The candidates go to the workspace.
// merge_kernel: a CTA a request joins the beams' sums and takes the candidates of all slices in two
// steps: fp32 scores with a bound of their error leave hardly more than `keep`, which are scored in
// fp64 and ranked. So the order between beams does not hang on fp32 rounding of the scores.
//
// What bounds it: 2048 bf16 rows of 151936 under a softcap take 197 us in slice_kernel, at 40% of HBM's rate and 62%
// of the issue slots (15 instructions a logit, the capped exponentials among them), and 13 in merge_kernel (each by
// itself; a call 200 to 210). Whole slices held in registers took 252 us, slices in batches through registers 297. Up to
// some tens of rows the two launches and their chains of steps count: 4 x 32000 14 us, of which the merge is 11.
// A slice whose candidates are too many for its list, or come with few threads, is bisected by reading it again: 64 rows
// of 32000 equal logits 770 us, and of 128 or 256 allowed tokens in a run 690 (of 16, 64, 384 and more 15).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "headloss.h"
#include "headloss_beam.h"
#include "hl_pack.cuh"
#include "hl_tanh_poly.h"

namespace hl_beam {

constexpr int ST = 256;               // threads of a slice
constexpr int WORDS = 8;              // 16-byte words a thread
constexpr int SLICE_WORDS = ST * WORDS;
constexpr int MT = 512;               // threads of a merge
constexpr int MAX_BEAMS = 64, MAX_KEEP = 128;
constexpr int LIST = MT;              // survivors that are ranked at once
constexpr float NEG = -INFINITY;

struct __align__(16) Head {
    float top;   // the slice's largest logit
    float sum;   // of 2^((z - z(top)) K)
    int n;       // candidates
    int pad;
};
struct Cand {
    float x;
    int at;
};

struct Args {
    const void* logits;
    int64_t ld;
    int V;
    const float* scores;
    const uint8_t* ended;
    int64_t eos;
    int beams, keep, stay;
    float cap, inv_cap;
    float scale, K;       // logits_scale, logits_scale * log2(e)
    float cap_K, near;    // cap * K; the magnitudes that `poly` covers
    float far;            // FAR octaves in logits
    int precise;          // a cap whose exponentials are taken from differences of logits alone
    hl::f2 poly[6];       // z K = x poly(x^2), each coefficient twice
    int slices, cap_list; // slices a row, candidates a slice
    Head* heads;
    Cand* cands;
    float* out_scores;
    int32_t* parents;
    int64_t* tokens;
    uint8_t* out_ended;
};

// Bits in the order of the values (0 and -0 the same).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double x) {
    const uint64_t b = uint64_t(__double_as_longlong(x + 0.0));
    return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}

// z(x) - z(top), top >= x: exact without a cap. With one, for y = x / c, b = top / c and E = e^-2|.|,
// tanh y - tanh b = 2 F (e^-2(b - y) - 1) / ((1 + E_y) (1 + E_b)), F the larger E where the signs are equal, else 1: no
// cancellation, and an error (2^-19 up to 8 caps) that is relative to the difference.
template <bool CAP>
__device__ __forceinline__ float fall(float x, float top, float cap, float inv_cap) {
    if (x == top) return 0.f;
    if (!CAP) return x - top;
    const float y = x * inv_cap, b = top * inv_cap, ey = expf(-2.f * fabsf(y)), eb = expf(-2.f * fabsf(b));
    const float f = y < 0.f && b >= 0.f ? 1.f : fmaxf(ey, eb);
    return cap * __fdividef(2.f * f * expm1f(-2.f * ((top - x) * inv_cap)), (1.f + ey) * (1.f + eb));
}
template <int DT>
struct Words {
    static constexpr int SIZE = DT == HEADLOSS_FP32 ? 4 : 2, PER = 16 / SIZE;
    static constexpr uint32_t NONE = DT == HEADLOSS_FP32 ? 0xff800000u
                                     : DT == HEADLOSS_BF16 ? 0xff80ff80u : 0xfc00fc00u;
    // the larger of each pair (or value); a NaN loses
    static __device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
        if (DT == HEADLOSS_FP32) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
        if (DT == HEADLOSS_BF16) {
            const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                             *reinterpret_cast<const __nv_bfloat162*>(&b));
            return *reinterpret_cast<const uint32_t*>(&r);
        }
        const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ float2 pair(uint32_t a) {
        if (DT == HEADLOSS_BF16) return make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
        return __half22float2(*reinterpret_cast<const __half2*>(&a));
    }
    static __device__ __forceinline__ float top_of(uint32_t a) {
        if (DT == HEADLOSS_FP32) return __uint_as_float(a);
        const float2 f = pair(a);
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ float value(const char* row, int64_t e) {
        if (DT == HEADLOSS_FP32) return reinterpret_cast<const float*>(row)[e];
        if (DT == HEADLOSS_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[e]);
        return __half2float(reinterpret_cast<const __half*>(row)[e]);
    }
    // a word that is not the row's alone: elements lo .. of it, -inf outside
    static __device__ __forceinline__ void edge(const char* row, int lo, int V, uint32_t (&w)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (DT == HEADLOSS_FP32) {
                const int e = lo + k;
                if (e >= 0 && e < V) w[k] = reinterpret_cast<const uint32_t*>(row)[e];
            } else {
                const int e = lo + 2 * k;
                const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
                if (e >= 0 && e < V) w[k] = (w[k] & 0xffff0000u) | p[e];
                if (e + 1 >= 0 && e + 1 < V) w[k] = (w[k] & 0xffffu) | uint32_t(p[e + 1]) << 16;
            }
        }
    }
    // a value in both halves, rounded towards zero
    static __device__ __forceinline__ uint32_t packed(float v) {
        if (DT == HEADLOSS_FP32) return __float_as_uint(v);
        if (DT == HEADLOSS_BF16) return (__float_as_uint(v) >> 16) * 0x10001u;
        return uint32_t(__half_as_ushort(__float2half_rz(v))) * 0x10001u;
    }
    // a value in both halves, rounded upwards (past the largest: infinity)
    static __device__ __forceinline__ uint32_t packed_up(float v) {
        if (DT == HEADLOSS_FP32) return __float_as_uint(v);
        if (DT == HEADLOSS_BF16) return uint32_t(__bfloat16_as_ushort(__float2bfloat16_ru(v))) * 0x10001u;
        return uint32_t(__half_as_ushort(__float2half_ru(v))) * 0x10001u;
    }
    // whether every magnitude of two words is at most `most` (a NaN may hide behind a number)
    static __device__ __forceinline__ bool within(const uint32_t (&v)[4], const uint32_t (&w)[4], uint32_t most) {
        if (DT == HEADLOSS_FP32) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(__uint_as_float(v[k])), fabsf(__uint_as_float(w[k]))));
            return m <= __uint_as_float(most);
        }
        if (DT == HEADLOSS_BF16) {
            using P = hl::Pack16<__nv_bfloat16>;
            const uint32_t m = P::absmax2(P::absmax2(P::absmax2(v[0], v[1]), P::absmax2(v[2], v[3])),
                                          P::absmax2(P::absmax2(w[0], w[1]), P::absmax2(w[2], w[3]))) & 0x7fff7fffu;
            return __hble2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&most));
        }
        using P = hl::Pack16<__half>;
        const uint32_t m = P::absmax2(P::absmax2(P::absmax2(v[0], v[1]), P::absmax2(v[2], v[3])),
                                      P::absmax2(P::absmax2(w[0], w[1]), P::absmax2(w[2], w[3]))) & 0x7fff7fffu;
        return __hble2(*reinterpret_cast<const __half2*>(&m), *reinterpret_cast<const __half2*>(&most));
    }
    // whether a value (of two) is `least` or more, and not -inf
    static __device__ __forceinline__ bool reaches(uint32_t t, uint32_t least) {
        if (DT == HEADLOSS_FP32) return __uint_as_float(t) >= __uint_as_float(least) && __uint_as_float(t) > NEG;
        if (least == NONE) return t != NONE;
        if (DT == HEADLOSS_BF16)
            return !__hblt2(*reinterpret_cast<const __nv_bfloat162*>(&t), *reinterpret_cast<const __nv_bfloat162*>(&least));
        return !__hblt2(*reinterpret_cast<const __half2*>(&t), *reinterpret_cast<const __half2*>(&least));
    }
    static __device__ __forceinline__ void unpack(const uint32_t (&w)[4], hl::f2* x) {
        if (DT == HEADLOSS_FP32) {
            x[0] = hl::pk(__uint_as_float(w[0]), __uint_as_float(w[1]));
            x[1] = hl::pk(__uint_as_float(w[2]), __uint_as_float(w[3]));
        } else {
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
                const float2 f = pair(w[k]);
                x[k] = hl::pk(f.x, f.y);
            }
        }
    }
};

// 2^(z K - zt) of a capped logit, tanh through two MUFU operations: any x.
__device__ __forceinline__ float mass_any(float x, float zt, const Args& a) {
    if (x == NEG) return 0.f;
    const float y = x * a.inv_cap, w = hl::ex2f(-2.8853900817779268f * fabsf(y));
    return hl::ex2f(fmaf(a.cap_K, copysignf((1.f - w) * hl::rcpf(1.f + w), y), -zt));
}
// The same of N pairs of logits within HL_TANH_B_Y0 caps, added up: z K = x Q(x^2), the cap and K in
// the coefficients, each of which is fetched once for all pairs.
template <int N>
__device__ __forceinline__ hl::f2 mass_near(const hl::f2 (&x)[N], hl::f2 minus_zt, const Args& a) {
    hl::f2 t[N], q[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        t[j] = hl::mul2(x[j], x[j]);
        q[j] = hl::fma2(a.poly[5], t[j], a.poly[4]);
    }
#pragma unroll
    for (int i = 3; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = hl::fma2(q[j], t[j], a.poly[i]);
    hl::f2 s = 0ull;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const hl::f2 e = hl::ex2p(hl::fma2(x[j], q[j], minus_zt));
        s = j ? hl::add2(s, e) : e;
    }
    return s;
}

constexpr int HITS = ST;      // words with a candidate that a slice lists
constexpr int MANY = 48;      // so many are thinned out before their logits are looked at
constexpr float FAR = 64.f;   // octaves above a thread's shift at which it is raised
constexpr double PRECISE = 1024.0;  // cap * scale above which the slice is read again for its sum
constexpr int RING = 2 * SLICE_WORDS * 16;

template <int DT, bool CAP>
__global__ void __launch_bounds__(ST, 3) slice_kernel(const __grid_constant__ Args a) {
    using W = Words<DT>;
    extern __shared__ __align__(16) uint4 ring[];  // two batches
    __shared__ __align__(16) uint4 hit[HITS];
    __shared__ int hit_at[HITS];  // the word's place, and whether its sum went through mass_any
    __shared__ __align__(16) float tops[ST];
    __shared__ uint32_t group[32];
    __shared__ float part[ST / 32], shift[ST / 32];
    __shared__ long long extra[ST / 32];
    __shared__ int more_hits[3], count, found[ST / 32];
    __shared__ float bound_at;
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = int(blockIdx.x / unsigned(a.slices));
    const int slice = int(blockIdx.x) - row * a.slices;
    Head* head = a.heads + blockIdx.x;
    Cand* cands = a.cands + int64_t(blockIdx.x) * a.cap_list;
    if (!(a.scores[row] > NEG) || (a.ended && a.ended[row])) return;  // the merge does not look here either

    const char* base = static_cast<const char*>(a.logits) + row * a.ld * W::SIZE;
    const int off = int(reinterpret_cast<uintptr_t>(base) & 15) / W::SIZE;  // elements of the first word before the row
    const int words = (off + a.V + W::PER - 1) / W::PER;
    const int j0 = int(int64_t(words) * slice / a.slices), j1 = int(int64_t(words) * (slice + 1) / a.slices);
    if (tid == 0) more_hits[0] = more_hits[1] = more_hits[2] = count = 0;
    int hits = 0;  // listed words

    // the n-th largest of the threads' values, for all threads
    auto nth = [&](float mine, int n) {
        tops[tid] = mine;
        __syncthreads();
        int rank = 0;
        for (int k = 0; k < ST; k += 4) {
            const float4 u = *reinterpret_cast<const float4*>(&tops[k]);
            rank += (u.x > mine || (u.x == mine && k < tid)) + (u.y > mine || (u.y == mine && k + 1 < tid)) +
                    (u.z > mine || (u.z == mine && k + 2 < tid)) + (u.w > mine || (u.w == mine && k + 3 < tid));
        }
        if (rank == n - 1) bound_at = mine;
        __syncthreads();
        return bound_at;
    };
    // the keep-th largest and the largest of 32 values, a lane each (keep <= 32)
    auto sorted = [&](float v, float& largest) {
#pragma unroll
        for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
            for (int o = k >> 1; o; o >>= 1) {
                const float u = __shfl_xor_sync(0xffffffffu, v, o);
                const bool larger = ((lane & o) == 0) == ((lane & k) == 0);  // falling where the k bit is clear
                v = larger ? fmaxf(v, u) : fminf(v, u);
            }
        largest = __shfl_sync(0xffffffffu, v, 0);
        return __shfl_sync(0xffffffffu, v, a.keep - 1);
    };
    // A logit that `keep` of this batch's are not below: the keep-th largest of the maxima of 32 groups of
    // eight threads, sorted by every warp, or of the threads'. And the largest.
    auto batch_bound = [&](float mine, float& largest) {
        if (a.keep > 16) {
            const float r = nth(mine, a.keep);
            largest = nth(mine, 1);
            return r;
        }
        float v = mine;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        if ((lane & 7) == 0) tops[tid >> 3] = v;
        __syncthreads();
        return sorted(tops[lane], largest);
    };
    // The same of a list in any order, a word a thread: the groups go by the words' places, so that the
    // bound, and with it what enters the sum once more, is the same in every run.
    auto list_bound = [&](float mine, int place) {
        if (a.keep > 16) return nth(mine, a.keep);
        if (tid < 32) group[tid] = 0u;
        __syncthreads();
        if (mine > NEG) atomicMax(&group[place & 31], key_of(mine));
        __syncthreads();
        const uint32_t k = group[lane];
        float largest;
        return sorted(k == 0u ? NEG : __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k), largest);
    };

    float top = NEG, bound = NEG;  // of this thread; of the CTA
    // What a thread takes off its exponents: the first batch's largest, raised where one lies far above.
    float zt = NEG;
    uint32_t far2 = 0;
    hl::f2 s2 = 0ull;
    bool crowded = false;
    const hl::f2 K2 = hl::pk1(a.K);
    const uint32_t near2 = CAP ? W::packed(a.near) : 0u;
    // at this logit (not below the bound) a shift is raised; none is where the cap keeps all within range
    auto far_of = [&](float x) { return W::packed_up(CAP && 2.f * a.cap_K < FAR ? INFINITY : x + a.far); };
    auto z_of = [&](float x) { return CAP ? a.cap_K * tanhf(x * a.inv_cap) : x * a.K; };
    // Each thread copies and reads its own words, so that its own wait is all the copies need.
    auto fetch = [&](int jb, int stage) {
        const int je = min(j1, jb + SLICE_WORDS);
        const bool inside = jb * W::PER >= off && je * W::PER - off <= a.V;  // no word is shared with a neighbour
        const char* at = base + (int64_t(jb + tid) * W::PER - off) * W::SIZE;
        const uint32_t own = uint32_t(__cvta_generic_to_shared(&ring[stage * WORDS * ST + tid]));
        if (inside && jb + SLICE_WORDS == je) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(own + i * ST * 16), "l"(at + i * ST * 16)
                             : "memory");
            asm volatile("cp.async.commit_group;" ::: "memory");
            return;
        }
#pragma unroll 1
        for (int i = 0; i < WORDS; ++i) {
            const int j = jb + i * ST + tid;
            if (j < je) {
                const int lo = j * W::PER - off;
                uint4* to = &ring[(stage * WORDS + i) * ST + tid];
                if (inside || (lo >= 0 && lo + W::PER <= a.V)) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(to))),
                                 "l"(at + i * ST * 16)
                                 : "memory");
                } else {
                    uint32_t w[4] = {W::NONE, W::NONE, W::NONE, W::NONE};
                    W::edge(base, lo, a.V, w);
                    *to = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else if (j < je + 2 * ST) {
                ring[(stage * WORDS + i) * ST + tid] = make_uint4(W::NONE, W::NONE, W::NONE, W::NONE);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (j0 < j1) fetch(j0, 0);
    int stage = 0, turn = 0;
#pragma unroll 1
    for (int jb = j0; jb < j1 && !crowded; jb += SLICE_WORDS, stage ^= 1) {
        const int je = min(j1, jb + SLICE_WORDS);
        if (je < j1) {
            fetch(je, stage ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        const int pairs = (je - jb + 2 * ST - 1) / (2 * ST);  // of words a thread
        auto word = [&](int i, uint32_t (&w)[4]) {
            const uint4 u = ring[(stage * WORDS + i) * ST + tid];
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        };
        // (a NaN loses every comparison; of a word of NaNs alone it stays, and reaches any bound)
        auto word_top = [&](const uint32_t (&w)[4]) { return W::top2(W::top2(w[0], w[1]), W::top2(w[2], w[3])); };
        if (!(zt > NEG)) {  // nothing was allowed so far
            uint32_t t = W::NONE;
#pragma unroll 2
            for (int i = 0; i < 2 * pairs; ++i) {
                uint32_t w[4];
                word(i, w);
                t = W::top2(t, word_top(w));
            }
            float largest;
            bound = batch_bound(W::top_of(t), largest);
            __syncthreads();
            if (!(largest > NEG)) continue;
            zt = z_of(largest);
            if (!(zt > NEG)) zt = -3e38f;  // (the sum is taken again below)
            far2 = far_of(largest);
        }
        // three counters in turn: one barrier a batch stands between a counter's pushes, reads and reset
        int* pushed = &more_hits[turn];
        turn = turn == 2 ? 0 : turn + 1;
        uint32_t bound2 = W::packed(bound), all = W::NONE;  // (exact: the bound is a logit)
#pragma unroll 2
        for (int i = 0; i < 2 * pairs; i += 2) {
            uint32_t w[2][4];
            word(i, w[0]);
            word(i + 1, w[1]);
            const uint32_t t0 = word_top(w[0]), t1 = word_top(w[1]), t = W::top2(t0, t1);
            all = W::top2(all, t);
            int any = 0;
            if (CAP) any = !__all_sync(0xffffffffu, W::within(w[0], w[1], near2));
            // the words with a candidate go to a list, so that the code for them exists once
            if (W::reaches(t, bound2)) {
                const float x = W::top_of(t);
                if (W::reaches(t, far2) && x > NEG) {  // (not a NaN)
                    const float z = z_of(x);
                    s2 = hl::mul2(s2, hl::pk1(hl::ex2f(zt - z)));
                    zt = z;
                    far2 = far_of(x);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (W::reaches(k ? t1 : t0, bound2)) {
                        const int p = hits + atomicAdd(pushed, 1);
                        if (p < HITS) {
                            hit[p] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                            hit_at[p] = (jb + (i + k) * ST + tid) * 2 | any;
                        }
                    }
            }
            hl::f2 x[W::PER];
            W::unpack(w[0], x);
            W::unpack(w[1], x + W::PER / 2);
            if (CAP && any) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < W::PER; ++e) {
                    float lo, hi;
                    hl::upk(x[e], lo, hi);
                    s += mass_any(lo, zt, a) + mass_any(hi, zt, a);
                }
                s2 = hl::add2(s2, hl::pk(s, 0.f));
            } else if (CAP) {
                s2 = hl::add2(s2, mass_near(x, hl::pk1(-zt), a));
            } else {
                const hl::f2 minus_zt = hl::pk1(-zt);
#pragma unroll
                for (int e = 0; e < W::PER; ++e) s2 = hl::add2(s2, hl::ex2p(hl::fma2(x[e], K2, minus_zt)));
            }
        }
        top = fmaxf(top, W::top_of(all));
        __syncthreads();
        int listed = hits + *pushed;
        if (tid == 0) more_hits[turn == 2 ? 0 : turn + 1] = 0;
        if (listed > HITS) {  // more than fit (a row that rises): once more with this batch's own bound
            float largest;
            bound = fmaxf(bound, batch_bound(W::top_of(all), largest));
            __syncthreads();
            if (tid == 0) *pushed = 0;
            __syncthreads();
            bound2 = W::packed(bound);
#pragma unroll 1
            for (int i = 0; i < 2 * pairs; i += 2) {
                uint32_t w[2][4];
                word(i, w[0]);
                word(i + 1, w[1]);
                int any = 0;  // as above: which way their masses were taken
                if (CAP) any = !__all_sync(0xffffffffu, W::within(w[0], w[1], near2));
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (W::reaches(word_top(w[k]), bound2)) {
                        const int p = hits + atomicAdd(pushed, 1);
                        if (p < HITS) {
                            hit[p] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                            hit_at[p] = (jb + (i + k) * ST + tid) * 2 | any;
                        }
                    }
            }
            __syncthreads();
            listed = hits + *pushed;
            crowded = listed > HITS;
            __syncthreads();
        }
        hits = listed;
        // The list thinned out, before it is full and at the end: the keep-th largest of its words' maxima is
        // a bound too.
        if (hits > (je < j1 ? HITS / 2 : MANY) && hits > a.keep && !crowded) {
            uint4 h = make_uint4(W::NONE, W::NONE, W::NONE, W::NONE);
            int h_at = 0;
            if (tid < hits) h = hit[tid], h_at = hit_at[tid];
            const float u = W::top_of(W::top2(W::top2(h.x, h.y), W::top2(W::top2(h.z, h.w), W::NONE)));
            if (tid == 0) count = 0;
            bound = fmaxf(bound, list_bound(u, h_at >> 1));
            if (u >= bound && u > NEG) {
                const int p = atomicAdd(&count, 1);
                hit[p] = h;
                hit_at[p] = h_at;
            }
            __syncthreads();
            hits = count;
            __syncthreads();
            if (tid == 0) count = 0;
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // the slice's largest logit, and its sum: of each warp and its shift
    float sum = hl::hsum(s2), zw = zt;
#pragma unroll
    for (int o = 16; o; o >>= 1) zw = fmaxf(zw, __shfl_xor_sync(0xffffffffu, zw, o));
    sum = zt > NEG ? sum * hl::ex2f(zt - zw) : 0.f;  // (each thread's is its own)
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (lane == 0) part[warp] = sum, shift[warp] = zw, tops[warp] = top;
    __syncthreads();
    top = NEG;
#pragma unroll
    for (int k = 0; k < ST / 32; ++k) top = fmaxf(top, tops[k]);
    if (top == NEG) {  // nothing is allowed here
        if (tid == 0) *head = Head{NEG, 0.f, 0, 0};
        return;
    }
    zt = CAP ? a.cap_K * tanhf(top * a.inv_cap) : top * a.K;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < ST / 32; ++k)
        if (shift[k] > NEG) sum += part[k] * hl::ex2f(shift[k] - zt);
    // 2^(top K - zt) is taken off again: zt was rounded
    if (!CAP) sum *= hl::ex2f(-fmaf(top, a.K, -zt));
    long long more = 0;  // in units of 2^-40: the list's order is not the same in every run, so it must not matter
    if (!crowded) {
        const int n = hits;
        for (int k = tid; k < n * W::PER; k += ST) {
            const int h = k / W::PER, e = k % W::PER;
            const float x = W::value(reinterpret_cast<const char*>(&hit[h]), e);
            if (x >= bound && x > NEG) {
                const int p = atomicAdd(&count, 1);
                if (p < a.cap_list) cands[p] = Cand{x, (hit_at[h] >> 1) * W::PER - off + e};
                if (CAP) {
                    // the candidates have most of the mass: theirs enters more exactly, relative to the
                    // largest logit's own z
                    const hl::f2 one[1] = {hl::pk1(x)};
                    const float went = hit_at[h] & 1 ? mass_any(x, zt, a) : hl::lo_of(mass_near(one, hl::pk1(-zt), a));
                    more += __float2ll_rn((exp2f(fall<CAP>(x, top, a.cap, a.inv_cap) * a.K) - went) * 0x1p40f);
                }
            }
        }
    }
    if (CAP) {
#pragma unroll
        for (int o = 16; o; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
        if (lane == 0) extra[warp] = more;
    }
    __syncthreads();
    if (CAP) {
        more = 0;
#pragma unroll
        for (int k = 0; k < ST / 32; ++k) more += extra[k];
        sum += float(more) * 0x1p-40f;
    }
    int n = count;
    const int e0 = max(0, j0 * W::PER - off), e1 = min(a.V, j1 * W::PER - off);
    // not all was summed; a NaN, an infinity, zt beyond fp32; a cap that the passes above are too coarse for
    if (crowded || (CAP && a.precise) || !(sum > 0.5f && sum < INFINITY)) {
        float s = 0.f;
#pragma unroll 1
        for (int e = e0 + tid; e < e1; e += ST) {
            const float x = W::value(base, e);
            if (x > NEG) top = fmaxf(top, x);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        __syncthreads();
        if (lane == 0) tops[warp] = top;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < ST / 32; ++k) top = fmaxf(top, tops[k]);
#pragma unroll 1
        for (int e = e0 + tid; e < e1; e += ST) {
            const float x = W::value(base, e);
            if (x > NEG) s += exp2f(fall<CAP>(x, top, a.cap, a.inv_cap) * a.K);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        __syncthreads();
        if (lane == 0) part[warp] = s;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < ST / 32; ++k) sum += part[k];
    }
    if (crowded || n > a.cap_list) {
        // Many equal logits (or hardly any groups with one): the keep-th largest by bisection of the
        // ordered bits, then the lowest indices of those that equal it.
        // The slice is read again for it, so that the usual way keeps its registers.
        auto counted = [&](auto take) {
            int c = 0;
#pragma unroll 1
            for (int e = e0 + tid; e < e1; e += ST) {
                const float x = W::value(base, e);
                c += x > NEG && take(key_of(x), e);
            }
            c = __reduce_add_sync(0xffffffffu, c);
            __syncthreads();
            if (lane == 0) found[warp] = c;
            __syncthreads();
            c = 0;
#pragma unroll
            for (int k = 0; k < ST / 32; ++k) c += found[k];
            return c;
        };
        uint32_t T = 0;
#pragma unroll 1
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t t = T | 1u << bit;
            if (counted([&](uint32_t k, int) { return k >= t; }) >= a.keep) T = t;
        }
        const int need = a.keep - counted([&](uint32_t k, int) { return k > T; });
        int J = 0;
#pragma unroll 1
        for (int bit = 30; bit >= 0; --bit) {
            const int t = J | 1 << bit;
            if (counted([&](uint32_t k, int at) { return k == T && at < t; }) < need) J = t;
        }
        if (tid == 0) count = 0;
        __syncthreads();
#pragma unroll 1
        for (int e = e0 + tid; e < e1; e += ST) {
            const float x = W::value(base, e);
            const uint32_t k = key_of(x);
            if (x > NEG && (k > T || (k == T && e <= J))) {
                const int p = atomicAdd(&count, 1);
                if (p < a.cap_list) cands[p] = Cand{x, e};
            }
        }
        __syncthreads();
        n = count;
    }
    if (tid == 0) *head = Head{top, sum, min(n, a.cap_list), 0};
}

// ----------------------------------------------------------------- merge ----

struct Best {
    uint64_t key;   // of the fp64 score
    int beam;
    float x;
    int token;
};
// Whether a stands before b.
__device__ __forceinline__ bool before(const Best& a, const Best& b) {
    if (a.key != b.key) return a.key > b.key;
    if (a.beam != b.beam) return a.beam < b.beam;
    if (a.x != b.x) return a.x > b.x;
    return a.token < b.token;
}

constexpr int LISTS = 256, HELD = 1920;  // lists and candidates that are held in shared memory
constexpr uint64_t NO_KEY = 0;  // below every score that a candidate can have

__global__ void __launch_bounds__(MT) merge_kernel(const Args a) {
    __shared__ double log_mass[MAX_BEAMS], before_of[MAX_BEAMS];
    __shared__ float top_of[MAX_BEAMS], log_of[MAX_BEAMS];
    __shared__ double tanh_top[MAX_BEAMS];
    __shared__ uint8_t kind[MAX_BEAMS];  // 0: no candidates, 1: its row's, 2: ended
    __shared__ int size_of[LISTS], begin_of[LISTS + 1];
    __shared__ float high_of[HELD];
    __shared__ Cand cand_of[HELD];
    __shared__ uint8_t beam_of[HELD];
    __shared__ uint16_t alive[LIST];
    __shared__ int survivors;
    __shared__ Best list[LIST];
    __shared__ Best kept[MAX_KEEP];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r = blockIdx.x;
    const int B = a.beams, S = a.slices;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Head* heads = a.heads + r * B * S;
    const Cand* cands = a.cands + r * B * S * a.cap_list;
    if (tid == 0) count = survivors = 0;
    // the beams' sums: a warp a beam
    for (int b = warp; b < B; b += MT / 32) {
        const float s = a.scores[r * B + b];
        const bool over = a.ended && a.ended[r * B + b];
        const bool live = s > NEG;
        if (live && !over) {
            float top = NEG;
            for (int k = lane; k < S; k += 32) top = fmaxf(top, heads[b * S + k].top);
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float total = 0.f;
            if (top > NEG)
                for (int k = lane; k < S; k += 32) {
                    const Head h = heads[b * S + k];
                    if (h.top > NEG) {
                        const float d = a.cap > 0.f ? fall<true>(h.top, top, a.cap, a.inv_cap)
                                                    : fall<false>(h.top, top, 0.f, 0.f);
                        total += h.sum * exp2f(d * a.K);
                    }
                }
#pragma unroll
            for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (lane == 0) {
                kind[b] = top > NEG;
                top_of[b] = top;
                log_of[b] = total;
            }
        } else if (lane == 0) {
            kind[b] = live ? 2 : 0;
        }
        if (lane == 0) before_of[b] = double(s);
    }
    __syncthreads();
    // fp64 takes as long for one lane as for a warp: a lane a beam
    if (tid < B && kind[tid] == 1) {
        log_mass[tid] = log(double(log_of[tid]));
        log_of[tid] = float(log_mass[tid]);
    }
    if (a.cap > 0.f && tid >= MAX_BEAMS && tid < MAX_BEAMS + B && kind[tid - MAX_BEAMS] == 1)
        tanh_top[tid - MAX_BEAMS] = tanh(double(top_of[tid - MAX_BEAMS]) / a.cap);
    __syncthreads();

    // An entry's score in fp64, and in fp32 with a bound of its error.
    auto exact = [&](int b, const Cand& c) {
        Best t;
        t.beam = b;
        t.x = c.x;
        t.token = c.at;
        double d;
        if (c.x == top_of[b]) d = 0.0;
        else if (a.cap == 0.f) d = double(c.x) - double(top_of[b]);
        else d = double(a.cap) * (tanh(double(c.x) / a.cap) - tanh_top[b]);
        const double s = before_of[b] + (d * double(a.scale) - log_mass[b]);
        t.key = s > -INFINITY ? key_of(s) : NO_KEY;
        return t;
    };
    auto ended = [&](int b) {
        return Best{key_of(before_of[b]), b, 0.f, int(a.eos)};
    };
    // tanh by two MUFU operations is within 2^-21, so the score within 2^-20 of its parts
    auto rough = [&](int b, float x, float& off) {
        const float s = float(before_of[b]), l = log_of[b];
        float d = x - top_of[b];
        if (a.cap > 0.f) {
            const float y = x * a.inv_cap, w = hl::ex2f(-2.8853900817779268f * fabsf(y));
            d = a.cap * (copysignf((1.f - w) * hl::rcpf(1.f + w), y) - float(tanh_top[b]));
        }
        d = x == top_of[b] ? 0.f : d * a.scale;
        off = 9.5367432e-7f * (fabsf(s) + fabsf(d) + fabsf(l) + a.cap * a.scale + 1.f);
        return s + (d - l);
    };
    // f(beam, entry) for every candidate of the rows: a warp a list
    auto each = [&](auto f) {
        for (int l = warp; l < B * S; l += MT / 32) {
            const int b = l / S;
            if (kind[b] != 1) continue;
            const int n = heads[l].n;
            for (int e = lane; e < n; e += 32) f(b, cands[int64_t(l) * a.cap_list + e]);
        }
    };
    // The candidates once more in shared memory, where they fit; else they are read twice.
    const int lists = B * S;
    const bool fits = lists <= LISTS;
    int entries = 0;
    if (fits) {
        if (tid < lists) size_of[tid] = kind[tid / S] == 1 ? heads[tid].n : 0;
        __syncthreads();
        if (warp == 0) {  // where each list begins
            int run = 0;
            for (int l0 = 0; l0 < lists; l0 += 32) {
                const int n = l0 + lane < lists ? size_of[l0 + lane] : 0;
                int up = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane >= o) up += u;
                }
                if (l0 + lane < lists) begin_of[l0 + lane] = run + up - n;
                run += __shfl_sync(0xffffffffu, up, 31);
            }
            if (lane == 0) begin_of[lists] = run;
        }
        __syncthreads();
        entries = begin_of[lists];
    }
    const bool held = fits && entries <= HELD;
    // a bound: `keep` threads have a candidate whose score is not below it
    float mine = NEG;
    if (held) {
        for (int l = warp; l < lists; l += MT / 32) {
            const int b = l / S, n = size_of[l], at = begin_of[l];
            for (int e = lane; e < n; e += 32) {
                const Cand c = cands[int64_t(l) * a.cap_list + e];
                float off;
                const float s = rough(b, c.x, off), high = s + off;
                // (an overflow or NaN is left to fp64)
                high_of[at + e] = high > NEG ? high : INFINITY;
                cand_of[at + e] = c;
                beam_of[at + e] = uint8_t(b);
                mine = fmaxf(mine, s - off);
            }
        }
    } else {
        each([&](int b, const Cand& c) {
            float off;
            const float s = rough(b, c.x, off);
            mine = fmaxf(mine, s - off);
        });
    }
    if (tid < B && kind[tid] == 2) mine = fmaxf(mine, float(before_of[tid]));
    const uint32_t my_key = mine > NEG ? key_of(mine) : 0u;
    uint32_t T = 0;
    for (int bit = 31; bit >= 8; --bit) {  // from below, to 16 bits of the fraction
        const uint32_t t = T | 1u << bit;
        if (__syncthreads_count(my_key >= t) >= a.keep) T = t;
    }
    auto offer_list = [&](int b, const Cand& c) {
        const Best t = exact(b, c);
        if (t.key != NO_KEY) {
            const int p = atomicAdd(&count, 1);
            if (p < LIST) list[p] = t;
        }
    };
    if (held) {  // the survivors' places first, so that fp64 runs in full warps
        for (int e = tid; e < entries; e += MT)
            if (key_of(high_of[e]) >= T) {
                const int p = atomicAdd(&survivors, 1);
                if (p < LIST) alive[p] = uint16_t(e);
            }
        __syncthreads();
        if (survivors <= LIST) {
            if (tid < survivors) offer_list(beam_of[alive[tid]], cand_of[alive[tid]]);
        } else if (tid == 0) {
            count = LIST + 1;
        }
    } else {
        each([&](int b, const Cand& c) {
            float off;
            const float s = rough(b, c.x, off), high = s + off;
            if (!(high > NEG) || key_of(high) >= T) offer_list(b, c);
        });
    }
    if (tid < B && kind[tid] == 2) {
        const int p = atomicAdd(&count, 1);
        if (p < LIST) list[p] = ended(tid);
    }
    __syncthreads();
    const int n = count;
    __syncthreads();
    int m = min(n, a.keep);
    if (n <= LIST) {
        if (tid < n) {
            const Best t = list[tid];
            int rank = 0;
            for (int k = 0; k < n; ++k) rank += before(list[k], t);
            if (rank < m) kept[rank] = t;
        }
    } else {
        // Too many to rank (rows of equal logits): the best one after the last, `keep` times.
        for (int k = 0; k < a.keep; ++k) {
            const Best last = k ? kept[k - 1] : Best{~uint64_t(0), -1, INFINITY, -1};
            Best best = {NO_KEY, MAX_BEAMS, NEG, INT32_MAX};
            auto offer = [&](const Best& t) {
                if (t.key != NO_KEY && (k == 0 || before(last, t)) && before(t, best)) best = t;
            };
            each([&](int b, const Cand& c) { offer(exact(b, c)); });
            if (tid < B && kind[tid] == 2) offer(ended(tid));
            list[tid] = best;
            __syncthreads();
            for (int o = MT / 2; o; o >>= 1) {
                if (tid < o && before(list[tid + o], list[tid])) list[tid] = list[tid + o];
                __syncthreads();
            }
            if (tid == 0) kept[k] = list[0];
            __syncthreads();
            if (kept[k].key == NO_KEY) {  // the others score -inf: fewer candidates than `keep`
                m = k;
                break;
            }
        }
    }
    __syncthreads();
    // places: in order, or a parent's first child in its place
    __shared__ int place[MAX_KEEP];
    if (a.stay) {
        if (tid == 0) {
            uint64_t taken = 0;
            for (int k = 0; k < m; ++k) {
                const uint64_t bit = uint64_t(1) << kept[k].beam;
                place[k] = taken & bit ? -1 : kept[k].beam;
                taken |= bit;
            }
            int next = 0;
            for (int k = 0; k < a.keep; ++k)
                if (k >= m || place[k] < 0) {
                    while (taken >> next & 1) ++next;
                    place[k] = next;
                    taken |= uint64_t(1) << next;
                }
        }
        __syncthreads();
    }
    if (tid < a.keep) {
        const int64_t at = r * a.keep + (a.stay ? place[tid] : tid);
        if (tid < m) {
            const Best t = kept[tid];
            const uint64_t b = t.key >> 63 ? t.key & ~(uint64_t(1) << 63) : ~t.key;
            a.out_scores[at] = float(__longlong_as_double(int64_t(b)));
            a.parents[at] = t.beam;
            a.tokens[at] = t.token;
            if (a.out_ended) a.out_ended[at] = a.eos >= 0 && t.token == a.eos;
        } else {
            a.out_scores[at] = NEG;
            a.parents[at] = -1;
            a.tokens[at] = -1;
            if (a.out_ended) a.out_ended[at] = 0;
        }
    }
}

// ------------------------------------------------------------------ host ----

constexpr int64_t FILL = 900;  // CTAs: about three an SM, twice

struct Plan {
    int slices, cap_list;
    int64_t heads, bytes;
};
Plan plan_of(int64_t requests, int beams, int64_t V, int dtype, int keep) {
    Plan p;
    const int per = dtype == HEADLOSS_FP32 ? 4 : 8;
    const int64_t words = (V + per - 1 + per - 1) / per;  // of a row that starts anywhere in a word
    // batches of a row on CTAs of their own until those would fill three a SM twice
    const int64_t batches = (words + SLICE_WORDS - 1) / SLICE_WORDS, rows = requests * beams > 0 ? requests * beams : 1;
    const int64_t most = (FILL + rows - 1) / rows;
    p.slices = int(batches < most ? batches : most);
    p.cap_list = keep <= 16 ? 64 : 4 * keep;
    const int64_t n = requests * beams * p.slices;
    p.heads = n * int64_t(sizeof(Head));
    p.bytes = p.heads + n * p.cap_list * int64_t(sizeof(Cand));
    return p;
}
bool sizes_ok(int64_t requests, int beams, int64_t V, int keep) {
    return requests >= 0 && requests <= INT32_MAX && beams >= 1 && beams <= MAX_BEAMS && keep >= 1 &&
           keep <= MAX_KEEP && V >= 1 && V < (int64_t(1) << 31) - 4096 && requests * beams <= INT32_MAX;
}

template <int DT, bool CAP>
bool launch_slices(const Args& a, unsigned grid, cudaStream_t s) {
    if (cudaFuncSetAttribute(slice_kernel<DT, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, RING) != cudaSuccess)
        return false;
    slice_kernel<DT, CAP><<<grid, ST, RING, s>>>(a);
    return cudaGetLastError() == cudaSuccess;
}
template <int DT>
bool launch(const Args& a, unsigned grid, cudaStream_t s) {
    return a.cap > 0.f ? launch_slices<DT, true>(a, grid, s) : launch_slices<DT, false>(a, grid, s);
}

}  // namespace hl_beam

extern "C" int64_t headloss_beam_workspace(int64_t requests, int beams, int64_t V, int dtype, int keep) {
    using namespace hl_beam;
    if (!sizes_ok(requests, beams, V, keep) || dtype < HEADLOSS_FP32 || dtype > HEADLOSS_FP16) return -1;
    const Plan p = plan_of(requests, beams, V, dtype, keep);
    return requests * beams * p.slices > INT32_MAX ? -1 : p.bytes;
}

extern "C" int headloss_beam_select(const void* logits, int64_t requests, int beams, int64_t V, int64_t ld,
                                    int dtype, const float* scores, const uint8_t* ended, int64_t eos,
                                    int keep, int stay, float softcap, float logits_scale,
                                    float* out_scores, int32_t* parents, int64_t* tokens,
                                    uint8_t* out_ended, void* workspace, int64_t workspace_bytes,
                                    void* stream) {
    using namespace hl_beam;
    if (!sizes_ok(requests, beams, V, keep) || ld < V || eos < -1 || eos >= V || (ended && eos < 0) ||
        (stay != 0 && stay != 1) || (stay && keep != beams))
        return HEADLOSS_ERR_ARG;
    if (!(softcap >= 0.f) || !isfinite(softcap) || !(logits_scale > 0.f) || !isfinite(logits_scale))
        return HEADLOSS_ERR_ARG;
    const float inv_cap = softcap > 0.f ? float(1.0 / double(softcap)) : 0.f;
    const float K = float(double(logits_scale) * 1.4426950408889634);
    if (!isfinite(inv_cap) || !isfinite(K)) return HEADLOSS_ERR_ARG;
    if (dtype != HEADLOSS_FP32 && dtype != HEADLOSS_BF16 && dtype != HEADLOSS_FP16) return HEADLOSS_ERR_DTYPE;
    if (requests == 0) return HEADLOSS_OK;
    if (!logits || !scores || !out_scores || !parents || !tokens || !workspace) return HEADLOSS_ERR_ARG;
    auto bits = [](const void* q) { return reinterpret_cast<uintptr_t>(q); };
    if ((bits(logits) & (dtype == HEADLOSS_FP32 ? 3u : 1u)) || (bits(tokens) & 7u) || (bits(workspace) & 15u) ||
        ((bits(scores) | bits(out_scores) | bits(parents)) & 3u))
        return HEADLOSS_ERR_ALIGN;
    const Plan p = plan_of(requests, beams, V, dtype, keep);
    const int64_t grid = requests * beams * p.slices;
    if (grid > INT32_MAX || workspace_bytes < p.bytes) return HEADLOSS_ERR_ARG;
    Args a = {};
    a.logits = logits;
    a.ld = ld;
    a.V = int(V);
    a.scores = scores;
    a.ended = ended;
    a.eos = eos;
    a.beams = beams;
    a.keep = keep;
    a.stay = stay;
    a.cap = softcap;
    a.inv_cap = inv_cap;
    a.scale = logits_scale;
    a.K = K;
    a.cap_K = softcap * K;
    a.far = FAR / K;
    // Both fast ways to tanh are off by a share of the cap, up to 2^-21 of cap * scale in an exponent (a score of rows
    // whose logits lie at a third of the cap: 2e-6 at a cap of 30, 3e-5 at 1000, 5e-3 at 1e5). Above PRECISE a slice is
    // read again and its sum taken from differences: 2048 x 151936 bf16 3.3 ms, and 0.20.
    a.precise = double(softcap) * double(logits_scale) > PRECISE;
    // a cap whose powers leave fp32's normal range takes the other way to tanh throughout
    const double C[6] = {HL_TANH_B_C0, HL_TANH_B_C1, HL_TANH_B_C2, HL_TANH_B_C3, HL_TANH_B_C4, HL_TANH_B_C5};
    bool fits = softcap > 0.f;
    for (int i = 0; fits && i < 6; ++i) {
        const float c = float(C[i] * double(K) / pow(double(softcap), 2 * i));
        uint32_t u;
        memcpy(&u, &c, 4);
        a.poly[i] = uint64_t(u) << 32 | u;
        fits = isnormal(c);
    }
    a.near = fits ? HL_TANH_B_Y0 * softcap : -1.f;
    a.slices = p.slices;
    a.cap_list = p.cap_list;
    a.heads = static_cast<Head*>(workspace);
    a.cands = reinterpret_cast<Cand*>(static_cast<char*>(workspace) + p.heads);
    a.out_scores = out_scores;
    a.parents = parents;
    a.tokens = tokens;
    a.out_ended = out_ended;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool ok = dtype == HEADLOSS_FP32   ? launch<HEADLOSS_FP32>(a, unsigned(grid), s)
                    : dtype == HEADLOSS_BF16 ? launch<HEADLOSS_BF16>(a, unsigned(grid), s)
                                             : launch<HEADLOSS_FP16>(a, unsigned(grid), s);
    if (!ok) return HEADLOSS_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(requests));
    cfg.blockDim = dim3(MT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge_kernel, a) == cudaSuccess ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
}
