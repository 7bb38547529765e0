// hl_sample.cu -- drawing tokens from the head's logits (headloss_sample in
// include/headloss_sample.h, where the definition stands).
//
// One CTA a row, the row read from global memory in every pass:
//   largest logit; with top-k or top-p the cut of the order (x descending,
//   index ascending) by radix selection on the sortable key, eight bits a
//   level, counts and integer masses a bin; kept mass; the target's segment
//   and token by prefix sums in index order.
// The three filters keep a prefix of the order, so a row's kept set is a key
// tau, how many of the tokens at tau stay (the first by index), and min-p's
// comparison.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <math.h>
#include <stdint.h>

#include "headloss.h"
#include "headloss_sample.h"

namespace hl_sample {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr float UNIT = 1073741824.f;  // 2^30, the weight of the largest logit
constexpr double LOG2E = 1.4426950408889634;
constexpr float LN2 = 0.69314718055994531f;

struct Args {
    const void* logits;
    int64_t ld;
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

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

// A key whose unsigned order is the order of the floats; -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T* red, F f) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < WARPS; ++i) v = f(v, red[i]);
    return v;
}

// One row's view: a logit's sortable key and its integer weight.
template <typename DT>
struct Row {
    const DT* x;
    float cap, inv_cap, zm, c;
    __device__ float at(int j) const {
        const float v = to_f(x[j]);
        return v == v ? v : -CUDART_INF_F;
    }
    __device__ float z(float v) const {
        return cap > 0.f ? __fmul_rn(tanhf(__fmul_rn(v, inv_cap)), cap) : v;
    }
    __device__ float d(float v) const {
        const float zz = z(v);
        return zz == zm ? 0.f : __fmul_rn(__fsub_rn(zz, zm), c);
    }
    __device__ float e(float v) const { return v == -CUDART_INF_F ? 0.f : exp2f(d(v)); }
    __device__ static uint32_t weight(float e) { return __float2uint_rn(__fmul_rn(e, UNIT)); }
};

struct Cut {
    uint32_t key;  // tokens above the key stay, and
    int ties;      // this many at the key, the first by index
};

// The cut after the first tokens of the order whose count before them is below
// k (by_mass = false) or whose mass before them is below target.  Only tokens above
// `floor` are looked at; found = false where they are too few.
template <typename DT>
__device__ bool select(const Row<DT>& r, int V, bool by_mass, int64_t k, double target,
                       uint32_t floor, uint32_t* cnt, unsigned long long* mass, Cut* out,
                       unsigned long long* above_out) {
    __shared__ uint32_t s_digit;
    __shared__ unsigned long long s_before;
    __shared__ int s_found;
    uint32_t prefix = 0;
    unsigned long long before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += THREADS) cnt[i] = 0, mass[i] = 0;
        if (threadIdx.x == 0) s_found = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < V; j += THREADS) {
            const float v = r.at(j);
            const uint32_t key = key_of(v);
            if (key <= floor) continue;
            if (shift < 24 && (key >> (shift + 8)) != prefix) continue;
            const uint32_t b = (key >> shift) & 255u;
            atomicAdd(&cnt[b], 1u);
            if (by_mass) {
                const uint32_t w = r.weight(r.e(v));
                if (w) atomicAdd(&mass[b], (unsigned long long)w);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned long long m = before;
            for (int b = 255; b >= 0; --b) {
                if (!cnt[b]) continue;
                const unsigned long long n = m + (by_mass ? mass[b] : cnt[b]);
                if (by_mass ? double(n) >= target : int64_t(n) >= k) {
                    s_digit = b;
                    s_before = m;
                    s_found = 1;
                    break;
                }
                m = n;
            }
        }
        __syncthreads();
        if (!s_found) return false;
        prefix = (shift < 24 ? prefix << 8 : 0u) | s_digit;
        before = s_before;
        __syncthreads();
    }
    // all at one key: the same logit, so the same weight each
    if (threadIdx.x == 0) {
        out->key = prefix;
        const uint32_t n = cnt[prefix & 255u];
        if (by_mass) {
            const unsigned long long w = mass[prefix & 255u] / n;
            uint32_t t = 0;
            while (t < n && double(before + t * w) < target) ++t;
            out->ties = int(t);
        } else {
            out->ties = int(k - int64_t(before));
        }
        *above_out = before;
    }
    __syncthreads();
    return true;
}

template <typename DT>
__global__ void __launch_bounds__(THREADS) sample_kernel(Args a) {
    __shared__ uint32_t cnt[256];
    __shared__ unsigned long long mass[256];
    __shared__ unsigned long long red[WARPS];
    __shared__ float fred[WARPS];
    __shared__ int ired[WARPS];
    __shared__ Cut s_cut, s_kcut;
    __shared__ unsigned long long s_above;
    __shared__ int s_token;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
    Row<DT> r{reinterpret_cast<const DT*>(a.logits) + row * a.ld, a.cap, a.inv_cap, 0.f, 0.f};

    const float temp = a.temperature ? a.temperature[row] : 1.f;
    const double u = a.uniforms[row];
    int64_t k = a.top_k ? a.top_k[row] : 0;
    float p = a.top_p ? a.top_p[row] : 1.f;
    const float least = a.min_p ? a.min_p[row] : 0.f;
    const bool bad = !(temp >= 0.f && temp < CUDART_INF_F) || !(u >= 0.0 && u < 1.0) ||
                     !(p >= 0.f) || !(least >= 0.f && least <= 1.f);
    float top = -CUDART_INF_F;
    for (int j = tid; j < V; j += THREADS) top = fmaxf(top, r.at(j));
    top = block_reduce(top, fred, [](float x, float y) { return fmaxf(x, y); });
    if (bad || top == -CUDART_INF_F) {
        if (tid == 0) {
            a.tokens[row] = -1;
            if (a.logprobs) a.logprobs[row] = 0.f;
            if (a.draw_logprobs) a.draw_logprobs[row] = 0.f;
            if (a.n_kept) a.n_kept[row] = 0;
            if (bad) atomicOr(a.err, 1);
        }
        return;
    }
    r.zm = r.z(top);
    r.c = __fdiv_rn(a.K, temp);
    if (!(r.c < CUDART_INF_F)) {  // greedy
        r.c = a.K;
        k = 1;
    }
    if (k <= 0 || k > V) k = V;

    // the cut of the order
    Cut cut{0u, V};
    if (k < V) {
        select(r, V, false, k, 0.0, 0u, cnt, mass, &s_kcut, &s_above);
        cut = s_kcut;
    }
    if (p < 1.f) {
        unsigned long long m = 0;
        uint32_t wk = 0;
        for (int j = tid; j < V; j += THREADS) {
            const float v = r.at(j);
            if (key_of(v) > cut.key) m += r.weight(r.e(v));
            else if (key_of(v) == cut.key) wk = r.weight(r.e(v));
        }
        auto add = [](unsigned long long x, unsigned long long y) { return x + y; };
        m = block_reduce(m, red, add);
        wk = uint32_t(block_reduce((unsigned long long)wk, red,
                                   [](unsigned long long x, unsigned long long y) {
                                       return x > y ? x : y;
                                   }));
        const double target = double(p) * double(m + (k < V ? (unsigned long long)wk * cut.ties : 0));
        if (select(r, V, true, 0, target, cut.key, cnt, mass, &s_cut, &s_above)) {
            cut = s_cut;
        } else if (k < V) {  // the mass runs out among the ties of the top-k cut
            int t = 0;
            while (t < cut.ties && double(m + (unsigned long long)t * wk) < target) ++t;
            cut.ties = t;
        }
        if (p == 0.f || target == 0.0) cut = Cut{key_of(top), 1};
    }

    // kept mass by warp segments in index order (ties of the cut by index)
    const int seg = (V + WARPS - 1) / WARPS, j0 = min(V, warp * seg), j1 = min(V, j0 + seg);
    int eq = 0;
    for (int j = j0 + lane; j < j1; j += 32) eq += key_of(r.at(j)) == cut.key;
    for (int o = 16; o; o >>= 1) eq += __shfl_xor_sync(0xffffffffu, eq, o);
    __syncthreads();
    if (lane == 0) ired[warp] = eq;
    __syncthreads();
    int eq0 = 0;
    for (int i = 0; i < warp; ++i) eq0 += ired[i];
    unsigned long long m = 0;
    int kept = 0, e0 = eq0;
    float own = 0.f;
    for (int jj = j0; jj < j1; jj += 32) {
        const int j = jj + lane;
        const float v = j < j1 ? r.at(j) : -CUDART_INF_F;
        const uint32_t key = key_of(v);
        const unsigned tie = __ballot_sync(0xffffffffu, j < j1 && key == cut.key);
        const int nth = e0 + __popc(tie & ((1u << lane) - 1));
        e0 += __popc(tie);
        if (j < j1 && (key > cut.key || (key == cut.key && nth < cut.ties))) {
            const float e = r.e(v);
            const uint32_t w = e >= least ? r.weight(e) : 0u;
            m += w;
            kept += w > 0;
        }
        if (a.logprobs && v != -CUDART_INF_F) {
            const float z = r.z(v);
            own += z == r.zm ? 1.f : exp2f(__fmul_rn(__fsub_rn(z, r.zm), a.K));
        }
    }
    for (int o = 16; o; o >>= 1) {
        m += __shfl_xor_sync(0xffffffffu, m, o);
        kept += __shfl_xor_sync(0xffffffffu, kept, o);
        own += __shfl_xor_sync(0xffffffffu, own, o);
    }
    __syncthreads();
    if (lane == 0) red[warp] = m, ired[warp] = kept, fred[warp] = own;
    __syncthreads();
    unsigned long long W = 0, before = 0;
    kept = 0, own = 0.f;
    for (int i = 0; i < WARPS; ++i) {
        if (i == warp) before = W;
        W += red[i];
        kept += ired[i];
        own += fred[i];
    }
    unsigned long long t = (unsigned long long)floor(u * double(W));
    if (t > W - 1) t = W - 1;
    if (t < before || t >= before + m) return;
    // this warp's segment holds the token
    e0 = eq0;
    for (int jj = j0; jj < j1; jj += 32) {
        const int j = jj + lane;
        const float v = j < j1 ? r.at(j) : -CUDART_INF_F;
        const uint32_t key = key_of(v);
        const unsigned tie = __ballot_sync(0xffffffffu, j < j1 && key == cut.key);
        const int nth = e0 + __popc(tie & ((1u << lane) - 1));
        e0 += __popc(tie);
        uint32_t w = 0;
        if (j < j1 && (key > cut.key || (key == cut.key && nth < cut.ties))) {
            const float e = r.e(v);
            w = e >= least ? r.weight(e) : 0u;
        }
        unsigned long long sum = w;
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long n = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += n;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + sum > t);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                a.tokens[row] = j;
                const float z = r.z(v);
                if (a.logprobs)
                    a.logprobs[row] = (z == r.zm ? 0.f : __fsub_rn(z, r.zm) * a.K * LN2) - logf(own);
                if (a.draw_logprobs)
                    a.draw_logprobs[row] = r.d(v) * LN2 - logf(float(double(W) * (1.0 / UNIT)));
                if (a.n_kept) a.n_kept[row] = kept;
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
}

}  // namespace hl_sample

extern "C" int headloss_sample(const void* logits, int64_t N, int64_t V, int64_t ld, int dtype,
                               const double* uniforms, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p,
                               float softcap, float logits_scale, int64_t* tokens, float* logprobs,
                               float* draw_logprobs, int32_t* n_kept, int* err, void* stream) {
    using namespace hl_sample;
    if (N < 0 || N > INT32_MAX || V < 1 || V >= (int64_t(1) << 31) - 4096 || ld < V)
        return HEADLOSS_ERR_ARG;
    if (!(softcap >= 0.f) || !isfinite(softcap) || !(logits_scale > 0.f) || !isfinite(logits_scale))
        return HEADLOSS_ERR_ARG;
    if (dtype != HEADLOSS_FP32 && dtype != HEADLOSS_BF16 && dtype != HEADLOSS_FP16)
        return HEADLOSS_ERR_DTYPE;
    if (N == 0) return HEADLOSS_OK;
    if (!logits || !uniforms || !tokens || !err) return HEADLOSS_ERR_ARG;
    auto bits = [](const void* q) { return reinterpret_cast<uintptr_t>(q); };
    if ((bits(logits) & (dtype == HEADLOSS_FP32 ? 3u : 1u)) ||
        ((bits(uniforms) | bits(tokens)) & 7u) ||
        ((bits(temperature) | bits(top_k) | bits(top_p) | bits(min_p) | bits(logprobs) |
          bits(draw_logprobs) | bits(n_kept) | bits(err)) & 3u))
        return HEADLOSS_ERR_ALIGN;
    Args a;
    a.logits = logits;
    a.ld = ld;
    a.V = int(V);
    a.uniforms = uniforms;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.cap = softcap;
    a.inv_cap = softcap > 0.f ? float(1.0 / double(softcap)) : 0.f;
    a.K = float(double(logits_scale) * LOG2E);
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.draw_logprobs = draw_logprobs;
    a.n_kept = n_kept;
    a.err = err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == HEADLOSS_FP32) sample_kernel<float><<<unsigned(N), THREADS, 0, s>>>(a);
    else if (dtype == HEADLOSS_BF16) sample_kernel<__nv_bfloat16><<<unsigned(N), THREADS, 0, s>>>(a);
    else sample_kernel<__half><<<unsigned(N), THREADS, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? HEADLOSS_OK : HEADLOSS_ERR_CUDA;
}
