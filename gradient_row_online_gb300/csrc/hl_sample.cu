// hl_sample.cu -- headloss_sample's checks and dispatch (include/headloss_sample.h;
// the kernel is in hl_sample.cuh, instantiated a type a file).
#include <math.h>
#include <stdint.h>

#include "headloss_sample.h"
#include "hl_sample.cuh"

#ifdef HL_FAULT_INJECT
// Test builds alone: the calls that follow leave out the copies of row `drop_row` (-1: none), and
// their waits give up after `wait_ns` (0: the usual limit).
static int64_t g_drop_row = -1;
static unsigned long long g_wait_ns = hl_sample::WAIT_NS;
extern "C" void headloss_sample_test_inject(int64_t drop_row, unsigned long long wait_ns) {
    g_drop_row = drop_row;
    g_wait_ns = wait_ns ? wait_ns : hl_sample::WAIT_NS;
}
#endif

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
    // what the kernel multiplies by: with an infinity the row's largest logit would have no mass
    const float inv_cap = softcap > 0.f ? float(1.0 / double(softcap)) : 0.f;
    const float K = float(double(logits_scale) * 1.4426950408889634);
    if (!isfinite(inv_cap) || !isfinite(K)) return HEADLOSS_ERR_ARG;
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
    Args a = {};
    a.logits = logits;
    a.ld = ld;
    a.V = int(V);
    a.uniforms = uniforms;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.cap = softcap;
    a.inv_cap = inv_cap;
    a.K = K;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.draw_logprobs = draw_logprobs;
    a.n_kept = n_kept;
    a.err = err;
#ifdef HL_FAULT_INJECT
    a.drop_row = g_drop_row;
    a.wait_ns = g_wait_ns;
#endif
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return HEADLOSS_ERR_CUDA;
    return dtype == HEADLOSS_FP32   ? launch_fp32(a, N, device, sms, s)
           : dtype == HEADLOSS_BF16 ? launch_bf16(a, N, device, sms, s)
                                    : launch_fp16(a, N, device, sms, s);
}
