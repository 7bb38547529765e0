// The sampling kernel for bf16 logits.
#include "hl_sample.cuh"

namespace hl_sample {

int launch_bf16(const Args& a, int64_t N, int device, int sms, cudaStream_t st) {
    return a.cap > 0.f ? launch<__nv_bfloat16, true>(a, N, device, sms, st)
                       : launch<__nv_bfloat16, false>(a, N, device, sms, st);
}

}  // namespace hl_sample
