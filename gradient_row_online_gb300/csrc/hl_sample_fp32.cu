// The sampling kernel for fp32 logits.
#include "hl_sample.cuh"

namespace hl_sample {

int launch_fp32(const Args& a, int64_t N, int device, int sms, cudaStream_t st) {
    return a.cap > 0.f ? launch<float, true>(a, N, device, sms, st)
                       : launch<float, false>(a, N, device, sms, st);
}

}  // namespace hl_sample
