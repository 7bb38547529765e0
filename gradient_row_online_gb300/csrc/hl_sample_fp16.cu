// The sampling kernel for fp16 logits.
#include "hl_sample.cuh"

namespace hl_sample {

int launch_fp16(const Args& a, int64_t N, int device, int sms, cudaStream_t st) {
    return a.cap > 0.f ? launch<__half, true>(a, N, device, sms, st)
                       : launch<__half, false>(a, N, device, sms, st);
}

}  // namespace hl_sample
