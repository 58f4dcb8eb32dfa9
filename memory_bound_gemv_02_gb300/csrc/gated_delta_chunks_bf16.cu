// The chunk kernels of the gated delta rule for bf16.
#include "gated_delta_chunks.cuh"

namespace gemvk {

int launch_delta_chunks_bf16(const DeltaParams &p, int dk_padded, bool gradient, int sms, cudaStream_t stream) {
  return dispatch<false>(p, dk_padded, gradient, sms, stream);
}

}  // namespace gemvk
