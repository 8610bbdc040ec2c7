// Instantiations of the gradient's products for head dim 64.
#include "backward_kernel.cuh"

namespace gqa {

cudaError_t launch_bwd_d64(const BwdParams& p, bool bf16, cudaStream_t st) {
  return bf16 ? launch_backward<64, true>(p, st) : launch_backward<64, false>(p, st);
}

}  // namespace gqa
