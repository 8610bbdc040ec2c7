// Instantiations of the gradient's products for head dim 128.
#include "backward_kernel.cuh"

namespace gqa {

cudaError_t launch_bwd_d128(const BwdParams& p, bool bf16, cudaStream_t st) {
  return bf16 ? launch_backward<128, true>(p, st) : launch_backward<128, false>(p, st);
}

}  // namespace gqa
