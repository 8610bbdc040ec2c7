// inst_cache_d128.cu -- gqa_cache_attention's kernels for head dim 128.
#include "cache_attn.h"

namespace gqa {

cudaError_t launch_cache_attn_d128(const CacheAttnParams& p, bool bf16, bool c8, int nt, int grid,
                                  unsigned smem, int merge_x, int merge_y, cudaStream_t st) {
  if (nt == 2) return launch_cache_attn_types<128, 2, false>(p, bf16, c8, grid, smem, merge_x, merge_y, st);
  if (p.HPC == 8) return launch_cache_attn_types<128, 1, true>(p, bf16, c8, grid, smem, merge_x, merge_y, st);
  return launch_cache_attn_types<128, 1, false>(p, bf16, c8, grid, smem, merge_x, merge_y, st);
}

}  // namespace gqa
