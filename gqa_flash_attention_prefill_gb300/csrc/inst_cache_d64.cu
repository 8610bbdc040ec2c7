// inst_cache_d64.cu -- gqa_cache_attention's kernels for head dim 64.
#include "cache_attn.h"

namespace gqa {

cudaError_t launch_cache_attn_d64(const CacheAttnParams& p, bool bf16, bool c8, int nt, int grid,
                                  unsigned smem, int merge_x, int merge_y, cudaStream_t st) {
  if (nt == 4)  // e4m3: above 16 rows 16-bit pages take the 128-row kernel
    return bf16 ? launch_cache_attn<64, true, true, 4, false>(p, grid, smem, merge_x, merge_y, st)
                : launch_cache_attn<64, false, true, 4, false>(p, grid, smem, merge_x, merge_y, st);
  if (nt == 2) return launch_cache_attn_types<64, 2, false>(p, bf16, c8, grid, smem, merge_x, merge_y, st);
  if (p.HPC == 8) return launch_cache_attn_types<64, 1, true>(p, bf16, c8, grid, smem, merge_x, merge_y, st);
  return launch_cache_attn_types<64, 1, false>(p, bf16, c8, grid, smem, merge_x, merge_y, st);
}

}  // namespace gqa
