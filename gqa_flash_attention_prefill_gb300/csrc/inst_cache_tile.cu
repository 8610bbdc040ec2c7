// inst_cache_tile.cu -- gqa_cache_attention's kernels of 128-row tiles.
#include "cache_attn.h"

namespace gqa {

namespace {

template <int D, bool BF16, bool C8>
cudaError_t launch_tile(const CacheAttnParams& p, int grid, int mx, int my, cudaStream_t st) {
  static SmemAttr attr{};
  return launch_with_join<D, BF16, C8>(cache_tile_kernel<D, BF16, C8>, attr, p, 256, grid,
                                       kCtThreads, ct_smem(D, C8), mx, my, st);
}

template <int D>
cudaError_t launch_types(const CacheAttnParams& p, bool bf16, bool c8, int grid, int mx, int my,
                         cudaStream_t st) {
  if (bf16)
    return c8 ? launch_tile<D, true, true>(p, grid, mx, my, st)
              : launch_tile<D, true, false>(p, grid, mx, my, st);
  return c8 ? launch_tile<D, false, true>(p, grid, mx, my, st)
            : launch_tile<D, false, false>(p, grid, mx, my, st);
}

}  // namespace

cudaError_t launch_cache_tile(const CacheAttnParams& p, int d, bool bf16, bool c8, int grid,
                              int merge_x, int merge_y, cudaStream_t st) {
  return d == 64 ? launch_types<64>(p, bf16, c8, grid, merge_x, merge_y, st)
                 : launch_types<128>(p, bf16, c8, grid, merge_x, merge_y, st);
}

}  // namespace gqa
