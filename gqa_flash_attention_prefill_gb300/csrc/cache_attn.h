// cache_attn.h -- internal interface between gqa_cache_attention's host code
// and the kernel instantiations, one translation unit per head dim.
#pragma once
#include "cache_attn.cuh"
#include "cache_tile.cuh"
#include "launch.h"

namespace gqa {

// Shared memory a CTA may have, and what every kernel here is allowed: the ring
// takes as many slots as fit, so the size of one kernel differs between calls.
constexpr unsigned kSmemMax = 227u * 1024u;

// Rows per KV head (tokens times query heads of the longest sequence) above
// which the kernel of 128-row tiles takes over from the one whose warps stream
// all heads.  It reads a head's slices and pays a tile's products whatever the
// rows, and has to widen e4m3 keys through shared memory: with 8 sequences of
// 8k keys, 64 / 8 heads of 64, it takes 49..56 us (16-bit) or 65..81 us (e4m3)
// for 16..64 rows; the streaming kernel 46, 61, 65, 116, 122 us (16-bit) or 46,
// 54, 58, 92, 99 us (e4m3, bf16; 2 to 4% more in f16) for 16, 24, 32, 48, 64 rows.  At d = 128 (16 / 2
// heads) they meet at 16 rows (30 us, 16-bit) and between 32 and 40 (36..44 us,
// e4m3).
constexpr int kTileRows16 = 16, kTileRows8 = 32;

// 8-row tiles a warp takes at most for head dim d: the accumulators and the
// query fragments stay in registers.  (d = 64 has 4 for e4m3 pages alone: 16-bit
// ones leave this kernel at 16 rows.)
constexpr int cache_attn_max_nt(int d) { return d == 64 ? 4 : d == 128 ? 2 : 1; }
static_assert(kTileRows16 <= 16, "16-bit pages at d = 64 with four row tiles have no kernel");

cudaError_t launch_cache_attn_d64(const CacheAttnParams& p, bool bf16, bool c8, int nt, int grid,
                                  unsigned smem, int merge_x, int merge_y, cudaStream_t st);
cudaError_t launch_cache_attn_d128(const CacheAttnParams& p, bool bf16, bool c8, int nt, int grid,
                                   unsigned smem, int merge_x, int merge_y, cudaStream_t st);
cudaError_t launch_cache_attn_d256(const CacheAttnParams& p, bool bf16, bool c8, int nt, int grid,
                                   unsigned smem, int merge_x, int merge_y, cudaStream_t st);

// The 128-row form, d = 64 or 128.
cudaError_t launch_cache_tile(const CacheAttnParams& p, int d, bool bf16, bool c8, int grid,
                              int merge_x, int merge_y, cudaStream_t st);

namespace {

// Launches `kern`, and the join of cut units when merge_x > 0: one attribute
// slot per kernel remembers that it was allowed kSmemMax.  Threads that come
// here at once all set the same value.
template <int D, bool BF16, bool C8, typename Kern>
cudaError_t launch_with_join(Kern kern, SmemAttr& attr, const CacheAttnParams& p, int rt, int grid,
                             int threads, unsigned smem, int merge_x, int merge_y,
                             cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (attr.allowed[dev].load(std::memory_order_acquire) < kSmemMax) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    attr.allowed[dev].store(kSmemMax, std::memory_order_release);
  }
  e = launch_pdl(kern, p, grid, threads, smem, st);
  if (e != cudaSuccess || merge_x == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)merge_x, (unsigned)merge_y, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = la;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, cache_merge_kernel<D, BF16>, p, rt, BF16 && !C8 ? 0.f : kCaBias);
}

template <int D, bool BF16, bool C8, int NT, bool H8>
cudaError_t launch_cache_attn(const CacheAttnParams& p, int grid, unsigned smem, int merge_x,
                              int merge_y, cudaStream_t st) {
  static SmemAttr attr{};
  return launch_with_join<D, BF16, C8>(cache_attn_kernel<D, BF16, C8, NT, H8>, attr, p, 8 * NT,
                                       grid, 32 * (ca_warps(D, C8, NT) + 1), smem, merge_x, merge_y,
                                       st);
}

template <int D, int NT, bool H8>
cudaError_t launch_cache_attn_types(const CacheAttnParams& p, bool bf16, bool c8, int grid,
                                    unsigned smem, int mx, int my, cudaStream_t st) {
  if (bf16)
    return c8 ? launch_cache_attn<D, true, true, NT, H8>(p, grid, smem, mx, my, st)
              : launch_cache_attn<D, true, false, NT, H8>(p, grid, smem, mx, my, st);
  return c8 ? launch_cache_attn<D, false, true, NT, H8>(p, grid, smem, mx, my, st)
            : launch_cache_attn<D, false, false, NT, H8>(p, grid, smem, mx, my, st);
}

}  // namespace

}  // namespace gqa
