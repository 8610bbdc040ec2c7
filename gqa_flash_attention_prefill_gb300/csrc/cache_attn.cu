// cache_attn.cu -- host code of gqa_cache_attention: argument checks, the
// launch shape and the workspace.  Declared in include/gqa_prefill.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "cache_attn.h"
#include "gqa_prefill.h"

namespace gqa {

namespace {

struct CachePlan {
  bool tile;  // the kernel of 128-row tiles
  int RT;     // rows of a unit
  int G, HPC, HG, KW, NT, T, NS;
  uint32_t data_bytes, slot_bytes;
  int ctas, max_units;  // per launch of at most kMaxSeqs sequences
  size_t ml_off, head_off, hdr_off, bytes;
};

// Heads per CTA: the largest divisor of Hkv up to 8; the warps left over share
// the heads' keys.  A tile that would leave the ring fewer than four slots (two
// tiles) takes fewer warps per head, then fewer heads.
int ring_shape(int Hkv, int d, bool c8, int gk, int esz, int warps, CachePlan* pl) {
  int hpc = Hkv < 8 ? Hkv : 8;
  while (Hkv % hpc != 0) --hpc;
  int kw = 1;
  while (2 * kw * hpc <= warps) kw *= 2;  // a power of two, and so the keys per tile
  for (;;) {
    pl->HPC = hpc;
    pl->KW = kw;
    pl->T = 16 * gk * kw;
    pl->data_bytes = (uint32_t)pl->T * hpc * d * esz;
    pl->slot_bytes = pl->data_bytes + (c8 ? ((uint32_t)pl->T * Hkv + 127u) / 128u * 128u : 0u);
    pl->NS = (int)((kSmemMax - ca_fixed_smem(warps)) / pl->slot_bytes);
    if (pl->NS > kCaMaxSlots) pl->NS = kCaMaxSlots;
    if (pl->NS >= 4) break;
    if (kw > 1) {
      kw >>= 1;
    } else if (hpc > 1) {
      do --hpc;
      while (Hkv % hpc != 0);
    } else {
      if (pl->NS >= 2) break;
      return GQA_ERR_UNSUPPORTED;  // the scales of too many heads
    }
  }
  return GQA_OK;
}

int cache_plan(int num_seqs, int total_q, int max_seqlen_q, int Hq, int Hkv, int d, int dtype,
               int cache_type, CachePlan* pl) {
  if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 ||
      Hq % Hkv != 0)
    return GQA_ERR_INVALID;
  if (dtype != GQA_F16 && dtype != GQA_BF16) return GQA_ERR_INVALID;
  if (cache_type != GQA_CACHE_16 && cache_type != GQA_CACHE_E4M3) return GQA_ERR_INVALID;
  if (d != 64 && d != 128 && d != 256) return GQA_ERR_UNSUPPORTED;
  const bool c8 = cache_type == GQA_CACHE_E4M3;
  pl->G = Hq / Hkv;
  if (Hkv > 4096 || (long long)total_q * pl->G >= (1ll << 30)) return GQA_ERR_UNSUPPORTED;
  // Rows of the longest sequence (all of them, without the hint) decide how
  // many 8-row tiles share each key a warp loads.
  const long long rows = (long long)(max_seqlen_q > 0 ? max_seqlen_q : total_q) * pl->G;
  pl->tile = d <= 128 && rows > (c8 ? kTileRows8 : kTileRows16);
  pl->NT = 1;
  while (pl->NT < cache_attn_max_nt(d) && rows > 8 * pl->NT) pl->NT *= 2;
  const int gk = ca_gk(d, c8, pl->NT), esz = c8 ? 1 : 2;
  const int warps = ca_warps(d, c8, pl->NT);
  if (pl->tile) {
    pl->HPC = 1;
    pl->KW = 1;
    pl->T = ct_bn(d);
    pl->NS = 2;
    pl->data_bytes = pl->slot_bytes = 0;
    pl->RT = 256;
  } else {
    const int rc = ring_shape(Hkv, d, c8, gk, esz, warps, pl);
    if (rc != GQA_OK) return rc;
    pl->RT = 8 * pl->NT;
  }
  pl->HG = Hkv / pl->HPC;
  int sms = 152;
  unsigned int* status = nullptr;
  if (call_device(&sms, &status) != GQA_OK) sms = 152;
  pl->ctas = sms;
  const int seqs = num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs;
  const int rt = pl->RT;
  const long long units =
      (long long)pl->HG * (((long long)total_q * pl->G + rt - 1) / rt + (long long)seqs);
  if (units > (1ll << 26)) return GQA_ERR_UNSUPPORTED;
  pl->max_units = (int)units;
  auto al = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t prow = 2u * (size_t)pl->ctas * pl->HPC * rt;
  pl->ml_off = al(prow * d * 4u);
  pl->head_off = pl->ml_off + al(prow * 8u);
  pl->hdr_off = pl->head_off + al(32u + (size_t)pl->ctas);
  pl->bytes = pl->hdr_off + al(32u * (size_t)pl->max_units);
  return GQA_OK;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int run_attention(const void* q, const void* k_pages, const void* v_pages, const void* k_scales,
                  const void* v_scales, int cache_type, const int32_t* cu, const int32_t* pre,
                  const int32_t* indptr, const int32_t* indices, int entries, int page_size,
                  int num_pages, int num_seqs, int total_q, int max_seqlen_q, int Hq, int Hkv,
                  int d, int dtype, float scale, int window, const float* sinks,
                  int smooth_softmax, const uint32_t* mask, const int32_t* mask_indptr,
                  long long total_mask_words, const int32_t* depths, void* out, float* lse,
                  void* workspace, size_t workspace_bytes, void* stream) {
  CachePlan pl;
  const int rc =
      cache_plan(num_seqs, total_q, max_seqlen_q, Hq, Hkv, d, dtype, cache_type, &pl);
  if (rc == GQA_ERR_INVALID) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale)) return GQA_ERR_INVALID;
  if (sinks != nullptr && smooth_softmax != 0) return GQA_ERR_INVALID;
  if (entries < 0 || page_size < 8 || page_size % 8 != 0 || num_pages <= 0 ||
      (long long)num_pages * page_size >= (1ll << 31) || total_mask_words < 0)
    return GQA_ERR_INVALID;
  if (rc != GQA_OK) return rc;
  if (num_seqs == 0 || total_q == 0) return GQA_OK;  // no work, no launch
  const bool c8 = cache_type == GQA_CACHE_E4M3;
  if (q == nullptr || k_pages == nullptr || v_pages == nullptr || out == nullptr ||
      cu == nullptr || pre == nullptr || indptr == nullptr || indices == nullptr || entries == 0 ||
      !al16(q) || !al16(k_pages) || !al16(v_pages) || !al16(out))
    return GQA_ERR_INVALID;
  if (c8 && (k_scales == nullptr || v_scales == nullptr || !al16(k_scales) || !al16(v_scales)))
    return GQA_ERR_INVALID;
  if ((mask == nullptr) != (mask_indptr == nullptr) ||
      (reinterpret_cast<uintptr_t>(mask) & 3u) != 0)
    return GQA_ERR_INVALID;
  if (workspace == nullptr || workspace_bytes < pl.bytes ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return GQA_ERR_INVALID;
  // Tokens per copy: the largest power of two (8 at least) that divides the
  // tile and the page.
  int run = pl.T;
  while (page_size % run != 0) run >>= 1;
  if (c8 && run * Hkv % 16 != 0) return GQA_ERR_UNSUPPORTED;

  CacheAttnParams p;
  std::memset(&p, 0, sizeof(p));
  int sms = 0;
  if (call_device(&sms, &p.status) != GQA_OK) return GQA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.k_pages = static_cast<const uint8_t*>(k_pages);
  p.v_pages = static_cast<const uint8_t*>(v_pages);
  p.k_scales = static_cast<const uint8_t*>(k_scales);
  p.v_scales = static_cast<const uint8_t*>(v_scales);
  p.indices = indices;
  p.sinks = sinks;
  p.mask = mask;
  p.depths = depths;
  p.out = out;
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + pl.ml_off);
  p.head = reinterpret_cast<int32_t*>(ws + pl.head_off);
  p.hdr = reinterpret_cast<int32_t*>(ws + pl.hdr_off);
  p.ctas = pl.ctas;
  p.total_mask_words = total_mask_words;
  p.timeout_ns = wait_limit_ns();
  p.entries = entries;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.total_q = total_q;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = pl.G;
  p.HPC = pl.HPC;
  p.HG = pl.HG;
  p.KW = pl.KW;
  p.T = pl.T;
  while ((1 << p.log_T) < pl.T) ++p.log_T;
  p.div_g.set((uint32_t)pl.G);
  p.div_page.set((uint32_t)page_size);
  p.div_ctas.set((uint32_t)pl.ctas);
  while ((1 << p.log_run) < run) ++p.log_run;
  p.run = run;
  p.NS = pl.NS;
  p.slot_bytes = pl.slot_bytes;
  p.data_bytes = pl.data_bytes;
  p.window = window > 0 ? window : 0;
  p.smooth = smooth_softmax != 0 ? 1 : 0;
  p.whole_slack = pl.tile ? kCtWholeSlack : kCaWholeSlack;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.metadata_ready = metadata_ready_flag() ? 1 : 0;
  // A window bounds a unit's tiles on the host: where whole units dealt out
  // cost less than a join (the device's own rule), no join is launched.  The
  // hint may be wrong: then whole units are the slower choice, not a wrong one.
  const int seqs = num_seqs < kMaxSeqs ? num_seqs : kMaxSeqs;
  const long long new_max = max_seqlen_q > 0 ? max_seqlen_q : total_q;
  long long units = (long long)pl.HG * seqs * ((new_max * pl.G + pl.RT - 1) / pl.RT);
  if (units > pl.max_units) units = pl.max_units;
  bool join = true;
  if (p.window > 0) {
    const long long n = ((long long)p.window + new_max + pl.T - 3) / pl.T + 1;
    if ((units + pl.ctas - 1) / pl.ctas * n <= p.whole_slack) {
      p.whole = 1;
      join = false;
    }
  }
  // Blocks of the join: at most one unit is cut per CTA; a block per row of a
  // unit, 16 blocks an SM at most.
  int merge_x = 0, merge_y = 1;
  if (join) {
    merge_x = (int)(units < pl.ctas ? units : pl.ctas);
    merge_y = 16 * pl.ctas / merge_x;
    const long long live = pl.HPC * (new_max * pl.G < pl.RT ? new_max * pl.G : pl.RT);
    if (merge_y > live) merge_y = (int)live;
    if (merge_y < 1) merge_y = 1;
  }
  const unsigned smem = ca_fixed_smem(ca_warps(d, c8, pl.NT)) + (unsigned)pl.NS * pl.slot_bytes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int b0 = 0; b0 < num_seqs; b0 += kMaxSeqs) {
    p.cu = cu + b0;
    p.pre = pre + b0;
    p.indptr = indptr + b0;
    p.mask_indptr = mask_indptr != nullptr ? mask_indptr + b0 : nullptr;
    p.first_seq = b0;
    p.num_seqs = num_seqs - b0 < kMaxSeqs ? num_seqs - b0 : kMaxSeqs;
    const bool bf16 = dtype == GQA_BF16;
    const cudaError_t e =
        pl.tile    ? launch_cache_tile(p, d, bf16, c8, pl.ctas, merge_x, merge_y, st)
        : d == 64    ? launch_cache_attn_d64(p, bf16, c8, pl.NT, pl.ctas, smem, merge_x, merge_y, st)
        : d == 128 ? launch_cache_attn_d128(p, bf16, c8, pl.NT, pl.ctas, smem, merge_x, merge_y, st)
                   : launch_cache_attn_d256(p, bf16, c8, pl.NT, pl.ctas, smem, merge_x, merge_y, st);
    if (e != cudaSuccess) return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

}  // namespace

}  // namespace gqa

extern "C" {

int gqa_cache_attention(const void* q, const void* k_pages, const void* v_pages,
                        const void* k_scales, const void* v_scales, int cache_type,
                        const int32_t* cu_seqlens_q, const int32_t* prefix_lens,
                        const int32_t* kv_page_indptr, const int32_t* kv_page_indices,
                        int num_page_entries, int page_size, int num_pages, int num_seqs,
                        int total_q, int max_seqlen_q, int Hq, int Hkv, int d, int dtype,
                        float scale, int window, const float* sinks, int smooth_softmax,
                        const uint32_t* custom_mask, const int32_t* mask_indptr,
                        long long total_mask_words, const int32_t* depths, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return gqa::run_attention(q, k_pages, v_pages, k_scales, v_scales, cache_type, cu_seqlens_q,
                            prefix_lens, kv_page_indptr, kv_page_indices, num_page_entries,
                            page_size, num_pages, num_seqs, total_q, max_seqlen_q, Hq, Hkv, d,
                            dtype, scale, window, sinks, smooth_softmax, custom_mask, mask_indptr,
                            total_mask_words, depths, out, lse, workspace, workspace_bytes, stream);
}

int gqa_cache_attention_workspace(int num_seqs, int total_q, int max_seqlen_q, int Hq, int Hkv,
                                  int d, int dtype, int cache_type, size_t* bytes) {
  if (bytes == nullptr) return GQA_ERR_INVALID;
  gqa::CachePlan pl;
  const int rc =
      gqa::cache_plan(num_seqs, total_q, max_seqlen_q, Hq, Hkv, d, dtype, cache_type, &pl);
  if (rc == GQA_OK) *bytes = pl.bytes;
  return rc;
}

}  // extern "C"
