// cache_rows.cu -- the row operators around the paged cache: rotary positions
// (gqa_rope), writing the cache with the rotation fused (gqa_cache_write) and
// reading it back (gqa_cache_read).  Declared in include/gqa_prefill.h.
//
// All three move each value once and compute a few operations on it: they are
// bound by HBM when large and by the launch and two or three dependent loads
// (sequence, page table, page) when small.
#include <cuda_runtime.h>

#include <cmath>

#include "cache_rows.cuh"
#include "gqa_prefill.h"
#include "launch.h"

namespace gqa {

namespace {

constexpr int kRowThreads = 64;    // of the row kernel
constexpr int kMaxTokens = 8;      // tokens one of its CTAs handles at most
constexpr int kReadThreads = 128;  // of the read kernel, a warp per row

// Where the values of one call come from and go to.
struct RowsParams {
  // rotation (half == 0: none); the angles' tables are [half]
  const int32_t* positions;
  const double* inv_freq;
  int half;
  float factor;
  int inverse;
  // heads: hq rows of q (rotated, to q_out), hkv of k, hkv of v (never rotated)
  const void* q;
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;  // elements between rows
  void* q_out;
  void* k_out;  // rows (gqa_rope) or pages (gqa_cache_write)
  void* v_out;
  long long q_out_stride, k_out_stride;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int hq, hkv, d, rows;
  int tokens;  // tokens per CTA, <= kMaxTokens
  // sequences (gqa_cache_write)
  const int32_t* cu;
  const int32_t* pre;
  PageTable pt;
  unsigned int* status;
};

enum { kOutRows = 0, kOutCache16 = 1, kOutCache8 = 2 };
// How rotated values pair up: halves of the rotated part in vectors of 8,
// halves of any even size, or neighbours.
enum { kPairNone = 0, kPairHalf8 = 1, kPairHalf = 2, kPairNext = 3 };

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  x[0] = unpack_lo<BF16>(r.x), x[1] = unpack_hi<BF16>(r.x);
  x[2] = unpack_lo<BF16>(r.y), x[3] = unpack_hi<BF16>(r.y);
  x[4] = unpack_lo<BF16>(r.z), x[5] = unpack_hi<BF16>(r.z);
  x[6] = unpack_lo<BF16>(r.w), x[7] = unpack_hi<BF16>(r.w);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}
// 8 values times f as e4m3, rounded to nearest even, infinities to the largest.
__device__ __forceinline__ uint2 narrow8(const float (&x)[8], float f) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * f, x[4 * i + 1] * f),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * f, x[4 * i + 3] * f),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}
template <bool BF16>
__device__ __forceinline__ float load16(const uint16_t* p) {
  return unpack_lo<BF16>((uint32_t)*p);
}

// One CTA: up to `tokens` consecutive rows, all their heads (blockIdx.y takes
// every gridDim.y-th slice of the heads).  A thread owns two vectors of 8
// values at a fixed place of a fixed token and walks the heads, so the angles
// are found once: the CTA computes tokens * half pairs of (cos, sin) into
// shared memory and each thread keeps its own in registers.  The two vectors
// are neighbours, or, when halves pair up, the two that rotate into each
// other: every value is then read once.  The next head's loads are issued
// before this head's arithmetic, the first ones before the angles.
// Rotation, scale search and rounding run in fp32; the result is rounded once.
// (One vector a thread that read its partner's as well: 16k rows of 64 / 8
// heads 77 us, now 51.  Two heads' loads ahead, in registers that cost CTAs an
// SM: 53 us, a ragged prompt write of 9.6k tokens 40.1 where this takes 40.3.)
template <bool BF16, int OUT, int PAIR>
__global__ void __launch_bounds__(kRowThreads, 14) rows_kernel(const __grid_constant__ RowsParams p) {
  extern __shared__ float2 s_cs[];  // [tokens][half], then the steps [half]
  __shared__ int s_key[kMaxTokens];
  __shared__ long long s_slot[kMaxTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.x * p.tokens;
  const int ntok = min(p.tokens, p.rows - row0);
  grid_dep_launch_dependents();
  grid_dep_wait();

  // ---- this thread's vectors
  const int nt = (p.d + 15) >> 4;            // threads per head
  const int slices = kRowThreads / nt / p.tokens;  // heads in flight
  const int vec = tid % nt, rest = tid / nt;
  const int t = rest % p.tokens, slice = rest / p.tokens;
  const int rot = 2 * p.half, turning = p.half >> 3;  // threads of a head that rotate (halves)
  int ea = 16 * vec, eb = 16 * vec + 8;
  if (PAIR == kPairHalf8) {
    ea = vec < turning ? 8 * vec : 16 * vec;
    eb = vec < turning ? 8 * vec + p.half : 16 * vec + 8;
  }
  const int heads = p.hq + p.hkv + (OUT != kOutRows ? p.hkv : 0);
  const bool active = slice < slices && t < ntok;
  const bool two = eb < p.d;
  const int row = row0 + (active ? t : 0);
  const int step = slices * gridDim.y;
  const int first = blockIdx.y * slices + slice;
  // All lanes take every turn: the scale search shuffles over the warp.
  const int turns = (heads - (int)blockIdx.y * slices + step - 1) / step;
  // Head h of the row (q, then k, then v) starts at its base + h * d.
  const uint16_t* const q_row = static_cast<const uint16_t*>(p.q) + row * p.q_stride;
  const uint16_t* const k_row =
      static_cast<const uint16_t*>(p.k) + row * p.k_stride - (long long)p.hq * p.d;
  const uint16_t* const v_row = static_cast<const uint16_t*>(p.v) + row * p.v_stride -
                                (long long)(p.hq + p.hkv) * p.d;
  auto source = [&](int h) {
    const uint16_t* base = h < p.hq ? q_row : k_row;
    if (OUT != kOutRows && h >= p.hq + p.hkv) base = v_row;
    return base + h * p.d;
  };
  uint4 na = make_uint4(0u, 0u, 0u, 0u), nb = na;
  auto fetch = [&](int h) {
    if (!active || h >= heads) return;
    const uint16_t* src = source(h);
    na = *reinterpret_cast<const uint4*>(src + ea);
    if (two) nb = *reinterpret_cast<const uint4*>(src + eb);
  };
  fetch(first);

  // ---- tokens' places and angles
  if (PAIR != kPairNone) {
    unsigned long long* s_step = reinterpret_cast<unsigned long long*>(s_cs + p.tokens * p.half);
    for (int j = tid; j < p.half; j += kRowThreads) s_step[j] = phase_step(__ldg(p.inv_freq + j));
  }
  // A warp per token: its sequence, key index and page; the page number is
  // used only after the angles, which hide its load.
  int page = -1, in_page = 0;
  if (OUT != kOutRows && warp < ntok) {
    const int r = row0 + warp;
    const int b = warp_upper_bound(p.cu + 1, p.pt.num_seqs, r);
    if (lane == 0) {
      int key = 0;
      if (b < p.pt.num_seqs) {
        const int c0 = __ldg(p.cu + b), P = __ldg(p.pre + b);
        const int i0 = __ldg(p.pt.indptr + b), i1 = __ldg(p.pt.indptr + b + 1);
        const long long k = (long long)P + (r - c0);
        const long long at = i0 + k / p.pt.page_size;
        key = (int)k;
        in_page = (int)(k % p.pt.page_size);
        page = 0x7fffffff;  // bad, unless
        if (c0 >= 0 && c0 <= r && P >= 0 && k <= 0x7fffffffll && i0 >= 0 && at < i1 &&
            at < p.pt.entries)
          page = (int)min((unsigned)__ldg(p.pt.indices + at), 0x7fffffffu);  // negative: bad too
      }
      s_key[warp] = key;
    }
  }
  if (OUT != kOutRows || PAIR != kPairNone) __syncthreads();
  if (PAIR != kPairNone) {
    const unsigned long long* s_step =
        reinterpret_cast<const unsigned long long*>(s_cs + p.tokens * p.half);
    for (int i = tid; i < ntok * p.half; i += kRowThreads) {
      const int tt = i / p.half, j = i - tt * p.half;
      const int pos = p.positions != nullptr ? __ldg(p.positions + row0 + tt) : s_key[tt];
      float2 cs = phase_cos_sin(pos, s_step[j]);
      cs.x *= p.factor;
      cs.y *= p.inverse ? -p.factor : p.factor;
      s_cs[i] = cs;
    }
  }
  if (OUT != kOutRows && warp < ntok && lane == 0) {
    const bool bad = page >= p.pt.num_pages;
    if (bad) atomicOr(p.status, (unsigned)GQA_DEV_BAD_METADATA);
    s_slot[warp] = page < 0 || bad ? -1 : (long long)page * p.pt.page_size + in_page;
  }
  if (OUT != kOutRows || PAIR != kPairNone) __syncthreads();
  const long long slot = OUT != kOutRows ? s_slot[active ? t : 0] : 0;
  // The thread's angles: pairs of the two vectors, or the pairs within each.
  float2 cs[8];
  const bool turner = PAIR == kPairHalf8 ? vec < turning : ea < rot;
  if ((PAIR == kPairHalf8 || PAIR == kPairNext) && active && turner) {
    const float2* c = s_cs + t * p.half + 8 * vec;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      cs[i] = PAIR == kPairHalf8 || 16 * vec + 2 * i < rot ? c[i] : make_float2(1.f, 0.f);
  }

  // Destinations as the sources: base + h * d.
  constexpr int kOutBytes = OUT == kOutCache8 ? 1 : 2;
  uint16_t* const q_dst = static_cast<uint16_t*>(p.q_out) + row * p.q_out_stride;
  const long long dst_row = OUT == kOutRows ? row * p.k_out_stride : slot * p.hkv * p.d;
  void* const k_dst =
      static_cast<uint8_t*>(p.k_out) + (dst_row - (long long)p.hq * p.d) * kOutBytes;
  void* const v_dst =
      static_cast<uint8_t*>(p.v_out) + (dst_row - (long long)(p.hq + p.hkv) * p.d) * kOutBytes;

  for (int n = 0; n < turns; ++n) {
    const int h = first + n * step;
    const bool on = active && h < heads;
    const bool is_q = h < p.hq, is_k = !is_q && h < p.hq + p.hkv;
    float x[8], y[8];
    unpack8<BF16>(na, x);
    unpack8<BF16>(nb, y);
    if (n + 1 < turns) fetch(h + step);
    const bool turn = PAIR != kPairNone && on && turner && (is_q || is_k);
    if (PAIR == kPairHalf8 && turn) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = x[i], b = y[i];
        x[i] = a * cs[i].x - b * cs[i].y;
        y[i] = b * cs[i].x + a * cs[i].y;
      }
    }
    if (PAIR == kPairNext && turn) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        const float c = y[2 * i], d = y[2 * i + 1];
        if (ea + 2 * i < rot) {  // values past the rotated part stay
          x[2 * i] = a * cs[i].x - b * cs[i].y;
          x[2 * i + 1] = b * cs[i].x + a * cs[i].y;
        }
        if (eb + 2 * i < rot) {
          y[2 * i] = c * cs[4 + i].x - d * cs[4 + i].y;
          y[2 * i + 1] = d * cs[4 + i].x + c * cs[4 + i].y;
        }
      }
    }
    if (PAIR == kPairHalf && turn) {  // halves that do not fill vectors: partners one by one
      const uint16_t* src = source(h);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = (i < 8 ? ea : eb) + (i & 7);
        float& z = i < 8 ? x[i & 7] : y[i & 7];
        if (e < p.half) {
          const float2 c = s_cs[t * p.half + e];
          z = z * c.x - load16<BF16>(src + e + p.half) * c.y;
        } else if (e < rot) {
          const float2 c = s_cs[t * p.half + e - p.half];
          z = z * c.x + load16<BF16>(src + e - p.half) * c.y;
        }
      }
    }
    // A row without a place in the cache is nobody's: its q_out stays too.
    if (on && (OUT == kOutRows || (slot >= 0 && (is_q || OUT == kOutCache16)))) {
      uint16_t* dst = is_q ? q_dst : static_cast<uint16_t*>(is_k ? k_dst : v_dst);
      dst += h * p.d;
      *reinterpret_cast<uint4*>(dst + ea) = pack8<BF16>(x);
      if (two) *reinterpret_cast<uint4*>(dst + eb) = pack8<BF16>(y);
    }
    // Every lane comes here in the same turn; warps of query heads only pass by.
    if (OUT == kOutCache8 && __any_sync(0xffffffffu, on && !is_q)) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)  // NaN counts as absent
        amax = max3(amax, fabsf(x[i]), fabsf(y[i]));
      for (int o = nt >> 1; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (on && !is_q && slot >= 0) {
        const int e = e4m3_scale_exponent(amax);
        const float inv = pow2f(-e);
        uint8_t* dst = static_cast<uint8_t*>(is_k ? k_dst : v_dst) + h * p.d;
        *reinterpret_cast<uint2*>(dst + ea) = narrow8(x, inv);
        *reinterpret_cast<uint2*>(dst + eb) = narrow8(y, inv);
        if (vec == 0)
          (is_k ? p.k_scales + slot * p.hkv - p.hq : p.v_scales + slot * p.hkv - p.hq - p.hkv)[h] =
              (uint8_t)(e + 127);
      }
    }
  }
}

// ---------------------------------------------------------------- read back
struct ReadParams {
  const void* k_pages;
  const void* v_pages;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int32_t* kv_indptr;
  const int32_t* first_keys;  // or nullptr
  void* k_out;
  void* v_out;
  PageTable pt;
  int hkv, d, rows;
  unsigned int* status;
};

// Rows a CTA gathers: one a warp, so that the lookups of all run at once and
// nothing is shared (16 rows on 8 warps with a barrier after the lookups: 8 x
// 8192 keys 38.6 us, 64 x 128 keys 8.1; now 36.9 and 4.5).
constexpr int kReadRows = kReadThreads / 32;

// 4 e4m3 values times 2^e (as fp32 `s`), rounded to 16 bits (exact in bf16
// unless the result leaves bf16's normal range).
template <bool BF16>
__device__ __forceinline__ uint2 widen4(uint32_t w, float s) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
  return make_uint2(pack2<BF16>(a.x * s, a.y * s), pack2<BF16>(b.x * s, b.y * s));
}

// A warp per output row of k and v, all heads: it finds the row's place in the
// pool, then its lanes walk 16-value (e4m3) or 8-value (16-bit) vectors, 16-byte
// loads and stores.
template <bool BF16, bool C8>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x * kReadRows + warp;
  grid_dep_launch_dependents();
  grid_dep_wait();
  if (r >= p.rows) return;
  const int b = warp_upper_bound(p.kv_indptr + 1, p.pt.num_seqs, r);
  if (b >= p.pt.num_seqs) return;  // a row of no sequence
  // Every lane looks the same words up (one request a warp).
  const int r0 = __ldg(p.kv_indptr + b);
  const int f = p.first_keys != nullptr ? __ldg(p.first_keys + b) : 0;
  const int i0 = __ldg(p.pt.indptr + b), i1 = __ldg(p.pt.indptr + b + 1);
  const long long key = (long long)f + (r - r0);
  const long long at = i0 + key / p.pt.page_size;
  int page = -1;
  if (r0 >= 0 && r0 <= r && f >= 0 && i0 >= 0 && at < i1 && at < p.pt.entries)
    page = __ldg(p.pt.indices + at);
  if (page < 0 || page >= p.pt.num_pages) {
    if (lane == 0) atomicOr(p.status, (unsigned)GQA_DEV_BAD_METADATA);
    return;
  }
  const long long slot = (long long)page * p.pt.page_size + key % p.pt.page_size;
  const int per_row = p.hkv * p.d / (C8 ? 16 : 8);
  const uint4* const k = static_cast<const uint4*>(p.k_pages) + slot * per_row;
  const uint4* const v = static_cast<const uint4*>(p.v_pages) + slot * per_row;
  uint4* const ko = static_cast<uint4*>(p.k_out) + (long long)r * per_row * (C8 ? 2 : 1);
  uint4* const vo = static_cast<uint4*>(p.v_out) + (long long)r * per_row * (C8 ? 2 : 1);
  const int shift = p.d == 64 ? 2 : p.d == 128 ? 3 : 4;  // vectors of a head (e4m3)
  auto wide = [](uint4* dst, const uint4& raw, uint8_t e) {
    const float s = __int_as_float((int)e << 23);
    const uint2 a = widen4<BF16>(raw.x, s), c = widen4<BF16>(raw.y, s);
    const uint2 g = widen4<BF16>(raw.z, s), h = widen4<BF16>(raw.w, s);
    dst[0] = make_uint4(a.x, a.y, c.x, c.y);
    dst[1] = make_uint4(g.x, g.y, h.x, h.y);
  };
#pragma unroll 2
  for (int c = lane; c < per_row; c += 32) {
    const uint4 x = __ldg(k + c), y = __ldg(v + c);
    if (!C8) {
      ko[c] = x;
      vo[c] = y;
    } else {
      const uint8_t ek = __ldg(p.k_scales + slot * p.hkv + (c >> shift));
      const uint8_t ev = __ldg(p.v_scales + slot * p.hkv + (c >> shift));
      wide(ko + 2 * c, x, ek);
      wide(vo + 2 * c, y, ev);
    }
  }
}

// ---------------------------------------------------------------- host side
template <typename Kern, typename Params>
cudaError_t launch_rows(Kern kern, const Params& p, int gx, int gy, unsigned smem, cudaStream_t st,
                        int threads = kRowThreads) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)gx, (unsigned)gy, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <bool BF16, int OUT>
cudaError_t launch_pairs(const RowsParams& p, int pair, int gx, int gy, unsigned smem,
                         cudaStream_t st) {
  switch (pair) {
    case kPairNone: return launch_rows(rows_kernel<BF16, OUT, kPairNone>, p, gx, gy, smem, st);
    case kPairHalf8: return launch_rows(rows_kernel<BF16, OUT, kPairHalf8>, p, gx, gy, smem, st);
    case kPairHalf: return launch_rows(rows_kernel<BF16, OUT, kPairHalf>, p, gx, gy, smem, st);
    default: return launch_rows(rows_kernel<BF16, OUT, kPairNext>, p, gx, gy, smem, st);
  }
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// A row-strided tensor of 16-bit values read in 16-byte vectors.
bool row_ok(const void* p, long long stride, long long width) {
  return p != nullptr && aligned(p, 16) && stride >= width && stride % 8 == 0;
}

// Tokens per CTA and head slices.  Many rows: small CTAs (2 tokens at d = 64:
// 4 threads a head, 8 heads in flight), so that one's lookups and angles run
// beside another's loads (16k rows of 64 / 8 heads: 64 threads 52 us, 128 54,
// 256 64).  Few rows (the CTAs of that shape would not fill the SMs twice): one
// token per CTA and its heads spread over blockIdx.y, so that a thread has one
// head or two.
int launch_row_op(RowsParams& p, int out, int interleaved, bool bf16, void* stream) {
  int sms = 0;
  if (call_device(&sms, &p.status) != GQA_OK) return GQA_ERR_CUDA;
  const int nt = (p.d + 15) / 16, per = kRowThreads / nt;
  const int heads = p.hq + p.hkv + (out != kOutRows ? p.hkv : 0);
  int tokens = 8 / nt;
  if (tokens < 1) tokens = 1;
  if (tokens > kMaxTokens) tokens = kMaxTokens;
  if (out != kOutRows && tokens > kRowThreads / 32) tokens = kRowThreads / 32;  // a warp looks up a token
  int gy = 1;
  if ((long long)p.rows < 2ll * sms * tokens) {
    tokens = 1;
    gy = (heads + per - 1) / per;
    if (gy > 65535) gy = 65535;
  }
  p.tokens = tokens;
  const long long gx = ((long long)p.rows + tokens - 1) / tokens;
  const int pair = p.half == 0 ? kPairNone
                   : interleaved ? kPairNext
                   : p.half % 8 == 0 ? kPairHalf8 : kPairHalf;
  const unsigned smem = (unsigned)(tokens + 1) * (unsigned)p.half * 8u;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (out == kOutRows)
    e = bf16 ? launch_pairs<true, kOutRows>(p, pair, (int)gx, gy, smem, st)
             : launch_pairs<false, kOutRows>(p, pair, (int)gx, gy, smem, st);
  else if (out == kOutCache16)
    e = bf16 ? launch_pairs<true, kOutCache16>(p, pair, (int)gx, gy, smem, st)
             : launch_pairs<false, kOutCache16>(p, pair, (int)gx, gy, smem, st);
  else
    e = bf16 ? launch_pairs<true, kOutCache8>(p, pair, (int)gx, gy, smem, st)
             : launch_pairs<false, kOutCache8>(p, pair, (int)gx, gy, smem, st);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// True when [a, a + an) and [b, b + bn) share a byte.
bool overlap(const void* a, long long an, const void* b, long long bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}
// Output rows may not share memory with input rows: the next head is read
// before this one is written.
bool rows_overlap(const void* a, long long as, const void* b, long long bs, int rows, int wa,
                  int wb) {
  return overlap(a, ((rows - 1) * as + wa) * 2, b, ((rows - 1) * bs + wb) * 2);
}

bool rotation_ok(const double* inv_freq, int rot_dim, int interleaved, float factor, int d) {
  if (rot_dim <= 0 || rot_dim > d || rot_dim % 2 != 0) return false;
  if (interleaved != 0 && interleaved != 1) return false;
  return inv_freq != nullptr && aligned(inv_freq, 8) && std::isfinite(factor);
}

bool pages_ok(int num_page_entries, int page_size, int num_pages) {
  return num_page_entries >= 0 && page_size >= 8 && page_size % 8 == 0 && num_pages > 0 &&
         (long long)num_pages * page_size < (1ll << 31);
}

int run_rope(const gqa_rope_t* rope, const void* k, long long k_stride, void* k_out,
             long long k_out_stride, int rows, int Hkv, int d, int dtype, void* stream) {
  if (rope == nullptr || rows < 0 || Hkv < 0 || rope->Hq < 0 || d <= 0) return GQA_ERR_INVALID;
  if (dtype != GQA_F16 && dtype != GQA_BF16) return GQA_ERR_INVALID;
  if (!rotation_ok(rope->inv_freq, rope->rot_dim, rope->interleaved, rope->attn_factor, d) ||
      (rope->inverse != 0 && rope->inverse != 1))
    return GQA_ERR_INVALID;
  if (d % 8 != 0 || d > 1024 || rope->rot_dim > 512) return GQA_ERR_UNSUPPORTED;
  if ((long long)rope->Hq + Hkv > (1 << 20)) return GQA_ERR_UNSUPPORTED;
  if (rows == 0 || rope->Hq + Hkv == 0) return GQA_OK;
  if (rope->positions == nullptr) return GQA_ERR_INVALID;
  const long long qw = (long long)rope->Hq * d, kw = (long long)Hkv * d;
  if (rope->Hq > 0 && (!row_ok(rope->q, rope->q_stride, qw) ||
                       !row_ok(rope->q_out, rope->q_out_stride, qw) ||
                       rows_overlap(rope->q, rope->q_stride, rope->q_out, rope->q_out_stride, rows,
                                    (int)qw, (int)qw)))
    return GQA_ERR_INVALID;
  if (Hkv > 0 && (!row_ok(k, k_stride, kw) || !row_ok(k_out, k_out_stride, kw) ||
                  rows_overlap(k, k_stride, k_out, k_out_stride, rows, (int)kw, (int)kw)))
    return GQA_ERR_INVALID;
  // Nor with the other input's: both are read by the CTA that writes.
  if (rope->Hq > 0 && Hkv > 0 &&
      (rows_overlap(k, k_stride, rope->q_out, rope->q_out_stride, rows, (int)kw, (int)qw) ||
       rows_overlap(rope->q, rope->q_stride, k_out, k_out_stride, rows, (int)qw, (int)kw)))
    return GQA_ERR_INVALID;
  RowsParams p = {};
  p.positions = rope->positions;
  p.inv_freq = rope->inv_freq;
  p.half = rope->rot_dim / 2;
  p.factor = rope->attn_factor;
  p.inverse = rope->inverse;
  p.q = rope->q, p.q_stride = rope->q_stride;
  p.q_out = rope->q_out, p.q_out_stride = rope->q_out_stride;
  p.k = k, p.k_stride = k_stride, p.k_out = k_out, p.k_out_stride = k_out_stride;
  p.hq = rope->Hq, p.hkv = Hkv, p.d = d, p.rows = rows;
  return launch_row_op(p, kOutRows, rope->interleaved, dtype == GQA_BF16, stream);
}

int run_write(const void* k, long long k_stride, const void* v, long long v_stride,
              const int32_t* cu, const int32_t* pre, const int32_t* indptr, const int32_t* indices,
              int entries, int page_size, int num_pages, int num_seqs, int total_q, int Hkv, int d,
              int dtype, int cache_type, void* k_pages, void* v_pages, void* k_scales,
              void* v_scales, const gqa_rope_t* rope, void* stream) {
  if (num_seqs < 0 || total_q < 0 || Hkv <= 0 || d <= 0) return GQA_ERR_INVALID;
  if (dtype != GQA_F16 && dtype != GQA_BF16) return GQA_ERR_INVALID;
  if (cache_type != GQA_CACHE_16 && cache_type != GQA_CACHE_E4M3) return GQA_ERR_INVALID;
  if (!pages_ok(entries, page_size, num_pages)) return GQA_ERR_INVALID;
  const int Hq = rope != nullptr ? rope->Hq : 0;
  if (rope != nullptr && (Hq < 0 || rope->inverse != 0 ||
                          !rotation_ok(rope->inv_freq, rope->rot_dim, rope->interleaved,
                                       rope->attn_factor, d)))
    return GQA_ERR_INVALID;
  if (d != 64 && d != 128 && d != 256) return GQA_ERR_UNSUPPORTED;
  if ((long long)Hq + 2ll * Hkv > (1 << 20)) return GQA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0) return GQA_OK;
  const long long kw = (long long)Hkv * d, qw = (long long)Hq * d;
  if (cu == nullptr || pre == nullptr || indptr == nullptr || indices == nullptr || entries == 0 ||
      !row_ok(k, k_stride, kw) || !row_ok(v, v_stride, kw) || k_pages == nullptr ||
      v_pages == nullptr || !aligned(k_pages, 16) || !aligned(v_pages, 16))
    return GQA_ERR_INVALID;
  if (cache_type == GQA_CACHE_E4M3 && (k_scales == nullptr || v_scales == nullptr))
    return GQA_ERR_INVALID;
  if (Hq > 0 && (!row_ok(rope->q, rope->q_stride, qw) ||
                 !row_ok(rope->q_out, rope->q_out_stride, qw) ||
                 rows_overlap(rope->q, rope->q_stride, rope->q_out, rope->q_out_stride, total_q,
                              (int)qw, (int)qw) ||
                 rows_overlap(k, k_stride, rope->q_out, rope->q_out_stride, total_q, (int)kw,
                              (int)qw) ||
                 rows_overlap(v, v_stride, rope->q_out, rope->q_out_stride, total_q, (int)kw,
                              (int)qw)))
    return GQA_ERR_INVALID;
  RowsParams p = {};
  if (rope != nullptr) {
    p.positions = rope->positions;
    p.inv_freq = rope->inv_freq;
    p.half = rope->rot_dim / 2;
    p.factor = rope->attn_factor;
    p.q = rope->q, p.q_stride = rope->q_stride;
    p.q_out = rope->q_out, p.q_out_stride = rope->q_out_stride;
  }
  p.hq = Hq, p.hkv = Hkv, p.d = d, p.rows = total_q;
  p.k = k, p.k_stride = k_stride, p.v = v, p.v_stride = v_stride;
  p.k_out = k_pages, p.v_out = v_pages;
  p.k_scales = static_cast<uint8_t*>(k_scales), p.v_scales = static_cast<uint8_t*>(v_scales);
  p.cu = cu, p.pre = pre;
  p.pt = PageTable{indptr, indices, entries, page_size, num_pages, num_seqs};
  return launch_row_op(p, cache_type == GQA_CACHE_E4M3 ? kOutCache8 : kOutCache16,
                       rope != nullptr ? rope->interleaved : 0, dtype == GQA_BF16, stream);
}

int run_read(const void* k_pages, const void* v_pages, const void* k_scales, const void* v_scales,
             int cache_type, const int32_t* indptr, const int32_t* indices, int entries,
             int page_size, int num_pages, const int32_t* kv_indptr, const int32_t* first_keys,
             int num_seqs, int total_kv, int Hkv, int d, int dtype, void* k_out, void* v_out,
             void* stream) {
  if (num_seqs < 0 || total_kv < 0 || Hkv <= 0 || d <= 0) return GQA_ERR_INVALID;
  if (dtype != GQA_F16 && dtype != GQA_BF16) return GQA_ERR_INVALID;
  if (cache_type != GQA_CACHE_16 && cache_type != GQA_CACHE_E4M3) return GQA_ERR_INVALID;
  if (!pages_ok(entries, page_size, num_pages)) return GQA_ERR_INVALID;
  if (d != 64 && d != 128 && d != 256) return GQA_ERR_UNSUPPORTED;
  if (Hkv > (1 << 16)) return GQA_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_kv == 0) return GQA_OK;
  if (indptr == nullptr || indices == nullptr || entries == 0 || kv_indptr == nullptr ||
      k_pages == nullptr || v_pages == nullptr || k_out == nullptr || v_out == nullptr ||
      !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return GQA_ERR_INVALID;
  const bool c8 = cache_type == GQA_CACHE_E4M3;
  if (c8 && (k_scales == nullptr || v_scales == nullptr)) return GQA_ERR_INVALID;
  ReadParams p = {};
  p.k_pages = k_pages, p.v_pages = v_pages;
  p.k_scales = static_cast<const uint8_t*>(k_scales);
  p.v_scales = static_cast<const uint8_t*>(v_scales);
  p.kv_indptr = kv_indptr, p.first_keys = first_keys;
  p.k_out = k_out, p.v_out = v_out;
  p.pt = PageTable{indptr, indices, entries, page_size, num_pages, num_seqs};
  p.hkv = Hkv, p.d = d, p.rows = total_kv;
  int sms = 0;
  if (call_device(&sms, &p.status) != GQA_OK) return GQA_ERR_CUDA;
  const int grid = (int)(((long long)total_kv + kReadRows - 1) / kReadRows);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!c8)  // 16-bit pages are copied whatever their type
    e = launch_rows(read_kernel<true, false>, p, grid, 1, 0, st, kReadThreads);
  else if (dtype == GQA_BF16)
    e = launch_rows(read_kernel<true, true>, p, grid, 1, 0, st, kReadThreads);
  else
    e = launch_rows(read_kernel<false, true>, p, grid, 1, 0, st, kReadThreads);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

}  // namespace gqa

extern "C" {

int gqa_rope(const gqa_rope_t* rope, const void* k, long long k_stride, void* k_out,
             long long k_out_stride, int rows, int Hkv, int d, int dtype, void* stream) {
  return gqa::run_rope(rope, k, k_stride, k_out, k_out_stride, rows, Hkv, d, dtype, stream);
}

int gqa_cache_write(const void* k, long long k_stride, const void* v, long long v_stride,
                    const int32_t* cu_seqlens_q, const int32_t* prefix_lens,
                    const int32_t* kv_page_indptr, const int32_t* kv_page_indices,
                    int num_page_entries, int page_size, int num_pages, int num_seqs, int total_q,
                    int Hkv, int d, int dtype, int cache_type, void* k_pages, void* v_pages,
                    void* k_scales, void* v_scales, const gqa_rope_t* rope, void* stream) {
  return gqa::run_write(k, k_stride, v, v_stride, cu_seqlens_q, prefix_lens, kv_page_indptr,
                        kv_page_indices, num_page_entries, page_size, num_pages, num_seqs, total_q,
                        Hkv, d, dtype, cache_type, k_pages, v_pages, k_scales, v_scales, rope,
                        stream);
}

int gqa_cache_read(const void* k_pages, const void* v_pages, const void* k_scales,
                   const void* v_scales, int cache_type, const int32_t* kv_page_indptr,
                   const int32_t* kv_page_indices, int num_page_entries, int page_size,
                   int num_pages, const int32_t* kv_indptr, const int32_t* first_keys, int num_seqs,
                   int total_kv, int Hkv, int d, int dtype, void* k_out, void* v_out,
                   void* stream) {
  return gqa::run_read(k_pages, v_pages, k_scales, v_scales, cache_type, kv_page_indptr,
                       kv_page_indices, num_page_entries, page_size, num_pages, kv_indptr,
                       first_keys, num_seqs, total_kv, Hkv, d, dtype, k_out, v_out, stream);
}

}  // extern "C"
