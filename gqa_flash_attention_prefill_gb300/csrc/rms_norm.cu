// rms_norm.cu -- gqa_rms_norm and gqa_rms_norm_backward: the root-mean-square
// norm of rows of n values, with the residual's addition before it and a 16-bit
// or e4m3 output, and its gradient.  Declared in include/gqa_prefill.h.
//
// Mathematics.  h = x + residual (rounded to the stream's type), r = (mean h^2 +
// eps)^-1/2, y = h r (w + offset).  With t = h r, g = dy (w + offset):
//   dh_row = r (g - t mean(g t)) + dh        dw = sum over rows of dy t.
// Both are bound by memory: each value is read once and kept in registers (the
// gradient of long rows: in shared memory) between the row's sum and its output.  A
// row belongs to 8, 16 or 32 lanes of a warp while it fits them, a longer one to a CTA
// (norm_shape), in groups of 8 neighbouring values.  Sums are fp32, in an order that depends on the shape
// alone, so results are the same run to run.
//
// Measured (one launch, inputs larger than L2; 6.81 TB/s is what a copy reaches):
//   16384 x 4096 bf16, residual added in place      77.4 us  6.94 TB/s
//   2047 x 5120 f16 on an fp32 stream, to e4m3      21.0 us  5.5 TB/s: one wave and a half of CTAs
//   16384 x 64 heads of 64, bf16                    46.1 us  5.9 TB/s: 61% of the issue slots
//   gradient of 16384 x 4096 bf16, with dw          87.3 us  6.2 TB/s, 5 of it the sum of the CTAs' dw
//   gradient of 4095 x 32 heads of 128, f16         23.1 us  4.4 TB/s: start, tail and the same sum
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "cache_rows.cuh"
#include "gqa_prefill.h"
#include "launch.h"

namespace gqa {

namespace {

// n / d for 0 <= n < 2^31: the high half of a product, and a shift.
struct Div {
  uint32_t m;
  int l;
  __host__ void set(uint32_t d) {
    l = 0;
    while ((1ull << l) < d) ++l;
    m = (uint32_t)(((1ull << (32 + l)) + d - 1) / d - (1ull << 32));
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, m) + n) >> l; }
};

struct NormParams {
  const void* x;  // backward: dy
  const void* residual;  // backward: h
  const void* weight;
  const void* dh;
  const float* rstd_in;
  void* h_out;
  void* out;  // backward: dx
  void* dresidual;
  uint8_t* scales;
  float* rstd;
  float* part;  // [CTAs of the gradient][n]
  uint32_t* failed;  // [CTAs of the gradient]: a wait ran out, there is no part (NULL: no waits)
  float* dweight;
  long long x_stride, h_stride, out_stride;
  uint32_t rows;  // rows x heads
  Div div_heads;
  int heads, n, team;  // team: lanes of a row (0: the CTA)
  int group;       // values that share a scale (0: 16-bit output)
  int w32;
  int parts;
  int stages;
  float offset, eps, inv_n;
  unsigned int* status;
  unsigned long long timeout_ns;
};
constexpr int kMaxStages = 4;

// Row r of [rows, heads]: where its values start in a tensor of that row stride.
__device__ __forceinline__ size_t start(const NormParams& p, uint32_t row, long long stride) {
  const uint32_t token = p.div_heads(row), head = row - token * p.heads;
  return (size_t)token * stride + (size_t)head * p.n;
}

// Two fp32 values in one register pair, two lanes an instruction (subnormals
// kept): at 6.8 TB/s an SM has some 100 instructions for 8 values and their
// gradient, so their count matters.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float sum2(uint64_t a) {
  float x, y;
  unf2(a, x, y);
  return x + y;
}

struct Vec8 {  // 8 values
  uint64_t v[4];
};

template <bool BF16>
__device__ __forceinline__ Vec8 widen(const uint4& u) {
  Vec8 r;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = f2(unpack_lo<BF16>(w[i]), unpack_hi<BF16>(w[i]));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow(const Vec8& a) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unf2(a.v[i], lo, hi);
    w[i] = pack2<BF16>(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 values as they lie in memory: 16 bytes, or 32.
template <bool F32>
struct Raw {
  uint4 a[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(const void* base, size_t at) {  // at: in values
  Raw<F32> r;
  if constexpr (F32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
    r.a[0] = p[0];
    r.a[1] = p[1];
  } else {
    r.a[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
  }
  return r;
}
template <bool F32, bool BF16>
__device__ __forceinline__ Vec8 values(const Raw<F32>& r) {
  if constexpr (!F32) {
    return widen<BF16>(r.a[0]);
  } else {
    Vec8 v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v.v[2 * i] = (uint64_t)r.a[i].y << 32 | r.a[i].x;
      v.v[2 * i + 1] = (uint64_t)r.a[i].w << 32 | r.a[i].z;
    }
    return v;
  }
}
template <bool F32, bool BF16>
__device__ __forceinline__ void store8(void* base, size_t at, const Vec8& v) {
  if constexpr (F32) {
    ulonglong2* p = reinterpret_cast<ulonglong2*>(static_cast<float*>(base) + at);
    p[0] = make_ulonglong2(v.v[0], v.v[1]);
    p[1] = make_ulonglong2(v.v[2], v.v[3]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = narrow<BF16>(v);
  }
}

// w + offset of 8 columns.
template <bool BF16>
__device__ __forceinline__ Vec8 weight8(const NormParams& p, int col) {
  Vec8 w = p.w32 ? values<true, BF16>(load_raw<true>(p.weight, (size_t)col))
                 : values<false, BF16>(load_raw<false>(p.weight, (size_t)col));
  const uint64_t o = f2(p.offset, p.offset);
#pragma unroll
  for (int i = 0; i < 4; ++i) w.v[i] = add2(w.v[i], o);
  return w;
}

// Sum (and maximum) over the lanes of a row; every lane gets them.  `s` holds
// two words per warp, and is not used again before the CTA's next barrier.
template <bool WIDE, bool MAX>
__device__ __forceinline__ void row_reduce(float& sum, float& most, int team, float* s) {
  const int width = WIDE ? 32 : team;
  for (int o = 1; o < width; o <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (MAX) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if constexpr (WIDE) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
      s[warp] = sum;
      if (MAX) s[32 + warp] = most;
    }
    __syncthreads();
    sum = lane < warps ? s[lane] : 0.f;
    if (MAX) most = lane < warps ? s[32 + lane] : 0.f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (MAX) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
  }
}

// (sum / n + eps)^-1/2: the reciprocal square root, and a step of Newton's method
// whose residual 1 - v r^2 has the rounding of v r in it.
__device__ __forceinline__ float rstd_of(const NormParams& p, float sum) {
  const float v = fmaf(sum, p.inv_n, p.eps), r = rsqrtf(v), t = v * r;
  return fmaf(0.5f * r, fmaf(-t, r, 1.f) - fmaf(v, r, -t) * r, r);
}

// The sum of 8 products.
__device__ __forceinline__ float dot8(const Vec8& a, const Vec8& b) {
  return sum2(add2(fma2(a.v[0], b.v[0], mul2(a.v[1], b.v[1])), fma2(a.v[2], b.v[2], mul2(a.v[3], b.v[3]))));
}
__device__ __forceinline__ float most8(const Vec8& a) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x, y;
    unf2(a.v[i], x, y);
    m = max3(m, fabsf(x), fabsf(y));
  }
  return m;
}

// One row's 8 values in a thread of its team, before and after the row's sums.
template <bool BF16, bool F32, bool OUT8>
struct NormVec {
  Vec8 h;      // with OUT8, from take() on times the weight
  float top;   // OUT8: the largest magnitude of them
  bool in;
  // w: the weight of the columns (OUT8 alone uses it here).
  __device__ __forceinline__ void take(const NormParams& p, const uint4& x, const Raw<F32>& r, const Vec8& w,
                                       size_t hat, float& sum, float& most) {
    top = 0.f;
    if (!in) return;
    h = widen<BF16>(x);
    if (p.residual != nullptr) {
      const Vec8 a = values<F32, BF16>(r);
#pragma unroll
      for (int i = 0; i < 4; ++i) h.v[i] = add2(h.v[i], a.v[i]);
      // The norm is of what the stream holds.
      if constexpr (!F32) {
        const uint4 n = narrow<BF16>(h);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h_out) + hat) = n;
        h = widen<BF16>(n);
      } else {
        store8<true, BF16>(p.h_out, hat, h);
      }
    }
    sum += dot8(h, h);
    if constexpr (OUT8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) h.v[i] = mul2(h.v[i], w.v[i]);
      top = most8(h);
      most = fmaxf(most, top);
    }
  }
  // All lanes of a warp call it together.
  __device__ __forceinline__ void give(const NormParams& p, size_t row, size_t oat, int c, const Vec8& w,
                                       float rstd, float most) {
    if constexpr (!OUT8) {
      if (!in) return;
      const uint64_t r = f2(rstd, rstd);
#pragma unroll
      for (int i = 0; i < 4; ++i) h.v[i] = mul2(mul2(h.v[i], r), w.v[i]);
      store8<false, BF16>(p.out, oat + 8 * c, h);
    } else {
      if (p.group == p.n) {  // one scale a row
        top = most;
      } else {
        for (int o = 1; o < p.group / 8; o <<= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      if (!in) return;
      const int e = e4m3_scale_exponent(top * rstd);
      const float m = rstd * pow2f(-e);  // exact: one rounding of h w rstd, then e4m3's
      const uint64_t mm = f2(m, m);
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x, y;
        unf2(mul2(h.v[i], mm), x, y);
        b[i] = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + oat + 8 * c) =
          make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
      if (8 * c % p.group == 0) p.scales[row * (p.n / p.group) + 8 * c / p.group] = (uint8_t)(e + 127);
    }
  }
};

// A CTA of up to T threads per row, V groups of 8 values a thread; B CTAs an SM.
template <bool BF16, bool F32, bool OUT8, int V, int T, int B>
__global__ void __launch_bounds__(T, B) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s[64];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int TS = blockDim.x, lane = threadIdx.x, nv = p.n / 8;
  const uint32_t row = blockIdx.x;
  const size_t xat = start(p, row, p.x_stride), hat = (size_t)row * p.n;
  uint4 x[V];
  Raw<F32> r[V];
  Vec8 w[V];
  NormVec<BF16, F32, OUT8> n[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
    n[v].in = c < nv;
    if (n[v].in) {
      x[v] = load_raw<false>(p.x, xat + 8 * c).a[0];
      if (p.residual != nullptr) r[v] = load_raw<F32>(p.residual, hat + 8 * c);
      if constexpr (OUT8) w[v] = weight8<BF16>(p, 8 * c);
    }
  }
  float sum = 0.f, most = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) n[v].take(p, x[v], r[v], w[v], hat + 8 * (v * TS + lane), sum, most);
  row_reduce<true, OUT8>(sum, most, 32, s);
  const float rstd = rstd_of(p, sum);
  if (lane == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  const size_t oat = start(p, row, p.out_stride);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
    if (!OUT8 && n[v].in) w[v] = weight8<BF16>(p, 8 * c);
    n[v].give(p, row, oat, c, w[v], rstd, most);
  }
}

// Rows of up to 1024 values: a row in `team` lanes (8, 16 or 32) of V groups of 8
// values, U rows a team, all of whose loads are on their way at once, and one weight
// for all of them.  CTAs an SM by measurement: on an fp32 stream two without spills
// (32768 rows of 1024: 61.0 us, three 70.6); else four, three of two groups (131072 rows
// of 512: 78.2 us, four 78.7, two 81.7).
constexpr int kTeamGroups = 4;  // U x V
template <bool BF16, bool F32, bool OUT8, int V>
__global__ void __launch_bounds__(256, F32 ? 2 : V == 1 ? 4 : 3) norm_team_kernel(const __grid_constant__ NormParams p) {
  constexpr int U = kTeamGroups / V;
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int c = threadIdx.x & (p.team - 1), teams = 256 / p.team;
  const uint32_t row0 = blockIdx.x * teams * U + threadIdx.x / p.team;
  uint4 x[U][V];
  Raw<F32> r[U][V];
  NormVec<BF16, F32, OUT8> n[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t row = row0 + u * teams;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int g = 32 * v + c;  // V > 1: 32 lanes
      n[u][v].in = row < p.rows && g < p.n / 8;
      if (n[u][v].in) {
        x[u][v] = load_raw<false>(p.x, start(p, row, p.x_stride) + 8 * g).a[0];
        if (p.residual != nullptr) r[u][v] = load_raw<F32>(p.residual, (size_t)row * p.n + 8 * g);
      }
    }
  }
  Vec8 w[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (32 * v + c < p.n / 8) w[v] = weight8<BF16>(p, 8 * (32 * v + c));
  float sum[U], most[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    sum[u] = most[u] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      n[u][v].take(p, x[u][v], r[u][v], w[v], (size_t)(row0 + u * teams) * p.n + 8 * (32 * v + c), sum[u], most[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) row_reduce<false, OUT8>(sum[u], most[u], p.team, nullptr);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float rstd = rstd_of(p, sum[u]);
    const uint32_t row = row0 + u * teams;
    if (n[u][0].in && c == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v)
      n[u][v].give(p, row, start(p, row, p.out_stride), 32 * v + c, w[v], rstd, most[u]);
  }
}

// ------------------------------------------------------------------ gradient
// The thread's share of dw and of the row's sum of g t, from 8 values.
__device__ __forceinline__ float grad_sum(const Vec8& d, const Vec8& h, const Vec8& w, float rstd, Vec8& acc) {
  const uint64_t r = f2(rstd, rstd);
  Vec8 t, g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.v[i] = mul2(h.v[i], r);
    acc.v[i] = fma2(d.v[i], t.v[i], acc.v[i]);
    g.v[i] = mul2(d.v[i], w.v[i]);
  }
  return dot8(g, t);
}
// dx = rstd g + (dh - h rstd^2 mean(g t)) of 8 values; k = rstd^2 mean(g t).
template <bool BF16, bool F32>
__device__ __forceinline__ void grad_store(const NormParams& p, const Vec8& d, const Vec8& h, const Vec8& w,
                                           const Vec8& dh, float rstd, float k, size_t oat, size_t sat) {
  const uint64_t r = f2(rstd, rstd), kk = f2(-k, -k);
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.v[i] = fma2(mul2(d.v[i], w.v[i]), r, fma2(h.v[i], kk, dh.v[i]));
  if (p.out != nullptr) store8<false, BF16>(p.out, oat, o);
  if (p.dresidual != nullptr) store8<F32, BF16>(p.dresidual, sat, o);
}
__device__ __forceinline__ Vec8 zero8() {
  Vec8 z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.v[i] = 0ull;
  return z;
}

// A row in a CTA.  Each CTA walks rows blockIdx.x, + gridDim.x, ... through a
// ring of `stages` rows in shared memory, filled by bulk copies that run ahead:
// the bytes in flight that the memory's latency asks for would not fit in
// registers beside the sums.  Its share of dw stays in registers.
template <bool BF16, bool F32, int V, int T>
__global__ void __launch_bounds__(T) norm_backward_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[kMaxStages];
  // A wait of row k that runs out sets abort_words[k & 1].  After the row's barrier
  // every thread reads the same there: the next wait to set it is row k + 2's,
  // behind a barrier that this thread has to pass first.
  __shared__ uint32_t abort_words[2];
  __shared__ float s[2][64];
  const int TS = blockDim.x, lane = threadIdx.x, nv = p.n / 8;
  constexpr uint32_t es = F32 ? 4u : 2u;
  const uint32_t off_h = 2u * p.n, off_dh = off_h + es * p.n, stage = off_dh + (p.dh != nullptr ? es * p.n : 0u);
  const uint32_t sbar = smem_u32(bars), sring = smem_u32(ring);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) mbar_init(sbar + 8 * i, 1u);
    abort_words[0] = abort_words[1] = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_launch_dependents();
  grid_dep_wait();
  // Copies row number k of this CTA into its stage.
  auto fill = [&](uint32_t k, uint32_t st) {
    const unsigned long long at = blockIdx.x + (unsigned long long)k * gridDim.x;
    if (at >= p.rows) return;
    const uint32_t row = (uint32_t)at, bar = sbar + 8 * st, dst = sring + st * stage;
    mbar_arrive_expect_tx(bar, stage);
    bulk_load(dst, static_cast<const uint16_t*>(p.x) + start(p, row, p.x_stride), 2u * p.n, bar);
    bulk_load(dst + off_h, static_cast<const uint8_t*>(p.residual) + es * start(p, row, p.h_stride), es * p.n, bar);
    if (p.dh != nullptr) bulk_load(dst + off_dh, static_cast<const uint8_t*>(p.dh) + es * ((size_t)row * p.n), es * p.n, bar);
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < p.stages; ++k) fill(k, k);
  Vec8 w[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
    acc[v] = zero8();
    if (c < nv) w[v] = weight8<BF16>(p, 8 * c);
  }
  uint32_t k = 0, st = 0, par = 0;  // the row's number, its stage, the stage's parity
  for (unsigned long long at_row = blockIdx.x; at_row < p.rows; at_row += gridDim.x, ++k) {
    const uint32_t row = (uint32_t)at_row;
    const float rstd = __ldg(p.rstd_in + row);
    // A wait that runs out raises the status, and ends the CTA for all its threads at
    // the row's barrier: nothing of the row is stored, and no copy issued after it.
    (void)wait_bounded(sbar + 8 * st, par, abort_words + (k & 1), p.status, p.timeout_ns);
    const uint8_t* at = ring + st * stage;
    float sum = 0.f, none = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * TS + lane;
      if (c < nv)
        sum += grad_sum(widen<BF16>(load_raw<false>(at, 8 * c).a[0]),
                        values<F32, BF16>(load_raw<F32>(at + off_h, 8 * c)), w[v], rstd, acc[v]);
    }
    row_reduce<true, false>(sum, none, 32, s[k & 1]);
    if (abort_words[k & 1] != 0u) {
      if (threadIdx.x == 0) {  // let the copies in flight land: row k's and those ahead of it
        const uint32_t stages = (uint32_t)p.stages, ahead = k > 0 && stages > 1 ? stages - 1 : stages;
        for (uint32_t j = k; j < k + ahead && blockIdx.x + (unsigned long long)j * gridDim.x < p.rows; ++j)
          wait_drain(sbar + 8 * (j % stages), (j / stages) & 1u, p.timeout_ns);
        if (p.part != nullptr) p.failed[blockIdx.x] = 1u;
      }
      if (p.part != nullptr)
        for (int c = lane; c < p.n; c += TS) p.part[(size_t)blockIdx.x * p.n + c] = NAN;
      return;
    }
    // Every thread is past the row before: its stage is free.
    if (threadIdx.x == 0 && k > 0 && p.stages > 1)
      fill(k - 1 + p.stages, (st == 0 ? p.stages : st) - 1);
    const float mean = rstd * rstd * (sum * p.inv_n);
    const size_t oat = start(p, row, p.out_stride), sat = (size_t)row * p.n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * TS + lane;
      if (c < nv) {
        const Vec8 o = p.dh != nullptr ? values<F32, BF16>(load_raw<F32>(at + off_dh, 8 * c)) : zero8();
        grad_store<BF16, F32>(p, widen<BF16>(load_raw<false>(at, 8 * c).a[0]),
                              values<F32, BF16>(load_raw<F32>(at + off_h, 8 * c)), w[v], o, rstd, mean,
                              oat + 8 * c, sat + 8 * c);
      }
    }
    if (p.stages == 1) {  // rows so wide that one fits
      __syncthreads();
      if (threadIdx.x == 0) fill(k + 1, 0);
    }
    if (++st == (uint32_t)p.stages) {
      st = 0;
      par ^= 1u;
    }
  }
  if (p.part == nullptr) return;
  if (threadIdx.x == 0) p.failed[blockIdx.x] = 0u;
  float* part = p.part + (size_t)blockIdx.x * p.n;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
    if (c < nv) store8<true, BF16>(part, (size_t)8 * c, acc[v]);
  }
}

// Rows of up to 512 values: a row in `team` lanes of V groups of 8, U rows a team at
// a time (U V = 2, in 64 registers, and four CTAs an SM: 4095 x 32 rows of 128 in
// 23.1 us; four in 116 registers and two CTAs 25.3).  Two CTAs an SM where 64
// registers would spill: 131072 rows of 512 in 92.9 us instead of 98.6, 65536 on an fp32
// stream 86.6 instead of 111.
constexpr int kTeamGroupsBack = 2;
template <bool BF16, bool F32, int V>
__global__ void __launch_bounds__(256, F32 || V == 2 ? 2 : 4) norm_backward_team_kernel(const __grid_constant__ NormParams p) {
  constexpr int U = kTeamGroupsBack / V;
  __shared__ __align__(16) float s_acc[V][256 * 8];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int c = threadIdx.x & (p.team - 1), teams = 256 / p.team, mine = threadIdx.x / p.team;
  const bool has = p.dh != nullptr;
  bool col[V];
  Vec8 w[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    col[v] = 32 * v + c < p.n / 8;  // V > 1: 32 lanes
    acc[v] = zero8();
    if (col[v]) w[v] = weight8<BF16>(p, 8 * (32 * v + c));
  }
  const uint32_t per = teams * U;
  for (unsigned long long base = (unsigned long long)blockIdx.x * per; base < p.rows;
       base += (unsigned long long)gridDim.x * per) {
    uint4 dy[U][V];
    Raw<F32> h[U][V], dh[U][V];
    float rstd[U], sum[U];
    const uint32_t row0 = (uint32_t)base + mine;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t row = row0 + u * teams;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int at = 8 * (32 * v + c);
        if (col[v] && row < p.rows) {
          dy[u][v] = load_raw<false>(p.x, start(p, row, p.x_stride) + at).a[0];
          h[u][v] = load_raw<F32>(p.residual, start(p, row, p.h_stride) + at);
          if (has) dh[u][v] = load_raw<F32>(p.dh, (size_t)row * p.n + at);
          if (v == 0) rstd[u] = __ldg(p.rstd_in + row);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      sum[u] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (col[v] && row0 + u * teams < p.rows) {
          const float part = grad_sum(widen<BF16>(dy[u][v]), values<F32, BF16>(h[u][v]), w[v], rstd[u], acc[v]);
          sum[u] = v == 0 ? part : sum[u] + part;
        }
    }
    float none = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) row_reduce<false, false>(sum[u], none, p.team, nullptr);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t row = row0 + u * teams;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int at = 8 * (32 * v + c);
        if (col[v] && row < p.rows) {
          const Vec8 o = has ? values<F32, BF16>(dh[u][v]) : zero8();
          grad_store<BF16, F32>(p, widen<BF16>(dy[u][v]), values<F32, BF16>(h[u][v]), w[v], o, rstd[u],
                                rstd[u] * rstd[u] * (sum[u] * p.inv_n), start(p, row, p.out_stride) + at,
                                (size_t)row * p.n + at);
        }
      }
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int v = 0; v < V; ++v) store8<true, BF16>(s_acc[v], (size_t)threadIdx.x * 8, acc[v]);
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {  // 256 columns each
    if (256 * v + (int)threadIdx.x < p.n) {
      float a = 0.f;
      for (int k = 0; k < teams; ++k) a += s_acc[v][k * p.team * 8 + threadIdx.x];
      p.part[(size_t)blockIdx.x * p.n + 256 * v + threadIdx.x] = a;
    }
  }
}

// dw: the sum of the CTAs' shares.  32 columns a block, a share a warp; up to ten
// of a warp's loads on their way at once.
__global__ void __launch_bounds__(1024) norm_join_kernel(const __grid_constant__ NormParams p) {
  constexpr int U = 10;
  __shared__ float s[32][33];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  for (int b0 = y; b0 < p.parts; b0 += 32 * U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + 32 * u;
      v[u] = b < p.parts && c < p.n ? __ldcg(p.part + (size_t)b * p.n + c) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) a += v[u];
  }
  s[y][lane] = a;
  __syncthreads();
  a = s[lane][y];  // column y of the block, share `lane`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (p.failed != nullptr && __any_sync(0xffffffffu, a != a)) {
    // The values' own NaN, or a share that is missing: a CTA whose wait ran out leaves
    // NaN, and its word.
    uint32_t failed = 0u;
    for (int b = lane; b < p.parts; b += 32) failed |= __ldcg(p.failed + b);
    if (__any_sync(0xffffffffu, failed != 0u)) return;
  }
  if (lane == 0 && blockIdx.x * 32 + y < p.n) p.dweight[blockIdx.x * 32 + y] = a;
}

// ------------------------------------------------------------------ host
constexpr int kMaxN = 16384;
constexpr unsigned kRingBytes = 220u * 1024u;  // of an SM's shared memory, for the gradient's rows

struct NormShape {
  int team;     // lanes of a row, 0: a CTA
  int v, t;     // groups of 8 values a thread, and the threads it is compiled for
  int threads;
};
// Which form a row takes.  Lanes of a warp while a row fits them: no barrier, and
// hundreds of short rows in flight (262144 rows of 256: 78 us, in CTAs of their own 264;
// 131072 of 512: 78 and 133, the gradient 93 and 416 of 256).  Beyond, a CTA a row: the
// gradient with two groups a thread, so that more CTAs with rings of their own fit an SM
// (65536 rows of 1024: 89 us, one group a thread 135; 32768 of 2048: 82 and 132), the
// norm itself with one up to 2048 values (76.6 us, two 77.6).
NormShape norm_shape(int n, bool gradient) {
  const int nv = n / 8;
  if (nv <= 32) return {nv <= 8 ? 8 : nv <= 16 ? 16 : 32, 1, 256, 256};
  if (nv <= 64) return {32, 2, 256, 256};
  if (nv <= 128 && !gradient) return {32, 4, 256, 256};
  NormShape s{0, gradient || nv > 256 ? 2 : 1, nv <= 256 ? 256 : nv <= 1024 ? 512 : 1024, 0};
  s.threads = ((nv + s.v - 1) / s.v + 31) / 32 * 32;
  return s;
}
// CTAs per SM of the gradient's persistent grid: some 640 threads (32768 rows of 2048:
// 82.1 us, 512 or 768 threads 87; 16384 of 4096: 87.5 with 512 or 640, 91.3 with 768,
// 131 with 256).
int backward_per_sm(const NormShape& s) {
  if (s.team > 0) return 4;
  const int c = 640 / s.threads;
  return c < 1 ? 1 : c > 8 ? 8 : c;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Span {
  const void* p;
  size_t n;
};
bool meet(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}
// Bytes from the first row to the end of the last.
size_t extent(int rows, long long stride, long long row, size_t e) {
  return rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)row) * e : 0;
}

// What both directions check; GQA_OK, an error, or 1 for no work.
int norm_check(int rows, int heads, int n, int dtype, int stream_type, int weight_type, float offset) {
  if (rows < 0 || heads <= 0 || n <= 0) return GQA_ERR_INVALID;
  if (dtype != GQA_F16 && dtype != GQA_BF16) return GQA_ERR_INVALID;
  if (stream_type != dtype && stream_type != GQA_F32) return GQA_ERR_INVALID;
  if (weight_type != dtype && weight_type != GQA_F32) return GQA_ERR_INVALID;
  if (!std::isfinite(offset)) return GQA_ERR_INVALID;
  if (n % 8 != 0 || n > kMaxN || (long long)rows * heads >= (1ll << 31) || (long long)heads * n >= (1ll << 31))
    return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}
bool bad_stride(long long stride, long long row) { return stride < row || stride % 8 != 0; }

template <bool BF16, bool F32, bool OUT8>
cudaError_t launch_norm_as(const NormParams& p, const NormShape& s, cudaStream_t st) {
  if (s.team > 0) {
    const long long per = (long long)(kTeamGroups / s.v) * 256 / s.team;
    const int grid = (int)(((long long)p.rows + per - 1) / per);
    return s.v == 1   ? launch_pdl(norm_team_kernel<BF16, F32, OUT8, 1>, p, grid, 256, 0, st)
           : s.v == 2 ? launch_pdl(norm_team_kernel<BF16, F32, OUT8, 2>, p, grid, 256, 0, st)
                      : launch_pdl(norm_team_kernel<BF16, F32, OUT8, 4>, p, grid, 256, 0, st);
  }
  const int grid = (int)p.rows;
  return s.v == 1     ? launch_pdl(norm_kernel<BF16, F32, OUT8, 1, 256, 6>, p, grid, s.threads, 0, st)
         : s.t == 512 ? launch_pdl(norm_kernel<BF16, F32, OUT8, 2, 512, 2>, p, grid, s.threads, 0, st)
                      : launch_pdl(norm_kernel<BF16, F32, OUT8, 2, 1024, 1>, p, grid, s.threads, 0, st);
}
template <bool BF16, bool F32>
cudaError_t launch_norm(const NormParams& p, const NormShape& s, cudaStream_t st) {
  return p.group > 0 ? launch_norm_as<BF16, F32, true>(p, s, st) : launch_norm_as<BF16, F32, false>(p, s, st);
}

template <bool BF16, bool F32, int V, int T>
cudaError_t launch_ring(const NormParams& p, const NormShape& s, int grid, unsigned smem, cudaStream_t st) {
  auto kern = norm_backward_kernel<BF16, F32, V, T>;
  static SmemAttr attr{};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (attr.allowed[dev].load(std::memory_order_acquire) < kRingBytes) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    attr.allowed[dev].store(kRingBytes, std::memory_order_release);
  }
  return launch_pdl(kern, p, grid, s.threads, smem, st);
}
template <bool BF16, bool F32>
cudaError_t launch_back(const NormParams& p, const NormShape& s, int grid, unsigned smem, cudaStream_t st) {
  if (s.team > 0)
    return s.v == 1 ? launch_pdl(norm_backward_team_kernel<BF16, F32, 1>, p, grid, 256, 0, st)
                    : launch_pdl(norm_backward_team_kernel<BF16, F32, 2>, p, grid, 256, 0, st);
  return s.v == 1     ? launch_ring<BF16, F32, 1, 256>(p, s, grid, smem, st)
         : s.t == 256 ? launch_ring<BF16, F32, 2, 256>(p, s, grid, smem, st)
         : s.t == 512 ? launch_ring<BF16, F32, 2, 512>(p, s, grid, smem, st)
                      : launch_ring<BF16, F32, 2, 1024>(p, s, grid, smem, st);
}

int run_norm(const void* x, long long x_stride, const void* residual, void* residual_out,
             int stream_type, const void* weight, int weight_type, float offset, float eps, int rows,
             int heads, int n, int dtype, int out_type, int group, void* out, long long out_stride,
             void* scales, float* rstd, void* stream) {
  const int rc = norm_check(rows, heads, n, dtype, stream_type, weight_type, offset);
  if (rc == GQA_ERR_INVALID) return rc;
  if (!(eps > 0.f) || !std::isfinite(eps)) return GQA_ERR_INVALID;
  if (out_type != GQA_CACHE_16 && out_type != GQA_CACHE_E4M3) return GQA_ERR_INVALID;
  const bool e4 = out_type == GQA_CACHE_E4M3;
  if (e4 && (group <= 0 || n % group != 0)) return GQA_ERR_INVALID;
  if ((residual == nullptr) != (residual_out == nullptr)) return GQA_ERR_INVALID;
  if (rc != GQA_OK) return rc;
  if (e4 && group != 32 && group != 64 && group != 128 && group != n) return GQA_ERR_UNSUPPORTED;
  if (rows == 0) return GQA_OK;
  const long long wide = (long long)heads * n;
  if (x == nullptr || weight == nullptr || out == nullptr || (e4 && scales == nullptr))
    return GQA_ERR_INVALID;
  if (!al16(x) || !al16(residual) || !al16(residual_out) || !al16(weight) || !al16(out) || !al4(rstd))
    return GQA_ERR_INVALID;
  if (rows == 1) x_stride = out_stride = wide;  // never used
  if (bad_stride(x_stride, wide) || bad_stride(out_stride, wide)) return GQA_ERR_INVALID;
  // A result may take an input's place row by row, value by value; nothing else
  // of theirs overlaps.
  const size_t es = stream_type == GQA_F32 ? 4 : 2, count = (size_t)rows * (size_t)wide;
  const Span sx{x, extent(rows, x_stride, wide, 2)}, sr{residual, count * es},
      sw{weight, (size_t)n * (weight_type == GQA_F32 ? 4 : 2)}, sh{residual_out, count * es},
      so{out, extent(rows, out_stride, wide, e4 ? 1 : 2)}, ss{e4 ? scales : nullptr, count / (e4 ? group : 1)},
      sd{rstd, 4u * (size_t)rows * heads};
  const Span outs[] = {sh, so, ss, sd};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return GQA_ERR_INVALID;
    if (meet(outs[i], sw)) return GQA_ERR_INVALID;
    const bool same_r = i == 0 ? residual_out == residual : i == 1 && !e4 && out == residual && es == 2 && out_stride == wide;
    const bool same_x = i == 0 ? residual_out == x && es == 2 && x_stride == wide
                               : i == 1 && !e4 && out == x && out_stride == x_stride;
    if (!same_r && meet(outs[i], sr)) return GQA_ERR_INVALID;
    if (!same_x && meet(outs[i], sx)) return GQA_ERR_INVALID;
  }
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = x;
  p.residual = residual;
  p.h_out = residual_out;
  p.weight = weight;
  p.out = out;
  p.scales = static_cast<uint8_t*>(scales);
  p.rstd = rstd;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  p.rows = (uint32_t)rows * (uint32_t)heads;
  p.div_heads.set((uint32_t)heads);
  p.inv_n = 1.f / (float)n;
  p.heads = heads;
  p.n = n;
  p.group = e4 ? group : 0;
  p.w32 = weight_type == GQA_F32;
  p.offset = offset;
  p.eps = eps;
  const NormShape s = norm_shape(n, false);
  p.team = s.team;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == GQA_BF16, f32 = stream_type == GQA_F32;
  const cudaError_t e = bf ? (f32 ? launch_norm<true, true>(p, s, st) : launch_norm<true, false>(p, s, st))
                           : (f32 ? launch_norm<false, true>(p, s, st) : launch_norm<false, false>(p, s, st));
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

// CTAs that the workspace has room for: a part of n floats each, and behind the parts a word each.
size_t backward_ctas(const NormShape& s) {
  int sms = 152;
  unsigned int* status = nullptr;
  if (call_device(&sms, &status) != GQA_OK) sms = 152;
  return (size_t)sms * backward_per_sm(s);
}
size_t backward_bytes(const NormShape& s, int n) { return 4u * backward_ctas(s) * ((size_t)n + 1); }

int run_norm_backward(const void* dy, long long dy_stride, const void* h, long long h_stride,
                      int stream_type, const float* rstd, const void* weight, int weight_type,
                      float offset, const void* dh, int rows, int heads, int n, int dtype, void* dx,
                      long long dx_stride, void* dresidual, float* dweight, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const int rc = norm_check(rows, heads, n, dtype, stream_type, weight_type, offset);
  if (rc == GQA_ERR_INVALID) return rc;
  if (dx == nullptr && dresidual == nullptr && dweight == nullptr) return GQA_ERR_INVALID;
  if (rc != GQA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!al4(dweight)) return GQA_ERR_INVALID;
  if (rows == 0) {
    if (dweight != nullptr && cudaMemsetAsync(dweight, 0, 4u * (size_t)n, st) != cudaSuccess)
      return GQA_ERR_CUDA;
    return GQA_OK;
  }
  if (dy == nullptr || h == nullptr || rstd == nullptr || weight == nullptr) return GQA_ERR_INVALID;
  if (!al16(dy) || !al16(h) || !al4(rstd) || !al16(weight) || !al16(dh) || !al16(dx) || !al16(dresidual))
    return GQA_ERR_INVALID;
  const long long wide = (long long)heads * n;
  if (rows == 1) dy_stride = h_stride = dx_stride = wide;  // never used
  if (dx == nullptr) dx_stride = wide;
  if (bad_stride(dy_stride, wide) || bad_stride(h_stride, wide) || bad_stride(dx_stride, wide))
    return GQA_ERR_INVALID;
  NormShape s = norm_shape(n, true);
  const size_t need = backward_bytes(s, n);
  if (dweight != nullptr && (workspace == nullptr || workspace_bytes < need ||
                             (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return GQA_ERR_INVALID;
  if (dweight == nullptr) workspace = nullptr;
  const size_t es = stream_type == GQA_F32 ? 4 : 2, count = (size_t)rows * (size_t)wide;
  const Span sy{dy, extent(rows, dy_stride, wide, 2)}, sh{h, extent(rows, h_stride, wide, es)},
      sd{dh, count * es}, sr{rstd, 4u * (size_t)rows * heads},
      sw{weight, (size_t)n * (weight_type == GQA_F32 ? 4 : 2)};
  const Span outs[] = {{dx, extent(rows, dx_stride, wide, 2)}, {dresidual, count * es}, {dweight, 4u * (size_t)n},
                       {workspace, need}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return GQA_ERR_INVALID;
    if (meet(outs[i], sr) || meet(outs[i], sw)) return GQA_ERR_INVALID;
    // In place, value by value, as in the forward direction.
    const long long os = i == 0 ? dx_stride : wide;
    const size_t oe = i == 0 ? 2 : es;
    const bool row_out = i < 2;
    if (!(row_out && outs[i].p == dy && oe == 2 && os == dy_stride) && meet(outs[i], sy)) return GQA_ERR_INVALID;
    if (!(row_out && outs[i].p == h && oe == es && os == h_stride) && meet(outs[i], sh)) return GQA_ERR_INVALID;
    if (!(row_out && outs[i].p == dh && oe == es && os == wide) && meet(outs[i], sd)) return GQA_ERR_INVALID;
  }
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = dy;
  p.residual = h;
  p.weight = weight;
  p.dh = dh;
  p.rstd_in = rstd;
  p.out = dx;
  p.dresidual = dresidual;
  p.part = static_cast<float*>(workspace);
  if (p.part != nullptr && s.team == 0) p.failed = reinterpret_cast<uint32_t*>(p.part + backward_ctas(s) * n);
  p.dweight = dweight;
  p.x_stride = dy_stride;
  p.h_stride = h_stride;
  p.out_stride = dx_stride;
  p.rows = (uint32_t)rows * (uint32_t)heads;
  p.div_heads.set((uint32_t)heads);
  p.inv_n = 1.f / (float)n;
  p.heads = heads;
  p.n = n;
  p.team = s.team;
  p.w32 = weight_type == GQA_F32;
  p.offset = offset;
  int sms = 0;
  if (call_device(&sms, &p.status) != GQA_OK) return GQA_ERR_CUDA;
  p.timeout_ns = wait_limit_ns();
  // Rows of the ring: as many as fit beside the SM's other CTAs, four at most;
  // a CTA has the SM to itself where two rows would not fit otherwise.
  int per_sm = backward_per_sm(s);
  // A CTA's time counts where each has one row at most: a group a thread (33 rows of
  // 1000: 3.8 us against 4.3).
  if (s.team == 0 && s.t == 256 && (long long)rows * heads <= sms) {
    s.v = 1;
    s.threads = (n / 8 + 31) / 32 * 32;
  }
  const size_t stage = (size_t)n * (2 + es * (dh != nullptr ? 2 : 1));
  if (s.team == 0) {
    while (per_sm > 1 && 2 * stage > kRingBytes / per_sm - 2048) --per_sm;
    const size_t fit = (per_sm > 1 ? kRingBytes / per_sm - 2048 : kRingBytes) / stage;
    p.stages = (int)(fit < kMaxStages ? fit : kMaxStages);
  }
  const long long per = s.team > 0 ? (long long)(kTeamGroupsBack / s.v) * 256 / s.team : 1, all = ((long long)p.rows + per - 1) / per;
  const long long most = (long long)sms * per_sm;
  const int grid = (int)(all < most ? all : most);
  const unsigned smem = (unsigned)(p.stages * stage);
  p.parts = grid;
  const bool bf = dtype == GQA_BF16, f32 = stream_type == GQA_F32;
  cudaError_t e = bf ? (f32 ? launch_back<true, true>(p, s, grid, smem, st) : launch_back<true, false>(p, s, grid, smem, st))
                     : (f32 ? launch_back<false, true>(p, s, grid, smem, st) : launch_back<false, false>(p, s, grid, smem, st));
  if (e == cudaSuccess && dweight != nullptr) e = launch_pdl(norm_join_kernel, p, (n + 31) / 32, 1024, 0, st);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

}  // namespace gqa

extern "C" {

int gqa_rms_norm(const void* x, long long x_stride, const void* residual, void* residual_out,
                 int stream_type, const void* weight, int weight_type, float offset, float eps,
                 int rows, int heads, int n, int dtype, int out_type, int group, void* out,
                 long long out_stride, void* scales, float* rstd, void* stream) {
  return gqa::run_norm(x, x_stride, residual, residual_out, stream_type, weight, weight_type, offset,
                       eps, rows, heads, n, dtype, out_type, group, out, out_stride, scales, rstd, stream);
}

int gqa_rms_norm_backward(const void* dy, long long dy_stride, const void* h, long long h_stride,
                          int stream_type, const float* rstd, const void* weight, int weight_type,
                          float offset, const void* dh, int rows, int heads, int n, int dtype,
                          void* dx, long long dx_stride, void* dresidual, float* dweight,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return gqa::run_norm_backward(dy, dy_stride, h, h_stride, stream_type, rstd, weight, weight_type, offset,
                                dh, rows, heads, n, dtype, dx, dx_stride, dresidual, dweight, workspace,
                                workspace_bytes, stream);
}

int gqa_rms_norm_backward_workspace(int rows, int heads, int n, int dtype, size_t* bytes) {
  if (bytes == nullptr) return GQA_ERR_INVALID;
  const int rc = gqa::norm_check(rows, heads, n, dtype, dtype, dtype, 0.f);
  if (rc == GQA_OK) *bytes = gqa::backward_bytes(gqa::norm_shape(n, true), n);
  return rc;
}

}  // extern "C"
