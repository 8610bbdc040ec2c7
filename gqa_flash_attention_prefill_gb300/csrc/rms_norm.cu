// rms_norm.cu -- gqa_rms_norm and gqa_rms_norm_backward: the root-mean-square
// norm of rows of n values, with the residual's addition before it and a 16-bit
// or e4m3 output, and its gradient.  Declared in include/gqa_prefill.h.
//
// Mathematics.  h = x + residual (rounded to the stream's type), r = (mean h^2 +
// eps)^-1/2, y = h r (w + offset).  With t = h r, g = dy (w + offset):
//   dh_row = r (g - t mean(g t)) + dh        dw = sum over rows of dy t.
// Both are bound by memory: each value is read once and kept in registers
// between the row's sum and its output.  A row of up to 1024 values belongs to
// 8, 16 or 32 lanes of a warp, a longer one to a CTA; a thread holds V groups of
// 8 neighbouring values.  Sums are fp32, in an order that depends on the shape
// alone, so results are the same run to run.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "cache_rows.cuh"
#include "gqa_prefill.h"
#include "launch.h"

namespace gqa {

namespace {

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
  float* part;  // [gridDim.x][n]
  float* dweight;
  long long x_stride, h_stride, out_stride;
  long long rows;  // rows x heads
  int heads, n, team;  // team: lanes of a row (0: the CTA)
  int group;       // values that share a scale (0: 16-bit output)
  int w32;
  int parts;
  float offset, eps, inv_n;
};

struct Vec8 {
  float v[8];
};

template <bool BF16>
__device__ __forceinline__ Vec8 widen(const uint4& u) {
  Vec8 r;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = unpack_lo<BF16>(w[i]);
    r.v[2 * i + 1] = unpack_hi<BF16>(w[i]);
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow(const Vec8& a) {
  return make_uint4(pack2<BF16>(a.v[0], a.v[1]), pack2<BF16>(a.v[2], a.v[3]),
                    pack2<BF16>(a.v[4], a.v[5]), pack2<BF16>(a.v[6], a.v[7]));
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
      v.v[4 * i] = __uint_as_float(r.a[i].x);
      v.v[4 * i + 1] = __uint_as_float(r.a[i].y);
      v.v[4 * i + 2] = __uint_as_float(r.a[i].z);
      v.v[4 * i + 3] = __uint_as_float(r.a[i].w);
    }
    return v;
  }
}
template <bool F32, bool BF16>
__device__ __forceinline__ void store8(void* base, size_t at, const Vec8& v) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(v.v[0], v.v[1], v.v[2], v.v[3]);
    p[1] = make_float4(v.v[4], v.v[5], v.v[6], v.v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = narrow<BF16>(v);
  }
}

// w + offset of 8 columns.
template <bool BF16>
__device__ __forceinline__ Vec8 weight8(const NormParams& p, int col) {
  Vec8 w = p.w32 ? values<true, BF16>(load_raw<true>(p.weight, (size_t)col))
                 : values<false, BF16>(load_raw<false>(p.weight, (size_t)col));
#pragma unroll
  for (int i = 0; i < 8; ++i) w.v[i] += p.offset;
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

template <bool BF16, bool F32, bool OUT8, int V, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : 256) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s[64];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int TS = WIDE ? (int)blockDim.x : p.team;
  const int lane = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (TS - 1);
  const long long row = WIDE ? (long long)blockIdx.x
                             : ((long long)blockIdx.x * 256 + threadIdx.x) / TS;
  const bool live = row < p.rows;
  const long long token = live ? row / p.heads : 0;
  const int head = live ? (int)(row - token * p.heads) : 0;
  const int nv = p.n / 8;
  const size_t xat = (size_t)token * p.x_stride + (size_t)head * p.n;
  const size_t hat = (size_t)row * p.n;
  uint4 xr[V];
  Raw<F32> rr[V];
  const bool has = p.residual != nullptr;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
    if (live && c < nv) {
      xr[v] = load_raw<false>(p.x, xat + 8 * c).a[0];
      if (has) rr[v] = load_raw<F32>(p.residual, hat + 8 * c);
    }
  }
  Vec8 h[V];
  float sum = 0.f, most = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
    if (live && c < nv) {
      h[v] = widen<BF16>(xr[v]);
      if (has) {
        const Vec8 r = values<F32, BF16>(rr[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v].v[i] += r.v[i];
        // The norm is of what the stream holds.
        if constexpr (!F32) h[v] = widen<BF16>(narrow<BF16>(h[v]));
        store8<F32, BF16>(p.h_out, hat + 8 * c, h[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(h[v].v[i], h[v].v[i], sum);
      if constexpr (OUT8) {
        const Vec8 w = weight8<BF16>(p, 8 * c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[v].v[i] *= w.v[i];
          most = fmaxf(most, fabsf(h[v].v[i]));
        }
      }
    }
  }
  const bool whole = OUT8 && p.group == p.n;  // one scale a row
  row_reduce<WIDE, OUT8>(sum, most, TS, s);
  const float rstd = 1.f / sqrtf(fmaf(sum, p.inv_n, p.eps));
  if (live && lane == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  const size_t oat = (size_t)token * p.out_stride + (size_t)head * p.n;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
    const bool in = live && c < nv;
    if constexpr (!OUT8) {
      if (in) {
        const Vec8 w = weight8<BF16>(p, 8 * c);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v].v[i] = h[v].v[i] * rstd * w.v[i];
        store8<false, BF16>(p.out, oat + 8 * c, h[v]);
      }
    } else {
      float top = most;
      if (!whole) {
        top = 0.f;
        if (in) {
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(h[v].v[i]));
        }
        for (int o = 1; o < p.group / 8; o <<= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const int e = e4m3_scale_exponent(top * rstd);
      if (in) {
        const float m = pow2f(-e);
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* a = h[v].v + 4 * i;
          w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a[0] * rstd * m, a[1] * rstd * m),
                                                    __NV_SATFINITE, __NV_E4M3) |
                 (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a[2] * rstd * m, a[3] * rstd * m),
                                                    __NV_SATFINITE, __NV_E4M3) << 16;
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + oat + 8 * c) = make_uint2(w[0], w[1]);
        const int per = whole ? p.n : p.group;
        if (8 * c % per == 0) p.scales[(size_t)row * (p.n / per) + 8 * c / per] = (uint8_t)(e + 127);
      }
    }
  }
}

// Each CTA walks rows blockIdx.x, + gridDim.x, ..., the next row's values on
// their way while this one's are summed, and keeps its share of dw in registers.
template <bool BF16, bool F32, int V, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : 256) norm_backward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s[2][64];
  __shared__ float s_acc[WIDE ? 1 : 256 * 8];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int TS = WIDE ? (int)blockDim.x : p.team;
  const int lane = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (TS - 1);
  const int per_cta = WIDE ? 1 : 256 / TS;
  const int nv = p.n / 8;
  const long long step = (long long)gridDim.x * per_cta;
  const bool has = p.dh != nullptr;
  Vec8 w[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * TS + lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v].v[i] = 0.f;
    if (c < nv) w[v] = weight8<BF16>(p, 8 * c);
  }
  uint4 dy[V];
  Raw<F32> h[V], dh[V];
  float r = 0.f;
  auto fetch = [&](long long row) {
    if (row >= p.rows) return;
    const long long token = row / p.heads;
    const int head = (int)(row - token * p.heads);
    const size_t yat = (size_t)token * p.x_stride + (size_t)head * p.n;
    const size_t hat = (size_t)token * p.h_stride + (size_t)head * p.n;
    r = __ldg(p.rstd_in + row);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * TS + lane;
      if (c < nv) {
        dy[v] = load_raw<false>(p.x, yat + 8 * c).a[0];
        h[v] = load_raw<F32>(p.residual, hat + 8 * c);
        if (has) dh[v] = load_raw<F32>(p.dh, (size_t)row * p.n + 8 * c);
      }
    }
  };
  const long long row0 = (long long)blockIdx.x * per_cta;  // the first team's row
  const int mine = WIDE ? 0 : (int)threadIdx.x / TS;
  fetch(row0 + mine);
  int buf = 0;
  for (long long base = row0; base < p.rows; base += step, buf ^= 1) {
    const long long row = base + mine;
    const bool live = row < p.rows;
    const float rstd = r;
    Vec8 t[V], g[V];
    Raw<F32> old[V];
    float sum = 0.f, none = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * TS + lane;
      if (live && c < nv) {
        const Vec8 d = widen<BF16>(dy[v]);
        t[v] = values<F32, BF16>(h[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t[v].v[i] *= rstd;
          acc[v].v[i] = fmaf(d.v[i], t[v].v[i], acc[v].v[i]);
          g[v].v[i] = d.v[i] * w[v].v[i];
          sum = fmaf(g[v].v[i], t[v].v[i], sum);
        }
        if (has) old[v] = dh[v];
      }
    }
    fetch(row + step);
    row_reduce<WIDE, false>(sum, none, TS, s[buf]);
    const float mean = sum * p.inv_n;
    const long long token = live ? row / p.heads : 0;
    const size_t oat = (size_t)token * p.out_stride + (size_t)(live ? row - token * p.heads : 0) * p.n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * TS + lane;
      if (live && c < nv) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[v].v[i] = rstd * (g[v].v[i] - t[v].v[i] * mean);
        if (has) {
          const Vec8 o = values<F32, BF16>(old[v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[v].v[i] += o.v[i];
        }
        if (p.out != nullptr) store8<false, BF16>(p.out, oat + 8 * c, g[v]);
        if (p.dresidual != nullptr) store8<F32, BF16>(p.dresidual, (size_t)row * p.n + 8 * c, g[v]);
      }
    }
  }
  if (p.part == nullptr) return;
  float* part = p.part + (size_t)blockIdx.x * p.n;
  if constexpr (WIDE) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * TS + lane;
      if (c < nv) store8<true, BF16>(part, (size_t)8 * c, acc[v]);
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) s_acc[threadIdx.x * 8 + i] = acc[v].v[i];
      __syncthreads();
      const int at = v * TS * 8 + (int)threadIdx.x;  // the column
      if ((int)threadIdx.x < TS * 8 && at < p.n) {
        float a = 0.f;
        for (int k = 0; k < per_cta; ++k) a += s_acc[k * TS * 8 + threadIdx.x];
        part[at] = a;
      }
    }
  }
}

// dw: the sum of the CTAs' shares.  32 columns a block, 8 shares at a time.
__global__ void __launch_bounds__(256) norm_join_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s[8][32];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < p.n)
    for (int b = y; b < p.parts; b += 8) a += __ldcg(p.part + (size_t)b * p.n + c);
  s[y][lane] = a;
  __syncthreads();
  if (y == 0 && c < p.n) {
#pragma unroll
    for (int k = 1; k < 8; ++k) a += s[k][lane];
    p.dweight[c] = a;
  }
}

// ------------------------------------------------------------------ host
constexpr int kMaxN = 32768;

struct NormShape {
  int team, v, threads;  // team 0: a row per CTA
};
NormShape norm_shape(int n) {
  const int nv = n / 8;
  NormShape s{0, 1, 256};
  if (nv <= 128) {
    s.team = 8;
    while (s.team < 32 && s.team < nv) s.team *= 2;
    const int v = (nv + s.team - 1) / s.team;
    s.v = v <= 1 ? 1 : v <= 2 ? 2 : 4;
    return s;
  }
  s.v = nv <= 256 ? 1 : nv <= 1024 ? 2 : 4;
  s.threads = ((nv + s.v - 1) / s.v + 31) / 32 * 32;
  return s;
}
// CTAs of the gradient's persistent grid.
int backward_ctas(int sms, const NormShape& s) {
  return s.team > 0 ? 4 * sms : sms * (s.threads <= 256 ? 2 : 1);
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

template <bool BF16, bool F32, bool OUT8, bool WIDE>
cudaError_t launch_norm_v(const NormParams& p, const NormShape& s, int grid, cudaStream_t st) {
  return s.v == 1   ? launch_pdl(norm_kernel<BF16, F32, OUT8, 1, WIDE>, p, grid, s.threads, 0, st)
         : s.v == 2 ? launch_pdl(norm_kernel<BF16, F32, OUT8, 2, WIDE>, p, grid, s.threads, 0, st)
                    : launch_pdl(norm_kernel<BF16, F32, OUT8, 4, WIDE>, p, grid, s.threads, 0, st);
}
template <bool BF16, bool F32>
cudaError_t launch_norm(const NormParams& p, const NormShape& s, int grid, cudaStream_t st) {
  if (p.group > 0)
    return s.team > 0 ? launch_norm_v<BF16, F32, true, false>(p, s, grid, st)
                      : launch_norm_v<BF16, F32, true, true>(p, s, grid, st);
  return s.team > 0 ? launch_norm_v<BF16, F32, false, false>(p, s, grid, st)
                    : launch_norm_v<BF16, F32, false, true>(p, s, grid, st);
}
template <bool BF16, bool F32, bool WIDE>
cudaError_t launch_back_v(const NormParams& p, const NormShape& s, int grid, cudaStream_t st) {
  return s.v == 1   ? launch_pdl(norm_backward_kernel<BF16, F32, 1, WIDE>, p, grid, s.threads, 0, st)
         : s.v == 2 ? launch_pdl(norm_backward_kernel<BF16, F32, 2, WIDE>, p, grid, s.threads, 0, st)
                    : launch_pdl(norm_backward_kernel<BF16, F32, 4, WIDE>, p, grid, s.threads, 0, st);
}
template <bool BF16, bool F32>
cudaError_t launch_back(const NormParams& p, const NormShape& s, int grid, cudaStream_t st) {
  return s.team > 0 ? launch_back_v<BF16, F32, false>(p, s, grid, st)
                    : launch_back_v<BF16, F32, true>(p, s, grid, st);
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
  p.rows = (long long)rows * heads;
  p.heads = heads;
  p.n = n;
  p.group = e4 ? group : 0;
  p.w32 = weight_type == GQA_F32;
  p.offset = offset;
  p.eps = eps;
  p.inv_n = 1.f / (float)n;
  const NormShape s = norm_shape(n);
  p.team = s.team;
  const long long per = s.team > 0 ? 256 / s.team : 1;
  const int grid = (int)((p.rows + per - 1) / per);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == GQA_BF16, f32 = stream_type == GQA_F32;
  const cudaError_t e = bf ? (f32 ? launch_norm<true, true>(p, s, grid, st) : launch_norm<true, false>(p, s, grid, st))
                           : (f32 ? launch_norm<false, true>(p, s, grid, st) : launch_norm<false, false>(p, s, grid, st));
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

int sm_count() {
  int sms = 152;
  unsigned int* status = nullptr;
  if (call_device(&sms, &status) != GQA_OK) sms = 152;
  return sms;
}

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
  const NormShape s = norm_shape(n);
  const int sms = sm_count();
  const size_t need = 4u * (size_t)backward_ctas(sms, s) * n;
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
  p.dweight = dweight;
  p.x_stride = dy_stride;
  p.h_stride = h_stride;
  p.out_stride = dx_stride;
  p.rows = (long long)rows * heads;
  p.heads = heads;
  p.n = n;
  p.team = s.team;
  p.w32 = weight_type == GQA_F32;
  p.offset = offset;
  p.inv_n = 1.f / (float)n;
  const long long per = s.team > 0 ? 256 / s.team : 1, all = (p.rows + per - 1) / per;
  const int most = backward_ctas(sms, s);
  const int grid = (int)(all < most ? all : most);
  p.parts = grid;
  const bool bf = dtype == GQA_BF16, f32 = stream_type == GQA_F32;
  cudaError_t e = bf ? (f32 ? launch_back<true, true>(p, s, grid, st) : launch_back<true, false>(p, s, grid, st))
                     : (f32 ? launch_back<false, true>(p, s, grid, st) : launch_back<false, false>(p, s, grid, st));
  if (e == cudaSuccess && dweight != nullptr) e = launch_pdl(norm_join_kernel, p, (n + 31) / 32, 256, 0, st);
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
  if (rc == GQA_OK) *bytes = 4u * (size_t)gqa::backward_ctas(gqa::sm_count(), gqa::norm_shape(n)) * n;
  return rc;
}

}  // extern "C"
