// backward.cu -- gqa_prefill_backward: argument checks, the workspace, and the
// kernels around the products (backward_kernel.cuh): the plan, the rows'
// statistics, and the join of cut units.  Declared in include/gqa_prefill.h.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "backward.h"
#include "gqa_prefill.h"
#include "launch.h"

namespace gqa {

namespace {

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanBins = 64;
// Shares of the work that a CTA gets at the least: a unit is cut when it costs
// more than 1 / kShares of a CTA's part of the whole.  Tiles below which a
// unit is not cut.
constexpr int kShares = 1;
constexpr int kMinTiles = 8;
constexpr int kMinCost = 4 * kMinTiles;  // of a tile at the most expensive
// Pairs up to which a sequence's P and dS are held in two terms: 724 tokens of one query head, 256 of
// eight.  Error against 64 bits over that of results that are rounded alone, 1300 sequences of 1 to 700
// tokens, the worst of dq, dk and dv: with two terms 1.00 (1.06 where a result cancels), with one 1.43, up
// to 1.5 where pairs are few and twice over a handful; above the limit 1.49 at most, with scores of 8
// times the spread (a p or two a row) too.  Price: 2000 sequences of 30 tokens, 64 / 8 heads of 64, 964 -> 1048
// us; 100 of 300 tokens, above the limit, would take 669 instead of 576.
constexpr long long kTwoPairs = 1 << 19;

// Relative cost of a streamed tile: its products.
__host__ __device__ __forceinline__ int tile_cost(int kind) {
  return kind == kBwdKV ? 4 : kind == kBwdV ? 2 : 3;
}

// Sequence of tile x: the last b with first[b] <= x.
__device__ __forceinline__ int find_seq(const int32_t* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Whether a sequence's P and dS are held in two 16-bit terms: where it has few pairs (of a
// KV head's query rows and the keys that one sees), whatever stands beside it in the call.
__device__ __forceinline__ bool two_terms(const BwdParams& p, int P, int E) {
  return (long long)E * p.G * min(P + E, p.reach) <= kTwoPairs;
}

// Unit x of the list before cutting: first the query tiles, then the key tiles
// (twice at d = 256: dk, then dv).
__device__ __forceinline__ BwdUnit plan_unit(const BwdParams& p, int x, int nq, int nk) {
  BwdUnit u;
  const bool qa = x < nq;
  int t = qa ? x : x - nq;
  u.kind = qa ? kBwdQ : p.d == 256 ? (t < nk ? kBwdK : kBwdV) : kBwdKV;
  if (!qa && t >= nk) t -= nk;
  const int32_t* first = qa ? p.qtile0 : p.ktile0;
  const int b = find_seq(first, p.num_seqs, t);
  const int c0 = p.cu[b], E = p.cu[b + 1] - c0, P = p.pre[b], k0 = p.kvi[b];
  const int N = p.N;
  u.seq = b;
  u.P = P;
  u.E = E;
  u.a_off = (t - first[b]) * 128;
  u.slot = -1;
  u.stat = p.qtile0[b] * 128;
  int lo, hi;  // B's rows [lo, hi) that the unit streams
  if (qa) {
    u.a_base = c0;
    u.a_valid = min(128, E * p.G - u.a_off);
    u.b_base = k0;
    u.b_len = P + E;
  } else {
    u.a_base = k0;
    u.a_valid = min(128, P + E - u.a_off);
    u.b_base = c0;
    u.b_len = E * p.G;
  }
  bwd_bounds(qa, u.a_off, P, E, p.log_G, p.reach, lo, u.hi_min);
  bwd_bounds(qa, u.a_off + u.a_valid - 1, P, E, p.log_G, p.reach, u.lo_max, hi);
  ++hi;
  if (lo < 0) lo = 0;
  u.b_off = lo / N * N;
  u.n = hi > lo ? (hi - u.b_off + N - 1) / N : 0;
  return u;
}

// Metadata checks, and the tiles of the sequences before each one.
__global__ void __launch_bounds__(kPlanThreads) bwd_scan_kernel(const __grid_constant__ BwdParams p) {
  __shared__ int s_bad, s_carry[2], s_warp[2][32];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_bad = __ldg(p.cu) != 0;
    s_carry[0] = s_carry[1] = 0;
  }
  __syncthreads();
  // Tiles of each sequence, and their sums over the sequences before it.
  for (int b0 = 0; b0 < p.num_seqs; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n[2] = {0, 0};
    if (b < p.num_seqs) {
      const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), P = __ldg(p.pre + b);
      const int k0 = __ldg(p.kvi + b), k1 = __ldg(p.kvi + b + 1);
      if (c0 < 0 || c1 < c0 || c1 > p.total_q || P < 0 || k0 < 0 || k1 < k0 || k1 > p.total_kv ||
          (long long)k1 - k0 != (long long)P + c1 - c0) {
        s_bad = 1;
      } else {
        n[0] = ((c1 - c0) * p.G + 127) / 128;
        n[1] = (k1 - k0 + 127) / 128;
      }
    }
    int incl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int v = n[k];
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
      }
      incl[k] = v;
      if (lane == 31) s_warp[k][warp] = v;
    }
    __syncthreads();
    if (tid < 2) {
      int acc = s_carry[tid];
      for (int w = 0; w < 32; ++w) {
        const int v = s_warp[tid][w];
        s_warp[tid][w] = acc;
        acc += v;
      }
      s_carry[tid] = acc;
    }
    __syncthreads();
    if (b < p.num_seqs) {
      p.qtile0[b] = s_warp[0][warp] + incl[0] - n[0];
      p.ktile0[b] = s_warp[1][warp] + incl[1] - n[1];
    }
    __syncthreads();
  }
  const int nq = s_carry[0], nk = s_carry[1];
  if (s_bad) {  // nothing is written
    if (tid == 0) {
      atomicOr(p.status, 2u);  // GQA_DEV_BAD_METADATA
      p.hdr[kBwdQTiles] = p.hdr[kBwdKTiles] = 0;
      p.hdr[kBwdFailed] = 1;
    }
    return;
  }
  if (tid == 0) {
    p.qtile0[p.num_seqs] = nq;
    p.ktile0[p.num_seqs] = nk;
    p.hdr[kBwdFailed] = 0;
    p.hdr[kBwdQTiles] = nq;
    p.hdr[kBwdKTiles] = nk;
  }
  if (p.most_v != nullptr)
    for (long long i = tid; i < (long long)p.num_seqs * p.Hkv; i += kPlanThreads) p.most_v[i] = 0u;
}

// The list of units, by one CTA: their costs are summed, costly ones are cut, and
// the parts are sorted by cost, in bins (which CTA takes which unit changes no
// result, so the order inside a bin may be any).
__device__ __forceinline__ void bwd_plan(const BwdParams& p) {
  constexpr int kKept = 2048;
  __shared__ unsigned long long s_total;
  __shared__ int s_slots, s_joins, s_bins[kPlanBins], s_n[kKept];
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  const int nq = p.hdr[kBwdQTiles], nk = p.hdr[kBwdKTiles];
  const int total = nq + (p.d == 256 ? 2 : 1) * nk;
  auto kind_of = [&](int x) { return x < nq ? kBwdQ : p.d != 256 ? kBwdKV : x < nq + nk ? kBwdK : kBwdV; };
  auto tiles_of = [&](int x) { return x < kKept ? s_n[x] : plan_unit(p, x, nq, nk).n; };
  if (tid == 0) s_total = 0;
  __syncthreads();
  unsigned long long sum = 0;
  for (int x = tid; x < total; x += threads) {
    const int n = plan_unit(p, x, nq, nk).n;
    if (x < kKept) s_n[x] = n;
    sum += (unsigned long long)n * tile_cost(kind_of(x));
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) atomicAdd(&s_total, sum);
  __syncthreads();
  // The cost above which a unit is cut.  At most 2 sum / cap parts come of it;
  // should they not fit the workspace, the cap is doubled.
  long long cap = ((long long)s_total * p.Hkv + (long long)p.ctas * kShares - 1) / ((long long)p.ctas * kShares);
  if (cap < kMinCost) cap = kMinCost;
  auto parts_of = [&](int kind, int n) {
    const long long k = ((long long)n * tile_cost(kind) + cap - 1) / cap;
    return (int)(k < 1 ? 1 : k < n ? k : n);
  };
  auto bin_of = [&](int kind, int n) {  // 0: the costliest
    const long long k = n == 0 ? 0 : 1 + (long long)n * tile_cost(kind) * (kPlanBins - 2) / cap;
    return kPlanBins - 1 - (int)(k < kPlanBins - 1 ? k : kPlanBins - 1);
  };
  for (;;) {
    for (int i = tid; i < kPlanBins; i += threads) s_bins[i] = 0;
    if (tid == 0) s_slots = s_joins = 0;
    __syncthreads();
    for (int x = tid; x < total; x += threads) {
      const int kind = kind_of(x), n = tiles_of(x), parts = parts_of(kind, n);
      for (int i = 0; i < parts; ++i)
        atomicAdd(&s_bins[bin_of(kind, (int)((i + 1ll) * n / parts - (long long)i * n / parts))], 1);
      if (parts > 1) {
        atomicAdd(&s_slots, parts);
        atomicAdd(&s_joins, 1);
      }
    }
    __syncthreads();
    const bool fits = s_slots <= p.max_slots && s_joins <= p.max_joins;
    __syncthreads();  // all have read the counts, which are set anew below or in the next pass
    if (fits) break;
    cap *= 2;
  }
  if (tid < 32) {  // the bins' first places: two bins a lane
    static_assert(kPlanBins == 64, "two bins a lane");
    const int n0 = s_bins[2 * lane], n1 = s_bins[2 * lane + 1];
    int v = n0 + n1;
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    s_bins[2 * lane] = v - n0 - n1;
    s_bins[2 * lane + 1] = v - n1;
    if (lane == 31) {
      p.hdr[kBwdUnits] = v;
      p.hdr[kBwdJoins] = s_joins;
      p.hdr[kBwdNext] = 0;
      s_slots = s_joins = 0;
    }
  }
  __syncthreads();
  for (int x = tid; x < total; x += threads) {
    BwdUnit u = plan_unit(p, x, nq, nk);
    const int kind = u.kind, n = u.n, off = u.b_off, parts = parts_of(kind, n);
    int slot = -1;
    if (parts > 1) {
      slot = atomicAdd(&s_slots, parts);
      const BwdJoin j = {kind, u.a_base, u.a_off, u.a_valid, slot, parts, u.seq, 0};
      p.joins[atomicAdd(&s_joins, 1)] = j;
    }
    for (int i = 0; i < parts; ++i) {
      const int t0 = (int)((long long)i * n / parts), t1 = (int)((i + 1ll) * n / parts);
      u.n = t1 - t0;
      u.b_off = off + t0 * p.N;
      u.slot = parts > 1 ? slot + i : -1;
      u.kind = kind + (two_terms(p, u.P, u.E) ? kBwdTwo : 0);
      p.units[atomicAdd(&s_bins[bin_of(kind, u.n)], 1)] = u;
    }
  }
}

// ------------------------------------------------------------------ the rows' statistics
// Bound by memory: out and dout are read once, 8 values a lane, a row in d / 8
// neighbouring lanes.  The first CTA lists the units meanwhile.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const __grid_constant__ BwdParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, ROUNDS = 16 / RPW;  // 16 rows a warp
  __shared__ float s_nl[128], s_nd[128], s_w[128], s_o2[128];
  __shared__ unsigned int s_most[2];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = gridDim.x - 1;
  if (blockIdx.x == 0) {
    bwd_plan(p);
    return;
  }
  const int nq = p.hdr[kBwdQTiles] * p.Hkv, nk = BF16 ? 0 : p.hdr[kBwdKTiles] * p.Hkv;
  for (int x = blockIdx.x - 1; x < nq + nk; x += ctas) {
    const bool keys = x >= nq;
    const int y = keys ? x - nq : x, tile = y / p.Hkv, g = y - tile * p.Hkv;
    const int32_t* first = keys ? p.ktile0 : p.qtile0;
    const int b = find_seq(first, p.num_seqs, tile);
    const int r0 = (tile - first[b]) * 128;
    const int base = keys ? p.kvi[b] : p.cu[b];
    const int valid = keys ? min(128, p.kvi[b + 1] - base - r0) : min(128, (p.cu[b + 1] - base) * p.G - r0);
    if (!BF16 && tid < 2) s_most[tid] = 0u;
    if (!BF16) __syncthreads();
    float m2 = 0.f, md = 0.f;
    // Four rounds' loads at once, so that four CTAs fit an SM at any d (all rounds at
    // once took 116 registers at d = 128: 3598 f16 tokens, the whole gradient 162 us, now 159).
#pragma unroll 1
    for (int at = 0; at < ROUNDS; at += 4) {
      uint4 o[4], dn[4];
      float ls[4], dl[4], sk[4];  // the row's lse, dlse and sink: one address for its lanes
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = warp * 16 + (at + i) * RPW + lane / LPR;
        o[i] = dn[i] = make_uint4(0u, 0u, 0u, 0u);
        ls[i] = -INFINITY;
        dl[i] = sk[i] = 0.f;
        if (r < valid) {
          if (keys) {
            dn[i] = __ldg(reinterpret_cast<const uint4*>(p.v) +
                          ((size_t)(base + r0 + r) * p.Hkv + g) * LPR + lane % LPR);
          } else {
            const size_t row = (size_t)(base + ((r0 + r) >> p.log_G)) * p.Hq + g * p.G + ((r0 + r) & (p.G - 1));
            o[i] = __ldg(reinterpret_cast<const uint4*>(p.out) + row * LPR + lane % LPR);
            dn[i] = __ldg(reinterpret_cast<const uint4*>(p.dout) + row * LPR + lane % LPR);
            ls[i] = __ldg(p.lse + row);
            if (p.dlse != nullptr) dl[i] = __ldg(p.dlse + row);
            if (p.sinks != nullptr) sk[i] = __ldg(p.sinks + g * p.G + ((r0 + r) & (p.G - 1)));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = warp * 16 + (at + i) * RPW + lane / LPR;
        const uint32_t a[4] = {o[i].x, o[i].y, o[i].z, o[i].w},
                       e[4] = {dn[i].x, dn[i].y, dn[i].z, dn[i].w};
        float dot = 0.f, sq = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float el = unpack_lo<BF16>(e[k]), eh = unpack_hi<BF16>(e[k]);
          dot = fmaf(unpack_lo<BF16>(a[k]), el, dot);
          dot = fmaf(unpack_hi<BF16>(a[k]), eh, dot);
          if (!BF16) sq = fmaf(el, el, fmaf(eh, eh, sq));
        }
#pragma unroll
        for (int s = 1; s < LPR; s <<= 1) {
          dot += __shfl_xor_sync(0xffffffffu, dot, s);
          if (!BF16) sq += __shfl_xor_sync(0xffffffffu, sq, s);
        }
        if (!BF16) m2 = fmaxf(m2, sq);
        if (!keys && lane % LPR == 0) {
          float nl = -INFINITY, nd = 0.f, w = 0.f;
          if (r < valid) {
            const float lse = ls[i], dlt = dot - dl[i];
            nd = -dlt;
            if (lse != -INFINITY) {  // else: no key, no probability
              nl = -lse * kLog2e + (BF16 ? 0.f : kBwdBias);
              if (p.sinks != nullptr) w = expf(sk[i] - lse) * dlt;
            }
            if (!BF16) md = fmaxf(md, fabsf(dlt));
          }
          if (!BF16) s_o2[r] = sq;
          s_nl[r] = nl;
          s_nd[r] = nd;
          s_w[r] = w;
        }
      }
    }
    if (!BF16) {
      // NaN would lose every comparison: the bound then stays finite, and the
      // results are NaN by themselves.
      atomicMax(&s_most[0], __reduce_max_sync(0xffffffffu, __float_as_uint(m2)));
      atomicMax(&s_most[1], __reduce_max_sync(0xffffffffu, __float_as_uint(md)));
    }
    __syncthreads();
    if (!BF16 && tid == 0) {
      if (keys)
        atomicMax(p.most_v + (size_t)b * p.Hkv + g, s_most[0]);
      else
        p.tile_most[(size_t)g * p.max_qtiles + tile] = make_uint2(s_most[0], s_most[1]);
    }
    if (!keys) {
      const size_t at = (size_t)g * p.stat_rows + (size_t)tile * 128;
      if (!BF16 && tid < 128) p.row_o2[at + tid] = s_o2[tid];
      if (tid < 128) p.nlse[at + tid] = s_nl[tid];
      else p.nd[at + tid - 128] = s_nd[tid - 128];
      if (p.sinks != nullptr) {
        // Rows of one head are G apart: sums of pairs, in a warp and then over four.
        if (tid < 128) {
          float w = s_w[tid];
          for (int s = 16; s >= p.G; s >>= 1) w += __shfl_xor_sync(0xffffffffu, w, s);
          s_w[tid] = w;
        }
        __syncthreads();
        if (tid < p.G) {
          float w = s_w[tid];
          if (p.G <= 32) w = (w + s_w[tid + 32]) + (s_w[tid + 64] + s_w[tid + 96]);
          if (p.G == 64) w += s_w[tid + 64];
          p.sink_part[(size_t)(g * p.G + tid) * p.max_qtiles + tile] = w;
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ join
// Sums of the parts of cut units, in their order: a thread per row and 16 of its
// columns, all loads of two parts on their way at once; and the sinks' gradient,
// one block a head.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) bwd_join_kernel(const __grid_constant__ BwdParams p) {
  constexpr int A = bwd_accs(D), kPieces = D / 32;  // blocks for 128 rows of one accumulator
  grid_dep_launch_dependents();
  grid_dep_wait();
  if (p.hdr[kBwdFailed] != 0) return;
  const int tid = threadIdx.x;
  const int nj = p.hdr[kBwdJoins] * p.Hkv * A * kPieces, tiles = p.hdr[kBwdQTiles];
  const int ns = p.dsinks != nullptr ? p.Hq : 0;
  for (int x = blockIdx.x; x < nj + ns; x += gridDim.x) {
    if (x >= nj) {
      const int h = x - nj;
      __shared__ double s_sum[8];
      double acc = 0.0;
      for (int t = tid; t < tiles; t += 256) acc += (double)__ldcg(p.sink_part + (size_t)h * p.max_qtiles + t);
      for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
      if ((tid & 31) == 0) s_sum[tid >> 5] = acc;
      __syncthreads();
      if (tid == 0) {
        double a = 0.0;
        for (int w = 0; w < 8; ++w) a += s_sum[w];
        p.dsinks[h] = (float)(0.0 - a);
      }
      __syncthreads();
      continue;
    }
    const int a = x / kPieces % A, y = x / (kPieces * A), g = y % p.Hkv;
    const BwdJoin j = p.joins[y / p.Hkv];
    const int r = tid & 127, c = (x % kPieces) * 2 + (tid >> 7);  // columns [16 c, 16 c + 16)
    if ((a > 0 && j.kind != kBwdKV) || r >= j.a_valid) continue;
    const size_t stride = (size_t)p.Hkv * A * (D / 4) * 128;  // float4 between slots
    const float4* src = reinterpret_cast<const float4*>(p.part) +
                        (((size_t)j.slot * p.Hkv + g) * A + a) * (D / 4) * 128 + (size_t)(4 * c) * 128 + r;
    float4 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k < j.parts; ++k) {
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __ldcg(src + k * stride + (size_t)i * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i].x += v[i].x;
        s[i].y += v[i].y;
        s[i].z += v[i].z;
        s[i].w += v[i].w;
      }
    }
    void* dst = j.kind == kBwdQ ? p.dq : (j.kind == kBwdV || (j.kind == kBwdKV && a == 0)) ? p.dv : p.dk;
    const int ar = j.a_off + r;
    const size_t row = j.kind == kBwdQ
                           ? (size_t)(j.a_base + (ar >> p.log_G)) * p.Hq + g * p.G + (ar & (p.G - 1))
                           : (size_t)(j.a_base + ar) * p.Hkv + g;
    uint4* to = reinterpret_cast<uint4*>(dst) + row * (D / 8) + 2 * c;
    to[0] = make_uint4(pack2<BF16>(s[0].x, s[0].y), pack2<BF16>(s[0].z, s[0].w), pack2<BF16>(s[1].x, s[1].y),
                       pack2<BF16>(s[1].z, s[1].w));
    to[1] = make_uint4(pack2<BF16>(s[2].x, s[2].y), pack2<BF16>(s[2].z, s[2].w), pack2<BF16>(s[3].x, s[3].y),
                       pack2<BF16>(s[3].z, s[3].w));
  }
}

// ------------------------------------------------------------------ host
struct BwdPlan {
  int ctas, max_qtiles, max_ktiles, max_units, max_slots, max_joins;
  long long stat_rows;
  size_t units, joins, qt, kt, nlse, nd, sink, o2, most, most_v, part, bytes;
};

int bwd_layout(int num_seqs, int total_q, int total_kv, int Hq, int Hkv, int d, int dtype, BwdPlan* pl) {
  if (num_seqs < 0 || total_q < 0 || total_kv < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0)
    return GQA_ERR_INVALID;
  if (dtype != GQA_F16 && dtype != GQA_BF16) return GQA_ERR_INVALID;
  const int G = Hq / Hkv;
  if ((d != 64 && d != 128 && d != 256) || G > 128 || (G & (G - 1)) != 0) return GQA_ERR_UNSUPPORTED;
  // Packed rows, tiles and units are counted in 32 bits.
  const long long rows = (long long)total_q * G;
  const long long qt = rows / 128 + num_seqs, kt = (long long)total_kv / 128 + num_seqs;
  if (rows >= (1ll << 30) || total_kv >= (1 << 30) || num_seqs >= (1 << 24) ||
      (qt + 2 * kt + 4096) * Hkv >= (1ll << 31) || (qt * 128) >= (1ll << 31))
    return GQA_ERR_UNSUPPORTED;
  int sms = 152;
  unsigned int* status = nullptr;
  if (call_device(&sms, &status) != GQA_OK) sms = 152;
  sms *= bwd_per_sm(d);
  pl->ctas = sms;
  pl->max_qtiles = (int)qt;
  pl->max_ktiles = (int)kt;
  pl->stat_rows = qt * 128;
  // Parts of cut units: what the CTAs' shares can make of them, and no more than the
  // shapes can (a call of a few tokens cuts nothing, and needs no room for parts).
  const int N = bwd_n(d);
  auto parts = [&](int kind, long long rows_b) { return ((rows_b + N - 1) / N * tile_cost(kind) + kMinCost - 1) / kMinCost; };
  const long long pq = parts(kBwdQ, total_kv), pk = parts(d == 256 ? kBwdK : kBwdKV, rows);
  const long long by_shape = (pq > 1 ? qt * pq : 0) + (pk > 1 ? (d == 256 ? 2 : 1) * kt * pk : 0);
  const long long by_share = 2 * sms * kShares / Hkv + 1;
  pl->max_slots = (int)(by_shape < by_share ? by_shape : by_share);
  pl->max_joins = pl->max_slots / 2 + 1;
  pl->max_units = (int)(qt + (d == 256 ? 2 : 1) * kt) + pl->max_slots;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~static_cast<size_t>(255);
    return here;
  };
  take(4u * kBwdHdr);
  pl->units = take(sizeof(BwdUnit) * (size_t)pl->max_units);
  pl->joins = take(sizeof(BwdJoin) * (size_t)pl->max_joins);
  pl->qt = take(4u * (size_t)(num_seqs + 1));
  pl->kt = take(4u * (size_t)(num_seqs + 1));
  pl->nlse = take(4u * (size_t)Hkv * pl->stat_rows);
  pl->nd = take(4u * (size_t)Hkv * pl->stat_rows);
  pl->sink = take(4u * (size_t)Hq * pl->max_qtiles);
  const size_t f16 = dtype == GQA_F16 ? 1u : 0u;
  pl->o2 = take(f16 * 4u * (size_t)Hkv * pl->stat_rows);
  pl->most = take(f16 * 8u * (size_t)Hkv * pl->max_qtiles);
  pl->most_v = take(f16 * 4u * (size_t)num_seqs * Hkv);
  pl->part = take(4u * 128u * (size_t)d * bwd_accs(d) * Hkv * pl->max_slots);
  pl->bytes = at;
  return GQA_OK;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

template <int D, bool BF16>
cudaError_t launch_around(const BwdParams& p, cudaStream_t st) {
  cudaError_t e = launch_pdl(bwd_scan_kernel, p, 1, kPlanThreads, 0, st);
  if (e != cudaSuccess) return e;
  const long long items = ((long long)p.max_qtiles + (BF16 ? 0 : p.total_kv / 128 + p.num_seqs)) * p.Hkv;
  const long long room = 8ll * p.ctas;
  e = launch_pdl(bwd_prep_kernel<D, BF16>, p, 1 + (int)(items < room ? items : room), 256, 0, st);
  if (e != cudaSuccess) return e;
  e = D == 64 ? launch_bwd_d64(p, BF16, st) : D == 128 ? launch_bwd_d128(p, BF16, st) : launch_bwd_d256(p, BF16, st);
  if (e != cudaSuccess) return e;
  return launch_pdl(bwd_join_kernel<D, BF16>, p, 4 * p.ctas, 256, 0, st);
}

int run_backward(const void* q, const void* k, const void* v, const int32_t* cu, const int32_t* pre,
                 const int32_t* kvi, int num_seqs, int total_q, int total_kv, int Hq, int Hkv, int d,
                 int dtype, float scale, int window, const void* out, const float* lse,
                 const void* dout, const float* dlse, const float* sinks, void* dq, void* dk,
                 void* dv, float* dsinks, void* workspace, size_t workspace_bytes, void* stream) {
  BwdPlan pl;
  const int rc = bwd_layout(num_seqs, total_q, total_kv, Hq, Hkv, d, dtype, &pl);
  if (rc == GQA_ERR_INVALID) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale)) return GQA_ERR_INVALID;
  if ((sinks == nullptr) != (dsinks == nullptr) || !al4(sinks) || !al4(dsinks)) return GQA_ERR_INVALID;
  if (rc != GQA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (num_seqs == 0) {  // no rows; no token for the sinks either
    if (dsinks != nullptr && cudaMemsetAsync(dsinks, 0, 4u * (size_t)Hq, st) != cudaSuccess)
      return GQA_ERR_CUDA;
    return GQA_OK;
  }
  if (cu == nullptr || pre == nullptr || kvi == nullptr || !al4(cu) || !al4(pre) || !al4(kvi))
    return GQA_ERR_INVALID;
  if (total_q > 0 && (q == nullptr || out == nullptr || dout == nullptr || lse == nullptr || dq == nullptr))
    return GQA_ERR_INVALID;
  if (total_kv > 0 && (k == nullptr || v == nullptr || dk == nullptr || dv == nullptr))
    return GQA_ERR_INVALID;
  if (total_q > 0 && total_kv == 0) return GQA_ERR_INVALID;
  for (const void* x : {q, k, v, out, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv)})
    if (!al16(x)) return GQA_ERR_INVALID;
  if (!al4(lse) || !al4(dlse)) return GQA_ERR_INVALID;
  if (workspace == nullptr || workspace_bytes < pl.bytes ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return GQA_ERR_INVALID;
  // Results are written while other units still read the inputs.
  const size_t nq = 2u * (size_t)total_q * Hq * d, nk = 2u * (size_t)total_kv * Hkv * d,
               nl = 4u * (size_t)total_q * Hq;
  const Range in[] = {{q, nq}, {k, nk}, {v, nk}, {out, nq}, {dout, nq}, {lse, nl}, {dlse, nl},
                      {sinks, 4u * (size_t)Hq}, {cu, 4u * ((size_t)num_seqs + 1)},
                      {pre, 4u * (size_t)num_seqs}, {kvi, 4u * ((size_t)num_seqs + 1)}};
  const Range outs[] = {{dq, nq}, {dk, nk}, {dv, nk}, {dsinks, 4u * (size_t)Hq}, {workspace, pl.bytes}};
  for (int i = 0; i < 5; ++i) {
    for (const Range& r : in)
      if (overlap(outs[i], r)) return GQA_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return GQA_ERR_INVALID;
  }

  BwdParams p;
  std::memset(&p, 0, sizeof(p));
  int sms = 0;
  if (call_device(&sms, &p.status) != GQA_OK) return GQA_ERR_CUDA;
  const int G = Hq / Hkv, N = bwd_n(d);
  const int bh = G < N ? G : N, bt = N / bh;  // heads and tokens of a streamed query tile
  int rm = GQA_OK;
  auto map = [&](CUtensorMap* m, const void* base, int heads, int rows, int box_heads, int box_rows) {
    if (rm == GQA_OK && rows > 0) rm = rows_map(m, base, dtype, d, heads, rows, box_heads, box_rows);
  };
  map(&p.a_q, q, Hq, total_q, G, 128 / G);
  map(&p.a_do, dout, Hq, total_q, G, 128 / G);
  map(&p.a_k, k, Hkv, total_kv, 1, 128);
  map(&p.a_v, v, Hkv, total_kv, 1, 128);
  map(&p.b_q, q, Hq, total_q, bh, bt);
  map(&p.b_do, dout, Hq, total_q, bh, bt);
  map(&p.b_k, k, Hkv, total_kv, 1, N);
  map(&p.b_v, v, Hkv, total_kv, 1, N);
  if (rm != GQA_OK) return rm;
  char* ws = static_cast<char*>(workspace);
  p.cu = cu;
  p.pre = pre;
  p.kvi = kvi;
  p.v = v;
  p.out = out;
  p.dout = dout;
  p.lse = lse;
  p.dlse = dlse;
  p.sinks = sinks;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.dsinks = dsinks;
  p.hdr = reinterpret_cast<int32_t*>(ws);
  p.units = reinterpret_cast<BwdUnit*>(ws + pl.units);
  p.joins = reinterpret_cast<BwdJoin*>(ws + pl.joins);
  p.qtile0 = reinterpret_cast<int32_t*>(ws + pl.qt);
  p.ktile0 = reinterpret_cast<int32_t*>(ws + pl.kt);
  p.nlse = reinterpret_cast<float*>(ws + pl.nlse);
  p.nd = reinterpret_cast<float*>(ws + pl.nd);
  p.sink_part = reinterpret_cast<float*>(ws + pl.sink);
  if (dtype == GQA_F16) {
    p.row_o2 = reinterpret_cast<float*>(ws + pl.o2);
    p.tile_most = reinterpret_cast<uint2*>(ws + pl.most);
    p.most_v = reinterpret_cast<unsigned int*>(ws + pl.most_v);
  }
  p.part = reinterpret_cast<float*>(ws + pl.part);
  p.stat_rows = pl.stat_rows;
  p.max_qtiles = pl.max_qtiles;
  p.max_units = pl.max_units;
  p.max_slots = pl.max_slots;
  p.max_joins = pl.max_joins;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.total_kv = total_kv;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  while ((1 << p.log_G) < G) ++p.log_G;
  p.d = d;
  p.N = N;
  p.reach = window > 0 && window < (1 << 30) ? window : 1 << 30;
  p.ctas = pl.ctas;
  p.scale = scale;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.timeout_ns = wait_limit_ns();
  const bool bf = dtype == GQA_BF16;
  const cudaError_t e =
      d == 64    ? (bf ? launch_around<64, true>(p, st) : launch_around<64, false>(p, st))
      : d == 128 ? (bf ? launch_around<128, true>(p, st) : launch_around<128, false>(p, st))
                 : (bf ? launch_around<256, true>(p, st) : launch_around<256, false>(p, st));
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

}  // namespace gqa

extern "C" {

int gqa_prefill_backward(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                         const int32_t* prefix_lens, const int32_t* kv_indptr, int num_seqs,
                         int total_q, int total_kv, int Hq, int Hkv, int d, int dtype, float scale,
                         int window, const void* out, const float* lse, const void* dout,
                         const float* dlse, const float* sinks, void* dq, void* dk, void* dv,
                         float* dsinks, void* workspace, size_t workspace_bytes, void* stream) {
  return gqa::run_backward(q, k, v, cu_seqlens_q, prefix_lens, kv_indptr, num_seqs, total_q, total_kv,
                           Hq, Hkv, d, dtype, scale, window, out, lse, dout, dlse, sinks, dq, dk, dv,
                           dsinks, workspace, workspace_bytes, stream);
}

int gqa_prefill_backward_workspace(int num_seqs, int total_q, int total_kv, int Hq, int Hkv, int d,
                                   int dtype, size_t* bytes) {
  if (bytes == nullptr) return GQA_ERR_INVALID;
  gqa::BwdPlan pl;
  const int rc = gqa::bwd_layout(num_seqs, total_q, total_kv, Hq, Hkv, d, dtype, &pl);
  if (rc == GQA_OK) *bytes = pl.bytes;
  return rc;
}

}  // extern "C"
