// backward_kernel.cuh -- the products of the attention's gradient on tcgen05.
//
// Mathematics: backward.h.  A unit keeps 128 rows of one side in shared memory
// (A1, A2) and streams tiles of N rows of the other (B1, B2):
//                 A1  A2    B1  B2    S = A1 B1^T   T = A2 B2^T
//   dq unit       q   dout  k   v     S [queries, keys]
//   dk, dv unit   k   v     q   dout  S^T [keys, queries]
// Both products land in tensor memory with a row of A in each lane.  The
// softmax warps turn S into P and T into dS = P (T - D), write both back in 16
// bits over their own fp32 columns, and they are the left operand, in tensor
// memory, of the second products  acc1 += dS B1 (dq or dk)  and  acc0 += P B2
// (dv), whose right operand is the streamed tile read with its rows as the
// contraction.  So P and dS never pass through shared memory, and every row of
// the result has one writer: no atomics, the same bits run to run.  (The price
// is that S and T are computed for both kinds of unit: 7 products, not 5.)
//
// P and dS are rounded to the inputs' type because the tensor cores take no other
// left operand beside a 16-bit right one: half a step of each, as the forward
// kernels round P.  Everything else is fp32.  Over many pairs that makes a result's
// error some 1.43 times its own rounding; over a few it may be one p's alone, up to
// twice.  So the units of a sequence with few pairs (two_terms in backward.cu) hold P and
// dS as sums of two 16-bit terms, the second in the columns that the fp32 ones
// leave free.  Both kinds of unit are in one kernel, so that a sequence's bits do not
// depend on its company; the loops with the two terms beside them cost the others up to
// 1% (4096 tokens 462 -> 463 us, 3598 ragged ones 157 -> 158).
//
// CTA: 8 or 16 softmax warps (each warpgroup takes a share of the columns), a
// loading warp, a warp that issues the products.  Persistent: units are taken from a
// list sorted by cost with an atomic counter.
//
// What bounds it.  A 64-column tile of d = 64 takes an SM about 960 clocks; its
// products run for 512 (dq) or 640 (dk and dv: the ones from shared memory read
// all of its bandwidth), its softmax for 460-490, and they overlap as far as
// one warp gets the products issued (60-120 clocks each beside busy warps, 26 in
// 1500 clocks of a CTA's 1950).  4096 tokens of 64 / 8 heads of 64, bf16: 442 us of
// the call's 463, 1089 TFLOP/s of the seven products, tensor path 70% active, issue
// slots 55%; 3598 ragged f16 tokens of 32 / 8 heads of 128: 139 of 159 us, tensor path
// 59%.  2048 tokens of 16 / 4 heads of 256, bf16: 217 of 235 us, one stage, so that a
// tile's load, S, T and second products follow one another.  Registers: 96 a thread (two
// CTAs of ten warps, or one of 18, an SM), with 4 to 7 words spilled at d = 64 and 128: 0.06%
// and 0.4% of the instructions executed.
//
// Tile and CTAs.  d = 64: tiles of 64 columns and two CTAs an SM, which overlap each
// other's waits (one CTA with tiles of 128: 512 us, with two S tiles and two
// product warps 460 but 107 us instead of 95 with a window of 128, where a
// unit is three tiles long).  d = 128: tiles of 128, which the products read
// at full rate.  d = 256: 64, so that a tile of each operand fits.
#pragma once
#include "backward.h"
#include "launch.h"
#include "prefill_kernel.cuh"
#include "ptx.cuh"

namespace gqa {

constexpr int bwd_warps(int D) { return D == 64 ? 8 : 16; }  // softmax warps
constexpr int bwd_threads(int D) { return 32 * (bwd_warps(D) + 2); }
constexpr int kBwdRecs = 4;  // unit records in flight

constexpr int bwd_stages(int D) { return D == 64 ? 4 : D == 128 ? 2 : 1; }
constexpr uint32_t bwd_a_bytes(int D) { return 128u * D * 2u; }            // one tile
constexpr uint32_t bwd_b_bytes(int D) { return (uint32_t)bwd_n(D) * D * 2u; }
constexpr uint32_t bwd_stat_bytes(int D) { return 8u * bwd_n(D); }         // -lse, -D of a tile
constexpr uint32_t bwd_smem(int D) {
  return 1024u + 2u * bwd_a_bytes(D) +
         bwd_stages(D) * (2u * bwd_b_bytes(D) + bwd_stat_bytes(D)) + 64u * 8u + 16u +
         kBwdRecs * 64u;
}

// A truth value that picks a form of a generic lambda.
template <bool V>
struct Const {
  static constexpr bool value = V;
  __device__ constexpr operator bool() const { return V; }
};

struct BwdBar {
  static constexpr int kRecFull = 0, kRecEmpty = 4, kAFull = 8, kAEmpty = 9, kBFull = 10,
                       kBEmpty = 14, kLand = 18, kSFull = 19, kPFull = 20, kTFull = 22, kDFull = 23,
                       kAccDone = 24, kAccFree = 25, kDrain = 26, kCount = 27;
};

template <int D, bool BF16>
struct Bwd {
  static constexpr int N = bwd_n(D), NS = bwd_stages(D), NCH = D / 64,
                       WARPS = bwd_warps(D), PG = WARPS / 4, CW = N / PG;
  static constexpr uint32_t kABytes = bwd_a_bytes(D), kBBytes = bwd_b_bytes(D),
                            kStat = bwd_stat_bytes(D);
  static constexpr uint32_t kAChunk = 128u * 128u, kBChunk = N * 128u;
  static constexpr uint32_t kColT = N, kColAcc0 = D == 64 ? 128 : 256,
                            kColAcc1 = D == 64 ? 192 : D == 128 ? 384 : 256, kCols = 512 / bwd_per_sm(D);
  static_assert(kColT + N <= kColAcc0 && kColAcc1 + D <= kCols, "tensor memory");
};

// One tile of one unit in the hands of a softmax thread: lane row `r` of A,
// CW neighbouring columns of the tile.  lo, hi: the columns the row keeps.
struct BwdTile {
  uint32_t t_s, t_t;  // tensor-memory addresses of the thread's columns of S and T
  uint32_t stats;     // shared memory: -lse of the thread's columns; N floats on, -D (dk, dv units)
  float row_nlse, row_nd;
  int lo, hi;
  bool masked;  // whether some row of the tile has such an edge
};

template <int CW>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[CW]) {
  if constexpr (CW == 32)
    tmem_ld32(at, r);
  else
    tmem_ld16(at, r);
}
template <int W>
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[W]) {
  if constexpr (W == 16)
    tmem_st16(at, r);
  else
    tmem_st8(at, r);
}
__device__ __forceinline__ void ld_shared_f4(uint32_t at, float (&v)[4]) {
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(at));
}
// What this warp wrote to, or read from, tensor memory is done: one arrival.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

template <int KIND, int D, bool BF16, bool TWO>
__device__ __forceinline__ bool bwd_tile(const BwdTile& t, float sl2, float mul, uint32_t bar_s,
                                         uint32_t par_s, uint32_t bar_p, uint32_t bar_t,
                                         uint32_t par_t, uint32_t bar_d,
                                         volatile uint32_t* abort_flag, const BwdParams& p) {
  using K = Bwd<D, BF16>;
  constexpr int CW = K::CW;
  auto wait = [&](uint32_t bar, uint32_t par) {
    return __all_sync(0xffffffffu, wait_bounded(bar, par, abort_flag, p.status, p.timeout_ns));
  };
  if (!wait(bar_s, par_s)) return false;
  tc_fence_after();
  float x[CW];
  tmem_load<CW>(t.t_s, *reinterpret_cast<uint32_t(*)[CW]>(x));
  tmem_wait_ld();
  const uint64_t sc = f2(sl2, sl2);
#pragma unroll
  for (int c = 0; c < CW; c += 4) {
    float l[4];
    if constexpr (KIND == kBwdQ)
      l[0] = l[1] = l[2] = l[3] = t.row_nlse;
    else
      ld_shared_f4(t.stats + 4u * c, l);
    unf2(ffma2(f2(x[c], x[c + 1]), sc, f2(l[0], l[1])), x[c], x[c + 1]);
    unf2(ffma2(f2(x[c + 2], x[c + 3]), sc, f2(l[2], l[3])), x[c + 2], x[c + 3]);
  }
  if (t.masked) {
    // A bit per column: constant bits become predicates several at a time.
    const uint32_t below = t.hi >= 31 ? ~0u : t.hi < 0 ? 0u : (2u << t.hi) - 1u,
                   above = t.lo <= 0 ? ~0u : t.lo > 31 ? 0u : ~0u << t.lo, keep = below & above;
#pragma unroll
    for (int c = 0; c < CW; ++c)
      if ((keep & (1u << c)) == 0u) x[c] = -INFINITY;
  }
#pragma unroll
  for (int c = 0; c < CW; ++c) x[c] = ex2(x[c]);
  if constexpr (KIND == kBwdKV || KIND == kBwdV) {
    // P in 16 bits, over this thread's own columns of S.
    uint32_t pk[CW / 2];
#pragma unroll
    for (int c = 0; c < CW; c += 2) pk[c / 2] = pack2<BF16>(x[c], x[c + 1]);
    tmem_store<CW / 2>(t.t_s, pk);
    if constexpr (TWO) {
#pragma unroll
      for (int c = 0; c < CW; c += 2)
        pk[c / 2] = pack2<BF16>(x[c] - unpack_lo<BF16>(pk[c / 2]), x[c + 1] - unpack_hi<BF16>(pk[c / 2]));
      tmem_store<CW / 2>(t.t_s + CW / 2, pk);
    }
    tmem_wait_st();
  }
  warp_arrive(bar_p);  // S is read (and P written)
  if constexpr (KIND == kBwdV) return true;

  if (!wait(bar_t, par_t)) return false;
  tc_fence_after();
  uint32_t y[CW], dk[CW / 2];
  tmem_load<CW>(t.t_t, y);
  tmem_wait_ld();
  const uint64_t rnd = f2(t.row_nd, t.row_nd), mm = f2(mul, mul);
#pragma unroll
  for (int c = 0; c < CW; c += 4) {
    uint64_t n0 = rnd, n1 = rnd;
    if constexpr (KIND != kBwdQ) {
      float l[4];
      ld_shared_f4(t.stats + 4u * (uint32_t)K::N + 4u * c, l);
      n0 = f2(l[0], l[1]);
      n1 = f2(l[2], l[3]);
    }
    uint64_t a = fadd2(f2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), n0);
    uint64_t b = fadd2(f2(__uint_as_float(y[c + 2]), __uint_as_float(y[c + 3])), n1);
    if constexpr (!BF16) {  // f16: times a power of two, so that dS keeps its bits
      a = fmul2(a, mm);
      b = fmul2(b, mm);
    }
    float d0, d1, d2, d3;
    unf2(fmul2(a, f2(x[c], x[c + 1])), d0, d1);
    unf2(fmul2(b, f2(x[c + 2], x[c + 3])), d2, d3);
    dk[c / 2] = pack2<BF16>(d0, d1);
    dk[c / 2 + 1] = pack2<BF16>(d2, d3);
    if constexpr (TWO) {  // what the first term leaves, over T's values
      y[c / 2] = pack2<BF16>(d0 - unpack_lo<BF16>(dk[c / 2]), d1 - unpack_hi<BF16>(dk[c / 2]));
      y[c / 2 + 1] = pack2<BF16>(d2 - unpack_lo<BF16>(dk[c / 2 + 1]), d3 - unpack_hi<BF16>(dk[c / 2 + 1]));
    }
  }
  tmem_store<CW / 2>(t.t_t, dk);
  if constexpr (TWO)
    tmem_store<CW / 2>(t.t_t + CW / 2, *reinterpret_cast<uint32_t(*)[CW / 2]>(y));
  tmem_wait_st();
  warp_arrive(bar_d);
  return true;
}

// `cols` accumulator columns of this lane's row, times `mul`, to a row of the
// result or to a partial ([d / 4][128][4]), both from column `col0`.
template <int D, bool BF16>
__device__ __forceinline__ void bwd_store(uint32_t t_acc, int cols, int col0, float mul,
                                          uint16_t* row, float4* part, int r, bool zero) {
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    uint32_t o[32];
    if (!zero) {
      tmem_ld32(t_acc + c, o);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0u;
    }
    if (part != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        part[(size_t)((col0 + c) / 4 + i) * 128 + r] =
            make_float4(__uint_as_float(o[4 * i]) * mul, __uint_as_float(o[4 * i + 1]) * mul,
                        __uint_as_float(o[4 * i + 2]) * mul, __uint_as_float(o[4 * i + 3]) * mul);
    } else {
      // Four lanes exchange their rows' 16-byte pieces, so that a store writes 64
      // bytes a row: 8 lines an instruction instead of 32.
      uint32_t w[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[i][k] = pack2<BF16>(__uint_as_float(o[8 * i + 2 * k]) * mul, __uint_as_float(o[8 * i + 2 * k + 1]) * mul);
      const int lane = r & 31;
#pragma unroll
      for (int step = 1; step <= 2; ++step) {
        const bool up = (lane & step) != 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int a = step == 1 ? 2 * i : i, b = a + step;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[a][k] : w[b][k], step);
            w[a][k] = up ? got : w[a][k];
            w[b][k] = up ? w[b][k] : got;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint16_t* to = reinterpret_cast<uint16_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), (lane & ~3) + i));
        if (to != nullptr)
          reinterpret_cast<uint4*>(to + col0 + c)[lane & 3] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
      }
    }
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(bwd_threads(D), bwd_per_sm(D))
    backward_kernel(const __grid_constant__ BwdParams p) {
  using K = Bwd<D, BF16>;
  using B = BwdBar;
  constexpr int N = K::N, NS = K::NS, NCH = K::NCH, CW = K::CW;
  constexpr int WARPS = K::WARPS, kLoadWarp = WARPS, kMmaWarp = WARPS + 1;
  constexpr uint32_t kIdescS = idesc_f16(BF16, 128, N, false);
  constexpr uint32_t kIdescO = idesc_f16(BF16, 128, D, true);

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sA = smem_u32(smem);                      // [2] tiles
  const uint32_t sB = sA + 2u * K::kABytes;           // [NS][2] tiles
  const uint32_t sStat = sB + NS * 2u * K::kBBytes;        // [NS] -lse, -D
  uint8_t* tail = smem + 2u * K::kABytes + NS * (2u * K::kBBytes + K::kStat);
  uint64_t* bars = reinterpret_cast<uint64_t*>(tail);
  const uint32_t sBar = smem_u32(bars);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 64);  // [0] tensor memory, [1] abort
  int32_t* recs = reinterpret_cast<int32_t*>(misc + 4);     // [kBwdRecs][16]
  volatile uint32_t* abort_flag = misc + 1;
  auto bar = [&](int i) { return sBar + 8u * (uint32_t)i; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < B::kCount; ++i) {
      uint32_t cnt = 1u;
      if (i >= B::kRecEmpty && i < B::kRecEmpty + kBwdRecs) cnt = WARPS + 1u;
      if (i == B::kPFull || i == B::kPFull + 1 || i == B::kDFull || i == B::kAccFree)
        cnt = WARPS;
      mbar_init(bar(i), cnt);
    }
    misc[1] = 0u;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(misc), K::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  grid_dep_launch_dependents();
  grid_dep_wait();
  const int items = p.hdr[kBwdUnits] * p.Hkv;

  // ---------------------------------------------------------------- loads
  if (warp == kLoadWarp) {
    auto wait = [&](int b, uint32_t par) {
      return __all_sync(0xffffffffu,
                        wait_bounded(bar(b), par, abort_flag, p.status, p.timeout_ns));
    };
    uint32_t it = 0, ua = 0, lands = 0;
    for (uint32_t un = 0;; ++un) {
      const uint32_t rs = un % kBwdRecs;
      if (!wait(B::kRecEmpty + rs, ((un / kBwdRecs) & 1u) ^ 1u)) break;
      int item = (int)blockIdx.x;
      if (un > 0) {
        if (lane == 0) item = (int)gridDim.x + atomicAdd(&p.hdr[kBwdNext], 1);
        item = __shfl_sync(0xffffffffu, item, 0);
      }
      const bool end = item >= items;
      const int e = end ? 0 : item / p.Hkv, g = end ? 0 : item - e * p.Hkv;
      int word = 0;
      if (lane < 16) {
        word = end ? -1 : reinterpret_cast<const int32_t*>(p.units + e)[lane];
        if (lane == 13) word = g;
        recs[rs * 16 + lane] = word;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kRecFull + rs));
      if (end) break;
      auto field = [&](int i) { return __shfl_sync(0xffffffffu, word, i); };
      const int kind = field(0) & 3, n = field(1), a_base = field(2), a_off = field(3),
                b_base = field(5), b_off = field(6), b_len = field(7), stat = field(11);
      if (n == 0) continue;
      const bool qa = kind == kBwdQ;
      if (!wait(B::kAEmpty, (ua & 1u) ^ 1u)) break;
      if (lane == 0) {
        const uint32_t full = bar(B::kAFull), dst = sA;
        mbar_arrive_expect_tx(full, 2u * K::kABytes);
        // Queries are counted in packed rows, token by token: the G heads of a
        // KV head, one after the other.  A tile of 128 starts at a token.
        const int head = qa ? g * p.G : g, row = a_base + (qa ? a_off >> p.log_G : a_off);
        for (int c = 0; c < NCH; ++c) {
          tma_load_3d(dst + c * K::kAChunk, qa ? &p.a_q : &p.a_k, full, c * 64, head, row);
          tma_load_3d(dst + K::kABytes + c * K::kAChunk, qa ? &p.a_do : &p.a_v, full, c * 64, head,
                      row);
        }
      }
      ++ua;
      bool ok = true;
      for (int j = 0; j < n; ++j, ++it) {
        const uint32_t s = it % NS;
        if (!(ok = wait(B::kBEmpty + s, ((it / NS) & 1u) ^ 1u))) break;
        const int off = b_off + j * N, valid = b_len - off;
        const bool whole = valid >= N;
        const uint32_t dst = sB + s * 2u * K::kBBytes;
        const uint32_t full = bar(whole ? B::kBFull + s : B::kLand);
        if (lane == 0) {
          mbar_arrive_expect_tx(full, 2u * K::kBBytes + (qa ? 0u : K::kStat));
          const int head = qa ? g : g * p.G + (off & (p.G - 1));
          const int row = b_base + (qa ? off : off >> p.log_G);
          for (int c = 0; c < NCH; ++c) {
            tma_load_3d(dst + c * K::kBChunk, qa ? &p.b_k : &p.b_q, full, c * 64, head, row);
            tma_load_3d(dst + K::kBBytes + c * K::kBChunk, qa ? &p.b_v : &p.b_do, full, c * 64, head,
                        row);
          }
          if (!qa) {
            const size_t at = (size_t)g * p.stat_rows + stat + off;
            bulk_load(sStat + s * K::kStat, p.nlse + at, 4u * N, full);
            bulk_load(sStat + s * K::kStat + 4u * N, p.nd + at, 4u * N, full);
          }
        }
        if (!whole) {
          // Rows past the sequence's last are another's, or hold anything: they
          // become zeros, so that their zero probabilities add nothing.
          const bool landed = wait(B::kLand, lands & 1u);
          ++lands;
          if (!(ok = landed)) {
            ++it;
            break;
          }
          for (int c = 0; c < 2 * NCH; ++c)
            for (int x = valid * 128 + lane * 16; x < N * 128; x += 512)
              st_shared_v4(dst + c * K::kBChunk + x, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B::kBFull + s));
        }
      }
      if (!ok) break;
    }
    // Let every copy issued land before the CTA can exit: another warp may give up
    // after this one has issued its last.
    if (ua > 0) wait_drain(bar(B::kAFull), (ua - 1u) & 1u, p.timeout_ns);
    if (lands > 0) wait_drain(bar(B::kLand), (lands - 1u) & 1u, p.timeout_ns);
    for (uint32_t b = 0; b < NS; ++b)
      if (it > b)
        wait_drain(bar(B::kBFull + (it - 1u - b) % NS), ((it - 1u - b) / NS) & 1u, p.timeout_ns);
    __syncwarp();
  }

  // ---------------------------------------------------------------- products
  if (warp == kMmaWarp) {
    const uint64_t dA1 = smem_desc_sw128(sA, 16, 1024), dA2 = dA1 + (K::kABytes >> 4);
    const uint64_t dB0 = smem_desc_sw128(sB, 16, 1024);           // rows are N
    const uint64_t dBt0 = smem_desc_sw128(sB, K::kBChunk, 1024);  // rows are the contraction
    auto kstep = [](int kk, uint32_t chunk) -> uint64_t {
      return (uint64_t)(((uint32_t)(kk >> 2) * chunk + (uint32_t)(kk & 3) * 32u) >> 4);
    };
    auto wait = [&](int b, uint32_t par) {
      return __all_sync(0xffffffffu,
                        wait_bounded(bar(b), par, abort_flag, p.status, p.timeout_ns));
    };
    // it: tiles; td: tiles with a T; uc: units with tiles.
    uint32_t it = 0, td = 0, uc = 0;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      const uint32_t rs = un % kBwdRecs;
      if (!(ok = wait(B::kRecFull + rs, (un / kBwdRecs) & 1u))) break;
      const int word = recs[rs * 16], kind = word & 3, n = recs[rs * 16 + 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kRecEmpty + rs));
      if (word < 0) break;
      if (n == 0) continue;
      const bool has_t = kind != kBwdV, has_p = kind == kBwdKV || kind == kBwdV;
      if (!(ok = wait(B::kAFull, uc & 1u))) break;
      auto issue_s = [&](uint32_t t) -> bool {  // S of tile t, once it is in
        const uint32_t s = t % NS;
        if (!wait(B::kBFull + s, (t / NS) & 1u)) return false;
        tc_fence_after();
        const uint64_t b1 = dB0 + s * 2u * (K::kBBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem, dA1 + kstep(kk, K::kAChunk), b1 + kstep(kk, K::kBChunk),
                 kIdescS, kk > 0 ? 1u : 0u);
        mma_commit(bar(B::kSFull));
        return true;
      };
      // acc (+)= (the 16-bit tile at `src`) B: each warpgroup's columns stand at
      // the start of its fp32 ones.
      auto issue_acc = [&](auto two, uint32_t acc, uint32_t src, uint64_t b, bool first) {
#pragma unroll
        for (int kk = 0; kk < N / 16; ++kk)
          mma_ts(acc, src + (kk / (CW / 16)) * CW + (kk % (CW / 16)) * 8,
                 b + (uint64_t)(kk * 128), kIdescO, (first && kk == 0) ? 0u : 1u);
        if (two) {
#pragma unroll
          for (int kk = 0; kk < N / 16; ++kk)
            mma_ts(acc, src + (kk / (CW / 16)) * CW + (kk % (CW / 16)) * 8 + CW / 2,
                   b + (uint64_t)(kk * 128), kIdescO, 1u);
        }
      };
      if constexpr (NS > 1) {
        ok = issue_s(it);
        if (!ok) break;
      }
      auto tiles = [&](auto two) {
        for (int j = 0; j < n; ++j, ++it) {
          const uint32_t s = it % NS;
          if constexpr (NS == 1) {
            ok = issue_s(it);
            if (!ok) break;
          }
          const uint64_t dB = dB0 + s * 2u * (K::kBBytes >> 4), dBt = dBt0 + s * 2u * (K::kBBytes >> 4);
          if (has_t) {
            const uint64_t b2 = dB + (K::kBBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + K::kColT, dA2 + kstep(kk, K::kAChunk), b2 + kstep(kk, K::kBChunk), kIdescS,
                     kk > 0 ? 1u : 0u);
            mma_commit(bar(B::kTFull));
          }
          if (j == n - 1) mma_commit(bar(B::kAEmpty));
          if (!(ok = wait(B::kPFull + (it & 1u), (it >> 1) & 1u))) break;
          if (j == 0 && uc > 0 && !(ok = wait(B::kAccFree, (uc - 1u) & 1u))) break;
          tc_fence_after();
          if (has_p)
            issue_acc(two, tmem + K::kColAcc0, tmem, dBt + (K::kBBytes >> 4), j == 0);
          if constexpr (NS > 1) {
            if (j + 1 < n) ok = issue_s(it + 1);
            if (!ok) break;
          }
          if (has_t) {
            if (!(ok = wait(B::kDFull, td & 1u))) break;
            tc_fence_after();
            issue_acc(two, tmem + K::kColAcc1, tmem + K::kColT, dBt, j == 0);
            ++td;
          }
          mma_commit(bar(B::kBEmpty + s));
        }
      };
      // A branch a tile, or two forms of the loop: 157.7 or 161.4 us for 3598 ragged tokens
      // of d = 128, 469 or 464 for 4096 of d = 64.
      const bool two = (word & kBwdTwo) != 0;
      if constexpr (D == 128)
        tiles(two);
      else if (two)
        tiles(Const<true>{});
      else
        tiles(Const<false>{});
      if (!ok) break;
      mma_commit(bar(B::kAccDone));
      ++uc;
    }
    mma_commit(bar(B::kDrain));
    wait_drain(bar(B::kDrain), 0u, p.timeout_ns);
    __syncwarp();
  }

  // ---------------------------------------------------------------- softmax, results
  if (warp < WARPS) {
    constexpr int PG = K::PG;
    const int part = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = p.scale_log2;
    auto wait = [&](int b, uint32_t par) {
      return __all_sync(0xffffffffu,
                        wait_bounded(bar(b), par, abort_flag, p.status, p.timeout_ns));
    };
    uint32_t it = 0, td = 0, uc = 0;
    // The next unit's record, and what of global memory it needs: on its way while
    // this unit's results are stored.
    int next = -1;
    float next_nlse = 0.f, next_nd = 0.f, next_o2 = 0.f, next_v2 = 0.f;
    auto fetch = [&](uint32_t un) -> bool {
      const uint32_t rs = un % kBwdRecs;
      if (!wait(B::kRecFull + rs, (un / kBwdRecs) & 1u)) return false;
      const int32_t* rec = recs + rs * 16;
      next = rec[0];
      if (next < 0) return true;
      const int kind = next & 3;
      if (kind == kBwdQ) {
        const size_t at = (size_t)rec[13] * p.stat_rows + rec[11] + rec[3] + r;
        next_nlse = __ldcg(p.nlse + at);
        next_nd = __ldcg(p.nd + at);
        if constexpr (!BF16) next_o2 = __ldcg(p.row_o2 + at);
      } else if (!BF16 && kind != kBwdV) {
        // The largest of the query tiles that the unit streams.
        const int t0 = rec[6] >> 7, t1 = (min(rec[6] + rec[1] * N, rec[7]) + 127) >> 7;
        const uint2* most = p.tile_most + (size_t)rec[13] * p.max_qtiles + (rec[11] >> 7);
        uint32_t o2 = 0u, dm = 0u;
        for (int i = t0 + lane; i < t1; i += 32) {
          const uint2 m = __ldcg(most + i);
          o2 = max(o2, m.x);
          dm = max(dm, m.y);
        }
        next_o2 = __uint_as_float(__reduce_max_sync(0xffffffffu, o2));
        next_nd = __uint_as_float(__reduce_max_sync(0xffffffffu, dm));
      }
      if (!BF16 && kind != kBwdV) next_v2 = __uint_as_float(__ldcg(p.most_v + (size_t)rec[12] * p.Hkv + rec[13]));
      return true;
    };
    bool ok = fetch(0);
    for (uint32_t un = 0; ok && next >= 0; ++un) {
      const uint32_t rs = un % kBwdRecs;
      const int32_t* rec = recs + rs * 16;
      const int kind = next & 3, n = rec[1];
      const bool two_terms = (next & kBwdTwo) != 0;
      const bool qa = kind == kBwdQ;
      BwdTile t;
      t.row_nlse = next_nlse;
      t.row_nd = next_nd;
      float mul = 1.f, undo = 1.f;  // of dS, and of the results it enters
      if constexpr (!BF16) {
        const int k = bwd_exponent(next_o2, fabsf(next_nd), next_v2);
        mul = ldexpf(1.f, k - (int)kBwdBias);
        undo = ldexpf(1.f, -k);
      }
      const int a_off = rec[3], b_off = rec[6];
      // Columns the row keeps, counted from B's first row: key or packed row
      // c of tile j is kept iff lo0 <= b_off + j N + c <= hi0.
      int lo0, hi0;
      const int lo_max = rec[14], hi_min = rec[15];  // over A's rows: the largest lo0, the least hi0
      {
        bwd_bounds(qa, a_off + r, rec[8], rec[9], p.log_G, p.reach, lo0, hi0);
        lo0 -= part * CW;
        hi0 -= part * CW;
      }
      auto tiles = [&](auto two) {
        constexpr bool TWO = decltype(two)::value;
        for (int j = 0; j < n; ++j, ++it) {
          const uint32_t s = it % NS;
          const int off = b_off + j * N;
          t.t_s = t_lane + part * CW;
          t.t_t = t_lane + K::kColT + part * CW;
          t.stats = sStat + s * K::kStat + (uint32_t)part * CW * 4u;
          t.lo = lo0 - off;
          t.hi = hi0 - off;
          t.masked = lo_max > off || hi_min < off + N - 1;
          const uint32_t bs = bar(B::kSFull), ps = it & 1u, bp = bar(B::kPFull + (it & 1u)),
                         bt = bar(B::kTFull), bd = bar(B::kDFull);
          if (qa) {
            ok = bwd_tile<kBwdQ, D, BF16, TWO>(t, sl2, mul, bs, ps, bp, bt, td & 1u, bd, abort_flag, p);
          } else {
            // The statistics came with B (this thread has to see their barrier).
            if (!(ok = wait(B::kBFull + s, (it / NS) & 1u))) break;
            if constexpr (D < 256)
              ok = bwd_tile<kBwdKV, D, BF16, TWO>(t, sl2, mul, bs, ps, bp, bt, td & 1u, bd, abort_flag, p);
            else if (kind == kBwdK)
              ok = bwd_tile<kBwdK, D, BF16, TWO>(t, sl2, mul, bs, ps, bp, bt, td & 1u, bd, abort_flag, p);
            else
              ok = bwd_tile<kBwdV, D, BF16, TWO>(t, sl2, mul, bs, ps, bp, bt, td & 1u, bd, abort_flag, p);
          }
          if (!ok) break;
          if (kind != kBwdV) ++td;
        }
      };
      if (two_terms)
        tiles(Const<true>{});
      else
        tiles(Const<false>{});
      if (!ok || !(ok = fetch(un + 1u))) break;
      // Half of the warpgroups take dv and half dk of a unit with both, else each
      // an equal share of the columns of its one result.
      const bool both = kind == kBwdKV;
      const bool is_v = kind == kBwdV || (both && part < PG / 2);
      const float out_mul = is_v ? (BF16 ? 1.f : 1.f / 32768.f) : p.scale * undo;
      const uint32_t acc = is_v ? K::kColAcc0 : K::kColAcc1;
      static_assert(D / PG % 32 == 0, "bwd_store takes 32 columns at a time");
      const int cols = both ? D / (PG / 2) : D / PG, col0 = (both ? part % (PG / 2) : part) * cols;
      const int a_base = rec[2], slot = rec[10], g = rec[13];
      uint16_t* row = nullptr;
      float4* to_part = nullptr;
      if (slot >= 0) {
        to_part = reinterpret_cast<float4*>(p.part) +
               (((size_t)slot * p.Hkv + g) * bwd_accs(D) + (both && !is_v ? 1 : 0)) * (D / 4) * 128;
      } else if (r < rec[4]) {
        if (qa) {
          const int a = a_off + r;
          row = static_cast<uint16_t*>(p.dq) +
                ((size_t)(a_base + (a >> p.log_G)) * p.Hq + g * p.G + (a & (p.G - 1))) * D;
        } else {
          row = static_cast<uint16_t*>(is_v ? p.dv : p.dk) + ((size_t)(a_base + a_off + r) * p.Hkv + g) * D;
        }
      }
      if (n > 0) {
        if (!(ok = wait(B::kAccDone, uc & 1u))) break;
        tc_fence_after();
      }
      bwd_store<D, BF16>(t_lane + acc + col0, cols, col0, out_mul, row, to_part, r, n == 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kRecEmpty + rs));
      if (n > 0) {
        warp_arrive(bar(B::kAccFree));
        ++uc;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && *abort_flag) p.hdr[kBwdFailed] = 1;  // nothing is joined
  if (warp == kMmaWarp) tmem_dealloc(tmem, K::kCols);
}

namespace {

template <int D, bool BF16>
cudaError_t launch_backward(const BwdParams& p, cudaStream_t st) {
  auto kern = backward_kernel<D, BF16>;
  static SmemAttr attr{};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  constexpr unsigned smem = bwd_smem(D);
  static_assert(smem <= 227u * 1024u, "shared memory");
  if (attr.allowed[dev].load(std::memory_order_acquire) < smem) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr.allowed[dev].store(smem, std::memory_order_release);
  }
  return launch_pdl(kern, p, p.ctas, bwd_threads(D), smem, st);
}

}  // namespace

}  // namespace gqa
