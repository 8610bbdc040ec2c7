// cache_tile.cuh -- the form of gqa_cache_attention for many query rows per KV
// head (a draft tree of some tens of tokens, a short chunk): 128-row tiles on
// the tensor memory, sm_103a.
//
// The mathematics is cache_attn.cuh's; here the rows fill a 128-row tile, so
// the products go to tcgen05 and the bound moves from memory to the
// exponentials (128 keys x 128 rows take the special-function units 1024
// clocks, the two products 512 at d = 64).  Two CTAs per SM, so that one's
// softmax runs beside the other's products.
//
// A CTA of 8 warps:
//   0..3  softmax and output, thread = row = tensor-memory lane; they also
//         bring the rows of Q into shared memory;
//   4..6  bring K and V: 16-byte loads from the pages straight to registers,
//         e4m3 widened to f16 (exact, the scales stay apart), stored in the
//         128-byte swizzle the products read.  A tile is loaded while the one
//         before waits for its slot.  Keys no row sees become zeros;
//   7     plans the work and issues the products.
// The scales of an e4m3 tile go to shared memory as fp32: the softmax
// multiplies a key's scores by its K scale, and takes its V scale into the
// exponent (P) and out of the denominator, in pairs of keys.
#pragma once
#include "cache_attn.cuh"

namespace gqa {

constexpr int kCtThreads = 256;
constexpr int kCtLoaders = 96;
constexpr int kCtWholeSlack = 2;  // tiles a join is worth
__host__ __device__ constexpr int ct_bn(int D) { return D == 64 ? 128 : 64; }
// Q tile, two slots each of K and V, their scales, the tables of the sequences.
__host__ __device__ constexpr uint32_t ct_smem(int D) {
  return 1024u + 128u * D * 2u + 4u * ct_bn(D) * D * 2u + 2u * ct_bn(D) * 12u +
         4u * (5 * kMaxSeqs + 3) + kCaPieces * 64u + 32u * 8u + 32u;
}

struct CtBar {  // barrier numbers
  static constexpr int kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kSFree = 9,
                       kPFull = 10, kODone = 11, kQFull = 12, kDrain = 13, kPiece = 14;
};

template <int D, bool BF16, bool C8>
__global__ void __launch_bounds__(kCtThreads, 2)
    cache_tile_kernel(const __grid_constant__ CacheAttnParams p) {
  constexpr int BN = ct_bn(D), RT = 128;
  constexpr bool MBF = BF16 && !C8;  // product type
  constexpr float kBias = MBF ? 0.f : kCaBias;
  constexpr int kEsz = C8 ? 1 : 2;
  constexpr uint32_t kQBytes = 128u * D * 2u, kKVBytes = (uint32_t)BN * D * 2u;
  constexpr uint32_t kQChunk = 128u * 128u, kKVChunk = (uint32_t)BN * 128u;
  constexpr uint32_t kColS = 0, kColP = BN, kColO = BN + BN / 2;
  static_assert(kColO + D <= 256, "two CTAs share the tensor memory");
  constexpr uint32_t kIdescS = idesc_f16(MBF, 128, BN, false);
  constexpr uint32_t kIdescO = idesc_f16(MBF, 128, D, true);
  using B = CtBar;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_u32(smem), sK = sQ + kQBytes, sV = sK + 2u * kKVBytes;
  float* s_ks = reinterpret_cast<float*>(smem + kQBytes + 4u * kKVBytes);  // [2][BN]
  float* s_we = s_ks + 2 * BN;                                            // [2][BN]
  float* s_wi = s_we + 2 * BN;                                            // [2][BN]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_wi + 2 * BN);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 32);  // [0] abort [1] bad [2] most tiles [3] tmem
  int4* s_piece = reinterpret_cast<int4*>(misc + 8);
  int32_t* tiles = reinterpret_cast<int32_t*>(s_piece + 4 * kCaPieces);
  int32_t* units = tiles + (kMaxSeqs + 1);
  int32_t* s_cu = units + (kMaxSeqs + 1);
  int32_t* s_pre = s_cu + (kMaxSeqs + 1);
  int32_t* s_ipt = s_pre + kMaxSeqs;
  const uint32_t sBar = smem_u32(bars);
  const uint32_t sPiece = sBar + 8u * B::kPiece;
  volatile uint32_t* abort_flag = misc;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned long long tmo = p.timeout_ns;

  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(sBar + 8u * (B::kKFull + i), kCtLoaders);
      mbar_init(sBar + 8u * (B::kVFull + i), kCtLoaders);
      // Free once the product is done and, for e4m3, the softmax warps have
      // read the scales.
      mbar_init(sBar + 8u * (B::kKEmpty + i), C8 ? 5u : 1u);
      mbar_init(sBar + 8u * (B::kVEmpty + i), C8 ? 5u : 1u);
    }
    mbar_init(sBar + 8u * B::kSFull, 1u);
    mbar_init(sBar + 8u * B::kSFree, 128u);
    mbar_init(sBar + 8u * B::kPFull, 128u);
    mbar_init(sBar + 8u * B::kODone, 1u);
    mbar_init(sBar + 8u * B::kQFull, 128u);
    mbar_init(sBar + 8u * B::kDrain, 1u);
    for (int i = 0; i < kCaPieces; ++i) {
      mbar_init(sPiece + 8u * i, 1u);
      mbar_init(sPiece + 8u * (kCaPieces + i), 7u);  // 4 softmax and 3 loading warps
    }
    misc[0] = 0u;
    misc[1] = 0u;
    misc[2] = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_launch_dependents();
  if (!p.metadata_ready) grid_dep_wait();
  ca_tables(p, tiles, units, s_cu, s_pre, s_ipt, misc, RT, tid, kCtThreads);
  __syncthreads();
  const bool bad_meta = misc[1] != 0u;
  if (p.metadata_ready) grid_dep_wait();  // before any global write or other read
  if (bad_meta) {
    if (tid == 0) {
      atomicOr(p.status, 2u);  // GQA_DEV_BAD_METADATA
      if (blockIdx.x == 0) p.hdr[0] = 0;
    }
    return;
  }
  if (warp == 7) {
    tmem_alloc(smem_u32(misc + 3), 256u);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[3];
  // Every lane of a warp goes on or none.
  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, p.status, tmo)) != 0;
  };
  // The next piece from the planning warp; false when there is none.
  auto next_piece = [&](uint32_t pi, int4& d0, int4& d1, int4& d2, bool& ok) {
    const uint32_t ps = pi % kCaPieces;
    ok = wait_all(sPiece + 8u * ps, (pi / kCaPieces) & 1u);
    if (!ok) return false;
    d0 = s_piece[4 * ps];
    d1 = s_piece[4 * ps + 1];
    d2 = s_piece[4 * ps + 2];
    __syncwarp();
    if (lane == 0) mbar_arrive(sPiece + 8u * (kCaPieces + ps));
    return d0.x > 0;
  };

  if (warp == 7) {
    // -------------------------------------------------------------- plan, products
    const uint64_t dQ = smem_desc_sw128(sQ, 16, 1024);
    const uint64_t dK0 = smem_desc_sw128(sK, 16, 1024);
    const uint64_t dV0 = smem_desc_sw128(sV, kKVChunk, 1024);
    auto kstep = [](int kk, uint32_t chunk) -> uint64_t {
      return (uint64_t)(((uint32_t)(kk >> 2) * chunk + (uint32_t)(kk & 3) * 32u) >> 4);
    };
    auto issue_pv = [&](uint32_t it, bool first) -> bool {
      const uint32_t s = it & 1u;
      if (!wait_all(sBar + 8u * (B::kVFull + s), (it >> 1) & 1u)) return false;
      if (!wait_all(sBar + 8u * B::kPFull, it & 1u)) return false;
      tc_fence_after();
      const uint64_t dv = dV0 + s * (kKVBytes >> 4);
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        mma_ts(tmem + kColO, tmem + kColP + kk * 8, dv + (uint64_t)(kk * 128), kIdescO,
               (first && kk == 0) ? 0u : 1u);
      mma_commit(sBar + 8u * (B::kVEmpty + s));
      mma_commit(sBar + 8u * B::kODone);
      return true;
    };
    CaPlan plan = ca_plan(p, tiles, units, s_cu, s_pre, s_ipt, misc);
    // A piece is told to the other warps one ahead of its products.
    uint32_t told = 0;
    auto tell = [&](CaPiece& u, bool& more) -> bool {
      more = ca_next(p, plan.T, plan.walk, RT, u);
      const uint32_t ps = told % kCaPieces;
      if (!wait_all(sPiece + 8u * (kCaPieces + ps), ((told / kCaPieces) & 1u) ^ 1u)) return false;
      if (lane == 0) {
        ca_publish(p, plan, u, more, RT, s_piece + 4 * ps);
        mbar_arrive(sPiece + 8u * ps);
      }
      ++told;
      __syncwarp();
      return true;
    };
    CaPiece u = {};
    bool more = false;
    bool ok = tell(u, more);
    uint32_t it = 0, pc = 0;
    while (ok && more) {
      const int n = u.t1 - u.t0;
      CaPiece un = {};
      bool more_n = false;
      if (!(ok = tell(un, more_n))) break;
      if (!(ok = wait_all(sBar + 8u * B::kQFull, pc & 1u))) break;
      for (int j = 0; j < n; ++j, ++it) {
        const uint32_t s = it & 1u;
        if (!(ok = wait_all(sBar + 8u * (B::kKFull + s), (it >> 1) & 1u))) break;
        if (it > 0 && !(ok = wait_all(sBar + 8u * B::kSFree, (it - 1u) & 1u))) break;
        tc_fence_after();
        const uint64_t dk = dK0 + s * (kKVBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + kColS, dQ + kstep(kk, kQChunk), dk + kstep(kk, kKVChunk), kIdescS,
                 kk > 0 ? 1u : 0u);
        mma_commit(sBar + 8u * B::kSFull);
        mma_commit(sBar + 8u * (B::kKEmpty + s));
        // The second product of a tile goes after the next tile's first, so
        // that the tensor core works on S(j) while the softmax is at S(j - 1).
        if (j > 0 && !(ok = issue_pv(it - 1u, j == 1))) break;
      }
      if (!ok) break;
      if (!(ok = issue_pv(it - 1u, n == 1))) break;
      ++pc;
      u = un;
      more = more_n;
    }
    mma_commit(sBar + 8u * B::kDrain);  // completes when every product issued is done
    wait_drain(sBar + 8u * B::kDrain, 0u, tmo);
    __syncwarp();
  } else if (warp >= 4) {
    // -------------------------------------------------------------- K and V
    constexpr int kCpr = D * kEsz / 16;                          // 16-byte loads per key
    constexpr int kStep = kCtLoaders / kCpr;                     // keys a round of all threads
    constexpr int kLoads = (BN + kStep - 1) / kStep;             // of a thread, K or V
    static_assert(kCtLoaders % kCpr == 0, "a thread keeps its place in a key");
    // The thread loads 16 bytes, at place q, of keys j0, j0 + kStep, ..
    const int lt = tid - 128, q = lt % kCpr, j0 = lt / kCpr;
    const long long tok_bytes = (long long)p.Hkv * D * kEsz;
    uint4 raw[kLoads];
    int row[kLoads];        // pool rows of the tile's keys, -1 for a key no row sees
    uint32_t sc[kLoads];    // the keys' scale bytes, in the threads at place 0
    int4 d0 = {}, d1 = {}, d2 = {};
    uint32_t pi = 0, it = 0;
    bool ok = true;
    auto places = [&](int n0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int key = n0 + j0 + i * kStep;
        row[i] = -1;
        if (j0 + i * kStep < BN && key < d1.y && (p.window == 0 || key > d0.w - p.window)) {
          const int kp = p.div_page.div(key);
          int pg = __ldg(p.indices + d2.z + kp);
          if ((unsigned)pg >= (unsigned)p.num_pages) {
            atomicOr(p.status, 2u);  // GQA_DEV_BAD_METADATA
            pg = 0;
          }
          row[i] = pg * p.page_size + (key - kp * p.page_size);  // the pool has < 2^31 rows
        }
      }
    };
    auto fetch = [&](bool is_v) {
      const uint8_t* src =
          (is_v ? p.v_pages : p.k_pages) + (long long)d1.w * (D * kEsz) + 16 * q;
      const uint8_t* scales = (is_v ? p.v_scales : p.k_scales) + d1.w;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        sc[i] = 0u;
        if (row[i] >= 0) {
          raw[i] = __ldg(reinterpret_cast<const uint4*>(src + row[i] * tok_bytes));
          if (C8 && q == 0) sc[i] = __ldg(scales + (long long)row[i] * p.Hkv);
        }
      }
    };
    // 16-byte unit c of key row j goes to unit c ^ (j & 7) of its 128-byte row.
    auto put = [&](uint32_t base, int j, int unit, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
      st_shared_v4(base + (uint32_t)(unit >> 3) * kKVChunk + (uint32_t)j * 128u +
                       (uint32_t)(((unit & 7) ^ (j & 7)) << 4),
                   a, b, c, d);
    };
    auto store = [&](uint32_t it2, bool is_v) -> bool {
      const uint32_t s = it2 & 1u;
      if (!wait_all(sBar + 8u * ((is_v ? B::kVEmpty : B::kKEmpty) + s), ((it2 >> 1) & 1u) ^ 1u))
        return false;
      const uint32_t base = (is_v ? sV : sK) + s * kKVBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int j = j0 + i * kStep;
        if (BN % kStep != 0 && j >= BN) break;
        if constexpr (C8) {
          uint32_t h[8];
          e4m3x4_f16(raw[i].x, h[0], h[1]);
          e4m3x4_f16(raw[i].y, h[2], h[3]);
          e4m3x4_f16(raw[i].z, h[4], h[5]);
          e4m3x4_f16(raw[i].w, h[6], h[7]);
          put(base, j, 2 * q, h[0], h[1], h[2], h[3]);
          put(base, j, 2 * q + 1, h[4], h[5], h[6], h[7]);
          if (q == 0) {
            if (is_v) {
              s_we[s * BN + j] = sc[i] ? __uint_as_float(0x4B000000u | sc[i]) - 8388735.f : 0.f;
              s_wi[s * BN + j] = __uint_as_float((254u - sc[i]) << 23);
            } else {
              s_ks[s * BN + j] = __uint_as_float(sc[i] << 23);
            }
          }
        } else {
          put(base, j, q, raw[i].x, raw[i].y, raw[i].z, raw[i].w);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(sBar + 8u * ((is_v ? B::kVFull : B::kKFull) + s));
      return true;
    };
    // Loads run one half tile (K or V) ahead of the stores, across pieces.
    bool have = next_piece(pi++, d0, d1, d2, ok);
    if (have) {
      places(d0.z);
      fetch(false);
    }
    while (ok && have) {
      const int n = d0.x, first = d0.z;
      for (int j = 0; j < n; ++j, ++it) {
        if (!(ok = store(it, false))) break;
        fetch(true);
        if (!(ok = store(it, true))) break;
        int next = first + (j + 1) * BN;
        if (j + 1 == n) {
          have = next_piece(pi++, d0, d1, d2, ok);
          if (!have) break;
          next = d0.z;
        }
        places(next);
        fetch(false);
      }
    }
  } else {
    // -------------------------------------------------------------- softmax, output
    const int r = tid;  // row of the tile, lane of the tensor memory
    const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
    int4 d0 = {}, d1 = {}, d2 = {};
    uint32_t pi = 0, it = 0;
    bool ok = true;
    while (next_piece(pi++, d0, d1, d2, ok)) {
      const int n = d0.x, P = d0.w, E = d1.x, head = d1.w, cu0 = d2.x;
      const bool cut = (d0.y & 1) != 0;
      const int gr = d1.z + r;  // row of the sequence
      const int i = p.div_g.div(gr);
      const bool on = i < E;
      const int qh = head * p.G + (gr - i * p.G);
      const long long row = (long long)(cu0 + (on ? i : 0)) * p.Hq + qh;
      int dep = i;
      if (on && p.depths != nullptr) dep = __ldg(p.depths + cu0 + i);
      float sink = -INFINITY;
      if (p.sinks != nullptr) sink = __ldg(p.sinks + qh) * kLog2e;
      else if (p.smooth) sink = 0.f;
      // ---- this row of Q.  The last product that read the tile before is
      // done: its scores were read here.
      float rs = p.scale_log2;
      {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + row * D);
        uint4 w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = on ? __ldg(q + c) : make_uint4(0u, 0u, 0u, 0u);
        float f = 1.f;
        if constexpr (C8) {
          // f16 operands: the row scaled by the power of two that brings its
          // largest magnitude into [1, 2); smaller values round at 2^-25.
          float amax = 0.f;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = max3(amax, fabsf(unpack_lo<BF16>(x[k])), fabsf(unpack_hi<BF16>(x[k])));
          }
          const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126);
          f = __int_as_float((127 - e) << 23);
          rs *= __int_as_float((127 + e) << 23);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
          if constexpr (C8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = pack2<false>(unpack_lo<BF16>(x[k]) * f, unpack_hi<BF16>(x[k]) * f);
          }
          st_shared_v4(sQ + (uint32_t)(c >> 3) * kQChunk + (uint32_t)r * 128u +
                           (uint32_t)(((c & 7) ^ (r & 7)) << 4),
                       x[0], x[1], x[2], x[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(sBar + 8u * B::kQFull);
      }

      float M = -1e30f, L = 0.f;
      const uint64_t rs2 = f2(rs, rs);
      for (int j = 0; j < n; ++j, ++it) {
        const int n0 = d0.z + j * BN;
        const uint32_t s = it & 1u;
        // The scales were written by the loading warps: their own barriers
        // make them visible here.
        if (C8 && !(ok = wait_all(sBar + 8u * (B::kKFull + s), (it >> 1) & 1u))) break;
        if (C8 && !(ok = wait_all(sBar + 8u * (B::kVFull + s), (it >> 1) & 1u))) break;
        if (!(ok = wait_all(sBar + 8u * B::kSFull, it & 1u))) break;
        tc_fence_after();
        const bool edge = n0 + BN > P || p.window > 0 || !on;
        float alpha = 1.f;  // this tile's moves of the reference
#pragma unroll 1
        for (int c = 0; c < BN / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(t_lane + kColS + 32 * c, x);
          tmem_wait_ld();
          if (c == BN / 32 - 1) {
            tc_fence_before();
            mbar_arrive(sBar + 8u * B::kSFree);  // the next scores may come
          }
          uint64_t t2[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            t2[k] = f2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
          if constexpr (C8) {
            const ulonglong2* ks = reinterpret_cast<const ulonglong2*>(s_ks + s * BN + 32 * c);
            const ulonglong2* we = reinterpret_cast<const ulonglong2*>(s_we + s * BN + 32 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const ulonglong2 a = ks[k], b = we[k];
              t2[2 * k] = ffma2(fmul2(t2[2 * k], rs2), a.x, b.x);
              t2[2 * k + 1] = ffma2(fmul2(t2[2 * k + 1], rs2), a.y, b.y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) t2[k] = fmul2(t2[k], rs2);
          }
          if (edge) {  // keys this row keeps, one bit each
            const int x0 = n0 + 32 * c - P;  // first key's index among the new tokens
            uint32_t keep = 0u;
            if (on && x0 <= i) {
              keep = i - x0 >= 31 ? ~0u : (2u << (i - x0)) - 1u;
              if (p.mask != nullptr && x0 + 31 >= 0) {
                const int W = (E + 31) >> 5, w0 = x0 >> 5;  // floor
                const uint32_t* mw = p.mask + (long long)d2.y + (long long)i * W;
                const uint32_t lo = w0 >= 0 && w0 < W ? __ldg(mw + w0) : w0 < 0 ? ~0u : 0u;
                const uint32_t hi = w0 + 1 < W ? __ldg(mw + w0 + 1) : 0u;
                keep &= __funnelshift_r(lo, hi, x0 & 31);
              }
              if (p.window > 0) {
                if (p.depths == nullptr) {
                  const int gone = i - p.window + 1 - x0;  // keys below the window
                  if (gone > 0) keep = gone > 31 ? 0u : keep >> gone << gone;
                } else {
                  for (int k = 0; k < 32; ++k) {
                    if (!(keep >> k & 1u)) continue;
                    const int y = x0 + k, place = y >= 0 ? __ldg(p.depths + cu0 + y) : y;
                    if (place <= dep - p.window) keep &= ~(1u << k);
                  }
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float a, b;
              unf2(t2[k], a, b);
              t2[k] = f2(keep >> (2 * k) & 1u ? a : -INFINITY, keep >> (2 * k + 1) & 1u ? b : -INFINITY);
            }
          }
          float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            float a, b;
            unf2(t2[k], a, b), m0 = max3(m0, a, b);
            unf2(t2[k + 1], a, b), m1 = max3(m1, a, b);
            unf2(t2[k + 2], a, b), m2 = max3(m2, a, b);
            unf2(t2[k + 3], a, b), m3 = max3(m3, a, b);
          }
          const float mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
          const bool raise = mx > M + kCaSlack;
          if (c == 0 && it > 0) {  // P of the tile before has been read
            if (!(ok = wait_all(sBar + 8u * B::kODone, (it - 1u) & 1u))) break;
            tc_fence_after();
          }
          if (__any_sync(0xffffffffu, raise)) {  // rare after the first tiles
            const float a = raise ? ex2(M - mx) : 1.f;
            if (raise) M = mx;
            L *= a;
            alpha *= a;
            tmem_wait_st();
            for (int e = 0; e < c; ++e) {  // this tile's P so far
              uint32_t pk[16];
              tmem_ld16(t_lane + kColP + 16 * e, pk);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k)
                pk[k] = pack2<MBF>(unpack_lo<MBF>(pk[k]) * a, unpack_hi<MBF>(pk[k]) * a);
              tmem_st16(t_lane + kColP + 16 * e, pk);
              tmem_wait_st();
            }
          }
          const float ref = kBias - M;
          const uint64_t ref2 = f2(ref, ref);
          uint64_t l0 = 0, l1 = 0;
          uint32_t pk[16];
          const ulonglong2* wi = reinterpret_cast<const ulonglong2*>(s_wi + s * BN + 32 * c);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float a, b, e, f;
            unf2(fadd2(t2[k], ref2), a, b);
            unf2(fadd2(t2[k + 1], ref2), e, f);
            a = ex2(a), b = ex2(b), e = ex2(e), f = ex2(f);
            if constexpr (C8) {
              const ulonglong2 w = wi[k / 2];
              l0 = ffma2(f2(a, b), w.x, l0);
              l1 = ffma2(f2(e, f), w.y, l1);
            } else {
              l0 = fadd2(l0, f2(a, b));
              l1 = fadd2(l1, f2(e, f));
            }
            pk[k] = pack2<MBF>(a, b);
            pk[k + 1] = pack2<MBF>(e, f);
          }
          float a, b;
          unf2(fadd2(l0, l1), a, b);
          L += a + b;
          tmem_st16(t_lane + kColP + 16 * c, pk);
        }
        if (!ok) break;
        if (C8) {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(sBar + 8u * (B::kKEmpty + s));
            mbar_arrive(sBar + 8u * (B::kVEmpty + s));
          }
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {  // O so far, its products done
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(t_lane + kColO + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(t_lane + kColO + c * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(sBar + 8u * B::kPFull);
      }
      if (!ok) break;
      if (!(ok = wait_all(sBar + 8u * B::kODone, (it - 1u) & 1u))) break;
      tc_fence_after();
      // ---- the row: a partial, or the result
      if (cut) {
        const long long pr = (2ll * blockIdx.x + (d0.y >> 1)) * RT + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_lane + kColO + c * 32, o);
          tmem_wait_ld();
          if (on) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + pr * D + 32 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                   __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
          }
          __syncwarp();
        }
        if (on) *reinterpret_cast<float2*>(p.part_ml + pr * 2) = make_float2(M, L);
      } else {
        const bool any = L > 0.f;
        const float mm = fmaxf(M - kBias, sink), f = ex2(M - kBias - mm);
        const float den = fmaf(L, f, ex2(sink - mm));
        const float inv = any ? f / den : 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_lane + kColO + c * 32, o);
          tmem_wait_ld();
          if (on) {
            uint4* dst =
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + 32 * c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = pack2<BF16>(__uint_as_float(o[8 * k + 2 * e]) * inv,
                                   __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
              dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          __syncwarp();
        }
        if (on && p.lse != nullptr) p.lse[row] = any ? (mm + log2f(den)) * kLn2 : -INFINITY;
      }
    }
  }
  // The products are done (warp 7 drained them) and every row has been read.
  tc_fence_before();
  __syncthreads();
  if (warp == 7) {
    tc_fence_after();
    tmem_dealloc(tmem, 256u);
  }
}

}  // namespace gqa
