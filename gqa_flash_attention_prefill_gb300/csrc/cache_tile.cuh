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
//   4..6  bring K and V into the 128-byte swizzle the products read: 16-bit
//         pages by cp.async, e4m3 pages through registers, widened to f16, the
//         next tile's loads in flight meanwhile.  Keys no row sees become
//         zeros;
//   7     plans the work and issues the products.
//
// Scales of an e4m3 tile.  Widening multiplies a key's values by 2^(e - x)
// with x 7 below the largest exponent e of the tile, which keeps every value
// within f16 and exact where e lies at most 22 below the largest.  The tile's
// 2^x multiplies all its scores alike, and V's x joins the exponent of all its
// probabilities (and leaves the denominator) as w does in cache_attn.cuh.
// Below those 22 powers of two a K value rounds at 2^-33 of the tile's largest,
// less than the scores' own fp32; a V tile that spans more keeps its values
// unscaled and hands the softmax an exponent per key.  (Always a scale per key:
// the broadcast reads of three arrays took 1536 shared-memory clocks a tile of
// 128 keys, three times its products.)
#pragma once
#include "cache_attn.cuh"

namespace gqa {

constexpr int kCtThreads = 256;
constexpr int kCtLoaders = 96;
constexpr int kCtWholeSlack = 2;  // tiles a join is worth
__host__ __device__ constexpr int ct_bn(int D) { return D == 64 ? 128 : 64; }
// Q tile, two slots each of K and V, their scales, the tables of the sequences.
__host__ __device__ constexpr uint32_t ct_smem(int D) {
  return 1024u + 128u * D * 2u + 4u * ct_bn(D) * D * 2u + 2u * ct_bn(D) * 8u + 4u * 16u +
         4u * (5 * kMaxSeqs + 3) + kCaPieces * 64u + 32u * 8u + 64u;
}

struct CtBar {  // barrier numbers
  static constexpr int kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kSFree = 9,
                       kPFull = 10, kODone = 11, kQFull = 12, kDrain = 13, kPiece = 14;
};

// Keys x0 .. x0 + 31 (counted from the first new token) that row i of a
// sequence of E new tokens keeps, one bit each.
static __device__ __noinline__ uint32_t keep_bits(const CacheAttnParams& p, bool on, int i, int dep,
                                           int x0, int E, int cu0, long long mask0) {
  if (!on || x0 > i) return 0u;
  uint32_t keep = i - x0 >= 31 ? ~0u : (2u << (i - x0)) - 1u;
  if (p.mask != nullptr && x0 + 31 >= 0) {
    const int W = (E + 31) >> 5, w0 = x0 >> 5;  // floor
    const uint32_t* mw = p.mask + mask0 + (long long)i * W;
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
  return keep;
}

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
  // Exponents of a V tile that spans too many: w and 2^-w per key.
  float* s_we = reinterpret_cast<float*>(smem + kQBytes + 4u * kKVBytes);  // [2][BN]
  float* s_wi = s_we + 2 * BN;                                            // [2][BN]
  // Per tile, four deep: K's exponent x, V's, whether V's stand per key.
  int4* s_exp = reinterpret_cast<int4*>(s_wi + 2 * BN);
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_exp + 4);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 32);  // [0] abort [1] bad [2] most tiles
  int* s_red = reinterpret_cast<int*>(misc + 4);            // [3] tmem; the loaders' reductions
  int4* s_piece = reinterpret_cast<int4*>(misc + 16);
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
      // Free once the product is done.  What the softmax reads of a V slot it
      // has read before the product starts (P is full); s_exp is four deep:
      // entry t + 4 is written after the scores of t + 2, hence after t + 1 was
      // read.
      mbar_init(sBar + 8u * (B::kKEmpty + i), 1u);
      mbar_init(sBar + 8u * (B::kVEmpty + i), 1u);
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
    int row[kLoads];  // pool rows of the tile's keys, -1 for a key no row sees
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
    // 16-byte unit c of key row j goes to unit c ^ (j & 7) of its 128-byte row.
    auto unit_at = [&](uint32_t base, int j, int unit) {
      return base + (uint32_t)(unit >> 3) * kKVChunk + (uint32_t)j * 128u +
             (uint32_t)(((unit & 7) ^ (j & 7)) << 4);
    };
    auto slot_free = [&](uint32_t i, bool is_v) {
      return wait_all(sBar + 8u * ((is_v ? B::kVEmpty : B::kKEmpty) + (i & 1u)),
                      ((i >> 1) & 1u) ^ 1u);
    };
    // The next tile: the piece's, or the next piece's first.
    int left = 0, n0 = 0;
    auto next_tile = [&]() -> bool {
      if (left == 0) {
        if (!next_piece(pi++, d0, d1, d2, ok)) return false;
        left = d0.x;
        n0 = d0.z;
      } else {
        n0 += BN;
      }
      --left;
      places(n0);
      return true;
    };

    if constexpr (C8) {
      // The next half tile (K or V) is loaded, in registers of its own, while
      // this one is widened and stored.  One copy of the code serves both
      // kinds: the loops of all roles have to stay in the instruction cache
      // together.
      struct Half {
        uint4 raw[kLoads];
        uint32_t sc[kLoads];  // the keys' scale bytes, 0 for a key no row sees
      } cur, nxt;
      auto fetch = [&](Half& h, bool is_v) {
        const uint8_t* src = (is_v ? p.v_pages : p.k_pages) + (long long)d1.w * D + 16 * q;
        const uint8_t* scales = (is_v ? p.v_scales : p.k_scales) + d1.w;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          h.raw[i] = make_uint4(0u, 0u, 0u, 0u);
          h.sc[i] = 0u;
          if (row[i] >= 0) {
            h.raw[i] = __ldg(reinterpret_cast<const uint4*>(src + row[i] * tok_bytes));
            h.sc[i] = __ldg(scales + (long long)row[i] * p.Hkv);
          }
        }
      };
      // Largest and smallest scale byte of the tile's keys, over the three
      // warps: each puts its own into one of two sets of words in turn.
      uint32_t turn = 0;
      auto span = [&](const Half& h, int& top, int& low) {
        int hi = 0, lo = 255;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          hi = max(hi, (int)h.sc[i]);
          if (h.sc[i] != 0u) lo = min(lo, (int)h.sc[i]);
        }
        hi = __reduce_max_sync(0xffffffffu, hi);
        lo = __reduce_min_sync(0xffffffffu, lo);
        int* red = s_red + 6 * (turn++ & 1u);
        if (lane == 0) {
          red[2 * (warp - 4)] = hi;
          red[2 * (warp - 4) + 1] = lo;
        }
        named_bar_sync(1u, kCtLoaders);
        top = max(max(red[0], red[2]), red[4]);
        low = min(min(red[1], red[3]), red[5]);
      };
      auto store = [&](const Half& h, bool is_v) {
        const uint32_t s = it & 1u;
        const uint32_t base = (is_v ? sV : sK) + s * kKVBytes;
        int top, low;
        span(h, top, low);
        const bool apart = is_v && top - low > 22;  // exponents per key
        const int x = apart ? 0 : max(top, 8) - 127 - 7;  // the tile's exponent, >= -126
        if (lt == 0) {
          if (is_v) {
            s_exp[it & 3u].y = x;
            s_exp[it & 3u].z = apart ? 1 : 0;
          } else {
            s_exp[it & 3u].x = x;
          }
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int j = j0 + i * kStep;
          if (BN % kStep != 0 && j >= BN) break;
          uint32_t y[8];
          e4m3x4_f16(h.raw[i].x, y[0], y[1]);
          e4m3x4_f16(h.raw[i].y, y[2], y[3]);
          e4m3x4_f16(h.raw[i].z, y[4], y[5]);
          e4m3x4_f16(h.raw[i].w, y[6], y[7]);
          // 2^(e - x) as an f16 pair: at most 2^7, zero below 2^-24.
          const int e = apart ? 0 : max((int)h.sc[i] - 127 - x, -40);
          const float f = __int_as_float((127 + e) << 23);
          const uint32_t f2h = pack2<false>(f, f);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[k]) : "r"(y[k]), "r"(f2h));
          st_shared_v4(unit_at(base, j, 2 * q), y[0], y[1], y[2], y[3]);
          st_shared_v4(unit_at(base, j, 2 * q + 1), y[4], y[5], y[6], y[7]);
          if (apart && q == 0) {
            s_we[s * BN + j] = h.sc[i] ? (float)((int)h.sc[i] - 127) : 0.f;
            s_wi[s * BN + j] = __uint_as_float((254u - h.sc[i]) << 23);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(sBar + 8u * ((is_v ? B::kVFull : B::kKFull) + s));
      };
      bool have = next_tile(), v_next = false;
#pragma unroll 1
      for (bool first = true;; first = false) {
        const bool v_now = !v_next;  // of the half in `nxt` until now
        if (!first) cur = nxt;
        if (have) fetch(nxt, v_next);
        if (!first) {
          if (!slot_free(it, v_now)) break;
          store(cur, v_now);
          if (v_now) ++it;
        }
        if (!have) break;
        if (v_next) have = next_tile();
        v_next = !v_next;
      }
    } else {
      // Straight to shared memory; two halves (K or V) stay in flight.
      auto issue = [&](uint32_t i2, bool is_v) {
        const uint8_t* src =
            (is_v ? p.v_pages : p.k_pages) + (long long)d1.w * (D * kEsz) + 16 * q;
        const uint32_t base = (is_v ? sV : sK) + (i2 & 1u) * kKVBytes;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int j = j0 + i * kStep;
          if (BN % kStep != 0 && j >= BN) break;
          const uint8_t* g = src + (row[i] >= 0 ? row[i] : 0) * tok_bytes;
          // Source size 0 fills with zeros.
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(unit_at(base, j, q)),
                       "l"(g), "r"(row[i] >= 0 ? 16u : 0u)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // Half h (2 t: K of tile t, 2 t + 1: V) has landed.
      auto landed = [&](uint32_t h) {
        fence_proxy_async_smem();
        mbar_arrive(sBar + 8u * (((h & 1u) ? B::kVFull : B::kKFull) + ((h >> 1) & 1u)));
      };
      uint32_t h = 0;  // halves issued
      while (next_tile()) {
        if (!slot_free(it, false)) break;
        issue(it, false);
        if (++h > 2u) {
          asm volatile("cp.async.wait_group 2;" ::: "memory");
          landed(h - 3u);
        }
        if (!slot_free(it, true)) break;
        issue(it, true);
        if (++h > 2u) {
          asm volatile("cp.async.wait_group 2;" ::: "memory");
          landed(h - 3u);
        }
        ++it;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      for (uint32_t x = h > 2u ? h - 2u : 0u; x < h; ++x) landed(x);
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
      for (int j = 0; j < n; ++j, ++it) {
        const int n0 = d0.z + j * BN;
        const uint32_t s = it & 1u;
        // This tile's factor of the scores, and V's exponent.
        float rk = rs, ve = 0.f, vi = 1.f;
        bool apart = false;
        if constexpr (C8) {
          // The loaders' writes are visible after their own barriers.
          if (!(ok = wait_all(sBar + 8u * (B::kKFull + s), (it >> 1) & 1u))) break;
          if (!(ok = wait_all(sBar + 8u * (B::kVFull + s), (it >> 1) & 1u))) break;
          const int4 x = s_exp[it & 3u];
          rk = fmaxf(rs * __int_as_float((127 + x.x) << 23), 1e-37f);
          ve = (float)x.y;
          vi = __int_as_float((127 - x.y) << 23);
          apart = x.z != 0;
        }
        if (!(ok = wait_all(sBar + 8u * B::kSFull, it & 1u))) break;
        tc_fence_after();
        const bool edge = n0 + BN > P || p.window > 0 || !on;
        float alpha = 1.f, sum = 0.f;  // this tile's moves of the reference, its sum of P
        // Rolled: the unrolled loop and the loaders' did not fit the
        // instruction cache together (half the stalls).
#pragma unroll 1
        for (int c = 0; c < BN / 32; ++c) {
          uint32_t sr[32];
          float mx = tmem_ld32_max(t_lane + kColS + 32 * c, sr);
          tmem_wait_ld();
          if (c == BN / 32 - 1) {
            tc_fence_before();
            mbar_arrive(sBar + 8u * B::kSFree);  // the next tile's scores may come
          }
          if (__builtin_expect(edge || apart, 0)) {
            if (edge) {  // keys this row keeps, one bit each
              const uint32_t keep =
                  keep_bits(p, on, i, dep, n0 + 32 * c - P, E, cu0, (long long)d2.y);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(keep >> k & 1u)) sr[k] = 0xFF800000u;  // -inf
            }
            mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float a = __uint_as_float(sr[k]), b = __uint_as_float(sr[k + 1]);
              if (apart) {  // the whole exponent here, a key's own part of it included
                a = fmaf(a, rk, s_we[s * BN + 32 * c + k]);
                b = fmaf(b, rk, s_we[s * BN + 32 * c + k + 1]);
                sr[k] = __float_as_uint(a), sr[k + 1] = __float_as_uint(b);
              }
              mx = max3(mx, a, b);
            }
          }
          const float rc = apart ? 1.f : rk;
          mx = fmaf(mx, rc, ve);  // ve is 0 with exponents per key
          if (c == 0 && it > 0) {  // P of the tile before has been read
            if (!(ok = wait_all(sBar + 8u * B::kODone, (it - 1u) & 1u))) break;
            tc_fence_after();
          }
          const bool raise = mx > M + kCaSlack;
          if (__any_sync(0xffffffffu, raise)) {  // rare after the first tiles
            const float a = raise ? ex2(M - mx) : 1.f;
            if (raise) M = mx;
            L *= a;
            sum *= a;
            alpha *= a;
            tmem_wait_st();
#pragma unroll 1
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
          const float ref = ve - M + kBias;
          const uint64_t ref2 = f2(ref, ref), rk2 = f2(rc, rc);
          uint64_t l0 = 0, l1 = 0;
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float a, b, e, f;
            unf2(ffma2(f2(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1])), rk2, ref2), a, b);
            unf2(ffma2(f2(__uint_as_float(sr[2 * k + 2]), __uint_as_float(sr[2 * k + 3])), rk2, ref2), e, f);
            a = ex2(a), b = ex2(b), e = ex2(e), f = ex2(f);
            pk[k] = pack2<MBF>(a, b);
            pk[k + 1] = pack2<MBF>(e, f);
            if (C8 && __builtin_expect(apart, 0)) {
              const float* w = s_wi + s * BN + 32 * c + 2 * k;
              a *= w[0], b *= w[1], e *= w[2], f *= w[3];
            }
            l0 = fadd2(l0, f2(a, b));
            l1 = fadd2(l1, f2(e, f));
          }
          float a, b;
          unf2(fadd2(l0, l1), a, b);
          sum += a + b;
          tmem_st16(t_lane + kColP + 16 * c, pk);
        }
        if (!ok) break;
        L = fmaf(sum, vi, L);
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
