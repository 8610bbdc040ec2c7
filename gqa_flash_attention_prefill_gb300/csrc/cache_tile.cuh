// cache_tile.cuh -- the form of gqa_cache_attention for many query rows per KV
// head (a draft tree of some tens of tokens, a short chunk): two 128-row tiles
// on the tensor memory, sm_103a.
//
// The mathematics is cache_attn.cuh's; here the rows fill 128-row tiles, so the
// products go to tcgen05 and the bound moves from memory to the softmax and,
// for e4m3, to widening the keys.  A unit is 256 rows of one KV head, so a key
// is widened once for two row tiles.
//
// A CTA of 14 warps, one per SM:
//   0..7   softmax and output: warps 0..3 row tile 0, 4..7 row tile 1, thread =
//          row = tensor-memory lane; they also bring their rows of Q into
//          shared memory.  A second tile without rows takes no part;
//   8..11  bring K (two warps) and V (two) into the 128-byte swizzle the
//          products read, each warp half of a tile's keys on its own.  16-bit
//          pages: cp.async.  e4m3 pages: cp.async of the raw bytes some tiles
//          ahead, then each thread widens what it copied itself to f16.  Keys
//          no row sees become zeros;
//   12, 13 issue the products, a warp per row tile; 12 plans the work as well.
// A round of barriers around the products costs an issuing warp about as much
// as 64 keys of softmax (one warp for both tiles, 64-key tiles with double-
// buffered scores: 8 trees of 64 tokens over 8k e4m3 keys 176 us, 146 of them
// with softmax and widening left out), so a tile takes as many keys as the
// tensor memory holds beside P and O, and the two row tiles do not wait for
// each other: 156 us, 440 TFLOP/s.  A tile takes 4300 clocks: 2500 of softmax
// work, the rest its waits for exponents, scores and the product before, each
// some hundreds although the slots are rarely full.
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

constexpr int kCtLoaders = 128;
constexpr int kCtThreads = 256 + kCtLoaders + 64;
constexpr int kCtWholeSlack = 2;  // tiles a join is worth
__host__ __device__ constexpr int ct_bn(int D) { return D == 64 ? 128 : 64; }  // keys per tile
// Slots of K and of V ready for the products; raw e4m3 tiles on their way.
__host__ __device__ constexpr int ct_slots(bool C8) { return C8 ? 2 : 4; }
constexpr int kCtRaw = 4;
// A raw half tile (K or V): the values, and for each of its two warps 8 bytes a
// key for the scales.
__host__ __device__ constexpr uint32_t ct_raw_half(int D) { return (uint32_t)ct_bn(D) * (D + 16u); }
__host__ __device__ constexpr uint32_t ct_smem(int D, bool C8) {
  return 1024u + 2u * 128u * D * 2u + 2u * ct_slots(C8) * ct_bn(D) * D * 2u +
         (C8 ? 2u * kCtRaw * ct_raw_half(D) + 2u * ct_slots(C8) * ct_bn(D) * 4u : 0u) + 8u * 16u +
         64u * 8u + 128u + kCaPieces * 64u + 4u * (5 * kMaxSeqs + 3);
}

struct CtBar {  // barrier numbers: 4 for the slots, 2 for the row tiles
  static constexpr int kKFull = 0, kKEmpty = 4, kVFull = 8, kVEmpty = 12, kSFull = 16, kSFree = 18,
                       kPFull = 20, kODone = 22, kQFull = 24, kDrain = 26, kPiece = 28,
                       kExp = kPiece + 2 * kCaPieces;  // 8, one an entry of s_exp
  static_assert(kExp + 8 <= 64, "barriers");
};

// Keys x0 .. x0 + 31 (counted from the first new token) that row i of a
// sequence of E new tokens keeps, one bit each.
__device__ __forceinline__ uint32_t keep_bits(const CacheAttnParams& p, bool on, int i, int dep,
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

// New tokens x0 + 32 g, g < groups, that none of the tokens first .. last of a
// sequence of E new ones sees by the bitmap and the window, a bit each.  A
// token itself, which sees it as a rule, is looked at first.  Not inlined: in
// the loading warps' loop it cost 14 us of 161 whether it ran or not, called 3.
inline __device__ __noinline__ uint32_t ct_hidden(const uint32_t* mask, const int32_t* depths, int E,
                                                  int window, int first, int last, int x0,
                                                  int groups) {
  uint32_t hid = 0;
#pragma unroll 1
  for (int g = 0; g < groups; ++g) {
    const int x = x0 + 32 * g;
    if (x < 0 || x > last) continue;
    const int place = depths != nullptr ? __ldg(depths + x) : x;
    bool seen = false;
#pragma unroll 1
    for (int i = max(x, first); i <= last && !seen; ++i) {
      seen = mask == nullptr ||
             (__ldg(mask + (long long)i * ((E + 31) >> 5) + (x >> 5)) >> (x & 31) & 1u);
      if (seen && window > 0) seen = place > (depths != nullptr ? __ldg(depths + i) : i) - window;
    }
    if (!seen) hid |= 1u << g;
  }
  return hid;
}

// Products and commits as the one elected thread of a warp issues them, all
// under one election (one an instruction: 164.7 -> 158.6 us).
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, e;\n\t}"
      : "=r"(r)::"memory");
  return r != 0;
}
__device__ __forceinline__ void one_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void one_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void one_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

template <int D, bool BF16, bool C8>
__global__ void __launch_bounds__(kCtThreads, 1)
    cache_tile_kernel(const __grid_constant__ CacheAttnParams p) {
  constexpr int BN = ct_bn(D), RT = 256, NS = ct_slots(C8);
  constexpr bool MBF = BF16 && !C8;  // product type
  constexpr float kBias = MBF ? 0.f : kCaBias;
  constexpr int kEsz = C8 ? 1 : 2;
  constexpr uint32_t kQBytes = 128u * D * 2u, kKVBytes = (uint32_t)BN * D * 2u;
  constexpr uint32_t kQChunk = 128u * 128u, kKVChunk = (uint32_t)BN * 128u;
  constexpr uint32_t kColP = BN, kColO = BN + BN / 2;  // scores at column 0
  static_assert(kColO + D <= 256, "two row tiles share the tensor memory");
  constexpr uint32_t kIdescS = idesc_f16(MBF, 128, BN, false);
  constexpr uint32_t kIdescO = idesc_f16(MBF, 128, D, true);
  using B = CtBar;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_u32(smem), sK = sQ + 2u * kQBytes, sV = sK + NS * kKVBytes;
  const uint32_t sRaw = sV + NS * kKVBytes;  // [kCtRaw][K, V][values, scales]
  uint8_t* after = smem + 2u * kQBytes + 2u * NS * kKVBytes +
                   (C8 ? 2u * kCtRaw * ct_raw_half(D) : 0u);
  // Exponents of a V tile that spans too many: w and 2^-w per key.
  float* s_we = reinterpret_cast<float*>(after);  // [NS][BN]
  float* s_wi = s_we + (C8 ? NS * BN : 0);
  // Per tile, eight deep: K's exponent x, V's, whether V's stand per key.
  int4* s_exp = reinterpret_cast<int4*>(s_wi + (C8 ? NS * BN : 0));
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_exp + 8);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 64);  // [0] abort [1] bad [2] most tiles [3] tmem
  int4* s_piece = reinterpret_cast<int4*>(misc + 32);
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
    // A slot is free once both row tiles' products are done.  What the softmax
    // reads of a V slot it has read before those products start (P is full);
    // s_exp is eight deep: entry t + 8 is written after slot t + 7's turn, when
    // the scores of t + 7 - NS are done, which were issued after the softmax of
    // t + 6 - NS had read its entry.
    for (int i = 0; i < NS; ++i) {
      mbar_init(sBar + 8u * (B::kKFull + i), 2u);
      mbar_init(sBar + 8u * (B::kVFull + i), 2u);
      mbar_init(sBar + 8u * (B::kKEmpty + i), 2u);
      mbar_init(sBar + 8u * (B::kVEmpty + i), 2u);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sBar + 8u * (B::kSFull + i), 1u);
      mbar_init(sBar + 8u * (B::kSFree + i), 4u);
      mbar_init(sBar + 8u * (B::kPFull + i), 4u);
      mbar_init(sBar + 8u * (B::kODone + i), 1u);
      mbar_init(sBar + 8u * (B::kQFull + i), 4u);
      mbar_init(sBar + 8u * (B::kDrain + i), 1u);
    }
    for (int i = 0; i < 8; ++i) mbar_init(sBar + 8u * (B::kExp + i), 2u);
    for (int i = 0; i < kCaPieces; ++i) {
      mbar_init(sPiece + 8u * i, 1u);
      mbar_init(sPiece + 8u * (kCaPieces + i), 13u);  // 8 softmax, 4 loading, 1 issuing
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
      if (blockIdx.x == 0) p.head[0] = 0;
    }
    return;
  }
  if (tid == 0) ca_mark(p, 0);
  if (warp == 12) {
    tmem_alloc(smem_u32(misc + 3), 512u);
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
  // One arrival for a warp whose lanes are all done (32 arrivals: 158.6 us, one:
  // 155.7).
  auto warp_arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
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

  if (warp >= 12) {
    // -------------------------------------------------------------- plan, products
    const int t = warp - 12;  // row tile
    const uint64_t dQ = smem_desc_sw128(sQ + t * kQBytes, 16, 1024);
    const uint64_t dK0 = smem_desc_sw128(sK, 16, 1024);
    const uint64_t dV0 = smem_desc_sw128(sV, kKVChunk, 1024);
    const uint32_t tb = tmem + 256u * t;
    auto kstep = [](int kk, uint32_t chunk) -> uint64_t {
      return (uint64_t)(((uint32_t)(kk >> 2) * chunk + (uint32_t)(kk & 3) * 32u) >> 4);
    };
    uint32_t it = 0, c = 0, pieces = 0;  // tiles of the CTA, of the row tile; its pieces
    // O += P V of the tile before tile i2 of the CTA, c2 of the row tile.
    auto issue_pv = [&](uint32_t i2, uint32_t c2, bool first) -> bool {
      const uint32_t s = (i2 - 1u) % NS;
      if (!wait_all(sBar + 8u * (B::kVFull + s), ((i2 - 1u) / NS) & 1u)) return false;
      if (!wait_all(sBar + 8u * (B::kPFull + t), (c2 - 1u) & 1u)) return false;
      tc_fence_after();
      const uint64_t dv = dV0 + s * (kKVBytes >> 4);
      if (elected()) {
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          one_mma_ts(tb + kColO, tb + kColP + kk * 8, dv + (uint64_t)(kk * 128), kIdescO,
                     (first && kk == 0) ? 0u : 1u);
        one_commit(sBar + 8u * (B::kODone + t));
        one_commit(sBar + 8u * (B::kVEmpty + s));
      }
      __syncwarp();
      return true;
    };
    CaPlan plan = {};
    if (t == 0) plan = ca_plan(p, tiles, units, s_cu, s_pre, s_ipt, misc);
    // The other warps hear of up to seven pieces beyond the one at work, more
    // than the five tiles (of a piece each, at the least) that the loading
    // warps look ahead: they never wait for a piece that waits for them.
    uint32_t told = 0;
    bool more = true, ok = true;
    for (uint32_t pc = 0; ok; ++pc) {
      int4 d0, d1, d2;
      if (t == 0) {
        while (more && told < pc + kCaPieces) {
          CaPiece u = {};
          more = ca_next(p, plan.T, plan.walk, RT, u);
          const uint32_t ps = told % kCaPieces;
          if (!(ok = wait_all(sPiece + 8u * (kCaPieces + ps), ((told / kCaPieces) & 1u) ^ 1u)))
            break;
          if (lane == 0) {
            ca_publish(p, plan, u, more, RT, s_piece + 4 * ps);
            mbar_arrive(sPiece + 8u * ps);
          }
          ++told;
          __syncwarp();
        }
        if (!ok) break;
        d0 = s_piece[4 * (pc % kCaPieces)];
        d1 = s_piece[4 * (pc % kCaPieces) + 1];
        if (d0.x == 0) break;
      } else if (!next_piece(pc, d0, d1, d2, ok)) {
        break;
      }
      const int n = d0.x;
      if (d1.z + 128 * t >= d1.x * p.G) {  // no rows in this tile: its share of the slots
        for (int j = 0; j < n; ++j, ++it) {
          const uint32_t s = it % NS;
          if (!(ok = wait_all(sBar + 8u * (B::kKFull + s), (it / NS) & 1u))) break;
          if (lane == 0) mbar_arrive(sBar + 8u * (B::kKEmpty + s));
          if (!(ok = wait_all(sBar + 8u * (B::kVFull + s), (it / NS) & 1u))) break;
          if (lane == 0) mbar_arrive(sBar + 8u * (B::kVEmpty + s));
        }
        continue;
      }
      if (!(ok = wait_all(sBar + 8u * (B::kQFull + t), pieces & 1u))) break;
      ++pieces;
      for (int j = 0; j < n; ++j, ++it, ++c) {
        const uint32_t s = it % NS;
        if (!(ok = wait_all(sBar + 8u * (B::kKFull + s), (it / NS) & 1u))) break;
        if (c > 0 && !(ok = wait_all(sBar + 8u * (B::kSFree + t), (c - 1u) & 1u))) break;
        tc_fence_after();
        const uint64_t dk = dK0 + s * (kKVBytes >> 4);
        if (elected()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            one_mma_ss(tb, dQ + kstep(kk, kQChunk), dk + kstep(kk, kKVChunk), kIdescS,
                       kk > 0 ? 1u : 0u);
          one_commit(sBar + 8u * (B::kSFull + t));
          one_commit(sBar + 8u * (B::kKEmpty + s));
        }
        __syncwarp();
        // The second product of a tile goes after the next tile's first.
        if (j > 0 && !(ok = issue_pv(it, c, j == 1))) break;
      }
      if (ok) ok = issue_pv(it, c, n == 1);
    }
    mma_commit(sBar + 8u * (B::kDrain + t));  // completes when every product issued is done
    wait_drain(sBar + 8u * (B::kDrain + t), 0u, tmo);
    __syncwarp();
  } else if (warp >= 8) {
    // -------------------------------------------------------------- K and V
    constexpr int kCpr = D * kEsz / 16;  // 16-byte pieces of a key, and pieces of a lane
    constexpr int kStep = 32 / kCpr;     // keys a round of the warp's lanes
    const bool is_v = warp >= 10;
    constexpr int kOwn = BN / 64;        // 32-key groups of a warp, the tile's half
    const int half = warp & 1;           // keys BN / 2 * half .. of a tile
    const int q = lane % kCpr, k0 = lane / kCpr;  // the lane's place in a key, its first key
    const long long tok_bytes = (long long)p.Hkv * D * kEsz;
    const uint8_t* const pages = is_v ? p.v_pages : p.k_pages;
    const uint8_t* const scales = is_v ? p.v_scales : p.k_scales;
    const uint32_t sT = is_v ? sV : sK;
    const uint32_t full = sBar + 8u * (is_v ? B::kVFull : B::kKFull);
    const uint32_t empty = sBar + 8u * (is_v ? B::kVEmpty : B::kKEmpty);
    int4 d0 = {}, d1 = {}, d2 = {};
    uint32_t pi = 0, it = 0;
    bool ok = true;
    int left = 0, n0 = 0;
    int row[BN / 32];  // pool rows of the tile's keys lane, lane + 32, .., -1: no row sees it
    auto place = [&](int key) -> int {
      if (key >= d1.y || (p.window > 0 && key <= d0.w - p.window)) return -1;
      const int kp = p.div_page.div(key);
      int pg = __ldg(p.indices + d2.z + kp);
      if ((unsigned)pg >= (unsigned)p.num_pages) {
        atomicOr(p.status, 2u);  // GQA_DEV_BAD_METADATA
        pg = 0;
      }
      return pg * p.page_size + (key - kp * p.page_size);  // the pool has < 2^31 rows
    };
    // The next tile (the piece's, or the next piece's first) and its rows,
    // whose lookups are under way while the tile before is handled.
    auto next_tile = [&]() -> bool {
      if (left == 0) {
        if (!next_piece(pi++, d0, d1, d2, ok)) return false;
        left = d0.x;
        n0 = d0.z;
      } else {
        n0 += BN;
      }
      --left;
#pragma unroll
      for (int g = 0; g < BN / 32; ++g) row[g] = place(n0 + 32 * g + lane);
      if (n0 + BN > d0.w && (p.mask != nullptr || (p.depths != nullptr && p.window > 0))) {
        const int first = p.div_g.div(d1.z), last = min(p.div_g.div(d1.z + RT - 1), d1.x - 1);
        const uint32_t hid = ct_hidden(p.mask != nullptr ? p.mask + (long long)d2.y : nullptr,
                                       p.depths != nullptr ? p.depths + d2.x : nullptr, d1.x,
                                       p.window, first, last, n0 - d0.w + lane, BN / 32);
#pragma unroll
        for (int g = 0; g < BN / 32; ++g)
          if (hid >> g & 1u) row[g] = -1;
      }
      return true;
    };
    // 16-byte unit c of key row j goes to unit c ^ (j & 7) of its 128-byte row.
    auto unit_at = [&](uint32_t base, int j, int unit) {
      return base + (uint32_t)(unit >> 3) * kKVChunk + (uint32_t)j * 128u +
             (uint32_t)(((unit & 7) ^ (j & 7)) << 4);
    };
    // Asynchronous copies; a source size of 0 fills with zeros.
    auto copy16 = [](uint32_t dst, const uint8_t* src, bool live) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                   "r"(live ? 16u : 0u)
                   : "memory");
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    auto slot_free = [&](uint32_t i) { return wait_all(empty + 8u * (i % NS), ((i / NS) & 1u) ^ 1u); };

    bool more = next_tile();
    if constexpr (C8) {
      // Raw tile i to ring place i % kCtRaw: the lane's own pieces, and the
      // aligned word around the scale byte of every key of the tile, with the
      // byte's shift within it.
      uint32_t issued = 0;
      const uint32_t ring = sRaw + (is_v ? ct_raw_half(D) : 0u);
      const uint32_t words = (uint32_t)(BN * D + 8 * (BN * half + lane));  // of this warp
      auto issue = [&]() {
        const uint32_t at = ring + issued % kCtRaw * (2u * ct_raw_half(D));
#pragma unroll
        for (int g = 0; g < kOwn; ++g) {
          const int own = half ? row[kOwn + g] : row[g];
#pragma unroll
          for (int i = 0; i < kCpr; ++i) {
            const int k = k0 + i * kStep, r = __shfl_sync(0xffffffffu, own, k);
            const long long off = (long long)max(r, 0) * tok_bytes + d1.w * D + 16 * q;
            copy16(at + (uint32_t)((BN / 2 * half + 32 * g + k) * D + 16 * q), pages + off, r >= 0);
          }
        }
#pragma unroll
        for (int g = 0; g < BN / 32; ++g) {
          const long long so = (long long)max(row[g], 0) * p.Hkv + d1.w;
          const uint32_t sa = at + words + 256u * g;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sa),
                       "l"(scales + (so & ~3ll)), "r"(row[g] >= 0 ? 4u : 0u)
                       : "memory");
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(sa + 4u), "r"(8u * (uint32_t)(so & 3))
                       : "memory");
        }
        ++issued;
        more = next_tile();
      };
      // kCtRaw - 1 tiles ahead; every turn commits a group, empty at the end.
#pragma unroll 1
      for (int i = 0; i < kCtRaw - 1; ++i) {
        if (more) issue();
        commit();
      }
#pragma unroll 1
      for (; ok; ++it) {
        if (more) issue();
        commit();
        if (it >= issued) break;  // no tile left
        asm volatile("cp.async.wait_group %0;" ::"n"(kCtRaw - 1) : "memory");
        const uint32_t at = ring + it % kCtRaw * (2u * ct_raw_half(D));
        // Scale bytes of keys lane, lane + 32, .., 0 for a key no row sees.
        int sc[BN / 32], top = 0, low = 255;
#pragma unroll
        for (int g = 0; g < BN / 32; ++g) {
          const uint2 w = lds64(at + words + 256u * g);
          sc[g] = (int)((w.x >> w.y) & 255u);
          top = max(top, sc[g]);
          if (sc[g] != 0) low = min(low, sc[g]);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        low = __reduce_min_sync(0xffffffffu, low);
        const bool apart = is_v && top - low > 22;        // exponents per key
        const int x = apart ? 0 : max(top, (int)kCaLeast + 7) - 127 - 7;  // the tile's exponent
        if (half == 0 && lane == 0) {
          if (is_v) {
            s_exp[it & 7u].y = x;
            s_exp[it & 7u].z = apart ? 1 : 0;
          } else {
            s_exp[it & 7u].x = x;
          }
          mbar_arrive(sBar + 8u * (B::kExp + (it & 7u)));
        }
        if (!(ok = slot_free(it))) break;
        const uint32_t s = it % NS, base = sT + s * kKVBytes;
#pragma unroll 1
        for (int g = 0; g < kOwn; ++g) {
          const int own = half * kOwn + g == 0   ? sc[0]
                          : half * kOwn + g == 1 ? sc[1]
                          : half * kOwn + g == 2 ? sc[BN / 32 - 2] : sc[BN / 32 - 1];
          // 2^(e - x) as an f16 pair: at most 2^7, zero below 2^-24.
          const int e = apart ? 0 : max(own - 127 - x, -40);
          const float f = __int_as_float((127 + e) << 23);
          const uint32_t f2h = pack2<false>(f, f);
          const int j0 = BN / 2 * half + 32 * g;
          if (__builtin_expect(apart, 0)) {
            const int w = max(own, (int)kCaLeast);
            s_we[s * BN + j0 + lane] = (float)(w - 127);
            s_wi[s * BN + j0 + lane] = __uint_as_float((uint32_t)(254 - w) << 23);
          }
#pragma unroll
          for (int i = 0; i < kCpr; ++i) {
            const int k = k0 + i * kStep, j = j0 + k;
            const uint4 raw = lds128(at + (uint32_t)(j * D + 16 * q));
            const uint32_t m = __shfl_sync(0xffffffffu, f2h, k);
            uint32_t y[8];
            e4m3x4_f16(raw.x, y[0], y[1]);
            e4m3x4_f16(raw.y, y[2], y[3]);
            e4m3x4_f16(raw.z, y[4], y[5]);
            e4m3x4_f16(raw.w, y[6], y[7]);
#pragma unroll
            for (int n = 0; n < 8; ++n)
              asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[n]) : "r"(y[n]), "r"(m));
            st_shared_v4(unit_at(base, j, 2 * q), y[0], y[1], y[2], y[3]);
            st_shared_v4(unit_at(base, j, 2 * q + 1), y[4], y[5], y[6], y[7]);
          }
        }
        fence_proxy_async_smem();
        warp_arrive(full + 8u * s);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
      // Straight to the products' slots; two tiles stay in flight.
      auto landed = [&](uint32_t i) {
        fence_proxy_async_smem();
        warp_arrive(full + 8u * (i % NS));
      };
      while (more) {
        if (!slot_free(it)) break;
        const uint32_t base = sT + it % NS * kKVBytes;
#pragma unroll
        for (int g = 0; g < kOwn; ++g) {
          const int own = half ? row[kOwn + g] : row[g];
#pragma unroll
          for (int i = 0; i < kCpr; ++i) {
            const int k = k0 + i * kStep, r = __shfl_sync(0xffffffffu, own, k);
            const long long off =
                (long long)max(r, 0) * tok_bytes + (long long)d1.w * (D * kEsz) + 16 * q;
            copy16(unit_at(base, BN / 2 * half + 32 * g + k, q), pages + off, r >= 0);
          }
        }
        commit();
        if (++it > 2u) {
          asm volatile("cp.async.wait_group 2;" ::: "memory");
          landed(it - 3u);
        }
        more = next_tile();
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      for (uint32_t i = it > 2u ? it - 2u : 0u; i < it; ++i) landed(i);
    }
  } else {
    // -------------------------------------------------------------- softmax, output
    const int t = warp >> 2;    // row tile
    const int r = tid & 127;    // its row, lane of the tensor memory
    const uint32_t t_lane = tmem + 256u * t + ((uint32_t)((warp & 3) * 32) << 16);
    int4 d0 = {}, d1 = {}, d2 = {};
    uint32_t pi = 0, it = 0, c = 0;  // tiles of the CTA, and of this row tile
    bool ok = true;
    while (next_piece(pi++, d0, d1, d2, ok)) {
      const int n = d0.x, P = d0.w, E = d1.x, head = d1.w, cu0 = d2.x;
      const bool cut = (d0.y & 1) != 0;
      if (d1.z + 128 * t >= E * p.G) {  // no rows in this tile
        it += n;
        continue;
      }
      const int gr = d1.z + 128 * t + r;  // row of the sequence
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
        for (int k8 = 0; k8 < D / 8; ++k8) w[k8] = on ? __ldg(q + k8) : make_uint4(0u, 0u, 0u, 0u);
        float f = 1.f;
        if constexpr (C8) {
          // f16 operands: the row scaled by the power of two that brings its
          // largest magnitude into [1, 2); smaller values round at 2^-25.
          float amax = 0.f;
#pragma unroll
          for (int k8 = 0; k8 < D / 8; ++k8) {
            const uint32_t x[4] = {w[k8].x, w[k8].y, w[k8].z, w[k8].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = max3(amax, fabsf(unpack_lo<BF16>(x[k])), fabsf(unpack_hi<BF16>(x[k])));
          }
          const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126);
          f = __int_as_float((127 - e) << 23);
          rs *= __int_as_float((127 + e) << 23);
        }
#pragma unroll
        for (int k8 = 0; k8 < D / 8; ++k8) {
          uint32_t x[4] = {w[k8].x, w[k8].y, w[k8].z, w[k8].w};
          if constexpr (C8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = pack2<false>(unpack_lo<BF16>(x[k]) * f, unpack_hi<BF16>(x[k]) * f);
          }
          st_shared_v4(sQ + t * kQBytes + (uint32_t)(k8 >> 3) * kQChunk + (uint32_t)r * 128u +
                           (uint32_t)(((k8 & 7) ^ (r & 7)) << 4),
                       x[0], x[1], x[2], x[3]);
        }
        fence_proxy_async_smem();
        warp_arrive(sBar + 8u * (B::kQFull + t));
      }

      float M = -1e30f, L = 0.f;
      for (int j = 0; j < n; ++j, ++it, ++c) {
        const int n0 = d0.z + j * BN;
        const uint32_t s = it % NS;
        // The scores come first.  The barriers of the exponents and of V's slots
        // tell a phase only from the one before it, and a row tile that had no
        // rows in the tiles before waited for nothing there: it may be any
        // number of phases ahead of the loading warps.  The scores are counted
        // by the row tile's own tiles, and once they are here every entry and
        // slot of an earlier tile has been told.  (Exponents first, scores first
        // only after such tiles: 160 us where this order takes 157, for the code
        // it adds to the loop.)
        if (!(ok = wait_all(sBar + 8u * (B::kSFull + t), c & 1u))) break;
        // This tile's factor of the scores, and V's exponent.
        float rk = rs, ve = 0.f, vi = 1.f;
        bool apart = false;
        if constexpr (C8) {
          // The exponents are told before the values are widened.  K's slot may
          // be two tiles further on by now, so they have a barrier per entry;
          // V's slot waits for this tile's probabilities.
          if (!(ok = wait_all(sBar + 8u * (B::kExp + (it & 7u)), (it >> 3) & 1u))) break;
          const int4 x = s_exp[it & 7u];
          if (x.z != 0 && !(ok = wait_all(sBar + 8u * (B::kVFull + s), (it / NS) & 1u))) break;
          rk = fmaxf(rs * __int_as_float((127 + x.x) << 23), 1e-37f);
          ve = (float)x.y;
          vi = __int_as_float((127 - x.y) << 23);
          apart = x.z != 0;
        }
        tc_fence_after();
        const uint32_t col_p = t_lane + kColP;
        const bool edge = n0 + BN > P || p.window > 0;
        float alpha = 1.f, sum = 0.f;  // this tile's moves of the reference, its sum of P
        // Exponents of 32 scores and their sum; the packed pairs go to P.
        auto exps = [&](const uint32_t(&sr)[32], float scale, float ref, uint32_t(&pk)[16]) {
          const uint64_t sc2 = f2(scale, scale), ref2 = f2(ref, ref);
          uint64_t l0 = 0, l1 = 0;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float a, a2, e, f;
            unf2(ffma2(f2(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1])), sc2, ref2), a, a2);
            unf2(ffma2(f2(__uint_as_float(sr[2 * k + 2]), __uint_as_float(sr[2 * k + 3])), sc2, ref2), e, f);
            a = ex2(a), a2 = ex2(a2), e = ex2(e), f = ex2(f);
            pk[k] = pack2<MBF>(a, a2);
            pk[k + 1] = pack2<MBF>(e, f);
            l0 = fadd2(l0, f2(a, a2));
            l1 = fadd2(l1, f2(e, f));
          }
          float la, lb;
          unf2(fadd2(l0, l1), la, lb);
          sum += la + lb;
        };
        // P of the tile before has been read.
        if (c > 0 && !(ok = wait_all(sBar + 8u * (B::kODone + t), (c - 1u) & 1u))) break;
        tc_fence_after();
        bool plain = !edge && !apart;
        if (plain) {
          // No mask, no exponents per key: the next 32 scores load during these.
          // A score above the reference ends this form; the tile starts again
          // in the general one (its scores are still there).  Kept apart, since
          // the general form's code between the chunks cost 48 of 176 us.
          uint32_t x[2][32];
          float top[2];
          const float ref = ve - M + kBias;
          top[0] = tmem_ld32_max(t_lane, x[0]);
#pragma unroll
          for (int h = 0; h < BN / 32; ++h) {
            tmem_wait_ld();
            if (h + 1 < BN / 32)
              top[(h + 1) & 1] = tmem_ld32_max(t_lane + 32 * (h + 1), x[(h + 1) & 1]);
            plain = !__any_sync(0xffffffffu, fmaf(top[h & 1], rk, ve) > M + kCaSlack);
            if (!plain) break;
            if (h + 1 == BN / 32) {
              tc_fence_before();
              warp_arrive(sBar + 8u * (B::kSFree + t));  // the next tile's scores may come
            }
            uint32_t pk[16];
            exps(x[h & 1], rk, ref, pk);
            tmem_st16(col_p + 16 * h, pk);
          }
          if (!plain) {
            sum = 0.f;
            tmem_wait_ld();
            tmem_wait_st();
          }
        }
        if (!plain) {
#pragma unroll 1
          for (int h = 0; h < BN / 32; ++h) {
            uint32_t sr[32], pk[16];
            float mx = tmem_ld32_max(t_lane + 32 * h, sr);
            tmem_wait_ld();
            if (h + 1 == BN / 32) {
              tc_fence_before();
              warp_arrive(sBar + 8u * (B::kSFree + t));
            }
            if (edge) {  // keys this row keeps, one bit each
              const uint32_t keep =
                  keep_bits(p, on, i, dep, n0 + 32 * h - P, E, cu0, (long long)d2.y);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(keep >> k & 1u)) sr[k] = 0xFF800000u;  // -inf
            }
            if (edge || apart) {
              mx = -INFINITY;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (apart)  // the whole exponent here, a key's own part of it included
                  sr[k] = __float_as_uint(fmaf(__uint_as_float(sr[k]), rk, s_we[s * BN + 32 * h + k]));
                mx = fmaxf(mx, __uint_as_float(sr[k]));
              }
            }
            const float rc = apart ? 1.f : rk;
            mx = fmaf(mx, rc, ve);  // ve is 0 with exponents per key
            const bool raise = mx > M + kCaSlack;
            if (__any_sync(0xffffffffu, raise)) {
              const float to = raise ? mx + kCaHead : M, a = ex2(M - to);
              M = to;
              L *= a;
              sum *= a;
              alpha *= a;
              tmem_wait_st();
#pragma unroll 1
              for (int e = 0; e < h; ++e) {  // this tile's P so far
                tmem_ld16(col_p + 16 * e, pk);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  pk[k] = pack2<MBF>(unpack_lo<MBF>(pk[k]) * a, unpack_hi<MBF>(pk[k]) * a);
                tmem_st16(col_p + 16 * e, pk);
                tmem_wait_st();
              }
            }
            const float ref = ve - M + kBias;
            if (apart) {
              float part = 0.f;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float a = ex2(__uint_as_float(sr[2 * k]) + ref);
                const float e = ex2(__uint_as_float(sr[2 * k + 1]) + ref);
                pk[k] = pack2<MBF>(a, e);
                part = fmaf(a, s_wi[s * BN + 32 * h + 2 * k], part);
                part = fmaf(e, s_wi[s * BN + 32 * h + 2 * k + 1], part);
              }
              sum += part;
            } else {
              exps(sr, rc, ref, pk);
            }
            tmem_st16(col_p + 16 * h, pk);
          }
        }
        L = fmaf(sum, vi, L);
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {  // O so far, its products done
#pragma unroll 1
          for (int x8 = 0; x8 < D / 32; ++x8) {
            uint32_t o[32];
            tmem_ld32(t_lane + kColO + x8 * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(t_lane + kColO + x8 * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(sBar + 8u * (B::kPFull + t));
      }
      if (!ok) break;
      if (!(ok = wait_all(sBar + 8u * (B::kODone + t), (c - 1u) & 1u))) break;
      tc_fence_after();
      // ---- the row: a partial, or the result
      if (cut) {
        const long long pr = (2ll * blockIdx.x + (d0.y >> 1)) * RT + 128 * t + r;
#pragma unroll 1
        for (int x8 = 0; x8 < D / 32; ++x8) {
          uint32_t o[32];
          tmem_ld32(t_lane + kColO + x8 * 32, o);
          tmem_wait_ld();
          if (on) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + pr * D + 32 * x8);
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
        for (int x8 = 0; x8 < D / 32; ++x8) {
          uint32_t o[32];
          tmem_ld32(t_lane + kColO + x8 * 32, o);
          tmem_wait_ld();
          if (on) {
            uint4* dst =
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + 32 * x8);
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
  // The products are done (warps 12 and 13 drained them) and every row has been read.
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag != 0u) ca_mark(p, 1);
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512u);
  }
}

}  // namespace gqa
