// cache_attn.cuh -- attention of a few new tokens per sequence (one decoded
// token, or a tree of drafted ones) over a paged cache, 16-bit or e4m3, for
// sm_103a.  Reached through gqa_cache_attention.
//
// Mathematics.  One pass over the keys with a running reference per row, in
// the log2 domain.  With s = scale log2(e) <q, k> and, for an e4m3 cache, the
// key's value scale 2^w (w = 0 otherwise),
//   M   >= max (s + w) - kCaSlack           the row's reference, moved lazily
//   P_j  = 2^(s_j + w_j - M + kBias)        fp32, see below
//   O    = sum P_j V_j,  L = sum P_j 2^-w_j   (fp32; V_j the stored values)
//   out  = O / (L + 2^(x - M + kBias)),   lse = (M - kBias + log2(L + ..)) ln 2
// so the value scales cost no pass of their own and L keeps the unrounded
// probabilities.  The second product takes P in 16 bits.  Rounded once that would
// add as much as the rounding of out where both have as many bits: over few keys
// and heads the error against 64 bits was up to twice the output's own.  So P is
// the sum of two 16-bit terms there (16-bit pages, and e4m3 under an f16 out),
// good to 2^-16 (bf16) or 2^-22, and one f16 term for e4m3 under a bf16 out (two
// terms: 256 sequences of 1k..16k keys 360 us, one 350; 16-bit pages are bound by
// memory all the same, 168 us for 64 such sequences either way).  A reference moves to kCaHead above the score that made it,
// so it moves once or twice in a sequence (each move rescales O); kBias uses
// f16's range upwards: P stays below 2^15, and a key weighs in down to 2^-30 of
// the largest at the least.
//
// Layout.  A page holds page_size tokens x Hkv heads x d values: the K of one
// token's heads is one run of memory, and so is a page's.  A CTA therefore
// takes HPC heads at once (all of them up to 8), one warp per head (or
// several warps that share a head's keys when there are fewer heads), and a
// producer warp copies whole runs of a page into a shared-memory ring with
// cp.async.bulk: no tensor map, no gather of 64-byte head slices, every DRAM
// burst read whole.  The G query heads of the tokens are the rows of the
// products: few (8 for one token of a 64 / 8 head model), so the products are
// m16n8k16 warp instructions whose operands are converted from e4m3 in
// registers; a 128-row tensor-memory tile would be 94% padding there.  They
// are taken transposed, S^T = K Q^T and O^T = V^T P^T: the keys (the head's
// values) fill the 16-row side and the queries the 8-column side, so 8 rows
// waste nothing.  (With the rows on the 16-row side half of every product and
// of the softmax was padding: 256 sequences of 1k..16k e4m3 keys 689 us.)
//
// Fragment order.  A contraction may run in any order, so the fragments are
// laid out by what one wide shared-memory load brings.  Lane (g, t) = (lane /
// 4, lane % 4).  Row m of a 16-key score tile is key ca_key(m); lane (g, t)
// loads 16 bytes of keys ca_key(g) and ca_key(g + 8) and later, for the second
// product, 8 values at 8 g of the keys 4 t .. 4 t + 3, which are the keys that
// an 8x8 transpose of P hands it.  The transposition of V is the byte
// interleave of its conversion.
//
// Work split.  Every CTA takes an equal share of all (sequence, row tile,
// head group) key tiles laid end to end (lengths are device data: the split
// is found on the device), and a unit cut by a share boundary leaves fp32
// partials (O, M, L) that cache_merge_kernel joins.  When whole units dealt
// out cost no more than equal shares plus a join, they are dealt whole.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "prefill_kernel.cuh"
#include "ptx.cuh"

namespace gqa {

// Consumer warps; one producer warp follows them.  16 where the accumulators
// leave room for them (96 registers a thread), else 8 (168 registers).
__host__ __device__ constexpr int ca_warps(int D, bool C8, int NT) {
  return NT == 1 && (D == 64 || (D == 128 && C8)) ? 16 : 8;
}
constexpr int kCaMaxSlots = 16;                    // ring slots at most
constexpr int kCaPieces = 8;                       // pieces the planning warp may be ahead
// In powers of two: what a score may exceed its row's reference by before the
// reference moves, how far above the score it then moves, and the exponent
// that a probability at the reference gets.
constexpr float kCaSlack = 6.f, kCaHead = 4.f, kCaBias = 9.f;
constexpr int kCaWholeSlack = 6;                   // tiles a join is worth
// Least byte of a value scale that counts, 2^-100: the denominators hold 2^-w,
// which overflows for the zero bytes of slots that were never written.
constexpr uint32_t kCaLeast = 27;

// Division of 0 <= n < 2^31 by a divisor fixed for the launch: with l =
// ceil(log2 d) and m = ceil(2^(32 + l) / d) - 2^32, n / d = (hi(n m) + n) >> l
// exactly (the rounding of m adds less than n / 2^(32 + l) <= 1 / 2^(l + 1) to
// the quotient, less than the gap below the next multiple of 1 / d).
struct FastDiv {
  uint32_t m;
  int l;
  __host__ void set(uint32_t d) {
    l = 0;
    while ((1ull << l) < d) ++l;
    m = (uint32_t)(((1ull << (32 + l)) + d - 1) / d - (1ull << 32));
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> l);
  }
};

struct CacheAttnParams {
  const void* q;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int32_t* cu;
  const int32_t* pre;
  const int32_t* indptr;
  const int32_t* indices;
  const float* sinks;
  const uint32_t* mask;
  const int32_t* mask_indptr;
  const int32_t* depths;
  void* out;
  float* lse;
  unsigned int* status;
  float* part_o;     // [2 per CTA][HPC * RT rows][D]
  float* part_ml;    // [2 per CTA][HPC * RT rows][2] (M, L)
  int32_t* head;     // [0] units to look at; byte 16 + c: 1 when a wait of CTA c ran out
  int32_t* hdr;      // [8 u ..] unit u: pieces after its first, the first's CTA, first row, first
                     // head, first token, tokens
  long long total_mask_words;
  unsigned long long timeout_ns;
  int entries, num_pages, page_size;
  int num_seqs, first_seq, total_q;
  int Hq, Hkv, G;
  int HPC, HG;       // heads per CTA, head groups
  int ctas;          // of the launch
  int KW;            // warps that share a head's keys
  int T, log_T;      // keys per tile (16 GK KW, a power of two)
  FastDiv div_g, div_page, div_ctas;
  int run, log_run;  // tokens per copy, a power of two that divides T and the page
  int NS;            // ring slots
  uint32_t slot_bytes, data_bytes;  // a slot, and its values (scales follow)
  int window, smooth;
  int whole;         // units dealt whole whatever the lengths
  int whole_slack;   // tiles that a join is worth
  float scale_log2;
  int metadata_ready;
};

// Rows of a unit: NT tiles of 8.  GK: 16-key groups a warp takes per tile.
__host__ __device__ constexpr int ca_gk(int D, bool C8, int NT) {
  return NT == 1 && D == 64 && C8 ? 2 : 1;
}
// Key of row m of a 16-key score tile: the transposed P gives lane t the rows
// 2 t, 2 t + 1, 2 t + 8, 2 t + 9, which are keys 4 t .. 4 t + 3.
__device__ __forceinline__ int ca_key(int m) {
  return 4 * ((m & 7) >> 1) + (m & 1) + 2 * (m >> 3);
}
// Shared memory besides the ring: per warp an area of 8 rows x 64 columns
// fp32 and its rows' (M, L), the barriers, the tables of the sequences.
__host__ __device__ constexpr uint32_t ca_fixed_smem(int warps) {
  return 1024u + 128u + (uint32_t)warps * (8u * 64u * 4u + 8u * 8u) + 2u * kCaMaxSlots * 8u + 32u +
         4u * (5 * kMaxSeqs + 3) + kCaPieces * (16u * 4u + 2u * 8u);
}

// The CTA's mark for the join: cleared before any of its warps can give up, by a
// thread that has no sequence to look up in a small batch.  Bytes, so that a
// block of the join reads all in ten 16-byte loads (a word a CTA: a join of many
// small blocks 0.5 us longer); the ones that fill the last 16 are some CTA's too.
__device__ __forceinline__ void ca_mark(const CacheAttnParams& p, uint8_t gave_up) {
  uint8_t* marks = reinterpret_cast<uint8_t*>(p.head + 4);
  for (int c = blockIdx.x; c < (p.ctas + 15) / 16 * 16; c += p.ctas) marks[c] = gave_up;
}

struct CaTab {
  const int32_t* tiles;  // [B] exclusive scan of key tiles
  const int32_t* units;  // [B] exclusive scan of units
  const int32_t* cu0;    // [B + 1]
  const int32_t* pre;    // [B]
  const int32_t* ipt;    // [B]
};

// A piece of work: tiles [t0, t1) of the n tiles of one unit.
struct CaPiece {
  int b, rt, hg, unit;
  int P, E, lo, hi;  // keys [lo, hi), lo a multiple of T
  int n, t0, t1;
};

// Key range of row tile rt: rows rt * RT .. of the sequence's E * G.
__device__ __forceinline__ void ca_range(const CacheAttnParams& p, int P, int E, int rt, int RT,
                                         int& lo, int& hi, int& n) {
  const int i1 = min(p.div_g.div(rt * RT + RT - 1), E - 1);
  hi = P + i1 + 1;
  lo = 0;
  if (p.window > 0) {
    // The lowest position of the tile's rows: depths may be anything >= 0.
    const int a = P - p.window + 1 + (p.depths != nullptr ? 0 : p.div_g.div(rt * RT));
    if (a > 0) lo = a >> p.log_T << p.log_T;
  }
  n = (hi - lo + p.T - 1) >> p.log_T;
}

// Equal shares of W tiles over C <= W CTAs: the first W % C hold one more.
struct CaShares {
  int q, r;  // W / C, W % C
  __device__ __forceinline__ int lo(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int owner(int x) const {  // CTA of tile x
    const int big = r * (q + 1);
    return x < big ? x / (q + 1) : r + (x - big) / q;
  }
};

struct CaWalk {
  int at, end;  // share mode: tiles left; whole mode: end is the unit count
  int unit;     // whole mode: next unit, every gridDim.x-th
  bool whole;
  // Share mode: the sequence of the last piece, its row tile and the tiles of
  // the sequence before that (pieces come in order, so a long sequence's row
  // tiles are counted once).
  int b, rt, before;
};

// Largest i in [0, n) with a[i] <= x (a[0] = 0 <= x) for a non-decreasing
// shared-memory array, by a converged warp: 32 probes a step.
__device__ __forceinline__ int warp_find(const int32_t* a, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lo + lane * step;
    const int c = __popc(__ballot_sync(0xffffffffu, lane * step < n && a[i] <= x)) - 1;
    lo += c * step;
    n = min(step, n - c * step);
  }
  return lo;
}

// The next piece; called by a converged warp.
__device__ __forceinline__ bool ca_next(const CacheAttnParams& p, const CaTab& T, CaWalk& w, int RT,
                                        CaPiece& u) {
  const int32_t* key = w.whole ? T.units : T.tiles;
  const int x = w.whole ? w.unit : w.at;
  if (x >= w.end) return false;
  const int lo = warp_find(key, p.num_seqs, x);
  u.b = lo;
  u.P = T.pre[lo];
  u.E = T.cu0[lo + 1] - T.cu0[lo];
  int off = x - key[lo];
  if (w.whole) {
    u.rt = p.HG == 1 ? off : off / p.HG;
    u.hg = off - u.rt * p.HG;
    ca_range(p, u.P, u.E, u.rt, RT, u.lo, u.hi, u.n);
    u.t0 = 0;
    u.t1 = u.n;
    u.unit = x;
    w.unit += gridDim.x;
    return true;
  }
  if (w.b != lo) {
    w.b = lo;
    w.rt = 0;
    w.before = 0;
  }
  off -= w.before;
  for (;; ++w.rt) {  // ends: off lies within the sequence's tiles
    ca_range(p, u.P, u.E, w.rt, RT, u.lo, u.hi, u.n);
    const int all = u.n * p.HG;
    if (off < all) break;
    off -= all;
    w.before += all;
  }
  u.rt = w.rt;
  u.hg = p.HG == 1 ? 0 : off / u.n;
  u.t0 = off - u.hg * u.n;
  u.t1 = min(u.n, u.t0 + w.end - w.at);
  u.unit = T.units[lo] + u.rt * p.HG + u.hg;
  w.at += u.t1 - u.t0;
  return true;
}

// Per sequence its key tiles and units, and the checks of the metadata
// (misc[1] set when something is inconsistent, misc[2] raised to the most
// tiles of a unit).  Called by every thread of the CTA; a barrier follows.
__device__ __forceinline__ void ca_tables(const CacheAttnParams& p, int32_t* tiles, int32_t* units,
                                          int32_t* s_cu, int32_t* s_pre, int32_t* s_ipt,
                                          uint32_t* misc, int RT, int tid, int nthreads) {
  const int nseq = p.num_seqs;
  bool bad = tid == 0 && p.first_seq == 0 && __ldg(p.cu) != 0;
  int my_max = 0;
  for (int b = tid; b < nseq; b += nthreads) {
    const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), P = __ldg(p.pre + b);
    const int i0 = __ldg(p.indptr + b), i1 = __ldg(p.indptr + b + 1);
    const int E = c1 - c0;
    bool b_bad = c0 < 0 || c1 < c0 || c1 > p.total_q || P < 0 || P > 0x7fff0000 - E || i0 < 0 ||
                 i1 > p.entries;
    if (!b_bad) b_bad = i1 - i0 != (P + E > 0 ? p.div_page.div(P + E - 1) + 1 : 0);
    if (p.mask != nullptr) {
      const long long m0 = __ldg(p.mask_indptr + b), m1 = __ldg(p.mask_indptr + b + 1);
      b_bad |= m0 < 0 || m1 > p.total_mask_words || m1 - m0 != (long long)E * ((E + 31) / 32);
    }
    bad |= b_bad;
    long long w = 0;
    int nu = 0;
    if (!b_bad && E > 0) {
      nu = (E * p.G + RT - 1) / RT;
      for (int rt = 0; rt < nu; ++rt) {
        int lo, hi, n;
        ca_range(p, P, E, rt, RT, lo, hi, n);
        w += n;
        my_max = max(my_max, n);
      }
      w *= p.HG;
      nu *= p.HG;
    }
    s_cu[b] = c0;
    s_pre[b] = P;
    s_ipt[b] = i0;
    if (w > 0x7fffffffll) bad = true;  // more key tiles than the shares count
    tiles[b] = (int)w;
    units[b] = nu;
    if (b == nseq - 1) s_cu[nseq] = c1;
  }
  if (bad) misc[1] = 1u;
  const int lane = tid & 31;
  my_max = __reduce_max_sync(0xffffffffu, my_max);
  if (lane == 0 && my_max > 0) atomicMax(reinterpret_cast<int*>(misc + 2), my_max);
}

struct CaPlan {
  CaTab T;
  CaShares shares;
  CaWalk walk;
};

// The CTA's part of the work; called by one converged warp after ca_tables.
__device__ __forceinline__ CaPlan ca_plan(const CacheAttnParams& p, int32_t* tiles, int32_t* units,
                                          int32_t* s_cu, int32_t* s_pre, int32_t* s_ipt,
                                          const uint32_t* misc) {
  const int lane = threadIdx.x & 31, nseq = p.num_seqs;
  // Exclusive scans of the tiles and units, a run of sequences a lane.
  const int run = (nseq + 31) >> 5, b0 = min(lane * run, nseq), b1 = min(b0 + run, nseq);
  long long st = 0;
  int su = 0;
  for (int b = b0; b < b1; ++b) {
    st += tiles[b];
    su += units[b];
  }
  long long at = st;
  int au = su;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, at, o);
    const int y = __shfl_up_sync(0xffffffffu, au, o);
    if (lane >= o) {
      at += x;
      au += y;
    }
  }
  const long long total = __shfl_sync(0xffffffffu, at, 31);
  const int n_all = __shfl_sync(0xffffffffu, au, 31);
  at -= st;
  au -= su;
  for (int b = b0; b < b1; ++b) {
    const int w = tiles[b], nu = units[b];
    tiles[b] = (int)at;
    units[b] = au;
    at += w;
    au += nu;
  }
  __syncwarp();
  // More key tiles than the shares count: nothing is done.
  const int W = total > 0x7fffffffll ? 0 : (int)total;
  if (W != total && lane == 0) atomicOr(p.status, 2u);  // GQA_DEV_BAD_METADATA
  const int n_units = W > 0 ? n_all : 0, grid = gridDim.x, c = blockIdx.x;
  // No more shares than tiles: every share holds a tile, so the pieces of a
  // cut unit lie on consecutive CTAs.
  const int C = min(W, grid);
  const int per = W < grid ? 1 : p.div_ctas.div(W);  // tiles of the smaller shares
  CaPlan plan;
  plan.T = CaTab{tiles, units, s_cu, s_pre, s_ipt};
  plan.shares = CaShares{per, W < grid ? 0 : W - per * grid};
  // Whole units when the deepest deal costs no more than an equal share and
  // the join that cut units need.
  CaWalk& w = plan.walk;
  w.whole = p.whole != 0 || (long long)p.div_ctas.div(n_units + grid - 1) * (int)misc[2] <=
                                per + p.whole_slack;
  w.unit = c;
  w.b = -1;
  w.at = c < C ? plan.shares.lo(c) : 0;
  w.end = w.whole ? n_units : c < C ? plan.shares.lo(c + 1) : 0;
  if (c == 0 && lane == 0) p.head[0] = w.whole ? 0 : n_units;
  return plan;
}

// What the other warps need of a piece, in 3 x 16 bytes: tiles (0: no more),
// flags (1 cut, 2 the first piece of a cut unit), first key, prefix; tokens,
// end of the keys, first row, first head; first token, first mask word.  The
// unit's first piece also writes its entry for the join.
__device__ __forceinline__ void ca_publish(const CacheAttnParams& p, const CaPlan& plan,
                                           const CaPiece& u, bool more, int RT, int4* d) {
  const bool cut = more && (u.t0 > 0 || u.t1 < u.n);
  const int m0 = more && p.mask != nullptr ? __ldg(p.mask_indptr + u.b) : 0;
  const int cu0 = more ? plan.T.cu0[u.b] : 0;
  d[0] = make_int4(more ? u.t1 - u.t0 : 0, (cut ? 1 : 0) | (cut && u.t0 == 0 ? 2 : 0),
                   u.lo + (u.t0 << p.log_T), u.P);
  d[1] = make_int4(u.E, u.hi, u.rt * RT, u.hg * p.HPC);
  d[2] = make_int4(cu0, m0, more ? plan.T.ipt[u.b] : 0, 0);
  if (more && !plan.walk.whole && u.t0 == 0) {
    const int c = blockIdx.x;
    int4* hd = reinterpret_cast<int4*>(p.hdr + 8ll * u.unit);
    hd[0] = make_int4(cut ? plan.shares.owner(plan.walk.at - u.t1 + u.n - 1) - c : 0, c, u.rt * RT,
                      u.hg * p.HPC);
    hd[1] = make_int4(cu0, u.E, 0, 0);
  }
}

// L2 policies: keys that this CTA alone reads leave L2 first, so the call's
// tables, partials and results stay (one 131k sequence 35.7 -> 33.6 us, 256
// sequences 355 -> 351).
__device__ __forceinline__ uint64_t l2_policy(bool first) {
  uint64_t a, b;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(a));
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(b));
  return first ? a : b;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1], %2, [%3], %4;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
// Named barrier over `count` threads that tells whether all of them said yes.
__device__ __forceinline__ bool named_bar_all(uint32_t id, uint32_t count, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)yes)
      : "memory");
  return r != 0;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 values as two f16 pairs (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
// 8x8 transpose of 16-bit pairs over the warp: lane (g, t) gives (row g,
// columns 2 t, 2 t + 1) and receives (column g, rows 2 t, 2 t + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}

// D: head dim.  BF16: type of q and out.  C8: e4m3 cache (products in f16),
// else the cache has q's type.  NT: 8-row tiles per warp.
// H8: 8 heads per CTA, which makes the ring's strides constants.
template <int D, bool BF16, bool C8, int NT, bool H8>
__global__ void __launch_bounds__(32 * (ca_warps(D, C8, NT) + 1), 1)
    cache_attn_kernel(const __grid_constant__ CacheAttnParams p) {
  constexpr int NW = ca_warps(D, C8, NT);
  constexpr int kThreads = 32 * (NW + 1);
  constexpr int GK = ca_gk(D, C8, NT);
  constexpr int RT = 8 * NT;
  constexpr bool MBF = BF16 && !C8;          // product type
  // P as two terms of the product type, where one would round it as coarsely as
  // out is rounded: an f16 P under a bf16 out is fine enough.
  constexpr bool kTwoTerms = !(C8 && BF16);
  constexpr float kBias = MBF ? 0.f : kCaBias;
  constexpr int kEsz = C8 ? 1 : 2;
  constexpr int KS = D / 16;                 // k16 steps of the scores
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* scratch = reinterpret_cast<float*>(smem);                 // [NW][8][64]
  float2* s_ml = reinterpret_cast<float2*>(scratch + NW * 8 * 64);  // [NW][8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_ml + NW * 8);
  uint32_t* misc = reinterpret_cast<uint32_t*>(bars + 2 * kCaMaxSlots);  // [0] abort [1] bad
  uint64_t* pbars = reinterpret_cast<uint64_t*>(misc + 8);  // pieces: full, empty
  int4* s_piece = reinterpret_cast<int4*>(pbars + 2 * kCaPieces);  // [kCaPieces][4]
  int32_t* tiles = reinterpret_cast<int32_t*>(s_piece + 4 * kCaPieces);
  int32_t* units = tiles + (kMaxSeqs + 1);
  int32_t* s_cu = units + (kMaxSeqs + 1);
  int32_t* s_pre = s_cu + (kMaxSeqs + 1);
  int32_t* s_ipt = s_pre + kMaxSeqs;
  const uint32_t ring = (smem_u32(s_ipt + kMaxSeqs) + 127u) & ~127u;
  const uint32_t sBar = smem_u32(bars), sPiece = smem_u32(pbars);
  volatile uint32_t* abort_flag = misc;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nact = p.HPC * p.KW;  // consumer warps at work
  const unsigned long long tmo = p.timeout_ns;

  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < p.NS; ++i) {
      mbar_init(sBar + 8u * i, 1u);
      mbar_init(sBar + 8u * (kCaMaxSlots + i), (uint32_t)nact);
    }
    for (int i = 0; i < kCaPieces; ++i) {
      mbar_init(sPiece + 8u * i, 1u);
      mbar_init(sPiece + 8u * (kCaPieces + i), (uint32_t)nact);
    }
    misc[0] = 0u;
    misc[1] = 0u;
    misc[2] = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_launch_dependents();
  if (!p.metadata_ready) {
    grid_dep_wait();
    if (tid == kThreads - 1) ca_mark(p, 0);
  }

  ca_tables(p, tiles, units, s_cu, s_pre, s_ipt, misc, RT, tid, kThreads);
  __syncthreads();
  const bool bad_meta = misc[1] != 0u;
  if (p.metadata_ready) {
    grid_dep_wait();  // before any global write or other read
    if (tid == kThreads - 1) ca_mark(p, 0);
    __syncthreads();  // before a warp can give up
  }
  if (bad_meta) {
    if (tid == 0) {
      atomicOr(p.status, 2u);  // GQA_DEV_BAD_METADATA
      if (blockIdx.x == 0) p.head[0] = 0;
    }
    return;
  }
  const uint32_t row_bytes = H8 ? 8u * D * kEsz : (uint32_t)p.HPC * D * kEsz;  // a token in the ring
  const long long tok_bytes = (long long)p.Hkv * D * kEsz;      // in the pool

  if (warp == NW) {
    // -------------------------------------------------------------- producer
    // Plans the CTA's work, tells the consumers piece by piece, and fills the
    // ring; the other warps would only repeat the planning (17 warps doing so
    // cost 3000 clocks before the first load).
    CaPlan plan = ca_plan(p, tiles, units, s_cu, s_pre, s_ipt, misc);
    // The tile's runs are spread over the lanes; slots alternate K and V.
    uint32_t slot = 0, ph = 0, issued = 0, pi = 0;
    bool ok = true;
    CaPiece u = {};
    const int nrun = p.T / p.run;  // the tile's copies, one a lane
    for (;; ++pi) {
      const bool more = ca_next(p, plan.T, plan.walk, RT, u);
      // ---- tell the consumers
      const uint32_t ps = pi % kCaPieces;
      if (lane == 0)
        ok = wait_bounded(sPiece + 8u * (kCaPieces + ps), ((pi / kCaPieces) & 1u) ^ 1u, abort_flag,
                          p.status, tmo);
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      if (!ok) break;
      if (lane == 0) {
        ca_publish(p, plan, u, more, RT, s_piece + 4 * ps);
        mbar_arrive(sPiece + 8u * ps);
      }
      if (!more) break;
      const int npg = p.div_page.div(u.P + u.E - 1) + 1;
      const int32_t* table = p.indices + plan.T.ipt[u.b];
      const uint64_t policy = l2_policy(u.E * p.G <= RT);  // one row tile reads these keys
      for (int t = u.t0; ok && t < u.t1; ++t) {
        const int n0 = u.lo + t * p.T;
        // Tokens [skip, ntok) of the tile: keys below the window are not read.
        const int ntok = min(p.T, u.hi - n0);
        const int skip = p.window > 0 ? max(u.P - p.window + 1 - n0, 0) : 0;
        for (int kv = 0; kv < 2; ++kv) {
          if (lane == 0) {
            ok = wait_bounded(sBar + 8u * (kCaMaxSlots + slot), ph ^ 1u, abort_flag, p.status, tmo);
            if (ok) {
              uint32_t bytes = (uint32_t)(ntok - skip) * row_bytes;
              if (C8)
                bytes += (uint32_t)(((ntok + p.run - 1) >> p.log_run) - (skip >> p.log_run)) *
                         (uint32_t)(p.run * p.Hkv);
              mbar_arrive_expect_tx(sBar + 8u * slot, bytes);
            }
          }
          ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
          if (!ok) break;
          const uint32_t dst = ring + slot * p.slot_bytes, bar = sBar + 8u * slot;
          const uint8_t* pages = kv ? p.v_pages : p.k_pages;
          for (int r = lane; r < nrun && r * p.run < ntok; r += 32) {
            const int first = max(skip - r * p.run, 0);  // the run's first live token
            const int key = n0 + r * p.run, cnt = min(p.run, ntok - r * p.run) - first;
            if (cnt <= 0) continue;
            const int kp = p.div_page.div(key);
            int pg = __ldg(table + min(kp, npg - 1));
            if (pg < 0 || pg >= p.num_pages) {
              atomicOr(p.status, 2u);  // GQA_DEV_BAD_METADATA
              pg = 0;
            }
            const long long row = (long long)pg * p.page_size + (key - kp * p.page_size);
            const uint8_t* src = pages + (row + first) * tok_bytes + (long long)u.hg * row_bytes;
            const uint32_t to = dst + (uint32_t)(r * p.run + first) * row_bytes;
            if (p.HG == 1)
              bulk_load(to, src, (uint32_t)cnt * row_bytes, bar, policy);
            else
              for (int i = 0; i < cnt; ++i)
                bulk_load(to + i * row_bytes, src + i * tok_bytes, row_bytes, bar, policy);
            if (C8)  // the scales of all heads, whole runs: within the page
              bulk_load(dst + p.data_bytes + (uint32_t)(r * p.run * p.Hkv),
                        (kv ? p.v_scales : p.k_scales) + row * p.Hkv, (uint32_t)(p.run * p.Hkv),
                        bar, policy);
          }
          ++issued;
          if (++slot == (uint32_t)p.NS) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) ca_mark(p, 1);
    // Let every copy issued land before the CTA can exit.
    __syncwarp();
    if (lane < p.NS) {
      const uint32_t loads = issued / p.NS + ((uint32_t)lane < issued % p.NS ? 1u : 0u);
      if (loads > 0) wait_drain(sBar + 8u * lane, (loads - 1u) & 1u, tmo);
    }
    return;
  }
  if (warp >= nact) return;  // more warps than heads can use

  // ---------------------------------------------------------------- consumers
  const int hl = warp % p.HPC, kw = warp / p.HPC;
  const int g = lane >> 2, t = lane & 3;
  // Every lane of a warp goes on or none.
  auto wait_full = [&](uint32_t sl, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bounded(sBar + 8u * sl, parity, abort_flag, p.status, tmo)) != 0;
  };
  uint32_t slot = 0, ph = 0;
  // Warps that share a head's keys go on together or not at all: each takes
  // part in one such barrier per piece, the one that finds no piece or whose
  // wait ran out included, so none waits for a warp that has left.
  auto together = [&](bool yes) {
    return p.KW > 1 ? named_bar_all(1u + (uint32_t)hl, 32u * (uint32_t)p.KW, yes) : yes;
  };
  bool ok = true;
  for (uint32_t pi = 0;; ++pi) {
    // ---- the next piece
    const uint32_t ps = pi % kCaPieces;
    ok = __all_sync(0xffffffffu, wait_bounded(sPiece + 8u * ps, (pi / kCaPieces) & 1u, abort_flag,
                                              p.status, tmo)) != 0;
    if (!ok) {
      together(false);
      break;
    }
    const int4 d0 = s_piece[4 * ps], d1 = s_piece[4 * ps + 1], d2 = s_piece[4 * ps + 2];
    __syncwarp();
    if (lane == 0) mbar_arrive(sPiece + 8u * (kCaPieces + ps));
    const int n_tiles = d0.x, P = d0.w, E = d1.x, row0 = d1.z;
    const bool cut = (d0.y & 1) != 0;
    if (n_tiles == 0) {
      together(true);
      break;
    }
    const int head = d1.w + hl;  // KV head
    const int cu0 = d2.x;
    // Softmax rows of the thread: 2 t and 2 t + 1 of every 8-row tile.
    int ri[NT][2], rdep[NT][2];  // token index (-1: none) and depth
    float rs[NT][2];             // scale to the log2 domain
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = p.div_g.div(row0 + m * 8 + 2 * t + h);
        const bool on = i < E;
        ri[m][h] = on ? i : -1;
        rdep[m][h] = i;
        if (on && p.depths != nullptr) rdep[m][h] = __ldg(p.depths + cu0 + i);
        rs[m][h] = p.scale_log2;
      }
    // Query fragments: row g of every tile.
    uint32_t qf[NT][KS][2];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int r = row0 + m * 8 + g;
      const int i = p.div_g.div(r);
      const bool on = i < E;
      const uint16_t* qr = static_cast<const uint16_t*>(p.q) +
                           ((long long)(cu0 + (on ? i : 0)) * p.Hq + head * p.G + (r - i * p.G)) * D;
      if constexpr (C8) {
        // f16 operands: the row scaled by the power of two that brings its
        // largest magnitude into [1, 2); smaller values round at 2^-25.
        uint2 w[KS];
        float amax = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          w[s] = on ? __ldg(reinterpret_cast<const uint2*>(qr + 64 * (s >> 2) + 16 * t + 4 * (s & 3)))
                    : make_uint2(0u, 0u);
          amax = max3(amax, fabsf(unpack_lo<BF16>(w[s].x)), fabsf(unpack_hi<BF16>(w[s].x)));
          amax = max3(amax, fabsf(unpack_lo<BF16>(w[s].y)), fabsf(unpack_hi<BF16>(w[s].y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126);
        const float f = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qf[m][s][0] = pack2<false>(unpack_lo<BF16>(w[s].x) * f, unpack_hi<BF16>(w[s].x) * f);
          qf[m][s][1] = pack2<false>(unpack_lo<BF16>(w[s].y) * f, unpack_hi<BF16>(w[s].y) * f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)  // lane 4 r holds row r's exponent
          rs[m][h] *= __int_as_float((127 + __shfl_sync(0xffffffffu, e, 4 * (2 * t + h))) << 23);
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint2 w = on ? __ldg(reinterpret_cast<const uint2*>(
                                   qr + 32 * (s >> 1) + 8 * t + 4 * (s & 1)))
                             : make_uint2(0u, 0u);
          qf[m][s][0] = w.x;
          qf[m][s][1] = w.y;
        }
      }
    }
    float o[NT][D / 16][4];  // [tile][16 values][(value g, g + 8) x (row 2 t, 2 t + 1)]
    float M[NT][2], L[NT][2];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      M[m][0] = M[m][1] = -1e30f;
      L[m][0] = L[m][1] = 0.f;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) o[m][n][0] = o[m][n][1] = o[m][n][2] = o[m][n][3] = 0.f;
    }
    const uint32_t koff = (uint32_t)(kw * 16 * GK + ca_key(g)) * row_bytes +
                          (uint32_t)(hl * D * kEsz) + 16u * t;
    const uint32_t voff = (uint32_t)(kw * 16 * GK + 4 * t) * row_bytes +
                          (uint32_t)(hl * D * kEsz + 8 * kEsz * g);
    const uint32_t soff = p.data_bytes + (uint32_t)((kw * 16 * GK + ca_key(g)) * p.Hkv + head);

    int n0 = d0.z + kw * 16 * GK;  // this warp's first key
    for (int tl = 0; tl < n_tiles; ++tl, n0 += p.T) {
      // ---- scores of 16 GK keys
      if (!(ok = wait_full(slot, ph))) break;
      float s[NT][GK][4];  // [(key g, g + 8) x (row 2 t, 2 t + 1)]
      float ks[GK][2];
      {
        const uint32_t base = ring + slot * p.slot_bytes;
#pragma unroll
        for (int k = 0; k < GK; ++k) {
#pragma unroll
          for (int m = 0; m < NT; ++m) s[m][k][0] = s[m][k][1] = s[m][k][2] = s[m][k][3] = 0.f;
          const uint32_t ka = base + koff + (uint32_t)(16 * k) * row_bytes;
#pragma unroll
          for (int c4 = 0; c4 < D * kEsz / 64; ++c4) {
            const uint4 x = lds128(ka + 64u * c4), y = lds128(ka + 2u * row_bytes + 64u * c4);
            if constexpr (C8) {
              const uint32_t xx[4] = {x.x, x.y, x.z, x.w}, yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t a[4];
                e4m3x4_f16(xx[j], a[0], a[2]);
                e4m3x4_f16(yy[j], a[1], a[3]);
#pragma unroll
                for (int m = 0; m < NT; ++m)
                  mma16816<MBF>(s[m][k], a, qf[m][4 * c4 + j][0], qf[m][4 * c4 + j][1]);
              }
            } else {
              const uint32_t a[4] = {x.x, y.x, x.y, y.y}, b[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
              for (int m = 0; m < NT; ++m) {
                mma16816<MBF>(s[m][k], a, qf[m][2 * c4][0], qf[m][2 * c4][1]);
                mma16816<MBF>(s[m][k], b, qf[m][2 * c4 + 1][0], qf[m][2 * c4 + 1][1]);
              }
            }
          }
          if constexpr (C8) {
            const uint32_t sa = base + soff + (uint32_t)(16 * k * p.Hkv);
            ks[k][0] = __int_as_float((int)lds8(sa) << 23);
            ks[k][1] = __int_as_float((int)lds8(sa + 2u * p.Hkv) << 23);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sBar + 8u * (kCaMaxSlots + slot));
        if (++slot == (uint32_t)p.NS) {
          slot = 0;
          ph ^= 1u;
        }
      }
      // ---- V of the tile: its scales join the exponents
      if (!(ok = wait_full(slot, ph))) break;
      const uint32_t vbase = ring + slot * p.slot_bytes;
      float we[GK][2], wi[GK][2];  // the value scale's exponent, and 2^-exponent
      if constexpr (C8) {
#pragma unroll
        for (int k = 0; k < GK; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t e = max(lds8(vbase + soff + (uint32_t)((16 * k + 2 * j) * p.Hkv)), kCaLeast);
            we[k][j] = __uint_as_float(0x4B000000u | e) - 8388735.f;  // 2^23 + e - (2^23 + 127)
            wi[k][j] = __uint_as_float((254u << 23) - e * (1u << 23));
          }
      }
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int k = 0; k < GK; ++k)
#pragma unroll
          for (int c2 = 0; c2 < 4; ++c2) {
            float& x = s[m][k][c2];
            if constexpr (C8)
              x = fmaf(x, rs[m][c2 & 1] * ks[k][c2 >> 1], we[k][c2 >> 1]);
            else
              x *= rs[m][c2 & 1];
          }
      // Which keys need a look at the mask: any at or past the prefix's end
      // (causal, tree, end of the sequence) or below some row's window.
      const bool edge = n0 + 16 * GK > P || p.window > 0;
      uint32_t live[GK];  // which of the keys 4 t .. 4 t + 3 some row sees
#pragma unroll
      for (int k = 0; k < GK; ++k) live[k] = 15u;
      if (__builtin_expect(edge, 0)) {
#pragma unroll
        for (int k = 0; k < GK; ++k) {
          uint32_t seen[2];  // bit 4 g + t': rows 2 t', 2 t' + 1 of a tile see key g (+ 8)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            bool any = false;
            const int x = n0 + 16 * k + ca_key(g + 8 * j) - P;  // index among the new tokens
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int i = ri[m][h];
                bool keep = i >= 0 && x <= i;
                if (keep && x >= 0 && p.mask != nullptr)
                  keep = (__ldg(p.mask + (long long)d2.y + (long long)i * ((E + 31) >> 5) + (x >> 5)) >>
                          (x & 31)) & 1u;
                if (keep && p.window > 0) {
                  const int place = x >= 0 && p.depths != nullptr ? __ldg(p.depths + cu0 + x) : x;
                  keep = place > rdep[m][h] - p.window;
                }
                if (!keep) s[m][k][2 * j + h] = -INFINITY;
                any |= keep;
              }
            seen[j] = __ballot_sync(0xffffffffu, any);
            if constexpr (C8)  // keys that no row sees may have any scale
              if (!(seen[j] >> (4 * g) & 15u)) wi[k][j] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)  // key 4 t + j: row 2 t + j % 2 + 8 (j / 2) of the scores
            if (!(seen[j >> 1] >> (4 * (2 * t + (j & 1))) & 15u)) live[k] &= ~(1u << j);
        }
      }
      // ---- the references: moved when some score exceeds one by kCaSlack
      bool raise = false;
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = s[m][0][h];
#pragma unroll
          for (int k = 0; k < GK; ++k) mx = max3(mx, s[m][k][h], s[m][k][2 + h]);
          raise |= mx > M[m][h] + kCaSlack;
        }
      if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = s[m][0][h];
#pragma unroll
            for (int k = 0; k < GK; ++k) mx = max3(mx, s[m][k][h], s[m][k][2 + h]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            mx = mx > M[m][h] + kCaSlack ? mx + kCaHead : M[m][h];
            const float f = ex2(M[m][h] - mx);
            M[m][h] = mx;
            L[m][h] *= f;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              o[m][n][h] *= f;
              o[m][n][2 + h] *= f;
            }
          }
      }
      uint32_t pf[NT][GK][2], pr[kTwoTerms ? NT : 1][kTwoTerms ? GK : 1][2];  // P, and its rest
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const float r0 = M[m][0] - kBias, r1 = M[m][1] - kBias;
#pragma unroll
        for (int k = 0; k < GK; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float a = ex2(s[m][k][2 * j] - r0), b = ex2(s[m][k][2 * j + 1] - r1);
            if constexpr (C8) {
              L[m][0] = fmaf(a, wi[k][j], L[m][0]);
              L[m][1] = fmaf(b, wi[k][j], L[m][1]);
            } else {
              L[m][0] += a;
              L[m][1] += b;
            }
            const uint32_t near = pack2<MBF>(a, b);
            pf[m][k][j] = transpose8(near);
            if constexpr (kTwoTerms)
              pr[m][k][j] = transpose8(pack2<MBF>(a - unpack_lo<MBF>(near), b - unpack_hi<MBF>(near)));
          }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int k = 0; k < GK; ++k) {
        const uint32_t vk = vbase + voff + (uint32_t)(16 * k) * row_bytes;
        // Keys that no row sees may hold anything: zeros in their place.
#pragma unroll
        for (int c64 = 0; c64 < D / 64; ++c64) {
          if constexpr (C8) {
            uint2 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = lds64(vk + (uint32_t)j * row_bytes + 64u * c64);
            if (__builtin_expect(edge, 0)) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!(live[k] >> j & 1u)) w[j] = make_uint2(0u, 0u);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {  // values 2 n and 2 n + 1 of the lane's 8
              const uint32_t sel = (n & 1) ? 0x7362u : 0x5140u;
              const uint32_t x = __byte_perm(n < 2 ? w[0].x : w[0].y, n < 2 ? w[1].x : w[1].y, sel);
              const uint32_t y = __byte_perm(n < 2 ? w[2].x : w[2].y, n < 2 ? w[3].x : w[3].y, sel);
              uint32_t a[4];
              e4m3x4_f16(x, a[0], a[1]);
              e4m3x4_f16(y, a[2], a[3]);
#pragma unroll
              for (int m = 0; m < NT; ++m) {
                mma16816<MBF>(o[m][4 * c64 + n], a, pf[m][k][0], pf[m][k][1]);
                if constexpr (kTwoTerms)
                  mma16816<MBF>(o[m][4 * c64 + n], a, pr[m][k][0], pr[m][k][1]);
              }
            }
          } else {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = lds128(vk + (uint32_t)j * row_bytes + 128u * c64);
            if (__builtin_expect(edge, 0)) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!(live[k] >> j & 1u)) w[j] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint32_t x0 = n == 0 ? w[0].x : n == 1 ? w[0].y : n == 2 ? w[0].z : w[0].w;
              const uint32_t x1 = n == 0 ? w[1].x : n == 1 ? w[1].y : n == 2 ? w[1].z : w[1].w;
              const uint32_t x2 = n == 0 ? w[2].x : n == 1 ? w[2].y : n == 2 ? w[2].z : w[2].w;
              const uint32_t x3 = n == 0 ? w[3].x : n == 1 ? w[3].y : n == 2 ? w[3].z : w[3].w;
              const uint32_t a[4] = {__byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x7632),
                                     __byte_perm(x2, x3, 0x5410), __byte_perm(x2, x3, 0x7632)};
#pragma unroll
              for (int m = 0; m < NT; ++m) {
                mma16816<MBF>(o[m][4 * c64 + n], a, pf[m][k][0], pf[m][k][1]);
                if constexpr (kTwoTerms)
                  mma16816<MBF>(o[m][4 * c64 + n], a, pr[m][k][0], pr[m][k][1]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sBar + 8u * (kCaMaxSlots + slot));
      if (++slot == (uint32_t)p.NS) {
        slot = 0;
        ph ^= 1u;
      }
    }
    // A wait that ran out in one warp ends the piece for all that join rows
    // with it: nothing more is written.
    ok = together(ok);
    if (!ok) break;

    // ---- the unit's (or piece's) rows: join the warps of a head, write.
    // Warp area [8 rows][64 columns] in shared memory, a tile and 64 columns
    // at a time; with one warp per head only that warp takes part.
    const long long pslot = 2ll * blockIdx.x + (d0.y >> 1);
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) L[m][h] += __shfl_xor_sync(0xffffffffu, L[m][h], x);
    auto join = [&]() {
      if (p.KW == 1) __syncwarp();
      else named_bar_sync(1u + (uint32_t)hl, 32u * (uint32_t)p.KW);
    };
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      if (g == 0) {
        s_ml[warp * 8 + 2 * t] = make_float2(M[m][0], L[m][0]);
        s_ml[warp * 8 + 2 * t + 1] = make_float2(M[m][1], L[m][1]);
      }
#pragma unroll
      for (int c64 = 0; c64 < D / 64; ++c64) {
        // Rows 2 t and 2 t + 1, columns 8 g .. 8 g + 7 of the chunk, turned by
        // the row so that the 16-byte stores of 8 lanes fall into all banks.
        float* area = scratch + warp * 8 * 64;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = (8 * g + 4 * j + 16 * (t & 1) + 4 * (t >> 1)) & 63;
            const float(&x)[4] = o[m][4 * c64 + 2 * j], (&y)[4] = o[m][4 * c64 + 2 * j + 1];
            *reinterpret_cast<float4*>(area + (2 * t + h) * 64 + col) =
                make_float4(x[h], x[2 + h], y[h], y[2 + h]);
          }
        join();
        // Four rows a warp at a time, 8 columns a lane.
        for (int r = 4 * kw + (lane >> 3); r < 8; r += 4 * p.KW) {
          const int gr = row0 + m * 8 + r;  // row of the sequence
          const int i = p.div_g.div(gr);
          if (i >= E) continue;
          const int qh = head * p.G + (gr - i * p.G);
          float xs = -INFINITY;
          if (!cut && p.sinks != nullptr) xs = __ldg(p.sinks + qh) * kLog2e;
          else if (!cut && p.smooth) xs = 0.f;
          const int turn = 16 * ((r >> 1) & 1) + 4 * (r >> 2);
          const int col0 = (8 * (lane & 7) + turn) & 63, col1 = (8 * (lane & 7) + 4 + turn) & 63;
          float mf = -1e30f;
          for (int w = 0; w < p.KW; ++w) mf = fmaxf(mf, s_ml[(w * p.HPC + hl) * 8 + r].x);
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f;
          for (int w = 0; w < p.KW; ++w) {
            const int wr = (w * p.HPC + hl) * 8 + r;
            const float2 ml = s_ml[wr];
            const float f = ex2(ml.x - mf);
            const float4 x = *reinterpret_cast<const float4*>(scratch + wr * 64 + col0);
            const float4 y = *reinterpret_cast<const float4*>(scratch + wr * 64 + col1);
            v[0] = fmaf(x.x, f, v[0]), v[1] = fmaf(x.y, f, v[1]);
            v[2] = fmaf(x.z, f, v[2]), v[3] = fmaf(x.w, f, v[3]);
            v[4] = fmaf(y.x, f, v[4]), v[5] = fmaf(y.y, f, v[5]);
            v[6] = fmaf(y.z, f, v[6]), v[7] = fmaf(y.w, f, v[7]);
            l = fmaf(ml.y, f, l);
          }
          const int col = 64 * c64 + 8 * (lane & 7);
          if (cut) {
            const long long pr = pslot * (p.HPC * RT) + hl * RT + m * 8 + r;
            float4* dst = reinterpret_cast<float4*>(p.part_o + pr * D + col);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            if (c64 == 0 && (lane & 7) == 0)
              *reinterpret_cast<float2*>(p.part_ml + pr * 2) = make_float2(mf, l);
          } else {
            // With the sink above the keys the reference moves to it.
            const bool any = l > 0.f;
            const float mm = fmaxf(mf - kBias, xs), f = ex2(mf - kBias - mm);
            const float den = fmaf(l, f, ex2(xs - mm));
            const float inv = any ? f / den : 0.f;
            const long long row = (long long)(cu0 + i) * p.Hq + qh;
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + col) = make_uint4(
                pack2<BF16>(v[0] * inv, v[1] * inv), pack2<BF16>(v[2] * inv, v[3] * inv),
                pack2<BF16>(v[4] * inv, v[5] * inv), pack2<BF16>(v[6] * inv, v[7] * inv));
            if (c64 == 0 && (lane & 7) == 0 && p.lse != nullptr)
              p.lse[row] = any ? (mm + log2f(den)) * kLn2 : -INFINITY;
          }
        }
        join();
      }
    }
  }
  if (!ok && lane == 0) ca_mark(p, 1);
}

// Joins the partials of the units that share boundaries cut: with mf the
// largest reference (the sink's included),
//   out = sum O_s 2^(M_s - mf) / (sum L_s 2^(M_s - mf) + 2^(x - mf)).
// A CTA that gave up (GQA_DEV_TIMEOUT) leaves units without an entry and pieces
// without partials: then nothing is joined, since the workspace holds anything
// there.  An entry out of range, which only another writer of the workspace can
// leave, raises GQA_DEV_BAD_METADATA and is passed over.
// blockIdx.x walks the units, blockIdx.y the rows of a unit that exist.  A unit
// of few pieces takes a warp per row (per two rows at d = 64), the rows dealt to
// the blocks first; one of many (a long sequence over all CTAs) the whole block,
// its warps (half warps at d = 64) sharing the pieces.  Bound by latency: the
// loads of 4 pieces go out at once.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) cache_merge_kernel(const __grid_constant__ CacheAttnParams p,
                                                          int RT, float bias) {
  constexpr int kLanes = D == 64 ? 16 : 32;  // lanes of a row, 4 values each (twice at d = 256)
  constexpr int kRows = 32 / kLanes, kVec = D / (4 * kLanes);
  __shared__ float4 s_o[8][kRows][D / 4];
  __shared__ float2 s_ml[8][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / kLanes, ll = lane % kLanes;
  grid_dep_launch_dependents();
  grid_dep_wait();
  // The marks, the count and the block's first entry at once (the grid has no
  // more blocks than there are entries).
  bool gone = false;
  for (int o = threadIdx.x; o < (p.ctas + 15) / 16; o += 256) {
    const int4 x = __ldcg(reinterpret_cast<const int4*>(p.head) + 1 + o);
    gone |= (x.x | x.y | x.z | x.w) != 0;
  }
  const int n_units = __ldcg(p.head);
  auto entry = [&](int u, int4& a, int4& b) {
    const int4* hd = reinterpret_cast<const int4*>(p.hdr + 8ll * u);
    a = __ldcg(hd);
    b = __ldcg(hd + 1);
  };
  int4 h4, g4;
  entry(blockIdx.x, h4, g4);
  if (__syncthreads_or(gone)) return;
  const int rows = p.HPC * RT;
  for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
    if (u != blockIdx.x) entry(u, h4, g4);
    const int np = h4.x + 1;
    if (np == 1) continue;
    const int c0 = h4.y, r0 = h4.z, h0 = h4.w, cu0 = g4.x, E = g4.y;
    if (c0 < 0 || h4.x < 0 || (unsigned)c0 + (unsigned)h4.x >= (unsigned)p.ctas || h0 < 0 ||
        h0 > p.Hkv - p.HPC || cu0 < 0 || E < 0 || cu0 > p.total_q - E || r0 < 0 || r0 >= E * p.G) {
      if (threadIdx.x == 0) atomicOr(p.status, 2u);
      continue;
    }
    const bool wide = np > 8;  // the whole block per row
    const int per_head = min(RT, E * p.G - r0), live = p.HPC * per_head;
    const int groups = wide ? live : (live + kRows - 1) / kRows;
    const int step = wide ? gridDim.y : gridDim.y * 8;
    for (int x = wide ? blockIdx.y : warp * gridDim.y + blockIdx.y; x < groups; x += step) {
      const int row_x = wide ? x : x * kRows + sub;
      const bool on = row_x < live;
      const int lr = on ? row_x : 0;  // lanes past the last row repeat the first
      const int hl = lr / per_head, rr = lr - hl * per_head, r = hl * RT + rr;
      const int gr = r0 + rr, i = p.div_g.div(gr);
      const int qh = (h0 + hl) * p.G + (gr - i * p.G);
      float xs = -INFINITY;
      if (p.sinks != nullptr) xs = __ldg(p.sinks + qh) * kLog2e;
      else if (p.smooth) xs = 0.f;
      const int ds = wide ? 8 * kRows : 1;
      // Piece s of the unit: slot 2 c + 1 of its first CTA, slot 2 (c + s) after.
      float mf = -1e30f, l = 0.f;
      float4 acc[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](int k, const float4& v, float f) {
        acc[k].x = fmaf(v.x, f, acc[k].x), acc[k].y = fmaf(v.y, f, acc[k].y);
        acc[k].z = fmaf(v.z, f, acc[k].z), acc[k].w = fmaf(v.w, f, acc[k].w);
      };
      for (int s0 = wide ? warp * kRows + sub : 0; s0 < np; s0 += 4 * ds) {
        float2 ml[4];
        float4 v[4][kVec];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = s0 + j * ds;
          ml[j] = make_float2(-1e30f, 0.f);
#pragma unroll
          for (int k = 0; k < kVec; ++k) v[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (s < np) {
            const long long a = (2ll * (c0 + s) + (s == 0 ? 1 : 0)) * rows + r;
            ml[j] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + a);
#pragma unroll
            for (int k = 0; k < kVec; ++k)
              v[j][k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + a * D) + kLanes * k + ll);
          }
        }
        const float m = fmaxf(fmaxf(mf, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
        const float f0 = ex2(mf - m);
        l *= f0;
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          acc[k] = make_float4(acc[k].x * f0, acc[k].y * f0, acc[k].z * f0, acc[k].w * f0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float f = ex2(ml[j].x - m);
          l = fmaf(ml[j].y, f, l);
#pragma unroll
          for (int k = 0; k < kVec; ++k) add(k, v[j][k], f);
        }
        mf = m;
      }
      if (wide) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kVec; ++k) s_o[warp][sub][kLanes * k + ll] = acc[k];
        if (ll == 0) s_ml[warp][sub] = make_float2(mf, l);
        __syncthreads();
        if (warp == 0 && sub == 0) {
          mf = -1e30f;
          for (int w = 0; w < 8 * kRows; ++w) mf = fmaxf(mf, s_ml[w / kRows][w % kRows].x);
          l = 0.f;
#pragma unroll
          for (int k = 0; k < kVec; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int w = 0; w < 8 * kRows; ++w) {
            const float2 y = s_ml[w / kRows][w % kRows];
            const float f = ex2(y.x - mf);
            l = fmaf(y.y, f, l);
#pragma unroll
            for (int k = 0; k < kVec; ++k) add(k, s_o[w / kRows][w % kRows][kLanes * k + ll], f);
          }
        }
      }
      if (on && (!wide || (warp == 0 && sub == 0))) {
        const bool any = l > 0.f;
        const float mm = fmaxf(mf - bias, xs), f = ex2(mf - bias - mm);
        const float den = fmaf(l, f, ex2(xs - mm));
        const float inv = any ? f / den : 0.f;
        const long long row = (long long)(cu0 + i) * p.Hq + qh;
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + 4 * (kLanes * k + ll)) =
              make_uint2(pack2<BF16>(acc[k].x * inv, acc[k].y * inv),
                         pack2<BF16>(acc[k].z * inv, acc[k].w * inv));
        if (ll == 0 && p.lse != nullptr) p.lse[row] = any ? (mm + log2f(den)) * kLn2 : -INFINITY;
      }
      __syncwarp();
    }
  }
}

}  // namespace gqa
