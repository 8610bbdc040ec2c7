// backward.h -- the gradient of the prefill attention: what its kernels share.
//
// Mathematics.  With s = scale <q_i, k_j> over the kept pairs, lse and out of
// the forward pass, and D_i = <dout_i, out_i> - dlse_i,
//   p_ij = e^(s_ij - lse_i)            ds_ij = p_ij (<dout_i, v_j> - D_i)
//   dv_j = sum_i p_ij dout_i           dk_j = scale sum_i ds_ij q_i
//   dq_i = scale sum_j ds_ij k_j       dsink_h = -sum_i e^(sink_h - lse_ih) D_ih
// Four kernels in stream order:
//   scan  (1 CTA)  checks the metadata and counts the sequences' tiles;
//   prep           D and -lse log2(e) per query row, the sinks' partial sums; one
//                  more CTA lists the work units;
//   main           the products (backward_kernel.cuh);
//   join           sums of cut units, and the sinks' gradient.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace gqa {

// A work unit holds 128 rows of one side still (A) and streams the other side
// (B) past them in tiles of N rows: queries still and keys streamed for dq,
// keys still and queries streamed for dk and dv.  At d = 256 the tensor memory
// holds one accumulator, so dk and dv are units of their own.
enum BwdKind { kBwdQ = 0, kBwdKV = 1, kBwdK = 2, kBwdV = 3 };
constexpr int kBwdTwo = 4;  // added to the kind in a record: P and dS in two 16-bit terms

struct BwdUnit {      // one record of the plan, the same for every KV head
  int kind, n;        // n: tiles streamed (0: the rows get zeros)
  int a_base, a_off;  // the sequence's first row on A's side, A's first row in it
  int a_valid;        // rows of A that exist
  int b_base, b_off;  // the same of B's first tile
  int b_len;          // rows on B's side of the sequence
  int P, E;           // prefix keys, new tokens
  int slot;           // -1: writes the result; else fp32 partial `slot`
  int stat;           // the sequence's first row in the arrays of row statistics
  int seq;
  int g;              // the KV head, once a CTA takes the record
  int lo_max, hi_min; // of the columns that A's rows keep: the last first one, the first last one
};
static_assert(sizeof(BwdUnit) == 64, "copied as 16 words");

struct BwdJoin {  // a cut unit: its parts are slots slot .. slot + parts - 1
  int kind, a_base, a_off, a_valid, slot, parts, seq, pad;
};

// Words of the plan's header.
enum { kBwdUnits = 0, kBwdJoins = 1, kBwdNext = 2, kBwdFailed = 3, kBwdQTiles = 4, kBwdKTiles = 5, kBwdHdr = 64 };

struct BwdParams {
  CUtensorMap a_q, a_do, a_k, a_v;  // boxes of 128 rows
  CUtensorMap b_q, b_do, b_k, b_v;  // boxes of N rows
  const int32_t* cu;
  const int32_t* pre;
  const int32_t* kvi;
  const void* v;
  const void* out;
  const void* dout;
  const float* lse;
  const float* dlse;
  const float* sinks;
  void* dq;
  void* dk;
  void* dv;
  float* dsinks;
  // workspace
  int32_t* hdr;
  BwdUnit* units;
  BwdJoin* joins;
  int32_t* qtile0;    // [B+1] first 128-row query tile of each sequence (of one KV head)
  int32_t* ktile0;    // [B+1] first 128-key tile
  float* nlse;        // [Hkv][stat_rows] -lse log2(e) (+ 15 in f16); -inf: no such row
  float* nd;          // [Hkv][stat_rows] -D
  float* sink_part;   // [Hq][max_qtiles]
  float* row_o2;      // f16: [Hkv][stat_rows] |dout|^2
  uint2* tile_most;   // f16: [Hkv][max_qtiles] largest |dout|^2 and |D| of a query tile (bits of floats)
  unsigned int* most_v; // f16: [B][Hkv] largest |v|^2 of the sequence
  float* part;        // [slot][Hkv][accumulators][d/4][128][4]
  unsigned int* status;
  long long stat_rows;
  int max_qtiles, max_units, max_slots, max_joins;
  int num_seqs, total_q, total_kv;
  int Hq, Hkv, G, log_G;
  int d, N;             // N: rows of a streamed tile
  int reach;            // the window, or 2^30: more than any length
  int ctas;
  float scale, scale_log2;
  unsigned long long timeout_ns;
};

constexpr float kBwdBias = 15.f;  // f16: p is held times 2^15, so that it keeps its bits down to 2^-29

// Rows of a streamed tile: 64 at d = 256, where 128 would not fit in shared memory,
// and at d = 64, where two CTAs an SM overlap each other's waits.
__host__ __device__ constexpr int bwd_n(int D) { return D == 128 ? 128 : 64; }
__host__ __device__ constexpr int bwd_per_sm(int D) { return D == 64 ? 2 : 1; }
__host__ __device__ constexpr int bwd_accs(int D) { return D == 256 ? 1 : 2; }

cudaError_t launch_bwd_d64(const BwdParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_bwd_d128(const BwdParams& p, bool bf16, cudaStream_t st);
cudaError_t launch_bwd_d256(const BwdParams& p, bool bf16, cudaStream_t st);

// Rows of B that row `a` of a sequence on A's side keeps, both counted in their
// sequence: keys of a packed query row, or packed query rows of a key.
__device__ __forceinline__ void bwd_bounds(bool queries, int a, int P, int E, int log_G, int reach, int& lo,
                                           int& hi) {
  if (queries) {
    hi = P + (a >> log_G);
    lo = hi - reach + 1;
  } else {
    lo = max(a - P, 0) << log_G;
    const int i = a - P;  // key a's token, if it is a new one
    hi = ((i >= E - reach ? E : max(i + reach, 0)) << log_G) - 1;
  }
}

// dS = P (dP - D) is held in f16 times 2^k, with k from a bound of |dP - D| that
// leaves a factor of two to the largest f16: |dP_ij| <= |dout_i| |v_j|.  A dq unit has a
// k for each query row, a dk unit one for the query rows that it streams.
__device__ __forceinline__ int bwd_exponent(float o2, float dm, float v2) {
  const float bound = sqrtf(o2) * sqrtf(v2) + dm;
  if (!(bound > 0.f) || !(bound < 3e38f)) return 0;  // all zeros, or not finite
  int e;
  frexpf(bound, &e);  // bound < 2^e
  return max(-100, min(100, 14 - e));
}

}  // namespace gqa
