// cache_rows.cuh -- what the row operators around the paged cache share: the
// lookup of a row's sequence and page, the e4m3 rows with one power-of-two
// scale, and the rotation angles.
//
// An e4m3 row of a cache (one token, one KV head, d values x_0 .. x_{d-1}) is
// held as d bytes and one byte e + 127 of scale 2^e:
//   e = the least integer with max |x_i| <= 448 * 2^e, at least -60 and 0 for
//       a row of zeros;   value i = e4m3(x_i * 2^-e), rounded to nearest even.
// A power of two keeps the products exact: x_i * 2^-e rounds once, to e4m3,
// and value * 2^e is exact again in bf16 (4 significant bits), so a cache
// read back to bf16 holds what the attention over the e4m3 cache sees.
// e4m3 has the same relative precision over 2^-6 .. 448, so a scale of
// amax / 448 instead would gain at most one bit at its lower end.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace gqa {

// The page table of a call (device arrays but for the counts).
struct PageTable {
  const int32_t* indptr;   // [num_seqs + 1]
  const int32_t* indices;  // [entries]
  int entries, page_size, num_pages, num_seqs;
};

// Scale exponent of an e4m3 row from the bits of its largest magnitude:
// 448 = 1.75 * 2^8, so amax = m 2^E needs 2^(E - 8) when m <= 1.75, else
// 2^(E - 7).
__device__ __forceinline__ int e4m3_scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0u) return 0;
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -60), 127);
}
// 2^e as fp32, -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// First index i in [0, n) with a[i] > x (n when there is none) for a
// non-decreasing a, found by a converged warp: 32 probes a step, so 1024
// sequences take two dependent loads.  Any array gives an index in [0, n].
__device__ __forceinline__ int warp_upper_bound(const int32_t* a, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;  // the answer lies in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 31) >> 5;
    const int i = lo + (lane + 1) * step - 1;  // last index of this lane's block
    const bool le = i < lo + len && __ldg(a + i) <= x;
    const int c = __popc(__ballot_sync(0xffffffffu, le));  // blocks wholly <= x
    const int at = c * step;
    if (step == 1) return lo + at;
    lo += at;
    len = min(step, len - at);
  }
  return lo;
}

// cos and sin of position * frequency.  `step` is the angle per position in
// units of 2^-64 turns, so position * step modulo 2^64 is the phase within one
// turn, within 2^-33 of it at the farthest position: a product in fp32 would be
// off by 0.06 radians at a million positions, one in fp64 costs the slow units.
// The phase is taken from the nearest quarter turn before it is rounded to
// fp32, which leaves it within 2^-27.8 of a turn (from the nearest whole turn it
// would be 2^-26, three times what the rounding of the cosine is off by), and
// within 2^-31 near the zeros of sine and cosine.
__device__ __forceinline__ float2 phase_cos_sin(int pos, unsigned long long step) {
  const unsigned long long ph = (unsigned long long)(long long)pos * step;
  const uint32_t hi = (uint32_t)(ph >> 32);           // 2^-32 turns
  const uint32_t quarter = (hi + (1u << 29)) >> 30;   // 0 .. 3
  const float half_turns = (float)(int)(hi - (quarter << 30)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  const float x = quarter & 1u ? s : c, y = quarter & 1u ? c : s;
  return make_float2((quarter + 1u) & 2u ? -x : x, quarter & 2u ? -y : y);
}
// The step of a frequency in radians per position: turns modulo one, in 2^-64,
// off by one unit at most for |f| < 2^40.  A double's product with 1 / (2 pi) is
// rounded at 2^-56 turns at one radian, 2^-25 turns at position 2^31, so the 53
// bits of f are multiplied in integers by 128 bits of 1 / (2 pi), and the bits
// from 2^-1 to 2^-64 turns taken out.  (In fp64, with 1 / (2 pi) in two
// doubles and fma: as exact; the gradient of 2047 rows 10.5 us, here 9.5.)
__device__ __forceinline__ unsigned long long phase_step(double f) {
  constexpr unsigned long long kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // 2^128 / (2 pi)
  const long long bits = __double_as_longlong(f);
  const int ex = (int)(bits >> 52) & 2047;  // f = m * 2^(ex - 1075)
  const unsigned long long m = ((unsigned long long)bits & ((1ull << 52) - 1)) | (ex ? 1ull << 52 : 0);
  const unsigned long long mid = m * kHi, p1 = mid + __umul64hi(m, kLo);
  const unsigned long long p2 = __umul64hi(m, kHi) + (p1 < mid ? 1 : 0);
  const int t = max(1075 - ex, 1);  // m * (kHi, kLo) / 2^(64 + t), of which p1 and p2 count
  const unsigned long long step = t < 64    ? p1 >> t | p2 << (64 - t)
                                  : t < 128 ? p2 >> (t - 64)
                                            : 0ull;
  return bits < 0 ? 0ull - step : step;
}

}  // namespace gqa
