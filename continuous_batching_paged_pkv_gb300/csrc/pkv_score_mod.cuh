// Modified scores (pkv_score_mod): what a row sees and what its scores become.
#pragma once

#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

// Keys [lo, hi) that a row at position p of a slot of L keys sees, its key_begin and key_end as given
// (anything where the arrays are not); lo >= hi for none.
__device__ __forceinline__ void visible_keys(const StepArgs &a, int begin, int end, int p, int L, int &lo, int &hi) {
  lo = a.key_begin ? max(0, begin) : 0;
  if (a.window > 0) lo = max(lo, p - a.window + 1);
  hi = a.key_end ? min(L, end) : p + 1;
}

// The same for packed row `row`; lo = hi = 0 for none.
__device__ __forceinline__ void row_sees(const StepArgs &a, int64_t row, int p, int L, int &lo, int &hi) {
  visible_keys(a, a.key_begin ? __ldg(a.key_begin + row) : 0, a.key_end ? __ldg(a.key_end + row) : 0, p, L, lo, hi);
  if (lo >= hi) lo = hi = 0;
}

// cap * tanh(s / cap) in log2 units: with t = tanh(y) = 1 - 2 / (1 + e^2y) and
// x = s log2(e), it is C - 2 C / (1 + 2^(x k)), C = cap log2(e), k = 2 / cap.
// Two SFU operations; t is within 2^-21 of the tanh (2^x: 2^-22 of its value,
// at most a quarter of that in t; 1/x: 2^-23; the difference: 2^-24), and 1 and
// -1 come out exactly for large |s|, infinities included.
struct Cap {
  bool on;
  float k, c, c2;
  __device__ __forceinline__ explicit Cap(float softcap)
      : on(softcap > 0.f), k(2.f / softcap), c(softcap * 1.4426950408889634f), c2(-2.f * c) {}
  __device__ __forceinline__ float operator()(float x) const { return fmaf(c2, rcp_approx(1.f + ex2_approx(x * k)), c); }
};

// Variants of the chunk kernels: plain, or modified scores with or without the
// cap and the distance bias (every modified variant masks each row's interval).
constexpr int kModNone = 0, kModMask = 1, kModCap = 2, kModBias = 4;

inline int mode_of(const StepArgs &a) {
  return a.modified ? kModMask | (a.softcap > 0.f ? kModCap : 0) | (a.alibi_slopes ? kModBias : 0) : kModNone;
}

// What the rows of a chunk tile (or tile pair) see, reduced over the CTA into
// `u` (shared: smallest first key, largest end; INT32_MAX and 0 for none).
// Every thread of the CTA calls it; rows [0, count) are packed row row0 + i at
// position pos0 + i of a slot of L keys.
__device__ __forceinline__ void rows_see(const StepArgs &a, int64_t row0, int pos0, int count, int L, int *u) {
  if (threadIdx.x == 0) {
    u[0] = INT32_MAX;
    u[1] = 0;
  }
  __syncthreads();
  for (int i0 = 0; i0 < count; i0 += blockDim.x) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    int lo = 0, hi = 0;
    if (i < count) row_sees(a, row0 + i, pos0 + i, L, lo, hi);
    const int first = __reduce_min_sync(0xffffffffu, lo < hi ? lo : INT32_MAX);
    const int end = __reduce_max_sync(0xffffffffu, hi);
    if ((threadIdx.x & 31) == 0 && first < end) {
      atomicMin(u, first);
      atomicMax(u + 1, end);
    }
  }
  __syncthreads();
}

// One tile's scores of a row (raw products) become logits in log2 units.
// `away`: position of the row minus the tile's first key; `ahead`: the row may
// see keys past its own position, so the distance needs its absolute value.
template <int MODE>
__device__ __forceinline__ void tile_logits(uint32_t (&sv)[4][32], float sl2, const Cap &cap, float slope, int away,
                                            bool ahead) {
  const float kk = sl2 * cap.k;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float x = __uint_as_float(sv[c][i]);
      if constexpr ((MODE & kModCap) != 0)
        x = fmaf(cap.c2, rcp_approx(1.f + ex2_approx(x * kk)), cap.c);
      else
        x *= sl2;
      sv[c][i] = __float_as_uint(x);
    }
  if constexpr ((MODE & kModBias) != 0) {
    const float from = static_cast<float>(away);
    if (ahead) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          sv[c][i] = __float_as_uint(
              fmaf(-slope, fabsf(from - static_cast<float>(c * 32 + i)), __uint_as_float(sv[c][i])));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          sv[c][i] =
              __float_as_uint(fmaf(-slope, from - static_cast<float>(c * 32 + i), __uint_as_float(sv[c][i])));
    }
  }
}

// Scores outside [first, last] of the tile's 128 keys become -inf.
__device__ __forceinline__ void mask_tile(uint32_t (&sv)[4][32], int first, int last) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c * 32 + i < first || c * 32 + i > last) sv[c][i] = 0xff800000u;
}

}  // namespace
}  // namespace pkv
