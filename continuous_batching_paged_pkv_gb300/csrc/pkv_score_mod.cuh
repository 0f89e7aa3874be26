// Modified scores (pkv_score_mod): what a row sees and what its scores become.
#pragma once

#include <cuda_bf16.h>
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
  __device__ __forceinline__ float operator()(float x) const {
    return fmaf(c2, rcp_approx(1.f + ex2_approx(__fmul_rn(x, k))), c);
  }
  // Two scores, with the same results.
  __device__ __forceinline__ void both(float &x0, float &x1) const {
    float e0, e1;
    mul2(e0, e1, x0, x1, k, k);
    e0 = ex2_approx(e0), e1 = ex2_approx(e1);
    add2(e0, e1, 1.f, 1.f);
    fma2(x0, x1, rcp_approx(e0), rcp_approx(e1), c2, c2, c, c);
  }
};

// Variants of the chunk kernels: plain, or modified scores with or without the
// cap and the distance bias (every modified variant masks each row's interval).
constexpr int kModNone = 0, kModMask = 1, kModCap = 2, kModBias = 4;

// A bias without a cap is added by the tensor core. Within a tile whose first key
// is kt0 it is slope (j - kt0) - slope (p - kt0): the second part is one number
// per row and tile, the first an inner product of three bf16 numbers that add up
// to slope / scale in fp32's 24 bits with j - kt0 three times (0 .. 127, exact in
// bf16). So the product Q K^T takes one more step of 16 columns, over operands that
// a CTA writes once, and a softmax thread does nothing for the bias. Added to every
// score in the softmax threads instead, one addition each: 2048 rows at context
// 8192, head_dim 128, 238 us; 8192 causal rows of 16 heads of 64, 260 us.
__host__ __device__ constexpr bool ramp_mode(int mode) { return (mode & (kModCap | kModBias)) == kModBias; }

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

__device__ __forceinline__ uint32_t shift_left(uint32_t x, int n) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(n));
  return r;
}

// Operands of that step, without swizzle: groups of 8 rows 256 B apart, their two
// 16-byte halves 128 B apart.
constexpr int kRampBytes = 128 * 32;

__device__ __forceinline__ uint64_t ramp_desc(const uint8_t *rows) { return smem_desc_noswz(smem_addr(rows), 128, 256); }

__device__ __forceinline__ void store_ramp_row(uint8_t *rows, int r, uint4 v) {
  uint8_t *dst = rows + (r >> 3) * 256 + (r & 7) * 16;
  *reinterpret_cast<uint4 *>(dst) = v;
  *reinterpret_cast<uint4 *>(dst + 128) = make_uint4(0, 0, 0, 0);
}

// Row r of Q's part: the head's slope in score units.
__device__ __forceinline__ void store_ramp_slope(uint8_t *rows, int r, float x) {
  const float hi = __bfloat162float(__float2bfloat16_rn(x));
  const float mid = __bfloat162float(__float2bfloat16_rn(x - hi));
  store_ramp_row(rows, r, make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(x - hi - mid, 0.f), 0, 0));
}

// Row r of K's part: the key's place in its tile.
__device__ __forceinline__ void store_ramp_key(uint8_t *rows, int r, int key) {
  const float k = static_cast<float>(key);
  store_ramp_row(rows, r, make_uint4(pack_bf16x2(k, k), pack_bf16x2(k, 0.f), 0, 0));
}

__device__ __forceinline__ float ramp_slope(const StepArgs &a, int head) {
  return __ldg(a.alibi_slopes + head) * 1.4426950408889634f / a.scale_log2;
}

// Scores outside [first, last] of the tile's 128 keys become -inf: a bit per key,
// 32 at a time, since two comparisons a score cost more than its exponent
// (documents of ~1000 tokens, 8192 rows, 16 heads of 64: 75 us, now 58 us).
__device__ __forceinline__ void mask_tile(uint32_t (&sv)[4][32], int first, int last) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    // shifts by 32 or more give 0
    const uint32_t seen = shift_left(~0u, max(first - c * 32, 0)) & ~shift_left(~0u, max(last + 1 - c * 32, 0));
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(seen & (1u << i))) sv[c][i] = 0xff800000u;
  }
}

__device__ __forceinline__ float score(const uint32_t (&sv)[4][32], int i) {
  return __uint_as_float(sv[i >> 5][i & 31]);
}

// Largest of a row's 128 scores, or the smallest: three-input maxima, four independent chains.
template <bool MIN = false>
__device__ __forceinline__ float tile_max(const uint32_t (&sv)[4][32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 128; i += 2)
    m[(i >> 1) & 3] = MIN ? max3(m[(i >> 1) & 3], -score(sv, i), -score(sv, i + 1))
                          : max3(m[(i >> 1) & 3], score(sv, i), score(sv, i + 1));
  const float r = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  return MIN ? -r : r;
}

// Modified scores in a chunk kernel's softmax thread: one row, tile by tile.
// The scores of a tile arrive as raw products; top() gives a reference for the
// tile's running max (log2 units) and exponents() the pairs 2^x is taken of.
//
// Without a cap a tile's unseen scores become -inf as they are, and the bias is in
// the scores but for `near`. With a cap a tile stays raw where every row of the warp
// sees it whole (most tiles). The cap is then y P(y^2) with y = raw r, |y| <= 0.55 and P of degree 3, fitted here
// to the least largest error of y P(y^2) (2^-21.5 in fp32 arithmetic), its
// coefficients scaled so that a score costs 5 operations, the last of which also
// subtracts the reference (2^x and 1/x would be two SFU operations of each score
// beside the softmax's own 2^x); a bias is one more. Only the segment's own rows decide. The reference is then the
// largest raw score's logit plus the largest bias of a key the row sees: an upper
// bound, at most kSpread above the row's largest logit. Weights then start as low
// as 2^-80 instead of 1, which fp32 and bf16 hold as exactly; only weights under
// 2^-46 of the row's largest are lost. Every other tile has its logits written
// out, masked, and their maximum taken.
//
// Capped 2048-row chunk at context 8192, head_dim 128: 379 us with 2^x and 1/x for
// every score, 373 us with the cubic written out first, 292 us fused (270 us with two warpgroups).
//
// Products that a sum follows are rounded explicitly: the compiler must not fuse
// them in one variant and not in another, or a row's last bits would depend on
// whether decode rows share the step.
template <int MODE>
struct TileScores {
  static constexpr int kKeys = 128;
  static constexpr bool kRamp = ramp_mode(MODE);  // the scores arrive with their bias, but for the row's part of it
  static constexpr bool kCap = (MODE & kModCap) != 0, kBias = (MODE & kModBias) != 0 && !kRamp;
  static constexpr float kSpread = 80.f;  // log2 units
  Cap cap;
  float sl2, slope;  // scale and bias per key in log2 units
  float r, p0, p1, p2, p3;
  uint32_t rows;     // the warp's lanes with a row of the segment
  bool poly, flat;   // warp-uniform: the cap's r leaves the coefficients in range; a tile's added biases stay within kSpread
  struct Tile {  // what top() found of a tile
    bool raw;    // warp-uniform
    float near;  // bias of its first key (0 without a bias)
  };

  // `stored`: the row is one of the segment's. The queries of the others are whatever follows in the
  // packed axis, so their scores have no say in how the warp caps a tile.
  __device__ __forceinline__ TileScores(const StepArgs &a, int head, bool stored)
      : cap(kCap ? a.softcap : 0.f), sl2(a.scale_log2), slope(0.f), r(0.f),
        rows(kCap ? __ballot_sync(0xffffffffu, stored) : 0u) {
    if constexpr (kBias || kRamp) slope = __ldg(a.alibi_slopes + head) * 1.4426950408889634f;
    flat = !kBias || __all_sync(0xffffffffu, fabsf(slope) * (kKeys - 1) <= kSpread);
    if constexpr (kCap) {
      r = sl2 / cap.c;
      poly = r > 0x1p-17f && r < 0x1p17f;
      const float u = r * r, c = cap.c * r;
      p0 = 0.9999952912330627f * c;
      p1 = -0.3331194519996643f * c * u;
      p2 = 0.13069017231464386f * c * u * u;
      p3 = -0.04152349755167961f * c * u * u * u;
    }
  }

  // `away`: position of the row minus the tile's first key; keys [first, last] of the tile are the row's.
  __device__ __forceinline__ float top(uint32_t (&sv)[4][32], int away, int first, int last, Tile &tile) const {
    constexpr uint32_t kAll = 0xffffffffu;
    tile.raw = true;
    tile.near = 0.f;
    const bool inside = __all_sync(kAll, first <= 0 && last >= kKeys - 1);
    if constexpr (kRamp) {
      tile.near = __fmul_rn(-slope, static_cast<float>(away));
      // keys past the row's own position: 2 slope (j - p) too much
      if (__any_sync(kAll, min(last, kKeys - 1) > away)) {
        const float twice = -2.f * slope / sl2, from = static_cast<float>(away);
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          sv[i >> 5][i & 31] = __float_as_uint(fmaf(twice, fmaxf(static_cast<float>(i) - from, 0.f), score(sv, i)));
      }
      if (!inside) mask_tile(sv, first, last);
      return fmaf(tile_max(sv), sl2, tile.near);
    } else if constexpr (!kCap) {
      if (!inside) mask_tile(sv, first, last);
      return tile_max(sv) * sl2;
    } else {
      // rows that see keys past their own position take the distance's absolute value
      const bool ahead = kBias && __any_sync(kAll, min(last, kKeys - 1) > away);
      float mx = 0.f;
      bool raw = inside && poly && flat && !ahead;
      const float near = kBias ? __fmul_rn(-slope, static_cast<float>(away)) : 0.f;
      tile.near = near;
      if (raw) {
        mx = tile_max(sv);
        raw = (__ballot_sync(kAll, fmaxf(mx, -tile_max<true>(sv)) * r > 0.55f) & rows) == 0;
      }
      tile.raw = raw;
      if (raw) {
        const float t = cap(__fmul_rn(mx, sl2));
        return kBias ? t + fmaxf(near, fmaf(slope, kKeys - 1.f, near)) : t;
      }
      const float from = static_cast<float>(away);
      float b0 = 0.f, b1 = 0.f;
#pragma unroll
      for (int i = 0; i < kKeys; i += 2) {
        float x0 = cap(score(sv, i) * sl2), x1 = cap(score(sv, i + 1) * sl2);
        if constexpr (kBias) {
          if (ahead) {
            b0 = -slope * fabsf(from - static_cast<float>(i));
            b1 = -slope * fabsf(from - static_cast<float>(i + 1));
          } else {
            bias(b0, b1, i, near);
          }
          add2(x0, x1, b0, b1);
        }
        sv[i >> 5][i & 31] = __float_as_uint(x0);
        sv[(i + 1) >> 5][(i + 1) & 31] = __float_as_uint(x1);
      }
      if (!inside) mask_tile(sv, first, last);
      return tile_max(sv);
    }
  }

  // Biases (plus `first`) of keys i and i + 1, called for i = 0, 2, 4, ...: two
  // products every eight keys, packed additions in between (three roundings).
  __device__ __forceinline__ void bias(float &b0, float &b1, int i, float first) const {
    if (i % 8 == 0) {
      b0 = fmaf(slope, static_cast<float>(i), first);
      b1 = fmaf(slope, static_cast<float>(i + 1), first);
    } else {
      add2(b0, b1, 2.f * slope, 2.f * slope);
    }
  }

  // x0, x1: exponents of keys i and i + 1 (i = 0, 2, 4, ...) less the reference
  // (nm = -reference); b0, b1 carry the biases from one call to the next.
  template <bool RAW>
  __device__ __forceinline__ void exponents(float &x0, float &x1, float &b0, float &b1, const uint32_t (&sv)[4][32],
                                            int i, float nm, float near) const {
    const float s0 = score(sv, i), s1 = score(sv, i + 1);
    if constexpr (RAW && kBias)
      bias(b0, b1, i, near + nm);
    else
      b0 = b1 = nm;
    if constexpr (RAW && kCap) {
      float u0, u1, f0 = p3, f1 = p3;
      mul2(u0, u1, s0, s1, s0, s1);
      fma2(f0, f1, f0, f1, u0, u1, p2, p2);
      fma2(f0, f1, f0, f1, u0, u1, p1, p1);
      fma2(f0, f1, f0, f1, u0, u1, p0, p0);
      fma2(x0, x1, s0, s1, f0, f1, b0, b1);
    } else {
      const float unit = RAW ? sl2 : 1.f;
      fma2(x0, x1, s0, s1, unit, unit, b0, b1);
    }
  }

  // Weights of keys c * 32 .. c * 32 + 31 as bf16 pairs, added to the row sum's even and odd parts.
  template <bool RAW>
  __device__ __forceinline__ void weigh(uint32_t (&pk)[16], const uint32_t (&sv)[4][32], int c, float nm, float near,
                                        float &even, float &odd) const {
    float b0, b1;
    if constexpr (kRamp) nm += near;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x0, x1;
      exponents<RAW>(x0, x1, b0, b1, sv, c * 32 + 2 * i, nm, near);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      add2(even, odd, p0, p1);
      pk[i] = pack_bf16x2(p0, p1);
    }
  }
};

}  // namespace
}  // namespace pkv
