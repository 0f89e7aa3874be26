// Attention with modified scores, one warp per (row, q head): the plain
// statement of pkv_score_mod over any pool, key by key.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "pkv_score_mod.cuh"

namespace pkv {
namespace {

// The N values at head_dim element e of pool row `prow` (D elements a row).
template <int BITS, int N>
__device__ __forceinline__ void load_values(float (&x)[N], const void *pool, const __nv_bfloat16 *scales, int64_t prow,
                                            int D, int e) {
  if constexpr (BITS == 16) {
    const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(pool) + prow * D + e;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(p[i]);
  } else {
    const float d = __bfloat162float(scales[prow * (D / 32) + e / 32]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int c;
      if constexpr (BITS == 8) {
        c = static_cast<const int8_t *>(pool)[prow * D + e + i];
      } else {
        const int byte = static_cast<const uint8_t *>(pool)[(prow * D + e + i) / 2];
        c = static_cast<int32_t>(static_cast<uint32_t>(byte) << (i & 1 ? 24 : 28)) >> 28;
      }
      x[i] = static_cast<float>(c) * d;
    }
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(256) score_mod_kernel(const StepArgs a, const __nv_bfloat16 *k_scales,
                                                        const __nv_bfloat16 *v_scales) {
  constexpr int N = D / 32;  // elements per lane
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t row = w / a.num_q_heads;
  const int h = static_cast<int>(w % a.num_q_heads);
  if (row >= a.total_q) return;
  int s0 = 0, s1 = a.num_seqs;  // the segment with cu[s] <= row < cu[s + 1]
  while (s1 - s0 > 1) {
    const int mid = (s0 + s1) / 2;
    if (a.cu_seqlens_q[mid] <= row)
      s0 = mid;
    else
      s1 = mid;
  }
  const int slot = a.seq_slot[s0], first = a.cu_seqlens_q[s0], n = a.cu_seqlens_q[s0 + 1] - first;
  const bool bad = slot < 0 || slot >= a.max_slots || row >= first + n;
  const int L = bad ? 0 : a.context_lens[slot];
  if (bad || n > L || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size) {
    if (lane == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    return;
  }
  const int p = L - n + static_cast<int>(row - first);
  int lo, hi;
  row_sees(a, row, p, L, lo, hi);
  const int64_t at = (row * a.num_q_heads + h) * D + lane * N;
  float q[N], o[N], sum = 0.f, top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[at + i]);
    o[i] = 0.f;
  }
  const float scale = a.scale_log2 * 0.6931471805599453f;
  const float slope = a.alibi_slopes ? a.alibi_slopes[h] : 0.f;
  const int g = h / a.group;
  for (int j = lo; j < hi; ++j) {
    const int blk = a.block_tables[static_cast<int64_t>(slot) * a.max_blocks_per_slot + j / a.block_size];
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t prow = (static_cast<int64_t>(blk) * a.num_kv_heads + g) * a.block_size + j % a.block_size;
    float k[N], v[N], x = 0.f;
    load_values<BITS>(k, a.k_pool, k_scales, prow, D, lane * N);
    load_values<BITS>(v, a.v_pool, v_scales, prow, D, lane * N);
#pragma unroll
    for (int i = 0; i < N; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    x *= scale;
    if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
    x -= slope * fabsf(static_cast<float>(p - j));
    if (x > top) {
      const float corr = expf(top - x);
      top = x;
      sum *= corr;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] *= corr;
    }
    const float e = expf(x - top);
    sum += e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(e, v[i], o[i]);
  }
  const float inv = hi > lo ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) static_cast<__nv_bfloat16 *>(a.out)[at + i] = __float2bfloat16_rn(o[i] * inv);
}

}  // namespace

cudaError_t launch_score_mod(const StepArgs &a, const void *k_scales, const void *v_scales, int32_t bits,
                             cudaStream_t stream) {
  const int64_t warps = a.total_q * a.num_q_heads;
  const dim3 grid(static_cast<unsigned>((warps + 7) / 8));
  auto *ks = static_cast<const __nv_bfloat16 *>(k_scales);
  auto *vs = static_cast<const __nv_bfloat16 *>(v_scales);
  auto *kernel = bits == 16 ? (a.head_dim == 128 ? score_mod_kernel<128, 16> : score_mod_kernel<64, 16>)
                 : bits == 8 ? (a.head_dim == 128 ? score_mod_kernel<128, 8> : score_mod_kernel<64, 8>)
                             : score_mod_kernel<128, 4>;
  return launch_pdl(kernel, grid, dim3(256), 0, stream, a, ks, vs);
}

}  // namespace pkv
