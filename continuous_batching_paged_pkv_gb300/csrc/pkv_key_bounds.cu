// Bounds of a block's keys: per channel the smallest and the largest value over
// the block's filled rows, for the blocks that a step's cache write touched.
//
//   lo[b][h][d] = min over r <= r_last of k[b][h][r][d],  hi the same with max,
//
// r_last the row of the step's last token in block b. Reduced from the pool
// itself rather than folded into older bounds: rows behind r_last (rejected
// drafts, an earlier owner's keys) then never count, and the result does not
// depend on what was there. A selection of bf16 values: exact.
//
// A warp takes `chunk` consecutive tokens and one kv head, finds the tokens that
// end a block's run, and reduces those blocks one after the other: 16-byte loads,
// a row over head_dim / 8 lanes, several rows per instruction, packed bf16 minima
// and maxima, the lanes of one channel joined by shuffles. Block rows are read once
// (they were written just before, and often come from L2). 24,500 packed tokens,
// 8 heads of 128: 50 MB of keys in 11.0 us, bound by the ramp of one wave of warps
// and then HBM; 64 tokens: 3.1 us, a launch and its chain (rows, store; 11.8 and 3.4
// us where the mapping is read behind the wait for the kernel before).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Eight keys' channels of one row from `lane`'s place in it, as bf16 pairs.
template <int D, int BITS>
__device__ __forceinline__ uint4 load_vector(const void *keys, const __nv_bfloat16 *scales, int64_t row, int c8) {
  if constexpr (BITS == 16) {
    return __ldcg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(keys) + row * D) + c8);
  } else {
    const float d = __bfloat162float(scales[row * (D / 32) + c8 / 4]);
    const int8_t *codes = static_cast<const int8_t *>(keys) + (row * D + c8 * 8) * BITS / 8;
    uint32_t w[4];
    if constexpr (BITS == 8) {
      const uint2 raw = __ldcg(reinterpret_cast<const uint2 *>(codes));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t word = (q < 2 ? raw.x : raw.y) >> (16 * (q & 1));
        w[q] = pack_bf16x2(static_cast<float>(static_cast<int8_t>(word & 0xFF)) * d,
                           static_cast<float>(static_cast<int8_t>((word >> 8) & 0xFF)) * d);
      }
    } else {
      const uint32_t raw = __ldcg(reinterpret_cast<const uint32_t *>(codes));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = pack_bf16x2(static_cast<float>(static_cast<int32_t>(raw << (28 - 8 * q)) >> 28) * d,
                           static_cast<float>(static_cast<int32_t>(raw << (24 - 8 * q)) >> 28) * d);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(64) key_bounds_kernel(const int64_t *__restrict__ slot_mapping, int64_t num_tokens,
                                                         const void *__restrict__ keys,
                                                         const __nv_bfloat16 *__restrict__ scales,
                                                         uint4 *__restrict__ bounds, int64_t pool_rows,
                                                         int32_t block_size, int32_t num_kv_heads, int32_t chunk,
                                                         uint32_t *__restrict__ status) {
  constexpr int V = D / 8;          // 16-byte vectors of a row
  constexpr int R = 32 / V;         // rows per instruction
  constexpr int U = 8;              // loads in flight per lane
  const int lane = threadIdx.x & 31, c8 = lane % V, sub = lane / V;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int64_t t0 = unit / num_kv_heads * chunk;
  const int h = static_cast<int>(unit % num_kv_heads);
  const int count = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(chunk), num_tokens - t0)));
  // lane l: token t0 + l, and whether its block's run ends with it
  int64_t s = -1;
  bool last = false;
  if (lane < count) {
    s = __ldg(slot_mapping + t0 + lane);
    const int64_t next = t0 + lane + 1 < num_tokens ? __ldg(slot_mapping + t0 + lane + 1) : -1;
    if (s >= pool_rows) {
      if (status && h == 0) atomicOr(status, PKV_DEV_BAD_SLOT_MAPPING);
      s = -1;
    }
    last = s >= 0 && (next < 0 || next / block_size != s / block_size);
  }
  grid_dependency_wait();  // the mapping is final when this grid starts, the keys come from earlier work
  launch_dependents();     // as the cache write: everything before this kernel has finished
  for (uint32_t todo = __ballot_sync(kAll, last); todo; todo &= todo - 1) {
    const int64_t at = __shfl_sync(kAll, s, __ffs(todo) - 1);
    const int64_t bh = at / block_size * num_kv_heads + h;
    const int rows = static_cast<int>(at % block_size) + 1;
    uint4 lo, hi;
    for (int r0 = 0; r0 < rows; r0 += U * R) {
      uint4 v[U];
#pragma unroll
      for (int i = 0; i < U; ++i)  // rows behind the last take the last one again
        v[i] = load_vector<D, BITS>(keys, scales, bh * block_size + min(r0 + i * R + sub, rows - 1), c8);
      if (r0 == 0) lo = hi = v[0];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        lo = make_uint4(min2(lo.x, v[i].x), min2(lo.y, v[i].y), min2(lo.z, v[i].z), min2(lo.w, v[i].w));
        hi = make_uint4(max2(hi.x, v[i].x), max2(hi.y, v[i].y), max2(hi.z, v[i].z), max2(hi.w, v[i].w));
      }
    }
#pragma unroll
    for (int o = V; o < 32; o *= 2) {
      lo = make_uint4(min2(lo.x, __shfl_xor_sync(kAll, lo.x, o)), min2(lo.y, __shfl_xor_sync(kAll, lo.y, o)),
                      min2(lo.z, __shfl_xor_sync(kAll, lo.z, o)), min2(lo.w, __shfl_xor_sync(kAll, lo.w, o)));
      hi = make_uint4(max2(hi.x, __shfl_xor_sync(kAll, hi.x, o)), max2(hi.y, __shfl_xor_sync(kAll, hi.y, o)),
                      max2(hi.z, __shfl_xor_sync(kAll, hi.z, o)), max2(hi.w, __shfl_xor_sync(kAll, hi.w, o)));
    }
    if (sub < 2) bounds[bh * 2 * V + lane] = sub == 0 ? lo : hi;  // [lo][hi], one vector per lane
  }
}

}  // namespace

cudaError_t launch_key_bounds(const int64_t *slot_mapping, int64_t num_tokens, const void *keys, const void *scales,
                              void *bounds, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                              int32_t head_dim, int32_t bits, uint32_t *status, cudaStream_t stream) {
  // Tokens per warp: one while that keeps the SMs from being full, up to 16 where most tokens do not end a block and
  // would only cost a warp each. CTAs of two warps, so that an SM's next ones start as soon as some end: 24,500
  // tokens x 8 heads in blocks of 16 took 11.8 us so (12.3 with eight warps; 12.6 with 32 tokens per warp).
  int32_t chunk = 1;
  while (chunk < 16 && num_tokens * num_kv_heads / chunk > 152 * 32) chunk *= 2;
  const int64_t units = (num_tokens + chunk - 1) / chunk * num_kv_heads;
  const dim3 grid(static_cast<unsigned>((units + 1) / 2));
  auto *kernel = bits == 4        ? key_bounds_kernel<128, 4>
                 : head_dim == 128 ? (bits == 8 ? key_bounds_kernel<128, 8> : key_bounds_kernel<128, 16>)
                                   : (bits == 8 ? key_bounds_kernel<64, 8> : key_bounds_kernel<64, 16>);
  return launch_pdl(kernel, grid, dim3(64), 0, stream, slot_mapping, num_tokens, keys,
                    static_cast<const __nv_bfloat16 *>(scales), static_cast<uint4 *>(bounds), num_blocks * block_size,
                    block_size, num_kv_heads, chunk, status);
}

}  // namespace pkv

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

pkv_status key_bounds(int32_t bits, const int64_t *slot_mapping, int64_t num_tokens, const void *keys,
                      const void *scales, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                      int32_t head_dim, void *bounds, uint32_t *device_status, pkv_stream_t stream) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 ||
      num_kv_heads > 65536 || num_blocks > INT64_MAX / block_size)
    return PKV_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || (bits == 4 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  // one grid of CTAs of two warps, 16 tokens a warp where there are so many
  if ((num_tokens + 15) / 16 * num_kv_heads > 2ll * INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!slot_mapping || !keys || (bits != 16 && !scales) || !bounds || !aligned16(keys) || !aligned16(scales) ||
      !aligned16(bounds) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7) != 0)
    return PKV_ERR_INVALID_ARG;
  const cudaError_t e = pkv::launch_key_bounds(slot_mapping, num_tokens, keys, scales, bounds, num_blocks, block_size,
                                               num_kv_heads, head_dim, bits, device_status,
                                               reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

pkv_status pkv_key_bounds(const int64_t *slot_mapping, int64_t num_tokens, const void *k_pool, int64_t num_blocks,
                          int32_t block_size, int32_t num_kv_heads, int32_t head_dim, void *bounds,
                          uint32_t *device_status, pkv_stream_t stream) {
  return key_bounds(16, slot_mapping, num_tokens, k_pool, nullptr, num_blocks, block_size, num_kv_heads, head_dim,
                    bounds, device_status, stream);
}

pkv_status pkv_key_bounds_q8(const int64_t *slot_mapping, int64_t num_tokens, const int8_t *k_codes,
                             const void *k_scales, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                             int32_t head_dim, void *bounds, uint32_t *device_status, pkv_stream_t stream) {
  return key_bounds(8, slot_mapping, num_tokens, k_codes, k_scales, num_blocks, block_size, num_kv_heads, head_dim,
                    bounds, device_status, stream);
}

pkv_status pkv_key_bounds_q4(const int64_t *slot_mapping, int64_t num_tokens, const uint8_t *k_codes,
                             const void *k_scales, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                             int32_t head_dim, void *bounds, uint32_t *device_status, pkv_stream_t stream) {
  return key_bounds(4, slot_mapping, num_tokens, k_codes, k_scales, num_blocks, block_size, num_kv_heads, head_dim,
                    bounds, device_status, stream);
}

}  // extern "C"
