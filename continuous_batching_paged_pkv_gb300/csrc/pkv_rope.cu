// Rotary positions: a step's queries and keys rotated by their positions, the
// rotated keys and the values appended to the paged pool in the same pass.
//
// A pair (a, b) of a head at position p with rotation f per position becomes
//   (m (a cos(p f) - b sin(p f)), m (a sin(p f) + b cos(p f))),
// m the magnitude of an extended context (1 otherwise). Pair i is elements
// (i, i + rot_dim / 2) in the half layout, (2 i, 2 i + 1) interleaved; elements
// from rot_dim on pass through. The angle comes as a fraction of a turn: f is
// a 64-bit fixed-point phase, p * phase modulo 2^64 is exact for every 32-bit
// position, and its top 32 bits (2^-33 of a turn, 7e-10 rad) feed sincospi. An
// angle in fp32 radians would be off by 4e-3 at position 131072. Products and
// sums are fp32 and round once, to bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 64;  // head_dim / 2 at head_dim 128

// One CTA per token: its angles once into shared memory, then one pair per
// thread over the token's rows (q heads, then k heads, then v heads).
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  __shared__ float2 turn[kMaxPairs];  // (cos, sin) times the magnitude
  grid_dependency_wait();             // every input may come from the previous kernel in the stream
  const int rot_pairs = a.rot_dim / 2, row_pairs = a.head_dim / 2;
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  for (int64_t t = blockIdx.x; t < a.num_tokens; t += gridDim.x) {
    if (threadIdx.x < rot_pairs) {
      const uint64_t angle = static_cast<uint64_t>(static_cast<int64_t>(__ldg(a.positions + t))) *
                             __ldg(a.phases + threadIdx.x);
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &s, &c);
      turn[threadIdx.x] = make_float2(c * a.magnitude, s * a.magnitude);
    }
    __syncthreads();
    int64_t block = 0, row = 0;
    bool keep = false;
    if (a.num_kv_heads > 0) {
      const int64_t slot = __ldg(a.slot_mapping + t);
      keep = slot >= 0 && slot < a.num_blocks * a.block_size;
      if (slot >= 0 && !keep && threadIdx.x == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SLOT_MAPPING);
      block = keep ? slot / a.block_size : 0;
      row = keep ? slot % a.block_size : 0;
    }
    for (int i = threadIdx.x; i < heads * row_pairs; i += kThreads) {
      const int h = i / row_pairs, j = i % row_pairs;
      const __nv_bfloat16 *src;
      __nv_bfloat16 *dst;
      const bool is_q = h < a.num_q_heads, is_v = h >= a.num_q_heads + a.num_kv_heads;
      if (is_q) {
        src = a.q + t * a.q_stride + h * a.head_dim;
        dst = a.q_out + t * a.q_out_stride + h * a.head_dim;
      } else {
        if (!keep) continue;
        const int g = h - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
        src = is_v ? a.v + t * a.v_stride + g * a.head_dim : a.k + t * a.k_stride + g * a.head_dim;
        dst = (is_v ? a.v_pool : a.k_pool) +
              ((block * a.num_kv_heads + g) * a.block_size + row) * static_cast<int64_t>(a.head_dim);
      }
      const bool turned = j < rot_pairs && !is_v;
      const int i0 = a.interleaved || j >= rot_pairs ? 2 * j : j;
      const int i1 = a.interleaved || j >= rot_pairs ? 2 * j + 1 : j + rot_pairs;
      const __nv_bfloat16 x0 = src[i0], x1 = src[i1];
      if (turned) {
        const float2 w = turn[j];
        const float f0 = __bfloat162float(x0), f1 = __bfloat162float(x1);
        dst[i0] = __float2bfloat16_rn(f0 * w.x - f1 * w.y);
        dst[i1] = __float2bfloat16_rn(f0 * w.y + f1 * w.x);
      } else {
        dst[i0] = x0;
        dst[i1] = x1;
      }
    }
    __syncthreads();  // the angles are overwritten for the next token
  }
  // pkv_attention reads q before it waits for this grid: every store is
  // performed before its thread ends, and this kernel never signals early.
  __threadfence();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
  const int64_t grid = a.num_tokens < (int64_t(1) << 30) ? a.num_tokens : int64_t(1) << 30;
  return launch_pdl(rope_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a);
}

}  // namespace pkv

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether rows of `width` elements every `stride` from x share memory with
// those of y: their address ranges meet, and they are not columns of one
// buffer that stay apart.
bool rows_meet(const void *x, int64_t x_stride, int64_t x_width, const void *y, int64_t y_stride, int64_t y_width,
               int64_t rows) {
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
  const uintptr_t x1 = x0 + ((rows - 1) * x_stride + x_width) * 2, y1 = y0 + ((rows - 1) * y_stride + y_width) * 2;
  if (x1 <= y0 || y1 <= x0) return false;
  if (x_stride != y_stride || x_stride == 0) return true;
  const int64_t stride = x_stride * 2;
  const int64_t off = ((static_cast<int64_t>(y0 - x0) % stride) + stride) % stride;  // y's column, seen from x
  return !(off >= x_width * 2 && off + y_width * 2 <= stride);
}

// Rows of `width` elements need 16-byte vectors and rows that do not overlap.
bool bad_rows(const void *p, int64_t stride, int64_t width, int64_t rows) {
  return !p || !aligned16(p) || stride % 8 != 0 || (rows > 1 && stride < width) || stride > (int64_t(1) << 40);
}

pkv_status check_rope(const pkv_rope_table *rope, int32_t head_dim) {
  if (!rope) return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (rope->rot_dim < 2 || rope->rot_dim > head_dim || rope->rot_dim % 2 != 0 || !rope->phases ||
      (reinterpret_cast<uintptr_t>(rope->phases) & 7) != 0 || (rope->interleaved != 0 && rope->interleaved != 1) ||
      !(rope->magnitude - rope->magnitude == 0.f))  // infinite or NaN
    return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

}  // namespace

extern "C" {

pkv_status pkv_rope(const void *x, int64_t x_stride, const int32_t *positions, const pkv_rope_table *rope,
                    int64_t num_tokens, int32_t num_heads, int32_t head_dim, void *out, int64_t out_stride,
                    pkv_stream_t stream) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || num_heads <= 0 || num_heads > 65536) return PKV_ERR_INVALID_ARG;
  if (const pkv_status st = check_rope(rope, head_dim); st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  const int64_t width = static_cast<int64_t>(num_heads) * head_dim;
  if (bad_rows(x, x_stride, width, num_tokens) || bad_rows(out, out_stride, width, num_tokens) || !positions ||
      (reinterpret_cast<uintptr_t>(positions) & 3) != 0)
    return PKV_ERR_INVALID_ARG;
  if ((x != out || x_stride != out_stride) && rows_meet(x, x_stride, width, out, out_stride, width, num_tokens))
    return PKV_ERR_INVALID_ARG;
  pkv::RopeArgs a{};
  a.q = static_cast<const __nv_bfloat16 *>(x);
  a.q_out = static_cast<__nv_bfloat16 *>(out);
  a.q_stride = x_stride;
  a.q_out_stride = out_stride;
  a.positions = positions;
  a.phases = rope->phases;
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.magnitude = rope->magnitude;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_heads;
  a.head_dim = head_dim;
  const cudaError_t e = pkv::launch_rope(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_rope_cache_write(const void *q, int64_t q_stride, const void *k_new, int64_t k_stride,
                                const void *v_new, int64_t v_stride, const int32_t *positions,
                                const int64_t *slot_mapping, const pkv_rope_table *rope, int64_t num_tokens,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, void *q_out,
                                int64_t q_out_stride, void *k_pool, void *v_pool, int64_t num_blocks,
                                int32_t block_size, uint32_t *device_status, pkv_stream_t stream) {
  if (num_tokens < 0 || num_tokens > INT32_MAX || num_q_heads <= 0 || num_q_heads > 65536 || num_kv_heads <= 0 ||
      num_kv_heads > 65536 || num_blocks <= 0 || block_size <= 0)
    return PKV_ERR_INVALID_ARG;
  if (const pkv_status st = check_rope(rope, head_dim); st != PKV_OK) return st;
  if (num_tokens == 0) return PKV_OK;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim, kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (bad_rows(q, q_stride, qw, num_tokens) || bad_rows(q_out, q_out_stride, qw, num_tokens) ||
      bad_rows(k_new, k_stride, kw, num_tokens) || bad_rows(v_new, v_stride, kw, num_tokens) || !positions ||
      (reinterpret_cast<uintptr_t>(positions) & 3) != 0 || !slot_mapping ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7) != 0 || !k_pool || !v_pool || !aligned16(k_pool) ||
      !aligned16(v_pool))
    return PKV_ERR_INVALID_ARG;
  if (((q != q_out || q_stride != q_out_stride) &&
       rows_meet(q, q_stride, qw, q_out, q_out_stride, qw, num_tokens)) ||
      rows_meet(k_new, k_stride, kw, q_out, q_out_stride, qw, num_tokens) ||
      rows_meet(v_new, v_stride, kw, q_out, q_out_stride, qw, num_tokens))
    return PKV_ERR_INVALID_ARG;
  pkv::RopeArgs a{};
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.k = static_cast<const __nv_bfloat16 *>(k_new);
  a.v = static_cast<const __nv_bfloat16 *>(v_new);
  a.q_out = static_cast<__nv_bfloat16 *>(q_out);
  a.k_pool = static_cast<__nv_bfloat16 *>(k_pool);
  a.v_pool = static_cast<__nv_bfloat16 *>(v_pool);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.positions = positions;
  a.slot_mapping = slot_mapping;
  a.phases = rope->phases;
  a.rot_dim = rope->rot_dim;
  a.interleaved = rope->interleaved;
  a.magnitude = rope->magnitude;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.status = device_status;
  const cudaError_t e = pkv::launch_rope(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
