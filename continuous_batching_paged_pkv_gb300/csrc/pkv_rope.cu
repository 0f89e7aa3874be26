// Rotary positions: a step's queries and keys rotated by their positions, the
// rotated keys and the values appended to the paged pool in the same pass.
//
// A pair (a, b) of a head at position p with rotation f per position becomes
//   (m (a cos(p f) - b sin(p f)), m (a sin(p f) + b cos(p f))),
// m the magnitude of an extended context (1 otherwise). Pair i is elements
// (i, i + rot_dim / 2) in the half layout, (2 i, 2 i + 1) interleaved; elements
// from rot_dim on pass through. The angle comes as a fraction of a turn: f is
// a 64-bit fixed-point phase, p * phase modulo 2^64 is exact for every 32-bit
// position, and its top 32 bits feed sincospi as an fp32 fraction of half a turn:
// off by at most pi 2^-25 (9e-8 rad, the rounding to 24 bits) at any position. An
// angle in fp32 radians would be off by 4e-3 at position 131072. Products and
// sums are fp32 and round once, to bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 64;  // head_dim / 2 at head_dim 128

// The angles of token t: (cos, sin) times the magnitude of pair i into turn[i], one thread each.
__device__ __forceinline__ void token_turns(const RopeArgs &a, int64_t t, float2 *turn) {
  for (int i = threadIdx.x; i < a.rot_dim / 2; i += blockDim.x) {
    const uint64_t angle =
        static_cast<uint64_t>(static_cast<int64_t>(__ldg(a.positions + t))) * __ldg(a.phases + i);
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &s, &c);
    turn[i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
}

// Where token t's key and value go: offset of its kv head 0 row in the pool, or
// -1 where they are not kept. Head g's row is g * block_size rows further.
__device__ __forceinline__ int64_t pool_offset(const RopeArgs &a, int64_t t, bool report) {
  if (a.num_kv_heads == 0) return -1;
  const int64_t slot = __ldg(a.slot_mapping + t);
  if (slot < 0) return -1;
  if (slot >= a.num_blocks * a.block_size) {
    if (report && a.status) atomicOr(a.status, PKV_DEV_BAD_SLOT_MAPPING);
    return -1;
  }
  const int64_t block = slot / a.block_size, row = slot % a.block_size;
  return (block * a.num_kv_heads * a.block_size + row) * a.head_dim;
}

struct HeadRow {
  const __nv_bfloat16 *src;
  __nv_bfloat16 *dst;  // nullptr: nothing to do
  bool turned;
};

// Head h of token t, in the order q heads, k heads, v heads.
__device__ __forceinline__ HeadRow head_row(const RopeArgs &a, int64_t t, int h, int64_t pool) {
  HeadRow r;
  if (h < a.num_q_heads) {
    r.src = a.q + t * a.q_stride + h * a.head_dim;
    r.dst = a.q_out + t * a.q_out_stride + h * a.head_dim;
    r.turned = true;
    return r;
  }
  const bool is_v = h >= a.num_q_heads + a.num_kv_heads;
  const int g = h - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
  r.src = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + g * a.head_dim;
  r.dst = pool < 0 ? nullptr
                   : (is_v ? a.v_pool : a.k_pool) + pool + static_cast<int64_t>(g) * a.block_size * a.head_dim;
  r.turned = !is_v;
  return r;
}

// Any even rot_dim: one CTA per token, one pair of elements per thread, with two
// 2-byte loads and stores and an index division a pair, which bind it (59% ALU, 65%
// issue, 25% of DRAM). 24500 tokens of 64 + 8 heads of 128, 120 elements rotated: 393
// us, where whole vectors (rope_vectors_kernel, 128 elements) take 155.
__global__ void __launch_bounds__(kThreads) rope_pairs_kernel(const RopeArgs a) {
  __shared__ float2 turn[kMaxPairs];
  grid_dependency_wait();  // every input may come from the previous kernel in the stream
  const int rot_pairs = a.rot_dim / 2, row_pairs = a.head_dim / 2;
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int64_t t = blockIdx.x;
  const int64_t pool = pool_offset(a, t, threadIdx.x == 0);
  token_turns(a, t, turn);
  __syncthreads();
  for (int i = threadIdx.x; i < heads * row_pairs; i += kThreads) {
    const int j = i % row_pairs;
    const HeadRow r = head_row(a, t, i / row_pairs, pool);
    if (!r.dst) continue;
    const int i0 = a.interleaved || j >= rot_pairs ? 2 * j : j;
    const int i1 = a.interleaved || j >= rot_pairs ? 2 * j + 1 : j + rot_pairs;
    const __nv_bfloat16 x0 = r.src[i0], x1 = r.src[i1];
    if (r.turned && j < rot_pairs) {
      const float2 w = turn[j];
      const float f0 = __bfloat162float(x0), f1 = __bfloat162float(x1);
      r.dst[i0] = __float2bfloat16_rn(f0 * w.x - f1 * w.y);
      r.dst[i1] = __float2bfloat16_rn(f0 * w.y + f1 * w.x);
    } else {
      r.dst[i0] = x0;
      r.dst[i1] = x1;
    }
  }
  __threadfence();  // as in rope_vectors_kernel
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Half layout: vector x holds the first elements of eight pairs, y the second ones.
__device__ __forceinline__ void turn_halves(uint4 &x, uint4 &y, const float2 *w) {
  uint32_t *px = &x.x, *py = &y.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 w0 = w[2 * i], w1 = w[2 * i + 1];
    const float a0 = low(px[i]), a1 = high(px[i]), b0 = low(py[i]), b1 = high(py[i]);
    px[i] = pack_bf16x2(a0 * w0.x - b0 * w0.y, a1 * w1.x - b1 * w1.y);
    py[i] = pack_bf16x2(a0 * w0.y + b0 * w0.x, a1 * w1.y + b1 * w1.x);
  }
}

// Interleaved: a vector holds four pairs.
__device__ __forceinline__ void turn_pairs(uint4 &x, const float2 *w) {
  uint32_t *p = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f0 = low(p[i]), f1 = high(p[i]);
    p[i] = pack_bf16x2(f0 * w[i].x - f1 * w[i].y, f0 * w[i].y + f1 * w[i].x);
  }
}

// rot_dim in whole 16-byte vectors (half layout: a multiple of 16, interleaved:
// of 8). A unit is two vectors of a head: the two halves of eight pairs, or two
// neighbours. A thread keeps its place within the head (D / 16 units divide the
// CTA's threads), so it reads its eight angles from shared memory once and walks
// the token's heads with them, one unit at a time; the first is requested before
// the angles are computed. gridDim.y CTAs share a token's units where tokens are few.
//
// Bound by HBM: T (2 Hq + 4 Hkv) D 2 bytes move and the angles are shared by a
// token's heads. What counts is CTAs in flight (12 of 128 threads per SM at 40
// registers and 32 spilled bytes, or 24 of 64), since a CTA waits in turn for
// position, vectors and stores: 24500 tokens of 64 + 8 heads of 128 take 155 us
// (6480 GB/s, 96% of the measured copy rate); with three units in flight per thread
// and 80 registers they took 223 us, and one pair of elements per thread 379 us.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 12) rope_vectors_kernel(const RopeArgs a) {
  constexpr int U = D / 16;  // units per head
  __shared__ float2 turn[kMaxPairs];
  grid_dependency_wait();  // every input may come from the previous kernel in the stream
  const int64_t t = blockIdx.x;
  const int64_t pool = pool_offset(a, t, threadIdx.x == 0 && blockIdx.y == 0);
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int c = threadIdx.x % U;
  const int turned_vecs = a.rot_dim / 8;
  // this thread's two vectors of a head
  const bool halves = !INTERLEAVED && c < turned_vecs / 2;
  const int v0 = halves ? c : 2 * c, v1 = halves ? c + turned_vecs / 2 : 2 * c + 1;
  const int step = blockDim.x / U * gridDim.y;
  int h = blockIdx.y * (blockDim.x / U) + threadIdx.x / U;

  HeadRow r;
  uint4 x, y;
  auto load = [&]() {
    r.dst = nullptr;
    if (h < heads) r = head_row(a, t, h, pool);
    if (r.dst) {
      x = reinterpret_cast<const uint4 *>(r.src)[v0];
      y = reinterpret_cast<const uint4 *>(r.src)[v1];
    }
  };
  load();
  token_turns(a, t, turn);
  __syncthreads();
  float2 w[8];
  if (INTERLEAVED || halves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = turn[c * 8 + i];  // past the rotated part: not used
  }
  for (; h < heads; h += step, load()) {
    if (!r.dst) continue;
    if (r.turned) {
      if constexpr (INTERLEAVED) {
        if (v0 < turned_vecs) turn_pairs(x, w);
        if (v1 < turned_vecs) turn_pairs(y, w + 4);
      } else if (halves) {
        turn_halves(x, y, w);
      }
    }
    uint4 *dst = reinterpret_cast<uint4 *>(r.dst);
    dst[v0] = x;
    dst[v1] = y;
  }
  // pkv_attention reads q before it waits for this grid: every store is
  // performed before its thread ends, and this kernel never signals early.
  __threadfence();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
  const unsigned tokens = static_cast<unsigned>(a.num_tokens);
  if (a.rot_dim % (a.interleaved ? 8 : 16) != 0)
    return launch_pdl(rope_pairs_kernel, dim3(tokens), dim3(kThreads), 0, stream, a);
  const int units = (a.num_q_heads + 2 * a.num_kv_heads) * (a.head_dim / 16);
  // Fewer tokens than SMs: one unit per thread, a token over several CTAs. Else one
  // CTA per token, with more units per thread (fewer, smaller CTAs reuse the angles
  // longer) the more tokens there are to fill the SMs. Measured with 3 / 5 / 10
  // units: 256 tokens of 64 + 8 heads 4.8 / 4.8 / 6.3 us, 2048 of 32 + 8 14.8 /
  // 12.0 / 12.7 us, 24500 of 64 + 8 163 / 163 / 154 us (heads of 128). Over eight
  // shapes from 4 + 2 heads of 64 to 64 + 8 of 128 and 256 to 24500 tokens the rule
  // is within 0.5 us or 6% of the best of 1, 2, 3, 5 and 10 units, but for 256
  // tokens of 8 + 8 or 14 + 2 heads of 64 (3.4 us, 2.7 with one unit) and 2048 of
  // 64 + 8 heads of 128 (21.1 us, 18.4 with ten).
  const bool few = a.num_tokens < 152;
  const int per_thread = few ? 1 : a.num_tokens < 1024 ? 3 : a.num_tokens < 8192 ? 5 : 10;
  const int want = (units + per_thread - 1) / per_thread;
  const int passes = (want + kThreads - 1) / kThreads;
  const int threads = ((want + passes - 1) / passes + 31) / 32 * 32;
  const dim3 grid(tokens, few ? passes : 1);
  auto *kernel = a.head_dim == 128 ? (a.interleaved ? rope_vectors_kernel<128, true> : rope_vectors_kernel<128, false>)
                                   : (a.interleaved ? rope_vectors_kernel<64, true> : rope_vectors_kernel<64, false>);
  return launch_pdl(kernel, grid, dim3(threads), 0, stream, a);
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
  return !p || !aligned16(p) || stride % 8 != 0 || (rows > 1 && stride < width) || stride > (int64_t(1) << 60) / rows;
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
