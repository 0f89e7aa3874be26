// The blocks that a block-sparse step reads: an upper bound of every cached
// block's scores, and the best blocks by it.
//
// With lo, hi the bounds of a block's keys and q one query row of the kv head's
// group, no key k of the block has q . k above
//   s = sum_d max(q_d lo_d, q_d hi_d) = max(q, 0) . hi + min(q, 0) . lo,
// so a block's score, the maximum of s over the segment's rows and the group's
// heads, is one matrix product of depth 2 D and a maximum.
//
// Scoring kernel: persistent warps, each taking 16 candidate blocks of one (segment,
// kv head) at a time. Their bounds go from global memory straight into MMA operands
// (m16n8k16, blocks on M, the (row, head) columns on N): the order of the depth is
// free as long as both operands share it, so a thread's 16-byte piece of a row serves
// two steps. As soon as the lower bounds of a task are multiplied the next task's are
// requested into the same registers, then the upper ones. Each bound is read once; the
// kernel is bound by HBM. A second product
// of the magnitudes gives A = sum |terms|: a step of the tensor core adds 17 numbers
// to fp32 in an order of its own, within 17 * 2^-23 of the sum of their magnitudes;
// two steps make a piece, whose sum (at most A of the piece, so 34 * 2^-23 A over all
// of them) is added to the running one with at most 8 roundings of 2^-24 A: a score
// is within 38 * 2^-23 A of the exact sum, for which 64 * 2^-23 A is taken, and 2^-100
// for products that are too small for fp32.
//
// Choosing kernel: a CTA per (segment, kv head), of 4 warps or, where segments have
// many candidates, 32. A bound T that exactly k scores reach, or else the k-th largest
// score, comes from histograms of the ordered scores' digits and, as soon as few agree
// with it so far, from their ranks. With E the error bound,
// what is above T + 2 E is in (its exact score is above T + E, and fewer than k are),
// what is below T - 2 E is out (k others have exact scores from T - E on), and only the
// blocks between are summed again, in fp64 (products of two bf16 are exact there), and
// ranked by (score, lower place first). So the choice is that of the exact scores,
// whatever the order of the sums, and every run gives the same. Then the chosen places
// are written in growing order.
//
// 256 slots x 8 heads of 512 to 16384 keys in blocks of 32, 64 chosen: 39.6 us, for
// 150 MB of bounds; five slots of up to 131072 keys in blocks of 16, 128 chosen: 28.4
// to 29.6 us, 86 MB (2.3 to 3 us more where the scoring warps look their first blocks
// up behind the wait for the kernel before; 1 and 0.2 with digits alone). The choosing
// kernel's chain of loads, histograms and, in a CTA of seven there, an exact sum (4
// us) is 11 to 13 us of them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kScoreError = 0x1.01p-17f;  // of the sum of magnitudes, whose own error is in the last digits

// A segment of a selection item, checked against the step's metadata: its blocks, the candidates [first, first +
// cand) among them (cand 0 where every block is read), the first place of the tail that is always read.
struct Chosen {
  int row0, n, slot, blocks, read, first, last, cand;
  bool ok;
};

__device__ __forceinline__ Chosen chosen_segment(const StepArgs &a, int seg, int slot, int max_cols, int row0, int row1,
                                                 int L, int sslot) {
  Chosen c{};
  c.slot = slot;
  c.row0 = row0;
  c.n = row1 - row0;
  c.ok = seg >= 0 && seg < a.num_seqs && slot >= 0 && slot < a.max_slots && sslot == slot && c.n >= 1 && c.n <= L &&
         c.n * a.group <= max_cols && row0 >= 0 && static_cast<int64_t>(row0) + c.n <= a.total_q;
  if (!c.ok) return c;
  const int shift = 31 - __clz(a.block_size);  // block sizes are powers of two
  c.blocks = ((L - 1) >> shift) + 1;
  c.read = min(a.top_blocks, c.blocks);
  c.last = max(0, ((L - c.n) >> shift) - a.keep_last);
  c.first = min(a.keep_first, c.last);
  c.cand = c.blocks > c.read ? c.last - c.first : 0;
  c.ok = c.blocks <= a.max_blocks_per_slot && (c.blocks <= c.read || c.first + (c.blocks - c.last) <= c.read);
  return c;
}

// First entry of a (segment, kv head) among the sums of magnitudes, one per group of candidates.
__device__ __forceinline__ int64_t sum_index(int base, int hkv, int g, int cand) {
  return static_cast<int64_t>(base) / kScoreGroup * hkv +
         static_cast<int64_t>(g) * ((cand + kScoreBlocks - 1) / kScoreBlocks * (kScoreBlocks / kScoreGroup));
}

__device__ __forceinline__ uint32_t part(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// All bits of each 16-bit half whose value is negative.
__device__ __forceinline__ uint32_t negative(uint32_t x) { return prmt(x, 0, 0xBB99u); }

// A warp's scoring task: 16 candidates of one (segment, kv head). Its metadata, block IDs and bounds are loaded one
// step of the loop after the other, each a task ahead of the last, so that no latency is waited on.
struct ScoreTask {
  int seg, slot, c0, base, g;  // from the item
  int row0, row1, L, sslot;    // loaded by meta()
  int bid[2];                  // blocks of this thread's two candidates, loaded by blocks()
  int cand, cols;              // 0 candidates: nothing to do
};

template <int D, int NT>
__global__ void __launch_bounds__(384, 1) score_blocks_kernel(const StepArgs a, const __nv_bfloat16 *__restrict__ bounds,
                                                              const int32_t *__restrict__ items, int num_items,
                                                              int64_t candidates, float *__restrict__ scores,
                                                              float *__restrict__ sums) {
  constexpr int P = D / 32;                          // 32-value pieces of a row of lo (or hi), and of q
  constexpr int kPerItem = kScoreBlocks / kScoreGroup;
  constexpr bool kQAhead = NT == 1;                  // two columns' q would not fit beside the bounds
  const int lane = threadIdx.x & 31, t = lane & 3, hkv = a.num_kv_heads;

  // Tasks in the order of items, kv heads, groups; a warp goes on by `stride` of them, kept as its three digits.
  struct Place {
    int item, g, w;
  };
  const int warps = static_cast<int>(gridDim.x) * (blockDim.x / 32);
  auto place_of = [&](int task) { return Place{task / kPerItem / hkv, task / kPerItem % hkv, task % kPerItem}; };
  const Place stride = place_of(warps);
  auto advance = [&](Place &p) {
    p.w += stride.w;
    p.g += stride.g;
    p.item += stride.item;
    if (p.w >= kPerItem) p.w -= kPerItem, ++p.g;
    if (p.g >= hkv) p.g -= hkv, ++p.item;
  };
  auto item_of = [&](const Place &p) -> int4 {
    return p.item < num_items ? __ldg(reinterpret_cast<const int4 *>(items) + p.item) : make_int4(-1, 0, 0, 0);
  };
  auto meta = [&](ScoreTask &T, const Place &p, const int4 &it) {
    T.seg = it.x;
    T.slot = it.y;
    T.c0 = it.z + p.w * kScoreGroup;
    T.base = it.w;
    T.g = p.g;
    T.cand = 0;
    T.row0 = T.row1 = T.L = 0;
    T.sslot = -1;
    if (T.seg >= 0 && T.seg < a.num_seqs && T.slot >= 0 && T.slot < a.max_slots) {
      T.row0 = __ldg(a.cu_seqlens_q + T.seg);
      T.row1 = __ldg(a.cu_seqlens_q + T.seg + 1);
      T.L = __ldg(a.context_lens + T.slot);
      T.sslot = __ldg(a.seq_slot + T.seg);
    }
  };
  auto in_pool = [&](int bid) { return static_cast<uint32_t>(bid) < static_cast<uint64_t>(a.num_blocks); };
  // Check the metadata and look the blocks up. Rows past the last candidate take that one's again.
  auto blocks = [&](ScoreTask &T, const Place &p) {
    T.bid[0] = T.bid[1] = 0;
    if (p.item >= num_items) return;
    const Chosen c = chosen_segment(a, T.seg, T.slot, 8 * NT, T.row0, T.row1, T.L, T.sslot);
    if (!c.ok || T.c0 < 0 || T.base < 0 || T.base % kScoreBlocks != 0 ||
        static_cast<int64_t>(T.base) + (c.cand + kScoreBlocks - 1) / kScoreBlocks * kScoreBlocks > candidates) {
      if (lane == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
      return;
    }
    if (T.c0 >= c.cand) return;  // the item's last groups may be empty
    T.cand = c.cand;
    T.cols = c.n * a.group;
    const int32_t *table = a.block_tables + static_cast<int64_t>(T.slot) * a.max_blocks_per_slot + c.first;
#pragma unroll
    for (int r = 0; r < 2; ++r) T.bid[r] = __ldg(table + min(T.c0 + (lane >> 2) + 8 * r, T.cand - 1));
  };
  // A thread's pieces of lo (half 0) or hi (1) of its two rows; a block outside the pool reads block 0's.
  auto load_half = [&](uint4 (&x)[2][P], const ScoreTask &T, int half) {
    if (T.cand == 0) return;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int bid = in_pool(T.bid[r]) ? T.bid[r] : 0;
      const uint4 *row = reinterpret_cast<const uint4 *>(
                             bounds + ((static_cast<int64_t>(bid) * hkv + T.g) * 2 + half) * D) + t;
#pragma unroll
      for (int p = 0; p < P; ++p) x[r][p] = __ldcg(row + p * 4);
    }
  };
  // q of column nt * 8 + lane / 4; columns past the last take the first one again, which changes no maximum.
  int col_row[NT], col_head[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    col_row[nt] = (nt * 8 + (lane >> 2)) / a.group;
    col_head[nt] = (nt * 8 + (lane >> 2)) % a.group;
  }
  auto load_q = [&](uint4 (&q)[P], const ScoreTask &T, int nt) {
    if (T.cand == 0) return;
    const bool valid = nt * 8 + (lane >> 2) < T.cols;
    const uint4 *row = reinterpret_cast<const uint4 *>(
                           static_cast<const __nv_bfloat16 *>(a.q) +
                           (static_cast<int64_t>(T.row0 + (valid ? col_row[nt] : 0)) * a.num_q_heads + T.g * a.group +
                            (valid ? col_head[nt] : 0)) * D) + t;
#pragma unroll
    for (int p = 0; p < P; ++p) q[p] = __ldg(row + p * 4);
  };

  ScoreTask A, B, C;  // current, next (blocks known), after it (metadata loading)
  uint4 lo[2][P], hi[2][P], qa[NT][P], qb[kQAhead ? P : 1];
  Place at = place_of(static_cast<int>(blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32));
  meta(A, at, item_of(at));
  blocks(A, at);
  int left = at.item < num_items;  // whether A is a task
  advance(at);
  meta(B, at, item_of(at));
  blocks(B, at);
  int more = at.item < num_items;
  advance(at);  // `at` is C's from here on
  meta(C, at, item_of(at));
  Place ahead = at;
  advance(ahead);
  int4 next_item = item_of(ahead);
  // The list, the metadata and the block tables are final when this grid starts; q and the bounds come from earlier
  // work. The choosing kernel may start once that has finished.
  grid_dependency_wait();
  launch_dependents();
  load_half(lo, A, 0);
  load_half(hi, A, 1);
  if constexpr (kQAhead) load_q(qa[0], A, 0);

  while (left) {
    float s[NT][4], m[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = m[nt][i] = 0.f;
    if constexpr (!kQAhead) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) load_q(qa[nt], A, nt);
    }
    // One half's products, a piece's sum started anew (for the error bound), and those of the magnitudes.
    auto multiply = [&](const uint4 (&x)[2][P], int half) {
      if (A.cand == 0) return;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float d[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t af[4] = {part(x[0][p], 2 * k), part(x[1][p], 2 * k), part(x[0][p], 2 * k + 1), part(x[1][p], 2 * k + 1)};
          const uint32_t aa[4] = {af[0] & 0x7FFF7FFFu, af[1] & 0x7FFF7FFFu, af[2] & 0x7FFF7FFFu, af[3] & 0x7FFF7FFFu};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t q0 = part(qa[nt][p], 2 * k), q1 = part(qa[nt][p], 2 * k + 1);
            const uint32_t n0 = half ? ~negative(q0) : negative(q0), n1 = half ? ~negative(q1) : negative(q1);
            mma_bf16_16816(d[nt], af, q0 & n0, q1 & n1);
            mma_bf16_16816(m[nt], aa, q0 & n0 & 0x7FFF7FFFu, q1 & n1 & 0x7FFF7FFFu);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[nt][i] += d[nt][i];
      }
    };
    multiply(lo, 0);
    load_half(lo, B, 0);
    if constexpr (kQAhead) load_q(qb, B, 0);
    blocks(C, at);
    multiply(hi, 1);
    load_half(hi, B, 1);
    if (A.cand > 0) {
      float best[2] = {-INFINITY, -INFINITY};  // blocks lane / 4 and lane / 4 + 8; a NaN is no maximum
      uint32_t mag = 0;  // non-negative floats order as their bits do; a NaN is above infinity there
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          best[i >> 1] = fmaxf(best[i >> 1], s[nt][i]);
          mag = max(mag, __float_as_uint(m[nt][i]) & 0x7FFFFFFFu);
        }
      float *out = scores + static_cast<int64_t>(A.base) * hkv + static_cast<int64_t>(A.g) * A.cand + A.c0;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        best[r] = fmaxf(best[r], __shfl_xor_sync(kAll, best[r], 1));
        best[r] = fmaxf(best[r], __shfl_xor_sync(kAll, best[r], 2));
        const int j = (lane >> 2) + 8 * r;
        if (t == 0 && A.c0 + j < A.cand) {
          const bool in = in_pool(A.bid[r]);
          if (!in && a.status) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
          out[j] = in ? best[r] + 0.f : -INFINITY;
        }
      }
      mag = __reduce_max_sync(kAll, mag);
      if (lane == 0) sums[sum_index(A.base, hkv, A.g, A.cand) + A.c0 / kScoreGroup] = __uint_as_float(mag);
    }
    A = B;
    B = C;
    left = more;
    more = at.item < num_items;
    at = ahead;
    meta(C, at, next_item);
    advance(ahead);
    next_item = item_of(ahead);
    if constexpr (kQAhead) {
#pragma unroll
      for (int p = 0; p < P; ++p) qa[0][p] = qb[p];
    }
  }
}

// Order of floats (and doubles) as unsigned integers; no NaN, and zeros are positive.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

constexpr int kListed = 256;  // blocks between the bounds that are ranked in shared memory

// Sums and maxima over T threads, up to three of them behind one barrier; two buffers, so that one is enough.
template <int T>
struct Block {
  uint32_t (*buf)[3][32];
  int turn;
  template <typename Op, typename... X>
  __device__ __forceinline__ void reduce(Op op, X &...x) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    turn ^= 1;
    int i = 0;
    (
        [&] {
          const uint32_t w = op(x);
          if (lane == 0) buf[turn][i++][warp] = w;
        }(),
        ...);
    __syncthreads();
    i = 0;
    ((x = op(lane < T / 32 ? buf[turn][i++][lane] : 0u)), ...);
  }
  template <typename... X>
  __device__ __forceinline__ void sums(X &...x) {
    reduce([](uint32_t v) { return __reduce_add_sync(kAll, v); }, x...);
  }
  template <typename... X>
  __device__ __forceinline__ void maxima(X &...x) {
    reduce([](uint32_t v) { return __reduce_max_sync(kAll, v); }, x...);
  }
  __device__ __forceinline__ uint32_t sum(uint32_t x) {
    sums(x);
    return x;
  }
  // Sum over the warps before this one of x's sums over a warp.
  __device__ __forceinline__ uint32_t warps_before(uint32_t x) {
    const uint32_t w = __reduce_add_sync(kAll, x);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    turn ^= 1;
    if (lane == 0) buf[turn][0][warp] = w;
    __syncthreads();
    return __reduce_add_sync(kAll, lane < warp ? buf[turn][0][lane] : 0u);
  }
};

// Exact score of candidate j, by one warp. The columns' sums are taken in fp32 first (each within `error`, as the
// scores are), two lanes to a column; only those that may be the largest are summed again in fp64, whose
// instructions take 64 times as long, over all lanes.
template <int D>
__device__ __forceinline__ double exact_score(const StepArgs &a, const __nv_bfloat16 *bounds, const Chosen &c, int g,
                                              int j, float error) {
  const int lane = threadIdx.x & 31, mine = lane & 15, cols = c.n * a.group;  // at most 16 columns
  const int bid = __ldg(a.block_tables + static_cast<int64_t>(c.slot) * a.max_blocks_per_slot + c.first + j);
  if (bid < 0 || bid >= a.num_blocks) return -INFINITY;
  const __nv_bfloat16 *lo = bounds + (static_cast<int64_t>(bid) * a.num_kv_heads + g) * 2 * D;
  auto row = [&](int col) {
    return static_cast<const __nv_bfloat16 *>(a.q) +
           ((static_cast<int64_t>(c.row0) + col / a.group) * a.num_q_heads + g * a.group + col % a.group) * D;
  };
  float s = -INFINITY;
  if (mine < cols) {
    s = 0.f;
    const int at = (lane >> 4) * (D / 2);
    const uint4 *pq = reinterpret_cast<const uint4 *>(row(mine) + at), *pl = reinterpret_cast<const uint4 *>(lo + at),
                *ph = reinterpret_cast<const uint4 *>(lo + D + at);
#pragma unroll 2
    for (int v = 0; v < D / 16; ++v) {
      const uint4 q = __ldg(pq + v), l = __ldcg(pl + v), h = __ldcg(ph + v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t qq = part(q, i), n = negative(qq), b = (part(l, i) & n) | (part(h, i) & ~n);
        s = fmaf(__uint_as_float(qq << 16), __uint_as_float(b << 16), s);
        s = fmaf(__uint_as_float(qq & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u), s);
      }
    }
  }
  const float other = __shfl_xor_sync(kAll, s, 16);
  if (mine < cols) s += other;
  const bool odd = __any_sync(kAll, mine < cols && !(fabsf(s) < INFINITY));  // some sum is not finite
  float top = s;
#pragma unroll
  for (int o = 8; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  double best = -INFINITY;
  for (uint32_t todo = __ballot_sync(kAll, lane < cols && (odd || !(s < __fsub_rd(top, 2.f * error)))); todo;
       todo &= todo - 1) {
    const __nv_bfloat16 *q = row(__ffs(todo) - 1);
    double e = 0.0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float x = __bfloat162float(q[lane + 32 * i]);
      e = fma(static_cast<double>(x), static_cast<double>(__bfloat162float(lo[(x < 0.f ? 0 : D) + lane + 32 * i])), e);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) e += __shfl_xor_sync(kAll, e, o);
    if (e == e && e > best) best = e;
  }
  return best + 0.0;
}

// T threads; warp w has the candidates from w S on (S a multiple of 32), in turn over its lanes. Up to KEYS ordered
// scores are kept in shared memory (more are read again in every pass, from L2). A score that was settled by its
// exact value is marked as above or below all others.
template <int D, int T, int KEYS>
__global__ void __launch_bounds__(T) choose_blocks_kernel(const StepArgs a, const __nv_bfloat16 *__restrict__ bounds,
                                                          const int32_t *__restrict__ items, int64_t candidates,
                                                          float *scores, const float *__restrict__ sums,
                                                          double *exact, int32_t *__restrict__ selected) {
  // The metadata and the list are final when this grid starts (the scoring kernel starts after everything before the
  // call); only the scores need the scoring kernel to finish. Every path waits for it, so that the grid ends after it.
  launch_dependents();
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t s_buf[2][3][32];
  __shared__ int s_list[kListed];
  __shared__ double s_exact[kListed];
  __shared__ uint32_t s_listed, s_same, s_hist[256], s_digit[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.y;
  const int4 it = __ldg(reinterpret_cast<const int4 *>(items) + blockIdx.x);
  const int base = it.z, N = it.w;
  if (!(it.x >= 0 && it.x < a.num_seqs)) {
    if (tid == 0 && a.status && g == 0) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    grid_dependency_wait();
    return;
  }
  const Chosen c = chosen_segment(a, it.x, it.y, 16, __ldg(a.cu_seqlens_q + it.x), __ldg(a.cu_seqlens_q + it.x + 1),
                                  it.y >= 0 && it.y < a.max_slots ? __ldg(a.context_lens + it.y) : 0,
                                  __ldg(a.seq_slot + it.x));
  int32_t *out = selected + (static_cast<int64_t>(it.x) * a.num_kv_heads + g) * a.top_blocks;
  const bool ok = c.ok && c.cand == N && base >= 0 && base % kScoreBlocks == 0 &&
                  static_cast<int64_t>(base) + (N + kScoreBlocks - 1) / kScoreBlocks * kScoreBlocks <= candidates;
  if (!ok) {
    if (tid == 0 && a.status && g == 0) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    grid_dependency_wait();
    for (int i = tid; i < a.top_blocks; i += T) out[i] = -1;
    return;
  }
  if (N == 0) {  // every block
    grid_dependency_wait();
    for (int i = tid; i < a.top_blocks; i += T) out[i] = i < c.blocks ? i : -1;
    return;
  }
  grid_dependency_wait();
  // the blocks that are always read, and what is left empty
  const int tail = c.blocks - c.last;
  const uint32_t need = static_cast<uint32_t>(c.read - c.first - tail);
  for (int i = tid; i < c.first; i += T) out[i] = i;
  for (int i = tid; i < tail; i += T) out[c.first + need + i] = c.last + i;
  for (int i = c.read + tid; i < a.top_blocks; i += T) out[i] = -1;
  if (need == 0) return;
  const int64_t at = static_cast<int64_t>(base) * a.num_kv_heads + static_cast<int64_t>(g) * N;
  float *sc = scores + at;
  const bool resident = N <= KEYS;
  const int S = ((N + T - 1) / T) * 32, w0 = warp * S, w1 = min(w0 + S, N);
  // f(j, key, live) for this warp's candidates, all lanes together
  auto each = [&](auto f) {
#pragma unroll 2
    for (int j = w0 + lane; j - lane < w1; j += 32) {
      const bool live = j < w1;
      f(j, !live ? 0u : resident ? keys[j] : ordered(__ldcg(sc + j)), live);
    }
  };
  auto settle = [&](int j, bool chosen) {
    if (resident)
      keys[j] = chosen ? ~0u : 0u;
    else
      sc[j] = __uint_as_float(chosen ? 0x7FFFFFFFu : ~0u);
  };
  Block<T> block{s_buf, 0};
  // largest sum of magnitudes; least (its complement) and largest score
  uint32_t mag = 0, least = 0u, most = 0u;
  const float *group_sums = sums + sum_index(base, a.num_kv_heads, g, N);
  for (int i = tid; i < (N + kScoreGroup - 1) / kScoreGroup; i += T) mag = max(mag, __float_as_uint(__ldcg(group_sums + i)));
  for (int j0 = w0 + lane; j0 < w1; j0 += 8 * 32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __ldcg(sc + min(j0 + i * 32, w1 - 1));  // past the last: that one again
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t k = ordered(v[i]);
      if (resident && j0 + i * 32 < w1) keys[j0 + i * 32] = k;
      least = max(least, ~k), most = max(most, k);
    }
  }
  if (tid == 0) s_listed = s_same = 0;
  block.maxima(mag, least, most);
  const float error = __uint_as_float(mag) * kScoreError + 0x1p-100f;
  // x: a bound that `need` candidates reach and no larger one does, or that exactly `need` reach. Eight bits at a
  // time below the bits that all share: a histogram of the candidates that agree with x so far, and the digit of
  // the `left`-th largest of them.
  const int bits = 32 - __clz(~least ^ most);
  uint32_t x = bits == 32 ? 0u : most >> bits << bits, left = need;
  for (int shift = bits; shift > 0;) {
    const int width = min(shift, 8), top = shift;
    shift -= width;
    for (int i = tid; i < 256; i += T) s_hist[i] = 0;
    __syncthreads();
    each([&](int, uint32_t k, bool live) {
      if (live && (top == 32 || k >> top == x >> top)) atomicAdd(&s_hist[k >> shift & ((1u << width) - 1u)], 1u);
    });
    __syncthreads();
    if (warp == 0) {  // lane l: digits 255 - 8 l and the seven below it
      uint32_t n[8], mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += n[i] = s_hist[255 - 8 * lane - i];
      uint32_t upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += y;
      }
      if (upto >= left && upto - mine < left) {
        uint32_t above = upto - mine;
        for (int i = 0; i < 8; ++i) {
          if (above + n[i] >= left) {
            s_digit[0] = 255 - 8 * lane - i;
            s_digit[1] = left - above;
            s_digit[2] = n[i];
            break;
          }
          above += n[i];
        }
      }
    }
    __syncthreads();
    x |= s_digit[0] << shift;
    left = s_digit[1];
    const uint32_t same = s_digit[2];
    if (same == left) break;
    if (shift > 0 && same <= kListed) {  // few agree with x so far: ranked at once
      each([&](int, uint32_t k, bool live) {
        if (live && k >> shift == x >> shift) s_list[atomicAdd(&s_same, 1u)] = static_cast<int>(k);
      });
      __syncthreads();
      for (uint32_t i = tid; i < same; i += T) {
        const uint32_t k = static_cast<uint32_t>(s_list[i]);
        uint32_t above = 0, reach = 0;
        for (uint32_t o = 0; o < same; ++o) {
          above += static_cast<uint32_t>(s_list[o]) > k;
          reach += static_cast<uint32_t>(s_list[o]) >= k;
        }
        if (above < left && left <= reach) s_digit[0] = k;
      }
      __syncthreads();
      x = s_digit[0];
      break;
    }
  }
  const float T0 = unordered(x);
  float low = __fsub_rd(T0, 2.f * error), high = __fadd_ru(T0, 2.f * error);
  if (!(low <= T0)) low = -INFINITY;    // infinities and NaN among the terms: all are summed again
  if (!(high >= T0)) high = INFINITY;
  const uint32_t klow = ordered(low + 0.f), khigh = ordered(high + 0.f);
  uint32_t over = 0, between = 0;
  each([&](int, uint32_t k, bool live) {
    over += live && k > khigh;
    between += live && k >= klow && k <= khigh;
  });
  uint32_t mine = over + between;  // of this thread, where all between the bounds are in
  block.sums(over, between);
  const uint32_t m = between, r = need - over;  // r of m
  uint32_t from = klow;  // scores from here on are chosen
  if (m != r) {
    from = khigh + 1;  // what is settled is above or below
    if (m <= kListed) {
      each([&](int j, uint32_t k, bool live) {
        if (live && k >= klow && k <= khigh) s_list[atomicAdd(&s_listed, 1u)] = j;
      });
      __syncthreads();
      for (uint32_t i = warp; i < m; i += T / 32) {
        const double s = exact_score<D>(a, bounds, c, g, s_list[i], error);
        if (lane == 0) s_exact[i] = s;
      }
      __syncthreads();
      for (uint32_t i = tid; i < m; i += T) {
        const double s = s_exact[i];
        const int j = s_list[i];
        uint32_t better = 0;
        for (uint32_t o = 0; o < m; ++o) better += s_exact[o] > s || (s_exact[o] == s && s_list[o] < j);
        settle(j, better < r);
      }
    } else {
      // Many equal (or indistinguishable) scores: the same choice with the exact scores in memory, the r-th
      // largest of them found bit by bit, equal ones taken from the lowest place on.
      double *ex = exact + at;
      for (int j = warp; j < N; j += T / 32) {
        const uint32_t k = resident ? keys[j] : ordered(__ldcg(sc + j));
        if (k < klow || k > khigh) continue;
        const double s = exact_score<D>(a, bounds, c, g, j, error);
        if (lane == 0) ex[j] = s;
      }
      __syncthreads();
      auto between_at = [&](uint32_t k, bool live) { return live && k >= klow && k <= khigh; };
      uint64_t v = 0;
      for (int bit = 63; bit >= 0; --bit) {
        const uint64_t y = v | 1ull << bit;
        uint32_t n = 0;
        each([&](int j, uint32_t k, bool live) { n += between_at(k, live) && ordered(ex[j]) >= y; });
        if (block.sum(n) >= r) v = y;
      }
      uint32_t above = 0, equal = 0;
      each([&](int j, uint32_t k, bool live) {
        if (!between_at(k, live)) return;
        const uint64_t e = ordered(ex[j]);
        above += e > v;
        equal += e == v;
      });
      above = block.sum(above);
      uint32_t rank = block.warps_before(equal);
      each([&](int j, uint32_t k, bool live) {
        const bool here = between_at(k, live);
        const uint64_t e = here ? ordered(ex[j]) : 0;
        const uint32_t ties = __ballot_sync(kAll, here && e == v);
        if (here) settle(j, e > v || (e == v && rank + __popc(ties & ((1u << lane) - 1u)) < r - above));
        rank += __popc(ties);
      });
    }
    __syncthreads();
  }
  auto in = [&](uint32_t k, bool live) { return live && k >= from; };
  if (m != r) {
    mine = 0;
    each([&](int, uint32_t k, bool live) { mine += in(k, live); });
  }
  uint32_t place = block.warps_before(mine);
  each([&](int j, uint32_t k, bool live) {
    const bool here = in(k, live);
    const uint32_t all = __ballot_sync(kAll, here), p = place + __popc(all & ((1u << lane) - 1u));
    if (here && p < need) out[c.first + p] = c.first + j;
    place += __popc(all);
  });
}

}  // namespace

cudaError_t launch_select_blocks(const StepArgs &a, const void *bounds, const pkv_work_info &info, void *workspace,
                                 int32_t *selected, cudaStream_t stream) {
  const int64_t cand = info.scratch_blocks;
  const SelectLayout lay = select_layout(cand, a.num_kv_heads);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  double *exact = reinterpret_cast<double *>(ws + lay.exact);
  float *scores = reinterpret_cast<float *>(ws + lay.scores), *sums = reinterpret_cast<float *>(ws + lay.sums);
  auto *b = static_cast<const __nv_bfloat16 *>(bounds);
  const int32_t *pre = a.work + static_cast<int64_t>(info.num_decode_items) * PKV_WORK_WORDS_PER_ITEM;
  const int32_t *scr = pre + (static_cast<int64_t>(info.num_prefill_items) + info.num_combine_items) * PKV_WORK_WORDS_PER_ITEM;
  if (info.num_scratch_items > 0) {
    const bool wide = info.decode_rows_max * a.group > 8;
    auto *kernel = a.head_dim == 128 ? (wide ? score_blocks_kernel<128, 2> : score_blocks_kernel<128, 1>)
                                     : (wide ? score_blocks_kernel<64, 2> : score_blocks_kernel<64, 1>);
    constexpr int kWarps = 12;  // what the registers of an SM hold
    const int64_t tasks = static_cast<int64_t>(info.num_scratch_items) * a.num_kv_heads * (kScoreBlocks / kScoreGroup);
    if (tasks > INT32_MAX - 16 * 152 * kWarps) return cudaErrorInvalidValue;
    const int64_t ctas = (tasks + kWarps - 1) / kWarps;
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(ctas < 152 ? ctas : 152)), dim3(32 * kWarps), 0,
                                     stream, a, b, scr, static_cast<int>(info.num_scratch_items), cand, scores, sums);
    if (e != cudaSuccess) return e;
  }
  if (info.num_prefill_items == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(info.num_prefill_items), static_cast<unsigned>(a.num_kv_heads));
  auto go = [&](auto *kernel, int threads, int num_keys) {
    return launch_pdl(kernel, grid, dim3(threads), num_keys * 4, stream, a, b, pre, cand, scores, sums, exact, selected);
  };
  // Small CTAs where the segments have few candidates: 256 slots x 8 heads of 145 on average take 14.8 us with 128
  // threads, 16.0 with 64 (and 30 with one warp, whose longest segment sets the time); 5 slots x 8 heads of up to
  // 8190 take 15.8 us with 1024. The mean decides, so a long segment among many short ones gets a small CTA that
  // reads its scores from L2 in every pass: the whole selection of one slot of 8190 candidates among 63 of 254 takes
  // 97 us, that of the one by itself 26, of the 63 36 (L2 flushed before each call).
  if (cand <= 1024ll * info.num_prefill_items)
    return a.head_dim == 128 ? go(choose_blocks_kernel<128, 128, 2048>, 128, 2048)
                             : go(choose_blocks_kernel<64, 128, 2048>, 128, 2048);
  return a.head_dim == 128 ? go(choose_blocks_kernel<128, 1024, 10240>, 1024, 10240)
                           : go(choose_blocks_kernel<64, 1024, 10240>, 1024, 10240);
}

}  // namespace pkv
