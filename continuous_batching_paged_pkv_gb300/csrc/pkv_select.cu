// The blocks that a block-sparse step reads: an upper bound of every cached
// block's scores, and the best blocks by it.
//
// With lo, hi the bounds of a block's keys and q one query row of the kv head's
// group, no key k of the block has q . k above
//   s = sum_d max(q_d lo_d, q_d hi_d) = max(q, 0) . hi + min(q, 0) . lo,
// so a block's score, the maximum of s over the segment's rows and the group's
// heads, is one matrix product of depth 2 D and a maximum.
//
// Scoring kernel: CTA (128 candidate blocks, kv head); a warp takes 16 blocks.
// Their bounds go from global memory straight into MMA operands (m16n8k16, blocks
// on M, the (row, head) columns on N): the order of the depth is free as long as
// both operands share it, so a thread's 16-byte piece of a row serves two steps.
// Each bound is read once; the kernel is bound by HBM. A second product of the
// magnitudes gives A = sum |terms|: the tensor core adds 17 numbers to fp32 in an
// order of its own (each step within 17 * 2^-23 of its largest, the running sum
// rounded 2 D / 16 times), so a score is within 2^-18 A of the exact sum.
//
// Choosing kernel: CTA (segment, kv head). The k-th largest fp32 score T comes from
// a search over the bits of the ordered scores. With E the error bound, what is
// above T + 2 E is in, what is below T - 2 E is out, and only the blocks between
// are summed again, in fp64 (products of two bf16 are exact there), and ranked by
// (score, lower place first). So the choice is that of the exact scores, whatever
// the order of the sums, and every run gives the same. Then the chosen places are
// written in growing order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kScoreError = 0x1.01p-18f;  // of the sum of magnitudes, whose own error is in the last digits

// A segment of a selection item, checked against the step's metadata.
struct Chosen {
  int row0, n, slot;
  SparseBlocks b;
  int cand;  // candidates (0 where every block is read)
  bool ok;
};

__device__ __forceinline__ Chosen chosen_segment(const StepArgs &a, int seg, int slot, int max_cols) {
  Chosen c{};
  c.slot = slot;
  c.ok = seg >= 0 && seg < a.num_seqs && slot >= 0 && slot < a.max_slots;
  if (!c.ok) return c;
  c.row0 = __ldg(a.cu_seqlens_q + seg);
  c.n = __ldg(a.cu_seqlens_q + seg + 1) - c.row0;
  const int L = __ldg(a.context_lens + slot);
  c.ok = __ldg(a.seq_slot + seg) == slot && c.n >= 1 && c.n <= L && c.n * a.group <= max_cols && c.row0 >= 0 &&
         static_cast<int64_t>(c.row0) + c.n <= a.total_q &&
         L <= static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size;
  if (!c.ok) return c;
  c.b = sparse_blocks(L, c.n, a.block_size, a.top_blocks, a.keep_first, a.keep_last);
  c.cand = c.b.blocks > c.b.read ? static_cast<int>(c.b.last - c.b.first) : 0;
  c.ok = c.b.blocks <= c.b.read || c.b.first + (c.b.blocks - c.b.last) <= c.b.read;
  return c;
}

__device__ __forceinline__ uint32_t part(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// A bf16 pair's values above zero, and those below.
__device__ __forceinline__ uint32_t above(uint32_t x) {
  const uint32_t neg = (x >> 15) & 0x00010001u;
  return x & ~(neg * 0xFFFFu);
}
__device__ __forceinline__ uint32_t below(uint32_t x) {
  const uint32_t neg = (x >> 15) & 0x00010001u;
  return x & (neg * 0xFFFFu);
}

template <int D, int NT>
__global__ void __launch_bounds__(256) score_blocks_kernel(const StepArgs a, const __nv_bfloat16 *__restrict__ bounds,
                                                           const int32_t *__restrict__ items, int64_t candidates,
                                                           float *__restrict__ scores, float *__restrict__ sums) {
  grid_dependency_wait();  // q and the bounds come from earlier work
  launch_dependents();
  constexpr int P = D / 32;  // 32-value pieces of a row of lo (or hi), and of q
  __shared__ uint32_t largest;
  if (threadIdx.x == 0) largest = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.y;
  const int4 it = __ldg(reinterpret_cast<const int4 *>(items) + blockIdx.x);
  const int c0 = it.z, base = it.w;
  Chosen c = chosen_segment(a, it.x, it.y, 8 * NT);
  const bool ok = c.ok && c0 >= 0 && c0 < c.cand && base >= 0 && static_cast<int64_t>(base) + c.cand <= candidates;
  if (!ok) {
    if (threadIdx.x == 0) {
      if (a.status && g == 0) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
      sums[static_cast<int64_t>(blockIdx.x) * a.num_kv_heads + g] = 0.f;
    }
    return;
  }
  const int t = lane & 3, cols = c.n * a.group;
  const int32_t *table = a.block_tables + static_cast<int64_t>(c.slot) * a.max_blocks_per_slot;
  // rows lane / 4 and lane / 4 + 8 of the warp's 16 blocks
  uint4 lo[2][P], hi[2][P];
  bool live[2], bad[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int j = c0 + warp * 16 + (lane >> 2) + 8 * r;
    live[r] = j < c.cand;
    const int bid = live[r] ? __ldg(table + c.b.first + j) : 0;
    bad[r] = bid < 0 || bid >= a.num_blocks;
    const uint4 *row = reinterpret_cast<const uint4 *>(
                           bounds + (static_cast<int64_t>(live[r] && !bad[r] ? bid : 0) * a.num_kv_heads + g) * 2 * D) + t;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      lo[r][p] = live[r] && !bad[r] ? __ldcg(row + p * 4) : make_uint4(0, 0, 0, 0);
      hi[r][p] = live[r] && !bad[r] ? __ldcg(row + (P + p) * 4) : make_uint4(0, 0, 0, 0);
    }
  }
  float best[2] = {-INFINITY, -INFINITY}, mag = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = nt * 8 + (lane >> 2);
    const bool valid = col < cols;
    const uint4 *qrow = reinterpret_cast<const uint4 *>(
                            static_cast<const __nv_bfloat16 *>(a.q) +
                            ((static_cast<int64_t>(c.row0) + (valid ? col / a.group : 0)) * a.num_q_heads +
                             g * a.group + (valid ? col % a.group : 0)) * D) + t;
    float s[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint4 q = valid ? __ldg(qrow + p * 4) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 &x0 = half ? hi[0][p] : lo[0][p], &x1 = half ? hi[1][p] : lo[1][p];
          const uint32_t b0 = half ? above(part(q, 2 * k)) : below(part(q, 2 * k));
          const uint32_t b1 = half ? above(part(q, 2 * k + 1)) : below(part(q, 2 * k + 1));
          const uint32_t af[4] = {part(x0, 2 * k), part(x1, 2 * k), part(x0, 2 * k + 1), part(x1, 2 * k + 1)};
          float d[4] = {0.f, 0.f, 0.f, 0.f};  // each step's sum starts anew, for the error bound
          mma_bf16_16816(d, af, b0, b1);
          const uint32_t aa[4] = {af[0] & 0x7FFF7FFFu, af[1] & 0x7FFF7FFFu, af[2] & 0x7FFF7FFFu, af[3] & 0x7FFF7FFFu};
          mma_bf16_16816(m, aa, b0 & 0x7FFF7FFFu, b1 & 0x7FFF7FFFu);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] += d[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // block lane / 4 (+ 8 for i >= 2), column nt * 8 + 2 t + (i & 1)
      if (nt * 8 + 2 * t + (i & 1) >= cols) continue;
      mag = m[i] <= mag ? mag : m[i];  // keeps a NaN
      if (s[i] == s[i]) best[i >> 1] = fmaxf(best[i >> 1], s[i]);
    }
  }
  float *out = scores + static_cast<int64_t>(base) * a.num_kv_heads + static_cast<int64_t>(g) * c.cand;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    best[r] = fmaxf(best[r], __shfl_xor_sync(kAll, best[r], 1));
    best[r] = fmaxf(best[r], __shfl_xor_sync(kAll, best[r], 2));
    if (live[r] && t == 0) {
      if (bad[r] && a.status && g == 0) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
      out[c0 + warp * 16 + (lane >> 2) + 8 * r] = bad[r] ? -INFINITY : best[r] + 0.f;
    }
  }
  // non-negative floats order as their bits do; a NaN is above infinity there
  const uint32_t most = __reduce_max_sync(kAll, __float_as_uint(mag) & 0x7FFFFFFFu);
  if (lane == 0) atomicMax(&largest, most);
  __syncthreads();
  if (threadIdx.x == 0) sums[static_cast<int64_t>(blockIdx.x) * a.num_kv_heads + g] = __uint_as_float(largest);
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

// Block-wide sums; two buffers, so that one barrier per sum is enough.
template <int T>
struct Counter {
  uint32_t (*buf)[32];
  int turn;
  __device__ __forceinline__ uint32_t sum(uint32_t x) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t w = __reduce_add_sync(kAll, x);
    turn ^= 1;
    if (lane == 0) buf[turn][warp] = w;
    __syncthreads();
    return __reduce_add_sync(kAll, lane < T / 32 ? buf[turn][lane] : 0u);
  }
  __device__ __forceinline__ uint32_t least(uint32_t x) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t w = __reduce_min_sync(kAll, x);
    turn ^= 1;
    if (lane == 0) buf[turn][warp] = w;
    __syncthreads();
    return __reduce_min_sync(kAll, lane < T / 32 ? buf[turn][lane] : ~0u);
  }
  // Sum of the threads before this one.
  __device__ __forceinline__ uint32_t before(uint32_t x) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    turn ^= 1;
    if (lane == 31) buf[turn][warp] = incl;
    __syncthreads();
    const uint32_t prior = __reduce_add_sync(kAll, lane < warp ? buf[turn][lane] : 0u);
    return prior + incl - x;
  }
};

// Exact score of candidate j, by one warp.
template <int D>
__device__ __forceinline__ double exact_score(const StepArgs &a, const __nv_bfloat16 *bounds, const Chosen &c, int g,
                                              int j) {
  const int lane = threadIdx.x & 31;
  const int bid = __ldg(a.block_tables + static_cast<int64_t>(c.slot) * a.max_blocks_per_slot + c.b.first + j);
  if (bid < 0 || bid >= a.num_blocks) return -INFINITY;
  const __nv_bfloat16 *lo = bounds + (static_cast<int64_t>(bid) * a.num_kv_heads + g) * 2 * D;
  double l[D / 32], h[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    l[i] = __bfloat162float(lo[lane + 32 * i]);
    h[i] = __bfloat162float(lo[D + lane + 32 * i]);
  }
  double best = -INFINITY;
  for (int col = 0; col < c.n * a.group; ++col) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                             ((static_cast<int64_t>(c.row0) + col / a.group) * a.num_q_heads + g * a.group + col % a.group) * D;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float x = __bfloat162float(q[lane + 32 * i]);
      s += static_cast<double>(x) * (x < 0.f ? l[i] : h[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(kAll, s, o);
    if (s == s && s > best) best = s;
  }
  return best + 0.0;
}

// T threads, each with `per` consecutive candidates, so that threads are in the candidates' order; up to R of
// them in registers (else they are read again in every pass, from L2).
template <int D, int T>
__global__ void __launch_bounds__(T) choose_blocks_kernel(const StepArgs a, const __nv_bfloat16 *__restrict__ bounds,
                                                          const int32_t *__restrict__ items, int64_t candidates,
                                                          const float *__restrict__ scores,
                                                          const float *__restrict__ sums, int num_score_items,
                                                          const int32_t *__restrict__ score_items,
                                                          double *__restrict__ exact, int32_t *__restrict__ selected) {
  grid_dependency_wait();
  launch_dependents();
  extern __shared__ uint32_t taken[];  // a bit per candidate: chosen among those between the bounds
  __shared__ uint32_t s_count[2][32];
  __shared__ int s_list[kListed];
  __shared__ double s_exact[kListed];
  __shared__ uint32_t s_listed;
  constexpr int R = 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = blockIdx.y;
  const int4 it = __ldg(reinterpret_cast<const int4 *>(items) + blockIdx.x);
  const Chosen c = chosen_segment(a, it.x, it.y, 16);
  const int base = it.z, N = it.w;
  if (!(it.x >= 0 && it.x < a.num_seqs)) {
    if (tid == 0 && a.status && g == 0) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    return;
  }
  int32_t *out = selected + (static_cast<int64_t>(it.x) * a.num_kv_heads + g) * a.top_blocks;
  const bool ok = c.ok && c.cand == N && base >= 0 && static_cast<int64_t>(base) + N <= candidates &&
                  (N + 31) / 32 <= (a.max_blocks_per_slot + 31) / 32;
  if (!ok) {
    if (tid == 0 && a.status && g == 0) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    for (int i = tid; i < a.top_blocks; i += T) out[i] = -1;
    return;
  }
  const int first = static_cast<int>(c.b.first), tail = static_cast<int>(c.b.blocks - c.b.last);
  const int need = N > 0 ? static_cast<int>(c.b.read) - first - tail : 0;
  if (N == 0) {  // every block
    for (int i = tid; i < a.top_blocks; i += T) out[i] = i < c.b.blocks ? i : -1;
    return;
  }
  // the blocks that are always read, and what is left empty
  for (int i = tid; i < first; i += T) out[i] = i;
  for (int i = tid; i < tail; i += T) out[first + need + i] = static_cast<int>(c.b.last) + i;
  for (int i = static_cast<int>(c.b.read) + tid; i < a.top_blocks; i += T) out[i] = -1;
  if (need == 0) return;
  const int64_t at = static_cast<int64_t>(base) * a.num_kv_heads + static_cast<int64_t>(g) * N;
  const float *sc = scores + at;
  const int per = (N + T - 1) / T, j0 = min(tid * per, N), j1 = min(j0 + per, N);
  const bool in_regs = per <= R;
  uint32_t key[R];
  if (in_regs) {
#pragma unroll
    for (int i = 0; i < R; ++i) key[i] = j0 + i < j1 ? ordered(__ldcg(sc + j0 + i)) : 0u;
  }
  if (tid == 0) s_listed = 0;
  for (int i = tid; i < (N + 31) / 32; i += T) taken[i] = 0;
  // f(j, key) for this thread's candidates
  auto each = [&](auto f) {
    if (in_regs) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (j0 + i < j1) f(j0 + i, key[i]);
    } else {
      for (int j = j0; j < j1; ++j) f(j, ordered(__ldcg(sc + j)));
    }
  };
  Counter<T> count{s_count, 0};
  // the largest sum of magnitudes among the segment's scoring items
  uint32_t mag = 0;
  for (int i = tid; i < num_score_items; i += T) {
    const int4 si = __ldg(reinterpret_cast<const int4 *>(score_items) + i);
    if (si.x == it.x) mag = max(mag, __float_as_uint(__ldcg(sums + static_cast<int64_t>(i) * a.num_kv_heads + g)));
  }
  mag = ~count.least(~mag);
  const float error = __uint_as_float(mag) * kScoreError;
  // largest x that `need` candidates reach, bit by bit; done early where exactly `need` do
  uint32_t x = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t y = x | 1u << bit;
    uint32_t n = 0;
    each([&](int, uint32_t k) { n += k >= y; });
    n = count.sum(n);
    if (n >= static_cast<uint32_t>(need)) x = y;
    if (n == static_cast<uint32_t>(need)) break;
  }
  uint32_t lowest = ~0u;
  each([&](int, uint32_t k) { if (k >= x) lowest = min(lowest, k); });
  const float T0 = unordered(count.least(lowest));
  float low = __fsub_rd(T0, 2.f * error), high = __fadd_ru(T0, 2.f * error);
  if (!(low <= T0)) low = -INFINITY;    // infinities and NaN among the terms: all are summed again
  if (!(high >= T0)) high = INFINITY;
  const uint32_t klow = ordered(low + 0.f), khigh = ordered(high + 0.f);
  uint32_t over = 0, between = 0;
  each([&](int, uint32_t k) {
    over += k > khigh;
    between += k >= klow && k <= khigh;
  });
  over = count.sum(over);
  const uint32_t m = count.sum(between), r = static_cast<uint32_t>(need) - over;  // r of m, r >= 1
  const bool all = m == r;
  if (!all && m <= kListed) {
    each([&](int j, uint32_t k) {
      if (k >= klow && k <= khigh) s_list[atomicAdd(&s_listed, 1u)] = j;
    });
    __syncthreads();
    for (uint32_t i = warp; i < m; i += T / 32) {
      const double s = exact_score<D>(a, bounds, c, g, s_list[i]);
      if (lane == 0) s_exact[i] = s;
    }
    __syncthreads();
    for (uint32_t i = tid; i < m; i += T) {
      const double s = s_exact[i];
      const int j = s_list[i];
      uint32_t better = 0;
      for (uint32_t o = 0; o < m; ++o) better += s_exact[o] > s || (s_exact[o] == s && s_list[o] < j);
      if (better < r) atomicOr(&taken[j / 32], 1u << (j % 32));
    }
    __syncthreads();
  } else if (!all) {
    // Many equal (or indistinguishable) scores: the same choice with the exact scores in memory, the r-th
    // largest of them found bit by bit, equal ones taken from the lowest place on.
    double *ex = exact + at;
    for (int j = warp; j < N; j += T / 32) {
      const uint32_t k = ordered(__ldcg(sc + j));
      if (k < klow || k > khigh) continue;
      const double s = exact_score<D>(a, bounds, c, g, j);
      if (lane == 0) ex[j] = s;
    }
    __syncthreads();
    uint64_t v = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t y = v | 1ull << bit;
      uint32_t n = 0;
      each([&](int j, uint32_t k) { n += k >= klow && k <= khigh && ordered(ex[j]) >= y; });
      if (count.sum(n) >= r) v = y;
    }
    uint32_t above_v = 0, equal = 0;
    each([&](int j, uint32_t k) {
      if (k < klow || k > khigh) return;
      const uint64_t e = ordered(ex[j]);
      above_v += e > v;
      equal += e == v;
    });
    above_v = count.sum(above_v);
    uint32_t rank = count.before(equal);
    each([&](int j, uint32_t k) {
      if (k < klow || k > khigh) return;
      const uint64_t e = ordered(ex[j]);
      if (e > v || (e == v && rank++ < r - above_v)) atomicOr(&taken[j / 32], 1u << (j % 32));
    });
    __syncthreads();
  }
  auto in = [&](int j, uint32_t k) { return k > khigh || (k >= klow && (all || (taken[j / 32] >> (j % 32) & 1u))); };
  uint32_t mine = 0;
  each([&](int j, uint32_t k) { mine += in(j, k); });
  uint32_t place = count.before(mine);
  each([&](int j, uint32_t k) {
    if (in(j, k) && place < static_cast<uint32_t>(need)) out[first + place++] = first + j;
  });
}

}  // namespace

cudaError_t launch_select_blocks(const StepArgs &a, const void *bounds, const pkv_work_info &info, void *workspace,
                                 int32_t *selected, cudaStream_t stream) {
  const int64_t cand = info.scratch_blocks;
  const SelectLayout lay = select_layout(cand, info.num_scratch_items, a.num_kv_heads);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  double *exact = reinterpret_cast<double *>(ws + lay.exact);
  float *scores = reinterpret_cast<float *>(ws + lay.scores), *sums = reinterpret_cast<float *>(ws + lay.sums);
  auto *b = static_cast<const __nv_bfloat16 *>(bounds);
  const int32_t *pre = a.work + static_cast<int64_t>(info.num_decode_items) * PKV_WORK_WORDS_PER_ITEM;
  const int32_t *scr = pre + (static_cast<int64_t>(info.num_prefill_items) + info.num_combine_items) * PKV_WORK_WORDS_PER_ITEM;
  const unsigned heads = static_cast<unsigned>(a.num_kv_heads);
  if (info.num_scratch_items > 0) {
    const bool wide = info.decode_rows_max * a.group > 8;
    auto *kernel = a.head_dim == 128 ? (wide ? score_blocks_kernel<128, 2> : score_blocks_kernel<128, 1>)
                                     : (wide ? score_blocks_kernel<64, 2> : score_blocks_kernel<64, 1>);
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(info.num_scratch_items), heads), dim3(256), 0,
                                     stream, a, b, scr, cand, scores, sums);
    if (e != cudaSuccess) return e;
  }
  if (info.num_prefill_items == 0) return cudaSuccess;
  const int smem = (a.max_blocks_per_slot + 31) / 32 * 4;
  const dim3 grid(static_cast<unsigned>(info.num_prefill_items), heads);
  // few candidates per segment: small CTAs, several to an SM
  const bool small = cand <= 2048ll * info.num_prefill_items;
  auto go = [&](auto *kernel, int threads) -> cudaError_t {
    if (smem > 40 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, grid, dim3(threads), smem, stream, a, b, pre, cand, scores, sums,
                      static_cast<int>(info.num_scratch_items), scr, exact, selected);
  };
  if (a.head_dim == 128)
    return small ? go(choose_blocks_kernel<128, 256>, 256) : go(choose_blocks_kernel<128, 1024>, 1024);
  return small ? go(choose_blocks_kernel<64, 256>, 256) : go(choose_blocks_kernel<64, 1024>, 1024);
}

}  // namespace pkv
