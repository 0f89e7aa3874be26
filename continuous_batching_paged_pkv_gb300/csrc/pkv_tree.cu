// Attention of trees of drafted tokens (tcgen05, keys split over CTAs).
//
// A segment's n rows see the L - n keys before the segment and, of the segment's
// own n keys, those whose bit is set in the row's mask:
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(scale log2(e) q_i . k_j - m_i)
// over the keys j that row i sees, m_i a running maximum. One CTA takes one or two
// 128-row query tiles of one (segment, kv head) -- rows are P positions x G grouped
// q heads, row m = position m / G, head m % G -- and one span of the keys, 64 at a
// time. A segment of one span stores its rows; otherwise every span leaves a
// partial (unnormalised sum, maximum, denominator) that the span merge of the
// decode kernels joins in order, so results do not depend on the rest of the step.
//
//   softmax warpgroup w  thread = TMEM lane = row of query tile w: takes S_u into
//                        registers, masks it where the unit reaches the segment's
//                        own keys, writes P_u as bf16 over S_u, rescales O when the
//                        running maximum grew by more than 2^8
//   producer warp        TMA: Q, then K_0, K_1, V_0, K_2, V_1, ... of 64 keys each
//                        through one ring, a 16-key sub-tile a box
//   score issuer         S_u = Q_w K_u^T (SS) of both tiles in turn, into the two
//                        buffers of a tile alternately, one unit ahead
//   value issuer         O_w += P_u V_u (TS) of both tiles in turn
//
// A unit is a chain S, softmax, P V of which each step leaves most of the SM idle.
// With two buffers of S a tile's next scores are there when its softmax is done.
// Products that add to one accumulator follow each other at some 90 cycles (scores)
// to 120 (values), twice what the tensor core needs, so a second tile's go in
// between: where a segment has more than one query tile (W = 2) the issuers take the
// two tiles of a CTA step by step in turn, and the tiles share every key that is
// loaded (TMEM: two times two S of 64 columns and O, 512 columns). Else two CTAs
// share an SM (W = 1), each with half of its shared memory, TMEM and registers.
// There are two issuers because an issue blocks its thread until the tensor core
// takes it.
//
// Measured: 64 slots x 32 nodes, 64 + 8 heads of 128, up to 8192 keys: 146-154 us, 766
// MB of keys and values at 5.0 TB/s; a unit of two tiles takes 1370 cycles, HBM's share
// of an SM is 1400, the rest is the CTAs' starts and ends (5 us each). One slot x 64
// nodes, 32 + 8 heads, 32,768 keys: 39.5 us with the merge (8), 5 slots x 8 nodes 20.
//
// Every mbarrier wait is bounded; on expiry the CTA records PKV_DEV_TIMEOUT,
// drains its MMAs, waits for its copies and frees its TMEM before it returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kTileKeys = kTreeTileKeys;  // spans are whole tiles
constexpr int kUnitKeys = 64, kUnitSubs = kUnitKeys / kSubKeys;
static_assert(kTreeMinSpanTiles * kTileKeys >= PKV_TREE_MAX_ROWS, "rows of a segment without a history are one span");
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kFull = 0xffffffffu;

template <int D, int W>
struct Cfg {
  static constexpr int kThreads = 128 * (W + 1);
  static constexpr int kWarpProducer = 4 * W, kWarpScores = 4 * W + 1, kWarpValues = 4 * W + 2;
  static constexpr int kLaunchRegs = W == 1 ? 128 : 168, kSoftmaxRegs = W == 1 ? 192 : 208, kOtherRegs = W == 1 ? 64 : 88;
  static_assert(W * kSoftmaxRegs + kOtherRegs == (W + 1) * kLaunchRegs, "register shares must add up to the launch's");
  static constexpr int kSlotBytes = kUnitKeys * D * 2;  // a ring slot holds a unit of K or V
  static constexpr int kSlots = D == 128 ? 5 * W : W == 1 ? 12 : 20;
  static constexpr int kSubBytes = kSubKeys * D * 2;         // one 16-key sub-tile, one box
  static constexpr int kGroupStep = D == 128 ? 2048 : 1024;  // from 8 keys to the next 8
  static constexpr int kHalfStep = 1024;                     // from one 64-column half of them to the other (D = 128)
  static constexpr int kQHalf = 128 * 128;                   // 64 columns of a query tile
  static constexpr int kQBytes = (D / 64) * kQHalf;
  static constexpr int kRingOffset = W * kQBytes;
  static constexpr int kBarOffset = kRingOffset + kSlots * kSlotBytes;
  static constexpr int kTmemCols = W * 256, kOCol = 128;  // tile w: its S and P buffers from 256 w on, O 128 columns behind
  // barriers
  static constexpr int kQFull = 0;
  static constexpr int kSlotFull = 1, kSlotEmpty = kSlotFull + kSlots;                      // + slot
  static constexpr int kSFull = kSlotEmpty + kSlots, kPVDone = kSFull + 2 * W;              // + 2 w + buffer
  static constexpr int kPReady = kPVDone + 2 * W, kDrain = kPReady + 2 * W, kNumBars = kDrain + 2;
  static_assert(kNumBars * 8 + 8 <= 512, "barriers, TMEM address and abort flag fit their 512 bytes");
  static constexpr int kSmem = kBarOffset + 512;
  static_assert((W == 1 ? 2 * (kSmem + 1024) : kSmem + 1024) <= kSmSmem, "shared memory of an SM");
  static_assert(tmem_apart(kTmemCols, kSmem), "beside a kernel that it lets start before it has its tensor memory");
};

// Wait that also gives up as soon as another role of this CTA has aborted, or after a second. The clock is looked at
// only now and then: every wait here is on the path of the tiles.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > 1000000000ull) {
        *abort = 1;
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool warp_wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(kFull, wait_or_abort(bar, parity, abort));
}

// Word k of a row's mask as far as the segment's n nodes go; every bit set before it (the history).
__device__ __forceinline__ uint32_t mask_word(const uint32_t *mask, int words, int n, int k) {
  if (k < 0) return ~0u;
  if (k >= words || k * 32 >= n) return 0u;
  const uint32_t m = __ldg(mask + k);
  return n - k * 32 >= 32 ? m : m & ((1u << (n - k * 32)) - 1u);
}

// Whether a row sees any of the places [r0, r1) among its segment's nodes, negative ones in the history. r1 - r0 is a
// multiple of 32, or r1 is the segment's end.
__device__ __forceinline__ bool sees_some(const uint32_t *mask, int words, int n, int r0, int r1) {
  if (r0 < 0) return true;
#pragma unroll 1
  for (int r = r0; r < r1; r += 32)
    if (__funnelshift_r(mask_word(mask, words, n, r >> 5), mask_word(mask, words, n, (r >> 5) + 1), r & 31)) return true;
  return false;
}

// Position in the ring of slots.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int k = 1) {
    slot += k;
    if (slot >= N) {
      slot -= N;
      phase ^= 1;
    }
  }
};

// 32 bytes with one store: a whole sector of L2, where lanes store to rows far apart.
__device__ __forceinline__ void store_32(void *p, const uint32_t *r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <int D, int W>
__global__ void __maxnreg__((Cfg<D, W>::kLaunchRegs))
    tree_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v, const StepArgs a, const int32_t *__restrict__ items,
                int rows_per_tile) {
  using C = Cfg<D, W>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::kBarOffset);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + C::kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = __shfl_sync(kFull, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int g = blockIdx.x % a.num_kv_heads;  // the longest items of all heads first
  // As in the other attention kernels: the work item, step metadata, q, the masks and the cached history are final
  // when this grid starts; the producer waits for the kernel before it at the first tile with rows of this step, and
  // everything that stores waits first.
  launch_dependents();
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmap_q);
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
  }
  // The item names the slot and the span, so that the block table is read beside the metadata, not behind it.
  const int4 it = __ldg(reinterpret_cast<const int4 *>(items) + blockIdx.x / a.num_kv_heads);
  const int seg = it.x, slot = it.y, pbase = it.w;
  const int span = (it.z >> 16 & 0xFF) + 1, tile0 = (it.z & 0xFFFF) * span;
  const int qt0 = static_cast<int>(static_cast<uint32_t>(it.z) >> 24);
  const int G = a.group, P = rows_per_tile;

  bool bad = seg < 0 || seg >= a.num_seqs || slot < 0 || slot >= a.max_slots;
  const int32_t *bt_row = a.block_tables + static_cast<int64_t>(bad ? 0 : slot) * a.max_blocks_per_slot;
  // lane l: key 16 (l % 8) of tile t0 + l / 8 of the span, and its block's ID (anything behind the table's end)
  auto key_of = [&](int t0) { return static_cast<int64_t>(tile0 + t0 + (lane >> 3)) * kTileKeys + (lane & 7) * kSubKeys; };
  auto group_ids = [&](int t0) -> int {
    const int64_t i = key_of(t0) / a.block_size;
    return i < a.max_blocks_per_slot ? __ldg(bt_row + i) : 0;
  };
  int ids0 = 0;
  if (!bad && warp == C::kWarpProducer) ids0 = group_ids(0);
  int row0 = 0, n = 0, L = 0;
  if (!bad) {
    row0 = __ldg(a.cu_seqlens_q + seg);
    n = __ldg(a.cu_seqlens_q + seg + 1) - row0;
    L = __ldg(a.context_lens + slot);
    const int64_t tiles = (static_cast<int64_t>(L) + kTileKeys - 1) / kTileKeys;
    bad = __ldg(a.seq_slot + seg) != slot || n < 1 || n > L || L > kTreeMaxKeys || n > PKV_TREE_MAX_ROWS || n > 32 * a.mask_words ||
          static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size || qt0 * P >= n ||
          tile0 >= tiles || row0 < 0 || static_cast<int64_t>(row0) + n > a.total_q ||
          (pbase >= 0 ? pbase > a.num_partials - n : tile0 != 0 || tiles > span);
  }
  if (bad || (smem_addr(smem) & 1023) != 0) {  // (the swizzled tiles need their alignment)
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    grid_dependency_wait();  // this grid ends after the kernel before it
    return;
  }
  const int ntiles = min(span, (L - 1) / kTileKeys + 1 - tile0);
  const int base = tile0 * kTileKeys;
  const int kv_end = static_cast<int>(min(static_cast<int64_t>(L), static_cast<int64_t>(base) + ntiles * kTileKeys));
  const int units = (kv_end - base + kUnitKeys - 1) / kUnitKeys;
  const int active = W == 2 && (qt0 + 1) * P < n ? 2 : 1;  // query tiles with rows

  // The producer starts on its own: it initialises the barriers, requests Q and fills the ring before it meets the
  // other warps, which clear the rest of the Q tiles and allocate TMEM meanwhile. Pool rows of the 16-key sub-tiles
  // come eight units (four tiles) per warp-wide load, those of the next eight beside them, raw block IDs of the eight
  // after that; an ID outside the pool is reported and reads block 0's rows.
  struct {
    Ring<C::kSlots> at;
    int next = 0;  // place in the order K_0, K_1, V_0, K_2, V_1, ..., V_units-1
    int rows = 0, rows_next = 0, ids = 0, group = 0;
    bool waited = false;
  } load;
  auto group_rows = [&](int t0, int blk) -> int {
    if (key_of(t0) >= kv_end) return 0;
    if (blk < 0 || blk >= a.num_blocks) {
      if (a.status) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
      blk = 0;
    }
    return (blk * a.num_kv_heads + g) * a.block_size + static_cast<int>(key_of(t0) % a.block_size);
  };
  // Request the next slot's boxes. The slot has to be free.
  auto fill = [&]() {
    const bool is_k = load.next == 0 || (load.next % 2 == 1 && load.next != 2 * units - 1);
    const int u = is_k ? (load.next + 1) / 2 : load.next == 2 * units - 1 ? units - 1 : load.next / 2 - 1;
    if ((u >> 3) > load.group + 1 || (!is_k && (u >> 3) > load.group)) {  // on to the next eight units
      ++load.group;
      load.rows = load.rows_next;
      load.rows_next = group_rows(4 * load.group + 4, load.ids);
      load.ids = group_ids(4 * load.group + 8);
    }
    if (!load.waited && base + (u + 1) * kUnitKeys > L - n) {
      grid_dependency_wait();
      load.waited = true;
    }
    const int count = min(kUnitSubs, (kv_end - base - u * kUnitKeys + kSubKeys - 1) / kSubKeys);  // sub-tiles with a key
    const int row = __shfl_sync(kFull, (u >> 3) == load.group ? load.rows : load.rows_next, (u & 7) * 4 + (lane & 3));
    uint64_t *full = bar + C::kSlotFull + load.at.slot;
    if (lane == 0) mbar_arrive_expect_tx(full, count * C::kSubBytes);
    __syncwarp();
    if (lane < count) {
      uint8_t *dst = smem + C::kRingOffset + load.at.slot * C::kSlotBytes + lane * C::kSubBytes;
      const CUtensorMap *map = is_k ? &tmap_k : &tmap_v;
      const uint64_t policy = l2_evict_first_policy();
      if constexpr (D == 128)
        tma_load_5d_hint(dst, map, 0, 0, 0, (row & (a.block_size - 1)) >> 3, row >> (31 - __clz(a.block_size)), full, policy);
      else
        tma_load_2d_hint(dst, map, 0, row, full, policy);
    }
    load.at.next();
    ++load.next;
  };
  if (warp == C::kWarpProducer) {
    if (lane == 0) {
      for (int i = 0; i < C::kNumBars; ++i)
        mbar_init(bar + i, i >= C::kPReady && i < C::kDrain ? 4 : 1);
      fence_barrier_init();
      *abort_flag = 0;
      mbar_arrive_expect_tx(bar + C::kQFull, active * (D / 64) * G * P * 128);
      for (int w = 0; w < active; ++w)
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(smem + w * C::kQBytes + h * C::kQHalf, &tmap_q, h * 64, g * G, row0 + (qt0 + w) * P, bar + C::kQFull);
    }
    load.ids = group_ids(4);
    load.rows = group_rows(0, ids0);
    __syncwarp();
    fill();  // the first keys go ahead of the rest of the ring
    load.rows_next = group_rows(4, load.ids);
    load.ids = group_ids(8);
  } else {
    // Rows of the Q tiles beyond G * P whole groups stay zero.
    const int qrows = G * P, chunks = (128 - qrows) * 8;
    const int other = threadIdx.x < 32 * C::kWarpProducer ? threadIdx.x : threadIdx.x - 32;  // place among the other warps
    for (int i = other; i < chunks * (D / 64) * W; i += blockDim.x - 32) {
      const int h = i / chunks, rem = i % chunks;
      *reinterpret_cast<uint4 *>(smem + h * C::kQHalf + (qrows + rem / 8) * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == C::kWarpScores) {
      tmem_alloc(tmem_slot, C::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 4 * W) {
    setmaxnreg_dec<C::kOtherRegs>();
    if (warp == C::kWarpProducer) {
      // ---------------------------------------------------------- producer
      warp_wait_or_abort(bar + C::kSlotFull, 0, abort_flag);
      while (load.next < 2 * units) {
        if (load.next >= C::kSlots &&
            !warp_wait_or_abort(bar + C::kSlotEmpty + load.at.slot, load.at.phase ^ 1, abort_flag))
          break;
        fill();
      }
    } else if (warp == C::kWarpScores) {
      // ---------------------------------------------------------- score issuer
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kUnitKeys, 0, 0);
      const uint64_t q_desc = smem_desc_sw128(smem_addr(smem), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_addr(smem + C::kRingOffset), 16, C::kGroupStep);
      Ring<C::kSlots> at;
      bool ok = warp_wait_or_abort(bar + C::kQFull, 0, abort_flag);
      for (int u = 0; ok && u < units; ++u) {
        if (!(ok = warp_wait_or_abort(bar + C::kSlotFull + at.slot, at.phase, abort_flag))) break;
        const uint64_t k0 = k_desc + at.slot * (C::kSlotBytes >> 4);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (w >= active) break;
          // the buffer holds P_{u-2} until its product is done
          if (u >= 2 && !(ok = warp_wait_or_abort(bar + C::kPVDone + 2 * w + (u & 1), ((u - 2) >> 1) & 1, abort_flag))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma_ss_warp(tmem + w * 256 + (u & 1) * kUnitKeys,
                           q_desc + ((w * C::kQBytes + (kk >> 2) * C::kQHalf + (kk & 3) * 32) >> 4),
                           k0 + (((kk >> 2) * C::kHalfStep + (kk & 3) * 32) >> 4), idesc_qk, kk > 0 ? 1u : 0u);
          tc_commit_warp(bar + C::kSFull + 2 * w + (u & 1));
        }
        if (!ok) break;
        tc_commit_warp(bar + C::kSlotEmpty + at.slot);
        at.next(u == 0 ? 1 : 2);
      }
      tc_commit_warp(bar + C::kDrain);
      if (!warp_wait_or_abort(bar + C::kDrain, 0, abort_flag) && lane == 0 && a.status) atomicOr(a.status, PKV_DEV_TIMEOUT);
    } else if (warp == C::kWarpValues) {
      // ---------------------------------------------------------- value issuer
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t v_desc = smem_desc_sw128(smem_addr(smem + C::kRingOffset), C::kHalfStep, C::kGroupStep);
      Ring<C::kSlots> at;
      at.next(units > 1 ? 2 : 1);
      bool ok = true;
      for (int u = 0; ok && u < units; ++u) {
        if (!(ok = warp_wait_or_abort(bar + C::kSlotFull + at.slot, at.phase, abort_flag))) break;
        const uint64_t v0 = v_desc + at.slot * (C::kSlotBytes >> 4);
        const int ksteps = (min(kUnitKeys, kv_end - base - u * kUnitKeys) + kSubKeys - 1) / kSubKeys;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (w >= active) break;
          if (!(ok = warp_wait_or_abort(bar + C::kPReady + 2 * w + (u & 1), (u >> 1) & 1, abort_flag))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < kUnitSubs; ++ks)
            if (ks < ksteps)
              tc_mma_ts_warp(tmem + w * 256 + C::kOCol, tmem + w * 256 + (u & 1) * kUnitKeys + ks * 8,
                             v0 + (ks * C::kSubBytes >> 4), idesc_pv, (u > 0 || ks > 0) ? 1u : 0u);
          tc_commit_warp(bar + C::kPVDone + 2 * w + (u & 1));
        }
        if (!ok) break;
        tc_commit_warp(bar + C::kSlotEmpty + at.slot);
        at.next(u + 2 == units ? 1 : 2);
      }
      tc_commit_warp(bar + C::kDrain + 1);
      if (!warp_wait_or_abort(bar + C::kDrain + 1, 0, abort_flag) && lane == 0 && a.status)
        atomicOr(a.status, PKV_DEV_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<C::kSoftmaxRegs>();
    const int w = W == 1 ? 0 : warp >> 2, quarter = warp & 3;
    if (w < active) {
      const int mrow = quarter * 32 + lane;
      const uint32_t s_base = tmem + w * 256 + (static_cast<uint32_t>(quarter * 32) << 16), o_col = s_base + C::kOCol;
      const int i = (qt0 + w) * P + mrow / G, h = g * G + mrow % G;  // the row's node and q head
      const bool stored = mrow < G * P && i < n;
      const uint32_t *mask = a.masks + (static_cast<int64_t>(row0) + (stored ? i : 0)) * a.mask_words;
      const float sl2 = a.scale_log2;
      float m_used = -INFINITY;  // log2 units
      float l_sum = 0.f, l_odd = 0.f;  // even and odd keys
      bool ok = true;
      for (int u = 0; u < units; ++u) {
        const int kt0 = base + u * kUnitKeys, b = u & 1;
        const uint32_t s_col = s_base + b * kUnitKeys;
        if (!(ok = warp_wait_or_abort(bar + C::kSFull + 2 * w + b, (u >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t sv[2][32];
        tmem_ld32(s_col, sv[0]);
        tmem_ld32(s_col + 32, sv[1]);
        tmem_wait_ld();
        if (kt0 + kUnitKeys > L - n) {  // the unit reaches the segment's own keys (or the end)
          const int r0 = kt0 - (L - n);  // its first key as a node, negative in the history
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int k = r0 + 32 * c;
            const uint32_t seen = k <= -32 ? ~0u
                                           : __funnelshift_r(mask_word(mask, a.mask_words, n, k >> 5),
                                                             mask_word(mask, a.mask_words, n, (k >> 5) + 1), k & 31);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(seen & (1u << x))) sv[c][x] = 0xff800000u;
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < kUnitKeys; x += 2)
          top[(x >> 1) & 3] = max3(top[(x >> 1) & 3], __uint_as_float(sv[x >> 5][x & 31]), __uint_as_float(sv[x >> 5][(x & 31) + 1]));
        const float m_new = fmaxf(m_used, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sl2);
        // before a row's first visible key there is nothing to rescale
        const bool fresh = m_used == -INFINITY;
        const bool need = !fresh && m_new > m_used + kRescaleThreshold;
        if (fresh) m_used = m_new;
        if (__any_sync(kFull, need)) {
          // (a row that needs it saw keys before, so u > 0)
          if (u > 0 && !(ok = warp_wait_or_abort(bar + C::kPVDone + 2 * w + (b ^ 1), ((u - 1) >> 1) & 1, abort_flag))) break;
          tc_fence_after();
          const float corr = need ? ex2_approx(m_used - m_new) : 1.f;
          if (need) m_used = m_new;
          l_sum *= corr;
          l_odd *= corr;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t ov[16];
            tmem_ld16(o_col + c * 16, ov);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * corr);
            tmem_st16(o_col + c * 16, ov);
          }
        }
        const float nm = m_used == -INFINITY ? 0.f : -m_used;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float x0, x1;
            fma2(x0, x1, __uint_as_float(sv[c][2 * x]), __uint_as_float(sv[c][2 * x + 1]), sl2, sl2, nm, nm);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            add2(l_sum, l_odd, p0, p1);
            pk[x] = pack_bf16x2(p0, p1);
          }
          tmem_st16(s_col + c * 16, pk);
        }
        // Zero the V rows past the context inside the final 16-key step: a block may hold stale or NaN rows there,
        // and 0 * NaN would reach O. (Both tiles' warps write the same zeros, each before its own product.)
        const int valid = kv_end - kt0, tail = valid < kUnitKeys ? (kSubKeys - valid % kSubKeys) % kSubKeys : 0;
        if (tail) {  // the last unit, whose values are the last slot's
          const int s = 2 * units - 1;
          if (!(ok = warp_wait_or_abort(bar + C::kSlotFull + s % C::kSlots, (s / C::kSlots) & 1, abort_flag))) break;
          uint8_t *v = smem + C::kRingOffset + (s % C::kSlots) * C::kSlotBytes;
          for (int x = threadIdx.x & 127; x < tail * (D / 8); x += 128) {
            const int r = valid + x / (D / 8), chunk = x % (D / 8);
            *reinterpret_cast<uint4 *>(v + (r >> 3) * C::kGroupStep + (chunk >> 3) * C::kHalfStep + (r & 7) * 128 +
                                       (chunk & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + C::kPReady + 2 * w + b);
      }
      if (ok && warp_wait_or_abort(bar + C::kPVDone + 2 * w + ((units - 1) & 1), ((units - 1) >> 1) & 1, abort_flag)) {
        tc_fence_after();
        grid_dependency_wait();  // the kernel before may write the same output or use the same workspace
        const float l = l_sum + l_odd;
        // A row that sees no key of the span gives zeros, whatever O holds. Its maximum alone does not tell: scores that
        // are all NaN leave it at -infinity too, and have to come through.
        const bool unseen = m_used == -INFINITY && !sees_some(mask, a.mask_words, n, base - (L - n), kv_end - (L - n));
        __syncwarp();
        const bool wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;  // rows of 128 or 256 bytes
        if (pbase < 0) {
          const float inv = unseen ? 0.f : 1.f / l;
          __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + (static_cast<int64_t>(row0 + i) * a.num_q_heads + h) * D;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_col + c * 32, ov);
            tmem_wait_ld();
            uint32_t pk[16];
#pragma unroll
            for (int x = 0; x < 16; ++x)
              pk[x] = unseen ? 0u : pack_bf16x2(__uint_as_float(ov[2 * x]) * inv, __uint_as_float(ov[2 * x + 1]) * inv);
            if (stored && wide_out) {
              store_32(dst + c * 32, pk);
              store_32(dst + c * 32 + 16, pk + 8);
            } else if (stored) {
#pragma unroll
              for (int v = 0; v < 4; ++v)
                reinterpret_cast<uint4 *>(dst)[c * 4 + v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
            }
          }
        } else {
          const int64_t e = (static_cast<int64_t>(pbase) + (stored ? i : 0)) * a.num_q_heads + h;
          float *dst = a.partial_acc + e * D;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_col + c * 32, ov);
            tmem_wait_ld();
            if (unseen)
#pragma unroll
              for (int x = 0; x < 32; ++x) ov[x] = 0;
            if (stored)
#pragma unroll
              for (int v = 0; v < 4; ++v) store_32(dst + c * 32 + v * 8, ov + 8 * v);
          }
          if (stored) {
            // (the first span of a row has a maximum, unless all its scores are NaN: a segment of several spans has a
            // history. A later one of the segment's own keys alone may have none, and no weight in the merge.)
            reinterpret_cast<float2 *>(a.partial_ml)[e] = make_float2(m_used, l);
          }
        }
      }
    }
  }

  grid_dependency_wait();  // this grid ends after the kernel before it, whatever its roles did
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, PKV_DEV_TIMEOUT);
    if (warp == C::kWarpProducer) {  // the copies in flight still write to this CTA's shared memory
      int late = 0;
      wait_or_abort(bar + C::kQFull, 0, &late);
      for (int i = max(0, load.next - C::kSlots); i < load.next; ++i)
        wait_or_abort(bar + C::kSlotFull + i % C::kSlots, (i / C::kSlots) & 1, &late);
    }
  }
  if (warp == C::kWarpScores) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int W>
cudaError_t launch_t(const StepArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     int32_t num_items, const int32_t *items, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};  // one bit per device
  if (const cudaError_t e = allow_smem_once(tree_kernel<D, W>, Cfg<D, W>::kSmem, configured); e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(num_items) * static_cast<unsigned>(a.num_kv_heads));
  return launch_pdl(tree_kernel<D, W>, grid, dim3(Cfg<D, W>::kThreads), Cfg<D, W>::kSmem, stream, tq, tk, tv, a, items,
                    prefill_rows_per_tile(a.group));
}

}  // namespace

cudaError_t launch_tree(const StepArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                        int32_t num_items, const int32_t *items, cudaStream_t stream) {
  if (num_items <= 0) return cudaSuccess;
  const bool two = tree_tiles_per_cta(a.decode_rows_max, a.group) == 2;
  if (a.head_dim == 128)
    return two ? launch_t<128, 2>(a, tq, tk, tv, num_items, items, stream)
               : launch_t<128, 1>(a, tq, tk, tv, num_items, items, stream);
  return two ? launch_t<64, 2>(a, tq, tk, tv, num_items, items, stream)
             : launch_t<64, 1>(a, tq, tk, tv, num_items, items, stream);
}

}  // namespace pkv
