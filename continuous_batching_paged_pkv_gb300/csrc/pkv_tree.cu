// Attention of trees of drafted tokens (tcgen05, keys split over CTAs).
//
// A segment's n rows see the L - n keys before the segment and, of the segment's
// own n keys, those whose bit is set in the row's mask:
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(scale log2(e) q_i . k_j - m_i)
// over the keys j that row i sees, m_i a running maximum. One CTA takes one or two
// 128-row query tiles of one (segment, kv head) -- rows are P positions x G grouped
// q heads, row m = position m / G, head m % G -- and one span of the keys, in tiles
// of 128. A segment of one span stores its rows; otherwise every span leaves a
// partial (unnormalised sum, maximum, denominator) that the span merge of the
// decode kernels joins in order, so results do not depend on the rest of the step.
//
//   softmax warpgroup w  thread = TMEM lane = row of query tile w: takes S_j into
//                        registers, masks it where the tile reaches the segment's
//                        own keys, writes P_j as bf16 over S_j, rescales O when the
//                        running maximum grew by more than 2^8
//   producer warp        TMA: Q, then K_0, V_0, K_1, V_1, ... through one ring, a
//                        16-key sub-tile a box
//   issuer warp w        S = Q_w K_j^T (SS), then O_w += P_j V_j (TS) when P_j is
//                        written; S_{j+1} follows when that product is done, since
//                        P shares S's columns
//
// A tile is a chain S, softmax, P V; what hides it is a second chain. Where a
// segment has more than one query tile (W = 2) the two tiles of a CTA share every
// key that it loads, and one's softmax runs under the other's products (TMEM: two
// times S and O, 512 columns). Else two CTAs share an SM (W = 1), each with half of
// its shared memory, TMEM and registers.
//
// Every mbarrier wait is bounded; on expiry the CTA records PKV_DEV_TIMEOUT,
// drains its MMAs and frees its TMEM before it returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "pkv_score_mod.cuh"

namespace pkv {
namespace {

constexpr int kTileKeys = kTreeTileKeys;
constexpr int kSubPerTile = kTileKeys / kSubKeys;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kFull = 0xffffffffu;

template <int D, int W>
struct Cfg {
  static constexpr int kThreads = 128 * (W + 1);
  static constexpr int kWarpProducer = 4 * W, kWarpIssue = 4 * W + 1;  // issuers: kWarpIssue + w
  static constexpr int kLaunchRegs = W == 1 ? 128 : 168, kSoftmaxRegs = W == 1 ? 192 : 208, kOtherRegs = W == 1 ? 64 : 88;
  static_assert(W * kSoftmaxRegs + kOtherRegs == (W + 1) * kLaunchRegs, "register shares must add up to the launch's");
  // A ring slot holds half a tile of K or V, or a whole one where the ring is large enough for some of those.
  static constexpr int kSlotKeys = D == 128 && W == 1 ? 64 : 128;
  static constexpr int kSlotsPerTile = kTileKeys / kSlotKeys;
  static constexpr int kSlotBytes = kSlotKeys * D * 2;
  static constexpr int kSlots = D == 64 ? 6 * W : 5;
  static constexpr int kSubBytes = kSubKeys * D * 2;    // one 16-key sub-tile, one box
  static constexpr int kSubsPerSlot = kSlotKeys / kSubKeys;
  static constexpr int kGroupStep = D == 128 ? 2048 : 1024;  // from 8 keys to the next 8
  static constexpr int kHalfStep = 1024;                     // from one 64-column half of them to the other (D = 128)
  static constexpr int kQHalf = 128 * 128;                   // 64 columns of a query tile
  static constexpr int kQBytes = (D / 64) * kQHalf;
  static constexpr int kRingOffset = W * kQBytes;
  static constexpr int kBarOffset = kRingOffset + kSlots * kSlotBytes;
  static constexpr int kTmemCols = W * 256, kOCol = 128;  // tile w: S and P from 256 w on, O 128 columns behind
  // barriers
  static constexpr int kQFull = 0;
  static constexpr int kSlotFull = 1, kSlotEmpty = kSlotFull + kSlots;  // + slot
  static constexpr int kSFull = kSlotEmpty + kSlots, kPReady = kSFull + W, kPVDone = kPReady + W, kDrain = kPVDone + W;  // + w
  static constexpr int kNumBars = kDrain + W;
  static_assert(kNumBars * 8 + 8 <= 512, "barriers, TMEM address and abort flag fit their 512 bytes");
  static constexpr int kSmem = kBarOffset + 512;
  static_assert((W == 1 ? 2 * (kSmem + 1024) : kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Wait that also gives up as soon as another role of this CTA has aborted.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 15u) == 0) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > 1000000000ull) {
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

// Position in the ring of slots.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x % a.num_kv_heads;  // the longest items of all heads first
  grid_dependency_wait();  // q, metadata, masks and this step's keys come from earlier work
  launch_dependents();
  const int4 it = reinterpret_cast<const int4 *>(items)[blockIdx.x / a.num_kv_heads];
  const int seg = it.x, ntiles = it.y, tile0 = it.z & 0xFFFFFF, qt0 = static_cast<int>(static_cast<uint32_t>(it.z) >> 24);
  const int pbase = it.w;
  const int G = a.group, P = rows_per_tile;

  bool bad = seg < 0 || seg >= a.num_seqs || ntiles < 1;
  int row0 = 0, n = 0, L = 0, slot = 0;
  if (!bad) {
    row0 = a.cu_seqlens_q[seg];
    n = a.cu_seqlens_q[seg + 1] - row0;
    slot = a.seq_slot[seg];
    bad = slot < 0 || slot >= a.max_slots;
  }
  if (!bad) {
    L = a.context_lens[slot];
    bad = n < 1 || n > L || n > PKV_TREE_MAX_ROWS || n > 32 * a.mask_words ||
          static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size || qt0 * P >= n ||
          static_cast<int64_t>(tile0) * kTileKeys >= L ||
          static_cast<int64_t>(tile0) + ntiles > (static_cast<int64_t>(L) + kTileKeys - 1) / kTileKeys || row0 < 0 ||
          static_cast<int64_t>(row0) + n > a.total_q || (pbase >= 0 && pbase > a.num_partials - n);
  }
  if (bad || (smem_addr(smem) & 1023) != 0) {  // (the swizzled tiles need their alignment)
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    return;
  }
  const int base = tile0 * kTileKeys;
  const int kv_end = static_cast<int>(min(static_cast<int64_t>(L), static_cast<int64_t>(base) + ntiles * kTileKeys));
  const int active = W == 2 && (qt0 + 1) * P < n ? 2 : 1;  // query tiles with rows

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bar + i, i >= C::kPReady && i < C::kPReady + W ? 4 : i >= C::kSlotEmpty && i < C::kSFull ? active : 1);
    fence_barrier_init();
    *abort_flag = 0;
  }
  // Rows of the Q tiles beyond G * P whole groups stay zero.
  {
    const int qrows = G * P, chunks = (128 - qrows) * 8;
    for (int i = threadIdx.x; i < chunks * (D / 64) * W; i += blockDim.x) {
      const int h = i / chunks, rem = i % chunks;
      *reinterpret_cast<uint4 *>(smem + h * C::kQHalf + (qrows + rem / 8) * 128 + (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == C::kWarpIssue) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 4 * W) {
    setmaxnreg_dec<C::kOtherRegs>();
    if (warp == C::kWarpProducer) {
      // ---------------------------------------------------------- producer
      // Pool rows of the 16-key sub-tiles, four tiles per warp-wide load (lane l: sub-tile l % 8 of tile t0 + l / 8),
      // raw block IDs one group ahead; an ID outside the pool is reported and reads block 0's rows.
      const int32_t *bt_row = a.block_tables + static_cast<int64_t>(slot) * a.max_blocks_per_slot;
      auto key_of = [&](int t0) { return base + (t0 + (lane >> 3)) * kTileKeys + (lane & 7) * kSubKeys; };
      auto inside = [&](int t0) { return t0 + (lane >> 3) < ntiles && key_of(t0) < kv_end; };
      auto group_ids = [&](int t0) -> int { return inside(t0) ? __ldg(bt_row + key_of(t0) / a.block_size) : 0; };
      auto group_rows = [&](int t0, int blk) -> int {
        if (!inside(t0)) return 0;
        if (blk < 0 || blk >= a.num_blocks) {
          if (a.status) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
          blk = 0;
        }
        return (blk * a.num_kv_heads + g) * a.block_size + key_of(t0) % a.block_size;
      };
      int rows_cur = group_rows(0, group_ids(0)), ids_next = group_ids(4);
      if (lane == 0) {
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
        mbar_arrive_expect_tx(bar + C::kQFull, active * (D / 64) * G * P * 128);
        for (int w = 0; w < active; ++w)
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(smem + w * C::kQBytes + h * C::kQHalf, &tmap_q, h * 64, g * G, row0 + (qt0 + w) * P, bar + C::kQFull);
      }
      const uint64_t policy = l2_evict_first_policy();
      const int bs_shift = 31 - __clz(a.block_size);  // block sizes are powers of two
      Ring<C::kSlots> at;
      int used = 0;  // slots filled so far
      bool ok = true;
      for (int j = 0; ok && j < ntiles; ++j) {
        if (j > 0 && (j & 3) == 0) {
          rows_cur = group_rows(j, ids_next);
          ids_next = group_ids(j + 4);
        }
        const int vs = min(kSubPerTile, (kv_end - base - j * kTileKeys + kSubKeys - 1) / kSubKeys);  // sub-tiles with a key
        for (int p = 0; ok && p < 2 * C::kSlotsPerTile; ++p) {  // K's slots, then V's
          const bool is_k = p < C::kSlotsPerTile;
          const int sub0 = (is_k ? p : p - C::kSlotsPerTile) * C::kSubsPerSlot;
          const int count = max(0, min(C::kSubsPerSlot, vs - sub0));
          if (used >= C::kSlots) ok = warp_wait_or_abort(bar + C::kSlotEmpty + at.slot, at.phase ^ 1, abort_flag);
          if (!ok) break;
          const int row = __shfl_sync(kFull, rows_cur, (j & 3) * 8 + ((sub0 + lane) & 7));
          uint64_t *full = bar + C::kSlotFull + at.slot;
          if (lane == 0) mbar_arrive_expect_tx(full, count * C::kSubBytes);
          __syncwarp();
          if (lane < count) {
            uint8_t *dst = smem + C::kRingOffset + at.slot * C::kSlotBytes + lane * C::kSubBytes;
            const CUtensorMap *map = is_k ? &tmap_k : &tmap_v;
            if constexpr (D == 128)
              tma_load_5d_hint(dst, map, 0, 0, 0, (row & (a.block_size - 1)) >> 3, row >> bs_shift, full, policy);
            else
              tma_load_2d_hint(dst, map, 0, row, full, policy);
          }
          at.next();
          ++used;
        }
      }
    } else if (warp - C::kWarpIssue < active && warp >= C::kWarpIssue) {
      // ---------------------------------------------------------- issuers
      if (lane == 0) {
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, C::kSlotKeys, 0, 0);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
        const int w = warp - C::kWarpIssue;
        const uint32_t q_base = smem_addr(smem + w * C::kQBytes), ring = smem_addr(smem + C::kRingOffset);
        const uint32_t s_col = tmem + w * 256, o_col = s_col + C::kOCol;
        Ring<C::kSlots> at;
        bool ok = wait_or_abort(bar + C::kQFull, 0, abort_flag);
        for (int j = 0; ok && j < ntiles; ++j) {
          // S's columns hold P_{j-1} until its product is done
          if (j > 0 && !(ok = wait_or_abort(bar + C::kPVDone + w, (j - 1) & 1, abort_flag))) break;
          for (int p = 0; ok && p < C::kSlotsPerTile; ++p) {
            if (!(ok = wait_or_abort(bar + C::kSlotFull + at.slot, at.phase, abort_flag))) break;
            tc_fence_after();
            const uint32_t k_base = ring + at.slot * C::kSlotBytes;
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_ss(s_col + p * C::kSlotKeys,
                        smem_desc_sw128(q_base + (kk >> 2) * C::kQHalf + (kk & 3) * 32, 16, 1024),
                        smem_desc_sw128(k_base + (kk >> 2) * C::kHalfStep + (kk & 3) * 32, 16, C::kGroupStep), idesc_qk,
                        kk > 0 ? 1u : 0u);
            tc_commit(bar + C::kSlotEmpty + at.slot);
            at.next();
          }
          if (!ok) break;
          tc_commit(bar + C::kSFull + w);
          if (!(ok = wait_or_abort(bar + C::kPReady + w, j & 1, abort_flag))) break;
          const int ksteps = (min(kTileKeys, kv_end - base - j * kTileKeys) + kSubKeys - 1) / kSubKeys;
          for (int p = 0; p < C::kSlotsPerTile; ++p) {
            if (!(ok = wait_or_abort(bar + C::kSlotFull + at.slot, at.phase, abort_flag))) break;
            tc_fence_after();
            const uint32_t v_base = ring + at.slot * C::kSlotBytes;
            for (int ks = p * C::kSubsPerSlot; ks < min(ksteps, (p + 1) * C::kSubsPerSlot); ++ks)
              tc_mma_ts(o_col, s_col + ks * 8,
                        smem_desc_sw128(v_base + (ks - p * C::kSubsPerSlot) * C::kSubBytes, C::kHalfStep, C::kGroupStep),
                        idesc_pv, (j > 0 || ks > 0) ? 1u : 0u);
            tc_commit(bar + C::kSlotEmpty + at.slot);
            at.next();
          }
          tc_commit(bar + C::kPVDone + w);
        }
        tc_commit(bar + C::kDrain + w);
        if (!wait_or_abort(bar + C::kDrain + w, 0, abort_flag) && a.status) atomicOr(a.status, PKV_DEV_TIMEOUT);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<C::kSoftmaxRegs>();
    const int w = W == 1 ? 0 : warp >> 2, quarter = warp & 3;
    if (w < active) {
      const int mrow = quarter * 32 + lane;
      const uint32_t s_col = tmem + w * 256 + (static_cast<uint32_t>(quarter * 32) << 16), o_col = s_col + C::kOCol;
      const int i = (qt0 + w) * P + mrow / G, h = g * G + mrow % G;  // the row's node and q head
      const bool stored = mrow < G * P && i < n;
      const uint32_t *mask = a.masks + (static_cast<int64_t>(row0) + (stored ? i : 0)) * a.mask_words;
      const TileScores<kModNone> ts(a, 0, stored);
      float m_used = -INFINITY;  // log2 units
      float l_sum = 0.f, l_odd = 0.f;
      bool ok = true;
      for (int j = 0; j < ntiles; ++j) {
        const int kt0 = base + j * kTileKeys;
        if (!(ok = warp_wait_or_abort(bar + C::kSFull + w, j & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t sv[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + c * 32, sv[c]);
        tmem_wait_ld();
        if (kt0 + kTileKeys > L - n) {  // the tile reaches the segment's own keys (or the end)
          const int r0 = kt0 - (L - n);  // the tile's first key as a node, negative in the history
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int b = r0 + 32 * c;
            const uint32_t seen = b <= -32 ? ~0u
                                           : __funnelshift_r(mask_word(mask, a.mask_words, n, b >> 5),
                                                             mask_word(mask, a.mask_words, n, (b >> 5) + 1), b & 31);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(seen & (1u << x))) sv[c][x] = 0xff800000u;
          }
        }
        const float m_new = fmaxf(m_used, tile_max(sv) * ts.sl2);
        // before a row's first visible key there is nothing to rescale
        const bool fresh = m_used == -INFINITY;
        const bool need = !fresh && m_new > m_used + kRescaleThreshold;
        if (fresh) m_used = m_new;
        if (__any_sync(kFull, need)) {  // S_j exists, so O holds the products up to tile j - 1
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
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
          ts.template weigh<true>(pk, sv, c, nm, 0.f, l_sum, l_odd);
          tmem_st16(s_col + c * 16, pk);
        }
        // Zero the V rows past the context inside the final 16-key step: a block may hold stale or NaN rows there,
        // and 0 * NaN would reach O. (Both tiles' warps write the same zeros, each before its own product.)
        const int valid = kv_end - kt0, tail = valid < kTileKeys ? (kSubKeys - valid % kSubKeys) % kSubKeys : 0;
        if (tail) {
          // V's slot: behind the slots of the tiles before and of this tile's K
          const int s = (2 * j + 1) * C::kSlotsPerTile + valid / C::kSlotKeys;
          if (!(ok = warp_wait_or_abort(bar + C::kSlotFull + s % C::kSlots, (s / C::kSlots) & 1, abort_flag))) break;
          uint8_t *v = smem + C::kRingOffset + (s % C::kSlots) * C::kSlotBytes;
          for (int x = threadIdx.x & 127; x < tail * (D / 8); x += 128) {
            const int r = valid % C::kSlotKeys + x / (D / 8), chunk = x % (D / 8);
            *reinterpret_cast<uint4 *>(v + (r >> 3) * C::kGroupStep + (chunk >> 3) * C::kHalfStep + (r & 7) * 128 +
                                       (chunk & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + C::kPReady + w);
      }
      if (ok && warp_wait_or_abort(bar + C::kPVDone + w, (ntiles - 1) & 1, abort_flag)) {
        tc_fence_after();
        const float l = l_sum + l_odd;
        const bool unseen = m_used == -INFINITY;  // no key of the span: zeros, whatever O holds
        if (pbase < 0) {
          const float inv = unseen ? 0.f : 1.f / l;
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                 (static_cast<int64_t>(row0 + i) * a.num_q_heads + h) * D);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_col + c * 32, ov);
            tmem_wait_ld();
            if (stored) {
              uint32_t pk[16];
#pragma unroll
              for (int x = 0; x < 16; ++x)
                pk[x] = unseen ? 0u
                               : pack_bf16x2(__uint_as_float(ov[2 * x]) * inv, __uint_as_float(ov[2 * x + 1]) * inv);
#pragma unroll
              for (int v = 0; v < 4; ++v) dst[c * 4 + v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
            }
          }
        } else {
          const int64_t e = (static_cast<int64_t>(pbase) + (stored ? i : 0)) * a.num_q_heads + h;
          uint4 *dst = reinterpret_cast<uint4 *>(a.partial_acc + e * D);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_col + c * 32, ov);
            tmem_wait_ld();
            if (stored)
#pragma unroll
              for (int v = 0; v < 8; ++v)
                dst[c * 8 + v] = unseen ? make_uint4(0, 0, 0, 0)
                                        : make_uint4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
          }
          if (stored) {
            // a row that sees nothing at all: sums of 0 over a denominator that is not 0 merge to zeros
            bool none = unseen && L == n;
            for (int k = 0; none && k < a.mask_words; ++k) none = mask_word(mask, a.mask_words, n, k) == 0;
            reinterpret_cast<float2 *>(a.partial_ml)[e] = none ? make_float2(0.f, 1.f) : make_float2(m_used, l);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0 && a.status) atomicOr(a.status, PKV_DEV_TIMEOUT);
  if (warp == C::kWarpIssue) {
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
