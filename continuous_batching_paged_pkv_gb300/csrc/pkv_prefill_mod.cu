// Prompt-chunk attention with modified scores for head_dim 64 (tcgen05, two
// CTAs per SM).
//
// One CTA takes one 128-row query tile of one (segment, kv head): rows are P
// positions x G grouped q heads (row m = position m / G, head m % G), keys come
// in tiles of 128 from the 16-key sub-tile of the first key that some row sees
// to the last such key. Per tile the tensor core has half the work that it has
// at head_dim 128 (twelve MMAs), the softmax as much as there, so the softmax
// sets the pace: its one warpgroup is a chain of TMEM load, maximum, exponents
// and TMEM store that leaves its pipes idle in between. Hence two CTAs per SM,
// each within half of TMEM, shared memory and registers: one's softmax runs while
// the other's scores or products are computed, and a CTA's start (metadata, Q, the
// first keys) hides behind the other's tiles.
//
//   warps 0-3  softmax: thread = TMEM lane = row; takes S_j into registers
//              (and gives S back at once), capped, biased, masked; P_j as bf16,
//              the row sum in fp32 registers, O rescaled when the running max
//              grew by more than 2^8; normalisation and store.
//   warp 4     TMA producer of K (Q first), three stages of 128 keys
//   warp 5     QK issuer: S_j = Q K_j^T (SS, M 128, N 128)
//   warp 6     PV issuer: O += P_j V_j (TS, N 64)
//   warp 7     TMA producer of V, two stages
//
// TMEM columns: [0, 128) S, [128, 192) P (bf16 pairs), [192, 256) O. P has
// columns of its own, so S_{j+1} is computed while P_j is still to be written.
// The kernel launches with 128 registers per thread; the softmax warpgroup raises
// its share to 192 and the other lowers its own to 64. A distance bias without a
// cap comes with the scores (one more MMA per tile). Every mbarrier wait is bounded; on
// expiry the CTA records PKV_DEV_TIMEOUT, drains its MMAs and frees its TMEM before
// it returns.
//
// What it takes is two CTAs' chains of some 2800 cycles per tile (of which the
// weights 960, their MMAs' issue 110 each) and, in short loops, a CTA's 6000 cycles
// before its first tile and after its last. 8192 rows, 16 heads of 64, one stream
// as the context: causal 207 us (665 TFLOP/s of what is seen), biased 217; windows of
// 512 keys 49 us, of 128 keys 33 us; documents of 16 to 2048 tokens 57 us, biased
// 63 us. The kernel for plain scores, with this one's masks and biases in its softmax
// threads, took 1059 us (causal), 89 us (128 keys) and 228 us (documents, biased).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "pkv_score_mod.cuh"

namespace pkv {
namespace {

constexpr int D = 64;
constexpr int kKeysPerTile = 128;
constexpr int kSubPerTile = kKeysPerTile / kSubKeys;
constexpr int kTmemCols = 256, kPCol = 128, kOCol = 192;
constexpr int kThreads = 256;
constexpr int kWarpK = 4, kWarpQK = 5, kWarpV = 7;  // the PV issuer is the fourth, warp 6
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 192, kOtherRegs = 64;
static_assert(kSoftmaxRegs + kOtherRegs == 2 * kLaunchRegs, "register shares must add up to the launch's");
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kKStages = 3, kVStages = 2;
constexpr int kTileBytes = kKeysPerTile * D * 2;  // Q, K or V tile: 128 rows x 128 B
constexpr int kBoxBytes = kSubKeys * D * 2;
constexpr int kBarOffset = (1 + kKStages + kVStages) * kTileBytes;
constexpr int kRampOffset = kBarOffset + 256;  // after the barriers and flags: the bias step's operands
template <int MODE>
constexpr int kSmem = kRampOffset + (ramp_mode(MODE) ? 2 * kRampBytes : 0) + 1024;  // + alignment slack
static_assert(2 * (kSmem<kModBias> + 1024) <= 228 * 1024, "two CTAs per SM");

enum Bar : int {
  kQFull = 0,
  kKFull = 1,                     // +stage
  kKEmpty = kKFull + kKStages,    // +stage
  kVFull = kKEmpty + kKStages,    // +stage
  kVEmpty = kVFull + kVStages,    // +stage
  kSFull = kVEmpty + kVStages,    // S_j computed
  kSFree,                         // S_j in registers: one arrival per softmax warp
  kPReady,                        // P_j written: one arrival per softmax warp
  kPVDone,                        // P_j V_j done: P free, O complete up to tile j
  kDrain,
  kDrainPV,
  kNumBars
};
static_assert(kNumBars * 8 + 16 <= 256, "barriers, TMEM address, abort flag and key range fit their 256 bytes");

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
  return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

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

template <int MODE>
__global__ void __maxnreg__(kLaunchRegs) prefill_mod_kernel(const __grid_constant__ CUtensorMap tmap_q,
                                                            const __grid_constant__ CUtensorMap tmap_k,
                                                            const __grid_constant__ CUtensorMap tmap_v,
                                                            const StepArgs a, const int32_t *__restrict__ items,
                                                            int rows_per_tile) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  uint8_t *sQ = smem, *sK = smem + kTileBytes, *sV = sK + kKStages * kTileBytes;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + kBarOffset);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint8_t *sRamp = smem + kRampOffset;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.y;
  // As in the head_dim 128 kernel: the work item, step metadata, q and the cached
  // history are final when this grid starts; the producers wait for the kernel
  // before it at the first tile that holds rows of this step.
  launch_dependents();
  const int4 it = reinterpret_cast<const int4 *>(items)[blockIdx.x];
  const int seg = it.x, slot = it.y, tile = it.z;
  const int G = a.group, P = rows_per_tile;

  bool bad = seg < 0 || seg >= a.num_seqs || slot < 0 || slot >= a.max_slots || tile < 0;
  int row0 = 0, n = 0, L = 0;
  if (!bad) {
    row0 = a.cu_seqlens_q[seg];
    n = a.cu_seqlens_q[seg + 1] - row0;
    L = a.context_lens[slot];
    bad = a.seq_slot[seg] != slot || n < 2 || n > L ||
          static_cast<int64_t>(L) > static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size ||
          static_cast<int64_t>(tile) * P >= n || row0 < 0 || static_cast<int64_t>(row0) + n > a.total_q;
  }
  if (bad) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    grid_dependency_wait();  // as below: this grid ends after the kernel before it
    return;
  }
  const int pos0 = tile * P;          // first query row of the tile within the segment
  const int rows = min(P, n - pos0);  // query positions present in this tile
  int *u = const_cast<int *>(abort_flag) + 1;
  rows_see(a, static_cast<int64_t>(row0) + pos0, L - n + pos0, rows, L, u);
  // keys [kv_begin, kv_end) are visible to some row; tiles start at their first 16-key sub-tile
  const int kv_begin = min(u[0], u[1]), kv_end = u[1];
  const int base = kv_begin & ~(kSubKeys - 1);
  const int ntiles = (kv_end - base + kKeysPerTile - 1) / kKeysPerTile;  // 0: no row of the tile sees a key
  if (ntiles == 0) grid_dependency_wait();  // else the producers do, before a row is stored
  // With a bias the nearest keys come first (as in the head_dim 128 kernel), but the cached ones before this step's.
  constexpr bool kDown = (MODE & kModBias) != 0;
  const int old = kDown ? min(max(L - n - base, 0) / kKeysPerTile, ntiles) : 0;
  auto tile_at = [&](int j) { return !kDown ? j : j < old ? old - 1 - j : ntiles - 1 - (j - old); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar + i, i == kSFree || i == kPReady ? 4 : 1);
    fence_barrier_init();
    *abort_flag = 0;
  }
  // Rows of the Q tile beyond G * P whole groups stay zero.
  {
    const int qrows = G * P;
    for (int i = threadIdx.x; i < (128 - qrows) * 8; i += blockDim.x)
      *reinterpret_cast<uint4 *>(sQ + (qrows + i / 8) * 128 + (i % 8) * 16) = make_uint4(0, 0, 0, 0);
    if constexpr (ramp_mode(MODE)) {
      const int r = threadIdx.x & 127;
      if (threadIdx.x < 128)
        store_ramp_slope(sRamp, r, r < qrows ? ramp_slope(a, g * G + r % G) : 0.f);
      else
        store_ramp_key(sRamp + kRampBytes, r, r);
    }
    fence_proxy_async_smem();
  }
  if (warp == kWarpQK) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 4) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == kWarpK || warp == kWarpV) {
      // ---------------------------------------------------------- producers
      // Pool rows of the 16-key sub-tiles, four tiles per warp-wide load (lane l:
      // sub-tile l % 8 of the tile at step t0 + l / 8), raw block IDs one group
      // ahead; an ID outside the pool is reported and reads block 0's rows.
      const bool is_k = warp == kWarpK;
      const CUtensorMap *map = is_k ? &tmap_k : &tmap_v;
      uint8_t *ring = is_k ? sK : sV;
      uint64_t *full = bar + (is_k ? kKFull : kVFull), *empty = bar + (is_k ? kKEmpty : kVEmpty);
      const int stages = is_k ? kKStages : kVStages;
      const int32_t *bt_row = a.block_tables + static_cast<int64_t>(slot) * a.max_blocks_per_slot;
      auto key_of = [&](int t0) { return base + tile_at(t0 + (lane >> 3)) * kKeysPerTile + (lane & 7) * kSubKeys; };
      auto group_ids = [&](int t0) -> int {
        const int key = key_of(t0);
        return key >= base && key < kv_end ? __ldcg(bt_row + key / a.block_size) : 0;
      };
      auto group_rows = [&](int t0, int blk) -> int {
        const int key = key_of(t0);
        if (key < base || key >= kv_end) return 0;
        if (blk < 0 || blk >= a.num_blocks) {
          if (a.status && is_k) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
          return 0;
        }
        return (blk * a.num_kv_heads + g) * a.block_size + key % a.block_size;
      };
      // A scratch pool and its block table come whole from the kernel before, which may still be running:
      // wait before the table is read, and read it through L2 (not as data that never changes).
      bool waited = false;
      if (a.kv_from_previous) {
        grid_dependency_wait();
        waited = true;
      }
      int rows_cur = group_rows(0, group_ids(0)), ids_next = group_ids(4);
      if (lane == 0) {
        prefetch_tensormap(map);
        if (is_k) {
          mbar_arrive_expect_tx(bar + kQFull, G * P * 128);
          tma_load_3d(sQ, &tmap_q, 0, g * G, row0 + pos0, bar + kQFull);
        }
      }
      int s = 0;
      uint32_t phase = 0;  // (j / stages) & 1
      for (int j = 0; j < ntiles; ++j) {
        if (j >= stages && !warp_wait_or_abort(empty + s, phase ^ 1, abort_flag)) break;
        if (j > 0 && (j & 3) == 0) {
          rows_cur = group_rows(j, ids_next);
          ids_next = group_ids(j + 4);
        }
        const int kt0 = base + tile_at(j) * kKeysPerTile;
        const int vs = min(kSubPerTile, (kv_end - kt0 + kSubKeys - 1) / kSubKeys);  // sub-tiles with a visible key
        const int row = __shfl_sync(kFull, rows_cur, (j & 3) * 8 + (lane & 7));
        // At the first tile with rows of this step, and with no such tile at the last one: the kernel before
        // may write the same output, and the next kernel waits for this grid only.
        if (!waited && (kt0 + kKeysPerTile > L - n || j == ntiles - 1)) {
          grid_dependency_wait();
          waited = true;
        }
        if (lane == 0) mbar_arrive_expect_tx(full + s, vs * kBoxBytes);
        __syncwarp();
        if (lane < vs) tma_load_2d(ring + s * kTileBytes + lane * kBoxBytes, map, 0, row, full + s);
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
    } else if (warp == kWarpQK) {
      // ---------------------------------------------------------- QK issuer
      if (lane == 0) {
        constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kKeysPerTile, 0, 0);
        const uint32_t q_base = smem_addr(sQ);
        bool ok = wait_or_abort(bar + kQFull, 0, abort_flag);
        tc_fence_after();
        for (int j = 0; ok && j < ntiles; ++j) {
          if (j > 0 && !(ok = wait_or_abort(bar + kSFree, (j - 1) & 1, abort_flag))) break;
          if (!(ok = wait_or_abort(bar + kKFull + j % kKStages, (j / kKStages) & 1, abort_flag))) break;
          tc_fence_after();
          const uint32_t k_base = smem_addr(sK + (j % kKStages) * kTileBytes);
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma_ss(tmem, smem_desc_sw128(q_base + kk * 32, 16, 1024), smem_desc_sw128(k_base + kk * 32, 16, 1024),
                      idesc_qk, kk > 0 ? 1u : 0u);
          if constexpr (ramp_mode(MODE)) tc_mma_ss(tmem, ramp_desc(sRamp), ramp_desc(sRamp + kRampBytes), idesc_qk, 1u);
          tc_commit(bar + kSFull);
          tc_commit(bar + kKEmpty + j % kKStages);
        }
        tc_commit(bar + kDrain);
        if (!wait_or_abort(bar + kDrain, 0, abort_flag) && a.status) atomicOr(a.status, PKV_DEV_TIMEOUT);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- PV issuer
      if (lane == 0) {
        constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
        for (int j = 0; j < ntiles; ++j) {
          if (!wait_or_abort(bar + kPReady, j & 1, abort_flag)) break;
          if (!wait_or_abort(bar + kVFull + j % kVStages, (j / kVStages) & 1, abort_flag)) break;
          tc_fence_after();
          const int valid = min(kKeysPerTile, kv_end - base - tile_at(j) * kKeysPerTile);
          const int ksteps = (valid + kSubKeys - 1) / kSubKeys;
          const uint32_t v_base = smem_addr(sV + (j % kVStages) * kTileBytes);
          for (int ks = 0; ks < ksteps; ++ks)
            tc_mma_ts(tmem + kOCol, tmem + kPCol + ks * 8, smem_desc_sw128(v_base + ks * kBoxBytes, kTileBytes, 1024),
                      idesc_pv, (j > 0 || ks > 0) ? 1u : 0u);
          tc_commit(bar + kPVDone);
          tc_commit(bar + kVEmpty + j % kVStages);
        }
        tc_commit(bar + kDrainPV);
        if (!wait_or_abort(bar + kDrainPV, 0, abort_flag) && a.status) atomicOr(a.status, PKV_DEV_TIMEOUT);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kSoftmaxRegs>();
    const int mrow = warp * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const int pos = mrow / G, hh = mrow % G;
    const int p_row = L - n + pos0 + pos;
    const bool stored = mrow < G * P && pos < rows;
    int lo = 0, hi = INT32_MAX;  // visible keys of this row; rows that are not stored mask nothing
    if (stored) row_sees(a, static_cast<int64_t>(row0) + pos0 + pos, p_row, L, lo, hi);
    TileScores<MODE> ts(a, g * G + hh, stored);
    float m_used = -INFINITY;            // log2 units
    float l_sum = 0.f, l_odd = 0.f;      // row sum, as even and odd columns (packed adds)
    bool ok = true;
    int tile_next = tile_at(0);
    for (int j = 0; j < ntiles; ++j) {
      const int tile_j = tile_next, kt0 = base + tile_j * kKeysPerTile;
      tile_next = kDown ? (j + 1 == old ? ntiles : tile_j) - 1 : j + 1;  // tile_at(j + 1) at less
      if (!(ok = warp_wait_or_abort(bar + kSFull, j & 1, abort_flag))) break;
      tc_fence_after();
      // Zero the V rows past the last visible key inside the final 16-key step,
      // and before the first visible one inside the first: a block may hold stale
      // or NaN rows there, and 0 * NaN would reach O.
      auto clear_values = [&]() -> bool {
        const int valid = kv_end - kt0;
        const int head = tile_j == 0 ? kv_begin - base : 0;
        const int tail = tile_j == ntiles - 1 ? (kSubKeys - valid % kSubKeys) % kSubKeys : 0;
        if (head + tail == 0) return true;
        if (!warp_wait_or_abort(bar + kVFull + j % kVStages, (j / kVStages) & 1, abort_flag)) return false;
        uint8_t *v = sV + (j % kVStages) * kTileBytes;
        for (int i = threadIdx.x; i < (head + tail) * 8; i += 128) {
          const int r = i / 8 < head ? i / 8 : valid + i / 8 - head;
          *reinterpret_cast<uint4 *>(v + r * 128 + (i % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        return true;
      };
      // No row of this warp sees a key of the tile (another warp's rows do): zero weights.
      if (__all_sync(kFull, !stored || lo > kt0 + kKeysPerTile - 1 || hi <= kt0)) {
        if (lane == 0) mbar_arrive(bar + kSFree);
        if (j > 0 && !(ok = warp_wait_or_abort(bar + kPVDone, (j - 1) & 1, abort_flag))) break;
        tc_fence_after();
        const uint32_t zero[16] = {};
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(tmem + lane_base + kPCol + c * 16, zero);
        if (!(ok = clear_values())) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kPReady);
        continue;
      }
      uint32_t sv[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tmem + lane_base + c * 32, sv[c]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + kSFree);
      typename TileScores<MODE>::Tile found;
      const float m_new = fmaxf(m_used, ts.top(sv, p_row - kt0, lo - kt0, hi - 1 - kt0, found));
      // before a row's first visible key there is nothing to rescale
      const bool fresh = m_used == -INFINITY;
      const bool need = !fresh && m_new > m_used + kRescaleThreshold;
      if (fresh) m_used = m_new;
      // P's columns are free and O holds tile j - 1's products
      if (j > 0 && !(ok = warp_wait_or_abort(bar + kPVDone, (j - 1) & 1, abort_flag))) break;
      tc_fence_after();
      if (__any_sync(kFull, need)) {
        const float corr = need ? ex2_approx(m_used - m_new) : 1.f;
        if (need) m_used = m_new;
        l_sum *= corr;
        l_odd *= corr;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t ov[16];
          tmem_ld16(tmem + lane_base + kOCol + c * 16, ov);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * corr);
          tmem_st16(tmem + lane_base + kOCol + c * 16, ov);
        }
      }
      const float nm = m_used == -INFINITY ? 0.f : -m_used;
      auto weigh = [&](auto is_raw) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
          ts.template weigh<decltype(is_raw)::value>(pk, sv, c, nm, found.near, l_sum, l_odd);
          tmem_st16(tmem + lane_base + kPCol + c * 16, pk);
        }
      };
      if (!TileScores<MODE>::kCap || found.raw)
        weigh(std::true_type{});
      else
        weigh(std::false_type{});
      if (!(ok = clear_values())) break;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + kPReady);
    }
    if (ok && (ntiles == 0 || warp_wait_or_abort(bar + kPVDone, (ntiles - 1) & 1, abort_flag))) {
      tc_fence_after();
      const float inv = 1.f / (l_sum + l_odd);
      const bool none = lo >= hi;  // a row that sees nothing gives zeros, whatever O holds
      __nv_bfloat16 *orow = reinterpret_cast<__nv_bfloat16 *>(a.out) +
                            (static_cast<size_t>(row0 + pos0 + pos) * a.num_q_heads + g * G + hh) * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(tmem + lane_base + kOCol + c * 32, ov);
        tmem_wait_ld();
        if (stored) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = none ? 0u : pack_bf16x2(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv);
          uint4 *dst = reinterpret_cast<uint4 *>(orow + c * 32);
#pragma unroll
          for (int v = 0; v < 4; ++v) dst[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0 && a.status) atomicOr(a.status, PKV_DEV_TIMEOUT);
  if (warp == kWarpQK) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int MODE>
cudaError_t launch_t(const StepArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     int32_t rows_per_tile, int32_t num_items, const int32_t *items, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};  // one bit per device
  if (const cudaError_t e = allow_smem_once(prefill_mod_kernel<MODE>, kSmem<MODE>, configured); e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(num_items), static_cast<unsigned>(a.num_kv_heads));
  return launch_pdl(prefill_mod_kernel<MODE>, grid, dim3(kThreads), kSmem<MODE>, stream, tq, tk, tv, a, items,
                    rows_per_tile);
}

}  // namespace

cudaError_t launch_prefill_mod(const StepArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                               int32_t rows_per_tile, int32_t num_items, const int32_t *items, cudaStream_t stream) {
  if (num_items <= 0) return cudaSuccess;
  if (a.head_dim != D) return cudaErrorInvalidValue;  // head_dim 128 runs on SM pairs
  switch (mode_of(a)) {
    case kModMask: return launch_t<kModMask>(a, tq, tk, tv, rows_per_tile, num_items, items, stream);
    case kModMask | kModCap: return launch_t<kModMask | kModCap>(a, tq, tk, tv, rows_per_tile, num_items, items, stream);
    case kModMask | kModBias:
      return launch_t<kModMask | kModBias>(a, tq, tk, tv, rows_per_tile, num_items, items, stream);
    default:
      return launch_t<kModMask | kModCap | kModBias>(a, tq, tk, tv, rows_per_tile, num_items, items, stream);
  }
}

}  // namespace pkv
