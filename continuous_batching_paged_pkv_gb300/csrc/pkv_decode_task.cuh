// Work-item bookkeeping shared by the split-KV decode kernels (bf16 and
// 8-bit pools): one task is (decode segment, key span of PKV_SPLIT_KEYS keys,
// kv head). A warp expands a task (issues the loads of its metadata and block
// IDs), then finalises it (checks the metadata against the work item and
// derives the key range and the pool row of each 16-key sub-tile).
#pragma once

#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "pkv_score_mod.cuh"

namespace pkv {
namespace {

// One task's metadata. Scalars are uniform across the warp; `bid` is per lane:
// the physical block of the task's sub-tile number `lane`.
struct Task {
  int t;  // task index, -1 if none
  int seg, slot, span, pbase, g;
  int row0, row1, L, sslot;
  int nrows;  // rows of the segment (1, or a short run of causal rows)
  int key0, key1, units;
  int bid;  // per lane: block of sub-tile `lane`
  int row;  // per lane: tensor-map row of sub-tile `lane`, -1 if its block ID is outside the pool
  bool raw_ok, finalized, ok;
  bool reads_new;  // the span reaches this step's rows (written by the kernel before in the stream)
  // modified scores only
  int subs;        // 16-key sub-tiles that the work item names (0: the segment sees nothing)
  int begin, end;  // per lane: key_begin / key_end of row `lane` as given (finalize issues the loads)
};

__device__ __forceinline__ int4 load_item(const int32_t *items, int t, int hkv) {
  return __ldg(reinterpret_cast<const int4 *>(items) + t / hkv);
}

// Issue every load the task needs; nothing here waits for a result. MOD:
// modified scores, whose items name the sub-tiles of the span that some row sees.
template <bool MOD = false>
__device__ __forceinline__ void expand(Task &T, int t, int4 raw, const StepArgs &a, int lane) {
  T.t = t;
  T.finalized = false;
  T.ok = false;
  T.reads_new = true;
  T.units = 0;
  T.bid = 0;
  T.row = -1;
  if (t < 0) return;
  T.seg = raw.x;
  T.slot = raw.y;
  T.span = raw.z;
  T.pbase = raw.w;
  T.g = t % a.num_kv_heads;
  if constexpr (MOD) {
    const uint32_t w = static_cast<uint32_t>(raw.z);
    T.span = static_cast<int>(w & 0x7FFFFFu);
    T.key0 = T.span * PKV_SPLIT_KEYS + static_cast<int>((w >> 23) & 15u) * kSubKeys;
    T.subs = static_cast<int>(w >> 27);
  } else {
    T.key0 = T.span * PKV_SPLIT_KEYS;
  }
  T.raw_ok = T.seg >= 0 && T.seg < a.num_seqs && T.slot >= 0 && T.slot < a.max_slots && T.span >= 0;
  if (!T.raw_ok) return;
  T.row0 = __ldg(a.cu_seqlens_q + T.seg);
  T.row1 = __ldg(a.cu_seqlens_q + T.seg + 1);
  T.L = __ldg(a.context_lens + T.slot);
  T.sslot = __ldg(a.seq_slot + T.seg);
  const int64_t key = static_cast<int64_t>(T.key0) + lane * kSubKeys;
  if ((MOD ? lane < T.subs : lane * kSubKeys < PKV_SPLIT_KEYS) &&
      key < static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size)
    T.bid = __ldg(a.block_tables + static_cast<int64_t>(T.slot) * a.max_blocks_per_slot + key / a.block_size);
}

// Check the metadata against the work item and derive the key range.
template <bool MOD = false>
__device__ __forceinline__ void finalize(Task &T, const StepArgs &a, int lane, int max_cols, int max_rows) {
  if (T.finalized) return;
  T.finalized = true;
  if (T.t < 0) return;
  T.nrows = T.row1 - T.row0;
  T.ok = T.raw_ok && T.sslot == T.slot && T.nrows >= 1 && T.nrows <= max_rows && T.nrows * a.group <= max_cols && T.nrows <= T.L &&
         T.L >= 1 &&
         static_cast<int64_t>(T.L) <= static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size &&
         (T.key0 < T.L || (MOD && T.subs == 0)) && T.row0 >= 0 &&
         static_cast<int64_t>(T.row0) + T.nrows <= a.total_q;
  if constexpr (MOD)  // at most a span's sub-tiles, and the partials inside the workspace
    T.ok = T.ok && T.subs <= PKV_SPLIT_KEYS / kSubKeys && (T.pbase < 0 || T.pbase <= a.num_partials - T.nrows);
  if (!T.ok) {
    if (lane == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    return;
  }
  if constexpr (MOD) {
    T.key1 = T.subs == 0 ? T.key0 : T.key0 + min(T.L - T.key0, T.subs * kSubKeys);
    T.begin = lane < T.nrows && a.key_begin ? __ldg(a.key_begin + T.row0 + lane) : 0;
    T.end = lane < T.nrows && a.key_end ? __ldg(a.key_end + T.row0 + lane) : INT32_MAX;
  } else {
    T.key1 = min(T.L, T.key0 + PKV_SPLIT_KEYS);
  }
  T.units = (T.key1 - T.key0 + kSubKeys - 1) / kSubKeys;
  T.reads_new = T.key1 > T.L - T.nrows;
  const bool in_pool = T.bid >= 0 && T.bid < a.num_blocks;
  T.row = in_pool ? (T.bid * a.num_kv_heads + T.g) * a.block_size + (T.key0 + lane * kSubKeys) % a.block_size : -1;
  if (lane < T.units && !in_pool && a.status) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
}

// What the columns of a task see and how their scores change, set up when the
// task becomes current (modified scores). A thread's columns are nt * 8 +
// 2 (lane % 4) + c, each a (row, q head) pair; a single row needs one interval.
template <int NT, bool MULTI>
struct TaskMod {
  static constexpr int N = MULTI ? NT : 1, C = MULTI ? 2 : 1;
  int lo[N][C], hi[N][C];  // visible keys [lo, hi) of the column
  float row[N][C];         // index of the column's row within the segment
  float slope[NT][2];      // distance bias per key, log2 units
  int u_lo, u_hi;          // from the first to past the last key that some row of the segment sees
  int a_lo, a_hi;          // keys that every row of the segment sees
  int pos0;                // position of the segment's first row

  __device__ __forceinline__ void set(const Task &T, const StepArgs &a, int lane) {
    const int n = T.ok ? T.nrows : 0;
    pos0 = T.L - n;
    int lo_l = INT32_MAX, hi_l = 0;
    if (lane < n) {
      visible_keys(a, T.begin, T.end, pos0 + lane, T.L, lo_l, hi_l);
      if (lo_l >= hi_l) lo_l = INT32_MAX, hi_l = 0;
    }
    u_lo = __reduce_min_sync(0xffffffffu, lo_l);
    u_hi = __reduce_max_sync(0xffffffffu, hi_l);
    a_lo = __reduce_max_sync(0xffffffffu, lane < n ? lo_l : 0);
    a_hi = __reduce_min_sync(0xffffffffu, lane < n ? hi_l : INT32_MAX);
    // Of a single span the item must name all the keys that the rows see.
    if (T.ok && T.pbase < 0 && u_lo < u_hi && (u_lo < T.key0 || u_hi > T.key1) && lane == 0 && a.status)
      atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = nt * 8 + (lane & 3) * 2 + c;
        const bool valid = col < n * a.group;
        if (MULTI || (nt == 0 && c == 0)) {
          const int i = MULTI && valid ? col / a.group : 0;
          lo[nt][c] = __shfl_sync(0xffffffffu, lo_l, i);
          hi[nt][c] = __shfl_sync(0xffffffffu, hi_l, i);
          row[nt][c] = static_cast<float>(i);
        }
        slope[nt][c] = valid && a.alibi_slopes
                           ? __ldg(a.alibi_slopes + T.g * a.group + (MULTI ? col % a.group : col)) * 1.4426950408889634f
                           : 0.f;
      }
  }

  // Whether the row of column (nt, c) sees no key.
  __device__ __forceinline__ bool nothing(int nt, int c) const { return hi[MULTI ? nt : 0][MULTI ? c : 0] == 0; }

  // A sub-tile's scores (log2 units) of keys kbase + ka and kbase + ka + 8
  // become logits; keys past the loaded ones (`v` of them) or outside the
  // column's interval become -inf. Most sub-tiles lie inside every row's interval.
  __device__ __forceinline__ void logits(float (&x)[NT][2][2], int kbase, int ka, int v, const Cap &cap, bool bias) const {
    if (cap.on) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) cap.both(x[nt][c][0], x[nt][c][1]);
    }
    if (bias) {
      const float away = static_cast<float>(pos0 - kbase) - static_cast<float>(ka);  // row 0 from key kbase + ka
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float d = MULTI ? away + row[MULTI ? nt : 0][MULTI ? c : 0] : away;
          x[nt][c][0] = fmaf(-slope[nt][c], fabsf(d), x[nt][c][0]);
          x[nt][c][1] = fmaf(-slope[nt][c], fabsf(d - 8.f), x[nt][c][1]);
        }
    }
    if (v < kSubKeys || kbase < a_lo || kbase + kSubKeys > a_hi) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int k = ka + 8 * i, j = kbase + k;
            if (!(k < v && j >= lo[MULTI ? nt : 0][MULTI ? c : 0] && j < hi[MULTI ? nt : 0][MULTI ? c : 0]))
              x[nt][c][i] = -INFINITY;
          }
    }
  }
};

}  // namespace
}  // namespace pkv
