// The rows of an accepted path move to the front of their segment's drafts.
//
// For depth d the row at place L - n + path[d] of the slot goes to place L - n + d.
// A path grows, so path[d] >= d: a copy's target is the source of no later copy,
// and only sources of earlier copies are overwritten. A warp takes one (segment,
// pool array, kv head), reads some rows before it writes any of them (four loads a
// lane: eight bf16 rows of 128), and goes through the path in order; nothing else
// touches these rows. Bound by latency (metadata, path, block table, row): a step
// moves a few rows per slot. Up to 6 of 32 nodes in 256 slots x 8 heads: 3.7 us
// (5.8 with eight loads a lane, whose registers leave half as many warps to an SM).
#include <cuda_runtime.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// Moves rows of `width` T words each; lane % lanes is the word, lane / lanes the row within an instruction.
template <typename T>
__device__ __forceinline__ void move_rows(uint8_t *base, int64_t row_bytes, int count, int lane, int64_t from,
                                          int64_t to) {
  const int words = static_cast<int>(row_bytes / sizeof(T));
  int lanes = 1;
  while (lanes < words && lanes < 32) lanes *= 2;
  const int per = 32 / lanes, sub = lane / lanes;
  constexpr int kRounds = 4;
  for (int w0 = 0; w0 < words; w0 += lanes) {
    const int w = w0 + lane % lanes;
    for (int d0 = 0; d0 < count; d0 += kRounds * per) {
      T v[kRounds];
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int d = d0 + i * per + sub;
        const int64_t src = __shfl_sync(kAll, from, d & 31), dst = __shfl_sync(kAll, to, d & 31);
        if (d < count && w < words && src >= 0 && dst >= 0)
          v[i] = *reinterpret_cast<const T *>(base + src * row_bytes + static_cast<int64_t>(w) * sizeof(T));
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int d = d0 + i * per + sub;
        const int64_t src = __shfl_sync(kAll, from, d & 31), dst = __shfl_sync(kAll, to, d & 31);
        if (d < count && w < words && src >= 0 && dst >= 0)
          *reinterpret_cast<T *>(base + dst * row_bytes + static_cast<int64_t>(w) * sizeof(T)) = v[i];
      }
      __syncwarp();
    }
  }
}

__global__ void __launch_bounds__(128) accept_rows_kernel(const AcceptArgs a) {
  // The next kernel may read the rows that move here as history, before its own wait: it must not start before
  // they are in place, so this one gives no early signal. The metadata and the paths are final when it starts; it
  // waits for the kernel before it ahead of the rows, and before it ends.
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int per_seg = a.num_arrays * a.num_kv_heads;
  const int64_t seg = unit / per_seg;
  if (seg >= a.num_seqs) {
    grid_dependency_wait();
    return;
  }
  const int arr = static_cast<int>(unit % per_seg) / a.num_kv_heads, h = static_cast<int>(unit % per_seg) % a.num_kv_heads;
  const bool reports = unit % per_seg == 0 && lane == 0 && a.status;
  const int row0 = __ldg(a.cu_seqlens_q + seg), n = __ldg(a.cu_seqlens_q + seg + 1) - row0, slot = __ldg(a.seq_slot + seg);
  bool ok = slot >= 0 && slot < a.max_slots && n >= 0 && row0 >= 0 && static_cast<int64_t>(row0) + n <= a.total_q;
  const int L = ok ? __ldg(a.context_lens + slot) : 0;
  ok = ok && n <= L && L <= static_cast<int64_t>(a.max_blocks_per_slot) * a.block_size;
  if (!ok) {
    if (reports) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    grid_dependency_wait();
    return;
  }
  const int32_t *path = a.paths + seg * a.max_path;
  const int32_t *table = a.block_tables + static_cast<int64_t>(slot) * a.max_blocks_per_slot;
  uint8_t *base = arr == 0 ? a.arrays[0] : arr == 1 ? a.arrays[1] : arr == 2 ? a.arrays[2] : a.arrays[3];
  const int64_t row_bytes = arr == 0 ? a.row_bytes[0] : arr == 1 ? a.row_bytes[1] : arr == 2 ? a.row_bytes[2] : a.row_bytes[3];
  // 32 depths at a time: lane l has depth d0 + l
  int before = -1;  // path entry of the depth before
  for (int d0 = 0; d0 < a.max_path; d0 += 32) {
    const int d = d0 + lane;
    const int p = d < a.max_path ? __ldg(path + d) : -1;
    int prev = __shfl_up_sync(kAll, p, 1);
    if (lane == 0) prev = before;
    const bool ends = p < 0, wrong = !ends && (p <= prev || p >= n);
    const uint32_t stop = __ballot_sync(kAll, ends || wrong);
    const int count = stop ? __ffs(stop) - 1 : 32;
    if (stop && lane == count && wrong && unit % per_seg == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_SEGMENT);
    int64_t from = -1, to = -1;
    bool bad = false;
    if (lane < count && p != d) {  // a row that is in its place stays
      const int src = L - n + p, dst = L - n + d;
      const int sb = __ldg(table + src / a.block_size), db = __ldg(table + dst / a.block_size);
      bad = sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks;
      if (!bad) {
        from = (static_cast<int64_t>(sb) * a.num_kv_heads + h) * a.block_size + src % a.block_size;
        to = (static_cast<int64_t>(db) * a.num_kv_heads + h) * a.block_size + dst % a.block_size;
      }
    }
    if (bad && unit % per_seg == 0 && a.status) atomicOr(a.status, PKV_DEV_BAD_BLOCK);
    if (d0 == 0) grid_dependency_wait();
    if (row_bytes % 16 == 0)
      move_rows<uint4>(base, row_bytes, count, lane, from, to);
    else if (row_bytes % 8 == 0)
      move_rows<uint2>(base, row_bytes, count, lane, from, to);
    else
      move_rows<uint32_t>(base, row_bytes, count, lane, from, to);
    if (stop) return;
    before = __shfl_sync(kAll, p, 31);
  }
}

}  // namespace

cudaError_t launch_accept_rows(const AcceptArgs &a, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.num_seqs) * a.num_arrays * a.num_kv_heads;
  return launch_pdl(accept_rows_kernel, dim3(static_cast<unsigned>((units + 3) / 4)), dim3(128), 0, stream, a);
}

}  // namespace pkv

extern "C" pkv_status pkv_accept_rows(const int32_t *cu_seqlens_q, int32_t num_seqs, int64_t total_q,
                                      const int32_t *seq_slot, const int32_t *context_lens, const int32_t *block_tables,
                                      int32_t max_slots, int32_t max_blocks_per_slot, int32_t block_size,
                                      int32_t num_kv_heads, const int32_t *paths, int32_t max_path, void *const *arrays,
                                      const int64_t *row_bytes, int32_t num_arrays, int64_t num_blocks,
                                      uint32_t *device_status, pkv_stream_t stream) {
  if (num_seqs < 0 || total_q < 0 || max_slots <= 0 || max_blocks_per_slot <= 0 || block_size <= 0 ||
      num_kv_heads <= 0 || num_kv_heads > 65536 || max_path < 0 || num_arrays < 1 || num_arrays > 4 || !arrays ||
      !row_bytes || num_blocks <= 0 || num_blocks > INT64_MAX / block_size / num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_seqs) * num_arrays * num_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  pkv::AcceptArgs a{};
  for (int32_t i = 0; i < num_arrays; ++i) {
    if (!arrays[i] || (reinterpret_cast<uintptr_t>(arrays[i]) & 15) != 0 || row_bytes[i] <= 0 || row_bytes[i] % 4 != 0 ||
        row_bytes[i] > (1 << 20) || row_bytes[i] > INT64_MAX / (num_blocks * block_size * num_kv_heads))
      return PKV_ERR_INVALID_ARG;
    a.arrays[i] = static_cast<uint8_t *>(arrays[i]);
    a.row_bytes[i] = row_bytes[i];
  }
  if (num_seqs == 0 || max_path == 0) return PKV_OK;
  if (!cu_seqlens_q || !seq_slot || !context_lens || !block_tables || !paths) return PKV_ERR_INVALID_ARG;
  a.cu_seqlens_q = cu_seqlens_q;
  a.seq_slot = seq_slot;
  a.context_lens = context_lens;
  a.block_tables = block_tables;
  a.paths = paths;
  a.total_q = total_q;
  a.num_blocks = num_blocks;
  a.num_seqs = num_seqs;
  a.max_slots = max_slots;
  a.max_blocks_per_slot = max_blocks_per_slot;
  a.block_size = block_size;
  a.num_kv_heads = num_kv_heads;
  a.max_path = max_path;
  a.num_arrays = num_arrays;
  a.status = device_status;
  const cudaError_t e = pkv::launch_accept_rows(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
