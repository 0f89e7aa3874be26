// Internal interfaces between the C-ABI layer (pkv_api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"

namespace pkv {

// Keys per 16-row sub-tile: the unit every kernel loads with one TMA box per
// 64-column half of head_dim.
constexpr int kSubKeys = 16;

struct StepArgs {
  const void *q;
  const void *k_pool;
  const void *v_pool;
  const int32_t *cu_seqlens_q;
  const int32_t *seq_slot;
  const int32_t *context_lens;
  const int32_t *block_tables;
  int32_t num_seqs, max_slots, max_blocks_per_slot, block_size;
  int64_t num_blocks, total_q;
  int32_t num_q_heads, num_kv_heads, group, head_dim;
  int32_t decode_rows_max;  // most rows of a segment on the decode path (1 for plain decode)
  float scale_log2;  // softmax scale times log2(e)
  const int32_t *work;
  void *out;
  float *partial_acc;  // [num_partials][Hq][D]
  float *partial_ml;   // [num_partials][Hq][2]  (running max in log2 units, sum)
  uint32_t *status;
  // Workspace word the decode kernel hands out tasks from past its first
  // three static rounds (nullptr: every task is assigned statically). The
  // launch zeroes it on the stream first.
  uint32_t *task_counter;
  // The chunk kernel's K/V pool is written by the kernel right before it (the
  // 8-bit and 4-bit paths' widening pass), and so is its block table: wait for
  // it before reading either.
  // Otherwise only the tiles holding this step's rows wait for the cache write.
  int32_t kv_from_previous;
  // `out` is page-locked host memory reached through its device address: the
  // chunk kernel then stages its rows in shared memory and stores whole rows,
  // which the host link carries at its copy rate (one 16-byte piece of 32
  // different rows per store it carries far slower).
  int32_t out_on_host;
  // Modified scores (pkv_score_mod; all zero for plain attention).
  int32_t modified;
  float softcap;
  int32_t window;
  const float *alibi_slopes;
  const int32_t *key_begin, *key_end;
  int32_t num_partials;  // span partials in the workspace: a modified list's items must stay among them
  // Block-sparse steps: int32 [num_seqs][Hkv][top_blocks], the places of the blocks that a segment reads.
  const int32_t *selected;
  int32_t top_blocks, keep_first, keep_last;
  // Trees: uint32 [total_q][mask_words], the step's rows that a row sees.
  const uint32_t *masks;
  int32_t mask_words;
};

// pkv_work_info::modified: which planner made a list, and StepArgs::modified.
constexpr int32_t kListPlain = 0, kListMod = 1, kListSparse = 2, kListTree = 3;

// pkv_attention with the output's location: out_on_host marks `out` as host
// memory (pkv_step's output written straight to the caller's host buffer).
// `mod`: the scores' modification (pkv_attention_mod), or nullptr.
pkv_status attention(const void *q, const int32_t *cu_seqlens_q, int32_t num_seqs, int64_t total_q,
                     const int32_t *seq_slot, const int32_t *context_lens, const int32_t *block_tables,
                     int32_t max_slots, int32_t max_blocks_per_slot, int32_t block_size, const void *k_pool,
                     const void *v_pool, int64_t num_blocks, int32_t num_q_heads, int32_t num_kv_heads,
                     int32_t head_dim, float scale, const int32_t *work, const pkv_work_info *info, void *out,
                     void *workspace, uint64_t workspace_bytes, uint32_t *device_status, pkv_stream_t stream,
                     bool out_on_host, const pkv_score_mod *mod = nullptr);

// Keys per decode span of a segment whose rows read `keys` keys, in the lists of listed sub-tiles (pkv_host.cpp).
int32_t span_keys(int64_t keys, int32_t max_slots, int32_t num_kv_heads);

// Rows of more spans than this are merged with four lanes per column.
constexpr int kLongMergeSpans = 64;

// Bytes of workspace after the span partials: the decode kernel's task counter.
constexpr uint64_t kCounterBytes = 256;

// Candidate blocks of one scoring item of the selection, and those that a warp scores at once.
constexpr int kScoreBlocks = 128, kScoreGroup = 16;

// Workspace of pkv_select_blocks: exact scores (fp64) and scores (fp32) of every (candidate, kv head), and per
// (group of candidates, kv head) the largest sum of magnitudes. A segment's candidates start at a multiple of
// kScoreBlocks, and so do its parts of these arrays. Offsets in bytes.
struct SelectLayout {
  uint64_t exact, scores, sums, bytes;
};
inline SelectLayout select_layout(int64_t candidates, int32_t num_kv_heads) {
  auto up = [](uint64_t x) { return (x + 255) & ~uint64_t(255); };
  const uint64_t n = static_cast<uint64_t>(candidates) * num_kv_heads;
  SelectLayout l;
  l.exact = 0;
  l.scores = up(n * 8);
  l.sums = l.scores + up(n * 4);
  l.bytes = l.sums + up(n / kScoreGroup * 4);
  return l;
}

// Blocks of a slot of L keys, n of them this step's rows, in a block-sparse step: all of them, the candidates
// [first, last), and how many are read. Everything else is always kept.
struct SparseBlocks {
  int64_t blocks, first, last, read;
};
inline SparseBlocks sparse_blocks(int64_t L, int64_t n, int32_t block_size, int32_t top, int32_t keep_first,
                                  int32_t keep_last) {
  SparseBlocks b;
  b.blocks = (L + block_size - 1) / block_size;
  b.last = (L - n) / block_size - keep_last;
  if (b.last < 0) b.last = 0;
  b.first = keep_first < b.last ? keep_first : b.last;
  b.read = top < b.blocks ? top : b.blocks;
  return b;
}

// Workspace of the span partials: sums, (max, denominator) pairs, the task counter.
inline uint64_t partial_bytes(int64_t partials, int32_t num_q_heads, int32_t head_dim) {
  auto up = [](uint64_t x) { return (x + 255) & ~uint64_t(255); };
  return partials == 0 ? 0
                       : up(static_cast<uint64_t>(partials) * num_q_heads * head_dim * 4) +
                             up(static_cast<uint64_t>(partials) * num_q_heads * 2 * 4) + kCounterBytes;
}
cudaError_t launch_cache_write(const void *k_new, const void *v_new, const int64_t *slot_mapping,
                               int64_t num_tokens, void *k_pool, void *v_pool, int64_t num_blocks,
                               int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                               uint32_t *status, cudaStream_t stream);

// Rotation of a step's rows (pkv_rope.cu): q rows to q_out; with kv heads, k
// rows rotated and v rows copied into the pool rows of slot_mapping.
struct RopeArgs {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_pool, *v_pool;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
  const int32_t *positions;
  const int64_t *slot_mapping;
  const uint64_t *phases;  // [rot_dim / 2] fractions of a turn per position
  int64_t num_tokens, num_blocks;
  int32_t num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved, block_size;
  float magnitude;
  uint32_t *status;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream);

constexpr int kCopyArrays = 5;  // most pool arrays of one call
cudaError_t launch_copy_blocks(const int32_t *pairs, int64_t num_pairs, void *const *arrays,
                               const int64_t *block_bytes, int32_t num_arrays, int64_t num_blocks, uint32_t *status,
                               cudaStream_t stream);

// Bounds of the blocks that a step touched (pkv_key_bounds.cu); bits 16 (bf16 pool, no scales), 8 or 4.
cudaError_t launch_key_bounds(const int64_t *slot_mapping, int64_t num_tokens, const void *keys, const void *scales,
                              void *bounds, int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                              int32_t head_dim, int32_t bits, uint32_t *status, cudaStream_t stream);

// Selection of a block-sparse step's blocks (pkv_select.cu); `workspace` laid out by select_layout.
cudaError_t launch_select_blocks(const StepArgs &a, const void *bounds, const pkv_work_info &info, void *workspace,
                                 int32_t *selected, cudaStream_t stream);

// Trees (pkv_tree.cu).
cudaError_t launch_tree(const StepArgs &a, const CUtensorMap &tmap_q, const CUtensorMap &tmap_k,
                        const CUtensorMap &tmap_v, int32_t num_items, const int32_t *items, cudaStream_t stream);

// Rows of accepted paths (pkv_accept.cu).
struct AcceptArgs {
  const int32_t *cu_seqlens_q, *seq_slot, *context_lens, *block_tables, *paths;
  uint8_t *arrays[4];
  int64_t row_bytes[4];
  int64_t total_q, num_blocks;
  int32_t num_seqs, max_slots, max_blocks_per_slot, block_size, num_kv_heads, max_path, num_arrays;
  uint32_t *status;
};
cudaError_t launch_accept_rows(const AcceptArgs &a, cudaStream_t stream);

// `beside_chunk`: the chunk kernel of the same step runs at the same time
// (head_dim 128 takes the small per-SM footprint described below).
cudaError_t launch_decode(const StepArgs &a, const CUtensorMap &tmap_k, const CUtensorMap &tmap_v,
                          int32_t num_items, const int32_t *items, bool beside_chunk, cudaStream_t stream);

// One CTA per (row of a multi-span segment, group of q heads): merges that
// row's span partials. The first `num_long` items (rows of more than two
// span groups) may take four lanes per column.
cudaError_t launch_merge(const StepArgs &a, int32_t num_items, int32_t num_long, const int32_t *items,
                         cudaStream_t stream);

// Block-scaled pools (bits = 8, or 4 at head_dim 128): quantising cache write,
// decode over the codes, and the widening of prompt-chunk histories into a
// bf16 scratch pool.
cudaError_t launch_cache_write_quant(const void *k_new, const void *v_new, const int64_t *slot_mapping,
                                  int64_t num_tokens, void *k_codes, void *k_scales, void *v_codes, void *v_scales,
                                  int64_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t bits, uint32_t *status, cudaStream_t stream);
cudaError_t launch_decode_quant(const StepArgs &a, const CUtensorMap &tmap_k_codes, const CUtensorMap &tmap_v_codes,
                             const void *k_scales, const void *v_scales, int32_t num_items, const int32_t *items,
                             int32_t bits, cudaStream_t stream);
cudaError_t launch_widen_quant(const StepArgs &a, const void *k_codes, const void *k_scales, const void *v_codes,
                            const void *v_scales, void *k_out, void *v_out, int32_t *scratch_table,
                            int64_t scratch_blocks, int32_t num_items, const int32_t *items, int32_t bits,
                            cudaStream_t stream);

cudaError_t launch_prefill(const StepArgs &a, const CUtensorMap &tmap_q, int32_t rows_per_tile,
                           int32_t num_items, const int32_t *items, cudaStream_t stream);
// head_dim 64 with modified scores.
cudaError_t launch_prefill_mod(const StepArgs &a, const CUtensorMap &tmap_q, const CUtensorMap &tmap_k,
                               const CUtensorMap &tmap_v, int32_t rows_per_tile, int32_t num_items,
                               const int32_t *items, cudaStream_t stream);
// head_dim 128: items are tile pairs, run by clusters of two CTAs.
// `beside_decode`: the step also has decode rows, whose kernel runs at the
// same time; the chunk kernel then keeps fewer K/V stages so that a decode CTA
// fits beside each of its CTAs.
cudaError_t launch_prefill_pair(const StepArgs &a, const CUtensorMap &tmap_q, const CUtensorMap &tmap_k,
                                const CUtensorMap &tmap_v, int32_t rows_per_tile, int32_t num_items,
                                const int32_t *items, bool beside_decode, cudaStream_t stream);

// A step with both prompt chunks and decode rows (head_dim 128) runs one CTA
// of each kernel on every SM: the chunk kernel with kPairStagesBesideDecode
// K/V stages (129 KiB of shared memory, 7 warps x 232 registers), the decode
// kernel with kDecodeWarpsBesideChunk warps of kDecodeStagesBesideChunk
// stages (81 KiB, 2 warps x at most 208 registers); together they stay within
// an SM's 228 KiB of shared memory and 64 Ki registers. The tensor-bound chunk
// tiles and the HBM-bound decode streams then share every SM instead of
// queueing for SMs.
constexpr int kPairStagesBesideDecode = 3;
constexpr int kDecodeWarpsBesideChunk = 4;
constexpr int kDecodeStagesBesideChunk = 2;

// Launch with programmatic stream serialization: the kernel may start while
// the previous kernel in the stream drains; it calls griddepcontrol.wait
// before touching any input.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Raises a kernel's dynamic shared-memory limit to `smem`, once per device,
// and asks for the largest shared-memory carve-out of the SM's L1 storage: a
// CTA of another kernel can join an SM only under the carve-out that SM was
// configured with, so the kernels meant to share SMs (a chunk CTA beside a
// decode CTA) must all ask for the same, largest one.
// `done` holds one bit per device (devices past 63 set the attributes on every
// call); two host threads racing on a first call both set them, which is harmless.
template <typename Kernel>
cudaError_t allow_smem_once(Kernel *kernel, int smem, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Tensor memory. An allocation waits, without a limit, until the SM has the columns. A kernel that lets the next one
// start before it has allocated its own must therefore never share an SM with a CTA of that one which took them first:
// it would wait for columns, and the other for its end. Shared memory keeps them apart. Every kernel that allocates
// takes at least kTmemSmemLeast bytes, so that three CTAs never fit, and one with all 512 columns takes so much that
// none fits beside it. (A kernel that allocates before it signals has nothing to fear.)
constexpr int kSmSmem = 228 * 1024, kCtaSmem = 1024;  // of an SM; what each CTA takes beyond its own
constexpr int kTmemSmemLeast = 99584;
constexpr bool tmem_apart(int columns, int smem) {
  return smem >= kTmemSmemLeast && 3 * (kTmemSmemLeast + kCtaSmem) > kSmSmem &&
         (columns <= 256 || smem + kTmemSmemLeast + 2 * kCtaSmem > kSmSmem);
}

// Positions per prefill tile: whole GQA groups fit one 128-row MMA tile.
inline int32_t prefill_rows_per_tile(int32_t group) { return 128 / group; }

// Trees (pkv_tree.cu): keys come in tiles of 128; a CTA takes two query tiles where some segment of the step has
// more than one, else one: 64 slots x 32 nodes of 8 q heads a kv head (two tiles a tree), up to 8192 keys, take 149 us
// (163 with one tile everywhere), one slot of 64 nodes of 4, 32,768 keys, 39.8 (42.3); where a tree is one tile, two
// leave half of a CTA idle, which costs a mixed step nothing: 64 trees of 8 nodes of 8 take 142 us, 63 of them beside
// one of 32 nodes 130 (L2 flushed before each call). Spans of kTreeMinSpanTiles to kTreeSpanTiles tiles.
constexpr int kTreeTileKeys = 128, kTreeMinSpanTiles = 2, kTreeSpanTiles = 64;
constexpr int kTreeMaxSpans = 0xFFFF;  // what an item's span and a merge item's count hold
constexpr int kTreeMaxKeys = kTreeMaxSpans * kTreeSpanTiles * kTreeTileKeys;  // the longest context, in the longest spans
inline int32_t tree_tiles_per_cta(int32_t rows_max, int32_t group) {
  return rows_max > prefill_rows_per_tile(group) ? 2 : 1;
}
int64_t tree_span_tiles(int64_t tiles, int32_t q_tiles, int32_t max_slots, int32_t num_kv_heads);

}  // namespace pkv
