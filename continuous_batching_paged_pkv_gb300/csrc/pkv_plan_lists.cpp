// Host planning of block-sparse steps and of steps of trees: the work lists of
// pkv_plan_work_sparse and pkv_plan_work_tree, and the trees' ancestor masks.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <vector>

#include "pkv.h"
#include "pkv_internal.h"

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Item {
  int32_t w[4];
  int64_t cost;
};

struct Shape {
  int32_t max_slots, max_blocks_per_slot, block_size, num_q_heads, num_kv_heads, head_dim;
  int32_t group() const { return num_q_heads / num_kv_heads; }
};

// The checks that every planner makes before it looks at the segments.
pkv_status check_step(const int32_t *cu, int32_t num_seqs, const int32_t *seq_slot, const int32_t *context_lens,
                      const Shape &sh, pkv_work_info *info, int32_t kind) {
  if (!info || num_seqs < 0 || !cu || (num_seqs > 0 && (!seq_slot || !context_lens)) || sh.max_slots <= 0 ||
      sh.max_blocks_per_slot <= 0)
    return PKV_ERR_INVALID_ARG;
  std::memset(info, 0, sizeof(*info));
  info->modified = kind;
  if (sh.num_kv_heads <= 0 || sh.num_q_heads <= 0 || sh.num_q_heads % sh.num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  if (sh.group() > 16 || (sh.head_dim != 64 && sh.head_dim != 128) ||
      (sh.block_size != 16 && sh.block_size != 32 && sh.block_size != 64))
    return PKV_ERR_UNSUPPORTED;
  return cu[0] < 0 ? PKV_ERR_INVALID_ARG : PKV_OK;
}

// One segment: its rows and context, PKV_OK with n = 0 for an empty one.
pkv_status check_segment(const int32_t *cu, int32_t s, const int32_t *seq_slot, const int32_t *context_lens,
                         const Shape &sh, std::vector<uint8_t> &used, int32_t &n, int32_t &slot, int32_t &L) {
  if (cu[s + 1] < cu[s]) return PKV_ERR_INVALID_ARG;
  n = cu[s + 1] - cu[s];
  slot = seq_slot[s];
  if (slot < 0 || slot >= sh.max_slots) return PKV_ERR_OUT_OF_RANGE;
  if (used[slot]) return PKV_ERR_INVALID_ARG;
  used[slot] = 1;
  L = context_lens[slot];
  if (n > L || L < 0) return PKV_ERR_INVALID_ARG;
  return static_cast<int64_t>(L) > static_cast<int64_t>(sh.max_blocks_per_slot) * sh.block_size ? PKV_ERR_OUT_OF_RANGE
                                                                                                : PKV_OK;
}

// Longest first, ties in their original order.
void sort_items(std::vector<Item> &v) {
  std::stable_sort(v.begin(), v.end(), [](const Item &a, const Item &b) { return a.cost > b.cost; });
}

// Counts, sizes and, where there is room, the words.
pkv_status finish(std::vector<Item> &dec, std::vector<Item> &pre, std::vector<Item> &comb, std::vector<Item> &scr,
                  int64_t partials, const Shape &sh, int32_t *work, int64_t work_capacity, pkv_work_info *info) {
  const int64_t items = static_cast<int64_t>(dec.size() + pre.size() + comb.size() + scr.size());
  if (partials > INT32_MAX || items > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  sort_items(dec);
  sort_items(comb);
  info->num_decode_items = static_cast<int32_t>(dec.size());
  info->num_prefill_items = static_cast<int32_t>(pre.size());
  info->num_combine_items = static_cast<int32_t>(comb.size());
  info->num_scratch_items = static_cast<int32_t>(scr.size());
  info->num_long_combine_items = static_cast<int32_t>(
      std::count_if(comb.begin(), comb.end(), [](const Item &it) { return it.cost > pkv::kLongMergeSpans; }));
  info->num_partials = static_cast<int32_t>(partials);
  info->work_words = items * PKV_WORK_WORDS_PER_ITEM;
  info->workspace_bytes = info->workspace_bytes_q8 = pkv::partial_bytes(partials, sh.num_q_heads, sh.head_dim);
  if (info->num_scratch_items > 0)
    info->workspace_bytes = info->workspace_bytes_q8 =
        std::max(info->workspace_bytes,
                 pkv::select_layout(info->scratch_blocks, sh.num_kv_heads).bytes);
  if (!work || work_capacity < info->work_words) return PKV_ERR_WORKSPACE_TOO_SMALL;
  for (const auto *v : {&dec, &pre, &comb, &scr})
    for (const Item &it : *v) {
      std::memcpy(work, it.w, sizeof(it.w));
      work += PKV_WORK_WORDS_PER_ITEM;
    }
  return PKV_OK;
}

pkv_status plan_sparse(const int32_t *cu, int32_t num_seqs, const int32_t *seq_slot, const int32_t *context_lens,
                       const Shape &sh, const pkv_sparse &sp, int32_t *work, int64_t work_capacity,
                       pkv_work_info *info) {
  if (const pkv_status st = check_step(cu, num_seqs, seq_slot, context_lens, sh, info, pkv::kListSparse); st != PKV_OK)
    return st;
  constexpr int64_t kSubsPerSpan = PKV_SPLIT_KEYS / pkv::kSubKeys;
  const int32_t most_rows = std::max<int32_t>(1, 16 / sh.group());
  std::vector<Item> dec, pre, comb, scr;
  std::vector<uint8_t> used(static_cast<size_t>(sh.max_slots), 0);
  int64_t partials = 0, candidates = 0;
  for (int32_t s = 0; s < num_seqs; ++s) {
    int32_t n, slot, L;
    if (const pkv_status st = check_segment(cu, s, seq_slot, context_lens, sh, used, n, slot, L); st != PKV_OK) return st;
    if (n == 0) continue;
    if (n > most_rows) return PKV_ERR_UNSUPPORTED;
    info->decode_rows_max = std::max(info->decode_rows_max, n);
    const pkv::SparseBlocks b = pkv::sparse_blocks(L, n, sh.block_size, sp.top_blocks, sp.keep_first, sp.keep_last);
    // selection: candidates only where not every block is read
    const int64_t cand = b.blocks > b.read ? b.last - b.first : 0;
    if (b.blocks > b.read && b.first + (b.blocks - b.last) > sp.top_blocks) return PKV_ERR_INVALID_ARG;
    if (candidates + cand > INT32_MAX - pkv::kScoreBlocks || cand > (1 << 20)) return PKV_ERR_UNSUPPORTED;
    pre.push_back({{s, slot, static_cast<int32_t>(candidates), static_cast<int32_t>(cand)}, cand});
    for (int64_t c = 0; c < cand; c += pkv::kScoreBlocks)
      scr.push_back({{s, slot, static_cast<int32_t>(c), static_cast<int32_t>(candidates)}, 0});
    candidates += ceil_div(cand, pkv::kScoreBlocks) * pkv::kScoreBlocks;
    // attention: spans over the list of blocks, whose last one may be partly filled
    const int64_t keys = L - (b.blocks - b.read) * sh.block_size;
    const int32_t sk = pkv::span_keys(keys, sh.max_slots, sh.num_kv_heads);
    const int64_t spans = ceil_div(keys, sk);
    if (keys > (int64_t(1) << 23) * PKV_SPLIT_KEYS || spans >= (1 << 16)) return PKV_ERR_UNSUPPORTED;
    if (partials + spans * n > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < spans; ++i) {
      const int64_t k0 = i * sk / pkv::kSubKeys, k1 = ceil_div(std::min(keys, (i + 1) * sk), pkv::kSubKeys);
      const uint32_t w = static_cast<uint32_t>(k0 / kSubsPerSpan) | static_cast<uint32_t>(k0 % kSubsPerSpan) << 23 |
                         static_cast<uint32_t>(k1 - k0) << 27;
      dec.push_back({{s, slot, static_cast<int32_t>(w), spans > 1 ? static_cast<int32_t>(partials + i * n) : -1}, k1 - k0});
    }
    if (spans > 1) {
      for (int32_t i = 0; i < n; ++i)
        comb.push_back({{s, slot, static_cast<int32_t>(spans) | (i << 16) | ((n - 1) << 24),
                         static_cast<int32_t>(partials + i)}, spans});
      partials += spans * n;
    }
  }
  sort_items(pre);
  info->scratch_blocks = candidates;
  return finish(dec, pre, comb, scr, partials, sh, work, work_capacity, info);
}

pkv_status plan_tree(const int32_t *cu, int32_t num_seqs, const int32_t *seq_slot, const int32_t *context_lens,
                     const Shape &sh, int32_t *work, int64_t work_capacity, pkv_work_info *info) {
  if (const pkv_status st = check_step(cu, num_seqs, seq_slot, context_lens, sh, info, pkv::kListTree); st != PKV_OK)
    return st;
  const int32_t rows_per_tile = pkv::prefill_rows_per_tile(sh.group());
  std::vector<Item> dec, none, comb;
  std::vector<uint8_t> used(static_cast<size_t>(sh.max_slots), 0);
  int64_t partials = 0;
  for (int32_t s = 0; s < num_seqs; ++s) {  // the kernel's variant follows the largest segment
    if (cu[s + 1] < cu[s]) return PKV_ERR_INVALID_ARG;
    info->decode_rows_max = std::max(info->decode_rows_max, cu[s + 1] - cu[s]);
  }
  if (info->decode_rows_max > PKV_TREE_MAX_ROWS) return PKV_ERR_UNSUPPORTED;
  const int32_t step = pkv::tree_tiles_per_cta(info->decode_rows_max, sh.group());
  for (int32_t s = 0; s < num_seqs; ++s) {
    int32_t n, slot, L;
    if (const pkv_status st = check_segment(cu, s, seq_slot, context_lens, sh, used, n, slot, L); st != PKV_OK) return st;
    if (n == 0) continue;
    if (L > pkv::kTreeMaxKeys) return PKV_ERR_UNSUPPORTED;
    const int32_t q_tiles = static_cast<int32_t>(ceil_div(n, rows_per_tile));
    const int64_t tiles = ceil_div(L, pkv::kTreeTileKeys);
    const int64_t span = pkv::tree_span_tiles(tiles, q_tiles, sh.max_slots, sh.num_kv_heads);
    const int64_t spans = ceil_div(tiles, span);
    if (spans > pkv::kTreeMaxSpans || partials + spans * n > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < spans; ++i)
      for (int32_t t = 0; t < q_tiles; t += step) {
        const uint32_t w = static_cast<uint32_t>(i) | static_cast<uint32_t>(span - 1) << 16 | static_cast<uint32_t>(t) << 24;
        dec.push_back({{s, slot, static_cast<int32_t>(w), spans > 1 ? static_cast<int32_t>(partials + i * n) : -1},
                       std::min(span, tiles - i * span)});
      }
    if (spans > 1) {
      for (int32_t i = 0; i < n; ++i)
        comb.push_back({{s, slot, static_cast<int32_t>(spans | static_cast<int64_t>(i) << 16 |
                                                       static_cast<int64_t>(n - 1) << 24),
                         static_cast<int32_t>(partials + i)}, spans});
      partials += spans * n;
    }
  }
  return finish(dec, none, comb, none, partials, sh, work, work_capacity, info);
}

// No exception leaves a C entry: sizes that the host has no memory for are refused.
template <typename Fn, typename... Args>
pkv_status no_throw(Fn fn, Args &&...args) {
  try {
    return fn(args...);
  } catch (...) {
    return PKV_ERR_INVALID_ARG;
  }
}

}  // namespace

// Tiles of a span: as many spans as still leave one CTA to an SM (two where a segment's rows are one query tile)
// if all slots were as long, and no span longer than kTreeSpanTiles, so that the slots' different lengths even
// out (64 slots of up to 8192 keys: 154 us; 179 with spans of at most 32 tiles, whose starts and partials cost more).
// It depends on the segment and the tables' shape, not on the rest of the step. So a slot that stands idle counts as
// one of the same length, and few live slots of many get longer spans and fewer CTAs than the GPU holds: 5 slots x 8
// nodes of up to 8192 keys take 26.6 us with 5 slots in the tables, 45 with 16 and 74 with 64; one slot x 64 nodes,
// 32,768 keys, 45 us alone and 113 beside 15 or 63 idle ones (L2 flushed before each call).
int64_t pkv::tree_span_tiles(int64_t tiles, int32_t q_tiles, int32_t max_slots, int32_t num_kv_heads) {
  const int64_t ctas = q_tiles > 1 ? 152 : 304, units = ceil_div(q_tiles, 2);
  const int64_t spans = std::max<int64_t>(1, ctas / (static_cast<int64_t>(max_slots) * num_kv_heads * units));
  return std::min<int64_t>(kTreeSpanTiles, std::max<int64_t>(kTreeMinSpanTiles, ceil_div(tiles, spans)));
}

extern "C" {

pkv_status pkv_plan_work_sparse(const int32_t *cu, int32_t num_seqs, const int32_t *seq_slot,
                                const int32_t *context_lens, int32_t max_slots, int32_t max_blocks_per_slot,
                                int32_t block_size, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                const pkv_sparse *sparse, int32_t *work, int64_t work_capacity, pkv_work_info *info) {
  if (!sparse || sparse->top_blocks < 1 || sparse->keep_first < 0 || sparse->keep_last < 0) return PKV_ERR_INVALID_ARG;
  const Shape sh{max_slots, max_blocks_per_slot, block_size, num_q_heads, num_kv_heads, head_dim};
  return no_throw(plan_sparse, cu, num_seqs, seq_slot, context_lens, sh, *sparse, work, work_capacity, info);
}

pkv_status pkv_plan_work_tree(const int32_t *cu, int32_t num_seqs, const int32_t *seq_slot, const int32_t *context_lens,
                              int32_t max_slots, int32_t max_blocks_per_slot, int32_t block_size, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, int32_t *work, int64_t work_capacity,
                              pkv_work_info *info) {
  const Shape sh{max_slots, max_blocks_per_slot, block_size, num_q_heads, num_kv_heads, head_dim};
  return no_throw(plan_tree, cu, num_seqs, seq_slot, context_lens, sh, work, work_capacity, info);
}

pkv_status pkv_tree_masks(const int32_t *parents, const int32_t *cu, int32_t num_seqs, int32_t mask_words,
                          uint32_t *masks, int32_t *depths) {
  if (num_seqs < 0 || !cu || cu[0] < 0 || mask_words < 1 || mask_words > PKV_TREE_MAX_ROWS / 32)
    return PKV_ERR_INVALID_ARG;
  for (int32_t s = 0; s < num_seqs; ++s)  // before `parents` is read: it has as many entries as the last offset says
    if (cu[s + 1] < cu[s]) return PKV_ERR_INVALID_ARG;
  for (int32_t s = 0; s < num_seqs; ++s) {  // everything is checked before anything is written
    if (cu[s + 1] > cu[s] && !parents) return PKV_ERR_INVALID_ARG;
    if (cu[s + 1] - cu[s] > 32 * mask_words) return PKV_ERR_OUT_OF_RANGE;
    for (int32_t r = cu[s]; r < cu[s + 1]; ++r)
      if (parents[r] < -1 || parents[r] >= r - cu[s]) return PKV_ERR_INVALID_ARG;
  }
  for (int32_t s = 0; s < num_seqs; ++s)
    for (int32_t r = cu[s]; r < cu[s + 1]; ++r) {
      const int32_t i = r - cu[s], p = parents[r];
      if (masks) {
        uint32_t *m = masks + static_cast<int64_t>(r) * mask_words;
        for (int32_t w = 0; w < mask_words; ++w)
          m[w] = p < 0 ? 0u : masks[(static_cast<int64_t>(cu[s]) + p) * mask_words + w];
        m[i / 32] |= 1u << (i % 32);
      }
      if (depths) depths[r] = p < 0 ? 0 : depths[cu[s] + p] + 1;
    }
  return PKV_OK;
}

}  // extern "C"
