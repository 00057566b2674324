// Arguments and launchers of the attention layers' kernels (gdn_kv.hip,
// gdn_attn.hip, gdn_attn_bf16.hip, gdn_rope.hip, gdn_weights.hip, gdn_evict.hip) and
// of the delta rule over trees (gdn_tree.hip).
#pragma once

#include "gdn_internal.h"

namespace gdn {

// The verify into pool slots over trees.
struct TreeArgs : StepArgs {
  const int32_t* parent;  // [batch][k]: parent node of each draft, -1 for the committed state
};

// Arguments of the paged-cache kernels (gdn_kv.hip).
struct KvPlanArgs {
  const int32_t *kv_len, *new_len, *n_free;
  int32_t *free_pages, *block_table, *cu_new, *slot_map, *position, *kv_len_out, *n_free_out, *dev_err;
  int32_t batch, max_tokens, page, n_pages, max_pages;
};
struct KvWriteArgs {
  const void *k, *v;
  void *k_cache, *v_cache;
  const int32_t* slot_map;
  int32_t* dev_err;
  int64_t k_stride, v_stride;  // bytes between tokens
  int32_t n_tokens, heads, row_bytes, page, n_pages;  // row_bytes: one head's D elements
};
constexpr int kKvPlanMaxBatch = 4096;

// Arguments of the attention kernels (gdn_attn.hip), prefill and tree.  Rows
// of a sequence are its (token, query head of one KV head's group) pairs, token
// major; keys are the sequence's cached tokens followed by its own.
struct AttnArgs {
  const void *q, *k, *v, *k_cache, *v_cache;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* block_table;
  const int32_t* ctx_len;     // null: no cached tokens
  const int32_t* cu_seqlens;  // prefill
  const int32_t* parent;      // tree
  const int32_t* n_row;       // tree, may be null
  void* o;
  float* part;                // partial outputs [token][H_q][n_split][D], then (max, sum) [token][H_q][n_split][2]
  int32_t* dev_err;
  int32_t n_seqs, n_tokens;   // tree: batch, batch * n
  int32_t nodes;              // tree: n; prefill: 0
  int32_t Hq, Hk, G, D, page, n_pages, max_pages;
  int32_t n_split;
  float scale_log2;           // scale * log2(e)
};

// Rotary positions (gdn_rope.hip).  Strides in bytes.
struct RopeArgs {
  const void *q, *k, *v;
  void *q_out, *k_out, *k_cache, *v_cache;
  int64_t q_stride, q_out_stride, k_stride, k_out_stride, v_stride;
  const uint64_t* turns;
  const int32_t *position, *slot_map;
  int32_t* dev_err;
  int32_t n_tokens, Hq, Hk, D, R, page, n_pages;
  bool inverse;
  float amplitude;
};

// Attention weights of cached tokens (gdn_weights.hip).
struct WeightArgs {
  const void *q, *k_cache;
  int64_t q_stride;  // elements between tokens
  const int32_t *block_table, *kv_len, *have_len, *n_row;
  const float* score_in;
  float* score_out;
  void* workspace;
  int32_t* dev_err;
  int32_t batch, n, width;
  int32_t Hk, G, D, page, n_pages, max_pages;
  float scale_log2;
};

// Eviction (gdn_evict.hip).
struct EvictArgs {
  const int32_t *kv_len, *budget, *token_pos, *row_state, *block_table, *n_free;
  const float* score;
  int32_t* free_pages;
  float* score_out;
  int32_t *token_pos_out, *kv_len_out, *row_state_out, *n_free_out, *move_src, *move_dst, *n_moves, *dev_err;
  int32_t batch, width, sink, recent, max_moves, page, n_pages, max_pages;
};
struct MoveArgs {
  void *k_cache, *v_cache;
  const int32_t *move_src, *move_dst, *n_moves;
  int32_t* dev_err;
  int32_t batch, max_moves, heads, row_bytes, page, n_pages;
};
constexpr int kEvictMaxBatch = 4096, kEvictMaxWidth = 1 << 18;  // width: a bit per token in LDS

// Launchers: return 0 on success, else the hipError_t value.
int launch_verify_tree(const TreeArgs& a, bool bf16, void* stream);
int launch_kv_plan(const KvPlanArgs& a, void* stream);
int launch_kv_write(const KvWriteArgs& a, void* stream);
// A launch has fewer than 2^32 threads along x.
inline bool grid_fits(int64_t workgroups, int threads) { return workgroups <= 0xffffffffll / threads; }
// Splits of the key axis of an attention call (1: none), by its row tiles and
// `keys`, the most keys that a row can have, since only the device knows the
// lengths; bf16 trees are split on the device.
int attn_splits(int64_t tokens, int n_seqs, int Hk, int G, int D, int nodes, bool bf16, int64_t keys);
// Workspace of a call: tokens = rows of q (trees: batch x nodes).
size_t attn_part_bytes(int64_t tokens, int n_seqs, int Hk, int G, int D, int nodes, bool bf16);
int launch_attn(const AttnArgs& a, bool bf16, void* stream);
int launch_rope(const RopeArgs& a, bool bf16, bool pairs, void* stream);
size_t weights_workspace_bytes(int32_t batch, int32_t n, int32_t width, int Hk, int G, int D, bool bf16);
int launch_weights(const WeightArgs& a, bool bf16, void* stream);
int launch_evict_plan(const EvictArgs& a, void* stream);
int launch_kv_move(const MoveArgs& a, void* stream);
constexpr int kPromptRows = 256;  // rows of a workgroup of the bf16 prompt attention
int launch_prompt_bf16(const AttnArgs& a, int64_t tiles, void* stream);
int launch_tree_bf16(const AttnArgs& a, void* stream);
size_t tree_bf16_part_bytes(int64_t batch, int Hk, int G, int D, int nodes);

}  // namespace gdn
