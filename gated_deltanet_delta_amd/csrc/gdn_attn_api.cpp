// C ABI of the paged KV cache, the attention over it, and the verify over a
// tree of drafts: argument validation and dispatch, as gdn_api.cpp does for
// the layer's other entry points.  Host code only.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "gdn.h"
#include "gdn_host.h"
#include "gdn_ops.h"

namespace {

using gdn::fail;
using gdn::launched;
using gdn::ok;

constexpr int32_t kMaxLen = (1 << 30) - 1;  // cached tokens of a sequence
// rows of a packed call: a sequence's cached plus new tokens fit 31 bits, rounded
// up to whole tiles and with the tiles that are requested ahead of the last
constexpr int32_t kMaxTokens = (1 << 30) - 4096;

gdn_status check_attn(const gdn_attn_geometry* g) {
  if (!g) return fail(GDN_ERR_NULL, "attention geometry: NULL, required: a gdn_attn_geometry");
  if (g->n_kv_heads < 1) return fail(GDN_ERR_GEOMETRY, "n_kv_heads: %d, required: >= 1", g->n_kv_heads);
  if (g->n_q_heads < 1 || g->n_q_heads % g->n_kv_heads != 0)
    return fail(GDN_ERR_GEOMETRY, "n_q_heads: %d, required: a multiple of n_kv_heads = %d", g->n_q_heads,
                g->n_kv_heads);
  if (g->d_head < 1) return fail(GDN_ERR_GEOMETRY, "d_head: %d, required: >= 1", g->d_head);
  if (g->page_tokens < 1) return fail(GDN_ERR_GEOMETRY, "page_tokens: %d, required: >= 1", g->page_tokens);
  if (g->n_pages < 1) return fail(GDN_ERR_GEOMETRY, "n_pages: %d, required: >= 1", g->n_pages);
  if (g->max_pages < 1) return fail(GDN_ERR_GEOMETRY, "max_pages: %d, required: >= 1", g->max_pages);
  if (static_cast<int64_t>(g->n_pages) * g->page_tokens > INT32_MAX)
    return fail(GDN_ERR_GEOMETRY, "n_pages * page_tokens: %lld, required: <= %d",
                static_cast<long long>(g->n_pages) * g->page_tokens, INT32_MAX);
  if (static_cast<int64_t>(g->max_pages) * g->page_tokens > kMaxLen)
    return fail(GDN_ERR_GEOMETRY, "max_pages * page_tokens: %lld, required: <= %d",
                static_cast<long long>(g->max_pages) * g->page_tokens, kMaxLen);
  if (g->max_tree < 1 || g->max_tree > 64)
    return fail(GDN_ERR_GEOMETRY, "max_tree: %d, required: 1..64", g->max_tree);
  if (g->dtype != GDN_F32 && g->dtype != GDN_BF16)
    return fail(GDN_ERR_GEOMETRY, "dtype: %d, required: GDN_F32 (0) or GDN_BF16 (1)", g->dtype);
  if (!std::isfinite(g->scale) || g->scale <= 0.f)
    return fail(GDN_ERR_GEOMETRY, "scale: %g, required: finite and > 0", g->scale);
  if (g->scale > 0x1p127f)  // the kernels take scale log2(e), which has to be finite
    return fail(GDN_ERR_UNSUPPORTED, "scale: %g, supported by this library: <= 2^127", g->scale);
  if (g->d_head != 64 && g->d_head != 128 && g->d_head != 256)
    return fail(GDN_ERR_UNSUPPORTED, "d_head: %d, supported by this library: 64, 128 or 256", g->d_head);
  if (g->page_tokens % 16 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "page_tokens: %d, supported by this library: a multiple of 16", g->page_tokens);
  if (g->n_kv_heads > 1024)
    return fail(GDN_ERR_UNSUPPORTED, "n_kv_heads: %d, supported by this library: <= 1024", g->n_kv_heads);
  if (g->n_q_heads / g->n_kv_heads > 64)
    return fail(GDN_ERR_UNSUPPORTED, "n_q_heads/n_kv_heads: %d, supported by this library: <= 64",
                g->n_q_heads / g->n_kv_heads);
  return ok();
}

int elem(const gdn_attn_geometry* g) { return g->dtype == GDN_BF16 ? 2 : 4; }

// A row stride: at least the row, and whole 16-byte vectors.
gdn_status check_stride(const gdn_attn_geometry* g, int64_t stride, int heads, const char* name) {
  const int64_t row = static_cast<int64_t>(heads) * g->d_head;
  if (stride < row || stride * elem(g) % 16 != 0 || stride >= (1 << 24))
    return fail(GDN_ERR_RANGE, "%s: %lld, required: >= %lld and < 2^24 elements, and a multiple of 16 bytes", name,
                static_cast<long long>(stride), static_cast<long long>(row));
  return GDN_OK;
}

// own: the largest number of keys that a sequence has among the call's tokens
int attn_split(const gdn_attn_geometry* g, int64_t tokens, int n_seqs, int nodes, int64_t own, bool cached) {
  const int64_t keys = own + (cached ? static_cast<int64_t>(g->max_pages) * g->page_tokens : 0);
  return gdn::attn_splits(tokens, n_seqs, g->n_kv_heads, g->n_q_heads / g->n_kv_heads, g->d_head, nodes,
                          g->dtype == GDN_BF16, keys);
}
size_t attn_bytes(const gdn_attn_geometry* g, int64_t tokens, int n_seqs, int nodes) {
  return gdn::attn_part_bytes(tokens, n_seqs, g->n_kv_heads, g->n_q_heads / g->n_kv_heads, g->d_head, nodes,
                              g->dtype == GDN_BF16);
}

// The most that attn_bytes() gives for 1 .. most rows (or batch rows), whose calls
// take splits_of() parts: fewer with more rows.  Among calls of as many parts the
// one of the most rows needs the most.
template <class Splits, class Bytes>
size_t most_bytes(int64_t most, Splits splits_of, Bytes bytes_of) {
  size_t best = 0;
  for (int64_t n = most; n >= 1;) {
    best = std::max(best, bytes_of(n));
    const int parts = splits_of(n);
    int64_t lo = 0, hi = n;  // the largest below n with more parts: lo has more (or is 0), hi has not
    while (hi - lo > 1) {
      const int64_t mid = lo + (hi - lo) / 2;
      if (splits_of(mid) > parts) lo = mid;
      else hi = mid;
    }
    n = lo;
  }
  return best;
}

gdn::AttnArgs attn_args(const gdn_attn_geometry* g, int32_t n_split, void* workspace, int64_t tokens) {
  gdn::AttnArgs a{};
  a.Hq = g->n_q_heads;
  a.Hk = g->n_kv_heads;
  a.G = g->n_q_heads / g->n_kv_heads;
  a.D = g->d_head;
  a.page = g->page_tokens;
  a.n_pages = g->n_pages;
  a.max_pages = g->max_pages;
  a.n_split = n_split;
  a.n_tokens = static_cast<int32_t>(tokens);
  a.part = static_cast<float*>(workspace);  // not used where the call needs none
  a.scale_log2 = static_cast<float>(static_cast<double>(g->scale) * 1.4426950408889634);
  return a;
}

gdn_status check_workspace(const void* workspace, size_t workspace_bytes, size_t need) {
  if (workspace_bytes < need)
    return fail(GDN_ERR_WORKSPACE, "workspace_bytes: %zu, required: >= %zu", workspace_bytes, need);
  if (need > 0) GDN_NEED_PTR(workspace, "workspace");
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_check_attn_geometry(const gdn_attn_geometry* g, char* msg, size_t msg_len) {
  const gdn_status s = check_attn(g);
  if (msg && msg_len) {
    std::strncpy(msg, gdn_last_error(), msg_len - 1);
    msg[msg_len - 1] = '\0';
  }
  return s;
}

gdn_status gdn_kv_plan(const gdn_attn_geometry* g, const int32_t* kv_len, const int32_t* new_len,
                       int32_t* free_pages, const int32_t* n_free, int32_t* block_table, int32_t batch,
                       int32_t max_tokens, int32_t* cu_new, int32_t* slot_map, int32_t* position,
                       int32_t* kv_len_out, int32_t* n_free_out, int32_t* dev_err, void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if (batch < 1 || batch > gdn::kKvPlanMaxBatch)
    return fail(GDN_ERR_RANGE, "batch: %d, required: 1..%d", batch, gdn::kKvPlanMaxBatch);
  if (max_tokens < 0) return fail(GDN_ERR_RANGE, "max_tokens: %d, required: >= 0", max_tokens);
  GDN_NEED_PTR4(kv_len, "kv_len");
  GDN_NEED_PTR4(new_len, "new_len");
  GDN_NEED_PTR4(free_pages, "free_pages");
  GDN_NEED_PTR4(n_free, "n_free");
  GDN_NEED_PTR4(block_table, "block_table");
  GDN_NEED_PTR4(cu_new, "cu_new");
  if (max_tokens > 0) {
    GDN_NEED_PTR4(slot_map, "slot_map");
    GDN_NEED_PTR4(position, "position");
  }
  GDN_NEED_PTR4(kv_len_out, "kv_len_out");
  GDN_NEED_PTR4(n_free_out, "n_free_out");
  if (kv_len_out == kv_len) return fail(GDN_ERR_RANGE, "kv_len_out: the same buffer as kv_len, required: another one");
  if (n_free_out == n_free) return fail(GDN_ERR_RANGE, "n_free_out: the same buffer as n_free, required: another one");
  gdn::KvPlanArgs a{};
  a.kv_len = kv_len;
  a.new_len = new_len;
  a.n_free = n_free;
  a.free_pages = free_pages;
  a.block_table = block_table;
  a.cu_new = cu_new;
  a.slot_map = slot_map;
  a.position = position;
  a.kv_len_out = kv_len_out;
  a.n_free_out = n_free_out;
  a.dev_err = dev_err;
  a.batch = batch;
  a.max_tokens = max_tokens;
  a.page = g->page_tokens;
  a.n_pages = g->n_pages;
  a.max_pages = g->max_pages;
  return launched(gdn::launch_kv_plan(a, stream), "gdn_kv_plan");
}

gdn_status gdn_kv_write(const gdn_attn_geometry* g, void* k_cache, void* v_cache, const void* k, int64_t k_stride,
                        const void* v, int64_t v_stride, const int32_t* slot_map, int32_t n_tokens,
                        int32_t* dev_err, void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if (n_tokens < 0) return fail(GDN_ERR_RANGE, "n_tokens: %d, required: >= 0", n_tokens);
  if ((s = check_stride(g, k_stride, g->n_kv_heads, "k_stride")) != GDN_OK) return s;
  if ((s = check_stride(g, v_stride, g->n_kv_heads, "v_stride")) != GDN_OK) return s;
  GDN_NEED_PTR(k_cache, "k_cache");
  GDN_NEED_PTR(v_cache, "v_cache");
  if (n_tokens == 0) return ok();
  GDN_NEED_PTR(k, "k");
  GDN_NEED_PTR(v, "v");
  GDN_NEED_PTR4(slot_map, "slot_map");
  gdn::KvWriteArgs a{};
  a.k = k;
  a.v = v;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.slot_map = slot_map;
  a.dev_err = dev_err;
  a.k_stride = k_stride * elem(g);
  a.v_stride = v_stride * elem(g);
  a.n_tokens = n_tokens;
  a.heads = g->n_kv_heads;
  a.row_bytes = g->d_head * elem(g);
  a.page = g->page_tokens;
  a.n_pages = g->n_pages;
  return launched(gdn::launch_kv_write(a, stream), "gdn_kv_write");
}

size_t gdn_attn_prefill_workspace_bytes(const gdn_attn_geometry* g, int32_t n_tokens, int32_t n_seqs) {
  if (check_attn(g) != GDN_OK || n_tokens < 0 || n_seqs < 1) return 0;
  return attn_bytes(g, n_tokens, n_seqs, 0);
}

size_t gdn_attn_tree_workspace_bytes(const gdn_attn_geometry* g, int32_t batch, int32_t n) {
  if (check_attn(g) != GDN_OK || batch < 1 || n < 1 || n > g->max_tree) return 0;
  return attn_bytes(g, static_cast<int64_t>(batch) * n, batch, n);
}

size_t gdn_attn_prefill_workspace_max_bytes(const gdn_attn_geometry* g, int32_t max_tokens, int32_t max_seqs) {
  if (check_attn(g) != GDN_OK || max_tokens < 0 || max_seqs < 1) return 0;
  // one sequence has the fewest row tiles, so the most parts
  return most_bytes(
      max_tokens, [&](int64_t n) { return attn_split(g, n, 1, 0, INT64_MAX / 2, false); },
      [&](int64_t n) { return attn_bytes(g, n, 1, 0); });
}

size_t gdn_attn_tree_workspace_max_bytes(const gdn_attn_geometry* g, int32_t max_batch, int32_t max_n) {
  if (check_attn(g) != GDN_OK || max_batch < 1 || max_n < 1 || max_n > g->max_tree) return 0;
  size_t best = 0;
  for (int n = 1; n <= max_n; ++n)
    best = std::max(best, most_bytes(
                              max_batch,
                              [&](int64_t b) { return attn_split(g, b * n, static_cast<int>(b), n, INT64_MAX / 2, false); },
                              [&](int64_t b) { return attn_bytes(g, b * n, static_cast<int>(b), n); }));
  return best;
}

gdn_status gdn_attn_prefill(const gdn_attn_geometry* g, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride, const int32_t* cu_seqlens,
                            int32_t n_seqs, int32_t n_tokens, const void* k_cache, const void* v_cache,
                            const int32_t* block_table, const int32_t* ctx_len, void* workspace,
                            size_t workspace_bytes, void* o, int32_t* dev_err, void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if (n_seqs < 1) return fail(GDN_ERR_RANGE, "n_seqs: %d, required: >= 1", n_seqs);
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return fail(GDN_ERR_RANGE, "n_tokens: %d, required: 0..%d", n_tokens, kMaxTokens);
  if ((s = check_stride(g, q_stride, g->n_q_heads, "q_stride")) != GDN_OK) return s;
  if ((s = check_stride(g, k_stride, g->n_kv_heads, "k_stride")) != GDN_OK) return s;
  if ((s = check_stride(g, v_stride, g->n_kv_heads, "v_stride")) != GDN_OK) return s;
  const int n_split = attn_split(g, n_tokens, n_seqs, 0, n_tokens, ctx_len != nullptr);
  s = check_workspace(workspace, workspace_bytes, attn_bytes(g, n_tokens, n_seqs, 0));
  if (s != GDN_OK) return s;
  GDN_NEED_PTR4(cu_seqlens, "cu_seqlens");
  if (ctx_len) {
    GDN_NEED_PTR4(ctx_len, "ctx_len");
    GDN_NEED_PTR4(block_table, "block_table");
    GDN_NEED_PTR(k_cache, "k_cache");
    GDN_NEED_PTR(v_cache, "v_cache");
  }
  if (n_tokens == 0) return ok();
  GDN_NEED_PTR(q, "q");
  GDN_NEED_PTR(k, "k");
  GDN_NEED_PTR(v, "v");
  GDN_NEED_PTR(o, "o");
  gdn::AttnArgs a = attn_args(g, n_split, workspace, n_tokens);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.ctx_len = ctx_len;
  a.cu_seqlens = cu_seqlens;
  a.o = o;
  a.dev_err = dev_err;
  a.n_seqs = n_seqs;
  return launched(gdn::launch_attn(a, g->dtype == GDN_BF16, stream), "gdn_attn_prefill");
}

gdn_status gdn_attn_tree(const gdn_attn_geometry* g, const void* q, int64_t q_stride, const void* k,
                         int64_t k_stride, const void* v, int64_t v_stride, const int32_t* parent,
                         const int32_t* n_row, int32_t batch, int32_t n, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, const int32_t* ctx_len, void* workspace,
                         size_t workspace_bytes, void* o, int32_t* dev_err, void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if (n < 1 || n > g->max_tree) return fail(GDN_ERR_RANGE, "n: %d, required: 1..max_tree = %d", n, g->max_tree);
  if (batch < 1 || batch > INT32_MAX / n)
    return fail(GDN_ERR_RANGE, "batch: %d, required: 1..%d for n = %d", batch, INT32_MAX / n, n);
  if ((s = check_stride(g, q_stride, g->n_q_heads, "q_stride")) != GDN_OK) return s;
  if ((s = check_stride(g, k_stride, g->n_kv_heads, "k_stride")) != GDN_OK) return s;
  if ((s = check_stride(g, v_stride, g->n_kv_heads, "v_stride")) != GDN_OK) return s;
  const int64_t rows = static_cast<int64_t>(batch) * n;
  const int n_split = attn_split(g, rows, batch, n, n, true);
  s = check_workspace(workspace, workspace_bytes, attn_bytes(g, rows, batch, n));
  if (s != GDN_OK) return s;
  GDN_NEED_PTR(q, "q");
  GDN_NEED_PTR(k, "k");
  GDN_NEED_PTR(v, "v");
  GDN_NEED_PTR4(parent, "parent");
  if (n_row) GDN_NEED_PTR4(n_row, "n_row");
  GDN_NEED_PTR(k_cache, "k_cache");
  GDN_NEED_PTR(v_cache, "v_cache");
  GDN_NEED_PTR4(block_table, "block_table");
  GDN_NEED_PTR4(ctx_len, "ctx_len");
  GDN_NEED_PTR(o, "o");
  gdn::AttnArgs a = attn_args(g, n_split, workspace, rows);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.ctx_len = ctx_len;
  a.parent = parent;
  a.n_row = n_row;
  a.nodes = n;
  a.o = o;
  a.dev_err = dev_err;
  a.n_seqs = batch;
  return launched(gdn::launch_attn(a, g->dtype == GDN_BF16, stream), "gdn_attn_tree");
}

gdn_status gdn_verify_tree_slots(const gdn_geometry* g, float* state, float* conv_state, int32_t* conv_pos,
                                 const void* x, const void* a_in, const void* b_in, const float* conv_w,
                                 const int32_t* slot, int32_t batch, int32_t k, const int32_t* k_row,
                                 const int32_t* parent, const int32_t* snap_slot, void* o, int32_t* dev_err,
                                 void* stream) {
  gdn_status s = gdn_check_geometry(g, nullptr, 0);
  if (s != GDN_OK) return s;
  if (batch < 1 || batch > g->n_slots)
    return fail(GDN_ERR_RANGE, "batch: %d, required: 1..n_slots = %d", batch, g->n_slots);
  if (k < 1 || k > g->max_draft) return fail(GDN_ERR_RANGE, "k: %d, required: 1..max_draft = %d", k, g->max_draft);
  if (static_cast<int64_t>(batch) * (k + 1) > g->n_slots)
    return fail(GDN_ERR_RANGE,
                "batch * (k + 1): %lld, required: <= n_slots = %d (rows and snapshots need distinct slots)",
                static_cast<long long>(batch) * (k + 1), g->n_slots);
  GDN_NEED_PTR(state, "state");
  if (g->conv_width > 0) {
    GDN_NEED_PTR(conv_state, "conv_state");
    GDN_NEED_PTR4(conv_pos, "conv_pos");
    GDN_NEED_PTR(conv_w, "conv_w");
  }
  GDN_NEED_PTR(x, "x");
  GDN_NEED_PTR(a_in, "a");
  GDN_NEED_PTR(b_in, "b");
  GDN_NEED_PTR4(slot, "slot");
  if (k_row) GDN_NEED_PTR4(k_row, "k_row");
  GDN_NEED_PTR4(parent, "parent");
  GDN_NEED_PTR4(snap_slot, "snap_slot");
  GDN_NEED_PTR(o, "o");
  gdn::TreeArgs a{};
  a.Hk = g->n_k_heads;
  a.Hv = g->n_v_heads;
  a.D = g->d_k;
  a.C = g->conv_channels;
  a.W = g->conv_width;
  a.R = g->conv_ring;
  a.n_slots = g->n_slots;
  a.flags = g->flags;
  a.q_scale = g->q_scale;
  a.l2_eps = g->l2_eps;
  a.state = state;
  a.conv_state = conv_state;
  a.conv_pos = conv_pos;
  a.x = x;
  a.a = a_in;
  a.b = b_in;
  a.conv_w = conv_w;
  a.slot = slot;
  a.k_row = k_row;
  a.parent = parent;
  a.snap_slot = snap_slot;
  a.o = o;
  a.dev_err = dev_err;
  a.batch = batch;
  a.k = k;
  GDN_DEBUG_DISTINCT("gdn_verify_tree_slots", slot, batch, snap_slot, batch, k, k_row);
  return launched(gdn::launch_verify_tree(a, g->dtype_in == GDN_BF16, stream), "gdn_verify_tree_slots");
}

}  // extern "C"
