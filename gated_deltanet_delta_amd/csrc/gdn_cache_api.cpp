// C ABI of what stands around the paged KV cache: rotary positions, attention
// weights of cached tokens, eviction plans and their moves.  Argument validation
// and dispatch, as gdn_attn_api.cpp does for the attention.  Host code only.
#include <cmath>
#include <cstring>

#include "gdn.h"
#include "gdn_host.h"
#include "gdn_ops.h"

namespace {

using gdn::check_attn;
using gdn::check_stride;
using gdn::check_workspace;
using gdn::elem;
using gdn::fail;
using gdn::launched;
using gdn::ok;

constexpr int32_t kMaxTokens = 1 << 30;
constexpr int32_t kMaxMoves = 1 << 30;
constexpr int32_t kWeightsMaxWidth = 1 << 29;  // a workgroup of 256 threads to 64 keys: 2^31 threads along x
constexpr long double kTwoPiLong = 6.283185307179586476925286766559L;
constexpr double kTwoPi = static_cast<double>(kTwoPiLong);

// The base of the frequencies; rot_dims > 2.
double scaled_base(const gdn_rope* r) {
  return r->scaling == GDN_ROPE_BASE ? r->base * std::pow(r->factor, r->rot_dims / (r->rot_dims - 2.0)) : r->base;
}

gdn_status check_rope(const gdn_rope* r) {
  if (!r) return fail(GDN_ERR_NULL, "rope: NULL, required: a gdn_rope");
  if (r->rot_dims < 2 || r->rot_dims % 2 != 0)
    return fail(GDN_ERR_GEOMETRY, "rot_dims: %d, required: even and >= 2", r->rot_dims);
  if (r->layout != GDN_ROPE_HALF && r->layout != GDN_ROPE_PAIRS)
    return fail(GDN_ERR_GEOMETRY, "layout: %d, required: GDN_ROPE_HALF (0) or GDN_ROPE_PAIRS (1)", r->layout);
  if (r->scaling < GDN_ROPE_NONE || r->scaling > GDN_ROPE_PARTS)
    return fail(GDN_ERR_GEOMETRY, "scaling: %d, required: 0..%d", r->scaling, GDN_ROPE_PARTS);
  if ((r->flags & ~GDN_ROPE_INVERSE) != 0)
    return fail(GDN_ERR_GEOMETRY, "flags: %#x, required: 0 or GDN_ROPE_INVERSE (1)", r->flags);
  if (!std::isfinite(r->base) || r->base <= 1.0) return fail(GDN_ERR_GEOMETRY, "base: %g, required: finite and > 1", r->base);
  if (r->scaling != GDN_ROPE_NONE && (!std::isfinite(r->factor) || r->factor < 1.0))
    return fail(GDN_ERR_GEOMETRY, "factor: %g, required: finite and >= 1", r->factor);
  if (r->scaling == GDN_ROPE_PARTS) {
    if (!std::isfinite(r->context) || r->context < 1.0)
      return fail(GDN_ERR_GEOMETRY, "context: %g, required: finite and >= 1", r->context);
    if (!std::isfinite(r->low) || !std::isfinite(r->high) || r->low < 0.0 || r->high <= r->low)
      return fail(GDN_ERR_GEOMETRY, "low, high: %g, %g, required: finite, 0 <= low < high", r->low, r->high);
  }
  if (!std::isfinite(r->amplitude) || r->amplitude <= 0.f)
    return fail(GDN_ERR_GEOMETRY, "amplitude: %g, required: finite and > 0", r->amplitude);
  if (r->rot_dims % 16 != 0)
    return fail(GDN_ERR_UNSUPPORTED, "rot_dims: %d, supported by this library: a multiple of 16", r->rot_dims);
  if (!std::isfinite(scaled_base(r)))
    return fail(GDN_ERR_GEOMETRY, "base, factor: %g, %g, required: a finite base s^(R/(R-2))", r->base, r->factor);
  return ok();
}

// An output that is the input itself has its stride.
gdn_status check_in_place(const void* in, int64_t stride, const void* out, int64_t out_stride, const char* name) {
  if (in == out && stride != out_stride)
    return fail(GDN_ERR_RANGE, "%s: %lld, required: %lld, the stride of the input that it overwrites", name,
                static_cast<long long>(out_stride), static_cast<long long>(stride));
  return GDN_OK;
}

gdn_status check_width(int32_t width, int32_t most) {
  if (width < 1 || width > most) return fail(GDN_ERR_RANGE, "width: %d, required: 1..%d", width, most);
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_check_rope(const gdn_rope* r, char* msg, size_t msg_len) {
  const gdn_status s = check_rope(r);
  if (msg && msg_len) {
    std::strncpy(msg, gdn_last_error(), msg_len - 1);
    msg[msg_len - 1] = '\0';
  }
  return s;
}

gdn_status gdn_rope_turns(const gdn_rope* r, double* freq, uint64_t* turns) {
  const gdn_status s = check_rope(r);
  if (s != GDN_OK) return s;
  if (!turns) return fail(GDN_ERR_NULL, "turns: NULL, required: a host pointer");
  const int R = r->rot_dims;
  const double base = scaled_base(r);
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    if (r->scaling == GDN_ROPE_LINEAR) f /= r->factor;
    if (r->scaling == GDN_ROPE_PARTS) {
      const double n = r->context * f / kTwoPi;
      const double g = std::fmin(1.0, std::fmax(0.0, (n - r->low) / (r->high - r->low)));
      f *= (1.0 - g) / r->factor + g;
    }
    if (freq) freq[i] = f;
    // f <= 1, so below 2^62; the quotient in 64 bits of mantissa, as positions multiply its error
    turns[i] = static_cast<uint64_t>(std::nearbyint(f / kTwoPiLong * 0x1p64L));
  }
  return ok();
}

gdn_status gdn_rope_rotate(const gdn_attn_geometry* g, const gdn_rope* r, const uint64_t* turns, const int32_t* position,
                           int32_t n_tokens, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride,
                           const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, const void* v,
                           int64_t v_stride, void* k_cache, void* v_cache, const int32_t* slot_map, int32_t* dev_err,
                           void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if ((s = check_rope(r)) != GDN_OK) return s;
  if (r->rot_dims > g->d_head)
    return fail(GDN_ERR_GEOMETRY, "rot_dims: %d, required: <= d_head = %d", r->rot_dims, g->d_head);
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return fail(GDN_ERR_RANGE, "n_tokens: %d, required: 0..%d", n_tokens, kMaxTokens);
  if (q) {
    if ((s = check_stride(g, q_stride, g->n_q_heads, "q_stride")) != GDN_OK) return s;
    if ((s = check_stride(g, q_out_stride, g->n_q_heads, "q_out_stride")) != GDN_OK) return s;
    if ((s = check_in_place(q, q_stride, q_out, q_out_stride, "q_out_stride")) != GDN_OK) return s;
  }
  if (k) {
    if ((s = check_stride(g, k_stride, g->n_kv_heads, "k_stride")) != GDN_OK) return s;
    if ((s = check_stride(g, k_out_stride, g->n_kv_heads, "k_out_stride")) != GDN_OK) return s;
    if ((s = check_in_place(k, k_stride, k_out, k_out_stride, "k_out_stride")) != GDN_OK) return s;
  }
  if (k_cache && (s = check_stride(g, v_stride, g->n_kv_heads, "v_stride")) != GDN_OK) return s;
  if (n_tokens == 0) return ok();
  if (!q && !k) return fail(GDN_ERR_NULL, "q, k: both NULL, required: one of them at least");
  GDN_NEED_PTR(turns, "turns");
  GDN_NEED_PTR4(position, "position");
  if (q) {
    GDN_NEED_PTR(q, "q");
    GDN_NEED_PTR(q_out, "q_out");
  }
  if (k) {
    GDN_NEED_PTR(k, "k");
    GDN_NEED_PTR(k_out, "k_out");
  }
  if (k_cache) {
    GDN_NEED_PTR(k, "k");
    GDN_NEED_PTR(v, "v");
    GDN_NEED_PTR(k_cache, "k_cache");
    GDN_NEED_PTR(v_cache, "v_cache");
    GDN_NEED_PTR4(slot_map, "slot_map");
  }
  gdn::RopeArgs a{};
  a.q = q;
  a.q_out = q_out;
  a.q_stride = q_stride * elem(g);
  a.q_out_stride = q_out_stride * elem(g);
  a.k = k;
  a.k_out = k_out;
  a.k_stride = k_stride * elem(g);
  a.k_out_stride = k_out_stride * elem(g);
  a.v = v;
  a.v_stride = v_stride * elem(g);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.turns = turns;
  a.position = position;
  a.slot_map = slot_map;
  a.dev_err = dev_err;
  a.n_tokens = n_tokens;
  a.Hq = g->n_q_heads;
  a.Hk = g->n_kv_heads;
  a.D = g->d_head;
  a.R = r->rot_dims;
  a.page = g->page_tokens;
  a.n_pages = g->n_pages;
  a.inverse = (r->flags & GDN_ROPE_INVERSE) != 0;
  a.amplitude = r->amplitude;
  return launched(gdn::launch_rope(a, g->dtype == GDN_BF16, r->layout == GDN_ROPE_PAIRS, stream), "gdn_rope_rotate");
}

size_t gdn_attn_weights_workspace_bytes(const gdn_attn_geometry* g, int32_t batch, int32_t n, int32_t width) {
  if (check_attn(g) != GDN_OK || batch < 1 || batch > 65535 || n < 1 || n > g->max_tree || check_width(width, kWeightsMaxWidth) != GDN_OK)
    return 0;
  return gdn::weights_workspace_bytes(batch, n, width, g->n_kv_heads, g->n_q_heads / g->n_kv_heads, g->d_head,
                                      g->dtype == GDN_BF16);
}

gdn_status gdn_attn_weights(const gdn_attn_geometry* g, const void* q, int64_t q_stride, const int32_t* n_row,
                            int32_t batch, int32_t n, const void* k_cache, const int32_t* block_table,
                            const int32_t* kv_len, const int32_t* have_len, const float* score_in, float* score_out,
                            int32_t width, void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if (n < 1 || n > g->max_tree) return fail(GDN_ERR_RANGE, "n: %d, required: 1..max_tree = %d", n, g->max_tree);
  if (batch < 1 || batch > 65535) return fail(GDN_ERR_RANGE, "batch: %d, required: 1..65535", batch);
  if ((s = check_width(width, kWeightsMaxWidth)) != GDN_OK) return s;
  if ((s = check_stride(g, q_stride, g->n_q_heads, "q_stride")) != GDN_OK) return s;
  s = check_workspace(workspace, workspace_bytes, gdn_attn_weights_workspace_bytes(g, batch, n, width));
  if (s != GDN_OK) return s;
  GDN_NEED_PTR(q, "q");
  GDN_NEED_PTR(k_cache, "k_cache");
  GDN_NEED_PTR4(block_table, "block_table");
  GDN_NEED_PTR4(kv_len, "kv_len");
  if (n_row) GDN_NEED_PTR4(n_row, "n_row");
  if (have_len) GDN_NEED_PTR4(have_len, "have_len");
  if (score_in) GDN_NEED_PTR4(score_in, "score_in");
  GDN_NEED_PTR4(score_out, "score_out");
  gdn::WeightArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.block_table = block_table;
  a.kv_len = kv_len;
  a.have_len = have_len;
  a.n_row = n_row;
  a.score_in = score_in;
  a.score_out = score_out;
  a.workspace = workspace;
  a.dev_err = dev_err;
  a.batch = batch;
  a.n = n;
  a.width = width;
  a.Hk = g->n_kv_heads;
  a.G = g->n_q_heads / g->n_kv_heads;
  a.D = g->d_head;
  a.page = g->page_tokens;
  a.n_pages = g->n_pages;
  a.max_pages = g->max_pages;
  a.scale_log2 = static_cast<float>(static_cast<double>(g->scale) * 1.4426950408889634);
  return launched(gdn::launch_weights(a, g->dtype == GDN_BF16, stream), "gdn_attn_weights");
}

gdn_status gdn_evict_plan(const gdn_attn_geometry* g, const int32_t* kv_len, const int32_t* budget, const float* score,
                          const int32_t* token_pos, const int32_t* row_state, const int32_t* block_table,
                          int32_t* free_pages, const int32_t* n_free, int32_t batch, int32_t width, int32_t sink,
                          int32_t recent, float* score_out, int32_t* token_pos_out, int32_t* kv_len_out,
                          int32_t* row_state_out, int32_t* n_free_out, int32_t* move_src, int32_t* move_dst,
                          int32_t* n_moves, int32_t max_moves, int32_t* dev_err, void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if (batch < 1 || batch > gdn::kEvictMaxBatch)
    return fail(GDN_ERR_RANGE, "batch: %d, required: 1..%d", batch, gdn::kEvictMaxBatch);
  if ((s = check_width(width, gdn::kEvictMaxWidth)) != GDN_OK) return s;
  if (max_moves < 1 || max_moves > kMaxMoves)
    return fail(GDN_ERR_RANGE, "max_moves: %d, required: 1..%d", max_moves, kMaxMoves);
  if (sink < 0) return fail(GDN_ERR_RANGE, "sink: %d, required: >= 0", sink);
  if (recent < 0) return fail(GDN_ERR_RANGE, "recent: %d, required: >= 0", recent);
  GDN_NEED_PTR4(kv_len, "kv_len");
  GDN_NEED_PTR4(budget, "budget");
  GDN_NEED_PTR4(score, "score");
  GDN_NEED_PTR4(token_pos, "token_pos");
  GDN_NEED_PTR4(row_state, "row_state");
  GDN_NEED_PTR4(block_table, "block_table");
  GDN_NEED_PTR4(free_pages, "free_pages");
  GDN_NEED_PTR4(n_free, "n_free");
  GDN_NEED_PTR4(score_out, "score_out");
  GDN_NEED_PTR4(token_pos_out, "token_pos_out");
  GDN_NEED_PTR4(kv_len_out, "kv_len_out");
  GDN_NEED_PTR4(row_state_out, "row_state_out");
  GDN_NEED_PTR4(n_free_out, "n_free_out");
  GDN_NEED_PTR4(move_src, "move_src");
  GDN_NEED_PTR4(move_dst, "move_dst");
  GDN_NEED_PTR4(n_moves, "n_moves");
  if (kv_len_out == kv_len) return fail(GDN_ERR_RANGE, "kv_len_out: the same buffer as kv_len, required: another one");
  if (row_state_out == row_state)
    return fail(GDN_ERR_RANGE, "row_state_out: the same buffer as row_state, required: another one");
  if (n_free_out == n_free) return fail(GDN_ERR_RANGE, "n_free_out: the same buffer as n_free, required: another one");
  if (move_src == move_dst) return fail(GDN_ERR_RANGE, "move_dst: the same buffer as move_src, required: another one");
  gdn::EvictArgs a{};
  a.kv_len = kv_len;
  a.budget = budget;
  a.score = score;
  a.token_pos = token_pos;
  a.row_state = row_state;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.score_out = score_out;
  a.token_pos_out = token_pos_out;
  a.kv_len_out = kv_len_out;
  a.row_state_out = row_state_out;
  a.n_free_out = n_free_out;
  a.move_src = move_src;
  a.move_dst = move_dst;
  a.n_moves = n_moves;
  a.dev_err = dev_err;
  a.batch = batch;
  a.width = width;
  a.sink = sink;
  a.recent = recent;
  a.max_moves = max_moves;
  a.page = g->page_tokens;
  a.n_pages = g->n_pages;
  a.max_pages = g->max_pages;
  return launched(gdn::launch_evict_plan(a, stream), "gdn_evict_plan");
}

gdn_status gdn_kv_move(const gdn_attn_geometry* g, void* k_cache, void* v_cache, const int32_t* move_src,
                       const int32_t* move_dst, const int32_t* n_moves, int32_t batch, int32_t max_moves,
                       int32_t* dev_err, void* stream) {
  gdn_status s = check_attn(g);
  if (s != GDN_OK) return s;
  if (batch < 1 || batch > gdn::kEvictMaxBatch)
    return fail(GDN_ERR_RANGE, "batch: %d, required: 1..%d", batch, gdn::kEvictMaxBatch);
  if (max_moves < 1 || max_moves > kMaxMoves)
    return fail(GDN_ERR_RANGE, "max_moves: %d, required: 1..%d", max_moves, kMaxMoves);
  GDN_NEED_PTR(k_cache, "k_cache");
  GDN_NEED_PTR(v_cache, "v_cache");
  GDN_NEED_PTR4(move_src, "move_src");
  GDN_NEED_PTR4(move_dst, "move_dst");
  GDN_NEED_PTR4(n_moves, "n_moves");
  gdn::MoveArgs a{};
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.move_src = move_src;
  a.move_dst = move_dst;
  a.n_moves = n_moves;
  a.dev_err = dev_err;
  a.batch = batch;
  a.max_moves = max_moves;
  a.heads = g->n_kv_heads;
  a.row_bytes = g->d_head * elem(g);
  a.page = g->page_tokens;
  a.n_pages = g->n_pages;
  return launched(gdn::launch_kv_move(a, stream), "gdn_kv_move");
}

}  // extern "C"
