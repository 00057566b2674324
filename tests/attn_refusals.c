/* Every host-side check of the paged-cache, attention and tree-verify entry
 * points, driven from C (see abi_refusals.c): no call here passes validation
 * or has any work, so nothing is launched and no GPU is needed.
 * Exit status: 0, or the number of the failed check. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdn.h"

static gdn_attn_geometry base(void) {
  gdn_attn_geometry g;
  memset(&g, 0, sizeof g);
  g.n_q_heads = 24;
  g.n_kv_heads = 4;
  g.d_head = 256;
  g.page_tokens = 16;
  g.n_pages = 100;
  g.max_pages = 50;
  g.max_tree = 8;
  g.dtype = GDN_BF16;
  g.scale = 0.0625f;
  return g;
}

#define P ((void*)(uintptr_t)0x10000)
#define PF ((float*)(uintptr_t)0x10000)
#define PI ((int32_t*)(uintptr_t)0x10000)
#define PJ ((int32_t*)(uintptr_t)0x20000)
#define ODD ((void*)(uintptr_t)0x10008)
#define ODDI ((int32_t*)(uintptr_t)0x10002)
#define BIG ((size_t)1 << 40)
#define CHECK(id, cond)                                                     \
  do {                                                                      \
    if (!(cond)) {                                                          \
      fprintf(stderr, "check %d failed: %s (%s)\n", id, #cond, gdn_last_error()); \
      return id;                                                            \
    }                                                                       \
  } while (0)

static int has(const char* needle) { return strstr(gdn_last_error(), needle) != NULL; }

int main(void) {
  char msg[256];
  gdn_attn_geometry g = base();
  CHECK(1, gdn_check_attn_geometry(&g, msg, sizeof msg) == GDN_OK && msg[0] == '\0');
  CHECK(2, gdn_check_attn_geometry(NULL, msg, sizeof msg) == GDN_ERR_NULL);
  struct { int field; int value; gdn_status st; const char* needle; } cases[] = {
      {0, 23, GDN_ERR_GEOMETRY, "n_q_heads: 23, required: a multiple of n_kv_heads = 4"},
      {0, 0, GDN_ERR_GEOMETRY, "n_q_heads: 0"},
      {0, 260, GDN_ERR_UNSUPPORTED, "n_q_heads/n_kv_heads: 65"},
      {1, 0, GDN_ERR_GEOMETRY, "n_kv_heads: 0"},
      {2, 0, GDN_ERR_GEOMETRY, "d_head: 0"},
      {2, 96, GDN_ERR_UNSUPPORTED, "d_head: 96, supported by this library: 64, 128 or 256"},
      {3, 0, GDN_ERR_GEOMETRY, "page_tokens: 0"},
      {3, 24, GDN_ERR_UNSUPPORTED, "page_tokens: 24"},
      {4, 0, GDN_ERR_GEOMETRY, "n_pages: 0"},
      {4, 1 << 28, GDN_ERR_GEOMETRY, "n_pages * page_tokens: 4294967296"},
      {5, 0, GDN_ERR_GEOMETRY, "max_pages: 0"},
      {5, 1 << 26, GDN_ERR_GEOMETRY, "max_pages * page_tokens: 1073741824, required: <= 1073741823"},
      {6, 0, GDN_ERR_GEOMETRY, "max_tree: 0"},
      {6, 65, GDN_ERR_GEOMETRY, "max_tree: 65"},
      {7, 2, GDN_ERR_GEOMETRY, "dtype: 2"}};
  for (unsigned i = 0; i < sizeof cases / sizeof cases[0]; ++i) {
    gdn_attn_geometry b = base();
    int32_t* f[] = {&b.n_q_heads, &b.n_kv_heads, &b.d_head, &b.page_tokens, &b.n_pages, &b.max_pages, &b.max_tree, &b.dtype};
    *f[cases[i].field] = cases[i].value;
    CHECK(100 + (int)i, gdn_check_attn_geometry(&b, msg, sizeof msg) == cases[i].st && strstr(msg, cases[i].needle));
    CHECK(200 + (int)i, gdn_check_attn_geometry(&b, msg, 8) == cases[i].st && strlen(msg) <= 7);
    CHECK(300 + (int)i, gdn_check_attn_geometry(&b, NULL, 0) == cases[i].st);
    CHECK(400 + (int)i, gdn_attn_prefill_workspace_bytes(&b, 100, 1) == 0 && gdn_attn_tree_workspace_bytes(&b, 1, 1) == 0);
    CHECK(500 + (int)i, gdn_kv_write(&b, P, P, P, 1024, P, 1024, PI, 4, NULL, NULL) == cases[i].st);
    CHECK(600 + (int)i, gdn_kv_plan(&b, PI, PI, PI, PI, PI, 4, 4, PI, PI, PI, PJ, PJ, NULL, NULL) == cases[i].st);
  }
  gdn_attn_geometry n = base();
  n.scale = 0.f;
  CHECK(3, gdn_check_attn_geometry(&n, NULL, 0) == GDN_ERR_GEOMETRY && has("scale: 0"));
  n.scale = -1.f;
  CHECK(4, gdn_check_attn_geometry(&n, NULL, 0) == GDN_ERR_GEOMETRY);

  /* plan */
  CHECK(10, gdn_kv_plan(&g, PI, PI, PI, PI, PI, 0, 4, PI, PI, PI, PJ, PJ, NULL, NULL) == GDN_ERR_RANGE && has("batch: 0"));
  CHECK(11, gdn_kv_plan(&g, PI, PI, PI, PI, PI, 4097, 4, PI, PI, PI, PJ, PJ, NULL, NULL) == GDN_ERR_RANGE);
  CHECK(12, gdn_kv_plan(&g, PI, PI, PI, PI, PI, 4, -1, PI, PI, PI, PJ, PJ, NULL, NULL) == GDN_ERR_RANGE && has("max_tokens: -1"));
  CHECK(13, gdn_kv_plan(&g, NULL, PI, PI, PI, PI, 4, 4, PI, PI, PI, PJ, PJ, NULL, NULL) == GDN_ERR_NULL && has("kv_len"));
  CHECK(14, gdn_kv_plan(&g, PI, PI, PI, PI, ODDI, 4, 4, PI, PI, PI, PJ, PJ, NULL, NULL) == GDN_ERR_ALIGN && has("block_table"));
  CHECK(15, gdn_kv_plan(&g, PI, PI, PI, PI, PI, 4, 4, PI, NULL, PI, PJ, PJ, NULL, NULL) == GDN_ERR_NULL && has("slot_map"));
  CHECK(16, gdn_kv_plan(&g, PI, PI, PI, PI, PI, 4, 4, PI, PI, PI, PI, PJ, NULL, NULL) == GDN_ERR_RANGE && has("kv_len_out"));
  CHECK(17, gdn_kv_plan(&g, PI, PI, PI, PI, PI, 4, 4, PI, PI, PI, PJ, PI, NULL, NULL) == GDN_ERR_RANGE && has("n_free_out"));
  /* write */
  CHECK(20, gdn_kv_write(&g, P, P, P, 1024, P, 1024, PI, -1, NULL, NULL) == GDN_ERR_RANGE);
  CHECK(21, gdn_kv_write(&g, P, P, P, 1023, P, 1024, PI, 4, NULL, NULL) == GDN_ERR_RANGE && has("k_stride: 1023"));
  CHECK(22, gdn_kv_write(&g, P, P, P, 1024, P, 1028, PI, 4, NULL, NULL) == GDN_ERR_RANGE && has("v_stride: 1028"));
  CHECK(23, gdn_kv_write(&g, ODD, P, P, 1024, P, 1024, PI, 4, NULL, NULL) == GDN_ERR_ALIGN && has("k_cache"));
  CHECK(24, gdn_kv_write(&g, P, P, P, 1024, P, 1024, NULL, 4, NULL, NULL) == GDN_ERR_NULL && has("slot_map"));
  CHECK(25, gdn_kv_write(&g, P, P, NULL, 1024, NULL, 1024, NULL, 0, NULL, NULL) == GDN_OK);
  /* prefill */
  CHECK(30, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 0, 9, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE && has("n_seqs: 0"));
  CHECK(31, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 1, -1, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE);
  CHECK(32, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 1, 1 << 30, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE);
  CHECK(33, gdn_attn_prefill(&g, P, 6136, P, 1024, P, 1024, PI, 1, 9, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE && has("q_stride"));
  size_t w = gdn_attn_prefill_workspace_bytes(&g, 9, 1);
  CHECK(42, gdn_attn_prefill(&g, P, 1 << 24, P, 1024, P, 1024, PI, 1, 9, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE && has("q_stride: 16777216"));
  CHECK(43, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1LL << 33, PI, 1, 9, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE && has("v_stride"));
  CHECK(34, w > 0 && gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 1, 9, P, P, PI, PI, P, w - 1, P, NULL, NULL) == GDN_ERR_WORKSPACE);
  CHECK(35, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 1, 9, P, P, PI, PI, NULL, w, P, NULL, NULL) == GDN_ERR_NULL && has("workspace"));
  CHECK(36, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, NULL, 1, 9, P, P, PI, PI, P, w, P, NULL, NULL) == GDN_ERR_NULL && has("cu_seqlens"));
  CHECK(37, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 1, 9, P, P, NULL, PI, P, w, P, NULL, NULL) == GDN_ERR_NULL && has("block_table"));
  CHECK(38, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 1, 9, P, ODD, PI, PI, P, w, P, NULL, NULL) == GDN_ERR_ALIGN && has("v_cache"));
  CHECK(39, gdn_attn_prefill(&g, P, 6144, P, 1024, P, 1024, PI, 1, 9, NULL, NULL, NULL, NULL, P, w, ODD, NULL, NULL) == GDN_ERR_ALIGN && has("o: address"));
  CHECK(40, gdn_attn_prefill(&g, NULL, 6144, NULL, 1024, NULL, 1024, PI, 1, 0, NULL, NULL, NULL, NULL, NULL, 0, NULL, NULL, NULL) == GDN_OK);
  CHECK(41, gdn_attn_prefill_workspace_bytes(&g, -1, 1) == 0 && gdn_attn_prefill_workspace_bytes(&g, 9, 0) == 0);
  /* tree */
  CHECK(50, gdn_attn_tree(&g, P, 6144, P, 1024, P, 1024, PI, NULL, 2, 9, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE && has("n: 9, required: 1..max_tree = 8"));
  CHECK(51, gdn_attn_tree(&g, P, 6144, P, 1024, P, 1024, PI, NULL, 0, 8, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE && has("batch: 0"));
  CHECK(52, gdn_attn_tree(&g, P, 6144, P, 1024, P, 1024, PI, NULL, 1 << 28, 8, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_RANGE);
  CHECK(53, gdn_attn_tree(&g, P, 6144, P, 1024, P, 1024, NULL, NULL, 2, 8, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_NULL && has("parent"));
  CHECK(54, gdn_attn_tree(&g, P, 6144, P, 1024, P, 1024, PI, ODDI, 2, 8, P, P, PI, PI, P, BIG, P, NULL, NULL) == GDN_ERR_ALIGN && has("n_row"));
  CHECK(55, gdn_attn_tree(&g, P, 6144, P, 1024, P, 1024, PI, NULL, 2, 8, P, P, PI, NULL, P, BIG, P, NULL, NULL) == GDN_ERR_NULL && has("ctx_len"));
  w = gdn_attn_tree_workspace_bytes(&g, 2, 8);
  CHECK(56, w > 0 && gdn_attn_tree(&g, P, 6144, P, 1024, P, 1024, PI, NULL, 2, 8, P, P, PI, PI, P, w - 1, P, NULL, NULL) == GDN_ERR_WORKSPACE);
  CHECK(57, gdn_attn_tree_workspace_bytes(&g, 0, 8) == 0 && gdn_attn_tree_workspace_bytes(&g, 2, 9) == 0);
  /* the delta rule over a tree */
  gdn_geometry d;
  memset(&d, 0, sizeof d);
  d.n_k_heads = 16;
  d.n_v_heads = 48;
  d.d_k = d.d_v = 128;
  d.conv_width = 4;
  d.conv_channels = 10240;
  d.conv_ring = 8;
  d.max_draft = 4;
  d.n_slots = 20;
  d.dtype_in = d.dtype_out = GDN_BF16;
  d.flags = GDN_FLAG_L2NORM_QK;
  d.q_scale = 1.f;
  d.l2_eps = 1e-6f;
  CHECK(60, gdn_verify_tree_slots(&d, PF, PF, PI, P, P, P, PF, PI, 4, 5, NULL, PI, PI, P, NULL, NULL) == GDN_ERR_RANGE && has("k: 5"));
  CHECK(61, gdn_verify_tree_slots(&d, PF, PF, PI, P, P, P, PF, PI, 5, 4, NULL, PI, PI, P, NULL, NULL) == GDN_ERR_RANGE && has("batch * (k + 1): 25"));
  CHECK(62, gdn_verify_tree_slots(&d, PF, PF, PI, P, P, P, PF, PI, 21, 4, NULL, PI, PI, P, NULL, NULL) == GDN_ERR_RANGE);
  CHECK(63, gdn_verify_tree_slots(&d, PF, PF, PI, P, P, P, PF, PI, 4, 4, NULL, NULL, PI, P, NULL, NULL) == GDN_ERR_NULL && has("parent"));
  CHECK(64, gdn_verify_tree_slots(&d, PF, PF, PI, P, P, P, PF, PI, 4, 4, ODDI, PI, PI, P, NULL, NULL) == GDN_ERR_ALIGN && has("k_row"));
  CHECK(65, gdn_verify_tree_slots(&d, PF, PF, PI, P, P, P, PF, PI, 4, 4, NULL, PI, NULL, P, NULL, NULL) == GDN_ERR_NULL && has("snap_slot"));
  CHECK(66, gdn_verify_tree_slots(NULL, PF, PF, PI, P, P, P, PF, PI, 4, 4, NULL, PI, PI, P, NULL, NULL) == GDN_ERR_NULL);
  d.n_v_heads = 47;
  CHECK(67, gdn_verify_tree_slots(&d, PF, PF, PI, P, P, P, PF, PI, 4, 4, NULL, PI, PI, P, NULL, NULL) == GDN_ERR_GEOMETRY);
  printf("attention refusals ok\n");
  return 0;
}
