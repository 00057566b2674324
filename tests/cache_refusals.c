/* Every host-side check of the rotary, weights, eviction and move entry points,
 * driven from C (see abi_refusals.c): no call here passes validation or has any
 * work, so nothing is launched and no GPU is needed.
 * Exit status: 0, or the number of the failed check. */
#include <math.h>
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

static gdn_rope rope(void) {
  gdn_rope r;
  memset(&r, 0, sizeof r);
  r.rot_dims = 64;
  r.layout = GDN_ROPE_HALF;
  r.scaling = GDN_ROPE_PARTS;
  r.base = 1e4;
  r.factor = 4.0;
  r.context = 4096.0;
  r.low = 1.0;
  r.high = 32.0;
  r.amplitude = 1.0f;
  return r;
}

#define P ((void*)(uintptr_t)0x10000)
#define PT ((uint64_t*)(uintptr_t)0x10000)
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

/* The rotary call with one argument replaced. */
typedef struct rot {
  const uint64_t* turns;
  const int32_t* position;
  int32_t n;
  const void* q;
  int64_t qs;
  void* qo;
  int64_t qos;
  const void* k;
  int64_t ks;
  void* ko;
  int64_t kos;
  const void* v;
  int64_t vs;
  void *kc, *vc;
  const int32_t* slot;
} rot;
static rot rot_ok(void) {
  rot a = {PT, PI, 4, P, 6144, PF, 6144, P, 1024, PF, 1024, P, 1024, P, P, PI};
  return a;
}
static gdn_status call(const gdn_attn_geometry* g, const gdn_rope* r, const rot* a) {
  return gdn_rope_rotate(g, r, a->turns, a->position, a->n, a->q, a->qs, a->qo, a->qos, a->k, a->ks, a->ko, a->kos, a->v,
                         a->vs, a->kc, a->vc, a->slot, NULL, NULL);
}
#define ROT(id, change, status, needle)                          \
  do {                                                           \
    rot a = rot_ok();                                            \
    change;                                                      \
    CHECK(id, call(&g, &r, &a) == (status) && has(needle));      \
  } while (0)

int main(void) {
  char msg[256];
  gdn_attn_geometry g = base();
  gdn_rope r = rope();
  double freq[32];
  uint64_t turns[32];

  CHECK(1, gdn_check_rope(&r, msg, sizeof msg) == GDN_OK && msg[0] == '\0');
  CHECK(2, gdn_check_rope(NULL, msg, sizeof msg) == GDN_ERR_NULL && strstr(msg, "rope"));
  CHECK(3, gdn_rope_turns(&r, freq, turns) == GDN_OK && freq[0] == 1.0 && turns[0] == 2935890503282001226ull);
  CHECK(4, gdn_rope_turns(&r, NULL, turns) == GDN_OK);
  CHECK(5, gdn_rope_turns(&r, freq, NULL) == GDN_ERR_NULL && has("turns: NULL"));
  struct { int field; double value; gdn_status st; const char* needle; } cases[] = {
      {0, 0, GDN_ERR_GEOMETRY, "rot_dims: 0"},
      {0, 63, GDN_ERR_GEOMETRY, "rot_dims: 63"},
      {0, -16, GDN_ERR_GEOMETRY, "rot_dims: -16"},
      {0, 24, GDN_ERR_UNSUPPORTED, "rot_dims: 24, supported by this library: a multiple of 16"},
      {1, 2, GDN_ERR_GEOMETRY, "layout: 2"},
      {1, -1, GDN_ERR_GEOMETRY, "layout: -1"},
      {2, 4, GDN_ERR_GEOMETRY, "scaling: 4"},
      {2, -1, GDN_ERR_GEOMETRY, "scaling: -1"},
      {3, 2, GDN_ERR_GEOMETRY, "flags: 0x2"},
      {4, 1.0, GDN_ERR_GEOMETRY, "base: 1"},
      {4, (double)INFINITY, GDN_ERR_GEOMETRY, "base: inf"},
      {4, (double)NAN, GDN_ERR_GEOMETRY, "base: "},
      {5, 0.5, GDN_ERR_GEOMETRY, "factor: 0.5"},
      {6, 0.0, GDN_ERR_GEOMETRY, "context: 0"},
      {7, -1.0, GDN_ERR_GEOMETRY, "low, high: -1"},
      {8, 1.0, GDN_ERR_GEOMETRY, "low, high: 1, 1"},
      {9, 0.0, GDN_ERR_GEOMETRY, "amplitude: 0"},
      {9, (double)INFINITY, GDN_ERR_GEOMETRY, "amplitude: inf"}};
  for (unsigned i = 0; i < sizeof cases / sizeof cases[0]; ++i) {
    gdn_rope b = rope();
    double* d[] = {&b.base, &b.factor, &b.context, &b.low, &b.high};
    if (cases[i].field == 0) b.rot_dims = (int32_t)cases[i].value;
    else if (cases[i].field == 1) b.layout = (int32_t)cases[i].value;
    else if (cases[i].field == 2) b.scaling = (int32_t)cases[i].value;
    else if (cases[i].field == 3) b.flags = (uint32_t)cases[i].value;
    else if (cases[i].field == 9) b.amplitude = (float)cases[i].value;
    else *d[cases[i].field - 4] = cases[i].value;
    rot a = rot_ok();
    CHECK(100 + (int)i, gdn_check_rope(&b, msg, sizeof msg) == cases[i].st && strstr(msg, cases[i].needle));
    CHECK(200 + (int)i, gdn_check_rope(&b, msg, 8) == cases[i].st && strlen(msg) <= 7);
    CHECK(300 + (int)i, gdn_rope_turns(&b, freq, turns) == cases[i].st);
    CHECK(400 + (int)i, call(&g, &b, &a) == cases[i].st);
  }
  gdn_attn_geometry small = base();
  small.d_head = 64;
  r.rot_dims = 80;
  rot whole = rot_ok();
  whole.qs = whole.qos = 24 * 64;
  whole.ks = whole.kos = whole.vs = 4 * 64;
  CHECK(6, call(&small, &r, &whole) == GDN_ERR_GEOMETRY && has("rot_dims: 80, required: <= d_head = 64"));
  r = rope();
  gdn_attn_geometry bad = base();
  bad.n_q_heads = 23;
  rot okay = rot_ok();
  CHECK(7, call(&bad, &r, &okay) == GDN_ERR_GEOMETRY);
  CHECK(8, call(NULL, &r, &okay) == GDN_ERR_NULL);
  CHECK(9, call(&g, NULL, &okay) == GDN_ERR_NULL);
  ROT(10, a.n = -1, GDN_ERR_RANGE, "n_tokens: -1");
  ROT(11, a.n = (1 << 30) + 1, GDN_ERR_RANGE, "n_tokens: 1073741825");
  ROT(12, a.qs = 6143, GDN_ERR_RANGE, "q_stride: 6143");
  ROT(13, a.qs = 6145, GDN_ERR_RANGE, "q_stride: 6145");
  ROT(14, a.qos = 1 << 24, GDN_ERR_RANGE, "q_out_stride: 16777216");
  ROT(15, a.ks = 0, GDN_ERR_RANGE, "k_stride: 0");
  ROT(16, a.kos = 1016, GDN_ERR_RANGE, "k_out_stride: 1016");
  ROT(17, a.vs = -1024, GDN_ERR_RANGE, "v_stride: -1024");
  ROT(18, (a.qo = P, a.qos = 6152), GDN_ERR_RANGE, "q_out_stride: 6152, required: 6144, the stride of the input");
  ROT(19, (a.ko = P, a.kos = 2048), GDN_ERR_RANGE, "k_out_stride: 2048, required: 1024");
  ROT(20, (a.q = NULL, a.k = NULL, a.kc = NULL), GDN_ERR_NULL, "q, k: both NULL");
  ROT(21, a.turns = NULL, GDN_ERR_NULL, "turns");
  ROT(22, a.turns = (uint64_t*)ODD, GDN_ERR_ALIGN, "turns");
  ROT(23, a.position = NULL, GDN_ERR_NULL, "position");
  ROT(24, a.position = ODDI, GDN_ERR_ALIGN, "position");
  ROT(25, a.qo = NULL, GDN_ERR_NULL, "q_out");
  ROT(26, a.q = ODD, GDN_ERR_ALIGN, "q:");
  ROT(27, a.ko = NULL, GDN_ERR_NULL, "k_out");
  ROT(28, a.k = NULL, GDN_ERR_NULL, "k:");
  ROT(29, a.v = NULL, GDN_ERR_NULL, "v:");
  ROT(30, a.vc = NULL, GDN_ERR_NULL, "v_cache");
  ROT(31, a.kc = ODD, GDN_ERR_ALIGN, "k_cache");
  ROT(32, a.slot = NULL, GDN_ERR_NULL, "slot_map");
  rot none = rot_ok();
  none.n = 0;
  CHECK(33, call(&g, &r, &none) == GDN_OK);

#define W(gg, q, qs, b, n, kc, bt, kv, si, so, width, ws, wb) \
  gdn_attn_weights(gg, q, qs, NULL, b, n, kc, bt, kv, NULL, si, so, width, ws, wb, NULL, NULL)
  CHECK(40, W(&bad, P, 6144, 4, 1, P, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_GEOMETRY);
  CHECK(41, W(&g, P, 6144, 4, 0, P, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_RANGE && has("n: 0"));
  CHECK(42, W(&g, P, 6144, 4, 9, P, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_RANGE && has("n: 9, required: 1..max_tree = 8"));
  CHECK(43, W(&g, P, 6144, 0, 1, P, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_RANGE && has("batch: 0"));
  CHECK(44, W(&g, P, 6144, 65536, 1, P, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_RANGE && has("batch: 65536"));
  CHECK(45, W(&g, P, 6144, 4, 1, P, PI, PI, PF, PF, 0, P, BIG) == GDN_ERR_RANGE && has("width: 0"));
  CHECK(46, W(&g, P, 6144, 4, 1, P, PI, PI, PF, PF, (1 << 30) + 1, P, BIG) == GDN_ERR_RANGE && has("width"));
  CHECK(39, W(&g, P, 6144, 4, 1, P, PI, PI, PF, PF, (1 << 29) + 1, P, BIG) == GDN_ERR_RANGE && has("width: 536870913, required: 1..536870912"));
  CHECK(47, W(&g, P, 6136, 4, 1, P, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_RANGE && has("q_stride: 6136"));
  const size_t need = gdn_attn_weights_workspace_bytes(&g, 4, 1, 100);
  CHECK(48, need > 0 && W(&g, P, 6144, 4, 1, P, PI, PI, PF, PF, 100, P, need - 1) == GDN_ERR_WORKSPACE);
  CHECK(49, W(&g, P, 6144, 4, 1, P, PI, PI, PF, PF, 100, NULL, need) == GDN_ERR_NULL && has("workspace"));
  CHECK(50, W(&g, P, 6144, 4, 1, P, PI, PI, PF, PF, 100, ODD, need) == GDN_ERR_ALIGN && has("workspace"));
  CHECK(51, W(&g, NULL, 6144, 4, 1, P, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_NULL && has("q"));
  CHECK(52, W(&g, P, 6144, 4, 1, NULL, PI, PI, PF, PF, 100, P, BIG) == GDN_ERR_NULL && has("k_cache"));
  CHECK(53, W(&g, P, 6144, 4, 1, P, NULL, PI, PF, PF, 100, P, BIG) == GDN_ERR_NULL && has("block_table"));
  CHECK(54, W(&g, P, 6144, 4, 1, P, PI, NULL, PF, PF, 100, P, BIG) == GDN_ERR_NULL && has("kv_len"));
  CHECK(55, W(&g, P, 6144, 4, 1, P, PI, PI, PF, NULL, 100, P, BIG) == GDN_ERR_NULL && has("score_out"));
  CHECK(56, W(&g, P, 6144, 4, 1, P, PI, PI, (float*)ODDI, PF, 100, P, BIG) == GDN_ERR_ALIGN && has("score_in"));
  CHECK(57, gdn_attn_weights(&g, P, 6144, ODDI, 4, 1, P, PI, PI, NULL, PF, PF, 100, P, BIG, NULL, NULL) == GDN_ERR_ALIGN && has("n_row"));
  CHECK(58, gdn_attn_weights(&g, P, 6144, NULL, 4, 1, P, PI, PI, ODDI, PF, PF, 100, P, BIG, NULL, NULL) == GDN_ERR_ALIGN && has("have_len"));
  CHECK(59, gdn_attn_weights_workspace_bytes(&bad, 4, 1, 100) == 0 && gdn_attn_weights_workspace_bytes(&g, 0, 1, 100) == 0 &&
                gdn_attn_weights_workspace_bytes(&g, 4, 9, 100) == 0 && gdn_attn_weights_workspace_bytes(&g, 4, 1, 0) == 0 &&
                gdn_attn_weights_workspace_bytes(&g, 65536, 1, 100) == 0);
  /* it grows with batch, n and width */
  size_t before = 0;
  g.max_tree = 64;
  for (int n = 1; n <= 64; ++n) {
    const size_t now = gdn_attn_weights_workspace_bytes(&g, 4, n, 1000);
    CHECK(60, now >= before && gdn_attn_weights_workspace_bytes(&g, 5, n, 1000) >= now &&
                  gdn_attn_weights_workspace_bytes(&g, 4, n, 1001) >= now);
    before = now;
  }
  g = base();

  {
    const int32_t* in[] = {PI, PI, PI, PI, PI, PI, PI};  /* kv_len budget score token_pos row_state block_table n_free */
    int32_t* out[] = {PI, PF == NULL ? NULL : PI, PJ, PJ, PJ, PI, PJ, PI, PI};
    const char* in_names[] = {"kv_len", "budget", "score", "token_pos", "row_state", "block_table", "n_free"};
    const char* out_names[] = {"free_pages", "score_out", "token_pos_out", "kv_len_out", "row_state_out", "n_free_out", "move_src", "move_dst", "n_moves"};
    int32_t* out_ok[] = {PI, PI, PI, PJ, PJ, PJ, PI, PJ, PI};
    memcpy(out, out_ok, sizeof out);
#define E(gg, batch, width, sink, recent, moves)                                                                              \
  gdn_evict_plan(gg, in[0], in[1], (const float*)in[2], in[3], in[4], in[5], out[0], in[6], batch, width, sink, recent,         \
                 (float*)out[1], out[2], out[3], out[4], out[5], out[6], out[7], out[8], moves, NULL, NULL)
    CHECK(70, E(&bad, 4, 100, 0, 0, 10) == GDN_ERR_GEOMETRY);
    CHECK(71, E(&g, 0, 100, 0, 0, 10) == GDN_ERR_RANGE && has("batch: 0"));
    CHECK(72, E(&g, 4097, 100, 0, 0, 10) == GDN_ERR_RANGE && has("batch: 4097, required: 1..4096"));
    CHECK(73, E(&g, 4, 0, 0, 0, 10) == GDN_ERR_RANGE && has("width: 0"));
    CHECK(78, E(&g, 4, (1 << 18) + 1, 0, 0, 10) == GDN_ERR_RANGE && has("width: 262145, required: 1..262144"));
    CHECK(74, E(&g, 4, 100, -1, 0, 10) == GDN_ERR_RANGE && has("sink: -1"));
    CHECK(75, E(&g, 4, 100, 0, -1, 10) == GDN_ERR_RANGE && has("recent: -1"));
    CHECK(76, E(&g, 4, 100, 0, 0, 0) == GDN_ERR_RANGE && has("max_moves: 0"));
    CHECK(77, E(&g, 4, 100, 0, 0, (1 << 30) + 1) == GDN_ERR_RANGE && has("max_moves"));
    for (int i = 0; i < 7; ++i) {
      const int32_t* was = in[i];
      in[i] = NULL;
      CHECK(80 + i, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_NULL && has(in_names[i]));
      in[i] = ODDI;
      CHECK(90 + i, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_ALIGN && has(in_names[i]));
      in[i] = was;
    }
    for (int i = 0; i < 9; ++i) {
      int32_t* was = out[i];
      out[i] = NULL;
      CHECK(500 + i, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_NULL && has(out_names[i]));
      out[i] = ODDI;
      CHECK(510 + i, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_ALIGN && has(out_names[i]));
      out[i] = was;
    }
    out[3] = PI;
    CHECK(520, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_RANGE && has("kv_len_out: the same buffer"));
    out[3] = PJ, out[4] = PI;
    CHECK(521, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_RANGE && has("row_state_out: the same buffer"));
    out[4] = PJ, out[5] = PI;
    CHECK(522, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_RANGE && has("n_free_out: the same buffer"));
    out[5] = PJ, out[7] = PI;
    CHECK(523, E(&g, 4, 100, 0, 0, 10) == GDN_ERR_RANGE && has("move_dst: the same buffer"));
  }

#define M(gg, kc, vc, s, d, n, b, m) gdn_kv_move(gg, kc, vc, s, d, n, b, m, NULL, NULL)
  CHECK(530, M(&bad, P, P, PI, PI, PI, 4, 10) == GDN_ERR_GEOMETRY);
  CHECK(531, M(&g, P, P, PI, PI, PI, 0, 10) == GDN_ERR_RANGE && has("batch: 0"));
  CHECK(532, M(&g, P, P, PI, PI, PI, 4097, 10) == GDN_ERR_RANGE && has("batch: 4097"));
  CHECK(533, M(&g, P, P, PI, PI, PI, 4, 0) == GDN_ERR_RANGE && has("max_moves: 0"));
  CHECK(534, M(&g, NULL, P, PI, PI, PI, 4, 10) == GDN_ERR_NULL && has("k_cache"));
  CHECK(535, M(&g, P, ODD, PI, PI, PI, 4, 10) == GDN_ERR_ALIGN && has("v_cache"));
  CHECK(536, M(&g, P, P, NULL, PI, PI, 4, 10) == GDN_ERR_NULL && has("move_src"));
  CHECK(537, M(&g, P, P, PI, ODDI, PI, 4, 10) == GDN_ERR_ALIGN && has("move_dst"));
  CHECK(538, M(&g, P, P, PI, PI, NULL, 4, 10) == GDN_ERR_NULL && has("n_moves"));

  printf("cache refusals ok\n");
  return 0;
}
