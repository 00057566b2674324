// Attention for gfx950: causal over packed prompts with cached prefixes, and
// over a tree of drafts behind a paged cache.
//
//   s_rj = scale q_r . k_j,   o_r = sum_j e^(s_rj - m_r) v_j / sum_j e^(s_rj - m_r)
//
// in one pass over the keys: with the running maximum m and sum l of a row, a
// tile of keys gives m' = max(m, max_j s_j), and O and l are scaled by
// e^(m - m') before the tile's terms are added.  Exponentials are taken base 2
// of logits scaled by scale log2(e).
//
// Rows of a sequence are its (token, query head) pairs for one KV head, token
// major, so the query heads of a group share the K and V tiles; keys are the
// sequence's cached tokens (through the block table) followed by its own.  The
// products are formed transposed, S^T = K Q^T and O^T = V^T P^T: a query row is
// then a column of every accumulator, its statistics are scalars of the lanes
// that hold it, and the accumulators of P^T are the operand of the second
// product as they are.
//
// With more than one split of the key axis each split writes its unscaled sums
// with (m, l), and attn_combine_kernel joins them in a fixed order.
#include <algorithm>

#include "gdn_attn_device.h"

namespace gdn {

namespace {

__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
// Maximum over the four lanes of a column (lanes l % 16).
__device__ __forceinline__ float quarter_max(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));  // of rows of 16 lanes: 0 0 2 2 and 1 1 3 3
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));  // of halves: 0 0 and 1 1
}
}  // namespace

// ---------------------------------------------------------------------------
// fp32: 64 rows x 32 keys per step, four waves of 16 rows each, K and V rows
// staged through LDS.  16x16x4 matrix instructions: with c = l % 16, g = l / 16,
// lane l holds rows 4 g + i of column (query row) c of a product, and element
// (c, g) of an operand.  What index of a row an operand's element stands for is
// free as long as both operands agree, and is taken so that four instructions'
// operands are 16 bytes of LDS: instruction 4 s + i of the logits contracts
// elements 16 s + 4 g + i of K and Q; instruction i of half h of the keys
// contracts keys 16 h + 4 g + i (where the weights are), and row c of V^T's block
// dt stands for d = 64 (dt / 4) + 4 c + dt % 4.  (bf16: gdn_attn_bf16.hip.)
//
// Bound by the matrix instructions and, as much again, the vector instructions of
// softmax, addresses and copies between them: 1024 tokens of 8 heads on 2, d 64,
// behind 4096 cached ones 132 us (73 TFLOP/s; a large fp32 product reaches 154); short prompts (301, 1 and
// 777 tokens) 30 us, of which the join of the splits is 6.  One of the two arrays
// of rows in flight lies in private memory (48, 80 and 144 bytes per lane at d 64,
// 128 and 256), so these rows make a way through it at every step.  Trees: 4 rows of
// one node at 8K, 24 heads on 4, d 256, 227 us (267 MB, 1.2 TB/s), of 16 nodes 437 us;
// 64 rows of 8 nodes up to 16K, 32 heads on 8, d 128, 2680 us.
// ---------------------------------------------------------------------------
constexpr int kGenRows = 64, kGenKeys = 32, kGenThreads = 256;
constexpr int kMaxSplits = 64;  // parts of a row

template <int D>
struct GenShape {
  static constexpr int ES = 4;
  static constexpr int VEC = 16 / ES;               // elements of a 16-byte vector
  static constexpr int LD = D + VEC;                // LDS row, 16 bytes of padding against bank conflicts
  static constexpr int VPR = D / VEC;               // vectors of a row
  static constexpr int TILE_BYTES = kGenKeys * LD * ES;
};

template <int D, bool TREE>
__global__ __launch_bounds__(kGenThreads) void attn_f32_kernel(AttnArgs A) {
  using Sh = GenShape<D>;
  constexpr int ES = Sh::ES, LD = Sh::LD, NT = D / 16;
  constexpr int QF = D / 4;  // k-steps of the logits
  typedef float E;
  extern __shared__ __align__(16) char lds[];  // K tile, V tile, P of a tile (rare), flags
  E* Ks = reinterpret_cast<E*>(lds);
  E* Vs = reinterpret_cast<E*>(lds + Sh::TILE_BYTES);
  float* Ps = reinterpret_cast<float*>(lds + 2 * Sh::TILE_BYTES);  // [4 waves][32 keys][16 rows]
  uint32_t* bad_keys = reinterpret_cast<uint32_t*>(Ps + 4 * kGenKeys * 16);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, col = lane & 15, g = lane >> 4;
  const int kvh = blockIdx.y, z = blockIdx.z;
  const bool reporter = tid == 0;

  // ---- the sequence and this tile's rows ----
  Seq q;
  uint64_t path = 0;
  int64_t r0;
  if constexpr (TREE) {
    const int per = (A.nodes * A.G + kGenRows - 1) / kGenRows;
    const int s = blockIdx.x / per;
    r0 = static_cast<int64_t>(blockIdx.x - s * per) * kGenRows;
    q = tree_seq(A, s, reporter, &path);
  } else {
    const int s = find_seq(A, blockIdx.x, kGenRows);
    r0 = (blockIdx.x - tile_start(A, s, kGenRows)) * kGenRows;
    q = packed_seq(A, s, reporter);
  }
  const int64_t rows = static_cast<int64_t>(q.n) * A.G;
  if (q.n == 0 || r0 >= rows) return;
  const int32_t left = static_cast<int32_t>(rows - r0 < kGenRows ? rows - r0 : kGenRows);  // rows of the tile
  const int t_first = uniform(static_cast<int32_t>(r0 / A.G));
  const int h_first = uniform(static_cast<int32_t>(r0 - static_cast<int64_t>(t_first) * A.G));
  const int32_t r = wave * 16 + col;
  const bool row_ok = r < left;
  const int32_t rh = h_first + (row_ok ? r : 0);
  const int t = t_first + rh / A.G;   // this lane's token
  const int head = kvh * A.G + rh % A.G;
  const int t_last = t_first + (h_first + left - 1) / A.G;
  uint64_t my_path = 0;
  if constexpr (TREE)
    my_path = (static_cast<uint64_t>(__shfl(static_cast<uint32_t>(path >> 32), t, 64)) << 32) |
              static_cast<uint32_t>(__shfl(static_cast<uint32_t>(path), t, 64));

  // ---- this split's keys ----
  const int32_t n_keys = TREE ? q.ctx + q.n : q.ctx + t_last + 1;  // both lengths are below 2^30
  const int32_t tiles = (n_keys + kGenKeys - 1) / kGenKeys;
  const int32_t per_split = (tiles + A.n_split - 1) / A.n_split;
  const int32_t tile_lo = z * per_split, tile_hi = min(tile_lo + per_split, tiles);
  const int32_t clear = TREE ? q.ctx : q.ctx + t_first + 1;        // keys every row of the tile attends

  // ---- Q operand ----
  float qf[QF];
  {
    const char* qp = static_cast<const char*>(A.q) + ((q.row0 + t) * A.q_stride + static_cast<int64_t>(head) * D) * ES;
#pragma unroll
    for (int s = 0; s < QF; s += 4) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(qp + (s * 4 + 4 * g) * ES);
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[s + i] = v[i];
    }
  }
  f32x4_t O[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) O[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;  // l: this lane's part of the sum

  // ---- tiles through registers: vector i of this thread belongs to key
  // kr0 + i KSTEP of a tile.  Page ids are read two tiles ahead, rows one ----
  constexpr int NV = kGenKeys * Sh::VPR / kGenThreads, KSTEP = kGenThreads / Sh::VPR;
  const int kr0 = tid / Sh::VPR, w = tid % Sh::VPR;
  int32_t page[NV], off[NV];
  uint4 kreg[NV], vreg[NV];
  auto read_ids = [&](int32_t kt) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t j = min(kt * kGenKeys + kr0 + i * KSTEP, q.ctx - 1);
      page[i] = off[i] = 0;
      if (j >= 0) {
        const int32_t e = static_cast<int32_t>(static_cast<uint32_t>(j) / static_cast<uint32_t>(A.page));
        off[i] = j - e * A.page;
        page[i] = A.block_table[static_cast<size_t>(q.index) * A.max_pages + e];
      }
    }
  };
  auto read_rows = [&](int32_t kt) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int32_t j = min(kt * kGenKeys + kr0 + i * KSTEP, n_keys - 1);  // past the last: the last, which no row attends there
      const char *kp, *vp;
      if (j < q.ctx) {
        int32_t pg = page[i];
        if (pg < 0 || pg >= A.n_pages) {
          report_error(A.dev_err, GDN_DEV_BAD_PAGE);
          pg = 0;
        }
        const size_t at = ((static_cast<size_t>(pg) * A.Hk + kvh) * A.page + off[i]) * static_cast<size_t>(D) * ES;
        kp = static_cast<const char*>(A.k_cache) + at;
        vp = static_cast<const char*>(A.v_cache) + at;
      } else {
        const int64_t row = q.row0 + (j - q.ctx), head_at = static_cast<int64_t>(kvh) * D;
        kp = static_cast<const char*>(A.k) + (row * A.k_stride + head_at) * ES;
        vp = static_cast<const char*>(A.v) + (row * A.v_stride + head_at) * ES;
      }
      kreg[i] = *reinterpret_cast<const uint4*>(kp + 16 * w);
      vreg[i] = *reinterpret_cast<const uint4*>(vp + 16 * w);
    }
  };
  if (tile_lo < tile_hi) {
    read_ids(tile_lo);
    read_rows(tile_lo);
    read_ids(tile_lo + 1);
  }

  for (int32_t kt = tile_lo; kt < tile_hi; ++kt) {
    const int32_t key0 = kt * kGenKeys;
    const bool masked = key0 + kGenKeys > clear;
    lds_barrier();
    if (masked && tid == 0) *bad_keys = 0;
    if (masked) lds_barrier();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int kr = kr0 + i * KSTEP;
      if (masked && any_nonfinite<false>(vreg[i])) atomicOr(bad_keys, 1u << kr);
      *reinterpret_cast<uint4*>(Ks + kr * LD + w * Sh::VEC) = kreg[i];
      *reinterpret_cast<uint4*>(Vs + kr * LD + w * Sh::VEC) = vreg[i];
    }
    if (kt + 1 < tile_hi) {
      read_rows(kt + 1);
      read_ids(kt + 2);
    }
    lds_barrier();
    // Values that are not finite must not reach rows that do not attend their
    // key (0 x inf is NaN): such V rows leave the product and are added below.
    uint32_t bad = 0;
    if (masked) {
      bad = *bad_keys;
      if (bad) {
        for (int e = tid; e < kGenKeys * Sh::VPR; e += kGenThreads)
          if ((bad >> (e / Sh::VPR)) & 1u)
            *reinterpret_cast<uint4*>(Vs + (e / Sh::VPR) * LD + (e % Sh::VPR) * Sh::VEC) = make_uint4(0, 0, 0, 0);
        lds_barrier();
      }
    }
    // ---- logits, keys 16 kt2 + 4 g + i ----
    f32x4_t x[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < QF; s += 4) {
      const f32x4_t k0 = *reinterpret_cast<const f32x4_t*>(Ks + col * LD + s * 4 + 4 * g);
      const f32x4_t k1 = *reinterpret_cast<const f32x4_t*>(Ks + (16 + col) * LD + s * 4 + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[0] = mfma_f32(k0[i], qf[s + i], x[0]);
        x[1] = mfma_f32(k1[i], qf[s + i], x[1]);
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bool seen = true;
        if (masked) {
          const int32_t own = key0 + 16 * k2 + 4 * g + i - q.ctx;
          if constexpr (TREE) seen = own < 0 || (own < q.n && ((my_path >> own) & 1ull));
          else seen = own <= t;
        }
        x[k2][i] = seen ? x[k2][i] * A.scale_log2 : -INFINITY;
        mx = fmaxf(mx, x[k2][i]);
      }
    mx = quarter_max(mx);
    const float m_new = fmaxf(m, mx);
    const float ref = m_new == -INFINITY ? 0.f : m_new;  // no key seen yet: all weights 2^-inf = 0
    const float scale = __builtin_amdgcn_exp2f(m - ref);
    m = m_new;
    l *= scale;
    f32x4_t P[2];
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        P[k2][i] = __builtin_amdgcn_exp2f(x[k2][i] - ref);
        l += P[k2][i];
      }
    if (__any(scale != 1.f)) {
#pragma unroll
      for (int i = 0; i < NT; ++i) O[i] *= scale;
    }
    // ---- O^T += V^T P^T; the contraction runs over keys 4 g + i of both halves ----
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int dt = 0; dt < NT; dt += 4) {
          const f32x4_t v = *reinterpret_cast<const f32x4_t*>(Vs + (16 * k2 + 4 * g + i) * LD + 16 * dt + 4 * col);
#pragma unroll
          for (int e = 0; e < 4; ++e) O[dt + e] = mfma_f32(v[e], P[k2][i], O[dt + e]);
        }
    if (bad) {  // same for the whole workgroup
      float* pw = Ps + wave * kGenKeys * 16;
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
        for (int i = 0; i < 4; ++i) pw[(16 * k2 + 4 * g + i) * 16 + col] = P[k2][i];
      lds_barrier();
      for (uint32_t left = bad; left != 0; left &= left - 1) {
        const int kr = __builtin_ctz(left);
        const int32_t j = key0 + kr, own = j - q.ctx;
        bool seen;
        if constexpr (TREE) seen = own < 0 || (own < q.n && ((my_path >> own) & 1ull));
        else seen = own <= t;
        if (!seen) continue;  // also keys past the last
        const char* vr = key_row<ES>(A, q, A.v_cache, A.v, A.v_stride, kvh, j);
        const float p = pw[kr * 16 + col];
#pragma unroll
        for (int dt = 0; dt < NT; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[dt][i] += p * load_in<false>(vr, 64 * (dt / 4) + 16 * g + 4 * i + dt % 4);
      }
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  if (!row_ok) return;
  const size_t orow = static_cast<size_t>(q.row0 + t) * A.Hq + head;
  auto write = [&](float* to, float by) {
#pragma unroll
    for (int dt = 0; dt < NT; dt += 4)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4_t*>(to + 16 * dt + 16 * g + 4 * i) =
            f32x4_t{O[dt][i], O[dt + 1][i], O[dt + 2][i], O[dt + 3][i]} * by;
  };
  if (A.n_split == 1) {
    write(static_cast<float*>(A.o) + orow * D, 1.0f / l);
  } else {
    const size_t part = orow * A.n_split + z;
    float* ml = A.part + static_cast<size_t>(A.n_tokens) * A.Hq * A.n_split * D;
    if (g == 0) {
      ml[part * 2] = m;
      ml[part * 2 + 1] = l;
    }
    if (tile_lo < tile_hi) write(A.part + part * D, 1.0f);
  }
}

// Joins the splits of a row: weights 2^(m_z - max m).  A wave takes one row:
// D / 4 lanes hold its elements, 256 / D groups of them every 256 / D-th split.
// A split that saw no key (its m is -inf and its sum 0) wrote no sums and is
// left out.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void attn_combine_kernel(AttnArgs A) {
  constexpr int LPR = D / 4, NG = kWave / LPR;
  const int lane = threadIdx.x & (kWave - 1), c = (lane % LPR) * 4, g = lane / LPR;
  const int64_t orow = static_cast<int64_t>(blockIdx.x) * 4 + uniform(static_cast<int32_t>(threadIdx.x / kWave));
  if (orow >= static_cast<int64_t>(A.n_tokens) * A.Hq) return;
  const int32_t tok = static_cast<int32_t>(orow / A.Hq);
  // rows that no workgroup computed (a refused sequence, padding) stay as they are
  if (A.nodes > 0) {
    uint64_t path;
    const int s = tok / A.nodes;
    if (tok - s * A.nodes >= tree_seq(A, s, false, &path).n) return;
  } else {
    // the last sequence that does not begin after the token
    const int s = last_seq(A, [&](int32_t t0, int) { return t0 <= tok; });
    const Seq q = packed_seq(A, s, false);
    if (q.n == 0 || tok < q.row0 || tok >= q.row0 + q.n) return;
  }
  const float* ml = A.part + static_cast<size_t>(A.n_tokens) * A.Hq * A.n_split * D + static_cast<size_t>(orow) * A.n_split * 2;
  const float* sums = A.part + static_cast<size_t>(orow) * A.n_split * D + c;
  static_assert(kMaxSplits <= kWave, "a lane per split");
  const bool mine = lane < A.n_split;
  const float mz = mine ? ml[2 * lane] : -INFINITY, lz = mine ? ml[2 * lane + 1] : 0.f;
  float m = mz;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
  const float ref = m == -INFINITY ? 0.f : m;
  const float weight = mz == -INFINITY && lz == 0.f ? 0.f : __builtin_amdgcn_exp2f(mz - ref);
  const float l = group_sum<kWave>(weight * lz);
  const uint64_t on = __ballot(!(mz == -INFINITY && lz == 0.f));
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int z0 = 0; z0 < A.n_split; z0 += NG) {  // the same turns in every lane: the weights come from other lanes
    const int z = min(z0 + g, A.n_split - 1);
    const f32x4_t x = load4(sums + static_cast<size_t>(z) * D);
    const float w = __shfl(weight, z, kWave);
    const bool seen = z0 + g < A.n_split && ((on >> z) & 1ull);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += seen ? w * x[e] : 0.f;
  }
#pragma unroll
  for (int d = LPR; d < kWave; d <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], d, kWave);
  if (g != 0) return;
  sum *= 1.0f / l;
  const size_t at = static_cast<size_t>(orow) * D + c;
  if constexpr (BF16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.o) + at) =
        make_uint2(pack2_bf16(sum[0], sum[1]), pack2_bf16(sum[2], sum[3]));
  else
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(A.o) + at) = sum;
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
namespace {

// Row tiles (per KV head) of a call.
int64_t row_tiles(int64_t tokens, int n_seqs, int G, int nodes, int bm) {
  if (nodes > 0) return static_cast<int64_t>(n_seqs) * ((static_cast<int64_t>(nodes) * G + bm - 1) / bm);
  return tokens * G / bm + n_seqs;
}

}  // namespace

// Parts of the key axis that a row tile is split into.  fp32: up to four
// workgroups per CU (that is what fits at d 64 and hides one's softmax behind the
// others' products: 2048 tokens of 8 heads 134 us with two, 100 us with four, 84 us
// with eight, where 256 tokens then take 19 us instead of 12).  bf16: one per CU
// (LDS holds one at d 128 and 256), none of fewer than 128 keys: parts are written
// and read once more, and with two per CU 512 tokens of 24 heads on 4, d 256, took
// 64 us instead of 40, 256 behind 8192 cached ones 102 instead of 77.  At d 64 two
// workgroups fit and the last part may begin beside others (4096 tokens 88 us in
// 130 workgroups, 64 us in 260).  The parts are those of rows that fill their block
// table: shorter ones leave parts empty.  fp32 trees take the prompts' rule, which
// was measured on prompts alone.
int attn_splits(int64_t tokens, int n_seqs, int Hk, int G, int D, int nodes, bool bf16, int64_t keys) {
  if (bf16 && nodes > 0) return 1;
  const int64_t wgs = row_tiles(tokens, n_seqs, G, nodes, bf16 && nodes == 0 ? kPromptRows : kGenRows) * Hk;
  if (wgs <= 0) return 1;
  const int64_t want = !bf16 ? 1024 / wgs : (D == 64 ? (255 + wgs) / wgs : 256 / wgs);
  const int64_t least = bf16 ? 128 : kGenKeys, parts = keys / least + (keys % least != 0);
  return static_cast<int>(std::max<int64_t>(std::min({want, parts, static_cast<int64_t>(kMaxSplits)}), 1));
}

size_t attn_part_bytes(int64_t tokens, int n_seqs, int Hk, int G, int D, int nodes, bool bf16) {
  if (bf16 && nodes > 0) return tree_bf16_part_bytes(n_seqs, Hk, G, D, nodes);
  const int n_split = attn_splits(tokens, n_seqs, Hk, G, D, nodes, bf16, INT64_MAX);
  return n_split <= 1 ? 0 : static_cast<size_t>(tokens) * Hk * G * n_split * (D + 2) * sizeof(float);
}

template <int D, bool BF16>
static int launch_attn_t(const AttnArgs& a, hipStream_t s) {
  const int64_t tiles = row_tiles(a.n_tokens, a.n_seqs, a.G, a.nodes, BF16 ? kPromptRows : kGenRows);
  if constexpr (BF16) {
    if (a.nodes > 0) return launch_tree_bf16(a, s);
    const int e = launch_prompt_bf16(a, tiles, s);
    if (e != 0) return e;
  } else {
    if (!grid_fits(tiles, kGenThreads)) return static_cast<int>(hipErrorInvalidValue);
    const dim3 grid(static_cast<unsigned>(tiles), a.Hk, a.n_split);
    const size_t lds = 2 * GenShape<D>::TILE_BYTES + 4 * kGenKeys * 16 * sizeof(float) + 16;
    if (a.nodes > 0) hipLaunchKernelGGL((attn_f32_kernel<D, true>), grid, dim3(kGenThreads), lds, s, a);
    else hipLaunchKernelGGL((attn_f32_kernel<D, false>), grid, dim3(kGenThreads), lds, s, a);
  }
  int e = static_cast<int>(hipGetLastError());
  if (e == 0 && a.n_split > 1) {
    const int64_t rows = static_cast<int64_t>(a.n_tokens) * a.Hq;  // few: a call of many rows is not split
    hipLaunchKernelGGL((attn_combine_kernel<D, BF16>), dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, s, a);
    e = static_cast<int>(hipGetLastError());
  }
  return e;
}

int launch_attn(const AttnArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (a.D) {
    case 64: return bf16 ? launch_attn_t<64, true>(a, s) : launch_attn_t<64, false>(a, s);
    case 128: return bf16 ? launch_attn_t<128, true>(a, s) : launch_attn_t<128, false>(a, s);
    case 256: return bf16 ? launch_attn_t<256, true>(a, s) : launch_attn_t<256, false>(a, s);
    default: return static_cast<int>(hipErrorInvalidValue);
  }
}

}  // namespace gdn
