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
// with (m, l), and combine_kernel joins them in a fixed order.
#include "gdn_attn_device.h"

namespace gdn {

namespace {

__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
}  // namespace

// ---------------------------------------------------------------------------
// fp32: 64 rows x 32 keys per step, four waves of 16 rows each, K and V rows
// staged through LDS.  16x16x4 matrix instructions: lane l holds rows (keys)
// 4 (l / 16) + i of column (query row) l % 16.  (bf16: gdn_flash.hip.)
// ---------------------------------------------------------------------------
constexpr int kGenRows = 64, kGenKeys = 32, kGenThreads = 256;

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
  const int64_t r = r0 + wave * 16 + col;
  const bool row_ok = r < rows;
  const int t = static_cast<int>((row_ok ? r : r0) / A.G);   // this lane's token
  const int head = kvh * A.G + static_cast<int>((row_ok ? r : r0) % A.G);
  const int t_first = static_cast<int>(r0 / A.G);
  const int64_t r_last = r0 + kGenRows < rows ? r0 + kGenRows - 1 : rows - 1;
  const int t_last = static_cast<int>(r_last / A.G);
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
    for (int s = 0; s < QF; ++s) qf[s] = *reinterpret_cast<const float*>(qp + (s * 4 + g) * 4);
  }
  f32x4_t O[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) O[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;  // l: this lane's part of the sum

  for (int32_t kt = tile_lo; kt < tile_hi; ++kt) {
    const int32_t key0 = kt * kGenKeys;
    const bool masked = key0 + kGenKeys > clear;
    __syncthreads();
    if (masked && tid == 0) *bad_keys = 0;
    if (masked) __syncthreads();
    for (int e = tid; e < kGenKeys * Sh::VPR; e += kGenThreads) {
      const int kr = e / Sh::VPR, w = e % Sh::VPR;
      const int32_t j = key0 + kr;
      uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
      if (j < n_keys) {
        kv = *reinterpret_cast<const uint4*>(key_row<ES>(A, q, A.k_cache, A.k, A.k_stride, kvh, j) + 16 * w);
        vv = *reinterpret_cast<const uint4*>(key_row<ES>(A, q, A.v_cache, A.v, A.v_stride, kvh, j) + 16 * w);
      }
      if (masked && any_nonfinite<false>(vv)) atomicOr(bad_keys, 1u << kr);
      *reinterpret_cast<uint4*>(Ks + kr * LD + w * Sh::VEC) = kv;
      *reinterpret_cast<uint4*>(Vs + kr * LD + w * Sh::VEC) = vv;
    }
    __syncthreads();
    // Values that are not finite must not reach rows that do not attend their
    // key (0 x inf is NaN): such V rows leave the product and are added below.
    uint32_t bad = 0;
    if (masked) {
      bad = *bad_keys;
      if (bad) {
        for (int e = tid; e < kGenKeys * Sh::VPR; e += kGenThreads)
          if ((bad >> (e / Sh::VPR)) & 1u)
            *reinterpret_cast<uint4*>(Vs + (e / Sh::VPR) * LD + (e % Sh::VPR) * Sh::VEC) = make_uint4(0, 0, 0, 0);
        __syncthreads();
      }
    }
    // ---- logits, keys 16 kt2 + 4 g + i ----
    float x[2][4];
    float mx = -INFINITY;
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      f32x4_t c = {0.f, 0.f, 0.f, 0.f};
      const E* kr = Ks + (16 * k2 + col) * LD;
#pragma unroll
      for (int s = 0; s < QF; ++s) c = mfma_f32(kr[s * 4 + g], qf[s], c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t j = key0 + 16 * k2 + 4 * g + i;
        bool seen = true;
        if (masked) {
          const int32_t own = j - q.ctx;
          if constexpr (TREE) seen = own < 0 || (own < q.n && ((my_path >> own) & 1ull));
          else seen = own <= t;
        }
        x[k2][i] = seen ? c[i] * A.scale_log2 : -INFINITY;
        mx = fmaxf(mx, x[k2][i]);
      }
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
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
#pragma unroll
    for (int i = 0; i < NT; ++i) O[i] *= scale;
    // ---- O^T += V^T P^T; the contraction runs over keys 4 g + i of both halves ----
#pragma unroll
    for (int dt = 0; dt < NT; ++dt) {
      const E* vc = Vs + 4 * g * LD + 16 * dt + col;
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[dt] = mfma_f32(vc[(16 * k2 + i) * LD], P[k2][i], O[dt]);
    }
    if (bad) {  // same for the whole workgroup
      float* pw = Ps + wave * kGenKeys * 16;
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
        for (int i = 0; i < 4; ++i) pw[(16 * k2 + 4 * g + i) * 16 + col] = P[k2][i];
      __syncthreads();
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
          for (int i = 0; i < 4; ++i) O[dt][i] += p * load_in<false>(vr, 16 * dt + 4 * g + i);
      }
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  if (!row_ok) return;
  const size_t orow = static_cast<size_t>(q.row0 + t) * A.Hq + head;
  if (A.n_split == 1) {
    const float inv = 1.0f / l;
#pragma unroll
    for (int dt = 0; dt < NT; ++dt)
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(A.o) + orow * D + 16 * dt + 4 * g) = O[dt] * inv;
  } else {
    const size_t part = orow * A.n_split + z;
    float* ml = A.part + static_cast<size_t>(A.n_tokens) * A.Hq * A.n_split * D;
    if (g == 0) {
      ml[part * 2] = m;
      ml[part * 2 + 1] = l;
    }
    if (tile_lo < tile_hi) {
#pragma unroll
      for (int dt = 0; dt < NT; ++dt)
        *reinterpret_cast<f32x4_t*>(A.part + part * D + 16 * dt + 4 * g) = O[dt];
    }
  }
}

// Joins the splits of a row: weights 2^(m_z - max m), in the order of z.  D/4
// lanes per row.  A split that saw no key (its m is -inf and its sum 0) wrote
// no sums and is left out.
template <int D, bool BF16>
__global__ __launch_bounds__(256) void attn_combine_kernel(AttnArgs A) {
  constexpr int LPR = D / 4, RPW = 256 / LPR;
  const int c = (threadIdx.x % LPR) * 4;
  const int64_t orow = static_cast<int64_t>(blockIdx.x) * RPW + threadIdx.x / LPR;
  const int64_t total = static_cast<int64_t>(A.n_tokens) * A.Hq;
  const int64_t tok = (orow < total ? orow : total - 1) / A.Hq;
  // rows that no workgroup computed (a refused sequence, padding) stay as they are
  bool live = orow < total;
  if (A.nodes > 0) {
    // the wave's rows may belong to several trees: each is checked by the whole wave
    const int s = static_cast<int>(tok / A.nodes);
    const int node = static_cast<int>(tok - static_cast<int64_t>(s) * A.nodes);
    uint64_t todo = __ballot(true);
    bool ok = false;
    while (todo != 0) {
      const int leader = __builtin_ctzll(todo);
      const int sl = __builtin_amdgcn_readlane(s, leader);
      uint64_t path;
      const Seq q = tree_seq(A, sl, false, &path);
      if (s == sl) ok = node < q.n;
      todo &= ~__ballot(s == sl);
    }
    live &= ok;
  } else {
    int lo = 0, hi = A.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (A.cu_seqlens[mid] <= tok) lo = mid;
      else hi = mid;
    }
    const Seq q = packed_seq(A, lo, false);
    live &= q.n > 0 && tok >= q.row0 && tok < q.row0 + q.n;
  }
  if (!live) return;
  const float* ml = A.part + static_cast<size_t>(A.n_tokens) * A.Hq * A.n_split * D +
                    static_cast<size_t>(orow) * A.n_split * 2;
  float m = -INFINITY;
  for (int z = 0; z < A.n_split; ++z) m = fmaxf(m, ml[2 * z]);
  const float ref = m == -INFINITY ? 0.f : m;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  for (int z = 0; z < A.n_split; ++z) {
    const float mz = ml[2 * z], lz = ml[2 * z + 1];
    if (mz == -INFINITY && lz == 0.f) continue;
    const float w = __builtin_amdgcn_exp2f(mz - ref);
    l += w * lz;
    sum += w * load4(A.part + (static_cast<size_t>(orow) * A.n_split + z) * D + c);
  }
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

int attn_splits(int64_t tokens, int n_seqs, int Hk, int G, int nodes, bool bf16) {
  if (bf16 && nodes > 0) return 1;
  // two workgroups per CU, and at most 64 parts to join
  const int64_t wgs = row_tiles(tokens, n_seqs, G, nodes, bf16 && nodes == 0 ? kFlashRows : kGenRows) * Hk;
  const int64_t want = wgs > 0 ? 512 / wgs : 1;
  return static_cast<int>(want < 1 ? 1 : (want > 64 ? 64 : want));
}

size_t attn_part_bytes(int64_t tokens, int n_seqs, int Hk, int G, int D, int nodes, bool bf16) {
  if (bf16 && nodes > 0) return flash_tree_part_bytes(n_seqs, Hk, G, D, nodes);
  const int n_split = attn_splits(tokens, n_seqs, Hk, G, nodes, bf16);
  return n_split <= 1 ? 0 : static_cast<size_t>(tokens) * Hk * G * n_split * (D + 2) * sizeof(float);
}

template <int D, bool BF16>
static int launch_attn_t(const AttnArgs& a, hipStream_t s) {
  const int64_t tiles = row_tiles(a.n_tokens, a.n_seqs, a.G, a.nodes, BF16 ? kFlashRows : kGenRows);
  if (tiles * a.Hk > INT32_MAX) return static_cast<int>(hipErrorInvalidValue);
  if constexpr (BF16) {
    if (a.nodes > 0) return launch_flash_tree(a, s);
    const int e = launch_flash_prefill(a, tiles, s);
    if (e != 0) return e;
  } else {
    const dim3 grid(static_cast<unsigned>(tiles), a.Hk, a.n_split);
    const size_t lds = 2 * GenShape<D>::TILE_BYTES + 4 * kGenKeys * 16 * sizeof(float) + 16;
    if (a.nodes > 0) hipLaunchKernelGGL((attn_f32_kernel<D, true>), grid, dim3(kGenThreads), lds, s, a);
    else hipLaunchKernelGGL((attn_f32_kernel<D, false>), grid, dim3(kGenThreads), lds, s, a);
  }
  int e = static_cast<int>(hipGetLastError());
  if (e == 0 && a.n_split > 1) {
    const int64_t rows = static_cast<int64_t>(a.n_tokens) * a.Hq, per = 256 / (D / 4);
    hipLaunchKernelGGL((attn_combine_kernel<D, BF16>), dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(256),
                       0, s, a);
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
