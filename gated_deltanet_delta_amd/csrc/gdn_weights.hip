// Attention weights that the newest tokens give to a row's cached tokens, for gfx950.
//
//   z = scale q . k_j,  lse = log sum over j <= last of e^z,  score[j] += sum over queries of e^(z - lse)
//
// over all queries (token t < n, head h) that attend j: last = kv_len - n + t.  The
// weights of one key are a column of the softmax, whose normaliser is known only once
// a query has seen all its keys, so there are three steps: maximum and sum of every
// (query, part of the keys); their join to one lse per query; the sums per key.
// V does not enter, so K is all that has to be read, and K is read once: at most 32 rows
// (queries of one KV head) store their logits for the last step, 4 bytes each
// beside a key's 2 D or 4 D; more rows compute them again.
//
// K goes from memory to registers as it lies (each lane 16 bytes of one key per step,
// the A or B operand of a 32 x 32 matrix instruction) and Q comes from LDS, where it
// lies in the order of the operands.  A wave owns its keys and walks over the rows,
// so waves share nothing but Q.  In base 2: z log2(e) is what is stored and compared.
#include "gdn_attn_device.h"

namespace gdn {

namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 16 bytes of an operand's row per lane and step: 8 bf16 or 4 fp32 elements, lanes
// l and l + 32 those of one row.  The two operands pair the same elements, so their
// order along the head is as they lie in memory.
template <bool BF16>
__device__ __forceinline__ f32x16_t mfma_step(uint4 a, uint4 b, f32x16_t c) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  } else {
    const f32x4_t x = __builtin_bit_cast(f32x4_t, a), y = __builtin_bit_cast(f32x4_t, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[i], y[i], c, 0, 0, 0);
    return c;
  }
}

// max / sum over the two lanes l and l ^ 32
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sizes of a call, the same on the host and on the device.
struct WeightPlan {
  int32_t R, row_tiles, Rp;    // rows of a KV head (n G), tiles of 32 of them, rows in whole tiles
  int32_t part_keys, parts;    // keys of a part, parts of a row of `width` tokens
  int32_t W;                   // row length of the logits or sums: width in whole tiles of keys
  bool stored;                 // logits are stored
  size_t lse, keys, total;     // byte offsets of lse [batch][Hk][Rp] and of the logits [batch][Hk][R][W] or
                               // the heads' sums [batch][Hk][W]; (max, sum) [batch][Hk][parts][Rp] is at 0
};

constexpr int kTileKeys = 32;
// Few rows: keys of a wave, and waves of a workgroup
constexpr int kStoredKeys = 64, kStoredWaves = 4;
// Many rows: 32-key blocks that a wave holds in registers (a Q operand then serves as many
// instructions), tiles that it takes one after the other, waves of a workgroup
constexpr int many_blocks(int D, bool bf16) { return D * (bf16 ? 2 : 4) <= 512 ? 2 : 1; }
constexpr int kManyTiles = 2, kManyWaves = 8;
// Row tiles whose Q lies in LDS at a time: 128 KB
constexpr int many_row_tiles(int D, bool bf16) { return (128 << 10) / (32 * D * (bf16 ? 2 : 4)); }

__host__ __device__ inline size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

WeightPlan weight_plan(int32_t batch, int32_t n, int32_t width, int Hk, int G, int D, bool bf16) {
  WeightPlan p{};
  p.R = n * G;
  p.row_tiles = (p.R + 31) / 32;
  p.Rp = p.row_tiles * 32;
  p.stored = p.row_tiles == 1;
  p.part_keys = p.stored ? kStoredKeys : kTileKeys * many_blocks(D, bf16);
  p.parts = static_cast<int32_t>((static_cast<int64_t>(width) + p.part_keys - 1) / p.part_keys);
  p.W = static_cast<int32_t>(round_up(width, 64));
  const size_t units = static_cast<size_t>(batch) * Hk;
  p.lse = round_up(units * p.parts * p.Rp * sizeof(float2), 256);
  p.keys = p.lse + round_up(units * p.Rp * sizeof(float), 256);
  p.total = p.keys + units * (p.stored ? p.R : 1) * p.W * sizeof(float);
  return p;
}

// Row i: its queries (0: idle or refused) and cached tokens.
struct WeightRow {
  int32_t n, kv;
};
__device__ __forceinline__ WeightRow weight_row(const WeightArgs& A, int i, bool report) {
  WeightRow r{A.n_row ? A.n_row[i] : A.n, A.kv_len[i]};
  if (r.n < 0 || r.n > A.n) {
    if (report) report_error(A.dev_err, GDN_DEV_BAD_K);
    r.n = 0;
  } else if (r.n > 0) {
    const int32_t have = A.have_len ? A.have_len[i] : 0;
    if (r.kv < r.n || r.kv > A.width || r.kv > static_cast<int64_t>(A.max_pages) * A.page || have < 0 || have > r.kv) {
      if (report) report_error(A.dev_err, GDN_DEV_BAD_LENGTH);
      r.n = 0;
    }
  }
  return WeightRow{uniform(r.n), uniform(r.kv)};
}

// Q of row tiles [t0, t0 + tiles) of KV head h of row i, in the order of the operands:
// [tile][step][lane] of 16 bytes.  Rows past the last are zeros.
template <int D, bool BF16, int THREADS>
__device__ __forceinline__ void load_q(const WeightArgs& A, int i, int h, int32_t rows, int t0, int tiles, uint4* lds) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32;
  for (int e = threadIdx.x; e < tiles * STEPS * 64; e += THREADS) {
    const int lane = e % 64, s = e / 64 % STEPS, r = (t0 + e / 64 / STEPS) * 32 + lane % 32;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const int t = r / A.G;
      const char* q = static_cast<const char*>(A.q) +
                      ((static_cast<int64_t>(i) * A.n + t) * A.q_stride + static_cast<int64_t>(h * A.G + r - t * A.G) * D) * ES;
      v = *reinterpret_cast<const uint4*>(q + (2 * s + lane / 32) * 16);
    }
    lds[e] = v;
  }
}

// This lane's 16-byte pieces of the K rows of 32 keys from key0 on, one key per pair of
// lanes; keys past the last repeat it (and are masked).
template <int D, bool BF16>
__device__ __forceinline__ void load_k(const WeightArgs& A, int i, int h, int32_t key0, int32_t kv,
                                       uint4 (&k)[D * (BF16 ? 2 : 4) / 32]) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32;
  const int lane = threadIdx.x & 63;
  const int32_t j = min(key0 + lane % 32, kv - 1);
  const int32_t e = j / A.page, off = j - e * A.page;
  int32_t page = A.block_table[static_cast<size_t>(i) * A.max_pages + e];
  if (page < 0 || page >= A.n_pages) {
    report_error(A.dev_err, GDN_DEV_BAD_PAGE);
    page = 0;
  }
  const char* p = static_cast<const char*>(A.k_cache) +
                  ((static_cast<size_t>(page) * A.Hk + h) * A.page + off) * (static_cast<size_t>(D) * ES) + lane / 32 * 16;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) k[s] = *reinterpret_cast<const uint4*>(p + s * 32);
}

// Element e of a 32 x 32 result is row 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32.
__device__ __forceinline__ int result_row(int e) { return 8 * (e / 4) + 4 * ((threadIdx.x & 63) / 32) + e % 4; }

}  // namespace

// Few rows: logits of a wave's keys (stored), maximum and sum of each row over them.
template <int D, bool BF16>
__global__ __launch_bounds__(64 * kStoredWaves) void weights_stored_kernel(WeightArgs A, WeightPlan P) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32;
  __shared__ uint4 qs[STEPS * 64];
  const int h = blockIdx.y, i = blockIdx.z, lane = threadIdx.x & 63;
  const WeightRow w = weight_row(A, i, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  if (w.n == 0 || static_cast<int64_t>(blockIdx.x) * kStoredWaves * kStoredKeys >= w.kv) return;
  load_q<D, BF16, 64 * kStoredWaves>(A, i, h, w.n * A.G, 0, 1, qs);
  __syncthreads();
  const int part = blockIdx.x * kStoredWaves + uniform(static_cast<int32_t>(threadIdx.x / 64));
  const int32_t lo = part * kStoredKeys, hi = min(lo + kStoredKeys, w.kv);
  if (lo >= hi) return;
  const int row = lane % 32;
  const int32_t last = w.kv - w.n + row / A.G;  // this row's last key
  const size_t unit = static_cast<size_t>(i) * A.Hk + h;
  float* z = reinterpret_cast<float*>(static_cast<char*>(A.workspace) + P.keys) + (unit * P.R + row) * P.W;
  float m = -INFINITY, l = 0.f;
  for (int32_t key0 = lo; key0 < hi; key0 += kTileKeys) {
    uint4 k[STEPS];
    load_k<D, BF16>(A, i, h, key0, w.kv, k);
    f32x16_t S;
#pragma unroll
    for (int e = 0; e < 16; ++e) S[e] = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) S = mfma_step<BF16>(k[s], qs[s * 64 + lane], S);
    float mx = m;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      S[e] = key0 + result_row(e) <= last ? S[e] * A.scale_log2 : -INFINITY;
      mx = fmaxf(mx, S[e]);
    }
    const float ref = mx == -INFINITY ? 0.f : mx;
    l *= __builtin_amdgcn_exp2f(m - ref);
    m = mx;
#pragma unroll
    for (int e = 0; e < 16; ++e) l += __builtin_amdgcn_exp2f(S[e] - ref);
    if (row < P.R) {
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<f32x4_t*>(z + key0 + result_row(e)) = f32x4_t{S[e], S[e + 1], S[e + 2], S[e + 3]};
    }
  }
  // the halves' maxima differ
  const float both = half_max(m), ref = both == -INFINITY ? 0.f : both;
  l = half_sum(l * __builtin_amdgcn_exp2f(m - ref));
  if (lane < 32) static_cast<float2*>(A.workspace)[(unit * P.parts + part) * P.Rp + row] = make_float2(both, l);
}

// Many rows: maximum and sum of every row over each of a wave's tiles of keys.
template <int D, bool BF16>
__global__ __launch_bounds__(64 * kManyWaves, 2) void weights_stats_kernel(WeightArgs A, WeightPlan P) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32, KB = many_blocks(D, BF16), RT = many_row_tiles(D, BF16);
  extern __shared__ __align__(16) uint4 q_lds[];
  const int h = blockIdx.y, i = blockIdx.z, lane = threadIdx.x & 63;
  const int32_t wave = uniform(static_cast<int32_t>(threadIdx.x / 64));
  const WeightRow w = weight_row(A, i, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  if (w.n == 0 || static_cast<int64_t>(blockIdx.x) * kManyWaves * kManyTiles * KB * kTileKeys >= w.kv) return;
  const int32_t rows = w.n * A.G, tiles = (rows + 31) / 32;
  const size_t unit = static_cast<size_t>(i) * A.Hk + h;
  for (int t0 = 0; t0 < tiles; t0 += RT) {
    const int nt = min(RT, tiles - t0);
    if (t0 > 0) __syncthreads();
    load_q<D, BF16, 64 * kManyWaves>(A, i, h, rows, t0, nt, q_lds);
    __syncthreads();
    for (int c = 0; c < kManyTiles; ++c) {
      const int part = (blockIdx.x * kManyTiles + c) * kManyWaves + wave;
      const int32_t key0 = part * (KB * kTileKeys);
      if (key0 >= w.kv) break;
      uint4 k[KB][STEPS];
#pragma unroll
      for (int b = 0; b < KB; ++b) load_k<D, BF16>(A, i, h, key0 + b * kTileKeys, w.kv, k[b]);
      const bool masked = key0 + KB * kTileKeys > w.kv - w.n + 1;
      for (int t = 0; t < nt; ++t) {
        f32x16_t S[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) S[b][e] = 0.f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const uint4 q = q_lds[(t * STEPS + s) * 64 + lane];
#pragma unroll
          for (int b = 0; b < KB; ++b) S[b] = mfma_step<BF16>(k[b][s], q, S[b]);
        }
        const int row = (t0 + t) * 32 + lane % 32;
        if (masked) {
          const int32_t last = w.kv - w.n + row / A.G;
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) S[b][e] = key0 + b * kTileKeys + result_row(e) <= last ? S[b][e] : -INFINITY;
        }
        float m = -INFINITY;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) m = fmaxf(m, S[b][e]);
        m = half_max(m) * A.scale_log2;
        const float off = m == -INFINITY ? 0.f : -m;
        float l = 0.f;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) l += __builtin_amdgcn_exp2f(fmaf(S[b][e], A.scale_log2, off));
        l = half_sum(l);
        if (lane < 32) static_cast<float2*>(A.workspace)[(unit * P.parts + part) * P.Rp + row] = make_float2(m, l);
      }
    }
  }
}

// Joins the parts of 32 rows of a KV head, in a fixed order: log2 of the sum of 2^z.
// Rows past the last get +inf, which takes every weight to 0.
__global__ __launch_bounds__(256) void weights_join_kernel(WeightArgs A, WeightPlan P) {
  __shared__ float2 parts[8][32];
  const int i = blockIdx.z, h = blockIdx.y, lr = threadIdx.x % 32, g = threadIdx.x / 32, row = blockIdx.x * 32 + lr;
  const WeightRow w = weight_row(A, i, false);
  if (w.n == 0) return;
  const size_t unit = static_cast<size_t>(i) * A.Hk + h;
  const float2* ml = static_cast<const float2*>(A.workspace) + unit * P.parts * P.Rp + row;
  const bool live = row < w.n * A.G;
  const int count = live ? (w.kv + P.part_keys - 1) / P.part_keys : 0;
  float m = -INFINITY, l = 0.f;
  auto add = [&](float2 x) {
    const float mx = fmaxf(m, x.x), ref = mx == -INFINITY ? 0.f : mx;
    l = l * __builtin_amdgcn_exp2f(m - ref) + x.y * __builtin_amdgcn_exp2f(x.x - ref);
    m = mx;
  };
#pragma unroll 4
  for (int p = g; p < count; p += 8) add(ml[static_cast<size_t>(p) * P.Rp]);
  parts[g][lr] = make_float2(m, l);
  __syncthreads();
  if (g != 0) return;
  for (int o = 1; o < 8; ++o) add(parts[o][lr]);
  float* lse = reinterpret_cast<float*>(static_cast<char*>(A.workspace) + P.lse);
  lse[unit * P.Rp + row] = live ? m + __builtin_amdgcn_logf(l) : INFINITY;
}

// Few rows: the weights of one key from the stored logits, all heads.
__global__ __launch_bounds__(256) void weights_sum_kernel(WeightArgs A, WeightPlan P) {
  const int i = blockIdx.y;
  const WeightRow w = weight_row(A, i, false);
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (w.n == 0 || j >= w.kv) return;
  const char* ws = static_cast<const char*>(A.workspace);
  const float* lse = reinterpret_cast<const float*>(ws + P.lse) + static_cast<size_t>(i) * A.Hk * P.Rp;
  const float* z = reinterpret_cast<const float*>(ws + P.keys) + static_cast<size_t>(i) * A.Hk * P.R * P.W + j;
  float sum = 0.f;
  for (int h = 0; h < A.Hk; ++h)
    for (int t = 0; t < w.n; ++t) {
      const bool seen = j <= w.kv - w.n + t;
#pragma unroll 4
      for (int g = 0; g < A.G; ++g) {
        const int r = t * A.G + g;
        const float p = __builtin_amdgcn_exp2f(z[(static_cast<size_t>(h) * P.R + r) * P.W] - lse[h * P.Rp + r]);
        sum += seen ? p : 0.f;
      }
    }
  const size_t at = static_cast<size_t>(i) * A.width + j;
  const bool old = A.score_in && (!A.have_len || j < A.have_len[i]);
  A.score_out[at] = (old ? A.score_in[at] : 0.f) + sum;
}

// Many rows: each head's weights of a wave's keys, the logits computed again with the
// operands the other way round, so that a lane holds one key's logits.
template <int D, bool BF16>
__global__ __launch_bounds__(64 * kManyWaves, 2) void weights_keys_kernel(WeightArgs A, WeightPlan P) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32, KB = many_blocks(D, BF16), RT = many_row_tiles(D, BF16);
  extern __shared__ __align__(16) uint4 q_lds[];
  __shared__ __align__(16) float lse[RT * 32];
  const int h = blockIdx.y, i = blockIdx.z, lane = threadIdx.x & 63;
  const int32_t wave = uniform(static_cast<int32_t>(threadIdx.x / 64));
  const WeightRow w = weight_row(A, i, false);
  if (w.n == 0 || static_cast<int64_t>(blockIdx.x) * kManyWaves * kManyTiles * KB * kTileKeys >= w.kv) return;
  const int32_t rows = w.n * A.G, tiles = (rows + 31) / 32;
  const size_t unit = static_cast<size_t>(i) * A.Hk + h;
  float* out = reinterpret_cast<float*>(static_cast<char*>(A.workspace) + P.keys) + unit * P.W;
  const float* all = reinterpret_cast<const float*>(static_cast<const char*>(A.workspace) + P.lse) + unit * P.Rp;
  for (int t0 = 0; t0 < tiles; t0 += RT) {
    const int nt = min(RT, tiles - t0);
    if (t0 > 0) __syncthreads();
    load_q<D, BF16, 64 * kManyWaves>(A, i, h, rows, t0, nt, q_lds);
    for (int r = threadIdx.x; r < nt * 32; r += 64 * kManyWaves) lse[r] = all[t0 * 32 + r];
    __syncthreads();
    for (int c = 0; c < kManyTiles; ++c) {
      const int32_t key0 = ((blockIdx.x * kManyTiles + c) * kManyWaves + wave) * (KB * kTileKeys);
      if (key0 >= w.kv) break;
      uint4 k[KB][STEPS];
#pragma unroll
      for (int b = 0; b < KB; ++b) load_k<D, BF16>(A, i, h, key0 + b * kTileKeys, w.kv, k[b]);
      const bool masked = key0 + KB * kTileKeys > w.kv - w.n + 1;
      float sum[KB];
#pragma unroll
      for (int b = 0; b < KB; ++b) sum[b] = 0.f;
      for (int t = 0; t < nt; ++t) {
        f32x16_t S[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) S[b][e] = 0.f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const uint4 q = q_lds[(t * STEPS + s) * 64 + lane];
#pragma unroll
          for (int b = 0; b < KB; ++b) S[b] = mfma_step<BF16>(q, k[b][s], S[b]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int row = t * 32 + result_row(e);
          const float off = -lse[row];
          const int32_t last = masked ? w.kv - w.n + (t0 * 32 + row) / A.G : 0;
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            const float p = __builtin_amdgcn_exp2f(fmaf(S[b][e], A.scale_log2, off));
            sum[b] += !masked || key0 + b * kTileKeys + lane % 32 <= last ? p : 0.f;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const float total = half_sum(sum[b]);
        float* at = out + key0 + b * kTileKeys + lane;  // within W, whole pairs of tiles
        if (lane < 32) *at = t0 > 0 ? *at + total : total;
      }
    }
  }
}

// Many rows: the heads' sums of one key.
__global__ __launch_bounds__(256) void weights_heads_kernel(WeightArgs A, WeightPlan P) {
  const int i = blockIdx.y;
  const WeightRow w = weight_row(A, i, false);
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (w.n == 0 || j >= w.kv) return;
  const float* k = reinterpret_cast<const float*>(static_cast<const char*>(A.workspace) + P.keys) +
                   static_cast<size_t>(i) * A.Hk * P.W + j;
  float sum = 0.f;
#pragma unroll 4
  for (int h = 0; h < A.Hk; ++h) sum += k[static_cast<size_t>(h) * P.W];
  const size_t at = static_cast<size_t>(i) * A.width + j;
  const bool old = A.score_in && (!A.have_len || j < A.have_len[i]);
  A.score_out[at] = (old ? A.score_in[at] : 0.f) + sum;
}

size_t weights_workspace_bytes(int32_t batch, int32_t n, int32_t width, int Hk, int G, int D, bool bf16) {
  // a call of fewer tokens may store logits that this one computes again
  const int few = n < 32 / G ? n : 32 / G;
  const size_t all = weight_plan(batch, n, width, Hk, G, D, bf16).total;
  const size_t stored = few > 0 ? weight_plan(batch, few, width, Hk, G, D, bf16).total : 0;
  return all > stored ? all : stored;
}

template <int D, bool BF16>
static int launch_weights_t(const WeightArgs& a, hipStream_t s) {
  const WeightPlan p = weight_plan(a.batch, a.n, a.width, a.Hk, a.G, a.D, BF16);
  const int64_t tiles = (static_cast<int64_t>(a.width) + 255) / 256;
  if (p.stored) {
    const int64_t wgs = (static_cast<int64_t>(p.parts) + kStoredWaves - 1) / kStoredWaves;
    if (!grid_fits(wgs, 64 * kStoredWaves)) return static_cast<int>(hipErrorInvalidValue);
    hipLaunchKernelGGL((weights_stored_kernel<D, BF16>), dim3(static_cast<unsigned>(wgs), a.Hk, a.batch),
                       dim3(64 * kStoredWaves), 0, s, a, p);
    hipLaunchKernelGGL(weights_join_kernel, dim3(1, a.Hk, a.batch), dim3(256), 0, s, a, p);
    hipLaunchKernelGGL(weights_sum_kernel, dim3(static_cast<unsigned>(tiles), a.batch), dim3(256), 0, s, a, p);
  } else {
    constexpr int per = kManyWaves * kManyTiles;
    const int64_t wgs = (static_cast<int64_t>(p.parts) + per - 1) / per;
    if (!grid_fits(wgs, 64 * kManyWaves)) return static_cast<int>(hipErrorInvalidValue);
    const int rt = p.row_tiles < many_row_tiles(D, BF16) ? p.row_tiles : many_row_tiles(D, BF16);
    const size_t lds = static_cast<size_t>(rt) * 32 * D * (BF16 ? 2 : 4);
    const dim3 grid(static_cast<unsigned>(wgs), a.Hk, a.batch);
    hipLaunchKernelGGL((weights_stats_kernel<D, BF16>), grid, dim3(64 * kManyWaves), lds, s, a, p);
    hipLaunchKernelGGL(weights_join_kernel, dim3(p.row_tiles, a.Hk, a.batch), dim3(256), 0, s, a, p);
    hipLaunchKernelGGL((weights_keys_kernel<D, BF16>), grid, dim3(64 * kManyWaves), lds, s, a, p);
    hipLaunchKernelGGL(weights_heads_kernel, dim3(static_cast<unsigned>(tiles), a.batch), dim3(256), 0, s, a, p);
  }
  return static_cast<int>(hipGetLastError());
}

int launch_weights(const WeightArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (a.D) {
    case 64: return bf16 ? launch_weights_t<64, true>(a, s) : launch_weights_t<64, false>(a, s);
    case 128: return bf16 ? launch_weights_t<128, true>(a, s) : launch_weights_t<128, false>(a, s);
    case 256: return bf16 ? launch_weights_t<256, true>(a, s) : launch_weights_t<256, false>(a, s);
    default: return static_cast<int>(hipErrorInvalidValue);
  }
}

}  // namespace gdn
