// Attention weights that the newest tokens give to a row's cached tokens, for gfx950.
//
//   z = scale q . k_j,  lse = log sum over j <= last of e^z,  score[j] += sum over queries of e^(z - lse)
//
// over all queries (token t < n, head h) that attend j: last = kv_len - n + t.  The
// weights of one key are a column of the softmax, whose normaliser is known only once
// a query has seen all its keys, so there are three steps: maximum and sum of every
// (query, part of the keys); their join to one lse per query; the sums per key.
// V does not enter, so K is all that has to be read.  At most 32 rows (queries of one KV
// head) store their logits for the last step, 4 bytes each beside a key's 2 D or 4 D, and K is
// read once; more rows compute them again, from K read a second time.
//
// K goes from memory to registers as it lies (each lane 16 bytes of one key per step,
// the A or B operand of a 32 x 32 matrix instruction) and Q comes from LDS, where it
// lies in the order of the operands.  A wave owns its keys and walks over the rows,
// so waves share nothing but Q, and one wave's loads hide behind the others' products.
// In base 2: z log2(e) is what is stored and compared.
//
// Bound by bytes.  24 heads on 4, d 256: one query at 4 x 8K tokens 21 - 23 us (67 MB: 14.0 - 16.2 us for
// the logits, 4.1 - 4.8 TB/s, 5.4 - 6.0 for the sums), 32 queries over 4 x 100K 377 - 420 us by the card (820 MB
// twice, 3.9 - 4.3 TB/s); 32 heads on 8, d 128, 4 queries in each of 64 ragged rows 114 - 116 us (330 MB of K, 170 MB of
// logits written and read).  With few rows the grids, the choice of the join and the workspace follow the score
// array's width: in one of 131072 the decode step takes 28.5 us, the 64 ragged rows 300, with 4.4 GB of
// workspace.  Many rows, measured and dropped: 64 keys per wave in 8
// waves instead of 32 in 16, 580 us; workgroups of a fixed number of keys, 473; one group of
// heads at a time, so that the second reading might find K in the last-level cache, 512 - 940.
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
  int32_t R, row_tiles, Rp;  // rows of a KV head (n G), tiles of 32 of them, rows in whole tiles
  int32_t W;                 // row length of the logits or sums: width in whole tiles of keys
  bool stored;               // few rows: logits are stored
  int32_t parts;             // few rows: parts (of kStoredKeys keys) of a row of `width` tokens
  // many rows: row tiles whose Q is in LDS together, and rounds of so many; a unit is a round of a KV head of a batch row
  int32_t round_tiles, rounds;
  // byte offsets; (maximum, sum) of a row over a part at 0, [batch Hk][parts][Rp] or [unit + workgroup][32
  // round_tiles]; (first workgroup, number of them) [unit] or lse [batch Hk][Rp]; the logits
  // [batch Hk][R][W] or a unit's sums [unit][W]
  size_t lse, keys, total;
};

constexpr int kTileKeys = 32;
// Few rows: waves of a workgroup, a tile of keys each
constexpr int kStoredWaves = 4, kStoredKeys = kStoredWaves * kTileKeys;
// Few rows: parts of a batch row's KV heads, and of all rows', up to which the last kernel joins them itself, a
// launch less against a join per 64 keys.  24 heads on 4, d 256, us with a kernel for the join / without: 4
// rows of 4000 tokens (128 parts) 18.7 / 16.7, of 8000 25.5 / 23.1, of 16000 42.9 / 43.4; 64 rows of 4000 129 / 132, of
// 8000 245 / 262; 16 rows of 4000, 8 KV heads 69.0 / 67.6.
constexpr int kFewParts = 320, kFewPartsAll = 4096;
// Many rows: waves of a workgroup, as the registers allow (a tile's K takes D / 4 (bf16) or D / 2 of them), and
// what they take at a time, a step of the keys
constexpr int many_waves(int D, bool bf16) { return D * (bf16 ? 2 : 4) <= 512 ? 16 : 8; }
constexpr int many_keys(int D, bool bf16) { return many_waves(D, bf16) * kTileKeys; }
// Row tiles whose Q lies in LDS at a time: 112 KB, and no more than 8 (each has 8 bytes per row and wave beside it)
constexpr int many_row_tiles(int D, bool bf16) {
  const int fit = (112 << 10) / (32 * D * (bf16 ? 2 : 4));
  return fit < 8 ? fit : 8;
}

__host__ __device__ inline size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

constexpr int kManyWorkgroups = 256;  // one per CU: 16 waves of 128 registers

WeightPlan weight_plan(int32_t batch, int32_t n, int32_t width, int Hk, int G, int D, bool bf16) {
  WeightPlan p{};
  p.R = n * G;
  p.row_tiles = (p.R + 31) / 32;
  p.Rp = p.row_tiles * 32;
  p.stored = p.row_tiles == 1;
  p.parts = static_cast<int32_t>((static_cast<int64_t>(width) + kStoredKeys - 1) / kStoredKeys);
  p.W = static_cast<int32_t>(round_up(width, 64));
  const int64_t heads = static_cast<int64_t>(batch) * Hk;
  // as many row tiles to a round as fit, or fewer where that leaves workgroups without work, but not so few that there are
  // more units of one step than workgroups (64 queries of 8 heads over 100 tokens, d 256: 20 us, with the most that fit 71;
  // 8 KV heads of 20000 tokens, d 128, 512 rows each: 233, with fewer 247; 4 rows of 5000 tokens, 4 KV heads, d 256, 192
  // query rows each: 54, with twice the rounds 60)
  const int64_t steps = (static_cast<int64_t>(width) + many_keys(D, bf16) - 1) / many_keys(D, bf16);
  const int64_t most = many_row_tiles(D, bf16), least = (p.row_tiles + most - 1) / most, fill = kManyWorkgroups / (steps * heads);
  const int64_t rounds = fill < least ? least : (fill < p.row_tiles ? fill : p.row_tiles);
  p.round_tiles = static_cast<int32_t>((p.row_tiles + rounds - 1) / rounds);
  p.rounds = (p.row_tiles + p.round_tiles - 1) / p.round_tiles;
  // A size that grows with each argument.  Units are heads x least; or, where there are more rounds than that, at
  // most kManyWorkgroups / steps, whose sums are kManyWorkgroups many_keys() at most, as W <= steps many_keys().
  const size_t base = heads * least, units = base + kManyWorkgroups;
  p.lse = round_up(p.stored ? heads * p.parts * p.Rp * sizeof(float2) : (units + kManyWorkgroups) * most * 32 * sizeof(float2), 256);
  p.keys = p.lse + round_up(p.stored ? heads * p.Rp * sizeof(float) : units * sizeof(int2), 256);
  const size_t sums = base * p.W + static_cast<size_t>(kManyWorkgroups) * many_keys(D, bf16);
  p.total = p.keys + (p.stored ? heads * p.R * static_cast<size_t>(p.W) : sums) * sizeof(float);
  return p;
}

// Row i: its queries (0: idle or refused) and cached tokens.
struct WeightRow {
  int32_t n, kv;
};
__device__ __forceinline__ WeightRow any_row(const WeightArgs& A, int i, bool report) {
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
  return r;
}
__device__ __forceinline__ WeightRow weight_row(const WeightArgs& A, int i, bool report) {
  const WeightRow r = any_row(A, i, report);
  return WeightRow{uniform(r.n), uniform(r.kv)};
}

// A workgroup's share of the keys of a unit (head h of row i, `tiles` row tiles from t0 on): steps [lo, hi) of
// its `steps`; `place` + lo is where it begins on the line of all units' steps.
struct Share {
  int i, h, t0, tiles;
  int64_t unit;
  WeightRow row;
  int32_t lo, hi, steps;
  int64_t place;
};
// The steps of all units lie on one line, row by row, head by head and round by round, and workgroup w of W = min(grid, total)
// takes places [w total / W, (w + 1) total / W), whatever the rows' lengths: f(share, w, W, total) for
// every unit that it has a part of, in order.  All waves together.
template <int KEYS, class F>
__device__ __forceinline__ void each_share(const WeightArgs& A, const WeightPlan& P, bool report, F f) {
  const int lane = threadIdx.x & 63;
  auto steps_of = [&](const WeightRow& r) { return r.n > 0 ? (r.kv + KEYS - 1) / KEYS : 0; };
  auto tiles_of = [&](const WeightRow& r) { return (r.n * A.G + 31) / 32; };
  auto units_of = [&](const WeightRow& r) { return (tiles_of(r) + P.round_tiles - 1) / P.round_tiles * A.Hk; };
  // inclusive sum over the lanes of the places of rows base + lane
  auto scan = [&](int base, int64_t* mine, bool tell) {
    const bool in = base + lane < A.batch;
    const WeightRow r = in ? any_row(A, base + lane, tell) : WeightRow{0, 0};
    int64_t inc = *mine = static_cast<int64_t>(steps_of(r)) * units_of(r);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t up = __shfl_up(inc, d, 64);
      if (lane >= d) inc += up;
    }
    return inc;
  };
  int64_t total = 0, mine = 0, inc = 0;
  for (int base = 0; base < A.batch; base += 64) {
    inc = scan(base, &mine, report);
    total += __shfl(inc, 63, 64);
  }
  total = uniform(total);
  const int64_t W = gridDim.x < total ? gridDim.x : total, w = blockIdx.x;
  if (w >= W) return;
  const int64_t first = uniform(w * total / W), last = uniform((w + 1) * total / W);
  // the row that holds place `first`: the last one that does not begin after it
  int i = 0;
  int64_t row_at = 0;
  for (int base = 0; base < A.batch; base += 64) {
    if (A.batch > 64) inc = scan(base, &mine, false);  // else it is at hand
    const int64_t chunk = __shfl(inc, 63, 64);
    if (row_at + chunk > first) {
      const int at = 63 - __builtin_clzll(__ballot(base + lane < A.batch && row_at + inc - mine <= first));
      i = base + at;
      row_at += __shfl(inc - mine, at, 64);
      break;
    }
    row_at += chunk;
  }
  i = uniform(i);
  row_at = uniform(row_at);
  for (int64_t at = first; at < last && i < A.batch;) {
    Share s;
    s.i = i;
    s.row = weight_row(A, i, false);
    s.steps = steps_of(s.row);
    const int units = units_of(s.row);
    if (at >= row_at + static_cast<int64_t>(s.steps) * units) {
      row_at += static_cast<int64_t>(s.steps) * units;
      ++i;
      continue;
    }
    const int u = static_cast<int>((at - row_at) / s.steps), rounds = units / A.Hk;
    s.h = u / rounds;
    const int round = u - s.h * rounds;
    s.t0 = round * P.round_tiles;
    s.tiles = min(P.round_tiles, tiles_of(s.row) - s.t0);
    s.unit = (static_cast<int64_t>(i) * A.Hk + s.h) * P.rounds + round;
    s.place = row_at + static_cast<int64_t>(u) * s.steps;
    s.lo = static_cast<int32_t>(at - s.place);
    s.hi = static_cast<int32_t>(last - s.place < s.steps ? last - s.place : s.steps);
    f(s, w, W, total);
    at = s.place + s.hi;
  }
}

// 16 bytes of Q of KV head h of row i, number e of row tiles [t0, ..) in the order of the operands: [tile][step][lane].
// Rows past the last repeat it, whose logits are infinite or NaN only where that row's are: zeros would meet an infinite
// key as NaN, which no weight of 0 takes out of a key's sum.
template <int D, bool BF16>
__device__ __forceinline__ uint4 q_piece(const WeightArgs& A, int i, int h, int32_t rows, int t0, int e) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32;
  const int lane = e % 64, s = e / 64 % STEPS, r = min((t0 + e / 64 / STEPS) * 32 + lane % 32, rows - 1);
  const int t = r / A.G;
  const char* q = static_cast<const char*>(A.q) +
                  ((static_cast<int64_t>(i) * A.n + t) * A.q_stride + static_cast<int64_t>(h * A.G + r - t * A.G) * D) * ES;
  return *reinterpret_cast<const uint4*>(q + (2 * s + lane / 32) * 16);
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
  __builtin_amdgcn_sched_barrier(0);  // all of them under way before the first is used
}

// Element e of a 32 x 32 result is row 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32.
__device__ __forceinline__ int result_row(int e) { return 8 * (e / 4) + 4 * ((threadIdx.x & 63) / 32) + e % 4; }

}  // namespace

// Few rows: logits of a tile of keys per wave (stored), maximum and sum of each row over the workgroup's.
template <int D, bool BF16>
__global__ __launch_bounds__(64 * kStoredWaves) void weights_stored_kernel(WeightArgs A, WeightPlan P) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32;
  __shared__ uint4 qs[STEPS * 64];
  __shared__ float2 ml[kStoredWaves][32];
  const int h = blockIdx.y, i = blockIdx.z, lane = threadIdx.x & 63;
  const int32_t wave = uniform(static_cast<int32_t>(threadIdx.x / 64));
  const WeightRow w = weight_row(A, i, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  const int64_t from = static_cast<int64_t>(blockIdx.x) * kStoredKeys;
  if (w.n == 0 || from >= w.kv) return;
  const int32_t key0 = static_cast<int32_t>(from) + wave * kTileKeys;
  // Q is asked for before K, and used first
  constexpr int PIECES = STEPS * 64 / (64 * kStoredWaves);
  uint4 q[PIECES], k[STEPS];
#pragma unroll
  for (int e = 0; e < PIECES; ++e) q[e] = q_piece<D, BF16>(A, i, h, w.n * A.G, 0, e * 64 * kStoredWaves + threadIdx.x);
  load_k<D, BF16>(A, i, h, key0, w.kv, k);
#pragma unroll
  for (int e = 0; e < PIECES; ++e) qs[e * 64 * kStoredWaves + threadIdx.x] = q[e];
  lds_barrier();
  const int row = lane % 32;
  const int32_t last = w.kv - w.n + row / A.G;  // this row's last key
  const size_t unit = static_cast<size_t>(i) * A.Hk + h;
  f32x16_t S;
#pragma unroll
  for (int e = 0; e < 16; ++e) S[e] = 0.f;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) S = mfma_step<BF16>(k[s], qs[s * 64 + lane], S);
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    S[e] = key0 + result_row(e) <= last ? S[e] * A.scale_log2 : -INFINITY;
    m = fmaxf(m, S[e]);
  }
  m = half_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int e = 0; e < 16; ++e) l += __builtin_amdgcn_exp2f(S[e] - ref);
  l = half_sum(l);
  if (row < P.R && key0 < w.kv) {
    float* z = reinterpret_cast<float*>(static_cast<char*>(A.workspace) + P.keys) + (unit * P.R + row) * P.W + key0;
#pragma unroll
    for (int e = 0; e < 16; e += 4) *reinterpret_cast<f32x4_t*>(z + result_row(e)) = f32x4_t{S[e], S[e + 1], S[e + 2], S[e + 3]};
  }
  if (lane < 32) ml[wave][row] = make_float2(m, l);
  lds_barrier();
  if (threadIdx.x < 32) {
    float both = -INFINITY, sum = 0.f;
#pragma unroll
    for (int o = 0; o < kStoredWaves; ++o) both = fmaxf(both, ml[o][row].x);
    const float to = both == -INFINITY ? 0.f : both;
#pragma unroll
    for (int o = 0; o < kStoredWaves; ++o) sum += ml[o][row].y * __builtin_amdgcn_exp2f(ml[o][row].x - to);
    static_cast<float2*>(A.workspace)[(unit * P.parts + blockIdx.x) * P.Rp + row] = make_float2(both, sum);
  }
}

// Many rows: maximum and sum of every row over a workgroup's share of the keys.
template <int D, bool BF16>
__global__ __launch_bounds__(64 * many_waves(D, BF16), many_waves(D, BF16) / 4) void weights_stats_kernel(WeightArgs A, WeightPlan P) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32, NW = many_waves(D, BF16), THREADS = 64 * NW;
  extern __shared__ __align__(16) uint4 q_lds[];
  const int held = P.round_tiles * 32;
  float2* ml = reinterpret_cast<float2*>(q_lds + static_cast<size_t>(held) * STEPS * 2);  // [wave][row of the round]
  const int lane = threadIdx.x & 63;
  const int32_t wave = uniform(static_cast<int32_t>(threadIdx.x / 64));
  each_share<many_keys(D, BF16)>(A, P, blockIdx.x == 0 && threadIdx.x < 64, [&](const Share& s, int64_t w, int64_t W, int64_t total) {
    const int32_t kv = s.row.kv;
    if (s.lo == 0 && threadIdx.x == 0) {
      // its last workgroup: the largest w' with w' total / W <= its last place
      const int64_t count = ((s.place + s.steps) * W - 1) / total - w + 1;
      reinterpret_cast<int2*>(static_cast<char*>(A.workspace) + P.lse)[s.unit] = make_int2(static_cast<int>(w), static_cast<int>(count));
    }
    __syncthreads();  // Q and the sums of what came before are read
    for (int e = threadIdx.x; e < s.tiles * STEPS * 64; e += THREADS) q_lds[e] = q_piece<D, BF16>(A, s.i, s.h, s.row.n * A.G, s.t0, e);
    for (int r = lane; r < s.tiles * 32; r += 64) ml[wave * held + r] = make_float2(-INFINITY, 0.f);
    __syncthreads();
#pragma unroll 1
    for (int32_t step = s.lo; step < s.hi; ++step) {
      const int32_t key0 = (step * NW + wave) * kTileKeys;
      if (key0 >= kv) break;
      uint4 k[STEPS];
      load_k<D, BF16>(A, s.i, s.h, key0, kv, k);
      const bool masked = key0 + kTileKeys > kv - s.row.n + 1;
      // lanes l + 32 read below what lanes l wrote in the step before
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int t = 0; t < s.tiles; ++t) {
        f32x16_t S;
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = 0.f;
#pragma unroll
        for (int o = 0; o < STEPS; ++o) S = mfma_step<BF16>(k[o], q_lds[(t * STEPS + o) * 64 + lane], S);
        const int row = t * 32 + lane % 32;
        if (masked) {
          const int32_t last = kv - s.row.n + (s.t0 * 32 + row) / A.G;
#pragma unroll
          for (int e = 0; e < 16; ++e) S[e] = key0 + result_row(e) <= last ? S[e] : -INFINITY;
        }
        const float2 was = ml[wave * held + row];
        float m = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, S[e]);
        m = fmaxf(half_max(m) * A.scale_log2, was.x);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) l += __builtin_amdgcn_exp2f(fmaf(S[e], A.scale_log2, -ref));
        l = fmaf(was.y, __builtin_amdgcn_exp2f(was.x - ref), half_sum(l));
        if (lane < 32) ml[wave * held + row] = make_float2(m, l);
      }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < s.tiles * 32; r += THREADS) {
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int o = 0; o < NW; ++o) m = fmaxf(m, ml[o * held + r].x);
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int o = 0; o < NW; ++o) l += ml[o * held + r].y * __builtin_amdgcn_exp2f(ml[o * held + r].x - ref);
      static_cast<float2*>(A.workspace)[(s.unit + w) * held + r] = make_float2(m, l);
    }
  });
}

// (maximum, sum) of the keys of two parts.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x), ref = m == -INFINITY ? 0.f : m;
  return make_float2(m, a.y * __builtin_amdgcn_exp2f(a.x - ref) + b.y * __builtin_amdgcn_exp2f(b.x - ref));
}

// Few rows: joins the parts of a KV head's rows, in a fixed order: log2 of the sum of 2^z.
__global__ __launch_bounds__(256) void weights_join_kernel(WeightArgs A, WeightPlan P) {
  __shared__ float2 parts[8][32];
  const int i = blockIdx.y, h = blockIdx.x, row = threadIdx.x % 32, g = threadIdx.x / 32;
  const WeightRow w = weight_row(A, i, false);
  if (w.n == 0) return;
  const size_t unit = static_cast<size_t>(i) * A.Hk + h;
  const float2* ml = static_cast<const float2*>(A.workspace) + unit * P.parts * P.Rp + row;
  const int count = (w.kv + kStoredKeys - 1) / kStoredKeys;
  float2 sum = make_float2(-INFINITY, 0.f);
#pragma unroll 8
  for (int p = g; p < count; p += 8) sum = join(sum, ml[static_cast<size_t>(p) * P.Rp]);
  parts[g][row] = sum;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int o = 1; o < 8; ++o) sum = join(sum, parts[o][row]);
  reinterpret_cast<float*>(static_cast<char*>(A.workspace) + P.lse)[unit * P.Rp + row] = sum.x + __builtin_amdgcn_logf(sum.y);
}

// Few rows: the weights of 64 keys from the stored logits; wave w takes heads w, w + 4, ..  JOIN: it joins the
// parts of its rows itself, which saves a launch where they are few (kFewParts).
template <bool JOIN>
__global__ __launch_bounds__(256) void weights_sum_kernel(WeightArgs A, WeightPlan P) {
  __shared__ float sums[4][64];
  const int i = blockIdx.y, lane = threadIdx.x & 63;
  const int32_t wave = uniform(static_cast<int32_t>(threadIdx.x / 64));
  const WeightRow w = weight_row(A, i, false);
  const int64_t from = static_cast<int64_t>(blockIdx.x) * 64, j = from + lane;
  if (w.n == 0 || from >= w.kv) return;
  const char* ws = static_cast<const char*>(A.workspace);
  const float* z = reinterpret_cast<const float*>(ws + P.keys) + static_cast<size_t>(i) * A.Hk * P.R * P.W + j;
  const int64_t span = j - (w.kv - w.n);  // tokens before `span` do not attend j
  const int32_t rows = w.n * A.G, first = span > 0 ? static_cast<int32_t>(span) * A.G : 0;
  float sum = 0.f;
  for (int h = wave; h < A.Hk; h += 4) {
    const size_t unit = static_cast<size_t>(i) * A.Hk + h;
    const float* lse = reinterpret_cast<const float*>(ws + P.lse) + unit * P.Rp;
    float joined = 0.f;  // of row `lane`
    if constexpr (JOIN) {
      // a lane per row and every 64 / 2^bits-th part, 2^bits >= rows
      const int bits = rows <= 8 ? 3 : (rows <= 16 ? 4 : 5), row = lane & ((1 << bits) - 1);
      const float2* ml = reinterpret_cast<const float2*>(ws) + unit * P.parts * P.Rp + row;
      const int count = (w.kv + kStoredKeys - 1) / kStoredKeys;
      float2 s = make_float2(-INFINITY, 0.f);
#pragma unroll 8
      for (int p = lane >> bits; p < count; p += 64 >> bits) s = join(s, ml[static_cast<size_t>(p) * P.Rp]);
      for (int d = 1 << bits; d < 64; d <<= 1) s = join(s, make_float2(__shfl_xor(s.x, d, 64), __shfl_xor(s.y, d, 64)));
      joined = s.x + __builtin_amdgcn_logf(s.y);
    }
#pragma unroll 8
    for (int r = 0; r < rows; ++r) {
      const float norm = JOIN ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(joined), r)) : lse[r];
      const float p = __builtin_amdgcn_exp2f(z[(static_cast<size_t>(h) * P.R + r) * P.W] - norm);
      sum += r >= first ? p : 0.f;
    }
  }
  sums[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || j >= w.kv) return;
  const size_t at = static_cast<size_t>(i) * A.width + j;
  const bool old = A.score_in && (!A.have_len || j < A.have_len[i]);
  A.score_out[at] = (old ? A.score_in[at] : 0.f) + ((sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]));
}

// Many rows: a unit's weights of the keys, the logits computed again with the
// operands the other way round, so that a lane holds one key's logits.
template <int D, bool BF16>
__global__ __launch_bounds__(64 * many_waves(D, BF16), many_waves(D, BF16) / 4) void weights_keys_kernel(WeightArgs A, WeightPlan P) {
  constexpr int ES = BF16 ? 2 : 4, STEPS = D * ES / 32, NW = many_waves(D, BF16), THREADS = 64 * NW;
  extern __shared__ __align__(16) uint4 q_lds[];
  __shared__ __align__(16) float lse[many_row_tiles(D, BF16) * 32];
  const int held = P.round_tiles * 32, lane = threadIdx.x & 63;
  const int32_t wave = uniform(static_cast<int32_t>(threadIdx.x / 64));
  each_share<many_keys(D, BF16)>(A, P, false, [&](const Share& s, int64_t, int64_t, int64_t) {
    const int32_t kv = s.row.kv, rows = s.row.n * A.G;
    float* out = reinterpret_cast<float*>(static_cast<char*>(A.workspace) + P.keys) + s.unit * P.W;
    const int2 meta = reinterpret_cast<const int2*>(static_cast<const char*>(A.workspace) + P.lse)[s.unit];
    __syncthreads();  // what came before is read
    for (int e = threadIdx.x; e < s.tiles * STEPS * 64; e += THREADS) q_lds[e] = q_piece<D, BF16>(A, s.i, s.h, rows, s.t0, e);
    // the parts of each row, joined in a fixed order: log2 of the sum of 2^z; past the last row
    // +inf, which takes every weight to 0
    for (int r = threadIdx.x; r < s.tiles * 32; r += THREADS) {
      const float2* ml = static_cast<const float2*>(A.workspace) + (s.unit + meta.x) * held + r;
      float2 sum = make_float2(-INFINITY, 0.f);
#pragma unroll 8
      for (int p = 0; p < meta.y; ++p) sum = join(sum, ml[static_cast<size_t>(p) * held]);
      lse[r] = s.t0 * 32 + r < rows ? sum.x + __builtin_amdgcn_logf(sum.y) : INFINITY;
    }
    __syncthreads();
#pragma unroll 1
    for (int32_t step = s.hi - 1; step >= s.lo; --step) {  // the last keys first: they may still be in the last-level cache
      const int32_t key0 = (step * NW + wave) * kTileKeys;
      if (key0 >= kv) continue;
      uint4 k[STEPS];
      load_k<D, BF16>(A, s.i, s.h, key0, kv, k);
      const bool masked = key0 + kTileKeys > kv - s.row.n + 1;
      float sum = 0.f;
#pragma unroll 1
      for (int t = 0; t < s.tiles; ++t) {
        f32x16_t S;
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = 0.f;
#pragma unroll
        for (int o = 0; o < STEPS; ++o) S = mfma_step<BF16>(q_lds[(t * STEPS + o) * 64 + lane], k[o], S);
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = __builtin_amdgcn_exp2f(fmaf(S[e], A.scale_log2, -lse[t * 32 + result_row(e)]));
        if (masked) {
#pragma unroll
          for (int e = 0; e < 16; ++e) S[e] = key0 + lane % 32 <= kv - s.row.n + ((s.t0 + t) * 32 + result_row(e)) / A.G ? S[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) sum += S[e];
      }
      const float total = half_sum(sum);
      if (lane < 32) out[key0 + lane] = total;  // within W
    }
  });
}

// Many rows: the units' sums of one key.
__global__ __launch_bounds__(256) void weights_units_kernel(WeightArgs A, WeightPlan P) {
  const int i = blockIdx.y;
  const WeightRow w = weight_row(A, i, false);
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (w.n == 0 || j >= w.kv) return;
  const float* k = reinterpret_cast<const float*>(static_cast<const char*>(A.workspace) + P.keys) +
                   static_cast<size_t>(i) * A.Hk * P.rounds * P.W + j;
  // a row of fewer queries has fewer rounds
  const int rounds = ((w.n * A.G + 31) / 32 + P.round_tiles - 1) / P.round_tiles;
  float sum = 0.f;
#pragma unroll 8
  for (int u = 0; u < A.Hk * P.rounds; ++u) {
    const float v = k[static_cast<size_t>(u) * P.W];
    sum += u % P.rounds < rounds ? v : 0.f;
  }
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
  if (p.stored) {
    const int64_t blocks = (static_cast<int64_t>(a.width) + 63) / 64;
    hipLaunchKernelGGL((weights_stored_kernel<D, BF16>), dim3(p.parts, a.Hk, a.batch), dim3(64 * kStoredWaves), 0, s, a, p);
    const dim3 grid(static_cast<unsigned>(blocks), a.batch);
    const int64_t parts = static_cast<int64_t>(p.parts) * a.Hk;
    if (parts <= kFewParts && parts * a.batch <= kFewPartsAll) {
      hipLaunchKernelGGL(weights_sum_kernel<true>, grid, dim3(256), 0, s, a, p);
    } else {
      hipLaunchKernelGGL(weights_join_kernel, dim3(a.Hk, a.batch), dim3(256), 0, s, a, p);
      hipLaunchKernelGGL(weights_sum_kernel<false>, grid, dim3(256), 0, s, a, p);
    }
  } else {
    constexpr int threads = 64 * many_waves(D, BF16);
    const size_t q = static_cast<size_t>(p.round_tiles) * 32 * D * (BF16 ? 2 : 4);
    const size_t ml = static_cast<size_t>(p.round_tiles) * 32 * many_waves(D, BF16) * sizeof(float2);
    const int64_t blocks = (static_cast<int64_t>(a.width) + 255) / 256;
    hipLaunchKernelGGL((weights_stats_kernel<D, BF16>), dim3(kManyWorkgroups), dim3(threads), q + ml, s, a, p);
    hipLaunchKernelGGL((weights_keys_kernel<D, BF16>), dim3(kManyWorkgroups), dim3(threads), q, s, a, p);
    hipLaunchKernelGGL(weights_units_kernel, dim3(static_cast<unsigned>(blocks), a.batch), dim3(256), 0, s, a, p);
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
