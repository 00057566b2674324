// Rotary positions of q and k for gfx950, the write of k and v into the paged KV
// cache in the same pass.
//
// Pair (x_a, x_b) of a head turns by the angle p f_i of its token's position p:
//   y_a = A (x_a c - x_b s),  y_b = A (x_a s + x_b c),  c, s = cos, sin(p f_i).
// f_i is held as turns_i, the fraction of a turn per position in units of 2^-64:
// p turns_i wraps modulo 2^64, that is, at whole turns, so the angle's error is p
// 2^-65 turns whatever p is.  Its upper 32 bits, less the nearest quarter turn,
// are what reaches fp32: at most an eighth of a turn, on which the Taylor
// polynomials below are good to 2^-25.
//
// A token's cosines and sines (R/2 pairs) are computed once by its workgroup into LDS
// and serve all its heads.  A unit of work is 16 dimensions of one head of one token,
// two groups of 8: of a rotated unit, the two halves of eight pairs; of a copied one, 16
// dimensions behind one another.
//
// Bound by bytes; a unit's loads are under way while the angles are made.  bf16, q and k
// out of place: 32771 tokens of 24 + 4 heads, d 256, 64 dimensions turned, with the cache
// 201 us (1141 MB, 5.7 TB/s); 5003 tokens of 32 + 8 heads, d 128, all turned, 21.7 (102
// MB, 4.7 TB/s).  A unit to each of 512 threads; with 2 or 4 units to a thread 202 / 23.3
// and 217 / 25.0, with 256 threads and 2, 4 or 8 units 206 / 24.3, 217 / 25.2 and 230 / 24.2,
// with 1024 threads and one unit 205 / 24.2; a thread's next unit loaded ahead is no
// faster.  4 tokens take 2 - 3 us, the launch and two loads behind one another.
#include "gdn_device.h"
#include "gdn_ops.h"

namespace gdn {

namespace {

constexpr int kRopeThreads = 512;
constexpr int kRopeMaxTokens = 16;  // of a workgroup

// cos and sin of x turns, |x| <= 1/8, as Taylor polynomials in y = 2 pi x, |y| <= pi / 4:
// the first terms left out are y^10 / 11! and y^12 / 12!, below 3e-9.
__device__ __forceinline__ void cos_sin_eighth(float x, float* c, float* s) {
  const float y = x * 6.283185307179586f, z = y * y;
  float u = 2.7557319e-6f;                        // 1/9!
  u = fmaf(u, z, -1.9841270e-4f);                 // -1/7!
  u = fmaf(u, z, 8.3333333e-3f);                  // 1/5!
  u = fmaf(u, z, -0.16666667f);                   // -1/3!
  *s = fmaf(y * z, u, y);
  float v = -2.7557319e-7f;                       // -1/10!
  v = fmaf(v, z, 2.4801587e-5f);                  // 1/8!
  v = fmaf(v, z, -1.3888889e-3f);                 // -1/6!
  v = fmaf(v, z, 4.1666667e-2f);                  // 1/4!
  *c = fmaf(z * z, v, fmaf(z, -0.5f, 1.0f));
}

// cos and sin of position p at turns per position, times the amplitude.
__device__ __forceinline__ float2 turned(int32_t p, uint64_t turns, bool inverse, float amplitude) {
  uint64_t a = turns * static_cast<uint64_t>(static_cast<int64_t>(p));
  if (inverse) a = 0 - a;
  const uint32_t t = static_cast<uint32_t>((a + (1ull << 31)) >> 32);  // 2^-32 turns
  const uint32_t quarter = (t + (1u << 29)) >> 30;                     // the nearest, 4 being 0
  const int32_t rest = static_cast<int32_t>(t - (quarter << 30));
  float c, s;
  cos_sin_eighth(static_cast<float>(rest) * 0x1p-32f, &c, &s);
  if (quarter & 1) {
    const float was = c;
    c = -s;
    s = was;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(amplitude * c, amplitude * s);
}

// Eight elements of a row.
template <bool BF16>
struct Eight;
template <>
struct Eight<true> {
  uint4 v;
  __device__ __forceinline__ void load(const char* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    v = make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7]));
  }
};
template <>
struct Eight<false> {
  float4 v[2];
  __device__ __forceinline__ void load(const char* p) {
    v[0] = reinterpret_cast<const float4*>(p)[0];
    v[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(char* p) const {
    reinterpret_cast<float4*>(p)[0] = v[0];
    reinterpret_cast<float4*>(p)[1] = v[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = v[i].x;
      f[4 * i + 1] = v[i].y;
      f[4 * i + 2] = v[i].z;
      f[4 * i + 3] = v[i].w;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  }
};

// Division by d >= 1 as a product: e / d = (e m) >> 32 with m = ceil(2^32 / d), where
// e (d - 1) < 2^32 (m d exceeds 2^32 by at most d - 1, so e m / 2^32 exceeds e / d by
// less than 1 / d).
struct Divisor {
  uint32_t d, m;
};
Divisor divisor(uint32_t d) { return Divisor{d, static_cast<uint32_t>(((1ull << 32) + d - 1) / d)}; }
__device__ __forceinline__ uint32_t divide(uint32_t e, Divisor v) {
  return v.d == 1 ? e : static_cast<uint32_t>((static_cast<uint64_t>(e) * v.m) >> 32);
}

}  // namespace

// How a token's units lie: those of q, then of k, then of v, per head `q_units`,
// `k_units` and D / 16 (v only with a cache).
struct RopePlan {
  Divisor token, q_units, k_units, v_units;  // token: all units of one (m = 0: a workgroup has one token)
  Divisor pairs;                             // R / 2
  uint32_t q_end, k_end;                     // first unit of k, of v
  int32_t tokens;                            // of a workgroup
};

template <bool BF16, bool PAIRS>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs A, RopePlan P) {
  constexpr int ES = BF16 ? 2 : 4;
  // cosine and sine of pairs 8 u .. 8 u + 7 of a token: [token][4][R / 16] of two pairs each, so that
  // lanes of neighbouring units read neighbouring words
  extern __shared__ __align__(16) float4 turn[];
  __shared__ int64_t cells[kRopeMaxTokens];  // byte offset of head 0 in the cache, -1: not cached
  const int tid = threadIdx.x, RU = A.R / 16;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.tokens;
  const int nt = static_cast<int>(A.n_tokens - t0 < P.tokens ? A.n_tokens - t0 : P.tokens);
  const uint32_t units = nt * P.token.d;

  struct Unit {
    Eight<BF16> a, b;
    char* out;        // its row's output (null: v has the cache's alone)
    uint32_t at, bt;  // byte offsets of the two groups within the head
    int32_t token, cached;  // cached: -1 no, else the head; v: bit 30
    int32_t pair;     // its unit of the rotation, -1: copied
  };
  auto fetch = [&](uint32_t e, Unit& u) {
    const uint32_t tt = divide(e, P.token);
    uint32_t r = e - tt * P.token.d;
    const int64_t t = t0 + tt;
    u.token = tt;
    const char* in;
    uint32_t h, p;
    if (r < P.q_end) {
      h = divide(r, P.q_units);
      p = r - h * P.q_units.d;
      in = static_cast<const char*>(A.q) + t * A.q_stride;
      u.out = static_cast<char*>(A.q_out) + t * A.q_out_stride;
      u.cached = -1;
    } else if (r < P.k_end) {
      r -= P.q_end;
      h = divide(r, P.k_units);
      p = r - h * P.k_units.d;
      in = static_cast<const char*>(A.k) + t * A.k_stride;
      u.out = static_cast<char*>(A.k_out) + t * A.k_out_stride;
      u.cached = A.k_cache ? static_cast<int32_t>(h) : -1;
    } else {
      r -= P.k_end;
      h = divide(r, P.v_units);
      p = r - h * P.v_units.d;
      in = static_cast<const char*>(A.v) + t * A.v_stride;
      u.out = nullptr;
      u.cached = static_cast<int32_t>(h) | (1 << 30);
    }
    const uint32_t head = h * A.D * ES;
    in += head;
    u.pair = u.out && p < static_cast<uint32_t>(RU) ? static_cast<int32_t>(p) : -1;
    u.at = (!PAIRS && u.pair >= 0 ? 8 * p : 16 * p) * ES;
    u.bt = !PAIRS && u.pair >= 0 ? u.at + A.R / 2 * ES : u.at + 8 * ES;
    if (u.out) u.out += head;
    u.a.load(in + u.at);
    u.b.load(in + u.bt);
  };

  // the first unit's loads are under way while the angles are made
  uint32_t e = tid;
  Unit u;
  if (e < units) fetch(e, u);
  const uint32_t head_bytes = A.D * ES;
  if (tid < nt && A.k_cache) {
    const int32_t slot = A.slot_map[t0 + tid];
    const bool in = slot >= 0 && slot < static_cast<int64_t>(A.n_pages) * A.page;
    if (!in && slot != -1) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
    const int32_t page = slot / A.page, off = slot - page * A.page;
    cells[tid] = in ? (static_cast<int64_t>(page) * A.Hk * A.page + off) * head_bytes : -1;
  }
  float2* turn2 = reinterpret_cast<float2*>(turn);
  for (int i = tid; i < nt * RU * 8; i += kRopeThreads) {
    const int tt = divide(i, P.pairs), pair = i - tt * (RU * 8);
    turn2[(tt * 4 + pair % 8 / 2) * RU * 2 + pair / 8 * 2 + pair % 2] =
        turned(A.position[t0 + tt], A.turns[pair], A.inverse, A.amplitude);
  }
  __syncthreads();

  while (e < units) {
    if (u.pair >= 0) {
      float a[8], b[8];
      u.a.get(a);
      u.b.get(b);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 cs = turn[(u.token * 4 + k) * RU + u.pair];
        // pairs 2 k and 2 k + 1 of the unit: (a_i, b_i), or neighbours of the 16
        float& xa = PAIRS ? (k < 2 ? a[4 * k] : b[4 * k - 8]) : a[2 * k];
        float& xb = PAIRS ? (k < 2 ? a[4 * k + 1] : b[4 * k - 7]) : b[2 * k];
        float& ya = PAIRS ? (k < 2 ? a[4 * k + 2] : b[4 * k - 6]) : a[2 * k + 1];
        float& yb = PAIRS ? (k < 2 ? a[4 * k + 3] : b[4 * k - 5]) : b[2 * k + 1];
        const float xc = xa * cs.x - xb * cs.y, xs = xa * cs.y + xb * cs.x;
        const float yc = ya * cs.z - yb * cs.w, ys = ya * cs.w + yb * cs.z;
        xa = xc;
        xb = xs;
        ya = yc;
        yb = ys;
      }
      u.a.set(a);
      u.b.set(b);
    }
    if (u.out) {
      u.a.store(u.out + u.at);
      u.b.store(u.out + u.bt);
    }
    if (u.cached >= 0) {
      const int64_t cell = cells[u.token];
      if (cell >= 0) {
        const int32_t h = u.cached & ~(1 << 30);
        char* row = static_cast<char*>(u.cached >> 30 ? A.v_cache : A.k_cache) + cell +
                    static_cast<int64_t>(h) * A.page * head_bytes;
        u.a.store(row + u.at);
        u.b.store(row + u.bt);
      }
    }
    e += kRopeThreads;
    if (e < units) fetch(e, u);
  }
}

// The call of n tokens from token t on.
static RopeArgs rope_part(const RopeArgs& a, int64_t t, int64_t n) {
  RopeArgs part = a;
  auto in = [t](const void* p, int64_t stride) { return p ? static_cast<const char*>(p) + t * stride : nullptr; };
  auto out = [t](void* p, int64_t stride) { return p ? static_cast<char*>(p) + t * stride : nullptr; };
  part.q = in(a.q, a.q_stride);
  part.k = in(a.k, a.k_stride);
  part.v = in(a.v, a.v_stride);
  part.q_out = out(a.q_out, a.q_out_stride);
  part.k_out = out(a.k_out, a.k_out_stride);
  part.position = a.position + t;
  part.slot_map = a.slot_map ? a.slot_map + t : nullptr;
  part.n_tokens = static_cast<int32_t>(n);
  return part;
}

int launch_rope(const RopeArgs& a, bool bf16, bool pairs, void* stream) {
  RopePlan p{};
  const uint32_t all = a.D / 16, rot = a.R / 16;
  const bool q_in_place = a.q == a.q_out, k_in_place = a.k == a.k_out;
  const uint32_t qu = q_in_place ? rot : all, ku = k_in_place && !a.k_cache ? rot : all;
  p.q_units = divisor(qu);
  p.k_units = divisor(ku);
  p.v_units = divisor(all);
  p.q_end = a.q ? a.Hq * qu : 0;
  p.k_end = p.q_end + (a.k ? a.Hk * ku : 0);
  p.token = divisor(p.k_end + (a.k_cache ? a.Hk * all : 0));
  p.pairs = divisor(a.R / 2);
  // a unit to a thread, or one token to a workgroup where it has more units; fewer tokens where there would be less than 1024 workgroups
  int64_t tokens = kRopeThreads / p.token.d;
  tokens = tokens < 1 ? 1 : (tokens > kRopeMaxTokens ? kRopeMaxTokens : tokens);
  while (tokens > 1 && a.n_tokens / tokens < 1024) --tokens;
  p.tokens = static_cast<int32_t>(tokens);
  if (tokens == 1) p.token.m = 0;  // a token may have more units than a product divides; else there are kRopeThreads at most
  const size_t lds = static_cast<size_t>(tokens) * a.R / 2 * sizeof(float2);
  hipStream_t s = static_cast<hipStream_t>(stream);
  // more tokens than a launch's workgroups take go in several launches
  const int64_t most = 0xffffffffll / kRopeThreads * tokens;
  for (int64_t t = 0; t < a.n_tokens; t += most) {
    const RopeArgs part = rope_part(a, t, a.n_tokens - t < most ? a.n_tokens - t : most);
    const dim3 grid(static_cast<unsigned>((part.n_tokens + tokens - 1) / tokens));
    if (bf16 && pairs) hipLaunchKernelGGL((rope_kernel<true, true>), grid, dim3(kRopeThreads), lds, s, part, p);
    else if (bf16) hipLaunchKernelGGL((rope_kernel<true, false>), grid, dim3(kRopeThreads), lds, s, part, p);
    else if (pairs) hipLaunchKernelGGL((rope_kernel<false, true>), grid, dim3(kRopeThreads), lds, s, part, p);
    else hipLaunchKernelGGL((rope_kernel<false, false>), grid, dim3(kRopeThreads), lds, s, part, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return static_cast<int>(err);
  }
  return 0;
}

}  // namespace gdn
