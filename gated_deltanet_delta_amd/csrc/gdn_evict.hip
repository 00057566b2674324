// Eviction from the paged KV cache for gfx950: which of a row's tokens stay, and the
// moves that close the gaps.
//
// Plan.  Each token j of a row has a key, its score as an unsigned integer of the same
// order, the largest for protected tokens.  The b tokens that stay are the b largest
// (key, ~j), found digit by digit from the top: of the tokens that agree with the b-th
// largest in the digits known, how many have which next digit.  Counts are kept in eight
// copies, lane l taking copy l % 8, since scores crowd into few digits.  After one digit the
// tokens left are few and move to a list in LDS; where they do not fit (many equal scores)
// the row is gone over again.  What stays is a bit per token in LDS; the kept tokens behind
// the budget fill the gaps below it, both in order, so a pair's number is a rank among bits.
// A row that loses e tokens moves min(b, e) at most, whatever its length.
//
// One workgroup plans one row and needs no memory beside its LDS and the outputs; one more
// puts the freed pages of all rows on the stack, where the ones that exist follow one another.  A CU
// issues one vector instruction a cycle for 64 tokens, so what bounds long rows is the
// number of instructions per token and pass: no branches and no addresses per token, one
// form of the loads for all steps.  Short rows are bound by latency: chains of loads,
// barriers between the digits, and the kernel's own instructions, which a launch fetches
// anew, so all passes take the same code.  us: 4 rows of 8192 19 - 20, 64 rows of 500 - 16384
// 32 - 34, 3 rows of 120000 cut to 16384 72.  (Keys of a row gone over in dependent steps, 2048
// counters in one copy: 27, 39 and 351; a branch per token and counter: 49, 45, 303; loads
// in a form per kind of step, whose results meet in copies of registers and are waited for
// there: 22, 34, 104.)
#include "gdn_attn_device.h"

namespace gdn {

namespace {

constexpr int kEvictThreads = 1024, kEvictWaves = kEvictThreads / kWave;
constexpr int kKeys = 8;                          // tokens of a thread and step
constexpr int kStep = kEvictThreads * kKeys;
constexpr int kWaveTokens = kWave * kKeys;        // a wave's of a step follow one another
constexpr int kGroupWords = 4;                    // words of the bits whose ranks share one base
constexpr int kDigits = 2048, kCopies = 8;        // counters: values of a digit, copies of each
constexpr int kMaxCandidates = 8192;
constexpr int kFewCandidates = 256;               // ranked by comparing all pairs
constexpr size_t kEvictLds = 156 << 10;
// Tokens behind a row's last count as kPast, below every token's key: a row keeps fewer than it has, so none of them stays.
constexpr uint32_t kPast = 0, kNan = 1, kProtected = 0xffffffffu;

// A score as an unsigned integer of the same order: NaN lowest, -0 = 0 (-0 + 0 is 0).
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t bits = __float_as_uint(s + 0.f);
  const uint32_t key = bits ^ (static_cast<uint32_t>(static_cast<int32_t>(bits) >> 31) | 0x80000000u);
  return s != s ? kNan : key;
}

struct EvictRow {
  int32_t c, b, settled, gone;
  bool ok, cut;  // lengths within limits; tokens leave
};
__device__ __forceinline__ EvictRow evict_row(const EvictArgs& A, int i, bool report) {
  EvictRow r{A.kv_len[i], A.budget[i], A.row_state[2 * i], A.row_state[2 * i + 1], false, false};
  const int64_t most = static_cast<int64_t>(A.max_pages) * A.page;
  r.ok = r.c >= 0 && r.c <= A.width && r.c <= most && r.settled >= 0 && r.settled <= r.c && r.gone >= 0 &&
         r.gone <= INT32_MAX - r.c;
  r.cut = r.ok && r.b >= 0 && r.b < r.c;
  const bool bad = r.cut && (r.b < static_cast<int64_t>(A.sink) + A.recent || min(r.b, r.c - r.b) > A.max_moves);
  if (report && (!r.ok || bad)) report_error(A.dev_err, GDN_DEV_BAD_LENGTH);
  r.cut = r.cut && !bad;
  return r;
}
__device__ __forceinline__ uint32_t pages_of(int32_t tokens, int32_t page) {
  return (static_cast<uint32_t>(tokens) + page - 1) / page;
}

// Digits of (key, n), n = ~j in `n_bits` bits: 11, 11 and 10 bits of the key, 11 of n and the rest.
constexpr int kAllDigits = 5;
__device__ __forceinline__ int digit_shift(int d, int n_bits) {
  return d < 3 ? (d == 0 ? 21 : (d == 1 ? 10 : 0)) : (d == 3 ? (n_bits > 11 ? n_bits - 11 : 0) : 0);
}
__device__ __forceinline__ uint32_t digit_mask(int d, int n_bits) {
  return d < 2 ? 2047 : (d == 2 ? 1023 : (d == 3 ? 2047 : (1u << (n_bits > 11 ? n_bits - 11 : 0)) - 1));
}

// Inclusive sums over the wave's lanes, which stay at 2^32 - 1 (DPP: shifts within 16 lanes, then the last lane of a
// row to the next ones).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_add(uint32_t v) {
  return __builtin_elementwise_add_sat(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);
  return dpp_add<0x143, 0xc>(v);
}
// Bits that any lane has, in every lane.
__device__ __forceinline__ uint32_t wave_or(uint32_t v) {
  v |= __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);   // lane ^ 1
  v |= __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);   // lane ^ 2
  v |= __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);  // 7 - i within 8 lanes
  v |= __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // 15 - i within 16 lanes
  return __builtin_amdgcn_readlane(v, 0) | __builtin_amdgcn_readlane(v, 16) | __builtin_amdgcn_readlane(v, 32) |
         __builtin_amdgcn_readlane(v, 48);
}
__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return __builtin_amdgcn_readlane(v, kWave - 1); }

// A buffer of n 32-bit words: words past its end read as 0, without a memory access.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t bounded(const void* p, int32_t n) {
  const uint64_t a = static_cast<uint64_t>(uniform(static_cast<int64_t>(reinterpret_cast<uint64_t>(p))));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(a), static_cast<short>(0), uniform(n) * 4, 0x00020000);
}
template <class V>
__device__ __forceinline__ V load_bounded(__amdgpu_buffer_rsrc_t r, int32_t byte) {
  return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b32(r, byte, 0, 0));
}

// The lowest n bits, n of any sign and size.
__device__ __forceinline__ uint64_t low_bits(int32_t n) { return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1); }
__device__ __forceinline__ uint64_t uniform_word(uint64_t v) { return static_cast<uint64_t>(uniform(static_cast<int64_t>(v))); }
// Number of bits of m below this lane's, plus `base`.
__device__ __forceinline__ uint32_t rank_in(uint64_t m, uint32_t base) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), base));
}

static_assert(kEvictMaxBatch == 4 * kEvictThreads && 2 * kEvictMaxBatch <= kDigits * kCopies, "four rows to a thread, two words to a row");

// Freed pages onto the stack, rows in order: those behind the budget of the rows that are cut, less the ids that are
// no pages of the cache, and how many the stack holds then.  The work of one workgroup, beside those that plan the rows,
// since a page's place depends on all before it: 8192 pages in 2.5 us, so it is done before they are up to some
// 100000 pages.  (512 rows that lose 1000 pages each: 163 us.  Each row's workgroup pushing its own, whatever the ids:
// 62; and 64 ragged rows 33.5, now 33.0.)  `lds` has two words for each row.
__device__ __forceinline__ void push_freed(const EvictArgs& A, uint32_t* lds, uint32_t (*sums)[kEvictWaves]) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = uniform(tid / kWave);
  uint32_t *start = lds, *first = lds + kEvictMaxBatch;  // number of a row's first page among the freed ones, its entry in the row's table
  const int32_t nf = *A.n_free;
  uint32_t pages[4], mine = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 4 * tid + k;
    pages[k] = 0;
    if (r < A.batch) {
      const EvictRow w = evict_row(A, r, true);
      first[r] = w.cut ? pages_of(w.b, A.page) : 0;
      pages[k] = w.cut ? pages_of(w.c, A.page) - first[r] : 0;
    }
    mine = __builtin_elementwise_add_sat(mine, pages[k]);
  }
  const uint32_t inc = wave_scan(mine);
  if (lane == kWave - 1) sums[0][wave] = inc;
  __syncthreads();
  const uint32_t others = wave_scan(lane < kEvictWaves ? sums[0][lane] : 0), total = last_lane(others);
  uint32_t at = inc - mine + (wave > 0 ? __builtin_amdgcn_readlane(others, wave - 1) : 0);  // exact where the stack takes them
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    start[4 * tid + k] = at;
    at += pages[k];
  }
  const bool stack_ok = nf >= 0 && static_cast<int64_t>(nf) + total <= A.n_pages;
  __syncthreads();
  uint32_t pushed = 0;
  if (stack_ok) {
    int turn = 0;
#pragma unroll 1
    for (uint32_t f0 = wave * kWaveTokens; f0 - wave * kWaveTokens < total; f0 += kStep, turn ^= 1) {
      int32_t page[kKeys];
      uint64_t there[kKeys];
      uint32_t count = 0, r = 0, begin = 0, end = 0;  // the row of this lane's page, which has pages [begin, end)
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        const uint32_t f = min(f0 + k * kWave + lane, total - 1);
        if (__ballot(f >= end) != 0) {
          r = 0;  // the last row that does not begin after f
#pragma unroll
          for (uint32_t d = kEvictMaxBatch / 2; d > 0; d /= 2) r += start[r + d] <= f ? d : 0;
          begin = start[r];
          end = r + 1 < kEvictMaxBatch ? start[r + 1] : total;
        }
        page[k] = A.block_table[static_cast<size_t>(r) * A.max_pages + first[r] + (f - begin)];
      }
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        const bool in = f0 + k * kWave + lane < total, ok = page[k] >= 0 && page[k] < A.n_pages;
        if (in && !ok) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
        there[k] = __ballot(in && ok);
        count += __popcll(there[k]);
      }
      if (lane == 0) sums[1 + turn][wave] = count;  // of the step before last: every wave has read it
      __syncthreads();
      const uint32_t ends = wave_scan(lane < kEvictWaves ? sums[1 + turn][lane] : 0);
      uint32_t to = pushed + (wave > 0 ? __builtin_amdgcn_readlane(ends, wave - 1) : 0);
      pushed += last_lane(ends);
#pragma unroll
      for (int k = 0; k < kKeys; ++k) {
        if (__builtin_amdgcn_inverse_ballot_w64(there[k])) A.free_pages[static_cast<int64_t>(nf) + rank_in(there[k], to)] = page[k];
        to += __popcll(there[k]);
      }
    }
  }
  if (tid == 0) {
    *A.n_free_out = static_cast<int32_t>(nf + pushed);
    if (!stack_ok) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
  }
}

}  // namespace

// LDS of a plan: the bits of `words` 64-token words, a rank per group of them, counters, candidates and one more.
// page_m: e / page = (2 (e / 16) page_m) >> 32.
struct EvictPlan {
  int32_t words, candidates;
  uint32_t page_m;
};

__global__ __launch_bounds__(kEvictThreads) void evict_plan_kernel(EvictArgs A, EvictPlan L) {
  extern __shared__ __align__(16) uint64_t kept[];
  uint32_t* rank0 = reinterpret_cast<uint32_t*>(kept + L.words);
  uint32_t* counts = rank0 + L.words / kGroupWords;
  uint2* candidates = reinterpret_cast<uint2*>(counts + kDigits * kCopies);
  __shared__ uint32_t sums[3][kEvictWaves], found[3], n_candidates, some_bits, all_bits;
  const int i = static_cast<int>(blockIdx.x) - 1, tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = uniform(tid / kWave);
  if (i < 0) return push_freed(A, counts, sums);

  // ---- freed pages of all rows: whether the stack takes them ----
  const int32_t nf = *A.n_free;
  uint32_t all = 0;
#pragma unroll 1
  for (int r = tid; r < A.batch; r += kEvictThreads) {
    const EvictRow w = evict_row(A, r, false);
    all = __builtin_elementwise_add_sat(all, w.cut ? pages_of(w.c, A.page) - pages_of(w.b, A.page) : 0);
  }
  EvictRow row = evict_row(A, i, false);
  all = wave_scan(all);
  if (lane == kWave - 1) sums[0][wave] = all;
  if (tid == 0) {
    n_candidates = some_bits = 0;
    all_bits = ~0u;
  }
#pragma unroll 1
  for (int e = tid; e < kDigits * kCopies / 4; e += kEvictThreads) reinterpret_cast<uint4*>(counts)[e] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const uint32_t total = last_lane(wave_scan(lane < kEvictWaves ? sums[0][lane] : 0));
  if (nf < 0 || static_cast<int64_t>(nf) + total > A.n_pages) row.cut = false;
  const int32_t c = row.c, b = row.cut ? row.b : c;
  const size_t at = static_cast<size_t>(i) * A.width, list = static_cast<size_t>(i) * A.max_moves;
  const float* score = A.score + at;
  const int32_t* token_pos = A.token_pos + at;
  int32_t moves = 0;

  if (row.cut) {
    // ---- the threshold, digit by digit ----
    // protected: positions below `sink` or from `recent` on, that is, outside [sink, recent)
    const int64_t recent64 = static_cast<int64_t>(c) + row.gone - A.recent;
    const int32_t recent = static_cast<int32_t>(recent64 > A.sink ? recent64 : A.sink);
    const uint32_t free_span = static_cast<uint32_t>(recent - A.sink);
    uint32_t T = 0, N = 0, need = b, knownT = 0, knownN = 0, among = 0;
    int32_t listed = -1;  // candidates in LDS, -1: they are not
    const int n_bits = 32 - __builtin_clz(c);  // c >= 1
    const __amdgpu_buffer_rsrc_t scores = bounded(score, c), positions = bounded(token_pos, row.settled);
    const uint32_t n_mask = (1u << n_bits) - 1;
    // Passes over all tokens of the row (or, with the candidates listed, over those).  kCount: counted by their
    // next digit; kClassify: those above the threshold's known digits stay, those that agree become candidates;
    // kBits: those from the threshold up stay.
    enum Pass { kCount, kClassify, kBits };
    Pass what = b > 0 ? kCount : kBits;
    if (b == 0) T = N = ~0u;  // above every (key, n)
    // words of the last group behind the row's
    if (tid < kGroupWords && (c + 63) / 64 + tid < L.words) kept[(c + 63) / 64 + tid] = 0;
#pragma unroll 1
    for (int d = 0;;) {
      const int shift = digit_shift(d, n_bits);
      const uint32_t mask = digit_mask(d, n_bits);
      if (listed >= 0) {
        const uint32_t of_key = d < 3 ? ~0u : 0u;
#pragma unroll 1
        for (int32_t e0 = wave * kWave; e0 < listed; e0 += kEvictThreads) {
          const uint2 x = candidates[min(e0 + lane, listed - 1)];
          const uint32_t other = ((x.x ^ T) & knownT) | ((x.y ^ N) & knownN), digit = ((x.x & of_key) | (x.y & ~of_key)) >> shift & mask;
          atomicAdd(&counts[digit * kCopies + lane % kCopies], e0 + lane < listed && other == 0 ? 1u : 0u);
        }
      } else {
        float s[kKeys];
        int32_t p[kKeys];
        // each step's loads are under way while the one before is worked on
#pragma unroll 1
        for (int32_t j0 = -kStep; j0 < c; j0 += kStep) {
          uint32_t key[kKeys];
          const int32_t first = j0 + wave * kWaveTokens, j = first + lane;  // this wave's first token of the step, this lane's
          // no token of a plain step is protected, by its index alone
          auto plain = [&](int32_t f) { return f >= row.settled && f + row.gone >= A.sink && static_cast<uint32_t>(f + row.gone) + kWaveTokens <= static_cast<uint32_t>(recent); };
          if (j0 >= 0) {
#pragma unroll
            for (int k = 0; k < kKeys; ++k) key[k] = score_key(s[k]);
            if (first + kWaveTokens <= row.settled) {
#pragma unroll
              for (int k = 0; k < kKeys; ++k) key[k] = static_cast<uint32_t>(p[k] - A.sink) >= free_span ? kProtected : key[k];
            } else if (!plain(first)) {
#pragma unroll
              for (int k = 0; k < kKeys; ++k) {
                const int32_t e = j + k * kWave;
                const uint32_t pos = e < row.settled ? p[k] : static_cast<uint32_t>(e) + row.gone;
                key[k] = pos - A.sink >= free_span ? kProtected : key[k];
                key[k] = e < c ? key[k] : kPast;
              }
            }
          }
          // one form of the loads for all steps: other forms meet in copies of registers, which wait for the loads
          const int32_t next = (j + kStep) * 4;
#pragma unroll
          for (int k = 0; k < kKeys; ++k) s[k] = load_bounded<float>(scores, next + k * kWave * 4);
#pragma unroll
          for (int k = 0; k < kKeys; ++k) p[k] = load_bounded<int32_t>(positions, next + k * kWave * 4);
          if (j0 < 0 || first >= c) continue;
          const int32_t word = first / 64 + lane;  // lane k stores the bits of tokens first + 64 k on
          if (what == kCount && d == 0) {
#pragma unroll
            for (int k = 0; k < kKeys; ++k) atomicAdd(&counts[(key[k] >> 21) * kCopies + lane % kCopies], 1u);
          } else if (what == kCount) {
#pragma unroll
            for (int k = 0; k < kKeys; ++k) {
              const uint32_t n = ~(j + k * kWave) & n_mask, other = ((key[k] ^ T) & knownT) | ((n ^ N) & knownN);
              if (other == 0) atomicAdd(&counts[((d < 3 ? key[k] : n) >> shift & mask) * kCopies + lane % kCopies], 1u);
            }
          } else if (what == kClassify) {
            uint64_t stay = 0, same[kKeys];
            uint32_t count = 0;
#pragma unroll
            for (int k = 0; k < kKeys; ++k) {
              const uint64_t w = __ballot(key[k] > (T | ~knownT));
              stay = lane == k ? w : stay;
              same[k] = __ballot(key[k] - T <= ~knownT);
              count += __popcll(same[k]);
            }
            if (lane < kKeys && word < L.words) kept[word] = stay;
            if (count != 0) {
              uint32_t to = 0;
              if (lane == 0) to = atomicAdd(&n_candidates, count);
              to = __builtin_amdgcn_readfirstlane(to);
              // every lane writes, those without a candidate behind the list's end
#pragma unroll
              for (int k = 0; k < kKeys; ++k) {
                const uint32_t rank = rank_in(same[k], to);
                candidates[__builtin_amdgcn_inverse_ballot_w64(same[k]) && rank < among ? rank : static_cast<uint32_t>(L.candidates)] =
                    make_uint2(key[k], ~(j + k * kWave) & n_mask);
                to += __popcll(same[k]);
              }
            }
          } else {
            uint64_t stay = 0;
#pragma unroll
            for (int k = 0; k < kKeys; ++k) {
              const uint64_t w = __ballot(key[k] > T || (key[k] == T && (~(j + k * kWave) & n_mask) >= N && key[k] != kPast));
              stay = lane == k ? w : stay;
            }
            if (lane < kKeys && word < L.words) kept[word] = stay;
          }
        }
      }
      __syncthreads();
      if (what == kBits) break;
      if (what == kClassify) {
        listed = among;
        if (listed <= kFewCandidates) break;
        uint32_t some = 0, every = ~0u;  // bits that one of the candidates has, that all have
#pragma unroll 1
        for (int32_t e = tid; e < listed; e += kEvictThreads) {
          some |= candidates[e].x;
          every &= candidates[e].x;
        }
        some = wave_or(some);
        every = ~wave_or(~every);
        if (lane == 0) {
          atomicOr(&some_bits, some);
          atomicAnd(&all_bits, every);
        }
        __syncthreads();
        // digits that all candidates share (equal scores) need no pass
        const uint32_t varies = some_bits & ~all_bits, shared = varies == 0 ? 0u : ~0u >> __builtin_clz(varies);
        T |= all_bits & ~shared;
        while (d < 2 && (~shared >> digit_shift(d + 1, n_bits) & digit_mask(d + 1, n_bits)) == digit_mask(d + 1, n_bits)) {
          ++d;
          knownT |= digit_mask(d, n_bits) << digit_shift(d, n_bits);
        }
        T &= knownT;
      } else {
        // from the highest digit down, two to a thread, which reads and clears their copies: four
        // times 16 bytes, in an order by lane that spreads them over the banks
        static_assert(kDigits == 2 * kEvictThreads && kCopies == 8, "two digits to a thread");
        const int top = kDigits - 1 - 2 * tid;
        uint4 part[4];
        uint32_t h[2] = {0, 0};  // of top - 1, top
        auto copies = [&](int q) -> uint4& { return reinterpret_cast<uint4*>(counts)[(top - 1) * (kCopies / 4) + q]; };
#pragma unroll
        for (int q = 0; q < 4; ++q) part[q] = copies((q + tid / 4) % 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int of = (q + tid / 4) % 4;
          const uint32_t sum = part[q].x + part[q].y + part[q].z + part[q].w;
          h[0] += of < 2 ? sum : 0;
          h[1] += of < 2 ? 0 : sum;
          copies(of) = make_uint4(0, 0, 0, 0);
        }
        const uint32_t inc = wave_scan(h[0] + h[1]);
        if (lane == kWave - 1) sums[2][wave] = inc;
        __syncthreads();
        const uint32_t others = wave_scan(lane < kEvictWaves ? sums[2][lane] : 0);
        const uint32_t start = wave > 0 ? __builtin_amdgcn_readlane(others, wave - 1) : 0;
        const uint32_t begin = start + inc - h[0] - h[1], middle = begin + h[1], end = middle + h[0];
        if (begin < need && need <= end) {
          const bool high = need <= middle;
          found[0] = high ? top : top - 1;
          found[1] = need - (high ? begin : middle);
          found[2] = high ? h[1] : h[0];
        }
        __syncthreads();
        need = found[1];
        among = found[2];
        const uint32_t bits = found[0] << shift, known = mask << shift;
        if (d < 3) {
          T |= bits;
          knownT |= known;
        } else {
          N |= bits;
          knownN |= known;
        }
      }
      if (need == among || d == kAllDigits - 1) {  // the threshold is there, or all of these stay: the digits left are zeros
        if (listed >= 0) break;
        what = kBits;
      } else if (listed < 0 && d < 2 && among <= static_cast<uint32_t>(L.candidates)) {
        what = kClassify;
      } else {
        ++d;
        what = kCount;
      }
    }

    // ---- which of the candidates stay ----
    if (listed >= 0) {
#pragma unroll 1
      for (int32_t e = tid; e < listed; e += kEvictThreads) {
        const uint2 x = candidates[e];
        bool stays = x.x > T || (x.x == T && x.y >= N);
        if (listed <= kFewCandidates) {  // no digits after the list
          uint32_t above = 0;
#pragma unroll 4
          for (int32_t o = 0; o < listed; ++o) {
            const uint2 y = candidates[o];
            above += y.x > x.x || (y.x == x.x && y.y > x.y);
          }
          stays = above < need;
        }
        const uint32_t j = ~x.y & n_mask;
        if (stays) atomicOr(reinterpret_cast<uint32_t*>(kept) + j / 32, 1u << (j % 32));
      }
      __syncthreads();
    }

    // ---- ranks: gaps below the budget and kept tokens behind it ----
    const int32_t words = (c + 63) / 64, groups = (words + kGroupWords - 1) / kGroupWords;
    auto gaps_of = [&](int32_t w) { return ~kept[w] & low_bits(b - 64 * w); };
    auto movers_of = [&](int32_t w) { return kept[w] & ~low_bits(b - 64 * w); };
    static_assert((1 << 18) / (64 * kGroupWords) <= kEvictThreads && kEvictMaxWidth <= 1 << 18, "a thread to a group");
    uint32_t gaps = 0, movers = 0;
#pragma unroll
    for (int e = 0; e < kGroupWords; ++e) {
      const int32_t w = min(tid * kGroupWords + e, words - 1);
      const bool on = tid * kGroupWords + e < words;
      gaps += on ? __popcll(gaps_of(w)) : 0;
      movers += on ? __popcll(movers_of(w)) : 0;
    }
    const uint32_t gap_end = wave_scan(gaps), mover_end = wave_scan(movers);
    if (lane == kWave - 1) {
      sums[0][wave] = gap_end;
      sums[1][wave] = mover_end;
    }
    __syncthreads();
    const uint32_t gap_sums = wave_scan(lane < kEvictWaves ? sums[0][lane] : 0);
    const uint32_t mover_sums = wave_scan(lane < kEvictWaves ? sums[1][lane] : 0);
    const uint32_t gap0 = gap_end - gaps + (wave > 0 ? __builtin_amdgcn_readlane(gap_sums, wave - 1) : 0);
    const uint32_t mover0 = mover_end - movers + (wave > 0 ? __builtin_amdgcn_readlane(mover_sums, wave - 1) : 0);
    // both sums are the same, and fit the lists; the least, so that every entry read below has been written
    moves = static_cast<int32_t>(min(static_cast<uint32_t>(A.max_moves), min(last_lane(gap_sums), last_lane(mover_sums))));
    // a group's base: of its gaps where it lies below the budget or holds it (no kept token lies
    // behind the budget before it), else of its movers
    const int32_t middle = b / (64 * kGroupWords);
    if (tid < groups) rank0[tid] = tid <= middle ? gap0 : mover0;
    __syncthreads();

    // ---- the lists, of indexes for now: a wave takes a group, its tokens in order ----
    int32_t* src = A.move_src + list;
    int32_t* dst = A.move_dst + list;
    const uint32_t last = static_cast<uint32_t>(A.max_moves) - 1;  // (scores that another stream changes meanwhile could make more)
#pragma unroll 1
    for (int32_t g = wave; g < groups; g += kEvictWaves) {
      uint64_t word[kGroupWords];
#pragma unroll
      for (int e = 0; e < kGroupWords; ++e) word[e] = uniform_word(kept[g * kGroupWords + e]);
      uint32_t base = uniform(static_cast<int32_t>(rank0[g]));
      auto write = [&](int32_t* to, uint64_t marks, int32_t w) {
        if (__builtin_amdgcn_inverse_ballot_w64(marks)) to[min(rank_in(marks, base), last)] = w * 64 + lane;
        base += __popcll(marks);
      };
      if (g <= middle) {
#pragma unroll
        for (int e = 0; e < kGroupWords; ++e) {
          const int32_t w = g * kGroupWords + e;
          write(dst, ~word[e] & (g < middle ? ~0ull : low_bits(b - 64 * w)), w);
        }
        base = 0;  // of the movers in the group that holds the budget
      }
      if (g >= middle) {
#pragma unroll
        for (int e = 0; e < kGroupWords; ++e) {
          const int32_t w = g * kGroupWords + e;
          write(src, word[e] & (g > middle ? ~0ull : ~low_bits(b - 64 * w)), w);
        }
      }
    }
  }

  // ---- scores and positions of the tokens that stay where they are ----
  const int32_t n = row.ok ? b : 0;
  constexpr int N = kKeys / 2;
#pragma unroll 1
  for (int32_t j0 = 0; j0 < n; j0 += N * kEvictThreads) {
    float s[N];
    int32_t p[N];
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] = score[min(j0 + k * kEvictThreads + tid, n - 1)];
    if (j0 < row.settled) {
#pragma unroll
      for (int k = 0; k < N; ++k) p[k] = token_pos[min(j0 + k * kEvictThreads + tid, n - 1)];
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int32_t j = j0 + k * kEvictThreads + tid;
      if (j < n && (!row.cut || (kept[j / 64] >> lane & 1))) {
        A.score_out[at + j] = s[k];
        A.token_pos_out[at + j] = j < row.settled ? p[k] : j + row.gone;
      }
    }
  }
  __syncthreads();  // the lists are there for the whole workgroup

  // ---- moves ----
  const int32_t* table = A.block_table + static_cast<size_t>(i) * A.max_pages;
  constexpr int M = 2;
#pragma unroll 1
  for (int32_t m0 = tid; m0 < moves; m0 += M * kEvictThreads) {
    int32_t j[M][2], p[M], e[M][2], page[M][2];  // source and destination
    float s[M];
#pragma unroll
    for (int k = 0; k < M; ++k) {
      // past the last pair this thread's own first one again: other entries become slots under way
      const int32_t m = m0 + k * kEvictThreads < moves ? m0 + k * kEvictThreads : m0;
      j[k][0] = A.move_src[list + m];
      j[k][1] = A.move_dst[list + m];
    }
#pragma unroll
    for (int k = 0; k < M; ++k) {
      s[k] = score[j[k][0]];
      p[k] = token_pos[j[k][0]];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        e[k][o] = static_cast<int32_t>(__umulhi(static_cast<uint32_t>(j[k][o]) / 16 * 2, L.page_m));
        page[k][o] = table[e[k][o]];
      }
    }
#pragma unroll
    for (int k = 0; k < M; ++k) {
      const int32_t m = m0 + k * kEvictThreads;
      if (m < moves) {
        int32_t slot[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const bool ok = page[k][o] >= 0 && page[k][o] < A.n_pages;
          slot[o] = ok ? page[k][o] * A.page + (j[k][o] - e[k][o] * A.page) : -1;
        }
        int32_t from = j[k][0];
        if (slot[0] < 0 || slot[1] < 0) {  // not moved: the gap keeps what it holds
          report_error(A.dev_err, GDN_DEV_BAD_PAGE);
          from = j[k][1];
          s[k] = score[from];
          p[k] = token_pos[from];
        }
        A.score_out[at + j[k][1]] = s[k];
        A.token_pos_out[at + j[k][1]] = from < row.settled ? p[k] : from + row.gone;
        A.move_src[list + m] = slot[0];
        A.move_dst[list + m] = slot[1];
      }
    }
  }
#pragma unroll 1
  for (int32_t m = moves + tid; m < A.max_moves; m += kEvictThreads) A.move_src[list + m] = A.move_dst[list + m] = -1;

  if (tid == 0) {
    A.n_moves[i] = moves;
    A.kv_len_out[i] = b;
    A.row_state_out[2 * i] = row.cut ? b : row.settled;
    A.row_state_out[2 * i + 1] = row.cut ? row.gone + (c - b) : row.gone;
  }
}

// How the pieces (16 bytes of K and of V) of moves lie: vph of a head, a power of two, vpt of a token.  A workgroup takes
// `moves` moves at a time; move = e / vpt of piece e is (e vpt_m) >> 32 (0: one move), page = slot / page tokens is
// (slot page_m) >> (32 + page_s).
struct MovePlan {
  int32_t vph_bits, vpt, moves;
  uint32_t vpt_m, page_m, page_s;
};

constexpr int kMoveThreads = 256;

// K and V rows of the moves: 16 bytes of each per thread and step, a row's moves over the workgroups along x.
//
// Bound by bytes, for few moves by two loads behind one another.  64 rows of up to 2048 moves, 468 MB in pieces of
// 256 bytes: 97 us, 4.8 TB/s; 4 rows of 128 moves 3 us in a graph of such calls.  Up to 8192 workgroups in all: 4096 103,
// 16384 93, but a call of 64 rows with room for 2048 moves and none to do takes 3.4 us, then 2.6 and 5.1.  Measured and
// dropped: two or four pieces of a thread under way at once 102 - 103; the moves of all rows on a line that is cut
// evenly 96 - 101, and 9 - 13 instead of 9 for 256 rows of 2 moves.
__global__ __launch_bounds__(kMoveThreads) void kv_move_kernel(MoveArgs A, MovePlan P) {
  const int i = blockIdx.y;
  const int32_t count = A.n_moves[i];
  if (count < 0 || count > A.max_moves) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(A.dev_err, GDN_DEV_BAD_LENGTH);
    return;
  }
  const int64_t cap = static_cast<int64_t>(A.n_pages) * A.page;
  const size_t list = static_cast<size_t>(i) * A.max_moves;
  for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * P.moves; m0 < count; m0 += static_cast<int64_t>(gridDim.x) * P.moves) {
    const int64_t left = count - m0;
    const uint32_t pieces = (left < P.moves ? static_cast<int32_t>(left) : P.moves) * P.vpt;
    for (uint32_t e = threadIdx.x; e < pieces; e += kMoveThreads) {
      const uint32_t m = static_cast<uint32_t>((static_cast<uint64_t>(e) * P.vpt_m) >> 32), v = e - m * P.vpt;
      const uint32_t h = v >> P.vph_bits, w = v & ((1u << P.vph_bits) - 1);
      const int32_t src = A.move_src[list + m0 + m], dst = A.move_dst[list + m0 + m];
      if (src < 0 || src >= cap || dst < 0 || dst >= cap) {
        if ((src < -1 || src >= cap) || (dst < -1 || dst >= cap)) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
        continue;
      }
      auto place = [&](uint32_t slot) {
        const uint32_t page = __umulhi(slot, P.page_m) >> P.page_s, off = slot - page * A.page;
        return ((static_cast<size_t>(page) * A.heads + h) * A.page + off) * A.row_bytes + 16 * w;
      };
      const size_t from = place(src), to = place(dst);
      const uint4 kv = *reinterpret_cast<const uint4*>(static_cast<const char*>(A.k_cache) + from);
      const uint4 vv = *reinterpret_cast<const uint4*>(static_cast<const char*>(A.v_cache) + from);
      *reinterpret_cast<uint4*>(static_cast<char*>(A.k_cache) + to) = kv;
      *reinterpret_cast<uint4*>(static_cast<char*>(A.v_cache) + to) = vv;
    }
  }
}

int launch_evict_plan(const EvictArgs& a, void* stream) {
  EvictPlan l{};
  l.words = (a.width + 1023) / 1024 * (4 * kGroupWords);  // what follows the ranks is 16-byte aligned
  const size_t fixed = static_cast<size_t>(l.words) * (sizeof(uint64_t) + sizeof(uint32_t) / kGroupWords) +
                       kDigits * kCopies * sizeof(uint32_t);
  static_assert((kEvictMaxWidth / 64) * 9 + kDigits * kCopies * 4 + kFewCandidates * 8 + 8 < kEvictLds, "the longest rows fit");
  const size_t room = (kEvictLds - fixed) / sizeof(uint2) - 1, most = room < kMaxCandidates ? room : kMaxCandidates;
  l.candidates = static_cast<int32_t>(static_cast<size_t>(a.width) < most ? a.width : most);
  // in units of 16 tokens: x / q = (2 x m) >> 32 with m = ceil(2^31 / q) for x (q - 1) < 2^31; x < 2^14, so
  // larger q give 0 as 2^14 does
  const uint32_t q = a.page / 16 < (1 << 14) ? a.page / 16 : 1 << 14;
  l.page_m = static_cast<uint32_t>(((1ull << 31) + q - 1) / q);
  hipLaunchKernelGGL(evict_plan_kernel, dim3(a.batch + 1), dim3(kEvictThreads), fixed + (l.candidates + 1) * sizeof(uint2),
                     static_cast<hipStream_t>(stream), a, l);
  return static_cast<int>(hipGetLastError());
}

int launch_kv_move(const MoveArgs& a, void* stream) {
  MovePlan p{};
  const uint32_t vph = a.row_bytes / 16;  // 8, 16, 32 or 64
  p.vph_bits = 31 - __builtin_clz(vph);
  p.vpt = static_cast<int32_t>(vph) * a.heads;
  p.moves = p.vpt < kMoveThreads ? kMoveThreads / p.vpt : 1;
  // e / d = (e m) >> 32 with m = ceil(2^32 / d) for e and d up to kMoveThreads: m d exceeds 2^32 by less than d, so
  // e m / 2^32 exceeds e / d by less than e / 2^32 < 1 / d
  p.vpt_m = p.moves == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + p.vpt - 1) / p.vpt);
  // s / d = (s m) >> (31 + l) with 2^(l - 1) < d <= 2^l and m = ceil(2^(31 + l) / d) for s < 2^31: m d exceeds
  // 2^(31 + l) by less than d <= 2^l, so s m / 2^(31 + l) exceeds s / d by less than 1 / d
  const int l = 32 - __builtin_clz(a.page - 1);
  p.page_m = static_cast<uint32_t>(((1ull << (31 + l)) + a.page - 1) / a.page);
  p.page_s = l - 1;
  const int64_t all = (static_cast<int64_t>(a.max_moves) + p.moves - 1) / p.moves, most = 8192 / a.batch;  // batch <= kEvictMaxBatch = 4096
  hipLaunchKernelGGL(kv_move_kernel, dim3(static_cast<unsigned>(all < most ? all : most), a.batch), dim3(kMoveThreads), 0,
                     static_cast<hipStream_t>(stream), a, p);
  return static_cast<int>(hipGetLastError());
}

}  // namespace gdn
