// Eviction from the paged KV cache for gfx950: which of a row's tokens stay, and the
// moves that close the gaps.
//
// Plan.  Each token j of a row has a key, its score as an unsigned integer of the same
// order, the largest for protected tokens; the b that stay are those above the b-th
// largest key T and, among the tokens with key T, the first by index.  T comes from
// counts of the keys' upper 11, middle 11 and lower 10 bits, each of the tokens that
// agree with T in the bits before.  The kept tokens behind the budget fill the gaps
// below it, both in order, so their numbers are ranks within two ballots: a row that
// loses e tokens moves min(b, e) at most, whatever its length.
//
// A workgroup plans one row.  Its keys stay in LDS up to 32768 tokens; the rest are made
// again from the scores in each of the five passes.  Bound by those passes: scores and
// positions are read once or from the L2.
#include "gdn_attn_device.h"

namespace gdn {

namespace {

constexpr int kEvictThreads = 1024, kEvictWaves = kEvictThreads / kWave;
constexpr int kLdsKeys = 32768;
constexpr uint32_t kZeroKey = 0x80000000u, kProtected = 0xffffffffu;

// A score as an unsigned integer of the same order: NaN lowest, -0 = 0.
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t bits = s == 0.f ? 0u : __float_as_uint(s);
  if (s != s) return 0;
  return bits >> 31 ? ~bits : bits | 0x80000000u;
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
__device__ __forceinline__ int32_t pages_of(int32_t tokens, int32_t page) {
  return static_cast<int32_t>((static_cast<uint32_t>(tokens) + page - 1) / page);
}

}  // namespace

__global__ __launch_bounds__(kEvictThreads) void evict_plan_kernel(EvictArgs A) {
  extern __shared__ uint32_t lds_keys[];
  __shared__ uint32_t hist[2048];
  __shared__ int64_t sums[kEvictWaves][2];
  __shared__ uint32_t waves[kEvictWaves][2];
  __shared__ uint32_t found[2];
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = uniform(tid / kWave);
  const uint64_t below = (1ull << lane) - 1;

  // ---- freed pages of the rows before this one, and of all ----
  int64_t before = 0, total = 0;
  for (int r = tid; r < A.batch; r += kEvictThreads) {
    const EvictRow w = evict_row(A, r, false);
    const int64_t pages = w.cut ? pages_of(w.c, A.page) - pages_of(w.b, A.page) : 0;
    total += pages;
    before += r < i ? pages : 0;
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    total += __shfl_xor(total, d, kWave);
    before += __shfl_xor(before, d, kWave);
  }
  if (lane == 0) {
    sums[wave][0] = total;
    sums[wave][1] = before;
  }
  __syncthreads();
  total = before = 0;
#pragma unroll
  for (int w = 0; w < kEvictWaves; ++w) {
    total += sums[w][0];
    before += sums[w][1];
  }
  const int32_t nf = *A.n_free;
  const bool stack_ok = nf >= 0 && nf + total <= A.n_pages;
  EvictRow row = evict_row(A, i, tid == 0);
  if (!stack_ok) row.cut = false;
  const int32_t c = row.c, b = row.cut ? row.b : c;
  if (tid == 0) {
    if (i == 0) {
      *A.n_free_out = stack_ok ? static_cast<int32_t>(nf + total) : nf;
      if (!stack_ok) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
    }
    A.kv_len_out[i] = b;
    A.row_state_out[2 * i] = row.cut ? b : row.settled;
    A.row_state_out[2 * i + 1] = row.cut ? row.gone + (c - b) : row.gone;
    if (!row.cut) A.n_moves[i] = 0;
  }
  const size_t at = static_cast<size_t>(i) * A.width, list = static_cast<size_t>(i) * A.max_moves;
  const int32_t* table = A.block_table + static_cast<size_t>(i) * A.max_pages;
  auto position = [&](int32_t j) { return j < row.settled ? A.token_pos[at + j] : j + row.gone; };
  if (!row.cut) {
    for (int32_t j = tid; row.ok && j < c; j += kEvictThreads) {
      const int32_t p = position(j);
      A.score_out[at + j] = A.score[at + j];
      A.token_pos_out[at + j] = p;
    }
    for (int32_t m = tid; m < A.max_moves; m += kEvictThreads) A.move_src[list + m] = A.move_dst[list + m] = -1;
    return;
  }

  // ---- keys ----
  const int64_t recent_from = static_cast<int64_t>(c) + row.gone - A.recent;
  auto make_key = [&](int32_t j) {
    const int32_t p = position(j);
    return p < A.sink || p >= recent_from ? kProtected : score_key(A.score[at + j]);
  };
  const int32_t in_lds = min(c, kLdsKeys);
  for (int32_t j = tid; j < in_lds; j += kEvictThreads) lds_keys[j] = make_key(j);
  __syncthreads();
  auto key_at = [&](int32_t j) { return j < kLdsKeys ? lds_keys[j] : make_key(j); };

  // ---- the b-th largest key, and how many of its equals stay ----
  uint32_t T = 0, need = b;
  if (b == 0) {
    T = kProtected;
  } else {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
      const uint32_t known = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
      for (int e = tid; e < 2048; e += kEvictThreads) hist[e] = 0;
      __syncthreads();
      for (int32_t j0 = wave * kWave; j0 < c; j0 += kEvictThreads) {
        const int32_t j = j0 + lane;
        const uint32_t key = j < c ? key_at(j) : 0;
        const bool in = j < c && ((key ^ T) & known) == 0;
        // the two keys that many tokens share take one addition per wave
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t often = k == 0 ? kZeroKey : kProtected;
          const uint64_t same = __ballot(in && key == often);
          if (same != 0 && lane == 0) atomicAdd(&hist[(often >> shift) & (bins - 1)], __popcll(same));
        }
        if (in && key != kZeroKey && key != kProtected) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // from the highest bin down, two per thread
      const int top = bins - 1 - 2 * tid;
      const uint32_t h0 = top >= 0 ? hist[top] : 0, h1 = top >= 1 ? hist[top - 1] : 0;
      uint32_t inc = h0 + h1;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t up = __shfl_up(inc, d, kWave);
        if (lane >= d) inc += up;
      }
      if (lane == kWave - 1) waves[wave][0] = inc;
      __syncthreads();
      uint32_t start = inc - h0 - h1;
      for (int w = 0; w < wave; ++w) start += waves[w][0];
      if (start < need && need <= start + h0) {
        found[0] = top;
        found[1] = need - start;
      } else if (start + h0 < need && need <= start + h0 + h1) {
        found[0] = top - 1;
        found[1] = need - start - h0;
      }
      __syncthreads();
      T |= found[0] << shift;
      need = found[1];
    }
  }

  // ---- ranks: a wave takes a run of tokens, 64 at a time ----
  const int32_t run = static_cast<int32_t>((static_cast<uint32_t>(c) + kEvictThreads - 1) / kEvictThreads) * kWave;
  const int64_t from = static_cast<int64_t>(wave) * run;
  const int32_t lo = static_cast<int32_t>(from < c ? from : c), hi = static_cast<int32_t>(from + run < c ? from + run : c);
  uint32_t equals = 0;
  for (int32_t j0 = lo; j0 < hi; j0 += kWave) equals += __popcll(__ballot(j0 + lane < c && key_at(j0 + lane) == T));
  if (lane == 0) waves[wave][0] = equals;
  __syncthreads();
  uint32_t equal0 = 0;
  for (int w = 0; w < wave; ++w) equal0 += waves[w][0];
  __syncthreads();
  // f(j, within the row, kept) for the run
  auto walk = [&](auto f) {
    uint32_t rank0 = equal0;
    for (int32_t j0 = lo; j0 < hi; j0 += kWave) {
      const int32_t j = j0 + lane;
      const uint32_t key = j < c ? key_at(j) : 0;
      const uint64_t same = __ballot(j < c && key == T);
      f(j, j < c, j < c && (key > T || (key == T && rank0 + __popcll(same & below) < need)));
      rank0 += __popcll(same);
    }
  };
  uint32_t holes = 0, movers = 0;
  walk([&](int32_t j, bool in, bool keep) {
    holes += __popcll(__ballot(in && j < b && !keep));
    movers += __popcll(__ballot(j >= b && keep));
  });
  if (lane == 0) {
    waves[wave][0] = holes;
    waves[wave][1] = movers;
  }
  __syncthreads();
  uint32_t hole0 = 0, mover0 = 0, count = 0;
  for (int w = 0; w < kEvictWaves; ++w) {
    if (w < wave) {
      hole0 += waves[w][0];
      mover0 += waves[w][1];
    }
    count += waves[w][0];
  }
  // the lists, of indexes for now; what stays where it is
  walk([&](int32_t j, bool in, bool keep) {
    const bool hole = in && j < b && !keep, mover = j >= b && keep;
    const uint64_t hs = __ballot(hole), ms = __ballot(mover);
    if (hole) A.move_dst[list + hole0 + __popcll(hs & below)] = j;
    if (mover) A.move_src[list + mover0 + __popcll(ms & below)] = j;
    if (keep && j < b) {
      const int32_t p = position(j);
      A.score_out[at + j] = A.score[at + j];
      A.token_pos_out[at + j] = p;
    }
    hole0 += __popcll(hs);
    mover0 += __popcll(ms);
  });
  __syncthreads();  // the lists are there for the whole workgroup

  // ---- moves ----
  auto slot_of = [&](int32_t j) {
    const int32_t e = j / A.page, page = table[e];
    if (page < 0 || page >= A.n_pages) {
      report_error(A.dev_err, GDN_DEV_BAD_PAGE);
      return -1;
    }
    return page * A.page + (j - e * A.page);
  };
  for (int32_t m = tid; m < A.max_moves; m += kEvictThreads) {
    int32_t src = -1, dst = -1;
    if (m < static_cast<int32_t>(count)) {
      const int32_t j = A.move_src[list + m], h = A.move_dst[list + m], p = position(j);
      A.score_out[at + h] = A.score[at + j];
      A.token_pos_out[at + h] = p;
      src = slot_of(j);
      dst = slot_of(h);
    }
    A.move_src[list + m] = src;
    A.move_dst[list + m] = dst;
  }
  if (tid == 0) A.n_moves[i] = static_cast<int32_t>(count);

  // ---- pages behind the budget: onto the stack ----
  const int32_t first = pages_of(b, A.page), freed = pages_of(c, A.page) - first;
  for (int32_t e = tid; e < freed; e += kEvictThreads) {
    const int32_t page = table[first + e];
    if (page < 0 || page >= A.n_pages) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
    A.free_pages[nf + before + e] = page;
  }
}

// K and V rows of the moves: 16 bytes of each per thread and step, a row's moves over
// the workgroups along x.
__global__ __launch_bounds__(256) void kv_move_kernel(MoveArgs A) {
  const int i = blockIdx.y;
  const int32_t count = A.n_moves[i];
  if (count < 0 || count > A.max_moves) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(A.dev_err, GDN_DEV_BAD_LENGTH);
    return;
  }
  const int vph = A.row_bytes / 16, vpt = vph * A.heads;  // vectors of one head, of one token
  const int64_t total = static_cast<int64_t>(count) * vpt, cap = static_cast<int64_t>(A.n_pages) * A.page;
  const size_t list = static_cast<size_t>(i) * A.max_moves;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total; e += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t m = e / vpt;
    const int v = static_cast<int>(e - m * vpt), h = v / vph, w = v - h * vph;
    const int32_t src = A.move_src[list + m], dst = A.move_dst[list + m];
    if (src < 0 || src >= cap || dst < 0 || dst >= cap) {
      if ((src < -1 || src >= cap) || (dst < -1 || dst >= cap)) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
      continue;
    }
    auto place = [&](int32_t slot) {
      const int32_t page = slot / A.page, off = slot - page * A.page;
      return ((static_cast<size_t>(page) * A.heads + h) * A.page + off) * A.row_bytes + 16 * w;
    };
    const size_t from = place(src), to = place(dst);
    const uint4 kv = *reinterpret_cast<const uint4*>(static_cast<const char*>(A.k_cache) + from);
    const uint4 vv = *reinterpret_cast<const uint4*>(static_cast<const char*>(A.v_cache) + from);
    *reinterpret_cast<uint4*>(static_cast<char*>(A.k_cache) + to) = kv;
    *reinterpret_cast<uint4*>(static_cast<char*>(A.v_cache) + to) = vv;
  }
}

int launch_evict_plan(const EvictArgs& a, void* stream) {
  const size_t lds = static_cast<size_t>(a.width < kLdsKeys ? a.width : kLdsKeys) * sizeof(uint32_t);
  hipLaunchKernelGGL(evict_plan_kernel, dim3(a.batch), dim3(kEvictThreads), lds, static_cast<hipStream_t>(stream), a);
  return static_cast<int>(hipGetLastError());
}

int launch_kv_move(const MoveArgs& a, void* stream) {
  const int64_t total = static_cast<int64_t>(a.max_moves) * a.heads * (a.row_bytes / 16);
  int64_t wgs = (total + 255) / 256;
  const int64_t most = a.batch < 4096 ? 4096 / a.batch : 1;
  if (wgs > most) wgs = most;
  hipLaunchKernelGGL(kv_move_kernel, dim3(static_cast<unsigned>(wgs), a.batch), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace gdn
