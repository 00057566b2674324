// The paged KV cache's bookkeeping and writes for gfx950.
//
// Plan: block tables and slot maps from the requests' lengths.  With
//   need_i = ceil((c_i + n_i) / P) - ceil(c_i / P)   (0 for a leaving row),
//   gone_i = ceil(c_i / P) for a leaving row, else 0,
// and exclusive sums N, E, L of need, gone and n over the rows, the free stack
// is F[0..f) followed by the leaving rows' pages, its top is f + sum gone, and
// the m-th new page of the call (m = N_i + j) is stack[top - 1 - m].  Every
// value follows from the lengths alone, so each workgroup computes the sums
// itself (they fit its LDS) and no workgroup waits for another.
//
// Both kernels are bound by latency where they are small: the plan by its chain
// of reads (lengths, sums, a search of the token's row, lengths, page), 4
// requests 3.6 us in a graph, 512 requests with tens of thousands of slots 7.7 us.  (Sums
// in 64 bits, divisions in 64 bits and 1024 tokens per workgroup: 5.2 and 16.3
// us.)  The write moves 16 bytes per thread and step: 32771 tokens of 4 heads,
// d 256, bf16 (268 MB read and written) 53 us, 5.1 TB/s, above the rate of a
// large copy; 4 tokens 2.2 us.
#include "gdn_device.h"
#include "gdn_ops.h"

namespace gdn {

namespace {

constexpr int kPlanThreads = 256;

// Sum of two values in 0 .. INT32_MAX that stays at INT32_MAX (sums of such
// values are the same in every order).
__device__ __forceinline__ int32_t add_sat(int32_t a, int32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Exclusive sums over the workgroup's threads of N values; total receives the
// whole sums.  One barrier: scratch is the call's own.
template <int N>
__device__ __forceinline__ void block_exclusive(int32_t (&v)[N], int32_t (*scratch)[N], int32_t (&total)[N]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int32_t inc[N];
#pragma unroll
  for (int n = 0; n < N; ++n) inc[n] = v[n];
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int32_t up = __shfl_up(inc[n], d, kWave);
      if (lane >= d) inc[n] = add_sat(inc[n], up);
    }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (lane == kWave - 1) scratch[wave][n] = inc[n];
    const int32_t up = __shfl_up(inc[n], 1, kWave);
    v[n] = lane > 0 ? up : 0;
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    total[n] = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / kWave; ++w) {
      if (w == wave) v[n] = add_sat(total[n], v[n]);
      total[n] = add_sat(total[n], scratch[w][n]);
    }
  }
}

// Largest row i with start[i] <= v (start non-decreasing, start[0] <= v).
__device__ __forceinline__ int row_of(const int32_t* start, int rows, int32_t v) {
  int lo = 0, hi = rows;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(KvPlanArgs A) {
  extern __shared__ int32_t plan_lds[];  // [3][batch + 1]: new tokens, new pages, pages given back, before each row
  __shared__ int32_t scratch[kPlanThreads / kWave][3];
  const int tid = threadIdx.x, B = A.batch;
  const uint32_t P = A.page;
  int32_t* tok0 = plan_lds;
  int32_t* need0 = tok0 + B + 1;
  int32_t* gone0 = need0 + B + 1;
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(tid * per, B), hi = min(lo + per, B);
  const int32_t most = A.max_pages * static_cast<int32_t>(P);  // below 2^30
  const int32_t f0 = *A.n_free;

  auto row_ok = [&](int32_t c, int32_t n) { return c >= 0 && c <= most && n >= -1 && n <= most - c; };
  auto pages_of = [&](int32_t tokens) { return static_cast<int32_t>((static_cast<uint32_t>(tokens) + P - 1) / P); };
  int32_t sum[3] = {0, 0, 0}, all[3];
  bool all_ok = true;
  for (int i = lo; i < hi; ++i) {
    const int32_t c = A.kv_len[i], n = A.new_len[i];
    const bool ok = row_ok(c, n);
    const int32_t have = ok ? pages_of(c) : 0;
    all_ok &= ok;
    sum[0] = add_sat(sum[0], tok0[i] = max(n, 0));
    sum[1] = add_sat(sum[1], need0[i] = ok && n > 0 ? pages_of(c + n) - have : 0);
    sum[2] = add_sat(sum[2], gone0[i] = ok && n == -1 ? have : 0);
  }
  block_exclusive(sum, scratch, all);
  for (int i = lo; i < hi; ++i) {  // each thread's own rows: its values, then the sums before them
    const int32_t n = tok0[i], need = need0[i], leaves = gone0[i];
    tok0[i] = sum[0];
    need0[i] = sum[1];
    gone0[i] = sum[2];
    sum[0] = add_sat(sum[0], n);
    sum[1] = add_sat(sum[1], need);
    sum[2] = add_sat(sum[2], leaves);
  }
  if (tid == 0) {
    tok0[B] = all[0];
    need0[B] = all[1];
    gone0[B] = all[2];
  }
  const int64_t tn = all[0], tneed = all[1], tgone = all[2];  // INT32_MAX: that many or more
  const bool stack_ok = f0 >= 0 && f0 + tgone <= A.n_pages;
  const int32_t gone = stack_ok ? static_cast<int32_t>(tgone) : 0;
  const int64_t top = stack_ok ? f0 + gone : 0;  // pages on the stack
  const bool first = blockIdx.x == 0;
  if (first && !all_ok) report_error(A.dev_err, GDN_DEV_BAD_LENGTH);
  if (first && tid == 0) {
    if (!stack_ok) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
    if (tn > A.max_tokens) report_error(A.dev_err, GDN_DEV_BAD_SEQLENS);
    if (stack_ok && tneed > top) report_error(A.dev_err, GDN_DEV_NO_PAGES);
  }
  __syncthreads();

  // page r of those given back, and stack entry s
  auto given_back = [&](int32_t r) {
    const int i = row_of(gone0, B, r);
    return A.block_table[static_cast<size_t>(i) * A.max_pages + (r - gone0[i])];
  };
  auto stack_at = [&](int64_t s) { return s < f0 ? A.free_pages[s] : given_back(static_cast<int32_t>(s - f0)); };
  // row i (c cached, n new tokens, within limits) gets the pages that it needs:
  // need0[i + 1], where they end, is exact up to top, or it needs none
  auto served = [&](int i, int32_t c, int32_t n) {
    return stack_ok && (need0[i + 1] <= top || n <= 0 || pages_of(c + n) == pages_of(c));
  };

  const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;
  const uint32_t n_slots = A.max_tokens;  // up to 2^31 - 1, so its index has no sign: the step past the last entry takes 32 bits
  // ---- rows: lengths, offsets ----
  for (int i = gtid; i < B; i += gsize) {
    const int32_t c = A.kv_len[i], n = A.new_len[i];
    A.cu_new[i] = min(tok0[i], A.max_tokens);
    A.kv_len_out[i] = !row_ok(c, n) || !served(i, c, n) ? c : (n < 0 ? 0 : c + n);
  }
  if (gtid == 0) {
    A.cu_new[B] = min(tok0[B], A.max_tokens);
    int64_t used = 0;  // rows are served up to the first that does not fit
    if (stack_ok) {
      if (tneed <= top) used = tneed;
      else {  // the largest start among the rows that still fit, plus their need
        int l = 0, h = B;  // need0[l] <= top
        while (h - l > 1) {
          const int mid = (l + h) >> 1;
          if (need0[mid] <= top) l = mid;
          else h = mid;
        }
        used = need0[l];
      }
    }
    *A.n_free_out = stack_ok ? static_cast<int32_t>(top - used) : f0;
  }
  if (!stack_ok) {
    for (uint32_t t = gtid; t < n_slots; t += gsize) {
      A.slot_map[t] = -1;
      A.position[t] = 0;
    }
    return;
  }
  // ---- pages given back: onto the stack ----
  for (int r = gtid; r < gone; r += gsize) A.free_pages[f0 + r] = given_back(r);
  // ---- new pages into the block tables ----
  const int32_t pages = static_cast<int32_t>(tneed < top ? tneed : top);
  for (int m = gtid; m < pages; m += gsize) {
    const int i = row_of(need0, B, m);
    if (need0[i + 1] > top) continue;
    A.block_table[static_cast<size_t>(i) * A.max_pages + pages_of(A.kv_len[i]) + (m - need0[i])] = stack_at(top - 1 - m);
  }
  // ---- slots and positions of the new tokens ----
  const int32_t total = min(tok0[B], A.max_tokens);
  for (uint32_t at = gtid; at < n_slots; at += gsize) {
    const int32_t t = static_cast<int32_t>(at);
    int32_t slot = -1, pos = 0;
    if (t < total) {
      const int i = row_of(tok0, B, t);
      const int32_t c = A.kv_len[i], n = A.new_len[i];
      if (row_ok(c, n)) {
        pos = c + (t - tok0[i]);
        if (served(i, c, n)) {
          const int32_t have = pages_of(c), e = static_cast<int32_t>(static_cast<uint32_t>(pos) / P);
          const int32_t page = e < have ? A.block_table[static_cast<size_t>(i) * A.max_pages + e]
                                        : stack_at(top - 1 - (need0[i] + (e - have)));
          if (page >= 0 && page < A.n_pages) slot = page * static_cast<int32_t>(P) + (pos - e * static_cast<int32_t>(P));
          else report_error(A.dev_err, GDN_DEV_BAD_PAGE);
        }
      }
    }
    A.slot_map[t] = slot;
    A.position[t] = pos;
  }
}

// K and V rows to their cache slots: one 16-byte vector per thread and step.
__global__ __launch_bounds__(256) void kv_write_kernel(KvWriteArgs A) {
  const int vph = A.row_bytes / 16;          // vectors of one head
  const int vpt = vph * A.heads;             // vectors of one token
  const int64_t total = static_cast<int64_t>(A.n_tokens) * vpt;
  const int64_t cap = static_cast<int64_t>(A.n_pages) * A.page;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = e / vpt;
    const int c = static_cast<int>(e - t * vpt), h = c / vph, w = c - h * vph;
    const int32_t slot = A.slot_map[t];
    if (slot < 0 || slot >= cap) {
      if (slot != -1) report_error(A.dev_err, GDN_DEV_BAD_PAGE);
      continue;
    }
    const int32_t page = slot / A.page, off = slot - page * A.page;
    const size_t dst = ((static_cast<size_t>(page) * A.heads + h) * A.page + off) * A.row_bytes + 16 * w;
    const size_t src = static_cast<size_t>(h) * A.row_bytes + 16 * w;
    const uint4 kv = *reinterpret_cast<const uint4*>(static_cast<const char*>(A.k) + t * A.k_stride + src);
    const uint4 vv = *reinterpret_cast<const uint4*>(static_cast<const char*>(A.v) + t * A.v_stride + src);
    *reinterpret_cast<uint4*>(static_cast<char*>(A.k_cache) + dst) = kv;
    *reinterpret_cast<uint4*>(static_cast<char*>(A.v_cache) + dst) = vv;
  }
}

int launch_kv_plan(const KvPlanArgs& a, void* stream) {
  // one workgroup per 256 tokens or rows, at most two per CU: every workgroup
  // scans all rows' lengths first, and then has one chain of dependent reads
  // (search, lengths, page) per round of 256
  const int64_t items = static_cast<int64_t>(a.max_tokens) > a.batch ? a.max_tokens : a.batch;
  int64_t wgs = (items + kPlanThreads - 1) / kPlanThreads;
  if (wgs < 1) wgs = 1;
  if (wgs > 512) wgs = 512;
  const size_t lds = 3 * (static_cast<size_t>(a.batch) + 1) * sizeof(int32_t);
  hipLaunchKernelGGL(kv_plan_kernel, dim3(static_cast<unsigned>(wgs)), dim3(kPlanThreads), lds,
                     static_cast<hipStream_t>(stream), a);
  return static_cast<int>(hipGetLastError());
}

int launch_kv_write(const KvWriteArgs& a, void* stream) {
  const int64_t total = static_cast<int64_t>(a.n_tokens) * a.heads * (a.row_bytes / 16);
  int64_t wgs = (total + 255) / 256;
  if (wgs > 4096) wgs = 4096;
  hipLaunchKernelGGL(kv_write_kernel, dim3(static_cast<unsigned>(wgs)), dim3(256), 0, static_cast<hipStream_t>(stream),
                     a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace gdn
