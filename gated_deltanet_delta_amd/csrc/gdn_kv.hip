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
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int kPlanThreads = 256;

// Exclusive sum over the workgroup's threads; *total receives the whole sum.
// One barrier pair per call.
__device__ __forceinline__ int64_t block_exclusive(int64_t v, int64_t* scratch, int64_t* total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int64_t inc = v;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t up = __shfl_up(inc, d, kWave);
    if (lane >= d) inc += up;
  }
  __syncthreads();
  if (lane == kWave - 1) scratch[wave] = inc;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / kWave; ++w) {
    if (w < wave) base += scratch[w];
    all += scratch[w];
  }
  *total = all;
  return base + inc - v;
}

__device__ __forceinline__ int32_t clamp32(int64_t v) { return static_cast<int32_t>(v < INT32_MAX ? v : INT32_MAX); }

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
  __shared__ int64_t scratch[kPlanThreads / kWave];
  const int tid = threadIdx.x, B = A.batch, P = A.page;
  int32_t* tok0 = plan_lds;
  int32_t* need0 = tok0 + B + 1;
  int32_t* gone0 = need0 + B + 1;
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(tid * per, B), hi = min(lo + per, B);
  const int64_t most = static_cast<int64_t>(A.max_pages) * P;

  struct Row {
    int64_t n, need, gone;
    bool ok;
  };
  auto row = [&](int i) {
    const int64_t c = A.kv_len[i], n = A.new_len[i];
    Row r;
    r.ok = c >= 0 && n >= -1 && c + (n > 0 ? n : 0) <= most;
    r.n = n > 0 ? n : 0;
    const int64_t have = r.ok ? (c + P - 1) / P : 0;
    r.need = r.ok && n > 0 ? (c + n + P - 1) / P - have : 0;
    r.gone = r.ok && n == -1 ? have : 0;
    return r;
  };
  int64_t sn = 0, sneed = 0, sgone = 0;
  bool all_ok = true;
  for (int i = lo; i < hi; ++i) {
    const Row r = row(i);
    sn += r.n;
    sneed += r.need;
    sgone += r.gone;
    all_ok &= r.ok;
  }
  int64_t tn, tneed, tgone;
  int64_t en = block_exclusive(sn, scratch, &tn);
  int64_t eneed = block_exclusive(sneed, scratch, &tneed);
  int64_t egone = block_exclusive(sgone, scratch, &tgone);
  for (int i = lo; i < hi; ++i) {
    const Row r = row(i);
    tok0[i] = clamp32(en);
    need0[i] = clamp32(eneed);
    gone0[i] = clamp32(egone);
    en += r.n;
    eneed += r.need;
    egone += r.gone;
  }
  if (tid == 0) {
    tok0[B] = clamp32(tn);
    need0[B] = clamp32(tneed);
    gone0[B] = clamp32(tgone);
  }
  const int32_t f0 = *A.n_free;
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
  // the row gets its pages (a row's need and its start are exact below INT32_MAX)
  auto served = [&](int i, int64_t need) { return stack_ok && (need == 0 || need0[i] + need <= top); };

  const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;
  // ---- rows: lengths, offsets ----
  for (int i = gtid; i < B; i += gsize) {
    const Row r = row(i);
    const int32_t c = A.kv_len[i];
    A.cu_new[i] = min(tok0[i], A.max_tokens);
    A.kv_len_out[i] = !r.ok || !served(i, r.need) ? c : (A.new_len[i] < 0 ? 0 : c + static_cast<int32_t>(r.n));
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
    for (int t = gtid; t < A.max_tokens; t += gsize) {
      A.slot_map[t] = -1;
      A.position[t] = 0;
    }
    return;
  }
  // ---- pages given back: onto the stack ----
  for (int r = gtid; r < gone; r += gsize) A.free_pages[f0 + r] = given_back(r);
  // ---- new pages into the block tables ----
  const int32_t pages = clamp32(tneed < top ? tneed : top);
  for (int m = gtid; m < pages; m += gsize) {
    const int i = row_of(need0, B, m);
    const Row r = row(i);
    if (!served(i, r.need)) continue;
    const int32_t have = static_cast<int32_t>((static_cast<int64_t>(A.kv_len[i]) + P - 1) / P);
    A.block_table[static_cast<size_t>(i) * A.max_pages + have + (m - need0[i])] = stack_at(top - 1 - m);
  }
  // ---- slots and positions of the new tokens ----
  const int32_t total = min(tok0[B], A.max_tokens);
  for (int t = gtid; t < A.max_tokens; t += gsize) {
    int32_t slot = -1, pos = 0;
    if (t < total) {
      const int i = row_of(tok0, B, t);
      const Row r = row(i);
      if (r.ok) {
        const int32_t c = A.kv_len[i];
        pos = c + (t - tok0[i]);
        if (served(i, r.need)) {
          const int32_t have = static_cast<int32_t>((static_cast<int64_t>(c) + P - 1) / P), e = pos / P;
          const int32_t page = e < have ? A.block_table[static_cast<size_t>(i) * A.max_pages + e]
                                        : stack_at(top - 1 - (need0[i] + (e - have)));
          if (page >= 0 && page < A.n_pages) slot = page * P + pos % P;
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
  // one workgroup per 1024 tokens or rows, at most one per CU: every workgroup
  // scans all rows' lengths first
  const int64_t items = static_cast<int64_t>(a.max_tokens) > a.batch ? a.max_tokens : a.batch;
  int64_t wgs = (items + 1023) / 1024;
  if (wgs < 1) wgs = 1;
  if (wgs > 256) wgs = 256;
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
