// Device helpers shared by the attention kernels (gdn_attn.hip, gdn_attn_bf16.hip):
// the sequences of a call, the rows of its keys, and partial results.
#pragma once

#include "gdn_device.h"
#include "gdn_ops.h"

namespace gdn {

// One sequence as a workgroup sees it.
struct Seq {
  int64_t row0;   // its first token among the call's
  int32_t n;      // its tokens (0: nothing to do)
  int32_t ctx;    // its cached tokens
  int32_t index;  // block-table row
};

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ Seq uniform(Seq q) {
  return Seq{uniform(q.row0), uniform(q.n), uniform(q.ctx), uniform(q.index)};
}

// Cached tokens of sequence s; false (and reported) if they do not fit the table.
__device__ __forceinline__ bool seq_ctx(const AttnArgs& A, int s, int32_t* ctx, bool report) {
  const int32_t c = A.ctx_len ? A.ctx_len[s] : 0;
  *ctx = c;
  if (c >= 0 && c <= static_cast<int64_t>(A.max_pages) * A.page) return true;
  if (report) report_error(A.dev_err, GDN_DEV_BAD_LENGTH);
  return false;
}

// Sequence s of a packed batch; n = 0 for one whose description is refused.
__device__ __forceinline__ Seq packed_seq(const AttnArgs& A, int s, bool report) {
  Seq q{0, 0, 0, s};
  const int32_t t0 = A.cu_seqlens[s], t1 = A.cu_seqlens[s + 1];
  if (t0 < 0 || t1 < t0 || t1 > A.n_tokens || A.cu_seqlens[0] != 0) {
    if (report) report_error(A.dev_err, GDN_DEV_BAD_SEQLENS);
    return q;
  }
  if (!seq_ctx(A, s, &q.ctx, report)) return q;
  q.row0 = t0;
  q.n = t1 - t0;
  return q;
}

// Row s of a batch of trees (all lanes of a wave call it together); n = 0 for
// one whose description is refused.  *path receives, in lane j, the bits of
// node j's path (its ancestors and itself).
__device__ __forceinline__ Seq tree_seq(const AttnArgs& A, int s, bool report, uint64_t* path) {
  const int lane = threadIdx.x & (kWave - 1);
  Seq q{0, 0, 0, s};
  const int32_t n = A.n_row ? A.n_row[s] : A.nodes;
  if (n < 1 || n > A.nodes) {
    if (report) report_error(A.dev_err, GDN_DEV_BAD_K);
    return q;
  }
  int par = lane < n ? A.parent[static_cast<size_t>(s) * A.nodes + lane] : -1;
  if (__ballot(par < -1 || (lane < n && par >= lane)) != 0) {
    if (report) report_error(A.dev_err, GDN_DEV_BAD_PARENT);
    return q;
  }
  // pointer doubling: after step i, bits of the 2^(i+1) nearest nodes of the path
  uint64_t bits = 1ull << lane;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const int src = par < 0 ? lane : par;
    const uint32_t lo = __shfl(static_cast<uint32_t>(bits), src, kWave);
    const uint32_t hi = __shfl(static_cast<uint32_t>(bits >> 32), src, kWave);
    const int up = __shfl(par, src, kWave);
    if (par >= 0) {
      bits |= (static_cast<uint64_t>(hi) << 32) | lo;
      par = up;
    }
  }
  *path = bits;
  if (!seq_ctx(A, s, &q.ctx, report)) return q;
  q.row0 = static_cast<int64_t>(s) * A.nodes;
  q.n = n;
  return q;
}

// Last sequence s with begins(cu_seqlens[s], s), a condition that no sequence
// meets after one that does not, of those up to the first that ends before it
// begins (which is refused, and so are those behind it: their bounds are in no
// order); 0 if none meets it.  All lanes of a wave together.
template <class F>
__device__ __forceinline__ int last_seq(const AttnArgs& A, F begins) {
  const int lane = threadIdx.x & (kWave - 1);
  int s = 0;
  for (int base = 0; base < A.n_seqs; base += kWave) {
    const int i = min(base + lane, A.n_seqs - 1);
    const bool in = base + lane < A.n_seqs;
    const int32_t t0 = A.cu_seqlens[i], t1 = A.cu_seqlens[i + 1];
    const uint64_t back = __ballot(in && t1 < t0);
    const uint64_t on = __ballot(in && begins(t0, i)) & (back ^ (back - 1));  // all lanes if none goes back
    if (on != 0) s = base + 63 - __builtin_clzll(on);
    if (on == 0 || back != 0) break;
  }
  return s;
}

// Row tiles of a packed batch: sequence s owns the tile ids from
// floor(cu[s] G / BM) + s on, at least ceil(n_s G / BM) of them, so a tile id
// finds its sequence without sums over the sequences before it.  Finds the
// last s with a first id <= id (all lanes of a wave together).
__device__ __forceinline__ int64_t tile_start(const AttnArgs& A, int s, int bm) {
  const int64_t t = A.cu_seqlens[s];
  return (t > 0 ? t : 0) * A.G / bm + s;
}
__device__ __forceinline__ int find_seq(const AttnArgs& A, int64_t id, int bm) {
  return last_seq(A, [&](int32_t t0, int i) { return (t0 > 0 ? static_cast<int64_t>(t0) : 0) * A.G / bm + i <= id; });
}

// The address of the K (or V) row of key j: in its page, or among the call's rows.
template <int ES>
__device__ __forceinline__ const char* key_row(const AttnArgs& A, const Seq& q, const void* cache, const void* fresh,
                                               int64_t stride, int kvh, int32_t j) {
  if (j < q.ctx) {
    const int32_t e = j / A.page, off = j - e * A.page;
    int32_t page = A.block_table[static_cast<size_t>(q.index) * A.max_pages + e];
    if (page < 0 || page >= A.n_pages) {
      report_error(A.dev_err, GDN_DEV_BAD_PAGE);
      page = 0;
    }
    return static_cast<const char*>(cache) +
           ((static_cast<size_t>(page) * A.Hk + kvh) * A.page + off) * static_cast<size_t>(A.D) * ES;
  }
  return static_cast<const char*>(fresh) +
         ((q.row0 + (j - q.ctx)) * stride + static_cast<int64_t>(kvh) * A.D) * ES;
}

// Whether any of the 16 bytes' elements is an infinity or a NaN.
template <bool BF16>
__device__ __forceinline__ bool any_nonfinite(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    else bad |= (w[i] & 0x7f800000u) == 0x7f800000u;
  }
  return bad;
}

}  // namespace gdn
