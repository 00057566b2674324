// Verify over a tree of drafts for gfx950: the gated delta rule from every
// node's parent,
//   S_j = alpha_j S_p (I - beta_j k_j k_j^T) + beta_j v_j k_j^T,  o_j = S_j q_j,
// each node's state, conv window and position written to a pool slot of its own.
//
// Per-token math and work split are the decode step's (one workgroup per (batch
// row, v-head, block of state rows), a state row read by D/4 lanes, the conv
// front end one channel per thread), so a chain of nodes gives the chain
// verify's results bit for bit.  Every lane owns the same part of all of the
// row's states, and the workgroup walks the tree depth first, a node's largest
// subtree last.  The state a node starts from is then in registers: the one just
// made, or one of at most three saved ones.  (A state is saved while a subtree of
// it that is not its largest is walked, whose size is less than half of the
// rest; the committed state counts as the root of all: 17, 8, 3, 1.)  All inputs
// are in LDS before the first node, so nothing in the walk waits for memory, and
// the stores, one state per node, set its time.
//
// 16 rows of 15 nodes, 48 heads, d 128 (50 MB read, 755 MB written, non-temporal):
// 170 us, 4.7 TB/s, the rate of a large copy.  Walked in order of the nodes with
// parents' states read back and a node's inputs loaded when it came up: 243 us.
// Plain stores 177 us; four waves per SIMD (registers spill) 199 us.  4 rows of
// 4 nodes, from HBM: 16.8 us.
#include "gdn_device.h"
#include "gdn_ops.h"

namespace gdn {

__device__ __forceinline__ float tree_dot4(f32x4_t a, float4 b) {
  float s = a.x * b.x;
  s = fmaf(a.y, b.y, s);
  s = fmaf(a.z, b.z, s);
  return fmaf(a.w, b.w, s);
}

template <int D, bool BF16, int W>
__global__ __launch_bounds__((StepShape<D, true>::THREADS)) void tree_kernel(TreeArgs A) {
  using Sh = StepShape<D, true>;
  constexpr int LPR = Sh::LPR;
  constexpr int NP = Sh::NP;
  constexpr int NG = D < kWave ? D : kWave;            // lanes per partial sum of squares
  constexpr int kMaxNodes = 16;                        // max_draft's limit: 4 bits per parent below
  static_assert(Sh::THREADS >= 2 * D && Sh::THREADS >= Sh::ROWS_WG, "one channel per thread");
  __shared__ float fe[2][2 * D + Sh::ROWS_WG];         // q | k | v of a node (two nodes in flight)
  __shared__ float ssq[2][2 * D / NG];                 // partial sums of squares of q and k
  constexpr int kHist = W == 4 ? 3 : 0;
  __shared__ float xs[kHist + kMaxNodes][2 * D + Sh::ROWS_WG];
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = tid / kWave;
  const int hb = blockIdx.x % Sh::WG_PER_HEAD;
  const int h = blockIdx.x / Sh::WG_PER_HEAD;
  const int b = blockIdx.y;
  const int G = A.Hv / A.Hk;
  const int kh = h / G;
  const int c4 = (lane % LPR) * 4;                     // first state column of this lane
  const int rloc0 = wave * Sh::ROWS_WAVE + lane / LPR; // this lane's first row within the block
  const int row0 = hb * Sh::ROWS_WG + rloc0;
  const int R = A.R, C = A.C, K = A.k;
  const bool reporter = tid == 0 && blockIdx.x == 0;

  // ---- the row: slot, node count, parents (4 bits each: parent + 1) ----
  const int slot = A.slot[b];
  if (slot < 0 || slot >= A.n_slots) {
    if (reporter) report_error(A.dev_err, GDN_DEV_BAD_SLOT);
    return;
  }
  int kn = K;
  if (A.k_row != nullptr) {
    kn = A.k_row[b];
    if (kn < 1 || kn > K) {
      if (reporter) report_error(A.dev_err, GDN_DEV_BAD_K);
      return;
    }
  }
  static_assert(kMaxNodes <= 16, "parents are packed in 64 bits");
  const int my_parent = lane < kn ? A.parent[static_cast<size_t>(b) * K + lane] : -1;
  if (__ballot(my_parent < -1 || (lane < kn && my_parent >= lane)) != 0) {
    if (reporter) report_error(A.dev_err, GDN_DEV_BAD_PARENT);
    return;
  }
  uint64_t parents = 0;
  for (int j = 0; j < kn; ++j)
    parents |= static_cast<uint64_t>(__builtin_amdgcn_readlane(my_parent, j) + 1) << (4 * j);
  auto parent_of = [&](int j) { return static_cast<int>((parents >> (4 * j)) & 15) - 1; };

  // ---- the walk's order: lane j holds node j's children, subtree size, depth,
  // lane kRoot those of the committed state, the parent of the nodes without one ----
  constexpr int kRoot = kWave - 1;
  auto parent_lane = [&](int j) { return parent_of(j) & kRoot; };
  int size = lane < kn ? 1 : 0, depth_l = 0;
  uint32_t children = 0;
  for (int j = kn - 1; j >= 0; --j) {
    const int sj = __builtin_amdgcn_readlane(size, j);
    if (lane == parent_lane(j)) {
      size += sj;
      children |= 1u << j;
    }
  }
  int largest = 0, largest_size = 0;  // the node's child with the largest subtree
  for (int j = 0; j < kn; ++j) {
    const int sj = __builtin_amdgcn_readlane(size, j), pj = parent_lane(j);
    if (lane == pj && sj > largest_size) {
      largest_size = sj;
      largest = j;
    }
    const int dj = __builtin_amdgcn_readlane(depth_l, pj) + 1;
    if (lane == j) depth_l = dj;
  }
  uint32_t last = 0;  // the nodes that are walked after their siblings
  for (int j = 0; j < kn; ++j)
    if (__builtin_amdgcn_readlane(largest, parent_lane(j)) == j) last |= 1u << j;
  const int my_snap = lane < kn ? A.snap_slot[static_cast<size_t>(b) * K + lane] : -1;

  const char* xb = static_cast<const char*>(A.x) + static_cast<size_t>(b) * K * C * (BF16 ? 2 : 4);
  const size_t xrow = static_cast<size_t>(C) * (BF16 ? 2 : 4);
  // the channel this thread runs the conv of: q / k of the k-head, or v of a row
  const bool fe_qk = tid < 2 * D;
  const bool fe_v = tid < Sh::ROWS_WG;
  const int ch_qk = tid < D ? kh * D + tid : A.Hk * D + kh * D + (tid - D);
  const int ch_v = 2 * A.Hk * D + h * D + hb * Sh::ROWS_WG + tid;
  const int chq = fe_qk ? ch_qk : 0, chv = fe_v ? ch_v : 0;  // clamped: every load stays in the row
  float4 wq = make_float4(0.f, 0.f, 0.f, 0.f), wv = wq;
  if constexpr (W == 4) {
    wq = *reinterpret_cast<const float4*>(A.conv_w + chq * 4);
    wv = *reinterpret_cast<const float4*>(A.conv_w + chv * 4);
  }
  const uint32_t pos = W > 0 ? (static_cast<uint32_t>(A.conv_pos[slot * kPosStride]) >> kPosShift) : 0u;

  // ---- the committed state and conv history ----
  auto state_at = [&](int s, int p) {
    return A.state + (static_cast<size_t>(s) * A.Hv + h) * D * D + static_cast<size_t>(row0 + p * Sh::RPW) * D + c4;
  };
  f32x4_t S[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) S[p] = load_nt4(state_at(slot, p));
  float hq0[3] = {0.f, 0.f, 0.f}, hv0[3] = {0.f, 0.f, 0.f};
  if constexpr (W == 4) {
    const float* ring = A.conv_state + static_cast<size_t>(slot) * R * C;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      const float* rr = ring + static_cast<size_t>(ring_row(pos + static_cast<uint32_t>(t - 3), R)) * C;
      hq0[t] = rr[chq];
      hv0[t] = rr[chv];
    }
  }
  const bool qk_writer = fe_qk && (h % G == 0) && hb == 0;
  const bool o_writer = (lane % LPR) == 0;
  f32x4_t K0[NP], K1[NP], K2[NP];  // saved states
  auto copy = [](f32x4_t(&to)[NP], const f32x4_t(&from)[NP]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) to[p] = from[p];
  };
  int n_saved = 0;
  uint64_t todo = 0;  // their children that are still to be walked, 16 bits each, the newest lowest

  // ---- inputs and gates of all nodes: every thread keeps its channels' in LDS
  // (rows 0 .. 2: the committed history), every lane its node's gates ----
  const size_t g0 = static_cast<size_t>(b) * K * A.Hv + h;
  const int gl = min(lane, kn - 1);
  const float alpha_l = sigmoid_fast(-load_in<BF16>(A.a, g0 + static_cast<size_t>(gl) * A.Hv));  // exp(-softplus(a)) = sigmoid(-a)
  const float beta_l = sigmoid_fast(load_in<BF16>(A.b, g0 + static_cast<size_t>(gl) * A.Hv));
  const int tq = min(tid, 2 * D - 1), tv = 2 * D + min(tid, Sh::ROWS_WG - 1);
  float xq[kMaxNodes], xv[kMaxNodes];
#pragma unroll
  for (int j = 0; j < kMaxNodes; ++j) {  // all in flight at once (nodes behind the last: the last)
    const char* xr = xb + min(j, kn - 1) * xrow;
    xq[j] = load_in<BF16>(xr, chq);
    xv[j] = load_in<BF16>(xr, chv);
  }
#pragma unroll
  for (int j = -kHist; j < kMaxNodes; ++j) {
    if (fe_qk) xs[kHist + j][tid] = j < 0 ? hq0[(j + 3) % 3] : xq[max(j, 0)];
    if (fe_v) xs[kHist + j][2 * D + tid] = j < 0 ? hv0[(j + 3) % 3] : xv[max(j, 0)];
  }

  int cur = kRoot;    // the node that was walked last (whose state S holds)
  uint32_t lost = 0;  // nodes without a snapshot, and their descendants
  for (int i = 0; i < kn; ++i) {
    // ---- the next node, and its parent's state ----
    const uint32_t kids = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(children), cur));
    int j;
    if (kids != 0) {
      j = __builtin_ctz((kids & ~last) != 0 ? kids & ~last : kids);
      const uint32_t others = kids & ~(1u << j);
      if (others != 0) {
        if (n_saved == 0) copy(K0, S);
        else if (n_saved == 1) copy(K1, S);
        else copy(K2, S);
        ++n_saved;
        todo = (todo << 16) | others;
      }
    } else {
      const uint32_t left = static_cast<uint32_t>(todo) & 0xffffu;
      j = __builtin_ctz((left & ~last) != 0 ? left & ~last : left);
      if (n_saved == 1) copy(S, K0);
      else if (n_saved == 2) copy(S, K1);
      else copy(S, K2);
      todo ^= 1u << j;
      if ((left & ~(1u << j)) == 0) {
        --n_saved;
        todo >>= 16;
      }
    }
    cur = j;
    const int par = parent_of(j);
    const bool skip = par >= 0 && ((lost >> par) & 1u);
    const int ss_in = __builtin_amdgcn_readlane(my_snap, j);
    const bool ss_ok = !skip && ss_in >= 0 && ss_in < A.n_slots;
    if (!ss_ok) {
      if (reporter && !skip) report_error(A.dev_err, GDN_DEV_BAD_SLOT);
      lost |= 1u << j;
    }
    const int ss = ss_ok ? ss_in : 0;
    const size_t gi = g0 + static_cast<size_t>(j) * A.Hv;
    // ---- front end, one channel per thread: conv along the path + SiLU ----
    float* f = fe[i & 1];
    float yq, yv;
    if constexpr (W == 4) {
      // the last three inputs along the path before node j, then its own
      float hq[4], hv[4];
      int at = kHist + j;
#pragma unroll
      for (int t = 3; t >= 0; --t) {
        hq[t] = xs[at][tq];
        hv[t] = xs[at][tv];
        at = at < kHist ? at - 1 : kHist + parent_of(at - kHist);
      }
      const int depth = __builtin_amdgcn_readlane(depth_l, j);
      yq = silu_fast(fmaf(wq.w, hq[3], fmaf(wq.z, hq[2], fmaf(wq.y, hq[1], wq.x * hq[0]))));
      yv = silu_fast(fmaf(wv.w, hv[3], fmaf(wv.z, hv[2], fmaf(wv.y, hv[1], wv.x * hv[0]))));
      if (ss_ok) {
        // the snapshot slot's history: its last three inputs, at their ring rows
        float* sring = A.conv_state + static_cast<size_t>(ss) * R * C;
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          float* rr = sring + static_cast<size_t>(ring_row(pos + static_cast<uint32_t>(depth + t) - 3u, R)) * C;
          if (qk_writer) rr[chq] = hq[t + 1];
          if (fe_v) rr[chv] = hv[t + 1];
        }
        if (h == 0 && hb == 0 && tid == 0)
          A.conv_pos[ss * kPosStride] = static_cast<int32_t>((pos + static_cast<uint32_t>(depth)) << kPosShift);
      }
    } else {
      yq = xs[j][tq];
      yv = xs[j][tv];
    }
    float sq = group_sum<NG < 32 ? NG : 32>(yq * yq);
    if constexpr (NG == 64)  // the two 32-lane halves, added in a fixed order
      sq = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sq), 0)) +
           __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sq), 32));
    if (fe_qk) {
      f[tid] = yq;
      if (tid % NG == 0) ssq[i & 1][tid / NG] = sq;
    }
    if (fe_v) f[2 * D + tid] = yv;
    lds_barrier();
    // ---- L2 norm of q and k, gates ----
    float sqq = 0.f, skk = 0.f;
#pragma unroll
    for (int e = 0; e < D / NG; ++e) {
      sqq += ssq[i & 1][e];
      skk += ssq[i & 1][D / NG + e];
    }
    float qs = A.q_scale, ks = 1.0f;
    if (A.flags & GDN_FLAG_L2NORM_QK) {
      qs = qs * __builtin_amdgcn_rsqf(sqq + A.l2_eps);
      ks = __builtin_amdgcn_rsqf(skk + A.l2_eps);
    }
    const float4 qr = *reinterpret_cast<const float4*>(f + c4);
    const float4 kr = *reinterpret_cast<const float4*>(f + D + c4);
    const float4 q = make_float4(qr.x * qs, qr.y * qs, qr.z * qs, qr.w * qs);
    const float4 k = make_float4(kr.x * ks, kr.y * ks, kr.z * ks, kr.w * ks);
    const float kq = group_sum<LPR>(tree_dot4(f32x4_t{k.x, k.y, k.z, k.w}, q));
    const float alpha = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, alpha_l), j));
    const float beta = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, beta_l), j));
    // ---- rank-1 delta update and output, one state row per lane group ----
    float ov[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const float v = f[2 * D + rloc0 + p * Sh::RPW];
      const float sk = group_sum<LPR>(tree_dot4(S[p], k));
      const float sqv = group_sum<LPR>(tree_dot4(S[p], q));
      const float u = beta * (v - alpha * sk);
      ov[p] = fmaf(alpha, sqv, u * kq);
      S[p].x = fmaf(u, k.x, alpha * S[p].x);
      S[p].y = fmaf(u, k.y, alpha * S[p].y);
      S[p].z = fmaf(u, k.z, alpha * S[p].z);
      S[p].w = fmaf(u, k.w, alpha * S[p].w);
    }
    if (ss_ok) {
#pragma unroll
      for (int p = 0; p < NP; ++p) store_nt4(state_at(ss, p), S[p]);
    }
    if (o_writer && !skip) {
#pragma unroll
      for (int p = 0; p < NP; ++p) store_out<BF16>(A.o, gi * D + row0 + p * Sh::RPW, ov[p]);
    }
  }
}

template <int D, bool BF16>
static int launch_tree_t(const TreeArgs& a, hipStream_t s) {
  using Sh = StepShape<D, true>;
  dim3 grid(a.Hv * Sh::WG_PER_HEAD, a.batch);
  if (a.W == 4) hipLaunchKernelGGL((tree_kernel<D, BF16, 4>), grid, dim3(Sh::THREADS), 0, s, a);
  else if (a.W == 0) hipLaunchKernelGGL((tree_kernel<D, BF16, 0>), grid, dim3(Sh::THREADS), 0, s, a);
  else return static_cast<int>(hipErrorInvalidValue);
  return static_cast<int>(hipGetLastError());
}

int launch_verify_tree(const TreeArgs& a, bool bf16, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (a.D) {
    case 16: return bf16 ? launch_tree_t<16, true>(a, s) : launch_tree_t<16, false>(a, s);
    case 32: return bf16 ? launch_tree_t<32, true>(a, s) : launch_tree_t<32, false>(a, s);
    case 64: return bf16 ? launch_tree_t<64, true>(a, s) : launch_tree_t<64, false>(a, s);
    case 128: return bf16 ? launch_tree_t<128, true>(a, s) : launch_tree_t<128, false>(a, s);
    default: return static_cast<int>(hipErrorInvalidValue);
  }
}

}  // namespace gdn
