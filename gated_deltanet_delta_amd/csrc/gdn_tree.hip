// Verify over a tree of drafts for gfx950: the gated delta rule from every
// node's parent,
//   S_j = alpha_j S_p (I - beta_j k_j k_j^T) + beta_j v_j k_j^T,  o_j = S_j q_j,
// each node's state, conv window and position written to a pool slot of its own.
//
// Per-token math, work split and memory order are the decode step's (one
// workgroup per (batch row, v-head, block of state rows), a state row read by
// D/4 lanes, the conv front end one channel per thread), so a chain of nodes
// gives the chain verify's results bit for bit.  A workgroup walks the row's
// nodes in order; every lane owns the same part of all of the row's states.
// The committed state and the last node's state stay in registers; any other
// parent's part is read back from the slot this lane wrote it to.
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

__device__ __forceinline__ float tree_dot4(f32x4_t a, float4 b) {
  float s = a.x * b.x;
  s = fmaf(a.y, b.y, s);
  s = fmaf(a.z, b.z, s);
  return fmaf(a.w, b.w, s);
}

template <int D, bool BF16, int W>
__global__ __launch_bounds__((StepShape<D, true>::THREADS)) void tree_kernel(StepArgs A) {
  using Sh = StepShape<D, true>;
  constexpr int LPR = Sh::LPR;
  constexpr int NP = Sh::NP;
  constexpr int NG = D < kWave ? D : kWave;            // lanes per partial sum of squares
  constexpr int kMaxNodes = 16;                        // max_draft's limit: 4 bits per parent below
  static_assert(Sh::THREADS >= 2 * D && Sh::THREADS >= Sh::ROWS_WG, "one channel per thread");
  __shared__ float fe[2][2 * D + Sh::ROWS_WG];         // q | k | v of a node (two nodes in flight)
  __shared__ float ssq[2][2 * D / NG];                 // partial sums of squares of q and k
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
  f32x4_t S0[NP], S[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) S0[p] = load_nt4(state_at(slot, p));
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
  uint32_t lost = 0;  // nodes without a snapshot, and their descendants
  int held = -1;      // the node whose state S holds (-1: none yet)

  for (int j = 0; j < kn; ++j) {
    const int par = parent_of(j);
    if (par >= 0 && ((lost >> par) & 1u)) {
      lost |= 1u << j;
      continue;
    }
    const int ss_in = A.snap_slot[static_cast<size_t>(b) * K + j];
    const bool ss_ok = ss_in >= 0 && ss_in < A.n_slots;
    if (!ss_ok) {
      if (reporter) report_error(A.dev_err, GDN_DEV_BAD_SLOT);
      lost |= 1u << j;
    }
    const int ss = ss_ok ? ss_in : 0;
    // ---- the parent's state ----
    if (par < 0) {
#pragma unroll
      for (int p = 0; p < NP; ++p) S[p] = S0[p];
    } else if (par != held) {
      const int ps = A.snap_slot[static_cast<size_t>(b) * K + par];  // in range: par is not lost
#pragma unroll
      for (int p = 0; p < NP; ++p) S[p] = load4(state_at(ps, p));
    }
    held = j;
    const float xq = load_in<BF16>(xb + j * xrow, chq), xv = load_in<BF16>(xb + j * xrow, chv);
    const size_t gi = (static_cast<size_t>(b) * K + j) * A.Hv + h;
    const float ga = load_in<BF16>(A.a, gi), gb = load_in<BF16>(A.b, gi);
    // ---- front end, one channel per thread: conv along the path + SiLU ----
    float* f = fe[j & 1];
    float yq, yv;
    int depth = 1;
    if constexpr (W == 4) {
      float hq[3], hv[3];  // the three inputs before node j on its path
      int at = par, back = 2;
#pragma unroll
      for (int t = 2; t >= 0; --t) {
        if (at >= 0) {
          hq[t] = load_in<BF16>(xb + at * xrow, chq);
          hv[t] = load_in<BF16>(xb + at * xrow, chv);
          at = parent_of(at);
        } else {
          hq[t] = back == 2 ? hq0[2] : (back == 1 ? hq0[1] : hq0[0]);
          hv[t] = back == 2 ? hv0[2] : (back == 1 ? hv0[1] : hv0[0]);
          --back;
        }
      }
      for (int up = par; up >= 0; up = parent_of(up)) ++depth;
      yq = silu_fast(fmaf(wq.w, xq, fmaf(wq.z, hq[2], fmaf(wq.y, hq[1], wq.x * hq[0]))));
      yv = silu_fast(fmaf(wv.w, xv, fmaf(wv.z, hv[2], fmaf(wv.y, hv[1], wv.x * hv[0]))));
      if (ss_ok) {
        // the snapshot slot's history: its last three inputs, at their ring rows
        float* sring = A.conv_state + static_cast<size_t>(ss) * R * C;
        const float nq[3] = {hq[1], hq[2], xq}, nv[3] = {hv[1], hv[2], xv};
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          float* rr = sring + static_cast<size_t>(ring_row(pos + static_cast<uint32_t>(depth + t) - 3u, R)) * C;
          if (qk_writer) rr[chq] = nq[t];
          if (fe_v) rr[chv] = nv[t];
        }
        if (h == 0 && hb == 0 && tid == 0)
          A.conv_pos[ss * kPosStride] = static_cast<int32_t>((pos + static_cast<uint32_t>(depth)) << kPosShift);
      }
    } else {
      yq = xq;
      yv = xv;
    }
    float sq = group_sum<NG < 32 ? NG : 32>(yq * yq);
    if constexpr (NG == 64)  // the two 32-lane halves, added in a fixed order
      sq = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sq), 0)) +
           __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sq), 32));
    if (fe_qk) {
      f[tid] = yq;
      if (tid % NG == 0) ssq[j & 1][tid / NG] = sq;
    }
    if (fe_v) f[2 * D + tid] = yv;
    lds_barrier();
    // ---- L2 norm of q and k, gates ----
    float sqq = 0.f, skk = 0.f;
#pragma unroll
    for (int i = 0; i < D / NG; ++i) {
      sqq += ssq[j & 1][i];
      skk += ssq[j & 1][D / NG + i];
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
    const float alpha = sigmoid_fast(-ga);  // exp(-softplus(a)) = sigmoid(-a)
    const float beta = sigmoid_fast(gb);
    // ---- rank-1 delta update and output, one state row per lane group ----
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int row = row0 + p * Sh::RPW;
      const float v = f[2 * D + rloc0 + p * Sh::RPW];
      const float sk = group_sum<LPR>(tree_dot4(S[p], k));
      const float sqv = group_sum<LPR>(tree_dot4(S[p], q));
      const float u = beta * (v - alpha * sk);
      const float ov = fmaf(alpha, sqv, u * kq);
      f32x4_t sn;
      sn.x = fmaf(u, k.x, alpha * S[p].x);
      sn.y = fmaf(u, k.y, alpha * S[p].y);
      sn.z = fmaf(u, k.z, alpha * S[p].z);
      sn.w = fmaf(u, k.w, alpha * S[p].w);
      S[p] = sn;
      if (ss_ok) *reinterpret_cast<f32x4_t*>(state_at(ss, p)) = sn;
      if (o_writer) store_out<BF16>(A.o, gi * D + row, ov);
    }
  }
}

template <int D, bool BF16>
static int launch_tree_t(const StepArgs& a, hipStream_t s) {
  using Sh = StepShape<D, true>;
  dim3 grid(a.Hv * Sh::WG_PER_HEAD, a.batch);
  if (a.W == 4) hipLaunchKernelGGL((tree_kernel<D, BF16, 4>), grid, dim3(Sh::THREADS), 0, s, a);
  else if (a.W == 0) hipLaunchKernelGGL((tree_kernel<D, BF16, 0>), grid, dim3(Sh::THREADS), 0, s, a);
  else return static_cast<int>(hipErrorInvalidValue);
  return static_cast<int>(hipGetLastError());
}

int launch_verify_tree(const StepArgs& a, bool bf16, void* stream) {
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
