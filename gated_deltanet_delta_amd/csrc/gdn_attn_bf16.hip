// Attention in bf16 for gfx950 (the formulas and the row and key order:
// gdn_attn.hip): 32x32x16 matrix instructions on key tiles that the waves of a
// workgroup share through LDS.
//
// A wave owns 32 rows.  S^T = K Q^T takes K as the A operand from LDS and Q^T
// from registers; lane l then holds row l % 32 and keys 8 (i / 4) + 4 (l / 32) +
// i % 4 of a block of 32.  O^T = V^T P^T contracts 16 keys per
// instruction: lane l's eight weights of one instruction are its accumulators
// 8 ks .. 8 ks + 7 as they are, and V^T's operand is read out of the V tile in
// the same key order with transposing LDS reads (ds_read_b64_tr_b16).
//
// Tiles go from memory to LDS without passing registers (global_load_lds, 16
// bytes per lane), up to NST - 1 of them in flight while one is used.  Rows lie
// unpadded in LDS, their 16-byte chunks permuted by an XOR with row bits so that
// both kinds of reads hit all banks: K reads take one chunk of 16 consecutive
// rows (chunk ^ row % 16), transposing reads four chunks of four consecutive
// rows (chunk ^ 4 (row % 4)).
//
// What bounds it.  Prompts: the matrix instructions and the exponentials, sums
// and conversions between them, which a wave does in turn; eight waves of one
// workgroup (two per SIMD) overlap them in part.  24 heads on 4, d 256, one
// prompt of 8192: 784 - 846 us by the card, 0.98 - 1.05 PFLOP/s, where a large library
// product reaches 1.6; ragged prompts behind prefixes of up to 20011 tokens, 32 heads
// on 8, d 128: 717 - 779 us, 0.91 - 0.98 PFLOP/s.  Rows per wave: 64 (four waves, one
// per SIMD) took 1452 us on the second, for want of a second wave to overlap with,
// and at d 256 do not fit the registers.  Two groups of waves that alternate
// products and weights between barriers: 995 and 1166 us against 785 and 896 then.
// Trees: the bytes of K and V (below).
#include "gdn_attn_device.h"
#include "gdn_rank.h"

namespace gdn {

namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kSchedMfma = 0x8, kSchedLds = 0x100;  // instruction classes of sched_group_barrier: MFMA, LDS reads

// 16 bytes per lane from memory to LDS at `lds` + 16 lane (lds: a byte address,
// the same in every lane).  Written out because the compiler, which cannot
// tell the buffers apart, would wait for these loads
// before every LDS read.  There is no register to return to; the readers are
// ordered by wait_tiles() and a barrier.
__device__ __forceinline__ void load_lds16(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(g) : "memory", "m0");
}
// The same from `base` (one address for all lanes) + off bytes.
__device__ __forceinline__ void load_lds16(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
// All but this wave's newest LEFT loads have landed.  The wait is the builtin,
// which the compiler takes into account: it then adds no wait of its own, among
// a tile's products, for loads issued before.
template <int LEFT>
__device__ __forceinline__ void wait_loads() {
  static_assert(LEFT >= 0 && LEFT < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | ((LEFT >> 4) << 14) | 0x0070);  // vmcnt LEFT, lgkmcnt 0
  asm volatile("" ::: "memory");
}
// One 32-bit word per lane from memory to LDS at `lds` + 4 lane.
__device__ __forceinline__ void load_lds4(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(g) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(p)));
}

__device__ __forceinline__ f32x16_t mfma32x32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
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

}  // namespace

// NW waves move KT-key tiles through NST buffers; the first RW of them compute,
// 32 rows each.
template <int D, int RW, int NW, int KT, int NST, bool TREE>
struct Tiles {
  static constexpr int THREADS = 64 * NW, BM = 32 * RW;
  static constexpr int ROW_BYTES = D * 2;
  static constexpr int TILE = KT * ROW_BYTES;            // K or V of a tile
  static constexpr int BUF = 2 * TILE;
  static constexpr int NS = D / 16, NT = D / 32;         // k-steps of the logits, 32-row tiles of O^T
  static constexpr int KB = KT / 32;                     // 32-key blocks per tile
  static constexpr int RPI = 1024 / ROW_BYTES;           // rows of one load instruction
  static constexpr int WROWS = KT / NW;                  // rows a wave loads
  static constexpr int LPT = 2 * (WROWS / RPI);          // load instructions of a wave and tile
  static constexpr int LPR = 64 / RPI;                   // lanes per row
  static constexpr int CH = D / 8;                       // 16-byte chunks of a row
  static constexpr int GROUP = 16;                       // tokens of a page come in multiples of this
  static constexpr int TPI = 64 * GROUP / KT;            // tiles whose groups the lanes' page ids cover
  static_assert(WROWS % RPI == 0 && WROWS > 0 && (NST & (NST - 1)) == 0 && RPI <= GROUP && WROWS % 2 == 0, "shape");
  // LDS: NST buffers, per wave two rounds of page ids, flags (keys whose V row is not finite)
  static constexpr size_t LDS_TILES = static_cast<size_t>(NST) * BUF;
  static constexpr size_t LDS_FLAGS = LDS_TILES + NW * 512;
  static constexpr size_t LDS = LDS_FLAGS + 16;

  __device__ static int k_perm(int row) { return D >= 128 ? row & 15 : (row >> 1) & 7; }
  __device__ static int v_perm(int row) { return D >= 128 ? (row & 3) * 4 : ((row >> 1) & 1) * 4; }

  const AttnArgs& A;
  char* lds;
  uint32_t lds0;
  int lane, wave, col, half;
  // the unit of work: one KV head of one sequence, a block of rows
  Seq q;
  int kvh;
  int32_t n_keys, clear;
  int64_t r0;            // its first row
  int t;                 // this lane's token
  uint64_t path;         // TREE: its row's nodes
  // base rows ((page * H_kv + kvh) P + offset) of the cached 16-token groups,
  // one per lane: lane i holds that of key 1024 ids_at + 16 i
  int32_t ids_at;
  int64_t ids;
  bf16x8_t qf[NS];
  f32x16_t O[NT];
  float m, l;            // running maximum (of unscaled logits), this lane's part of the sum

  __device__ Tiles(const AttnArgs& a, char* smem) : A(a), lds(smem) {
    lds0 = __builtin_amdgcn_readfirstlane(lds_address(smem));
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    col = lane & 31;
    half = lane >> 5;
  }

  // The unit: rows r0 .. r0 + BM - 1 (of n G) of KV head h of sequence q.
  __device__ void begin_keys(int64_t first_row, int h) {
    r0 = first_row;
    kvh = h;
    const int64_t rows = static_cast<int64_t>(q.n) * A.G;
    const int64_t r_last = r0 + BM < rows ? r0 + BM - 1 : rows - 1;
    n_keys = TREE ? q.ctx + q.n : q.ctx + static_cast<int32_t>(r_last / A.G) + 1;
    clear = TREE ? q.ctx : q.ctx + static_cast<int32_t>(r0 / A.G) + 1;
    ids_at = -1;
  }
  // Query head of this lane's row, and its token; -1: no row (the token is then
  // the unit's first).
  __device__ int row_head(int* token) const {
    const int32_t t0 = static_cast<int32_t>(r0 / A.G), h0 = static_cast<int32_t>(r0 - static_cast<int64_t>(t0) * A.G);
    const int32_t r = wave * 32 + col;
    const bool ok = wave < RW && r < static_cast<int64_t>(q.n) * A.G - r0;
    const int32_t rc = ok ? r : 0;
    *token = t0 + (h0 + rc) / A.G;
    return ok ? kvh * A.G + (h0 + rc) % A.G : -1;
  }
  // This lane's row and its Q; node_paths (TREE): lane j holds node j's path.
  __device__ void begin_rows(uint64_t node_paths) {
    int hd = row_head(&t);
    if (hd < 0) hd = kvh * A.G;  // reads some row of the call's
    if constexpr (TREE)
      path = (static_cast<uint64_t>(__shfl(static_cast<uint32_t>(node_paths >> 32), t, 64)) << 32) |
             static_cast<uint32_t>(__shfl(static_cast<uint32_t>(node_paths), t, 64));
    const uint16_t* qp = static_cast<const uint16_t*>(A.q) + (q.row0 + t) * A.q_stride + static_cast<int64_t>(hd) * D;
#pragma unroll
    for (int s = 0; s < NS; ++s) qf[s] = *reinterpret_cast<const bf16x8_t*>(qp + s * 16 + half * 8);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) O[i][e] = 0.f;
    m = -INFINITY;
    l = 0.f;
  }

  // Page ids of round `at` (keys 1024 at ..), one 16-token group per lane, into
  // this wave's LDS: requested a round ahead, so nothing waits for them.
  __device__ uint32_t ids_lds(int32_t at) const { return LDS_TILES + wave * 512 + (at & 1) * 256; }
  __device__ void request_ids(int32_t at) {
    const int32_t key = at * 1024 + lane * GROUP;  // below 2^30 + 2^11
    load_lds4(A.block_table + static_cast<size_t>(q.index) * A.max_pages + (key < q.ctx ? key / A.page : 0), lds0 + ids_lds(at));
  }
  // Takes round `at`, which has landed, into ids; asks for the next.
  __device__ void take_ids(int32_t at) {
    ids_at = at;
    const int32_t key = at * 1024 + lane * GROUP;
    int32_t page = *reinterpret_cast<const int32_t*>(lds + ids_lds(at) + 4 * lane);
    ids = 0;
    if (key < q.ctx) {
      if (page < 0 || page >= A.n_pages) {
        report_error(A.dev_err, GDN_DEV_BAD_PAGE);
        page = 0;
      }
      ids = (static_cast<int64_t>(page) * A.Hk + kvh) * A.page + (key - key / A.page * A.page);
    }
    if ((at + 1) * 1024 < q.ctx) request_ids(at + 1);
  }

  // Requests tile kt into buffer b.
  __device__ void request(int32_t kt, int b) {
    const int32_t key0 = kt * KT;
    // made anew for every tile (the empty asm hides that they never change):
    // offsets kept across tiles would be spilled, and a reload waits for all
    // loads in flight
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int lrow = ln / LPR, c = ln % LPR;  // this lane's row of an instruction's RPI, its chunk's place
    const int wrow = wave * WROWS;
    const uint32_t dst = lds0 + b * BUF + wrow * ROW_BYTES;
    if (key0 + KT <= q.ctx) {
      // all cached: 16-row groups lie in one page each
      if (ids_at != kt / TPI) {
        if (ids_at != kt / TPI - 1 || ids_at < 0) {  // the unit's first: not asked for before
          request_ids(kt / TPI);
          wait_loads<0>();
        }
        take_ids(kt / TPI);
      }
#pragma unroll
      for (int i = 0; i < WROWS / RPI; ++i) {
        const int row = wrow + i * RPI;  // first row of the instruction, within the tile
        const int src = (kt % TPI) * (KT / GROUP) + row / GROUP;
        const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(ids), src);
        const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(static_cast<uint64_t>(ids) >> 32), src);
        const int64_t base = (static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo) + row % GROUP) * ROW_BYTES;
        const uint32_t at = lrow * ROW_BYTES;
        load_lds16(static_cast<const char*>(A.k_cache) + base, at + 16 * (c ^ k_perm(row + lrow)), dst + i * 1024);
        load_lds16(static_cast<const char*>(A.v_cache) + base, at + 16 * (c ^ v_perm(row + lrow)), dst + TILE + i * 1024);
      }
    } else if (key0 >= q.ctx) {
      // all of the call's own rows (strides are below 2^24 elements); rows past
      // the last key repeat it, and no row attends them
      const int64_t first = q.row0 + (key0 - q.ctx);
      const char* kp = static_cast<const char*>(A.k) + (first * A.k_stride + static_cast<int64_t>(kvh) * D) * 2;
      const char* vp = static_cast<const char*>(A.v) + (first * A.v_stride + static_cast<int64_t>(kvh) * D) * 2;
      const uint32_t ks = static_cast<uint32_t>(A.k_stride) * 2, vs = static_cast<uint32_t>(A.v_stride) * 2;
      const int last = n_keys - 1 - key0;
#pragma unroll
      for (int i = 0; i < WROWS / RPI; ++i) {
        const int rr = wrow + i * RPI + lrow;
        const uint32_t r = min(rr, last);
        load_lds16(kp, r * ks + 16 * (c ^ k_perm(rr)), dst + i * 1024);
        load_lds16(vp, r * vs + 16 * (c ^ v_perm(rr)), dst + TILE + i * 1024);
      }
    } else {
      // both kinds: at most one tile of a sequence
#pragma unroll 1
      for (int i = 0; i < WROWS / RPI; ++i) {
        const int rr = wrow + i * RPI + lrow;
        const int32_t j = min(key0 + rr, n_keys - 1);
        const char* kp = key_row<2>(A, q, A.k_cache, A.k, A.k_stride, kvh, j);
        const char* vp = key_row<2>(A, q, A.v_cache, A.v, A.v_stride, kvh, j);
        load_lds16(kp + 16 * (c ^ k_perm(rr)), dst + i * 1024);
        load_lds16(vp + 16 * (c ^ v_perm(rr)), dst + TILE + i * 1024);
      }
    }
  }

  // Does this lane's row attend key j?
  __device__ bool attends(int32_t j) const {
    const int32_t own = j - q.ctx;
    if constexpr (TREE) return own < 0 || (own < q.n && ((path >> own) & 1ull));
    else return own <= t;
  }

  // Values that are not finite must not reach rows that do not attend their
  // key (0 x inf is NaN).  In a tile that some row attends in part: finds such
  // V rows and clears them in LDS; their terms are added apart in block().
  // All waves call it.
  __device__ uint64_t clear_bad(char* v) {
    uint32_t* flags = reinterpret_cast<uint32_t*>(lds + LDS_FLAGS);
    if (threadIdx.x < 2) flags[threadIdx.x] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < KT * CH; e += THREADS)
      if (any_nonfinite<true>(*reinterpret_cast<const uint4*>(v + e * 16))) atomicOr(&flags[e / CH / 32], 1u << (e / CH % 32));
    __syncthreads();
    const uint64_t bad = (static_cast<uint64_t>(flags[1]) << 32) | flags[0];
    if (bad != 0) {
      for (int e = threadIdx.x; e < KT * CH; e += THREADS)
        if ((bad >> (e / CH)) & 1ull) *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();  // the flags are read, and the rows cleared, by every wave
    return bad;
  }

  // LDS addresses of this lane's operands in a tile: K rows are read 16 bytes
  // at k-step s, V rows transposed at O^T tile dt.  The permutations touch the
  // low bits of s and dt alone, so a few addresses serve a whole tile, the rest
  // being constant offsets.
  static constexpr int KA = NS < 8 ? NS : 8, VA = NT < 4 ? NT : 4;
  __device__ void k_addresses(int b, uint32_t (&ka)[KA]) const {
    int ln = lane;  // made anew per tile, see request()
    asm volatile("" : "+v"(ln));
    const uint32_t buf = lds0 + b * BUF;
    const int kcol = ln & 31, kx = k_perm(kcol);  // blocks start at multiples of 32 rows
#pragma unroll
    for (int s = 0; s < KA; ++s) ka[s] = buf + kcol * ROW_BYTES + 16 * ((2 * s + (ln >> 5)) ^ kx);
  }
  __device__ void v_addresses(int b, uint32_t (&va)[VA]) const {
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const uint32_t buf = lds0 + b * BUF;
    const int g2 = (ln >> 4) & 1, mrow = (ln & 15) >> 2, quarter = ln & 3;
    const uint32_t vrow = buf + TILE + (4 * (ln >> 5) + mrow) * ROW_BYTES + 8 * (quarter & 1);
#pragma unroll
    for (int dt = 0; dt < VA; ++dt)  // rows of one read differ from mrow by multiples of 4
      va[dt] = vrow + 16 * ((dt * 4 + 2 * g2 + (quarter >> 1)) ^ v_perm(mrow));
  }

  // Logits of the tile in buffer b.
  __device__ void logits(int b, f32x16_t (&S)[KB]) const {
    typedef __attribute__((address_space(3))) const bf16x8_t* lds_k;
    uint32_t ka[KA];
    k_addresses(b, ka);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) S[kb][e] = 0.f;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const bf16x8_t a = *(lds_k)(ka[s % KA] + (s / KA) * 256 + kb * 32 * ROW_BYTES);
        S[kb] = mfma32x32(a, qf[s], S[kb]);
      }
    }
    // K operands four steps ahead, no more: registers are short
    __builtin_amdgcn_sched_group_barrier(kSchedLds, 4, 0);
#pragma unroll
    for (int s = 0; s < KB * NS; ++s) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
      if (s < KB * NS - 4) __builtin_amdgcn_sched_group_barrier(kSchedLds, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // Weights of a tile from its logits: rounded to bf16 for the product (what the
  // matrix instruction takes; fp32 operands run at a sixteenth of its rate), each
  // off by at most 2^-8 of itself.  Over the keys of a row that stays below the
  // output's own rounding: outputs are 0.0020 - 0.0023 of their size from the exact
  // ones, 0.0015 - 0.0017 where the outputs alone are rounded.  The sum takes the
  // rounded weights too, two to an instruction.
  // MASKED: some row does not attend every key of the tile; S then keeps the
  // unrounded weights.
  template <bool MASKED>
  __device__ void weights(int32_t key0, f32x16_t (&S)[KB], bf16x8_t (&P)[KB][2]) {
    float mx = -INFINITY;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if constexpr (MASKED) S[kb][e] = attends(key0 + kb * 32 + 8 * (e / 4) + 4 * half + e % 4) ? S[kb][e] : -INFINITY;
        mx = fmaxf(mx, S[kb][e]);
      }
    mx = half_max(mx);
    // The weights are taken against a maximum that may lag: O and l are scaled
    // only when some row's maximum has grown by more than 2^8 in weight, which
    // leaves sums and weights far inside their range.
    if (__any((mx - m) * A.scale_log2 > 8.f)) {
      const float m_new = fmaxf(m, mx);
      const float f = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - m_new) * A.scale_log2);
      m = m_new;
      l *= f;
#pragma unroll
      for (int i = 0; i < NT; ++i) O[i] *= f;
    }
    const float off = m == -INFINITY ? 0.f : -m * A.scale_log2;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        S[kb][e] = __builtin_amdgcn_exp2f(fmaf(S[kb][e], A.scale_log2, off));
        P[kb][e / 8][e % 8] = static_cast<__bf16>(S[kb][e]);
      }
#pragma unroll
      for (int e = 0; e < 16; e += 2)
        l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2_t{P[kb][e / 8][e % 8], P[kb][e / 8][e % 8 + 1]}, bf16x2_t{1.0f, 1.0f}, l, false);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // O^T += V^T P^T for the tile in buffer b.
  __device__ void terms(int b, const bf16x8_t (&P)[KB][2]) {
    typedef __attribute__((address_space(3))) s16x4_t* lds_v;
    uint32_t va[VA];
    v_addresses(b, va);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int dt = 0; dt < NT; ++dt) {
          const uint32_t at = va[dt % VA] + (dt / VA) * 256 + (kb * 32 + 16 * ks) * ROW_BYTES;
          const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v)(at));
          const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v)(at + 8 * ROW_BYTES));
          O[dt] = mfma32x32(__builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7)), P[kb][ks], O[dt]);
        }
    __builtin_amdgcn_sched_group_barrier(kSchedLds, 6, 1);
#pragma unroll
    for (int i = 0; i < KB * 2 * NT; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 1);
      if (i < KB * 2 * NT - 3) __builtin_amdgcn_sched_group_barrier(kSchedLds, 2, 1);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // The terms of the V rows that clear_bad() took out of a tile, for the rows
  // that attend them; S holds the weights.
  __device__ void bad_terms(int32_t key0, uint64_t bad, const f32x16_t (&S)[KB]) {
    for (; bad != 0; bad &= bad - 1) {
      const int kr = __builtin_ctzll(bad);
      const int32_t j = key0 + kr;
      float p = 0.f;  // the weight, in the lanes of half (kr / 4) % 2
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e) p = (kb * 32 + 8 * (e / 4) + e % 4) == (kr & ~4) ? S[kb][e] : p;
      p = __shfl(p, col + 32 * ((kr >> 2) & 1), 64);
      if (!attends(j)) continue;
      const uint16_t* vr = reinterpret_cast<const uint16_t*>(key_row<2>(A, q, A.v_cache, A.v, A.v_stride, kvh, j)) + 4 * half;
#pragma unroll
      for (int dt = 0; dt < NT; ++dt) {
#pragma unroll
        for (int i = 0; i < 16; ++i) O[dt][i] += p * bf16_bits_to_f32(vr[dt * 32 + 8 * (i / 4) + i % 4]);
        asm volatile("" ::: "memory");  // no more than one step's loads at a time in registers
      }
    }
  }

  // One tile in buffer b.
  template <bool MASKED>
  __device__ void tile(int32_t kt, int b) {
    uint64_t bad = 0;
    if constexpr (MASKED) bad = clear_bad(lds + b * BUF + TILE);
    if (wave < RW) {
      f32x16_t S[KB];
      bf16x8_t P[KB][2];
      logits(b, S);
      weights<MASKED>(kt * KT, S, P);
      terms(b, P);
      if constexpr (MASKED) bad_terms(kt * KT, bad, S);
    }
  }

  // Waits until at most `tiles` (0 .. NST - 2) of the newest requests are in flight.
  __device__ static void wait_tiles(int tiles) {
    if (tiles >= NST - 2) wait_loads<(NST - 2) * LPT>();
    else if (NST > 3 && tiles == 1) wait_loads<(NST > 3 ? LPT : 0)>();
    else wait_loads<0>();
  }
  __device__ static void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  // Tiles kt .. end - 1 of [lo, hi), up to tile kt + NST - 2 requested already.
  template <bool MASKED>
  __device__ void in_turn(int32_t kt, int32_t end, int32_t lo, int32_t hi) {
    for (; kt < end; ++kt) {
      wait_tiles(hi - 1 - kt);
      barrier();
      if (kt + NST - 1 < hi) request(kt + NST - 1, (kt + NST - 1 - lo) & (NST - 1));
      tile<MASKED>(kt, (kt - lo) & (NST - 1));
    }
  }
  // Tiles [lo, hi) of the unit, the first already requested into buffer 0;
  // leaves the sums in O, m, l.
  __device__ void keys(int32_t lo, int32_t hi) {
    wait_loads<0>();  // Q is at hand, so no later wait is for it
    // tiles that every row attends whole, then the others
    const int32_t mid = max(lo, min(hi, clear / KT));
#pragma unroll 1
    for (int i = 1; i < NST - 1 && lo + i < hi; ++i) request(lo + i, i);
    in_turn<false>(lo, mid, lo, hi);
    in_turn<true>(mid, hi, lo, hi);
    l = half_sum(l);
  }

  // Element (dt, i) of O is d = 32 dt + 8 (i / 4) + 4 half + i % 4.
  __device__ void write_out(int head) const {
    const float inv = 1.0f / l;
    uint16_t* o = static_cast<uint16_t*>(A.o) + (static_cast<size_t>(q.row0 + t) * A.Hq + head) * D + 4 * half;
#pragma unroll
    for (int dt = 0; dt < NT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint2*>(o + 32 * dt + 2 * i) = make_uint2(pack2_bf16(O[dt][i] * inv, O[dt][i + 1] * inv),
                                                                    pack2_bf16(O[dt][i + 2] * inv, O[dt][i + 3] * inv));
  }
  // Unscaled sums and (scaled maximum, sum) of this lane's row.
  __device__ void write_part(float* sums, float* ml) const {
#pragma unroll
    for (int dt = 0; dt < NT; ++dt)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4_t*>(sums + 32 * dt + 2 * i + 4 * half) =
            f32x4_t{O[dt][i], O[dt][i + 1], O[dt][i + 2], O[dt][i + 3]};
    if (half == 0) {
      ml[0] = m * A.scale_log2;
      ml[1] = l;
    }
  }
};

// Packed prompts: 256 rows per workgroup, 128 KB (D 64: 64 KB) of tiles.  64 keys
// where the registers hold a tile's logits beside O^T (d 128: 717 us on the ragged
// prompts above, 802 with 32 keys), else 32 (d 256: 784 us, with 64 keys, two
// buffers and spilled registers 1256).
template <int D>
constexpr int prompt_keys() { return D == 256 ? 32 : 64; }
template <int D>
using PromptTiles = Tiles<D, kPromptRows / 32, kPromptRows / 32, prompt_keys<D>(), 4, false>;

// Sum over the wave's lanes, in every lane.
__device__ __forceinline__ int32_t wave_sum(int32_t v) {
  v += __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);   // lane ^ 1
  v += __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);   // lane ^ 2
  v += __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);  // 7 - i within 8 lanes
  v += __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);  // 15 - i within 16 lanes
  return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
         __builtin_amdgcn_readlane(v, 48);
}

// A wave's lanes for ranked_block(), one sequence per lane.
template <int BM>
struct WaveLanes {
  typedef RowBlocks<BM> Blocks;
  Blocks mine;
  int lane;
  template <class F>
  __device__ int32_t sum(F f) const { return wave_sum(f(mine, lane)); }
  template <class F>
  __device__ int32_t max(F f) const {
    int32_t v = f(mine, lane);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = ::max(v, __shfl_xor(v, d, 64));
    return uniform(v);
  }
  template <class F>
  __device__ uint64_t ballot(F f) const { return __ballot(f(mine, lane)); }
  template <class F>
  __device__ int32_t at(F f, int l) const { return __builtin_amdgcn_readlane(f(mine, lane), l); }
};

// Row block number `rank` of a batch of at most 64 sequences (gdn_rank.h).
// Refused sequences have no blocks, and are reported at rank 0.  False: there are
// no more blocks.
template <int BM>
__device__ bool ranked_block_of(const AttnArgs& A, int64_t rank, int* seq, int64_t* r0) {
  const int lane = threadIdx.x & 63;
  Seq q{0, 0, 0, 0};
  const bool in = lane < A.n_seqs;
  if (in) q = packed_seq(A, lane, rank == 0);
  // sequences behind one that ends before it begins are refused with it (last_seq)
  const uint64_t back = __ballot(in && A.cu_seqlens[lane + 1] < A.cu_seqlens[lane]);
  if (((back ^ (back - 1)) >> lane & 1ull) == 0) q.n = 0;
  const WaveLanes<BM> lanes{RowBlocks<BM>(q.n, q.ctx, A.G), lane};
  int s;
  int32_t block;
  if (!ranked_block(lanes, static_cast<int32_t>(rank), &s, &block)) return false;
  *seq = uniform(s);
  *r0 = static_cast<int64_t>(block) * BM;
  return true;
}

// One workgroup per (block of rows, KV head, split of the key axis).
template <int D>
__global__ __launch_bounds__(PromptTiles<D>::THREADS, 2) void attn_prompt_kernel(AttnArgs A) {
  typedef PromptTiles<D> F;
  extern __shared__ __align__(1024) char smem[];
  F f(A, smem);
  int s;
  int64_t r0;
  if (A.n_seqs <= 64) {
    if (!ranked_block_of<F::BM>(A, blockIdx.x / A.Hk, &s, &r0)) return;
  } else {  // there are many blocks to even out what their order does not
    const int64_t id = gridDim.x / A.Hk - 1 - blockIdx.x / A.Hk;
    s = uniform(find_seq(A, id, F::BM));
    r0 = uniform((id - tile_start(A, s, F::BM)) * F::BM);
  }
  f.q = uniform(packed_seq(A, s, threadIdx.x == 0));
  if (f.q.n == 0 || r0 >= static_cast<int64_t>(f.q.n) * A.G) return;
  f.begin_keys(r0, blockIdx.x % A.Hk);
  const int32_t tiles = (f.n_keys + prompt_keys<D>() - 1) / prompt_keys<D>();
  const int32_t per = (tiles + A.n_split - 1) / A.n_split;
  const int32_t lo = min(static_cast<int32_t>(blockIdx.y) * per, tiles), hi = min(lo + per, tiles);
  if (lo < hi) f.request(lo, 0);
  f.begin_rows(0);
  if (lo < hi) f.keys(lo, hi);
  int t;
  const int head = f.row_head(&t);
  if (head < 0) return;
  if (A.n_split == 1) {
    f.write_out(head);
  } else {
    const size_t part = (static_cast<size_t>(f.q.row0 + t) * A.Hq + head) * A.n_split + blockIdx.y;
    float* ml = A.part + static_cast<size_t>(A.n_tokens) * A.Hq * A.n_split * D;
    f.write_part(A.part + part * D, ml + part * 2);
  }
}

// ---------------------------------------------------------------------------
// Trees of drafts: the key tiles of all units (KV head x block of rows of one
// row of the batch) lie on one line, row by row, kUnitCost places for what a
// unit costs apart from its tiles before each unit's, and workgroup w of W takes
// places [w T / W, (w + 1) T / W) of the T, whatever the rows' lengths.  A unit
// that lies in one workgroup's share is written out; the shares of one that
// does not go to the workspace (at most two per workgroup: its first, begun
// inside a unit, and its last, ended inside one) and are joined by
// tree_join_kernel.
// ---------------------------------------------------------------------------
struct TreeSplit {
  int32_t rows_per_unit, units_per_row;  // BM; row blocks x KV heads
  int32_t workgroups;                    // W
};
// Workspace: sums [2 W][BM][D], (max, sum) [2 W][BM][2], then per unit
// (first workgroup with a tile of it, number of workgroups; 0 or 1: nothing to join).
__host__ __device__ inline size_t tree_ml_offset(const TreeSplit& t, int D) {
  return static_cast<size_t>(2) * t.workgroups * t.rows_per_unit * D;
}
__host__ __device__ inline size_t tree_meta_offset(const TreeSplit& t, int D) {
  return tree_ml_offset(t, D) + static_cast<size_t>(4) * t.workgroups * t.rows_per_unit;
}

// 32-key tiles in four buffers; waves that have no rows only move tiles.  With
// few rows a call is bound by memory, and what reaches its rate is many waves
// with many loads in flight: 256 CUs x 8 waves, 64 - 96 KB per CU.  Between two
// units a workgroup's loads run dry once, so a unit counts as its tiles and
// kUnitCost more where the line is cut into shares: 64 ragged rows (below) 209 us
// with 0, 188 with 2, 174 with 4, 153 with 8, 151 with 12, 154 with 16, 161 with 32.
// 24 heads on 4, d 256: 4 rows of one node at 8K 47 us (134 MB, 2.9 TB/s; the
// join of the shares 6 of them); 4 rows of 16 nodes at 80 - 120K 356 us (1.64 GB,
// 4.6 TB/s, the rate of a large copy).  32 heads on 8, d 128, 64 rows of 8 nodes
// up to 16K, 16-token pages: 149 us (0.67 GB, 4.5 TB/s).  At d 256 25 - 27 registers
// of the addresses and row descriptions are spilled: stored once per workgroup,
// read back between units, and one of them within the tiles, where new page ids are
// taken (every 1024 keys).
constexpr int kTreeKeys = 32, kUnitCost = 12;
template <int D, int RW>
using TreeTiles = Tiles<D, RW, (RW > 2048 / 256 * D / 256 ? RW : 2048 / 256 * D / 256), kTreeKeys, 4, true>;

template <int D, int RW>
__global__ __launch_bounds__((TreeTiles<D, RW>::THREADS), 2) void attn_tree_kernel(AttnArgs A, TreeSplit ts) {
  typedef TreeTiles<D, RW> F;
  extern __shared__ __align__(1024) char smem[];
  F f(A, smem);
  const int lane = threadIdx.x & 63;
  int2* meta = reinterpret_cast<int2*>(A.part + tree_meta_offset(ts, D));

  // ---- the line: tiles of a unit of row s, and its units ----
  auto row_tiles = [&](int s, int32_t* units) {
    const int32_t n = A.n_row ? A.n_row[s] : A.nodes, c = A.ctx_len[s];
    *units = 0;
    if (n < 1 || n > A.nodes || c < 0 || c > static_cast<int64_t>(A.max_pages) * A.page) return 0;
    *units = (n * A.G + F::BM - 1) / F::BM * A.Hk;
    return (c + n + kTreeKeys - 1) / kTreeKeys;
  };
  // inclusive sum over the lanes of the places of rows base + lane
  auto scan = [&](int base, int64_t* mine) {
    int32_t units = 0;
    const int32_t tiles = base + lane < A.n_seqs ? row_tiles(base + lane, &units) : 0;
    int64_t inc = *mine = static_cast<int64_t>(tiles + kUnitCost) * units;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t up = __shfl_up(inc, d, 64);
      if (lane >= d) inc += up;
    }
    return inc;
  };
  int64_t total = 0, mine = 0, inc = 0;
  for (int base = 0; base < A.n_seqs; base += 64) {
    inc = scan(base, &mine);
    total += __shfl(inc, 63, 64);
  }
  total = uniform(total);
  // units without places (refused rows, row blocks past a row's nodes) have nothing to join
  for (int s = blockIdx.x; s < A.n_seqs; s += gridDim.x) {
    int32_t units;
    row_tiles(s, &units);
    for (int u = units + threadIdx.x; u < ts.units_per_row; u += F::THREADS)
      meta[static_cast<size_t>(s) * ts.units_per_row + u] = make_int2(0, 0);
    if (units == 0) {  // reports what is wrong with it
      uint64_t p;
      tree_seq(A, s, threadIdx.x == 0, &p);
    }
  }
  const int64_t W = ts.workgroups < total ? ts.workgroups : total;  // every workgroup has a place
  const int64_t w = blockIdx.x;
  if (w >= W) return;
  const int64_t first = uniform(w * total / W), last = uniform((w + 1) * total / W);

  // ---- the row that holds place `first`: the last one that does not begin after it ----
  int s = 0;
  int64_t row_at = 0;  // its first place
  for (int base = 0;; base += 64) {
    if (A.n_seqs > 64) inc = scan(base, &mine);  // else it is at hand
    const int64_t chunk = __shfl(inc, 63, 64);
    if (row_at + chunk > first) {
      const int at = 63 - __builtin_clzll(__ballot(base + lane < A.n_seqs && row_at + inc - mine <= first));
      s = base + at;
      row_at += __shfl(inc - mine, at, 64);
      break;
    }
    row_at += chunk;
  }
  s = uniform(s);
  row_at = uniform(row_at);

  int seen = -1;  // the row whose paths are at hand
  uint64_t paths = 0;
  Seq q{0, 0, 0, 0};
  for (int64_t at = first; at < last;) {
    int32_t units;
    const int32_t tiles = uniform(row_tiles(s, &units)), places = tiles + kUnitCost;
    units = uniform(units);
    if (at >= row_at + static_cast<int64_t>(places) * units) {
      row_at += static_cast<int64_t>(places) * units;
      ++s;
      continue;
    }
    const int32_t unit = static_cast<int32_t>((at - row_at) / places);
    const int64_t unit_at = row_at + static_cast<int64_t>(unit) * places;
    // this share's tiles: none if it holds only places before the first
    const int32_t lo = max(static_cast<int32_t>(at - unit_at) - kUnitCost, 0);
    const int32_t hi = static_cast<int32_t>(last - unit_at < places ? last - unit_at : places) - kUnitCost;
    at = unit_at + hi + kUnitCost;
    if (lo >= hi) continue;
    const int64_t r0 = static_cast<int64_t>(unit / A.Hk) * F::BM;
    // the first tile is requested before the row's paths and Q are waited for
    f.q = Seq{static_cast<int64_t>(s) * A.nodes, uniform(A.n_row ? A.n_row[s] : A.nodes), uniform(A.ctx_len[s]), s};
    f.begin_keys(r0, unit % A.Hk);
    f.request(lo, 0);
    if (seen != s) {
      q = uniform(tree_seq(A, s, threadIdx.x == 0, &paths));
      seen = s;
    }
    int2* unit_meta = meta + static_cast<size_t>(s) * ts.units_per_row + unit;
    if (q.n == 0) {  // parents refused
      if (lo == 0 && threadIdx.x == 0) *unit_meta = make_int2(0, 0);
      wait_loads<0>();
    } else {
      f.begin_rows(paths);
      f.keys(lo, hi);
      if (lo == 0 && threadIdx.x == 0) {
        // the last workgroup of the unit: the largest w' with w' T / W <= its last place
        const int64_t end = unit_at + places - 1;
        *unit_meta = make_int2(static_cast<int>(w), static_cast<int>(((end + 1) * W - 1) / total - w) + 1);
      }
      int t;
      const int head = f.row_head(&t);
      if (head >= 0) {
        if (lo == 0 && hi == tiles) {
          f.write_out(head);
        } else {
          const size_t row = (static_cast<size_t>(2) * w + (lo == 0 ? 1 : 0)) * F::BM + f.wave * 32 + f.col;
          f.write_part(A.part + row * D, A.part + tree_ml_offset(ts, D) + row * 2);
        }
      }
    }
    __syncthreads();  // every wave is done with the buffers
  }
}

// Joins the shares of a unit, in the order of the workgroups.  A wave takes one
// row: D / 4 lanes hold its elements, 256 / D groups of them every 256 / D-th share.
template <int D>
__global__ __launch_bounds__(256) void tree_join_kernel(AttnArgs A, TreeSplit ts) {
  constexpr int LPR = D / 4, NG = 64 / LPR;
  const int64_t u = blockIdx.x;
  const int s = static_cast<int>(u / ts.units_per_row), unit = static_cast<int>(u - static_cast<int64_t>(s) * ts.units_per_row);
  const int2 mt = *(reinterpret_cast<const int2*>(A.part + tree_meta_offset(ts, D)) + u);
  const int count = mt.y;
  if (count <= 1) return;
  const int lr = blockIdx.y * 4 + threadIdx.x / 64;  // row of the unit
  const int64_t r = static_cast<int64_t>(unit / A.Hk) * ts.rows_per_unit + lr;
  const int32_t n = A.n_row ? A.n_row[s] : A.nodes;
  if (lr >= ts.rows_per_unit || r >= static_cast<int64_t>(n) * A.G) return;
  const int lane = threadIdx.x & 63, c = (lane % LPR) * 4, g = lane / LPR;
  const float* ml = A.part + tree_ml_offset(ts, D);
  auto slot = [&](int i) {
    return (static_cast<size_t>(2) * (mt.x + i) + (i == 0 ? 1 : 0)) * ts.rows_per_unit + lr;
  };
  float m = -INFINITY;
  for (int i = lane; i < count; i += 64) m = fmaxf(m, ml[slot(i) * 2]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  const float ref = m == -INFINITY ? 0.f : m;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
#pragma unroll 4
  for (int i = g; i < count; i += NG) {
    const size_t at = slot(i);
    const float wt = __builtin_amdgcn_exp2f(ml[at * 2] - ref);
    l += wt * ml[at * 2 + 1];
    sum += wt * load4(A.part + at * D + c);
  }
#pragma unroll
  for (int d = LPR; d < 64; d <<= 1) {
    l += __shfl_xor(l, d, 64);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], d, 64);
  }
  if (g != 0) return;
  sum *= 1.0f / l;
  const int t = static_cast<int>(r / A.G), head = unit % A.Hk * A.G + static_cast<int>(r % A.G);
  const size_t at = ((static_cast<size_t>(s) * A.nodes + t) * A.Hq + head) * D + c;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.o) + at) =
      make_uint2(pack2_bf16(sum[0], sum[1]), pack2_bf16(sum[2], sum[3]));
}

namespace {

// Row blocks of 32, 64 or 128 rows, the smallest that holds the row's
// (node, head) pairs of one KV head, 128 at most; as many workgroups as fit the
// card at once: LDS holds 1, 2 or 4 of them per CU (D 256, 128, 64).
TreeSplit tree_split(int Hk, int G, int D, int nodes) {
  TreeSplit t;
  const int rows = nodes * G;
  t.rows_per_unit = rows <= 32 ? 32 : (rows <= 64 ? 64 : 128);
  t.units_per_row = (rows + t.rows_per_unit - 1) / t.rows_per_unit * Hk;
  t.workgroups = 256 * (D == 256 ? 1 : (D == 128 ? 2 : (t.rows_per_unit == 128 ? 2 : 4)));
  return t;
}

}  // namespace

size_t tree_bf16_part_bytes(int64_t batch, int Hk, int G, int D, int nodes) {
  const TreeSplit t = tree_split(Hk, G, D, nodes);
  return tree_meta_offset(t, D) * sizeof(float) + static_cast<size_t>(batch) * t.units_per_row * sizeof(int2);
}

template <int D, int RW>
static void launch_tree_rows(const AttnArgs& a, const TreeSplit& t, hipStream_t s) {
  typedef TreeTiles<D, RW> F;
  hipLaunchKernelGGL((attn_tree_kernel<D, RW>), dim3(t.workgroups), dim3(F::THREADS), F::LDS, s, a, t);
}

template <int D>
static int launch_tree_bf16_t(const AttnArgs& a, hipStream_t s) {
  const TreeSplit t = tree_split(a.Hk, a.G, D, a.nodes);
  if (!grid_fits(static_cast<int64_t>(a.n_seqs) * t.units_per_row, 256)) return static_cast<int>(hipErrorInvalidValue);
  if (t.rows_per_unit == 32) launch_tree_rows<D, 1>(a, t, s);
  else if (t.rows_per_unit == 64) launch_tree_rows<D, 2>(a, t, s);
  else launch_tree_rows<D, 4>(a, t, s);
  int e = static_cast<int>(hipGetLastError());
  if (e != 0) return e;
  const int rows = a.nodes * a.G < t.rows_per_unit ? a.nodes * a.G : t.rows_per_unit;
  hipLaunchKernelGGL((tree_join_kernel<D>), dim3(a.n_seqs * t.units_per_row, (rows + 3) / 4), dim3(256), 0, s, a, t);
  return static_cast<int>(hipGetLastError());
}

int launch_tree_bf16(const AttnArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (a.D) {
    case 64: return launch_tree_bf16_t<64>(a, s);
    case 128: return launch_tree_bf16_t<128>(a, s);
    case 256: return launch_tree_bf16_t<256>(a, s);
    default: return static_cast<int>(hipErrorInvalidValue);
  }
}

template <int D>
static int launch_prompt_bf16_t(const AttnArgs& a, int64_t tiles, hipStream_t s) {
  typedef PromptTiles<D> F;
  if (!grid_fits(tiles * a.Hk, F::THREADS)) return static_cast<int>(hipErrorInvalidValue);
  hipLaunchKernelGGL((attn_prompt_kernel<D>), dim3(static_cast<unsigned>(tiles * a.Hk), a.n_split), dim3(F::THREADS), F::LDS,
                     s, a);
  return static_cast<int>(hipGetLastError());
}

int launch_prompt_bf16(const AttnArgs& a, int64_t tiles, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (a.D) {
    case 64: return launch_prompt_bf16_t<64>(a, tiles, s);
    case 128: return launch_prompt_bf16_t<128>(a, tiles, s);
    case 256: return launch_prompt_bf16_t<256>(a, tiles, s);
    default: return static_cast<int>(hipErrorInvalidValue);
  }
}

}  // namespace gdn
