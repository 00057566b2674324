// The order of a packed batch's row blocks: by falling number of keys, so that
// the longest start first, whatever the order of the sequences.  Plain C++ over
// a set of lanes, so the same code runs on a wave and on the host.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define GDN_LANES __host__ __device__ inline
#else
#define GDN_LANES inline
#endif

namespace gdn {

// One sequence, cut into blocks of BM of its n G (token, head) rows.  Block b
// attends ctx + min(n, floor(((b + 1) BM - 1) / G) + 1) keys: more than block
// b - 1, except that the last two attend the same keys where the heads of the last
// token lie in both (0 < n G mod BM < G; G <= BM).
template <int BM>
struct RowBlocks {
  int32_t n, ctx, G, blocks;
  GDN_LANES RowBlocks(int32_t tokens, int32_t cached, int32_t group)
      : n(tokens), ctx(cached), G(group), blocks(static_cast<int32_t>((static_cast<int64_t>(tokens) * group + BM - 1) / BM)) {}
  // its first block of at least `keys` keys (blocks: it has none), which is also
  // the number of its blocks of fewer
  GDN_LANES int32_t first(int32_t keys) const {
    const int32_t need = keys - ctx;
    if (need <= 1) return 0;
    return need > n ? blocks : static_cast<int32_t>(static_cast<int64_t>(need - 1) * G / BM);
  }
  // number of its blocks of exactly `keys` keys: 0, 1 or 2
  GDN_LANES int32_t of(int32_t keys) const { return first(keys + 1) - first(keys); }
};

// Row block number r in falling order of keys, equal ones in order of their
// sequences; every block has one number, 0 to their count - 1.  The number of
// blocks of at least `keys` keys is a sum over the sequences, so a search over
// `keys` finds the block's, and the counts of exactly so many keys find its
// sequence.  Lanes holds one sequence per lane (at most 64; n = 0 where there is
// none): sum, max and ballot of f(sequence, lane) over the lanes, and its value
// at one of them.  False: there are no more blocks.
template <class Lanes>
GDN_LANES bool ranked_block(const Lanes& lanes, int32_t r, int* seq, int32_t* block) {
  typedef typename Lanes::Blocks Blocks;
  if (r >= lanes.sum([](const Blocks& q, int) { return q.blocks; })) return false;
  // the largest number of keys that more than r blocks have at least
  int32_t lo = 1, hi = 1 + lanes.max([](const Blocks& q, int) { return q.n > 0 ? q.ctx + q.n : 0; });
  auto at_least = [&](int32_t keys) { return lanes.sum([=](const Blocks& q, int) { return q.blocks - q.first(keys); }); };
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (at_least(mid) > r) lo = mid;
    else hi = mid;
  }
  // block number `skip` among those of exactly lo keys: 0, 1 or 2 per sequence
  const int32_t skip = r - at_least(lo + 1);
  const uint64_t one = lanes.ballot([=](const Blocks& q, int) { return q.of(lo) >= 1; });
  const uint64_t two = lanes.ballot([=](const Blocks& q, int) { return q.of(lo) >= 2; });
  auto before = [=](int lane) {
    const uint64_t mask = (1ull << lane) - 1;
    return static_cast<int32_t>(__builtin_popcountll(one & mask) + __builtin_popcountll(two & mask));
  };
  const uint64_t holds =
      lanes.ballot([=](const Blocks& q, int lane) { return before(lane) <= skip && skip < before(lane) + q.of(lo); });
  if (holds == 0) return false;
  const int s = __builtin_ctzll(holds);
  *seq = s;
  *block = lanes.at([=](const Blocks& q, int lane) { return q.first(lo) + skip - before(lane); }, s);
  return true;
}

}  // namespace gdn
