// The order of row blocks (gdn_rank.h) on the host: over lengths of 1 to 1024
// tokens, groups of 1 to 64 heads and batches of 1 to 64 sequences every number
// names a block of its own, all blocks are named, in falling order of their keys,
// and a number past the last names none.  Exit status 0, or 1 with the failing
// batch on stderr.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "gdn_rank.h"

namespace {

constexpr int BM = 256;

struct HostLanes {
  typedef gdn::RowBlocks<BM> Blocks;
  std::vector<Blocks> seqs;
  template <class F>
  int32_t sum(F f) const {
    int64_t v = 0;
    for (size_t i = 0; i < seqs.size(); ++i) v += f(seqs[i], static_cast<int>(i));
    return static_cast<int32_t>(v);
  }
  template <class F>
  int32_t max(F f) const {
    int32_t v = 0;  // as of a lane without a sequence
    for (size_t i = 0; i < seqs.size(); ++i) v = std::max(v, static_cast<int32_t>(f(seqs[i], static_cast<int>(i))));
    return v;
  }
  template <class F>
  uint64_t ballot(F f) const {
    uint64_t v = 0;
    for (size_t i = 0; i < seqs.size(); ++i) v |= static_cast<uint64_t>(f(seqs[i], static_cast<int>(i))) << i;
    return v;
  }
  template <class F>
  int32_t at(F f, int lane) const { return f(seqs[lane], lane); }
};

// Keys of block b by walking its rows' tokens, from the definition alone.
int64_t keys_of(int32_t n, int32_t ctx, int32_t G, int64_t b) {
  const int64_t rows = static_cast<int64_t>(n) * G, last = std::min((b + 1) * BM, rows) - 1;
  return ctx + last / G + 1;
}

bool check(const std::vector<std::pair<int32_t, int32_t>>& batch, int32_t G) {
  HostLanes lanes;
  std::vector<std::vector<char>> seen;
  int64_t total = 0;
  for (const auto& s : batch) {
    lanes.seqs.emplace_back(s.first, s.second, G);
    const int64_t blocks = (static_cast<int64_t>(s.first) * G + BM - 1) / BM;
    seen.emplace_back(blocks, 0);
    total += blocks;
  }
  int64_t longest = INT64_MAX;
  int s = 0;
  int32_t b = 0;
  const char* wrong = nullptr;
  for (int64_t r = 0; r < total && !wrong; ++r) {
    if (!gdn::ranked_block(lanes, static_cast<int32_t>(r), &s, &b)) wrong = "names no block";
    else if (s < 0 || s >= static_cast<int>(batch.size()) || b < 0 || b >= static_cast<int64_t>(seen[s].size())) wrong = "names a block that is not there";
    else if (seen[s][b]++) wrong = "names a block again";
    else if (keys_of(batch[s].first, batch[s].second, G, b) > longest) wrong = "is out of order";
    else longest = keys_of(batch[s].first, batch[s].second, G, b);
    if (wrong) fprintf(stderr, "number %lld of %lld %s; G %d,", static_cast<long long>(r), static_cast<long long>(total), wrong, G);
  }
  if (!wrong && gdn::ranked_block(lanes, static_cast<int32_t>(total), &s, &b)) {
    wrong = "past the last";
    fprintf(stderr, "a number past the last names a block; G %d,", G);
  }
  if (wrong) {
    for (const auto& q : batch) fprintf(stderr, " (%d, %d)", q.first, q.second);
    fprintf(stderr, "\n");
  }
  return !wrong;
}

}  // namespace

int main() {
  int64_t batches = 0;
  for (int32_t G = 1; G <= 64; ++G)
    for (int32_t n = 1; n <= 1024; ++n, batches += 2)
      if (!check({{n, 0}}, G) || !check({{n, 5}, {n, 5}}, G)) return 1;
  std::mt19937 rng(1);
  auto draw = [&](int lo, int hi) { return lo + static_cast<int>(rng() % static_cast<uint32_t>(hi - lo + 1)); };
  for (int i = 0; i < 4000; ++i, ++batches) {
    const int S = i % 8 == 0 ? 64 : draw(1, 64), G = draw(1, 64), kind = draw(0, 3);
    std::vector<std::pair<int32_t, int32_t>> batch;
    for (int s = 0; s < S; ++s) {
      if (kind == 0 && s > 0) batch.push_back(batch[0]);                              // all alike
      else if (kind == 1 && s > 0 && draw(0, 1)) batch.push_back(batch[draw(0, s - 1)]);  // some alike
      else if (kind == 2) {  // all end at the same number of keys
        const int n = draw(0, 300);
        batch.emplace_back(n, 300 - n);
      } else batch.emplace_back(draw(0, 5) ? draw(1, 400) : 0, draw(0, 1) ? draw(0, 400) : 0);
    }
    if (!check(batch, G)) return 1;
  }
  // the longest lengths: the last blocks' numbers and keys
  HostLanes far;
  far.seqs.emplace_back((1 << 30) - 4096, (1 << 30) - 16, 1);
  int s;
  int32_t b;
  if (!gdn::ranked_block(far, 0, &s, &b) || b != far.seqs[0].blocks - 1) return 1;
  if (!gdn::ranked_block(far, far.seqs[0].blocks - 1, &s, &b) || b != 0) return 1;
  printf("row blocks ok: %lld batches\n", static_cast<long long>(batches));
  return 0;
}
