// How the 8-bit linear layer shares its work out over clusters of blocks. For
// many tokens: whole waves of tiles first, then the steps of the tiles left
// over. For few: rows to clusters, inputs to their blocks, and as many tokens a
// launch as those hold. Plain arithmetic, for the host, the kernels and tests
// without a GPU.
#pragma once

#ifdef __CUDACC__
#define SFFN_HD __host__ __device__
#else
#define SFFN_HD
#endif

namespace sffn {

constexpr int kL8JoinSteps = 20;    // that take as long as leaving and joining a tile's parts, 8 us
constexpr int kL8LeastSteps = 16;   // of a share

struct L8Split {
  int steps, groups;        // of a tile; clusters
  int whole, left, parted;  // whole waves of tiles, tiles after them, clusters that share those
};

// The steps of the tiles left over go to as many clusters as get kL8LeastSteps each. None may be without steps, since a
// join waits for every cluster between a tile's first and last; and the last of many small parts adds all of them alone
// (256 x 8192 for 192 tokens: 218 us with shares of one step, 25 with 16, 34 not shared).
inline L8Split l8_split(int tiles, int steps, int groups) {
  L8Split w = {steps, groups, tiles / groups, tiles % groups, 0};
  const long long shares = (long long)w.left * steps / kL8LeastSteps;
  w.parted = (int)(shares < groups ? shares : groups);
  // sharing makes the tiles shorter by the clusters that would stand idle, and costs a join
  if ((long long)steps * (w.parted - w.left) <= (long long)kL8JoinSteps * w.parted) w.parted = w.left;
  return w;
}

// What a cluster computes: tiles cluster + i * groups for i < whole, then its share [from, to) of the steps left over.
struct L8Segment {
  int tile, s0, s1;
  bool part;    // others have the rest of the tile
  int slot;     // of the workspace, for its sums
};
struct L8Segments {
  int cluster, i = 0;
  long long at, to;
  SFFN_HD L8Segments(const L8Split& w, int c) : cluster(c) {
    const long long units = (long long)w.left * w.steps;
    at = c < w.parted ? units * c / w.parted : 0, to = c < w.parted ? units * (c + 1) / w.parted : 0;
  }
  SFFN_HD bool next(const L8Split& w, L8Segment& s) {
    if (i < w.whole) {
      s.tile = cluster + i * w.groups, s.s0 = 0, s.s1 = w.steps, s.part = false, s.slot = 0;
      ++i;
      return true;
    }
    if (at >= to) return false;
    const int t = (int)(at / w.steps);
    const long long begin = (long long)t * w.steps, end = begin + w.steps < to ? begin + w.steps : to;
    s.tile = w.whole * w.groups + t, s.s0 = (int)(at - begin), s.s1 = (int)(end - begin);
    s.part = s.s1 - s.s0 < w.steps, s.slot = at == (long long)w.left * w.steps * cluster / w.parted ? 0 : 1;
    at = end;
    return true;
  }
};

// The clusters from .. to that have steps of tile `left` of those left over, of which `cluster` is one (a few each way).
struct L8Sharers {
  int from, to;
};
SFFN_HD inline L8Sharers l8_sharers(const L8Split& w, int left, int cluster) {
  const long long units = (long long)w.left * w.steps, begin = (long long)left * w.steps, end = begin + w.steps;
  L8Sharers s = {cluster, cluster};
  while (units * s.from / w.parted > begin) --s.from;
  while (units * (s.to + 1) / w.parted < end) ++s.to;
  return s;
}
// Where sharer c of the tile has left its sums: its first steps are this tile's, or its last.
SFFN_HD inline int l8_slot(const L8Split& w, int left, int c) {
  return (long long)w.left * w.steps * c / w.parted >= (long long)left * w.steps ? 0 : 1;
}

// ----------------------------------------------------------------- few tokens

constexpr int kL8FewTokens = 32;            // of a launch, at most
constexpr int kL8FewSmem = 200 * 1024;      // of a block: its inputs of every token, sums of its cluster's rows
constexpr int kL8FewRows = 512;             // of a cluster, at most

struct L8Few {
  int nt;                  // column tiles of eight tokens: 1, 2 or 4
  int cs, clusters;        // blocks of a cluster, clusters
  int x_stride, off_sum;   // bytes of a token's codes held by a block, and where the sums begin
  int smem;
};

// The smallest cluster whose blocks hold their share of the tokens' codes, and larger ones while rows are too few to give
// every SM a tile. n outputs, kp inputs (a multiple of 128).
inline L8Few l8_few(int n, int kp, int tokens, int num_sms) {
  L8Few p = {};
  p.nt = tokens <= 8 ? 1 : tokens <= 16 ? 2 : 4;
  for (p.cs = 1;; p.cs *= 2) {
    const int own = (kp / 64 + p.cs - 1) / p.cs * 64, most = num_sms / p.cs, tiles = (n + 15) / 16;
    const int least = (n + kL8FewRows - 1) / kL8FewRows;
    p.x_stride = own + (own % 128 ? 0 : 64);
    p.clusters = most < tiles ? most : tiles;
    if (p.clusters < least) p.clusters = least;
    p.off_sum = 8 * p.nt * p.x_stride;
    p.smem = p.off_sum + (n + p.clusters - 1) / p.clusters * 8 * p.nt * 4;
    const bool spare = n < most * 16 && own > 1024;
    if (p.cs == 8 || (p.smem <= kL8FewSmem && !spare)) return p;
  }
}

// Tokens of a launch: 32, 16 or 8, the most that a cluster of eight holds with their padding and the sums (eight always).
inline int l8_few_tokens(int n, int kp, int num_sms) {
  int t = kL8FewTokens;
  while (t > 8 && l8_few(n, kp, t, num_sms).smem > kL8FewSmem) t /= 2;
  return t;
}

}  // namespace sffn
