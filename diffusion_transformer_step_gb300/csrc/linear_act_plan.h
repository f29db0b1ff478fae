// Which way a product with bias, activation and residual goes, and how its depth is split.  From the sizes and the
// operands' alignment alone: the split decides the order of sums, and equal calls give equal bits on any GB300.
#pragma once

namespace dit {

struct LinearActPlan {
  int bn;      // columns of a wide tile; 0: the kernel of few rows
  int splits;  // of the depth
};

// Clusters of c CTAs, one CTA per SM, that run at once. How many exactly depends on which SMs each processing cluster of a
// device has; these are what one GB300 of 152 SMs reports. Where fewer fit, the last ones wait for a second round: slower, with the same
// bits.
inline int clusters_at_once(int c) {
  const int n[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
  return n[c];
}

// Few rows, a cluster per 128 columns: as many splits as still run at once, of two blocks at least; up to 64 rows two CTAs share
// an SM.
inline int few_splits(int rows, int n, int kblocks) {
  const int blocks = (n + 127) / 128, most = kblocks / 2;
  int S = most < 8 ? most : 8;
  const int start = S;
  while (S > 1 && blocks > clusters_at_once(S)) --S;
  if (S < 3 && rows <= 64)
    for (S = start; S > 1 && blocks > 2 * clusters_at_once(S);) --S;
  return S > 1 ? S : 1;
}

// Many rows. Columns of a tile and splits of the depth, by the time that a pair's longest way takes: rounds of tiles, blocks
// of depth in each at what a block of 256, 192 or 128 columns costs, and what a split adds. Splits only where all of them run
// at once, of eight blocks at least. A block's MMAs take 0.27, 0.20 and 0.14 us, a little more where many SMs load. Rows of operands that do
// not start on 128-byte lines (`lines` false) are two lines each to load, which takes longer than that.
inline LinearActPlan wide_plan(int rows, int n, int kblocks, bool lines) {
  const int bns[3] = {256, 192, 128}, block_5ns[2][3] = {{60, 48, 35}, {92, 78, 64}}, split_5ns = 1100;
  LinearActPlan best{256, 1};
  long long least = 0;
  for (int i = 0; i < 3; ++i) {
    const long long tiles = (long long)((rows + 255) / 256) * ((n + bns[i] - 1) / bns[i]);
    const int pairs = clusters_at_once(2);
    for (int S = 1; S <= 4; ++S) {
      if (S > 1 && (kblocks / S < 8 || tiles > clusters_at_once(2 * S))) break;
      const long long way = (tiles + pairs - 1) / pairs * ((kblocks + S - 1) / S) * block_5ns[lines ? 0 : 1][i] + (S > 1 ? split_5ns : 0);
      if (least == 0 || way < least) least = way, best = LinearActPlan{bns[i], S};
    }
  }
  return best;
}

// Up to 128 rows a cluster per 128 columns of the output (65 x 4096 x 4096 10.7 us so, 13.8 in wide tiles, 128 x 12288 x 4096 23.7
// and 24.7; 100 x 8192 x 1024, two waves of clusters, 9.7 and 8.8). The same with up to 256 rows: 129 x 4096 x 4096 14.2 and
// 16.2, 256 x 4096 x 4096 16.6 and 16.6, 200 x 2048 x 1024 8.4 and 6.8, 250 x 8192 x 4096 25.6 and 18.2; left.
inline LinearActPlan linear_act_plan(int rows, int n, int kblocks, bool lines) {
  if (rows <= 128) return LinearActPlan{0, few_splits(rows, n, kblocks)};
  return wide_plan(rows, n, kblocks, lines);
}

}  // namespace dit
