// Tile and k-splits of the shared expert's bf16 products: the rule by itself, host code that a test compiles too.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace {

// Floats that a product's k-splits may take, and how many splits
constexpr int64_t PARTIAL = 512ll * 128 * 128;
constexpr int MAX_SPLITS = 16;

// Tile and k-splits of a product, by an estimate of its time from what the tiles measured (us per k-tile of 64, operands
// from HBM).  256 x 256: 1.5 with one workgroup on each CU.  128 x 128 in two stages: 0.85 where a CU has one workgroup, 1.05
// for two at once; in four stages (one workgroup fills a CU's LDS): 0.62, the loads' latency hidden by their depth instead
// of by the other workgroup.  64 x 128 in three stages: 0.53 and 0.75.  256 x 128 in three: 0.85.  So the large tiles are 1.4
// times as fast per product once every CU has one, and the small ones win where they would leave CUs idle: 777 tokens of the
// skewed workload's widths take 36 us forward in 64 x 128 or deep 128 x 128 tiles, 49 in 128 x 128, 82 in 256 x 256; 2048
// tokens 53, 62 and 93; 2048 tokens of the DeepSeek-V3-shaped widths 179, and 200 without the 256 x 128 tile; 16384 tokens
// 1213 in 256 x 256.  Splitting k costs the fp32 sums' way to memory and back and a second launch; 128 tokens of those widths
// take 44 us with splits and 80 without.
struct Choice {
  int tile, splits;
};
const struct {
  int bm, bn, per_cu;
  double alone, full, fixed;  // us: a k-tile with one workgroup on the CU, with per_cu of them, and a tile's two ends
} TILES[] = {{256, 256, 1, 1.5, 1.5, 5.0}, {128, 128, 2, 0.85, 1.05, 3.0}, {128, 128, 1, 0.62, 0.62, 3.0}, {64, 128, 2, 0.53, 0.75, 2.5}, {256, 128, 1, 0.85, 0.85, 3.5}};
int64_t tiles_of(int t, int64_t M, int64_t cols) { return ((M + TILES[t].bm - 1) / TILES[t].bm) * ((cols + TILES[t].bn - 1) / TILES[t].bn); }
double join_us(int64_t floats) { return 4.0 + 8.0 * floats / 3.5e6; }  // sums to memory and back

Choice choose(int64_t M, int64_t cols, int nkt) {
  Choice best{0, 1};
  double least = 1e30;
  for (int t = 0; t < 5; ++t) {
    const int64_t n = tiles_of(t, M, cols);
    for (int s = 1; s <= MAX_SPLITS; ++s) {
      if (s > 1 && (nkt / s < 4 || s * M * cols > PARTIAL)) break;
      const int64_t slots = 256 * TILES[t].per_cu, rounds = n * s / slots, rest = n * s % slots;
      const double kt = (double)((nkt + s - 1) / s);
      const double us = rounds * (kt * TILES[t].full + TILES[t].fixed) +
                        (rest ? kt * (rest <= 256 ? TILES[t].alone : TILES[t].full) + TILES[t].fixed : 0.0) +
                        (s > 1 ? join_us(s * M * cols) : 0.0);
      if (us < least) {
        least = us;
        best = {t, s};
      }
    }
  }
  return best;
}

struct Product {
  int64_t M, cols;  // cols: of a row of its partial sums
  int nkt;          // k-tiles of 64
};

// The same for the three gradients of one launch: the tile for all of them and each one's splits, towards sums of equal
// lengths.  Their workgroups fill the CUs one after another, so their times add up, but for the last one to start.
Choice choose_grads(const Product (&p)[3], int (&splits)[3]) {
  double least = 1e30;
  Choice best{0, 1};
  int64_t longest = 1;
  for (const Product& g : p) longest = std::max<int64_t>(longest, g.nkt);
  for (int t = 0; t < 3; ++t)
    for (int64_t len = longest; len >= 4 || len == longest; len = len * 3 / 4) {  // k-tiles of a sum, at most
      double work = 0, last = 0;
      int64_t floats = 0, n = 0;
      int sp[3];
      bool any = false;
      for (int i = 0; i < 3; ++i) {
        const int64_t nkt = p[i].nkt, cols = p[i].cols;
        int64_t s = std::min<int64_t>(MAX_SPLITS, (nkt + len - 1) / len);
        if (s > 1 && (nkt / s < 4 || floats + s * p[i].M * cols > PARTIAL)) s = 1;
        if (s > 1) floats += s * p[i].M * cols;
        sp[i] = (int)s;
        any |= s > 1;
        const int64_t tiles = tiles_of(t, p[i].M, cols) * s;
        const double kt = (double)((nkt + s - 1) / s);
        n += tiles;
        work += tiles * (kt * TILES[t].full + TILES[t].fixed);
        last = std::max(last, kt * TILES[t].alone + TILES[t].fixed);
      }
      const int64_t slots = 256 * TILES[t].per_cu;
      const double us = (n <= 256 ? last : std::max(last, work / slots + 0.4 * last)) + (any ? join_us(floats) : 0.0);
      if (us < least) {
        least = us;
        best.tile = t;
        for (int i = 0; i < 3; ++i) splits[i] = sp[i];
      }
      if (len <= 4) break;
    }
  return best;
}

}  // namespace
