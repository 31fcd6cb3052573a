// Which form an experts' product takes: how many row tiles it has, and how its CTAs share a tile.
// Host arithmetic only.
#pragma once

#include <algorithm>
#include <cstdint>

namespace tbe {

// How CTAs share a tile.
enum Share { kAlone, kPair, kSplit };
constexpr int kMostSplit = 8;

struct ProductForm {
  Share share;
  int cluster;  // CTAs of a tile
};

// Tiles of `tile` rows that `rows` rows of `experts` experts have at most: every expert but one has
// a tile for a single row.
inline int64_t most_row_tiles(int64_t rows, int64_t experts, int64_t tile) {
  const int64_t with_rows = std::min(experts, rows);
  return with_rows + (rows - with_rows) / tile;
}

// The same as expected of experts of unequal sizes: half of a last tile each, at least a tile each.
inline int64_t likely_row_tiles(int64_t rows, int64_t experts, int64_t tile) {
  const int64_t with_rows = std::min(experts, rows);
  return std::min(most_row_tiles(rows, experts, tile),
                  std::max(with_rows, rows / tile + (with_rows + 1) / 2));
}

// kb: blocks of 128 of k.
inline ProductForm product_form(int64_t rows, int64_t n, int64_t kb, int64_t experts, int sms) {
  // A split pays while its parts and their join fit one round with room to spare, so it counts a
  // tile more an expert (257 rows, 3 experts, 500 x 2048: 13.3 us in four parts, 18.4 in eight; 512
  // rows, 2048 x 2048: 12.3 whole, 14.3 in two).
  const int64_t tiles = (rows / 128 + std::min(experts, rows)) * ((n + 127) / 128);
  int split = 1;
  while (split < kMostSplit && tiles * split * 2 <= sms && kb >= split * 4) split *= 2;
  if (split > 1) return {kSplit, split};
  if (sms < 2) return {kAlone, 1};
  // Rounds of tiles over the multiprocessors (a pair takes two), times a tile's time: measured
  // on 65536 rows of 16 experts and 4096 columns, a block of k takes a pair 0.40 us and a lone
  // CTA 0.27, and a tile's start and end 1.43 and 0.76 us (k = 2048: 421 us in pairs, 501 alone;
  // 5000 rows, 8 experts, 1000 x 1008: 21.6 and 18.2).  One expert with a part of a tile: 16 rows,
  // 128000 x 4096: 120.8 in pairs, 104.4 alone; 1 row, 1024 x 128: 10.2 and 8.2.  Of 120 drawn
  // products (up to 65536 rows, 4096 columns, k of 4096) the chosen form, splits included, takes
  // 1.04 times the best form's time on average and 1.26 times at worst.
  const auto rounds = [](int64_t t, int64_t at_once) { return (t + at_once - 1) / at_once; };
  const int64_t alone =
      rounds(likely_row_tiles(rows, experts, 128) * ((n + 127) / 128), sms) * (kb * 27 + 76);
  const int64_t paired =
      rounds(likely_row_tiles(rows, experts, 256) * ((n + 255) / 256), sms / 2) * (kb * 40 + 143);
  return alone < paired ? ProductForm{kAlone, 1} : ProductForm{kPair, 2};
}

}  // namespace tbe
