// What the tiles of attention over shared prefixes are thought to take, by which they
// are divided between the workgroups.  Plain constexpr C++ with no HIP types, so the
// host tests compile it too.  Internal to the library (not part of the public ABI).
#pragma once

#include <stdint.h>

namespace dl {

constexpr int kStreamRows = 16, kSmallRows = 64;

// Lengths of tiles in units of about 0.1 us of a workgroup (of a wave, for the
// stream): what a tile's beginning and end take, and what a group of 32 tokens takes.
// Measured with heads of 128 on a full card: 0.8 us a group for 64 rows (0.9 to 1.2
// beside tiles of 128), 1.15 for 128, 1.6 for a wave's 16; a workgroup that goes on
// from one tile to the next loses 8 to 10 us, of which 5 pass until the first product.
//
// Heads of 256 have no tiles of a wave: a rest of up to 16 rows is a workgroup's as one
// of 64 is, and takes what that takes.  Counted as a wave's it got 1.8 times its share:
// 16 heads on 2, 16 sequences of 9 rows over four prefixes of 20,480 tokens took 158 us
// so, 119 as it is; 64 of one row with 3,000 tokens of their own over 4,096, 72 and 56;
// 16 of one row with 300 over 30,720, 37.2 and 36.9.
template <int D>
struct Cost {
  static constexpr int kRows = D == 256 ? 64 : 128;     // rows of a tile
  static constexpr bool kStreams = D != 256;            // up to 16 rows are a wave's
  static constexpr bool is_wave(int rows) { return kStreams && rows <= kStreamRows; }
  static constexpr int per_group(int rows) {
    const int units = (is_wave(rows) ? 16 : rows <= kSmallRows ? 9 : 12) * D / 128;
    return units > 1 ? units : 1;
  }
  static constexpr int begin(int rows) { return is_wave(rows) ? 40 : 80; }
  static constexpr int of(int rows, int groups) { return groups == 0 ? 0 : begin(rows) + groups * per_group(rows); }
};

// Contexts that are short by the table's width or the window, and few rows, take one
// launch, a tile of 16 rows a workgroup: at most short_tokens(D, short_tiles(..)) tokens
// that a row sees.  The tiles are counted as of sequences of equal rows.
//
// One launch costs by its longest tile and its rounds of workgroups (two a CU, heads of
// 256 one), the planned way about 15 us and then less a token.  Us in one launch and
// planned, 32 heads on 8 of 64, 40 on 8 of 128, 16 on 2 of 256:
//   64   256 tiles of 4,096 tokens 16.1, 24.9; 512 23.7, 26.0; 800 44.0, 45.5; 1,024
//        43.3, 34.0, of 2,048 26.9, 28.8; 2,016 of 2,048 51.2, 52.8, of 4,096 82.3, 76.9
//   128  256 tiles of 2,112 tokens 13.8, 26.5, of 2,816 16.6, 29.9; 512 of 2,816 30.7,
//        32.6; 768 of 1,536 30.8, 35.3; 800 of 1,536 42.8, 45.7, of 2,048 50.6, 47.2; 1,024
//        of 1,024 34.4, 34.2 or 36.2, 42.1, of 2,048 50.5, 39.2 or 51.2, 51.3; 1,376 of
//        512 41.1, 42.0, of 1,024 52.3, 49.4
//   256  24 tiles of 1,024 tokens 15.5, 20.1, of 2,048 24.4, 20.9; 64 of 1,536 20.1, 22.5;
//        200 of 2,560 29.9, 39.7; 304 of 1,536 39.4, 39.9, of 2,048 48.3, 42.7; 640 of 768
//        37.3, 41.7, of 1,536 57.4, 51.0; 800 of 512 40.9, 41.8, of 768 49.9, 45.8
// The most tokens are where one long sequence among short ones, that the width does not
// tell from a batch of long ones, still loses little: 15.6 and 16.9 us for one tile of
// 4,096 tokens and heads of 64, 16.4 and 17.3 for 2,816 and 128, 28.8 and 18.3 for 2,560
// and 256 (where 200 such tiles gain as much).
constexpr int64_t short_tiles(int64_t T, int n_seq, int hq, int hkv) {
  const int64_t rows = (T * (hq / hkv) + n_seq - 1) / n_seq;   // of a sequence
  return n_seq * ((rows + kStreamRows - 1) / kStreamRows) * hkv;
}
constexpr int short_tokens(int D, int64_t tiles) {
  if (D == 64) return tiles <= 800 ? 4096 : tiles <= 2048 ? 2304 : 0;
  if (D == 128) return tiles <= 512 ? 2816 : tiles <= 800 ? 1792 : tiles <= 1216 ? 1024 : 0;
  if (tiles <= 256) return tiles <= 109 ? 1024 + 14 * (int)tiles : 2560;
  return tiles <= 400 ? 1536 : tiles <= 640 ? 896 : tiles <= 800 ? 512 : 0;
}

}  // namespace dl
