// What the tiles of attention over shared prefixes are thought to take, by which they
// are divided between the workgroups.  Plain constexpr C++ with no HIP types, so the
// host tests compile it too.  Internal to the library (not part of the public ABI).
#pragma once

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

}  // namespace dl
