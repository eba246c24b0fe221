// How an expert's rows are spread over its row tiles.  Plain C++: the kernels and
// host code share it.
#pragma once

namespace zc {

// First of the blocks of rows that tile mt of `tiles` holds, where `blocks` of them
// are spread evenly: blocks * mt / tiles (tile mt ends with first_block(.., mt + 1, ..)).
// That product passes 31 bits from 2^21 rows on in blocks of 16 and tiles of 128, so
// it is taken of the remainder alone: below tiles^2, and no kernel has more than
// 2^15 row tiles of an expert (fewer than 2^22 rows in tiles of 128 or more).
constexpr int first_block(int blocks, int mt, int tiles) {
  const int each = blocks / tiles;
  return each * mt + (blocks - each * tiles) * mt / tiles;
}

// The same in one step, for products of at most 2^31 (fewer than 2^22 rows in blocks
// of 32 and tiles of 256: 2^17 * 2^14, 31 bits passed by one).
constexpr int first_block32(int blocks, int mt, int tiles) {
  return static_cast<int>(static_cast<unsigned>(blocks) * static_cast<unsigned>(mt) /
                          static_cast<unsigned>(tiles));
}

}  // namespace zc
