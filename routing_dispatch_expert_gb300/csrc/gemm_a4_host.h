// Host arithmetic of the 4-bit GEMM's launch (plain C++; no CUDA types, so it can be checked on a host without a GPU).
#pragma once

#include <cstdint>

namespace moe {
namespace a4 {

// Row tiles of `rows` rows in at most `groups` groups (both positive, groups <= rows): a group of m rows has
// (m - 1) / tile_rows + 1 of them, which sum to no more than this. For one group it is the number itself.
inline int64_t row_tiles_at_most(int64_t rows, int64_t groups, int64_t tile_rows) {
  return (rows - groups) / tile_rows + groups;
}

// Narrow tiles (`split` of them cover a wide one) where all of them run at once.
inline bool narrow_tiles(int64_t wide_tiles, int split, int sms) { return wide_tiles * split <= sms; }

// SM clocks after which a wait gives up: about two seconds, and 8 us for each K block of a tile, since the epilogue waits
// for all of them (a block takes 0.3 - 1 us; K may be 2^31).
inline long long wait_limit(int64_t k_blocks) { return 4000000000LL + 16000LL * k_blocks; }

}  // namespace a4
}  // namespace moe
