// The 4-bit K/V cache: its row format and the arguments of the kernels on it.
//
// A row of d channels is d / 64 groups of 64.  A group holds a scale s and a minimum m, both
// bfloat16, and a code c in 0..15 for each channel, which stands for m + c s.
//   codes   d / 2 bytes a row, in 32-bit words of 8 channels: channel 8 j + n of a group in
//           bits [4 n, 4 n + 4) of the group's word j; with two groups (d = 128) their words
//           alternate (word 2 j is group 0's, word 2 j + 1 group 1's).  A quarter of a row
//           then holds equal parts of both groups, and so does each eighth: the operand of a
//           matrix instruction, 16 channels or 16 keys deep, comes from one group only.
//   scales  4 bytes a group: s in the low half, m in the high half.
#pragma once

#include <stdint.h>

namespace stdb {

constexpr int kKv4Group = 64;  // channels that share a scale
constexpr int kKv4Rows = 16;   // a cache's capacity is a multiple of this

// First channel of word `w` of a row.
template <int D>
__host__ __device__ constexpr int kv4_word_channel(int w) {
  return D == 128 ? 64 * (w & 1) + 8 * (w >> 1) : 8 * w;
}

}  // namespace stdb
