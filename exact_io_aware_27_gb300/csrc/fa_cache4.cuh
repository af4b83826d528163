// Layout of the paged cache in 4 bits, uint8 [pages, Hkv, page / 16, 1152 G], for heads of
// G = 1 (d <= 64) or 2 groups of 64 channels.
//
// value = min + scale * code, code 0 .. 15, with a pair (scale, min) in bf16 for each row and
// group. Sixteen rows of a head are one block, so that the attention kernel copies K, V
// and their pairs of 16 keys with one bulk copy. Within a block everything is a 32-bit
// word: 8 codes, channels 8 w .. 8 w + 7 of a group (w = 0 .. 7), the lowest channel in the
// lowest bits; or a pair, scale in the lower half. The order of the words is the one in
// which a lane of the products (16 x 8 x 16, lane = 4 g + t) needs them, so that it loads 8 or
// 16 bytes at a time and a warp without bank conflicts:
//   K codes   row r, group j, word w = 2 t + u   at  8 G r + 2 G t + 2 j + u     (lanes g = r % 8)
//   V codes   row r, group j, word w = g         at  128 G + 128 j + 4 (4 g + t) + i
//                                                    with r = 2 t + i % 2 + 8 (i / 2)
//   pairs     row r, K (s = 0) or V (1), group j at  256 G + 2 G r + G s + j
#pragma once

#include "sm103.cuh"

namespace fa {

constexpr int kRows4 = 16;        // rows of a block
constexpr int kBlock4 = 1152;     // bytes of a block per group
__host__ __device__ constexpr int groups4(int d) { return d > 64 ? 2 : 1; }

FA_DEV int k_word4(int G, int r, int j, int w) {
  return 8 * G * r + 2 * G * (w >> 1) + 2 * j + (w & 1);
}
FA_DEV int v_word4(int G, int r, int j, int w) {
  return 128 * G + 128 * j + 4 * (4 * w + ((r & 7) >> 1)) + (r & 1) + 2 * (r >> 3);
}
FA_DEV int pair_word4(int G, int r, int s, int j) { return 256 * G + 2 * G * r + G * s + j; }

}  // namespace fa
