// The 4-bit key/value cache: its format and where each value lies.
//
// A value is minimum + scale * code, code = 0..15, with one fp16 (scale, minimum) per group
// of 32 channels of a token's head: 5 bits a value. A page of P tokens (P = 16..256) of one kv
// head is P / 16 sub-blocks, each self-contained and 20 d bytes long (n = d / 32 groups):
//     k codes 8 d | k scales d | k minima d | v codes 8 d | v (scale, minimum) pairs 2 d
// so that any run of sub-blocks is one contiguous copy. Inside a sub-block the codes lie as
// the tensor cores' operands want them: a lane gets all it needs of a token by one wide
// load, and the loads of a warp touch every shared-memory bank once:
//  - k, token u: four lanes c = 0..3 of n words; word j of lane c holds channels
//    32 j + 8 c .. + 7, channel i in bits 4 i (with n = 8, odd rows swap word halves).
//  - v, token u: row v_row(u) (even tokens of eight before odd ones); eight lanes g of n
//    half-words; half-word j of lane g holds channels 32 j + 4 g .. + 3 (the lane's place
//    in the row is turned by v_turn).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace s2 {
namespace c4 {

__host__ __device__ constexpr int sub_bytes(int d) { return 20 * d; }
__host__ __device__ constexpr int ks_at(int d) { return 8 * d; }
__host__ __device__ constexpr int km_at(int d) { return 9 * d; }
__host__ __device__ constexpr int vc_at(int d) { return 10 * d; }
__host__ __device__ constexpr int vp_at(int d) { return 18 * d; }

// Byte of word (j, c) of token u's k codes.
__host__ __device__ constexpr int k_word(int u, int j, int c, int n) {
  return u * 16 * n + 4 * (c * n + (n == 8 ? j ^ (4 * (u & 1)) : j));
}
__host__ __device__ constexpr int v_row(int u) { return (u & 8) | ((u & 7) >> 1) | ((u & 1) << 2); }
__host__ __device__ constexpr int v_turn(int row, int n) {
  return n == 8 ? 2 * (row & 3) : n == 4 ? 4 * ((row >> 1) & 1) : 0;
}
// Byte of half-word (j, g) of v row `row`, from the start of the v codes.
__host__ __device__ constexpr int v_piece(int row, int j, int g, int n) {
  return row * 16 * n + (g ^ v_turn(row, n)) * 2 * n + 2 * j;
}

// Sub-block of slot `slot` (page * P + place in the page) of kv head h.
__device__ inline size_t sub_of_slot(int slot, int h, int Hkv, int page_shift, int d) {
  const int page = slot >> page_shift, place = slot & ((1 << page_shift) - 1);
  return ((((size_t)page * Hkv + h) << (page_shift - 4)) + (place >> 4)) * sub_bytes(d);
}

}  // namespace c4
}  // namespace s2
