// kvq_kv4.cuh -- the format of the paged cache held in 4 bits.
//
// uint8 [num_pages, 2, num_heads_kv, page_size, 9 D / 16]: of a page the keys of
// every kv head, then the values.  A head's block of a page holds the codes of its
// tokens, D/2 bytes each, and behind them per token and group of 64 dims a
// 4-byte word: the scale in its low half, the zero in its high half, both bf16.
//   value of code c:  zero + scale (c - 8)
// A 32-bit word of codes holds eight dims 8w .. 8w + 7: nibble i < 4 is dim 2i,
// nibble i + 4 dim 2i + 1.  So one shift and one mask give the two codes of
// neighbouring dims, one in each half: a packed pair of bf16 values.
#pragma once

#include <stdint.h>

namespace kvq {
namespace kv4 {

constexpr int kGroup = 64;  // dims that share a scale and a zero

// Bytes of a token's row of one head, codes and scales.
__host__ __device__ constexpr int row_bytes(int head_dim) { return head_dim / 2 + head_dim / 16; }

// Codes i and i + 4 of a word as bf16 pairs 16 + c: the code lands on the upper four
// bits of the fraction of 16.
template <int I>
__device__ __forceinline__ uint32_t pair16(uint32_t w) {
  const uint32_t x = I == 0 ? w << 3 : w >> (4 * I - 3);
  return (x & 0x00780078u) | 0x41804180u;
}

}  // namespace kv4
}  // namespace kvq
