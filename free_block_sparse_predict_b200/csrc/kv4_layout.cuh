// Addresses inside a tile of the 4-bit cache: 16 tokens of one KV head (see
// sparge_kv4_t in include/sparge.h for the layout in bytes).
//
// The layout is the m16n8k16 fragment order.  Per 16-token tile the score
// product takes K as its A operand (rows = tokens, k = channels): lane
// (g, t) = (lane / 4, lane % 4) reads word (t, j) of tokens g and g + 8,
// whose eight codes are that lane's A entries of two k-steps.  The output
// product takes V transposed (rows = channels, k = tokens): lane (g, t) reads
// the words of g for tokens 2t, 2t + 1, 2t + 8, 2t + 9, which stand next to
// one another.
#pragma once

#include <cstdint>

namespace sparge {

struct Kv4Tile {
  int32_t d, ng;  // channels, scale groups
  __host__ __device__ int32_t k_word(int tok, int t, int j) const {
    return tok * (d / 2) + (t * (d / 32) + j) * 4;
  }
  __host__ __device__ static int v_pos(int tok) {
    return 4 * ((tok & 7) >> 1) + 2 * (tok >> 3) + (tok & 1);
  }
  __host__ __device__ int32_t v_word(int tok, int w, int g) const {
    return 8 * d + ((w * 8 + g) * 16 + v_pos(tok)) * 4;
  }
  __host__ __device__ int32_t k_scale(int tok) const { return 16 * d + tok * ng * 4; }
  __host__ __device__ int32_t v_scale(int tok) const { return k_scale(tok) + ng * 2; }
  __host__ __device__ int32_t bytes() const { return 16 * (d + 4 * ng); }
};

}  // namespace sparge
