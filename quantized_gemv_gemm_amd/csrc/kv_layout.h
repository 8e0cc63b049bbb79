// Where a token's elements lie in the paged K/V cache (host and device).
//
// A cache is [pages][kv_heads][block][D] elements; the block * D elements of one
// (page, head) are block / 16 tiles of 16 tokens, each 16 * D elements in the order
// in which the attention kernel's matrix operands are read: a load of a wavefront is
// whole 128-byte lines (K) or 512-byte runs (V), and what it brings is an operand as it
// stands, with nothing moved through LDS or between registers.
//   bf16:  K tile [D/32][4 g][16 p][8 e]        d = 32 c + 8 g + e
//          V tile [D/16][2 o][16 m][8 i]        token 8 o + i, d = 16 c + m
//   e4m3:  K tile [D/64][4 g][16 p][16 e]       d = 64 c + 16 g + e
//          V tile [D/32][2 o][16 m][2 u][8 i]   token 8 o + i, d = 32 c + 16 u + m
// Token t of a K tile is at place p with bits (t2, t3, t1, t0): two tiles together are
// then read as two operands of 16 tokens whose scores leave every lane with eight
// consecutive tokens of one query row, the run of tokens that a V load holds.
#pragma once

#include <stdint.h>

namespace tl {

constexpr int kKvTile = 16;       // tokens of a tile
constexpr int kTreeNodes = 64;    // nodes of a drafted tree (bits of a mask word)

#define TL_HD __host__ __device__ inline

// place of token t (0..15) in a K tile
TL_HD int kv_place(int t) { return (t & 3) | (t >> 3 & 1) << 2 | (t >> 2 & 1) << 3; }

// element offset of (token in [0, 16), d) inside a tile; `bytes` is the element size
TL_HD int kv_tile_k(int t, int d, int bytes) {
  const int e = 16 / bytes, w = 4 * e;
  return d / w * (16 * w) + d % w / e * (16 * e) + kv_place(t) * e + d % e;
}
TL_HD int kv_tile_v(int t, int d, int bytes) {
  const int u = 2 / bytes, w = 16 * u;
  return d / w * (16 * w) + t / 8 * (8 * w) + d % 16 * (8 * u) + d % w / 16 * 8 + t % 8;
}

// The same in bytes, as a token's part and a d's part.  K: 16-byte piece p of a row;
// V: element d.
TL_HD int kv_k_token(int t) { return kv_place(t) * 16; }
TL_HD int kv_k_piece(int p) { return p * 256; }
TL_HD int kv_v_token(int t, int bytes) { return t / 8 * 256 + t % 8 * bytes; }
TL_HD int kv_v_element(int d, int bytes) {
  return bytes == 2 ? d / 16 * 512 + d % 16 * 16 : d / 32 * 512 + d % 16 * 16 + d / 16 % 2 * 8;
}

}  // namespace tl
