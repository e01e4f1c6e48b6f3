// Shapes of the decode attention's launches: shared by the kernels and the
// entry points that lay workspaces out. Plain C++.
#pragma once
#include <limits.h>
#include <stdint.h>

namespace pkv {

// Query heads a head unit takes: one or two blocks of 8 (the N of a product).
inline int decode_rows(int group) { return group <= 8 ? 8 : 16; }

// CTAs of `warps` warps that an SM holds, and steps of a warp's ring.
// Four warps: three CTAs with two steps each, as the cost that a sequence has
// by itself hides behind the others' (256 sequences of 20 to 200 tokens, 8 x 4
// heads of 64: 23.8 us against 27.9 with two CTAs and three steps; 4 x 16
// heads of 77928 tokens 185 against 195). Blocks of 16 query heads and the
// decode step need the registers of two (a step of 128 sequences: 38.7 us
// against 40.9).
// Eight warps, one CTA, where the (sequence, unit) pairs are fewer than a
// quarter of the SMs: fewer parts to join (8 x 8 heads of 4096 tokens: 11.5 us
// against 14.7, 16 heads of 300: 5.4 against 6.0; but 64 pairs of 77928 tokens
// 195 against 185).
constexpr int decode_ctas_per_sm(int rows, bool fused, int warps) {
  return warps == 8 ? 1 : rows == 8 && !fused ? 3 : 2;
}
constexpr int decode_stages(int rows, bool fused, int warps) {
  return decode_ctas_per_sm(rows, fused, warps) == 3 ? 2 : 3;
}
inline int decode_warps(int n_seqs, int units, int num_sms) {
  return 4LL * n_seqs * units < num_sms ? 8 : 4;
}

// CTAs of a unit: one where the units alone fill the GPU.
inline int decode_ranks(int units, int rows, bool fused, int warps, int num_sms) {
  const int n = num_sms * decode_ctas_per_sm(rows, fused, warps) / units;
  return n > 1 ? n : 1;
}

// CTAs of any launch whose units have more than one.
inline int decode_most_ctas(int num_sms) { return 3 * num_sms; }

// Tokens that a warp takes at a time (8 KB of K and V).
constexpr int decode_step(int D) { return D == 64 ? 32 : 16; }

// Tiles that are not worth a join, while parts of them leave CTAs idle
// (with tiles of eight warps, 64 KB, 1, 2, 3 and 4 measured: 7.3, 5.3, 5.3, 5.3
// us for 16 heads of 300 tokens; 9.4, 10.2, 11.1, 12.0 for a step of two
// sequences of up to 1000, 8 x 2 heads; 12.3, 11.8, 12.1, 11.6 for 8 x 8 heads
// of 4096; with tiles of four, 32 KB: 16.4, 15.4, 14.7, 13.4 for the last).
constexpr int decode_part_tiles(int warps) { return warps == 8 ? 2 : 3; }

// A sequence's own cost in tiles, in the line that the ranks share (1, 2, 3
// and 5 tiles measured: a step of 128 sequences 38.8, 38.1, 38.8, 38.9 us).
constexpr int kSeqCost = 2;

// log2 of the tokens of a tile: a step of all warps, or the finest multiple
// that keeps the line of the longest possible sequences, every sequence's cost
// included, within 31 bits.
inline int decode_tile_shift(int D, int warps, int n_seqs, long long most_tokens) {
  int shift = 0;
  while ((1 << shift) < decode_step(D) * warps) ++shift;
  while (((most_tokens >> shift) + 1 + kSeqCost) * n_seqs > INT_MAX) ++shift;
  return shift;
}

}  // namespace pkv
