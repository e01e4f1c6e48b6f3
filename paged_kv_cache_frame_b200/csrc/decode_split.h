// How the decode attention's tiles are split over the ranks, and where a
// sequence's parts and their arrival counters lie. The kernel works it out
// from the lengths on the device; the host test from the same code. `Args` is
// DecodeArgs or the test's stand-in for it.
#pragma once
#include "decode_shape.h"
#include "host_device.h"

namespace pkv {

constexpr int kJoin = 32;    // parts that one CTA joins at once (a lane each)
constexpr int kGroup = 16;   // parts joined in a first round where there are more

// The first token that the query of a sequence of `len` sees, and its tiles.
template <typename Args>
PKV_HD int first_seen(const Args& a, int len) {
  return a.window > 0 && len > a.window ? len - a.window : 0;
}
template <typename Args>
PKV_HD uint32_t tiles_of(const Args& a, int len) {
  return ((uint32_t)(len - first_seen(a, len)) + (1u << a.tile_shift) - 1) >> a.tile_shift;
}
template <typename Args>
PKV_HD uint32_t parts_of(const Args& a, uint32_t tiles) {
  return (tiles + a.part_tiles - 1) / a.part_tiles;
}
template <typename Args>
PKV_HD int raw_len(const Args& a, int s) {
  return s < a.c.n_seqs ? index_at(a.c.lens + s) : 0;
}

// A rank's part of the tiles, and what is left of it. The host chooses tiles
// coarse enough for 31 bits.
struct Split {
  bool by_parts;      // a part a rank; else the line
  uint32_t each, more;   // the line: ranks below `more` take each + 1 places, the others `each`
  uint32_t t, end;    // places [t, end) of the line (or parts of all sequences) are left
  // Where place t lies: place `at` of the sequence's `size`.
  int seq;
  uint32_t at, size, tiles;
  int raw, later;     // the lengths of seq and seq + 1 as they stand: read a sequence ahead, as a load
                      // takes about a microsecond while the memory is busy

  PKV_HD uint32_t rank_of(uint32_t place) const {
    const uint32_t lower = more * (each + 1);
    return place < lower ? place / (each + 1) : more + (place - lower) / each;
  }
};

// The tokens of one sequence that the CTA takes.
struct Piece {
  int seq, raw;       // and the sequence's length as it stands: past the table's end there is no new token
  int tok0, tok1;     // tokens [tok0, tok1)
  int r0, parts;      // the sequence's first rank, and in how many it lies
};

// What rank `rank` takes of all sequences' parts and places of the line.
template <typename Args>
PKV_HD void split_range(const Args& a, uint32_t rank, uint32_t parts, uint32_t places, Split& l) {
  l.by_parts = parts <= (uint32_t)a.ranks;
  if (l.by_parts) {
    l.t = rank < parts ? rank : parts;
    l.end = rank + 1 < parts ? rank + 1 : parts;
    l.each = l.more = 0;
  } else {   // more places than ranks
    l.each = places / a.ranks;
    l.more = places - l.each * a.ranks;
    l.t = rank * l.each + (rank < l.more ? rank : l.more);
    l.end = l.t + l.each + (rank < l.more ? 1 : 0);
  }
}

// On to the next sequence's places.
template <typename Args>
PKV_HD void next_sequence(const Args& a, Split& l) {
  ++l.seq;
  l.raw = l.later;
  l.later = raw_len(a, l.seq + 1);
  l.tiles = tiles_of(a, held(a.c, l.raw));
  l.size = l.by_parts ? parts_of(a, l.tiles) : l.tiles ? l.tiles + kSeqCost : 0;
  l.at = 0;
}

// To the sequence of place t, behind sequence `seq`, whose end is place `base`.
template <typename Args>
PKV_HD void seek(const Args& a, Split& l, int seq, uint32_t base) {
  l.seq = seq;
  l.later = raw_len(a, l.seq + 1);
  for (;;) {
    next_sequence(a, l);
    if (l.seq >= a.c.n_seqs || l.t - base < l.size) break;
    base += l.size;
  }
  l.at = l.t - base;
}

template <typename Args>
PKV_HD bool next_piece(const Args& a, uint32_t rank, Split& l, Piece& p) {
  while (l.t < l.end) {
    while (l.at >= l.size && l.seq < a.c.n_seqs) next_sequence(a, l);
    if (l.seq >= a.c.n_seqs) return false;   // cannot be, unless the lengths change under the launch
    uint32_t tile0, tile1;
    if (l.by_parts) {
      tile0 = l.tiles * l.at / l.size;   // tiles <= part_tiles * ranks here
      tile1 = l.tiles * (l.at + 1) / l.size;
      p.r0 = l.t - l.at;
      p.parts = l.size;
      ++l.t;
      ++l.at;
    } else {
      const uint32_t left = l.end - l.t, here = l.size - l.at, n = left < here ? left : here;
      const uint32_t first = l.t - l.at;   // the sequence's first place; its tiles begin kSeqCost later
      tile0 = l.at > kSeqCost ? l.at - kSeqCost : 0;
      tile1 = l.at + n > kSeqCost ? l.at + n - kSeqCost : 0;
      p.r0 = tile0 == 0 ? rank : l.rank_of(first + kSeqCost);
      p.parts = (tile1 == l.tiles ? rank : l.rank_of(first + l.size - 1)) - p.r0 + 1;
      l.t += n;
      l.at += n;
    }
    if (tile0 == tile1) continue;
    p.seq = l.seq;
    p.raw = l.raw;
    const int len = held(a.c, l.raw), seen = first_seen(a, len);
    p.tok0 = seen + (int)(tile0 << a.tile_shift);
    p.tok1 = tile1 == l.tiles ? len : seen + (int)(tile1 << a.tile_shift);
    return true;
  }
  return false;
}

// Part p of a sequence that rank r0 begins: the slot of the workspace of that
// CTA, its second if it begins the sequence, else its first.
template <typename Args>
PKV_HD long long part_slot(const Args& a, int r0, int p, uint32_t unit) {
  return 2LL * ((long long)(r0 + p) * a.units + unit) + (p == 0 ? 1 : 0);
}

// How part `me` of `parts` is joined: more than kJoin parts in two rounds,
// kGroup neighbours first.
struct Join {
  bool two;
  int g0, of;      // the first round: the group's first part, and its parts
  int groups;      // the second: the groups
};
PKV_HD Join join_of(int me, int parts) {
  Join j;
  j.two = parts > kJoin;
  j.g0 = j.two ? me / kGroup * kGroup : 0;
  const int left = parts - j.g0;
  j.of = j.two ? (kGroup < left ? kGroup : left) : parts;
  j.groups = (parts + kGroup - 1) / kGroup;
  return j;
}
// The counters of its arrivals, of 4 for each of the launch's CTAs.
template <typename Args>
PKV_HD long long first_counter(const Args& a, int r0, const Join& j, uint32_t unit) {
  return part_slot(a, r0, j.g0, unit);
}
template <typename Args>
PKV_HD long long second_counter(const Args& a, int r0, uint32_t unit) {
  return 2LL * a.ranks * a.units + part_slot(a, r0, 0, unit);
}

}  // namespace pkv
