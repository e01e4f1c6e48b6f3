// Host test of the decode attention's split and of append's search, from the
// headers that the kernels include: random batches at the launches' own
// shapes. Exits non-zero on a failure.
#include <algorithm>
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "decode_split.h"

struct Cache {
  const int32_t* lens;
  int n_seqs, table_width, page_size;
};
struct Args {
  Cache c;
  int window, units, ranks, tile_shift, part_tiles;
};

static std::mt19937 rng(11);
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

#define CHECK(x)                                                       \
  do {                                                                 \
    if (!(x)) return std::printf("FAIL round %d: %s\n", round, #x), 1; \
  } while (0)

static long long seen_two[2][2];   // joins of two rounds: four or eight warps, the line or parts

static int batch(int round) {
  static const int kUnits[] = {1, 2, 3, 8, 16, 33, 200, 500}, kSeqs[] = {1, 2, 5, 36, 37, 64, 300}, kSms[] = {148, 148, 132, 20};
  const int D = pick(0, 1) ? 64 : 128, rows = pick(0, 1) ? 8 : 16, sms = kSms[pick(0, 3)];
  const bool fused = pick(0, 1);
  Args a;
  a.units = kUnits[pick(0, 7)];
  a.c.n_seqs = kSeqs[pick(0, 6)];
  a.c.page_size = pick(1, 300);
  a.c.table_width = pick(1, pick(0, 2) ? 300 : 3000);
  a.window = pick(0, 3) ? 0 : pick(1, 3000);
  const int most = a.c.page_size * a.c.table_width;
  std::vector<int32_t> lens(a.c.n_seqs);
  const int usual = pick(0, 2);   // lengths: all sorts, mostly short, all long
  for (int32_t& n : lens) n = usual == 0 ? pick(0, most) : usual == 1 ? pick(0, std::min(most, 40)) : most;
  if (usual == 1) lens[pick(0, a.c.n_seqs - 1)] = most;
  if (!pick(0, 3)) lens[pick(0, a.c.n_seqs - 1)] = most + pick(1, 5);
  if (!pick(0, 3)) lens[pick(0, a.c.n_seqs - 1)] = -pick(0, 5);
  a.c.lens = lens.data();
  const int warps = pkv::decode_warps(a.c.n_seqs, a.units, sms);
  a.ranks = pkv::decode_ranks(a.units, rows, fused, warps, sms);
  a.tile_shift = pkv::decode_tile_shift(D, warps, a.c.n_seqs, most);
  a.part_tiles = pkv::decode_part_tiles(warps);
  uint32_t parts = 0, places = 0;
  for (int n : lens) {
    const uint32_t tiles = pkv::tiles_of(a, pkv::held(a.c, n));
    parts += pkv::parts_of(a, tiles);
    places += tiles ? tiles + pkv::kSeqCost : 0;
  }
  struct Part {
    int tok0, tok1, rank, r0, parts;
  };
  std::map<int, std::vector<Part>> by_seq;
  std::set<long long> slots;
  std::map<long long, std::vector<std::tuple<int, int, int>>> counters;
  for (int r = 0; r < a.ranks; ++r) {
    pkv::Split l;
    pkv::split_range(a, r, parts, places, l);
    if (l.t >= l.end) continue;
    // as the kernel does: from some sequence in front of place t on
    int from = 0;
    uint32_t base = 0;
    for (const int start = pick(0, a.c.n_seqs - 1); from < start; ++from) {
      const uint32_t tiles = pkv::tiles_of(a, pkv::held(a.c, lens[from]));
      const uint32_t size = l.by_parts ? pkv::parts_of(a, tiles) : tiles ? tiles + pkv::kSeqCost : 0;
      if (base + size > l.t) break;
      base += size;
    }
    pkv::seek(a, l, from - 1, base);
    pkv::Piece p;
    while (pkv::next_piece(a, r, l, p)) {
      CHECK(p.seq >= 0 && p.seq < a.c.n_seqs && p.raw == lens[p.seq] && p.tok0 < p.tok1);
      by_seq[p.seq].push_back({p.tok0, p.tok1, r, p.r0, p.parts});
      CHECK(p.parts == 1 || a.ranks > 1);
      if (p.parts == 1) continue;
      const pkv::Join j = pkv::join_of(r - p.r0, p.parts);
      CHECK(j.of >= 1 && j.of <= pkv::kJoin && (!j.two || j.groups <= pkv::kJoin));
      seen_two[warps == 8][l.by_parts] += j.two;
      for (int u = 0; u < a.units; u += std::max(1, a.units - 1)) {
        const long long slot = pkv::part_slot(a, p.r0, r - p.r0, u), of_a_launch = 2LL * a.ranks * a.units;
        CHECK(slot >= 0 && slot < of_a_launch && slots.insert(slot).second);
        // the two rounds' counters are apart: the first below 2 a CTA, the second from there to 4
        const long long c1 = pkv::first_counter(a, p.r0, j, u), c2 = pkv::second_counter(a, p.r0, u);
        CHECK(c1 >= 0 && c1 < of_a_launch);
        counters[c1].push_back({p.seq * a.units + u, 1, j.of});
        if (j.two && r - p.r0 == j.g0) {
          CHECK(c2 >= of_a_launch && c2 < 2 * of_a_launch && c2 < 4LL * pkv::decode_most_ctas(sms));
          counters[c2].push_back({p.seq * a.units + u, 2, j.groups});
        }
        CHECK(c1 < 4LL * pkv::decode_most_ctas(sms));
      }
    }
  }
  for (auto& c : counters) {   // as many arrivals as are waited for, all of one sequence, unit and round
    CHECK((int)c.second.size() == std::get<2>(c.second[0]));
    for (auto& x : c.second) CHECK(x == c.second[0]);
  }
  for (int s = 0; s < a.c.n_seqs; ++s) {
    const int len = pkv::held(a.c, lens[s]);
    auto& p = by_seq[s];
    CHECK(p.empty() == (len == 0));
    if (p.empty()) continue;
    std::sort(p.begin(), p.end(), [](const Part& x, const Part& y) { return x.rank < y.rank; });
    CHECK(p[0].tok0 == pkv::first_seen(a, len) && p.back().tok1 == len);
    for (size_t i = 0; i < p.size(); ++i) {
      CHECK(p[i].rank == p[0].rank + (int)i && p[i].r0 == p[0].rank && p[i].parts == (int)p.size());
      CHECK(i == 0 || p[i].tok0 == p[i - 1].tok1);
    }
  }
  return 0;
}

static int search(int round) {
  std::vector<int32_t> cu{0};
  for (int n = pick(1, 3000); n > 0; --n) cu.push_back(cu.back() + (pick(0, 1) ? 0 : pick(0, 3)));
  const int n = (int)cu.size() - 1;
  for (int i = 0; i < 50; ++i) {
    const int t = pick(0, cu.back() + 3);
    int want = 0;
    while (want < n && cu[want + 1] <= t) ++want;
    CHECK(pkv::find_seq(cu.data(), n, t) == want);
  }
  for (int32_t& x : cu) x = pick(-5, 50);   // out of order: it ends, and within the sequences
  for (int i = 0; i < 20; ++i) {
    const int s = pkv::find_seq(cu.data(), n, pick(0, 50));
    CHECK(s >= 0 && s <= n);
  }
  return 0;
}

int main() {
  for (int round = 0; round < 4000; ++round)
    if (batch(round)) return 1;
  for (int round = 0; round < 200; ++round)
    if (search(round)) return 1;
  for (int w = 0; w < 2; ++w)
    for (int p = 0; p < 2; ++p)
      if (!seen_two[w][p]) return std::printf("FAIL no join of two rounds: %d warps, %s\n", w ? 8 : 4, p ? "parts" : "line"), 1;
  std::printf("ok %lld %lld %lld %lld\n", seen_two[0][0], seen_two[0][1], seen_two[1][0], seen_two[1][1]);
  return 0;
}
