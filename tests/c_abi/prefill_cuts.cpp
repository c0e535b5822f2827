// How prompt-side attention cuts its work over the CTAs, on the host: the kernel's
// own arithmetic (csrc/pkv_prefill_line.h) over random batches.  Every CTA walks its
// part of the line as the kernel's scheduler does; then
//   * every item's key tiles are some CTA's, once, and an item without keys is one CTA's;
//   * a CTA goes on with one item at most and leaves one unfinished at most;
//   * an item's first and last pieces are no shorter than asked for;
//   * the reduce's walk over the CTAs finds an item's pieces, all and in order;
//   * 32 and 64 bits agree where the host lets the scheduler count in 32.
// Prints the number of batches, cut items and pieces, or what is wrong.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "pkv_prefill_line.h"

using namespace pkv;

namespace {

unsigned long long state = 1;
unsigned draw(unsigned n) {                          // 0 .. n - 1
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return static_cast<unsigned>((state >> 33) % n);
}

struct Piece {
  int cta, from, to;
};
struct Item {
  int seq, kvh, tile, tiles;
  std::vector<Piece> pieces;
};
struct Batch {
  std::vector<int> n, L;
  int hkv, group, causal, ctas, least;
};

#define CHECK(x)                                                  \
  do {                                                            \
    if (!(x)) {                                                   \
      std::printf("line %d: %s\n", __LINE__, #x);                 \
      std::exit(1);                                               \
    }                                                             \
  } while (0)

template <int D, typename I>
std::vector<Item> walk(const Batch& b, long long* cut_items, long long* pieces) {
  constexpr int BN = prefill_key_tile(D);
  const int half = 128 / b.group, per = half * prefill_row_tiles(D);
  struct At {
    Item item;
    I at, cost;
    bool one;
    int price;
  };
  std::vector<At> line;
  I total = 0;
  for (size_t s = 0; s < b.n.size(); ++s) {
    const PrefillLine<I> l(b.n[s], b.L[s], per, half, b.causal);
    const I length = l.length();
    for (int h = 0; h < b.hkv; ++h) {
      for (int t = 0; t < l.tiles; ++t) {
        const int keys = l.keys(t);
        // the kernel steps from item to item by its cost, and begins by `begin`
        CHECK(t == 0 || l.begin(t) == l.begin(t - 1) + l.cost(t - 1));
        line.push_back({{static_cast<int>(s), h, t, (keys + BN - 1) / BN, {}},
                        total + l.begin(t), l.cost(t), l.one(t), l.one(t) ? l.item1 : l.item});
      }
      total += length;
    }
  }
  const PrefillShares<I> shares(total, b.ctas);
  CHECK(shares.begin(0) == 0 && shares.begin(b.ctas) == total);
  std::vector<PrefillCut> cuts(b.ctas, PrefillCut{});
  size_t first = 0;
  for (int c = 0; c < b.ctas; ++c) {
    const I x0 = shares.begin(c), x1 = shares.begin(c + 1);
    CHECK(x0 <= x1);
    while (first < line.size() && line[first].at + line[first].cost <= x0) ++first;
    int continued = 0, begun = 0;
    for (size_t i = first; x1 > x0 && i < line.size() && line[i].at < x1; ++i) {
      At& it = line[i];
      auto cut_in = [&](I x) {
        return prefill_cut<BN>(x - it.at, it.cost, it.one, it.price, it.item.tiles, b.least);
      };
      const int from = cut_in(x0), to = cut_in(x1), tiles = it.item.tiles;
      if (!(from < to || (tiles == 0 && it.at >= x0))) continue;
      if (tiles == 0) CHECK(from == 0 && to == 0);
      it.item.pieces.push_back({c, from, to});
      continued += from > 0;
      begun += from == 0 && to < tiles;
      if (from > 0) {
        int back = c - 1;
        while (back >= 0 && cut_in(shares.begin(back)) == from) --back;
        CHECK(back >= 0);
        cuts[c] = PrefillCut{cut_in(shares.begin(back)) == 0 ? 2 : 1, back, to == tiles, it.item.kvh, it.item.tile, 0};
      }
    }
    CHECK(continued <= 1 && begun <= 1);
  }
  std::vector<Item> items;
  for (const At& a : line) {
    const Item& it = a.item;
    items.push_back(it);
    if (it.tiles == 0) {
      CHECK(it.pieces.size() == 1);
      continue;
    }
    int upto = 0;
    for (const Piece& p : it.pieces) {
      CHECK(p.from == upto && p.to > p.from);
      if (it.pieces.size() > 1 && (p.from == 0 || p.to == it.tiles)) CHECK(p.to - p.from >= b.least);
      upto = p.to;
    }
    CHECK(upto == it.tiles);
    *pieces += it.pieces.size();
    if (it.pieces.size() == 1) continue;
    *cut_items += 1;
    // the reduce: from the CTA that has the second piece up to the one that has the last
    const int c0 = it.pieces[1].cta;
    CHECK(cuts[c0].kind == 2 && cuts[c0].first == it.pieces[0].cta);
    size_t found = 1;
    for (int c = c0;; ++c) {
      CHECK(c < b.ctas);
      if (cuts[c].kind == 0) continue;
      CHECK(found < it.pieces.size() && it.pieces[found].cta == c);
      CHECK(cuts[c].kind == (found == 1 ? 2 : 1));
      ++found;
      if (cuts[c].ends) break;
    }
    CHECK(found == it.pieces.size());
  }
  return items;
}

template <int D>
void run(int batches) {
  long long cut_items = 0, pieces = 0, both = 0;
  for (int i = 0; i < batches; ++i) {
    Batch b;
    const int kind = draw(5), seqs = kind == 0 ? 1 : 1 + draw(kind == 1 ? 200 : 6);
    const unsigned top = kind == 1 ? 40 : (kind == 2 ? 3000 : 400), far = kind == 3 ? 1 << draw(18) : 1 + draw(4000);
    for (int s = 0; s < seqs; ++s) {
      const int n = draw(4) == 0 ? draw(3) : draw(top);
      b.n.push_back(n);
      // (at times fewer keys than rows)
      b.L.push_back(draw(8) == 0 ? static_cast<int>(draw(n + 1)) : n + static_cast<int>(draw(far)));
    }
    b.hkv = 1 + draw(9);
    b.group = 1 + draw(32);
    b.causal = draw(3) != 0;
    b.ctas = 1 + draw(draw(2) ? 152 : 12);
    const int BN = prefill_key_tile(D);
    b.least = draw(4) == 0 ? 0x3fffffff : 1 + draw(2 * kPrefillMinPart / BN);
    const std::vector<Item> wide = walk<D, long long>(b, &cut_items, &pieces);
    // as the host decides it
    const int per = 128 / b.group * prefill_row_tiles(D);
    long long T = 0, most = 0;
    for (int s = 0; s < seqs; ++s) {
      T += b.n[s];
      most = b.L[s] > most ? b.L[s] : most;
    }
    const double items = static_cast<double>((T / per + seqs) * b.hkv);
    const double longest = static_cast<double>(most) * kPrefillKeyCost + kPrefillItemCost + static_cast<double>(per) * kPrefillTokenCost;
    if (T / per < kPrefillSmallItems && items * longest < 2147483648.0) {
      long long x = 0, y = 0;
      const std::vector<Item> narrow = walk<D, int>(b, &x, &y);
      CHECK(narrow.size() == wide.size());
      for (size_t j = 0; j < wide.size(); ++j) {
        CHECK(narrow[j].pieces.size() == wide[j].pieces.size());
        for (size_t k = 0; k < wide[j].pieces.size(); ++k)
          CHECK(narrow[j].pieces[k].cta == wide[j].pieces[k].cta && narrow[j].pieces[k].from == wide[j].pieces[k].from &&
                narrow[j].pieces[k].to == wide[j].pieces[k].to);
      }
      ++both;
    }
  }
  CHECK(cut_items > batches / 4 && both > batches / 4);
  std::printf("head_dim %d: %d batches, %lld cut items, %lld pieces, %lld counted in 32 bits as well\n", D, batches,
              cut_items, pieces, both);
}

}  // namespace

int main() {
  run<64>(3000);
  run<128>(3000);
  run<256>(3000);
  // the longest sequences, alone: 64 bits
  for (int causal = 0; causal < 2; ++causal) {
    Batch b{{3000, 1}, {kPrefillMostKeys, kPrefillMostKeys}, 3, 4, causal, 152, 4};
    long long x = 0, y = 0;
    walk<128, long long>(b, &x, &y);
    walk<256, long long>(b, &x, &y);
  }
  std::printf("ok\n");
  return 0;
}
