// How the prompt-side attention kernel cuts its work over the CTAs: plain
// arithmetic, which every CTA does for itself and a test does on the host.
#pragma once

#include <type_traits>

#include "pkv_prefill.h"

#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

template <typename I>
PKV_HD I line_min(I a, I b) { return a < b ? a : b; }
template <typename I>
PKV_HD I line_max(I a, I b) { return a > b ? a : b; }

// The work of one key head of a sequence, as a line: its items, of `per` tokens
// each (two row tiles of `half`, or one), one after the other, as long as they
// take.  I: the integers of lengths.
template <typename I>
struct PrefillLine {
  int n, L, per, half, tiles, causal, item, item1;
  PKV_HD PrefillLine(int n_, int L_, int per_, int half_, int causal_)
      : n(n_), L(L_), per(per_), half(half_), tiles((n_ + per_ - 1) / per_), causal(causal_),
        item(kPrefillItemCost + (causal_ ? per_ * kPrefillTokenCost : 0)),
        item1(kPrefillItemCost1 + (causal_ ? half_ * kPrefillTokenCost : 0)) {}
  // (products that wrap in 32 bits where their sum does not)
  static PKV_HD I mul(I a, I b) {
    using U = std::make_unsigned_t<I>;
    return static_cast<I>(static_cast<U>(a) * static_cast<U>(b));
  }
  // keys that item t sees
  PKV_HD int keys(int t) const {
    if (!causal) return L;
    const long long last = static_cast<long long>(t + 1) * per;
    return line_max(0, L - n + static_cast<int>(line_min(last, static_cast<long long>(n))));
  }
  PKV_HD bool one(int t) const {          // one row tile of two
    return half < per && n - static_cast<long long>(t) * per <= half;
  }
  PKV_HD I cost(int t) const {
    const I k = keys(t);
    return one(t) ? k * kPrefillKeyCost1 + item1 : k * kPrefillKeyCost + item;
  }
  // where item t begins (all before the last are whole)
  PKV_HD I begin(int t) const {
    I sum;                                          // of the keys before
    if (!causal) {
      sum = mul(t, L);
    } else {
      const int d = L - n, blind = d < 0 ? -d / per : 0;      // items that see none
      const I i = t, b = blind;
      sum = t <= blind ? 0 : static_cast<I>(static_cast<std::make_unsigned_t<I>>(mul(i - b, d)) + mul(per, (i * (i + 1) - b * (b + 1)) / 2));
    }
    return t * static_cast<I>(item) + sum * kPrefillKeyCost;
  }
  PKV_HD I length() const { return tiles > 0 ? begin(tiles - 1) + cost(tiles - 1) : 0; }
};

// Key tile, of BN keys, of an item at which the line is cut `x` into it: what
// comes before costs x, the item's own cost included (which the part behind pays
// once more, as that of every CTA that starts amid an item); its end belongs to it.
// No item's first or last part is shorter than `least` tiles (those between are a
// CTA's share, which may be less).
template <int BN, typename I>
PKV_HD int prefill_cut(I x, I cost, bool one, int item, int tiles, int least) {
  if (x >= cost) return tiles;
  const int key = BN * (one ? kPrefillKeyCost1 : kPrefillKeyCost);
  const I most = static_cast<I>(tiles) * key;
  const uint32_t keys = static_cast<uint32_t>(line_min(line_max(x - item + key / 2, static_cast<I>(0)), most));   // below 2^32: 3 a key, 2^24 keys
  const int p = static_cast<int>(one ? keys / (BN * kPrefillKeyCost1) : keys / (BN * kPrefillKeyCost));
  if (tiles < 2 * least) return 2 * p <= tiles ? 0 : tiles;
  if (p < least) return 2 * p <= least ? 0 : least;
  if (tiles - p < least) return 2 * (tiles - p) <= least ? tiles : tiles - least;
  return p;
}

// The line of all sequences and key heads in equal lengths, one a CTA.
template <typename I>
struct PrefillShares {
  I share, extra;
  PKV_HD PrefillShares(I total, int ctas) : share(total / ctas), extra(total - share * ctas) {}
  PKV_HD I begin(int cta) const { return share * cta + line_min(static_cast<I>(cta), extra); }
};

}  // namespace pkv
