// How the attention over a prefix and own pages is cut into items: host code alone.
#include "gdn_paged.h"

namespace gdn {
namespace {

// What a launch's items cost, in us: each its keys and what it takes to begin and end,
// `slots` of them at once; and the parts that are written and read back.  512 slots, two
// workgroups to a compute unit, are taken for all kernels; by their LDS and registers the
// compute units hold 256 of the one for few rows of fp32 beyond 128 channels, 768 of that
// of bf16 of 129 to 192, 1024 of the one for many rows up to 64.  An item has at least 128
// keys, or `least` where that leaves half of the slots free.  Of few rows of more than 256
// bytes, which two waves go through, 64: one token of 8 sequences over 1000 keys of 256
// channels, bf16, 12.7 us against 14.1, of 192 11.3 and 12.6, of 136 11.3 and 13.2, of 72
// and 96, fp32, 12.8 and 16.9; with the slots full, one token of 32 over 2000 keys of 8
// heads of 192, 25.8 against 20.6.  Of smaller rows (four waves) 128: one token of 4
// sequences over 4000 keys of 128 channels 13.3 us, with 64 keys 19.3.
struct Cost {
  double key, item;
  int slots, least;
};
Cost cost_of(int rows, int D, bool bf) {
  if (rows > 32) return {4.0 * rows * D / 1.6e6, 14.0, 512, 128};
  const int row = D * (bf ? 2 : 4);  // bytes
  return {2.0 * row / 9.0e3 * (bf ? 1.0 : 1.5) * (rows == 16 ? 1.0 : 1.3), 6.0, 512, row <= 256 ? 128 : 64};
}
struct Split {
  int chunk, n;  // keys of a split, splits
  double us;
};
// Of the numbers of splits of len keys that fill one to eight rounds of the slots, and
// one, the cheapest.
Split split(int64_t items, int64_t len, const Cost& c, double part_us) {
  Split best{1, 0, 0.0};
  const int64_t least = items * ((len + c.least - 1) / c.least) <= c.slots / 2 ? c.least : 128;
  for (int round = 0; round <= 8 && len > 0; ++round) {
    const int64_t n = round == 0 ? 1 : round * c.slots / items;
    if (n < 1) continue;
    const int64_t even = ((len + n - 1) / n + 63) / 64 * 64, k = n > 1 && even < least ? least : even;
    const int64_t count = (len + k - 1) / k, rounds = (items * count + c.slots - 1) / c.slots;
    const double us = rounds * (k * c.key + c.item) + count * part_us;
    if (round == 0 || us < best.us) best = Split{static_cast<int>(k), static_cast<int>(count), us};
  }
  return best;
}

}  // namespace

// Rows of an item.  The kernel for many rows from 65 on: 64 sequences' 512 rows and
// 32768 keys of 2 heads of 256 take 52 us with it, 167 us without.  Few rows, 16 or 32
// (the prefix's and own keys' in one launch): what the cost says.
void attn_plan(AttnArgs* a, bool bf, size_t* part, size_t* ml) {
  // (weights above the reference's: under 2^16 (gdn_prefix_attn.h), for each key)
  int lift = 17;
  while ((int64_t{1} << (lift - 17)) < static_cast<int64_t>(a->prefix) + a->max_len) ++lift;
  a->lift = static_cast<float>(lift);
  a->whole = static_cast<float>(int64_t{1} << lift);
  a->unit = 1.f / a->whole;
  const int64_t own = static_cast<int64_t>(a->max_q) * a->G, all = static_cast<int64_t>(a->N) * a->G;
  const double part_us = static_cast<double>(a->N) * a->Hq * a->D * 8 / 4.0e6;  // written and read, at 4 TB/s
  auto many = [&](int64_t n) { return bf && n > 64; };
  Split o{}, p{};
  auto choose = [&](int o_rows, int p_rows) {
    a->o_rows = o_rows;
    a->p_rows = p_rows;
    a->o_tiles = static_cast<int>((own + o_rows - 1) / o_rows);
    a->p_tiles = a->prefix > 0 ? static_cast<int>((all + p_rows - 1) / p_rows) : 0;
    o = split(static_cast<int64_t>(a->o_tiles) * a->Hk * a->S, a->max_len, cost_of(o_rows, a->D, bf), part_us);
    p = split(static_cast<int64_t>(a->p_tiles) * a->Hk, a->prefix, cost_of(p_rows, a->D, bf), part_us);
    return o.us + p.us;
  };
  const bool few_p = a->prefix > 0 && !many(all);
  if (many(own)) {
    choose(128, 128);
  } else {
    const double c16 = choose(16, few_p ? 16 : 128), c32 = choose(32, few_p ? 32 : 128);
    if (c16 <= c32) choose(16, few_p ? 16 : 128);
  }
  a->o_chunk = o.chunk;
  a->o_split = o.n;
  a->p_chunk = p.chunk;
  a->p_split = p.n;
  a->together = a->prefix == 0 && o.n <= 1;
  *part = *ml = 0;
  if (a->together) {
    a->o_chunk = a->max_len > 0 ? a->max_len : 1;
    a->o_split = 1;
    return;
  }
  const size_t rows = static_cast<size_t>(a->p_split + a->o_split) * a->N * a->Hq;
  *part = rows * a->D * sizeof(float);
  *ml = rows * sizeof(float2);
}

}  // namespace gdn
