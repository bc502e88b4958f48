// What the attention kernels share: items, keys in pages, the join of parts.
#pragma once

#include "gdn_dev.h"
#include "gdn_paged.h"

namespace gdn {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The statistics' reference maximum is moved when a score exceeds it by this (base 2):
// the weights stay below 2^8 and keep their relative precision, and moving it, which
// scales the result's registers, is rare.
constexpr float kSlack = 8.f;

// 16 bytes of zeros and of NaN (in either type): what the loads of keys behind the
// end, and of keys on pages that do not exist, are pointed to.
__device__ const uint4 kFill[2] = {{0, 0, 0, 0}, {0x7fc07fc0, 0x7fc07fc0, 0x7fc07fc0, 0x7fc07fc0}};

// 16 bytes (4 bytes) to LDS at the wave's base + 16 (4) * lane, issued by inline
// assembly like the buffer loads in gdn_dev.h; a pool may be larger than a
// descriptor's 4 GiB.  Inactive lanes write nothing.
__device__ __forceinline__ void load_lds16(const void* p, const void* lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(lds_addr(lds)) : "memory");
}
__device__ __forceinline__ void load_lds4(const void* p, const void* lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds_addr(lds)) : "memory");
}

// An item's keys: the prefix's p0 .. p1, then the sequence's own o0 .. o1, in tiles of
// KT (each part begins a tile).
template <int KT> struct Keys {
  const int32_t *plist, *olist;
  int p0, p1, o0, o1;
  int np, n;  // tiles of the prefix, of both
  __device__ __forceinline__ void count() {
    np = p1 > p0 ? (p1 - p0 + KT - 1) / KT : 0;
    n = np + (o1 > o0 ? (o1 - o0 + KT - 1) / KT : 0);
  }
  __device__ __forceinline__ bool own(int t) const { return t >= np; }
  __device__ __forceinline__ int first(int t) const { return t < np ? p0 + KT * t : o0 + KT * (t - np); }
  __device__ __forceinline__ int end(int t) const { return t < np ? p1 : o1; }
  __device__ __forceinline__ const int32_t* list(int t) const { return t < np ? plist : olist; }
};

// What an item works on: rows row0 .. row0 + rows of the tokens t0 .. t0 + n (n G rows
// in all) and key head hk; bad: the result is NaN.
struct Item {
  int t0, n, row0, hk, slot;
  int seen;  // own keys that the sequence's first token sees (may be negative)
  bool bad, empty;
};

// Items are numbered so that those which read the same keys of the prefix (row tiles
// of one split and key head) run on the same XCD, one after the other: workgroups go
// to the eight XCDs in turn.
__device__ __forceinline__ Item find_item(const AttnArgs& a, Keys<1>& ks) {
  Item it{};
  int b = blockIdx.x;
  const int pairs = a.p_split * a.Hk, p_items = (pairs + 7) / 8 * 8 * a.p_tiles;
  ks.plist = a.prefix_pages;
  ks.olist = nullptr;
  ks.p0 = ks.p1 = ks.o0 = ks.o1 = 0;
  if (!a.together && b < p_items) {
    const int pair = b / (8 * a.p_tiles) * 8 + b % 8, tile = b / 8 % a.p_tiles;
    if (pair >= pairs) {
      it.empty = true;
      return it;
    }
    it.slot = pair / a.Hk;
    it.hk = pair % a.Hk;
    it.n = a.N;
    it.row0 = tile * a.rows;
    ks.p0 = it.slot * a.p_chunk;
    ks.p1 = min(a.prefix, ks.p0 + a.p_chunk);
    return it;
  }
  if (!a.together) b -= p_items;
  // the splits of a sequence's keys outermost: those behind its end have nothing to do
  const int tile = b % a.o_tiles;
  b /= a.o_tiles;
  it.hk = b % a.Hk;
  b /= a.Hk;
  const int s = b % a.S, split = b / a.S;
  it.slot = a.p_split + split;
  it.row0 = tile * a.rows;
  const int end = a.cu ? min(a.cu[s + 1], a.N) : (s + 1) * a.per;
  it.t0 = a.cu ? max(a.cu[s], 0) : s * a.per;
  it.n = end - it.t0;
  const int len = a.lens[s];
  it.seen = len - it.n + 1;
  it.bad = len < 0 || len > a.max_len || it.n > a.max_q;
  const int last = min(it.n - 1, (it.row0 + a.rows - 1) / a.G);  // the tile's last token
  ks.olist = a.table + s * a.width;
  ks.o0 = split * a.o_chunk;
  ks.o1 = it.bad ? 0 : min(it.seen + last, ks.o0 + a.o_chunk);
  if (a.together && !it.bad) ks.p1 = a.prefix;
  it.empty = it.n <= 0 || (it.row0 >= it.n * a.G && !it.bad) || (!a.together && ks.o1 <= ks.o0);
  return it;
}

}  // namespace attn
}  // namespace gdn
