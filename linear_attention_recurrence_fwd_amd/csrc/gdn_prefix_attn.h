// What the attention kernels share: items, keys in pages, the join of parts.
#pragma once

#include "gdn_dev.h"
#include "gdn_paged.h"

namespace gdn {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The statistics' reference m is moved when a score exceeds it by this (base 2), so that
// moving it, which scales the result's registers, is rare.  The weights are held as
// 2^(score - m - lift): with lift = 17 + log2(all keys of a row) their sum stays under a
// half, and the sum of weighted values in fp32 for values up to its largest (relative to
// m alone, 1600 equal scores over values of 1e37 gave Inf).  At the other end products
// under 2^-126 lose bits: a factor of 2^17 earlier than with weights divided by their sum.
constexpr float kSlack = 16.f;
constexpr float kMost = 65536.f;  // and a lane's sixteen weights of a block by this together (times 2^-lift)

// 16 bytes of zeros and of NaN (in either type): what the loads of keys behind the
// end, and of keys on pages that do not exist, are pointed to.
__device__ const uint4 kFill[2] = {{0, 0, 0, 0}, {0x7fc07fc0, 0x7fc07fc0, 0x7fc07fc0, 0x7fc07fc0}};

// 16 bytes (4 bytes) of each lane to LDS at the wave's address + 16 (4) * lane, issued by
// inline assembly like the buffer loads in gdn_dev.h; a pool may be larger than a
// descriptor's 4 GiB.  Inactive lanes write nothing.  LDS addresses are plain numbers (of
// a pointer every cast is checked for null).
__device__ __forceinline__ uint32_t lds_of(const void* p) {
  typedef __attribute__((address_space(3))) const void lds_t;
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_t*)p));
}
__device__ __forceinline__ void load_lds16(const void* p, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
// From an address that is the same for the wave, and each lane's distance to it.  The
// address may just have come out of a vector register (readfirstlane): a vector memory
// instruction must not read such scalar registers within five wait states, which nobody
// but this block can see to.
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, uint32_t lds) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  base = reinterpret_cast<const void*>((static_cast<uint64_t>(hi) << 32) | lo);
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void load_lds4(const void* p, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}

// Where 16-byte piece p of row r of a tile lies: place p ^ swizzle(r) of the row.  LDS
// gives 256 bytes a cycle, 16 such pieces: to a wide read 16 lanes' (one piece of 16
// rows), to a transposing read 32 lanes' (AROUND = 4: four pieces of four rows, or 2: two
// of eight), to a read of single words 64 lanes' (AROUND = 0: four pieces of the rows r,
// r + 4, r + 8, r + 12).  The swizzle puts each of these on sixteen different places,
// modulo 16; rows of an odd number of 128 bytes have half of it from their parity.
// (By three bits for all, half of the LDS's cycles in use were conflicts.)
template <int PR, int AROUND> __device__ __forceinline__ int swizzle(int row) {
  if (AROUND == 0) return (((row >> 2) & 3) << 2) | (row & 3);
  if (AROUND == 4) return PR % 16 == 0 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  return PR % 16 == 0 ? ((row & 7) << 1) | ((row >> 3) & 1) : (((row >> 1) & 3) << 1) | ((row >> 3) & 1);
}

// What an item works on: rows from row0 on of the tokens t0 .. t0 + n - 1 (n G rows in
// all) and key head hk, keys k0 .. k1 - 1 in the pages of list; bad: the result is NaN.
struct Item {
  int t0, n, row0, hk, slot;
  const int32_t* list;
  int k0, k1;
  int seen;  // keys that the first token sees (may be negative); each further one sees one more
  bool bad, empty;
};

__device__ __forceinline__ Item item_of(const AttnArgs& a) {
  Item it{};
  int b = blockIdx.x;
  const int pairs = a.p_split * a.Hk, p_items = a.which & 1 ? pairs * a.p_tiles : 0;
  if (b < p_items) {
    const PairTile at = prefix_item(b, pairs, a.p_tiles);
    const int pair = at.pair, tile = at.tile;
    it.slot = pair / a.Hk;
    it.hk = pair % a.Hk;
    it.n = a.N;
    it.row0 = tile * a.p_rows;
    it.list = a.prefix_pages;
    it.k0 = it.slot * a.p_chunk;
    it.k1 = min(a.prefix, it.k0 + a.p_chunk);
    it.seen = 1 << 30;
    return it;
  }
  b -= p_items;
  // the splits of a sequence's keys outermost: those behind its end have nothing to do
  const int tile = b % a.o_tiles;
  b /= a.o_tiles;
  it.hk = b % a.Hk;
  b /= a.Hk;
  const int s = b % a.S, split = b / a.S;
  it.slot = a.p_split + split;
  it.row0 = tile * a.o_rows;
  const int end = a.cu ? min(a.cu[s + 1], a.N) : (s + 1) * a.per;
  it.t0 = a.cu ? max(a.cu[s], 0) : s * a.per;
  it.n = end - it.t0;
  const int len = a.lens[s];
  it.seen = len - it.n + 1;
  it.bad = len < 0 || len > a.max_len || it.n > a.max_q;
  const int last = min(it.n - 1, (it.row0 + a.o_rows - 1) / a.G);  // the tile's last token
  it.list = a.table + s * a.width;
  it.k0 = split * a.o_chunk;
  it.k1 = it.bad ? 0 : min(it.seen + last, it.k0 + a.o_chunk);
  it.empty = it.n <= 0 || (it.row0 >= it.n * a.G && !it.bad) || (!a.together && it.k1 <= it.k0);
  return it;
}

// Every lane finds the same: in scalar registers, what follows from it is worked out once
// for the wave.
__device__ __forceinline__ Item find_item(const AttnArgs& a) {
  Item it = item_of(a);
  for (int* x : {&it.t0, &it.n, &it.row0, &it.hk, &it.slot, &it.k0, &it.k1, &it.seen}) *x = __builtin_amdgcn_readfirstlane(*x);
  const uint64_t p = reinterpret_cast<uint64_t>(it.list);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32));
  it.list = reinterpret_cast<const int32_t*>(static_cast<uint64_t>(hi) << 32 | lo);
  it.bad = __builtin_amdgcn_readfirstlane(it.bad);
  it.empty = __builtin_amdgcn_readfirstlane(it.empty);
  return it;
}

// The last tile of a sequence with more tokens than max_q also has the rows that no
// tile covers.
template <typename T>
__device__ __forceinline__ void bad_rows(const AttnArgs& a, const Item& it, int nrows, int threads) {
  const int begin = it.row0 + a.o_rows;
  if (!it.bad || begin < a.max_q * a.G) return;
  for (int64_t i = threadIdx.x; i < static_cast<int64_t>(nrows - begin) * a.D; i += threads) {
    const int r = begin + static_cast<int>(i / a.D), c = static_cast<int>(i % a.D);
    const int64_t row = static_cast<int64_t>(it.t0 + r / a.G) * a.Hq + it.hk * a.G + r % a.G;
    static_cast<T*>(a.o)[row * a.D + c] = from_f32<T>(__builtin_nanf(""));
    if (a.lse && c == 0) a.lse[row] = __builtin_nanf("");
  }
}

hipError_t launch_many(const AttnArgs& a, unsigned items, hipStream_t st);  // items of 128 rows, bf16

}  // namespace attn
}  // namespace gdn
