// Host-side interfaces of the paged cache's operators (appending with norm and
// rotation; attention over a shared prefix and own pages): between their entry
// points (gdn_paged_api.hip) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Pool of pages; strides in bytes.
struct PagePool {
  int64_t ps, hs, ts;
  int pages, shift;         // tokens of a page: 1 << shift
};

struct AppendArgs {
  int64_t BT;               // tokens (rows of pos)
  int S, per;               // sequences; tokens of each where cu is null
  int Hq, Hk, D, R, P, A;
  int64_t qs, ks, vs;       // elements from one token's rows to the next one's
  int interleaved;
  float eps, w_offset;
  const void *q, *k, *v;
  const float *wq, *wk;     // may be null: no norm
  const float* rope;
  const uint8_t* axis;
  const int32_t* pos;
  int64_t first;
  const int32_t *table, *past, *cu;
  int64_t width;
  PagePool pool;
  void *oq, *kp, *vp;
};

// Rows of the tokens N by the G query heads of a key head: row r is token r / G (of
// the call, or of its sequence), head r % G.
struct AttnArgs {
  int N, S, per;            // tokens, sequences, tokens of each where cu is null
  int Hq, Hk, G, D;
  const void* q;
  const void *kp, *vp;
  PagePool pool;
  const int32_t *table, *lens, *prefix_pages, *cu;
  int64_t width;
  int prefix, max_q, max_len;
  float scale;
  void* o;
  float* lse;               // may be null
  // The plan.  together (no prefix, and own keys that are not split): an item writes the
  // result.  Otherwise items of the prefix (rows of all sequences) and of own keys leave
  // their parts in part / ml, [slot][N * Hq], the prefix's in the first p_split slots,
  // joined by another kernel.
  int together;
  int which;                // items of this launch: 1 the prefix's, 2 those of own keys (3 both)
  int p_rows, o_rows;       // rows of an item
  int p_tiles, p_split, p_chunk;  // items of the prefix: row tiles, splits, keys of a split
  int o_tiles, o_split, o_chunk;  // of own keys, the tiles of each sequence
  float* part;              // [slots][N * Hq][D], not divided by the sums
  float2* ml;               // [slots][N * Hq] reference m (base 2) and sum
  // The weights are held as 2^(score - m - lift), so that all of a row's together stay
  // under 1 and no sum of weighted values leaves fp32 while the values are in it.
  float lift, unit, whole;  // unit: 2^-lift, whole: 2^lift
};

// Items of the prefix and of own keys: workgroups of a launch.  (At most 2^26 rows by
// sequences: their products fit 64 bits.)
inline int64_t prefix_items(const AttnArgs& a) { return static_cast<int64_t>(a.p_split) * a.Hk * a.p_tiles; }
inline int64_t own_items(const AttnArgs& a) { return static_cast<int64_t>(a.o_tiles) * a.Hk * a.S * a.o_split; }

// Which pair of a split and a key head, and which tile of rows, an item of the prefix has.
// Items that read the same keys (the row tiles of a pair) run on the same XCD, one after
// the other: workgroups go to the eight XCDs in turn.  The pairs behind the last whole
// eight take turns over all of the XCDs, and no workgroup is empty (filled up to eight by
// empty ones, one pair's tiles all ran on one XCD: 8192 tokens over 2048 shared keys, 16
// heads of 128 on one key head, 1057 us instead of 246, on two 626 instead of 277).
struct PairTile {
  int pair, tile;
};
__host__ __device__ inline PairTile prefix_item(int b, int pairs, int tiles) {
  const int first = b / (8 * tiles) * 8, beside = pairs - first < 8 ? pairs - first : 8, at = b - first * tiles;
  return {first + at % beside, at / beside};
}

hipError_t launch_append(const AppendArgs& a, bool bf16, hipStream_t st);
// Fills the plan; the bytes of part and of ml.
void attn_plan(AttnArgs* a, bool bf16, size_t* part, size_t* ml);
hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t st);

}  // namespace gdn
