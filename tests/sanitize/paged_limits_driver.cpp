// The paged cache's attention at its limits, with its real launch code built for the host
// alone: sizes just inside have to be accepted and to make launches that the device can
// hold (fewer than 2^32 threads), those just outside have to be refused before anything is
// launched, by the size query and by the call alike.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "../../include/gdn.h"
#include "../../linear_attention_recurrence_fwd_amd/csrc/gdn_paged.h"

namespace {
long g_launches = 0, g_empty = 0;
uint64_t g_most = 0;
dim3 g_grid, g_block;
size_t g_shared;
hipStream_t g_stream;
void* fake(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 56); }
}  // namespace

extern "C" {
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t st) {
  g_grid = grid;
  g_block = block;
  g_shared = shared;
  g_stream = st;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* st) {
  *grid = g_grid;
  *block = g_block;
  *shared = g_shared;
  *st = g_stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 g, dim3 b, void**, size_t, hipStream_t) {
  ++g_launches;
  const uint64_t x = static_cast<uint64_t>(g.x) * b.x;
  if (x > g_most) g_most = x;
  if (!x || g.y != 1 || g.z != 1) ++g_empty;
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
}

namespace {
struct Case {
  const char* what;
  int dtype;
  int64_t N, S, Hq, Hk, D, prefix, max_q, max_len;
  bool taken;
};
}  // namespace

int main() {
  constexpr int64_t kRows = (int64_t{1} << 26) - 64;
  const Case cases[] = {
      // rows of one key head, with a prefix and own keys in one launch (fp32: tiles of 16 or 32 rows)
      {"all rows, one head", GDN_F32, kRows, 1, 1, 1, 8, 16, 1, 300, true},
      {"all rows, one head, long", GDN_F32, kRows, 1, 1, 1, 8, 5000, kRows, 1 << 18, true},
      {"all rows, eight heads", GDN_F32, kRows / 8, 1, 8, 8, 64, 100, kRows / 8, 300, true},
      {"all rows, sixteen to one", GDN_F32, kRows / 16, 4, 16, 1, 256, 16, kRows / 16, 300, true},
      {"all rows, one head, bf16", GDN_BF16, kRows, 1, 1, 1, 8, 16, kRows, 300, true},
      {"all rows, eight heads, bf16", GDN_BF16, kRows / 8, 1, 8, 8, 64, 1 << 30, kRows / 8, 300, true},
      {"one row more", GDN_F32, kRows + 1, 1, 1, 1, 8, 16, 1, 300, false},
      {"one row more, bf16", GDN_BF16, kRows + 1, 1, 1, 1, 8, 16, 1, 300, false},
      // single tokens of many sequences: an own item each, and the prefix's besides
      {"sequences", GDN_F32, (1 << 24) - 1, (1 << 24) - 1, 1, 1, 8, 0, 1, 16, true},
      {"one sequence more", GDN_F32, 1 << 24, 1 << 24, 1, 1, 8, 0, 1, 16, false},
      {"sequences with a prefix", GDN_F32, 15000000, 15000000, 1, 1, 8, 16, 1, 16, true},
      {"sequences with a prefix, too many", GDN_F32, (1 << 24) - 1, (1 << 24) - 1, 1, 1, 8, 16, 1, 16, false},
      {"sequences with a prefix, bf16 (two launches)", GDN_BF16, (1 << 24) - 1, (1 << 24) - 1, 1, 1, 8, 16, 1, 16, true},
      {"sequences by heads", GDN_BF16, (1 << 21) - 1, (1 << 21) - 1, 8, 8, 64, 100, 1, 300, true},
      {"sequences by heads, too many", GDN_BF16, 1 << 21, 1 << 21, 8, 8, 64, 100, 1, 300, false},
      // a ragged batch whose longest sequence is not known: as long as the batch
      {"ragged", GDN_BF16, 16384, 512, 32, 8, 128, 0, 16384, 4096, true},
      {"ragged with a prefix", GDN_BF16, 16384, 512, 32, 8, 128, 8192, 16384, 4096, true},
      {"ragged, fp32", GDN_F32, 16384, 512, 32, 8, 128, 8192, 16384, 4096, true},
      {"ragged, too many", GDN_BF16, 1 << 16, 1 << 12, 32, 8, 128, 0, 1 << 16, 4096, false},
      {"all bounds at once", GDN_F32, kRows, (1 << 30) - 1, 1, 1, 8, 1 << 30, kRows, 1 << 18, false},
  };
  void *q = fake(0), *o = fake(3), *kp = fake(4), *vp = fake(5), *ws = fake(8);
  float* lse = static_cast<float*>(fake(11));
  int32_t *table = static_cast<int32_t*>(fake(14)), *lens = static_cast<int32_t*>(fake(15)), *cu = static_cast<int32_t*>(fake(16)),
          *pages = static_cast<int32_t*>(fake(17));
  int bad = 0;
  for (const Case& c : cases) {
    const gdn_paged_dims d{c.N, c.S, c.Hq, c.Hk, c.D, 1 << 20, 64, 4096, c.Hk * 64 * c.D, 64 * c.D, c.D, c.dtype};
    const long before = g_launches;
    g_most = 0;
    size_t n = 0;
    const int query = gdn_prefix_attention_workspace_bytes(&d, c.prefix, c.max_q, c.max_len, &n);
    const int call = gdn_prefix_attention(&d, q, kp, vp, table, lens, pages, c.prefix, cu, c.max_q, c.max_len, 1.f, o, lse, ws,
                                          size_t{1} << 55, nullptr);
    const int want = c.taken ? GDN_OK : GDN_ERR_UNSUPPORTED;
    const bool launched = g_launches > before;
    if (query != want || call != want || launched != c.taken || g_most >= (uint64_t{1} << 32) || g_empty) {
      fprintf(stderr, "%s: query %d, call %d, %ld launches, %llu threads at most\n", c.what, query, call, g_launches - before,
              static_cast<unsigned long long>(g_most));
      ++bad;
    }
  }
  // every item of the prefix has a part of the work of its own, whatever their numbers
  for (int pairs : {1, 2, 3, 7, 8, 9, 15, 16, 23, 24, 129})
    for (int tiles : {1, 2, 5, 78, 1000}) {
      std::vector<char> seen(static_cast<size_t>(pairs) * tiles);
      for (int b = 0; b < pairs * tiles; ++b) {
        const gdn::PairTile at = gdn::prefix_item(b, pairs, tiles);
        if (at.pair < 0 || at.pair >= pairs || at.tile < 0 || at.tile >= tiles || seen[at.pair * tiles + at.tile]++) {
          fprintf(stderr, "item %d of %d pairs by %d tiles: pair %d, tile %d\n", b, pairs, tiles, at.pair, at.tile);
          return 1;
        }
      }
    }
  if (!bad) printf("ok: %zu cases, %ld launches\n", sizeof cases / sizeof *cases, g_launches);
  return bad != 0;
}
