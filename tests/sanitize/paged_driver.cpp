// Host-only sanitizer build of the C ABI of the paged cache (gdn_paged_api.hip): the
// launchers are replaced by stand-ins that read both ends of the workspace's regions,
// with the extent the kernels address, and the driver allocates the workspace with
// malloc at exactly the queried size.  The plan is the library's own
// (gdn_prefix_plan.hip).
#include <stdio.h>
#include <stdlib.h>

#include "../../include/gdn.h"
#include "../../linear_attention_recurrence_fwd_amd/csrc/gdn_paged.h"

namespace {
long g_launches = 0;
volatile unsigned char g_sink;
void touch(const void* p, size_t bytes) {
  if (!p || !bytes) return;
  const volatile unsigned char* c = static_cast<const volatile unsigned char*>(p);
  g_sink = c[0];
  g_sink = c[bytes - 1];
}
void* fake(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 48); }
}  // namespace

#define EXPECT(c)                                     \
  do {                                                \
    if (!(c)) {                                       \
      fprintf(stderr, "line %d: %s\n", __LINE__, #c); \
      exit(1);                                        \
    }                                                 \
  } while (0)

namespace gdn {
hipError_t launch_append(const AppendArgs& a, bool, hipStream_t) {
  EXPECT((int64_t{1} << a.pool.shift) > 0 && a.per >= 0);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_attn(const AttnArgs& a, bool bf, hipStream_t) {
  if (a.N == 0) return hipSuccess;
  // the splits cover all keys, and the tiles all rows
  const int64_t own = static_cast<int64_t>(a.max_q) * a.G, all = static_cast<int64_t>(a.N) * a.G;
  EXPECT(static_cast<int64_t>(a.o_tiles) * a.o_rows >= own && (a.o_rows <= 32 || bf));
  EXPECT(a.o_chunk > 0 && static_cast<int64_t>(a.o_split) * a.o_chunk >= a.max_len);
  if (a.together) {
    EXPECT(a.prefix == 0 && a.o_split == 1);
  } else {
    const size_t rows = static_cast<size_t>(a.p_split + a.o_split) * a.N * a.Hq;
    touch(a.part, rows * a.D * sizeof(float));
    touch(a.ml, rows * sizeof(float2));
    if (a.prefix > 0) {
      EXPECT(static_cast<int64_t>(a.p_tiles) * a.p_rows >= all && (a.p_rows <= 32 || bf));
      EXPECT(a.p_chunk > 0 && a.p_chunk % 32 == 0 && static_cast<int64_t>(a.p_split) * a.p_chunk >= a.prefix);
      EXPECT(static_cast<int64_t>(a.p_split - 1) * a.p_chunk < a.prefix);
    }
  }
  ++g_launches;
  return hipSuccess;
}
}  // namespace gdn

int main() {
  void *q = fake(0), *k = fake(1), *v = fake(2), *o = fake(3), *kp = fake(4), *vp = fake(5);
  float *w = static_cast<float*>(fake(9)), *rope = static_cast<float*>(fake(10)), *lse = static_cast<float*>(fake(11));
  int32_t *table = static_cast<int32_t*>(fake(14)), *lens = static_cast<int32_t*>(fake(15)), *cu = static_cast<int32_t*>(fake(16)),
          *pages = static_cast<int32_t*>(fake(17));
  long calls = 0;
  for (int dt : {GDN_F32, GDN_BF16})
    for (int64_t N : {0, 1, 7, 64, 500})
      for (int64_t S : {1, 7, 64})
        for (int64_t Hk : {1, 3})
          for (int64_t G : {1, 8, 17})
            for (int64_t D : {8, 72, 128, 256}) {
              const gdn_paged_dims d{N, S, Hk * G, Hk, D, 1000, 16, 500, Hk * 16 * D, 16 * D, D, dt};
              const gdn_turn t{9, D / 16 * 16, 0, 0, 0, 0, 3, 0, 1e-6f, 0.f};
              EXPECT(gdn_paged_append(&d, &t, q, k, v, w, w, rope, nullptr, nullptr, table, lens, cu, o, kp, vp, nullptr) == GDN_OK);
              for (int64_t prefix : {0, 1, 63, 2049, 70001})
                for (int64_t max_len : {0, 5, 300, 8000})
                  for (int64_t max_q : {int64_t{1}, N / 2, N}) {
                    if (max_q < 1 || max_q > N) continue;
                    size_t n = 0;
                    EXPECT(gdn_prefix_attention_workspace_bytes(&d, prefix, max_q, max_len, &n) == GDN_OK);
                    if (n > (size_t{2} << 30)) continue;
                    void* ws = n ? malloc(n) : nullptr;
                    EXPECT(gdn_prefix_attention(&d, q, kp, vp, table, lens, pages, prefix, cu, max_q, max_len, 1.f, o, lse, ws, n,
                                                nullptr) == GDN_OK);
                    if (n) EXPECT(gdn_prefix_attention(&d, q, kp, vp, table, lens, pages, prefix, cu, max_q, max_len, 1.f, o, lse, ws,
                                                       n - 1, nullptr) == GDN_ERR_WORKSPACE);
                    free(ws);
                    ++calls;
                  }
            }
  printf("ok: %ld calls, %ld launches\n", calls, g_launches);
  return 0;
}
