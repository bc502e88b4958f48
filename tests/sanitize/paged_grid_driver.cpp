// The entries of the rotation with several axes and of the paged cache with their real
// launch code, built for the host alone: the runtime's launch is replaced by one that
// looks at the grid.  A launch's threads are counted in 32 bits in each direction and a
// workgroup holds 1024 at most; every size that an entry accepts has to keep to that.
// Tensors and workspaces are places that nothing reads.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/gdn.h"

namespace {
long g_launches = 0, g_bad = 0;
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
  const uint64_t x = static_cast<uint64_t>(g.x) * b.x, y = static_cast<uint64_t>(g.y) * b.y, z = static_cast<uint64_t>(g.z) * b.z;
  const bool ok = x && y && z && x < (1ull << 32) && y <= 65535 && z <= 65535 && b.x * b.y * b.z <= 1024;
  if (!ok) {
    ++g_bad;
    fprintf(stderr, "grid %u x %u x %u of %u x %u x %u threads\n", g.x, g.y, g.z, b.x, b.y, b.z);
  }
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
}

int main() {
  long calls = 0, refused = 0;
  auto expect = [&](int rc, bool may_refuse, const char* what, int64_t a, int64_t b, int64_t c, int64_t d) {
    ++calls;
    if (rc == GDN_ERR_UNSUPPORTED && may_refuse) {
      ++refused;
      return;
    }
    if (rc != GDN_OK || g_bad) {
      fprintf(stderr, "status %d: %s %lld %lld %lld %lld\n", rc, what, static_cast<long long>(a), static_cast<long long>(b),
              static_cast<long long>(c), static_cast<long long>(d));
      exit(1);
    }
  };
  void *q = fake(0), *k = fake(1), *v = fake(2), *o = fake(3), *kp = fake(4), *vp = fake(5), *dq = fake(6), *dk = fake(7), *ws = fake(8);
  float *w = static_cast<float*>(fake(9)), *rope = static_cast<float*>(fake(10)), *lse = static_cast<float*>(fake(11)),
        *dw = static_cast<float*>(fake(12)), *dw2 = static_cast<float*>(fake(13));
  int32_t *table = static_cast<int32_t*>(fake(14)), *lens = static_cast<int32_t*>(fake(15)), *cu = static_cast<int32_t*>(fake(16)),
          *pages = static_cast<int32_t*>(fake(17));
  const size_t room = size_t{1} << 55;
  for (int dt : {GDN_F32, GDN_BF16}) {
    const int64_t tokens[][2] = {{1, 1}, {3, 7000}, {1, 1 << 24}, {1 << 24, 1}, {1, (1 << 26) + 1}, {1, (1 << 30) - 1}};
    for (auto& t : tokens)
      for (int64_t D : {8, 24, 64, 200, 512})
        for (int64_t H : {1, 64})
          for (int inter : {0, 1}) {
            const gdn_norm_dims d{t[0], t[1], H, 1, D, D / 16 * 16, 9, 0, 0, dt, inter, 1e-6f, 0.f};
            size_t n = 0;
            expect(gdn_norm_rope_bwd_workspace_bytes(&d, &n), false, "axes workspace", t[0], t[1], H, D);
            for (float* weight : {w, static_cast<float*>(nullptr)}) {
              expect(gdn_norm_rope_axes_fwd(&d, 3, q, k, weight, weight, rope, nullptr, nullptr, dq, dk, nullptr), false, "axes",
                     t[0], t[1], H, D);
              expect(gdn_norm_rope_axes_bwd(&d, 3, q, k, weight, weight, rope, nullptr, nullptr, v, o, dq, dk, dw, dw2, ws, n,
                                            nullptr), false, "axes bwd", t[0], t[1], H, D);
            }
          }
    // tokens by sequences of a cache
    const int64_t batch[][2] = {{1, 1}, {64, 64}, {4096, 3}, {1 << 20, 1 << 20}, {1 << 26, 1}, {(1 << 30) - 1, 7}, {100000, 40000}};
    for (auto& b : batch)
      for (int64_t D : {8, 64, 72, 128, 192, 256})
        for (int64_t Hk : {1, 8})
          for (int64_t G : {1, 16, 200}) {
            gdn_paged_dims d{b[0], b[1], Hk * G, Hk, D, 1 << 20, 64, 4096, Hk * 64 * D, 64 * D, D, dt};
            const gdn_turn t{9, D / 16 * 16, 0, 0, 0, 0, 3, 0, 1e-6f, 0.f};
            const bool wide = Hk * G * D > (1 << 30);
            if (!wide)
              expect(gdn_paged_append(&d, &t, q, k, v, w, w, rope, nullptr, nullptr, table, lens, cu, o, kp, vp, nullptr), false,
                     "append", b[0], b[1], G, D);
            for (int64_t prefix : {int64_t{0}, int64_t{1}, int64_t{100}, int64_t{5000}, int64_t{1} << 30})
              for (int64_t max_len : {0, 1, 300, 1 << 18})
                for (int64_t max_q : {int64_t{1}, int64_t{100}, b[0]}) {
                  if (max_q > b[0]) continue;
                  size_t n = 0;
                  const int rc = gdn_prefix_attention_workspace_bytes(&d, prefix, max_q, max_len, &n);
                  expect(rc, true, "attention workspace", b[0], b[1], max_q, max_len);
                  expect(gdn_prefix_attention(&d, q, kp, vp, table, lens, pages, prefix, cu, max_q, max_len, 1.f, o, lse, ws, room,
                                              nullptr), rc == GDN_ERR_UNSUPPORTED, "attention", b[0], b[1], prefix, max_len * 1000 + max_q);
                }
          }
  }
  printf("ok: %ld calls, %ld refused, %ld launches\n", calls, refused, g_launches);
  return g_launches < 20000;  // (sizes that are refused say nothing)
}
