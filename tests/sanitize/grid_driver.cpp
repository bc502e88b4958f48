// The decay operator's and the query/key norm's entries with their real launch
// code, built for the host alone: the runtime's launch is replaced by one that
// looks at the grid.  A launch's threads are counted in 32 bits in each direction
// and a workgroup holds 1024 at most; every size that an entry accepts has to keep
// to that.  Tensors and workspaces are places that nothing reads.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/gdn.h"

namespace {
long g_launches = 0, g_bad = 0;
dim3 g_grid, g_block;
size_t g_shared;
hipStream_t g_stream;
void* fake(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 48); }
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
  long calls = 0;
  auto expect = [&](int rc, int want, const char* what, int64_t a, int64_t b, int64_t c, int64_t d) {
    ++calls;
    if (rc != want) fprintf(stderr, "status %d\n", rc);
    if (rc != want || g_bad) {
      fprintf(stderr, "%s %lld %lld %lld %lld\n", what, static_cast<long long>(a), static_cast<long long>(b),
              static_cast<long long>(c), static_cast<long long>(d));
      exit(1);
    }
  };
  void *q = fake(0), *k = fake(1), *v = fake(2), *o = fake(3), *dO = fake(4), *dq = fake(5), *dk = fake(6), *dv = fake(7);
  float *lg = static_cast<float*>(fake(8)), *s0 = static_cast<float*>(fake(9)), *s1 = static_cast<float*>(fake(10));
  float *dS = static_cast<float*>(fake(11)), *ds = static_cast<float*>(fake(12)), *dlg = static_cast<float*>(fake(13));
  const uint8_t* m = static_cast<const uint8_t*>(fake(14));
  void* ws = fake(15);
  const size_t room = size_t{1} << 47;
  for (int dt : {GDN_F32, GDN_BF16}) {
    // tokens by heads of the norm
    const int64_t tokens[][2] = {{1, 1},       {3, 7000},          {1, 1 << 24},        {1 << 24, 1},
                                 {5, 1 << 24}, {1, (1 << 26) + 1}, {(1 << 26) - 1, 1}, {1, (1 << 30) - 1}};
    for (auto& t : tokens)
      for (int64_t D : {8, 24, 64, 200, 512})
        for (int64_t H : {1, 9, 64})
          for (int inter : {0, 1}) {
            const gdn_norm_dims d{t[0], t[1], H, 1, D, D / 16 * 16, 9, 0, 0, dt, inter, 1e-6f, 0.f};
            size_t n = 0;
            expect(gdn_norm_rope_bwd_workspace_bytes(&d, &n), GDN_OK, "norm workspace", t[0], t[1], H, D);
            expect(gdn_norm_rope_fwd(&d, q, k, lg, s0, s1, nullptr, dq, dk, nullptr), GDN_OK, "norm", t[0], t[1], H, D);
            expect(gdn_norm_rope_bwd(&d, q, k, lg, s0, s1, nullptr, v, dO, dq, dk, dS, ds, ws, n, nullptr), GDN_OK,
                   "norm bwd", t[0], t[1], H, D);
          }
    // batches by heads of the decay operator: up to kMost pairs and kRow elements a row
    constexpr int64_t kMost = (1 << 21) - 64, kRow = 1 << 22;
    const int64_t bh[][3] = {{1, 1, 1},         {1, 3, 255},        {2, 2, 128},      {kMost, 1, 1}, {kMost / 2, 2, 2},
                             {kMost / 4, 1, 4}, {kMost + 1, 1, 1},  {kMost / 2 + 1, 1, 2}, {1, 1, 1 << 14},
                             {100, 1, 1 << 14}, {64, 1 << 14, 1 << 14}};
    for (auto& h : bh)
      for (int64_t T : {1, 4, 5, 64, 4097})
        for (int64_t Dk : {8, 128, 192, 256})
          for (int64_t Dv : {8, 128, 192, 256})
            for (int algo : {GDN_ALGO_AUTO, GDN_ALGO_SCAN, GDN_ALGO_CHUNK}) {
              const gdn_dims d{h[0], T, h[1], h[2], Dk, Dv, dt, algo, 0};
              const int fit = h[0] * h[2] <= kMost && h[2] * (Dk > Dv ? Dk : Dv) <= kRow ? GDN_OK : GDN_ERR_UNSUPPORTED;
              const int64_t sizes = Dk * 1000 + Dv;
              expect(gdn_decay_fwd(&d, q, k, v, lg, 1.f, s0, m, o, s1, ws, room, nullptr), fit, "decay", h[0], h[2], T, sizes);
              expect(gdn_decay_fwd(&d, q, k, v, lg, 1.f, s0, m, o, s0, ws, room, nullptr), fit, "in place", h[0], h[2], T, sizes);
              expect(gdn_decay_bwd(&d, q, k, v, lg, 1.f, s0, m, dO, dS, dq, dk, dv, dlg, ds, ws, room, nullptr),
                     algo == GDN_ALGO_SCAN ? GDN_ERR_UNSUPPORTED : fit, "decay bwd", h[0], h[2], T, sizes);
            }
  }
  printf("ok: %ld calls, %ld launches\n", calls, g_launches);
  return 0;
}
