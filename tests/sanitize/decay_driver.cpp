// Host-only sanitizer build of the C ABI of the decay operator and the query/key
// norm (gdn_decay_api.hip): the kernel launchers are replaced by stand-ins that
// read both ends of every workspace region that they are handed, with the extent
// the kernels address, and the driver allocates the workspaces with malloc at
// exactly the queried sizes.  Tensors are placeholders that are never read.
#include <stdio.h>
#include <stdlib.h>

#include "../../include/gdn.h"
#include "../../linear_attention_recurrence_fwd_amd/csrc/gdn_decay.h"

namespace {
long g_launches = 0;
volatile unsigned char g_sink;
void touch(const void* p, size_t bytes) {
  if (!p || !bytes) return;
  const volatile unsigned char* c = static_cast<const volatile unsigned char*>(p);
  g_sink = c[0];
  g_sink = c[bytes - 1];
}
// Places of tensors that nothing reads here, far enough from each other and from the heap.
void* fake(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 48); }
size_t bh(const gdn::DecayDims& d) { return static_cast<size_t>(d.B) * d.Hv; }
size_t states(const gdn::DecayDims& d, int n) { return n * bh(d) * d.Dk * d.Dv * 4; }
}  // namespace

namespace gdn {
int decay_waves(int N) { return N <= 64 ? 4 : N <= 128 ? 8 : N <= 192 ? 12 : 8; }
size_t decay_sum_floats(int KD, int N) {
  auto up = [](int n) { return static_cast<size_t>(n <= 64 ? 64 : n <= 128 ? 128 : n <= 192 ? 192 : 256); };
  return up(KD) * up(N);
}
hipError_t launch_decay_walk(const DecayWalkArgs& a, bool, bool, hipStream_t) {
  for (int i = 0; i < a.nwalk; ++i) {
    const DecayWalk& w = a.walk[i];
    if (w.seg_sum && w.seg_native) touch(w.seg_sum, a.nseg * bh(a.d) * decay_sum_floats(w.KD, w.N) * 4);
    else if (w.seg_sum && !w.seg_start && !w.w) touch(w.seg_sum, states(a.d, a.nseg));
    touch(w.seg_steps, static_cast<size_t>(a.d.B) * a.nseg * 4);
    touch(w.seg_start, states(a.d, a.nseg));
    touch(w.seg_R, states(a.d, a.nseg));
    touch(w.grad, bh(a.d) * a.nseg * decay_waves(w.N) * 8);
    // the fp32 dq and dk walks of grouped heads leave rows for the sum over a group
    if (a.walk[0].e.p && a.d.G() > 1) touch(w.w, static_cast<size_t>(a.d.B) * a.d.T * a.d.Hv * w.N * 4);
  }
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_decay_keys(const DecayKeysArgs& a, hipStream_t) {
  if (a.nseg > 1) {
    touch(a.S, states(a.d, a.nseg));
    touch(a.R, states(a.d, a.nseg));
  }
  touch(a.grad, bh(a.d) * a.nseg * 4 * ((a.d.Dk + 63) / 64) * 8);
  const size_t rows = static_cast<size_t>(a.d.B) * a.d.T * a.d.Dk * 4;
  const int nk = a.d.G() / decay_heads_together(a.d.G());
  if (a.d.G() > 1) touch(a.pq, rows * a.d.Hv);
  if (nk > 1) touch(a.pk, rows * a.d.Hk * nk);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_decay_chain(const DecayChainArgs* a, int n, hipStream_t) {
  for (int i = 0; i < n; ++i) {
    touch(a[i].states, states(a[i].d, a[i].nseg));
    touch(a[i].seg_steps, static_cast<size_t>(a[i].d.B) * a[i].nseg * 4);
  }
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_decay_reduce(const DecayReduceArgs& a, hipStream_t) {
  touch(a.grad, bh(a.d) * a.n * 8);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_decay_group(const DecayGroupArgs& a, bool, hipStream_t) {
  const size_t rows = static_cast<size_t>(a.d.B) * a.d.T * a.d.Hk * a.d.Dk * 4;
  if (a.parts[0] > 1) touch(a.pq, rows * a.parts[0]);
  if (a.parts[1] > 1) touch(a.pk, rows * a.parts[1]);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_decay_step(const DecayStepArgs&, bool, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
int norm_rope_blocks(int64_t BT, int Hq, int Hk, int, bool) {
  const int64_t n = BT * (Hq + Hk);
  return static_cast<int>(n < 1024 ? n : 1024);
}
hipError_t launch_norm_rope_fwd(const NormRopeArgs&, bool, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_norm_rope_bwd(const NormRopeArgs& a, bool, hipStream_t) {
  touch(a.part, static_cast<size_t>(a.blocks) * 2 * a.D * 4);
  ++g_launches;
  return hipSuccess;
}
}  // namespace gdn

#define EXPECT(c)                                              \
  do {                                                         \
    if (!(c)) {                                                \
      fprintf(stderr, "line %d: %s\n", __LINE__, #c);          \
      exit(1);                                                 \
    }                                                          \
  } while (0)

int main() {
  void *q = fake(0), *k = fake(1), *v = fake(2), *o = fake(3), *dO = fake(4), *dq = fake(5), *dk = fake(6), *dv = fake(7);
  float *lg = static_cast<float*>(fake(8)), *s0 = static_cast<float*>(fake(9)), *s1 = static_cast<float*>(fake(10));
  float *dS = static_cast<float*>(fake(11)), *ds = static_cast<float*>(fake(12)), *dlg = static_cast<float*>(fake(13));
  const uint8_t* m = static_cast<const uint8_t*>(fake(14));
  const int64_t Ts[] = {0, 1, 2, 63, 64, 65, 200, 515, 1024, 2048, 40000};
  const int64_t heads[][2] = {{1, 1}, {1, 4}, {2, 6}, {3, 24}, {16, 64}, {40, 320}};
  const int64_t sizes[][2] = {{8, 8}, {64, 40}, {128, 128}, {192, 128}, {72, 256}, {256, 200}};
  long calls = 0;
  for (int64_t B : {1, 3, 70})
    for (int64_t T : Ts)
      for (auto& h : heads)
        for (auto& s : sizes)
          for (int dt : {GDN_F32, GDN_BF16})
            for (int algo : {GDN_ALGO_AUTO, GDN_ALGO_SCAN, GDN_ALGO_CHUNK, GDN_ALGO_CHUNK_TPAR}) {
              if (B * T * h[1] > 2000000) continue;  // (the partial rows are allocated)
              const gdn_dims d{B, T, h[0], h[1], s[0], s[1], dt, algo, 0};
              size_t n = 0;
              EXPECT(gdn_decay_fwd_workspace_bytes(&d, &n) == GDN_OK);
              if (n < (size_t{6} << 30)) {
                void* ws = n ? malloc(n) : nullptr;
                EXPECT(gdn_decay_fwd(&d, q, k, v, lg, 1.f, nullptr, m, o, s1, ws, n, nullptr) == GDN_OK);
                EXPECT(gdn_decay_fwd(&d, q, k, v, lg, 1.f, s0, nullptr, o, s1, ws, n, nullptr) == GDN_OK);
                EXPECT(gdn_decay_fwd(&d, q, k, v, lg, 1.f, s0, m, o, s0, ws, n, nullptr) == GDN_OK);  // in place
                if (n) EXPECT(gdn_decay_fwd(&d, q, k, v, lg, 1.f, s0, m, o, s0, ws, n - 1, nullptr) == GDN_ERR_WORKSPACE);
                free(ws);
                ++calls;
              }
              const int rc = gdn_decay_bwd_workspace_bytes(&d, &n);
              EXPECT(rc == (algo == GDN_ALGO_SCAN ? GDN_ERR_UNSUPPORTED : GDN_OK));
              if (rc == GDN_OK && n < (size_t{6} << 30)) {
                void* ws = malloc(n);
                EXPECT(gdn_decay_bwd(&d, q, k, v, lg, 1.f, s0, m, dO, dS, dq, dk, dv, dlg, ds, ws, n, nullptr) == GDN_OK);
                EXPECT(gdn_decay_bwd(&d, q, k, v, lg, 1.f, s0, m, dO, dS, dq, dk, dv, dlg, ds, ws, n - 1, nullptr) == GDN_ERR_WORKSPACE);
                free(ws);
                ++calls;
              }
            }
  for (int64_t B : {1, 7})
    for (int64_t T : {0, 1, 5, 3000})
      for (int64_t D : {8, 64, 192, 512})
        for (int dt : {GDN_F32, GDN_BF16}) {
          const gdn_norm_dims d{B, T, 5, 3, D, D / 16 * 16, 9, 0, 0, dt, 0, 1e-6f, 0.f};
          size_t n = 0;
          EXPECT(gdn_norm_rope_bwd_workspace_bytes(&d, &n) == GDN_OK);
          void* ws = n ? malloc(n) : nullptr;
          EXPECT(gdn_norm_rope_fwd(&d, q, k, lg, s0, s1, nullptr, dq, dk, nullptr) == GDN_OK);
          EXPECT(gdn_norm_rope_bwd(&d, q, k, lg, s0, s1, nullptr, v, dO, dq, dk, dS, ds, ws, n, nullptr) == GDN_OK);
          free(ws);
          ++calls;
        }
  printf("ok: %ld calls, %ld launches\n", calls, g_launches);
  return 0;
}
