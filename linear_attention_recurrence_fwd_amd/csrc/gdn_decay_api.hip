// C ABI of the decay operator and of the query/key norm with rotation (declared
// in include/gdn.h): argument validation, workspace layout and launch order.
// No allocation, no host sync.
#include "../../include/gdn.h"
#include "gdn_checks.h"
#include "gdn_decay.h"

#include <limits.h>

namespace {

using gdn::DecayDims;
using gdn::align_up;
using gdn::aligned;
using gdn::all_aligned;
using gdn::all_given;
using gdn::overlaps;
using gdn::Range;

// Bytes of the tensors with key heads, with value heads, of the states, mask and lg.
struct Sizes {
  size_t key, val, state, mask, lg;
  explicit Sizes(const gdn_dims* d) {
    const size_t bt = static_cast<size_t>(d->B) * d->T * (d->dtype == GDN_BF16 ? 2 : 4);
    key = bt * d->Hk * d->Dk;
    val = bt * d->Hv * d->Dv;
    state = static_cast<size_t>(d->B) * d->Hv * d->Dk * d->Dv * 4;
    mask = static_cast<size_t>(d->B) * d->T;
    lg = static_cast<size_t>(d->Hv) * 4;
  }
};

int check_dims(const gdn_dims* p, bool bwd, DecayDims* out) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->B < 1 || p->T < 0 || p->Hk < 1 || p->Hv < 1 || p->Dk < 1 || p->Dv < 1) return GDN_ERR_INVALID_ARG;
  if (p->Hv % p->Hk != 0) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (p->algo != GDN_ALGO_AUTO && p->algo != GDN_ALGO_SCAN && p->algo != GDN_ALGO_CHUNK &&
      p->algo != GDN_ALGO_CHUNK_TPAR)
    return GDN_ERR_INVALID_ARG;
  if (bwd && p->algo == GDN_ALGO_SCAN) return GDN_ERR_UNSUPPORTED;
  if (p->Dk % 8 || p->Dv % 8 || p->Dk > 256 || p->Dv > 256) return GDN_ERR_UNSUPPORTED;
  // counts that are held in 32 bits: steps, heads, (b, h) pairs times their slices
  // or segments, the threads of a launch over the pairs (dq's and dk's has up to
  // eight workgroups of 256 to a pair), and the bytes of 64 steps' rows (the
  // tensors themselves are addressed in 64)
  if (p->T > gdn::kDecayMaxT || p->Hv > gdn::kDecayMaxPairs || p->B > gdn::kDecayMaxPairs ||
      p->B * p->Hv > gdn::kDecayMaxPairs ||
      static_cast<double>(p->B) * p->T * p->Hv > 9.0e12 || p->Hv * (p->Dk > p->Dv ? p->Dk : p->Dv) > (1 << 22))
    return GDN_ERR_UNSUPPORTED;
  *out = DecayDims{static_cast<int>(p->B),  static_cast<int>(p->T),  static_cast<int>(p->Hk),
                   static_cast<int>(p->Hv), static_cast<int>(p->Dk), static_cast<int>(p->Dv)};
  return GDN_OK;
}

// Calls of a few steps take the steps in turn.  us in turn / by chunks, in a graph:
//   heads                        T = 1         T = 4         T = 6         T = 8
//   1 x 32, 128 x 128, bf16   4.9 /   9.4   7.6 /   9.4   9.5 /   9.5  11.5 /   9.4
//   16 x 32, 128 x 128, bf16 15.1 /  24.1  18.0 /  24.2  20.6 /  24.1  23.2 /  24.2
//   64 x 32, 128 x 128, bf16 46.2 /  81.1  62.0 /  81.4  71.0 /  82.0  78.9 /  82.2
//   8 x 8, 64 x 32, bf16      4.1 /   6.7   5.9 /   6.7   7.2 /   6.7   8.6 /   6.7
//   4 x 64, 192 x 128, bf16  12.3 /  16.4  16.7 /  16.5  19.7 /  16.1  22.6 /  16.8
//   1 x 32, 128 x 128, fp32   4.6 /  11.7   7.3 /  11.7   9.2 /  11.8  11.0 /  11.8
//   64 x 32, 128 x 128, fp32 47.0 / 102.6  64.3 / 103.8  73.5 / 104.5  83.0 / 105.8
// Four is where the first of them draw level; large batches and fp32 would gain in
// turn up to eight (by 4 to 30%), which this rule leaves.
constexpr int kFewSteps = 4;
bool use_step(const gdn_dims* p) {
  return p->algo == GDN_ALGO_SCAN || (p->algo == GDN_ALGO_AUTO && p->T <= kFewSteps);
}

// Segments up to which the forward's walks add up the sums before them themselves.
constexpr int kPrefixSegments = 8;

// Chunks per segment and segments.
struct Cut {
  int seg, n;
};
Cut cut(const gdn_dims* p, const DecayDims& d, bool bwd) {
  const int nc = d.nchunk();
  int n = 1;
  // one workgroup to a compute unit, and no second round of a few: at 48 (b, h)
  // and 16 chunks, 4 segments (192 workgroups) take 37 us, 6 (288) 47 us; at 64
  // and 32 chunks, 4 (256) take 72 us, 8 (512) 94 us
  if (p->algo != GDN_ALGO_CHUNK && nc > 1) n = gdn::kDecayMaxSeg / (d.B * d.Hv);
  if (n > nc) n = nc;
  if (n < 1) n = 1;
  // Segments pay where a pass over all chunks costs more than one over a
  // segment's, its sums (0.6 of a pass) and a launch and the states' traffic, in
  // chunks' times (3 us forward in bf16, 8 backward, 12 and more in fp32; the
  // states' part grows with their number).  128 x 128 heads, us, one pass against
  // segments: 8 heads, 130 steps 15 / 20, 512 steps 31 / 25; 64 heads, 512 steps
  // 31 / 35, 1024 steps 55 / 42; backward 64 heads, 512 steps 79 / 86, 1024 steps
  // 139 / 121; fp32 8 heads, 256 steps 55 / 32.  (The rule knows pairs and chunks
  // only: it leaves compute units idle at 129 to 255 (b, h), which stay one segment
  // each, and does not weigh a wide head's dearer chunks and states.)
  if (n > 1) {
    const float seg = static_cast<float>((nc + n - 1) / n), states = static_cast<float>(d.B) * d.Hv * n / 256.f;
    const float extra = p->dtype != GDN_BF16 ? 1.4f + states : bwd ? 1.5f + 6.f * states : 2.5f + 3.5f * states;
    if (static_cast<float>(nc) <= 1.6f * seg + extra) n = 1;
  }
  Cut c;
  c.seg = nc ? (nc + n - 1) / n : 1;
  c.n = nc ? (nc + c.seg - 1) / c.seg : 1;
  return c;
}

struct Layout {
  size_t S, R;            // segment states, forward and backward in time
  size_t steps;           // valid steps of the segments
  size_t grad;            // parts of dlg
  size_t pq, pk;          // rows of grouped heads
  size_t total;
};

// The waves that leave parts of dlg for a (b, h) and segment, and the parts in which a key
// head's value heads leave their dq and dk rows: the bf16 kernel goes through
// several value heads together, the fp32 walks through one.
int key_waves(const gdn_dims* p, const DecayDims& d) {
  return p->dtype == GDN_BF16 ? 4 * ((d.Dk + 63) / 64) : gdn::decay_waves(d.Dk);
}
int key_parts(const gdn_dims* p, const DecayDims& d, bool dq) {
  return p->dtype == GDN_BF16 && !dq ? d.G() / gdn::decay_heads_together(d.G()) : d.G();
}

Layout layout(const gdn_dims* p, const DecayDims& d, bool bwd) {
  Layout L{};
  size_t off = 0;
  auto take = [&](size_t nfloat) {
    const size_t o = off;
    off += align_up(nfloat * sizeof(float));
    return o;
  };
  const Cut c = cut(p, d, bwd);
  const size_t bh = static_cast<size_t>(d.B) * d.Hv;
  // (the forward's sums may lie in the walks' padded order)
  const size_t states = static_cast<size_t>(c.n) * bh * (bwd ? static_cast<size_t>(d.Dk) * d.Dv : gdn::decay_sum_floats(d.Dk, d.Dv));
  if (c.n > 1) {
    L.S = take(states);
    L.steps = take(static_cast<size_t>(d.B) * c.n);
  }
  if (bwd) {
    if (c.n > 1) L.R = take(states);
    L.grad = take(2 * bh * c.n * key_waves(p, d));  // fp64
    const size_t rows = static_cast<size_t>(d.B) * d.T * d.Hk * d.Dk;
    const int nq = key_parts(p, d, true), nk = key_parts(p, d, false);
    if (nq > 1) L.pq = take(rows * nq);
    if (nk > 1) L.pk = take(rows * nk);
  }
  L.total = off;
  return L;
}

template <typename P> P* at(void* ws, size_t off) { return reinterpret_cast<P*>(static_cast<char*>(ws) + off); }

gdn::DecayRows key_rows(const DecayDims& d, const void* p) { return gdn::DecayRows{p, d.Hk, d.Dk, d.G()}; }
gdn::DecayRows val_rows(const DecayDims& d, const void* p) { return gdn::DecayRows{p, d.Hv, d.Dv, 1}; }

// Walks whose state is [Dk, Dv] as stored (o, dv), and transposed (dq, dk).
gdn::DecayWalk walk_kv(const DecayDims& d) {
  gdn::DecayWalk w{};
  w.KD = d.Dk;
  w.N = d.Dv;
  w.sr = d.Dv;
  w.sc = 1;
  return w;
}
gdn::DecayWalk walk_vk(const DecayDims& d) {
  gdn::DecayWalk w{};
  w.KD = d.Dv;
  w.N = d.Dk;
  w.sr = 1;
  w.sc = d.Dv;
  return w;
}

int check_norm(const gdn_norm_dims* p, gdn::NormRopeArgs* a) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->B < 1 || p->T < 0 || p->Hq < 1 || p->Hk < 1 || p->D < 1 || p->R < 0 || p->P < 0) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_F32 && p->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (p->D % 8 || p->D > 512) return GDN_ERR_UNSUPPORTED;
  if (p->R > p->D) return GDN_ERR_INVALID_ARG;
  if (p->R % 16) return GDN_ERR_UNSUPPORTED;
  if (!(p->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (p->Hq > INT_MAX / 1024 || p->Hk > INT_MAX / 1024 || p->P > INT_MAX || p->B > INT_MAX || p->T > INT_MAX ||
      static_cast<double>(p->B) * p->T > INT_MAX / 2)
    return GDN_ERR_UNSUPPORTED;
  const int64_t qs = p->q_stride ? p->q_stride : p->Hq * p->D, ks = p->k_stride ? p->k_stride : p->Hk * p->D;
  const int64_t unit = p->dtype == GDN_BF16 ? 8 : 4;
  if (qs < p->Hq * p->D || ks < p->Hk * p->D || qs % unit || ks % unit || qs > INT_MAX || ks > INT_MAX)
    return GDN_ERR_INVALID_ARG;
  *a = gdn::NormRopeArgs{};
  a->BT = p->B * p->T;
  a->Hq = static_cast<int>(p->Hq);
  a->Hk = static_cast<int>(p->Hk);
  a->D = static_cast<int>(p->D);
  a->R = static_cast<int>(p->R);
  a->P = static_cast<int>(p->P);
  a->qs = qs;
  a->ks = ks;
  a->T = static_cast<int>(p->T);
  a->interleaved = p->interleaved != 0;
  a->eps = p->eps;
  a->w_offset = p->w_offset;
  a->blocks = gdn::norm_rope_blocks(a->BT, a->Hq, a->Hk, a->D, p->dtype == GDN_BF16);
  return GDN_OK;
}

// The rotation with A axes: weights for both norms or for none.
int check_axes(const gdn_norm_dims* p, int32_t A, const float* wq, const float* wk, gdn::NormRopeArgs* a) {
  const int rc = check_norm(p, a);
  if (rc) return rc;
  if (A < 1 || (wq == nullptr) != (wk == nullptr)) return GDN_ERR_INVALID_ARG;
  if (A > 4) return GDN_ERR_UNSUPPORTED;
  a->A = A;
  a->bare = wq == nullptr;
  return GDN_OK;
}

// Bytes of the dense rows, of the inputs' with their strides, of a weight, the
// table and the positions.
struct NormSizes {
  size_t q, k, qs, ks, w, rope, pos;
  NormSizes(const gdn_norm_dims* d, const gdn::NormRopeArgs& a) {
    const size_t es = d->dtype == GDN_BF16 ? 2 : 4, n = static_cast<size_t>(a.BT);
    const size_t qr = static_cast<size_t>(d->Hq) * d->D, kr = static_cast<size_t>(d->Hk) * d->D;
    q = n * qr * es;
    k = n * kr * es;
    qs = n ? ((n - 1) * a.qs + qr) * es : 0;
    ks = n ? ((n - 1) * a.ks + kr) * es : 0;
    w = static_cast<size_t>(d->D) * 4;
    rope = static_cast<size_t>(d->P) * d->R * 4;
    pos = n * 4;
  }
};

}  // namespace

extern "C" {

int gdn_decay_fwd_workspace_bytes(const gdn_dims* d, size_t* out) {
  DecayDims dd;
  const int rc = check_dims(d, false, &dd);
  if (rc) return rc;
  if (!out) return GDN_ERR_INVALID_ARG;
  *out = use_step(d) ? 0 : layout(d, dd, false).total;
  return GDN_OK;
}

int gdn_decay_bwd_workspace_bytes(const gdn_dims* d, size_t* out) {
  DecayDims dd;
  const int rc = check_dims(d, true, &dd);
  if (rc) return rc;
  if (!out) return GDN_ERR_INVALID_ARG;
  *out = layout(d, dd, true).total;
  return GDN_OK;
}

int gdn_decay_fwd(const gdn_dims* d, const void* q, const void* k, const void* v, const float* lg,
                  float scale, const float* state0, const uint8_t* mask, void* o, float* state_out,
                  void* ws, size_t ws_bytes, void* stream) {
  DecayDims dd;
  const int rc = check_dims(d, false, &dd);
  if (rc) return rc;
  if (!all_given(lg, state_out)) return GDN_ERR_INVALID_ARG;
  if (dd.T > 0 && !all_given(q, k, v, o)) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k, v, state0, o, state_out)) return GDN_ERR_INVALID_ARG;
  const bool bf = d->dtype == GDN_BF16;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Layout L = use_step(d) ? Layout{} : layout(d, dd, false);
  if (L.total > ws_bytes || (L.total > 0 && !ws)) return GDN_ERR_WORKSPACE;
  if (L.total > 0 && !aligned(ws)) return GDN_ERR_INVALID_ARG;
  const Sizes z(d);
  const Range out[] = {{o, z.val}, {state_out, z.state}, {ws, L.total}};
  const Range in[] = {{q, z.key}, {k, z.key}, {v, z.val}, {lg, z.lg}, {mask, z.mask},
                      {state0 == state_out ? nullptr : state0, z.state}};
  if (overlaps(out, in)) return GDN_ERR_INVALID_ARG;
  if (use_step(d)) {
    const gdn::DecayStepArgs a{dd, q, k, v, lg, scale, state0, mask, o, state_out};
    return gdn::launch_decay_step(a, bf, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  }
  const Cut c = cut(d, dd, false);
  gdn::DecayWalk w = walk_kv(dd);
  w.x = key_rows(dd, q);
  w.y = key_rows(dd, k);
  w.z = val_rows(dd, v);
  w.w = o;
  w.scale_p = w.scale_i = scale;
  w.scale_u = 1.f;
  w.start = state0;
  w.end = state_out;
  gdn::DecayWalkArgs a{dd, lg, mask, c.n, c.seg, 1, {w, w}};
  if (c.n > 1) {
    float *S = at<float>(ws, L.S), *steps = at<float>(ws, L.steps);
    // Few segments: each walk adds up the sums before its own.  Many, or a state
    // updated in place (which the first segment would read while the last one
    // writes it): a chain makes every start state first.
    const bool prefix = c.n <= kPrefixSegments && state_out != state0;
    gdn::DecayWalkArgs sum = a;
    sum.walk[0].seg_sum = S;
    sum.walk[0].seg_steps = steps;
    sum.walk[0].seg_native = prefix;
    if (gdn::launch_decay_walk(sum, true, bf, st) != hipSuccess) return GDN_ERR_HIP;
    if (prefix) {
      a.walk[0].seg_sum = S;
      a.walk[0].seg_steps = steps;
    } else {
      const gdn::DecayChainArgs ch{dd, lg, steps, c.n, S, state0, state_out, 0};
      if (gdn::launch_decay_chain(&ch, 1, st) != hipSuccess) return GDN_ERR_HIP;
      a.walk[0].seg_start = S;
      a.walk[0].end = nullptr;
    }
  }
  return gdn::launch_decay_walk(a, false, bf, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_decay_bwd(const gdn_dims* d, const void* q, const void* k, const void* v, const float* lg,
                  float scale, const float* state0, const uint8_t* mask, const void* dO,
                  const float* dS_final, void* dq, void* dk, void* dv, float* dlg, float* dstate,
                  void* ws, size_t ws_bytes, void* stream) {
  DecayDims dd;
  const int rc = check_dims(d, true, &dd);
  if (rc) return rc;
  if (!all_given(lg, dlg, dstate)) return GDN_ERR_INVALID_ARG;
  if (dd.T > 0 && !all_given(q, k, v, dO, dq, dk, dv)) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k, v, state0, dO, dS_final, dq, dk, dv, dstate)) return GDN_ERR_INVALID_ARG;
  const Layout L = layout(d, dd, true);
  if (L.total > ws_bytes || (L.total > 0 && !ws)) return GDN_ERR_WORKSPACE;
  if (L.total > 0 && !aligned(ws)) return GDN_ERR_INVALID_ARG;
  const Sizes z(d);
  const Range out[] = {{dq, z.key}, {dk, z.key}, {dv, z.val}, {dstate, z.state}, {dlg, z.lg}, {ws, L.total}};
  const Range in[] = {{q, z.key}, {k, z.key}, {v, z.val}, {lg, z.lg}, {mask, z.mask},
                      {dO, z.val}, {state0, z.state}, {dS_final, z.state}};
  if (overlaps(out, in)) return GDN_ERR_INVALID_ARG;
  const bool bf = d->dtype == GDN_BF16;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const Cut c = cut(d, dd, true);
  const int nq = key_parts(d, dd, true), nk = key_parts(d, dd, false);
  double* grad = at<double>(ws, L.grad);
  float *pq = at<float>(ws, L.pq), *pk = at<float>(ws, L.pk);  // (read and written with parts only)

  gdn::DecayWalk wv = walk_kv(dd);  // dv, dstate
  wv.x = key_rows(dd, k);
  wv.y = key_rows(dd, q);
  wv.z = val_rows(dd, dO);
  wv.w = dv;
  wv.reverse = 1;
  wv.scale_p = wv.scale_u = scale;
  wv.scale_i = 1.f;
  wv.start = dS_final;
  wv.end = dstate;

  float *S = nullptr, *R = nullptr;
  if (c.n > 1) {
    S = at<float>(ws, L.S);
    R = at<float>(ws, L.R);
    float* steps = at<float>(ws, L.steps);
    gdn::DecayWalk us = walk_kv(dd), ur = wv;
    us.y = key_rows(dd, k);
    us.z = val_rows(dd, v);
    us.scale_u = 1.f;
    us.seg_sum = S;
    us.seg_steps = steps;
    ur.seg_sum = R;
    const gdn::DecayWalkArgs sum{dd, lg, mask, c.n, c.seg, 2, {us, ur}};
    if (gdn::launch_decay_walk(sum, true, bf, st) != hipSuccess) return GDN_ERR_HIP;
    const gdn::DecayChainArgs ch[2] = {{dd, lg, steps, c.n, S, state0, nullptr, 0},
                                       {dd, lg, steps, c.n, R, dS_final, dstate, 1}};
    if (gdn::launch_decay_chain(ch, 2, st) != hipSuccess) return GDN_ERR_HIP;
    wv.seg_start = R;
    wv.end = nullptr;
  }
  const gdn::DecayWalkArgs av{dd, lg, mask, c.n, c.seg, 1, {wv, wv}};
  if (gdn::launch_decay_walk(av, false, bf, st) != hipSuccess) return GDN_ERR_HIP;
  if (bf) {
    const gdn::DecayKeysArgs ka{dd, lg, scale, mask, c.n, c.seg, q, k, v, dO, state0, dS_final, S, R, dq, dk, pq, pk, grad};
    if (gdn::launch_decay_keys(ka, st) != hipSuccess) return GDN_ERR_HIP;
  } else {
    gdn::DecayWalk wq = walk_vk(dd);  // dq
    wq.x = val_rows(dd, dO);
    wq.y = val_rows(dd, v);
    wq.z = key_rows(dd, k);
    wq.e = key_rows(dd, q);
    wq.w = nq > 1 ? pq : dq;
    wq.scale_p = wq.scale_i = scale;
    wq.scale_u = 1.f;
    wq.start = state0;
    wq.seg_start = S;
    wq.grad = grad;
    wq.R = dS_final;
    wq.seg_R = R;
    gdn::DecayWalk wk = walk_vk(dd);  // dk
    wk.x = val_rows(dd, v);
    wk.y = val_rows(dd, dO);
    wk.z = key_rows(dd, q);
    wk.w = nk > 1 ? pk : dk;
    wk.reverse = 1;
    wk.scale_p = wk.scale_u = scale;
    wk.scale_i = 1.f;
    wk.start = dS_final;
    wk.seg_start = R;
    const gdn::DecayWalkArgs aqk{dd, lg, mask, c.n, c.seg, 2, {wq, wk}};
    if (gdn::launch_decay_walk(aqk, false, false, st) != hipSuccess) return GDN_ERR_HIP;
  }
  if ((nq > 1 || nk > 1) && dd.T > 0) {
    const gdn::DecayGroupArgs ga{dd, {nq, nk}, pq, pk, dq, dk};
    if (gdn::launch_decay_group(ga, bf, st) != hipSuccess) return GDN_ERR_HIP;
  }
  const gdn::DecayReduceArgs ra{dd, c.n * key_waves(d, dd), grad, dlg};
  return gdn::launch_decay_reduce(ra, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

int gdn_norm_rope_fwd(const gdn_norm_dims* d, const void* q, const void* k, const float* wq,
                      const float* wk, const float* rope, const int32_t* pos, void* oq, void* ok,
                      void* stream) {
  gdn::NormRopeArgs a;
  const int rc = check_norm(d, &a);
  if (rc) return rc;
  if (!all_given(wq, wk) || (a.R > 0 && !rope)) return GDN_ERR_INVALID_ARG;
  if (a.BT > 0 && !all_given(q, k, oq, ok)) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k, wq, wk, rope, oq, ok)) return GDN_ERR_INVALID_ARG;
  const NormSizes z(d, a);
  const Range out[] = {{oq, z.q}, {ok, z.k}};
  const Range in[] = {{q, z.qs}, {k, z.ks}, {wq, z.w}, {wk, z.w}, {rope, z.rope}, {pos, z.pos}};
  if (overlaps(out, in)) return GDN_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.rope = rope;
  a.pos = pos;
  a.oq = oq;
  a.ok = ok;
  return gdn::launch_norm_rope_fwd(a, d->dtype == GDN_BF16, static_cast<hipStream_t>(stream)) == hipSuccess
             ? GDN_OK : GDN_ERR_HIP;
}

int gdn_norm_rope_bwd_workspace_bytes(const gdn_norm_dims* d, size_t* out) {
  gdn::NormRopeArgs a;
  const int rc = check_norm(d, &a);
  if (rc) return rc;
  if (!out) return GDN_ERR_INVALID_ARG;
  *out = align_up(static_cast<size_t>(a.blocks) * 2 * a.D * sizeof(float));
  return GDN_OK;
}

int gdn_norm_rope_bwd(const gdn_norm_dims* d, const void* q, const void* k, const float* wq,
                      const float* wk, const float* rope, const int32_t* pos, const void* dyq,
                      const void* dyk, void* dq, void* dk, float* dwq, float* dwk, void* ws,
                      size_t ws_bytes, void* stream) {
  gdn::NormRopeArgs a;
  const int rc = check_norm(d, &a);
  if (rc) return rc;
  if (!all_given(wq, wk, dwq, dwk) || (a.R > 0 && !rope)) return GDN_ERR_INVALID_ARG;
  if (a.BT > 0 && !all_given(q, k, dyq, dyk, dq, dk)) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k, wq, wk, rope, dyq, dyk, dq, dk, dwq, dwk)) return GDN_ERR_INVALID_ARG;
  const size_t need = align_up(static_cast<size_t>(a.blocks) * 2 * a.D * sizeof(float));
  if (need > ws_bytes || (need > 0 && !ws)) return GDN_ERR_WORKSPACE;
  const NormSizes z(d, a);
  const Range out[] = {{dq, z.q}, {dk, z.k}, {ws, need}};
  const Range in[] = {{q, z.qs},  {k, z.ks},  {dyq, z.q},     {dyk, z.k},
                      {wq, z.w}, {wk, z.w}, {rope, z.rope}, {pos, z.pos}};
  // (the weights' gradients are written when all inputs are read)
  const Range dw[] = {{dwq, z.w}, {dwk, z.w}};
  if (overlaps(out, in) || overlaps(dw, out)) return GDN_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.rope = rope;
  a.pos = pos;
  a.dyq = dyq;
  a.dyk = dyk;
  a.oq = dq;
  a.ok = dk;
  a.part = static_cast<float*>(ws);
  a.dwq = dwq;
  a.dwk = dwk;
  return gdn::launch_norm_rope_bwd(a, d->dtype == GDN_BF16, static_cast<hipStream_t>(stream)) == hipSuccess
             ? GDN_OK : GDN_ERR_HIP;
}

int gdn_norm_rope_axes_fwd(const gdn_norm_dims* d, int32_t A, const void* q, const void* k,
                           const float* wq, const float* wk, const float* rope, const uint8_t* axis,
                           const int32_t* pos, void* oq, void* ok, void* stream) {
  gdn::NormRopeArgs a;
  const int rc = check_axes(d, A, wq, wk, &a);
  if (rc) return rc;
  if (a.R > 0 && !rope) return GDN_ERR_INVALID_ARG;
  if (a.BT > 0 && !all_given(q, k, oq, ok)) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k, wq, wk, rope, oq, ok)) return GDN_ERR_INVALID_ARG;
  const NormSizes z(d, a);
  const Range out[] = {{oq, z.q}, {ok, z.k}};
  const Range in[] = {{q, z.qs}, {k, z.ks}, {wq, z.w}, {wk, z.w}, {rope, z.rope}, {pos, z.pos * A},
                      {axis, static_cast<size_t>(a.R / 2)}};
  if (overlaps(out, in)) return GDN_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.rope = rope;
  a.axis = axis;
  a.pos = pos;
  a.oq = oq;
  a.ok = ok;
  return gdn::launch_norm_rope_fwd(a, d->dtype == GDN_BF16, static_cast<hipStream_t>(stream)) == hipSuccess
             ? GDN_OK : GDN_ERR_HIP;
}

int gdn_norm_rope_axes_bwd(const gdn_norm_dims* d, int32_t A, const void* q, const void* k,
                           const float* wq, const float* wk, const float* rope, const uint8_t* axis,
                           const int32_t* pos, const void* dyq, const void* dyk, void* dq, void* dk,
                           float* dwq, float* dwk, void* ws, size_t ws_bytes, void* stream) {
  gdn::NormRopeArgs a;
  const int rc = check_axes(d, A, wq, wk, &a);
  if (rc) return rc;
  if (a.R > 0 && !rope) return GDN_ERR_INVALID_ARG;
  if (a.BT > 0 && !all_given(dyq, dyk, dq, dk)) return GDN_ERR_INVALID_ARG;
  if (!all_aligned(q, k, wq, wk, rope, dyq, dyk, dq, dk, dwq, dwk)) return GDN_ERR_INVALID_ARG;
  const bool bf = d->dtype == GDN_BF16;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const NormSizes z(d, a);
  a.rope = rope;
  a.axis = axis;
  a.pos = pos;
  a.oq = dq;
  a.ok = dk;
  if (a.bare) {
    // The rotation's VJP is the rotation back: a forward over the cotangents.
    const Range out[] = {{dq, z.q}, {dk, z.k}};
    const Range in[] = {{dyq, z.q}, {dyk, z.k}, {rope, z.rope}, {pos, z.pos * A}, {axis, static_cast<size_t>(a.R / 2)}};
    if (overlaps(out, in)) return GDN_ERR_INVALID_ARG;
    a.q = dyq;
    a.k = dyk;
    a.qs = d->Hq * d->D;
    a.ks = d->Hk * d->D;
    a.back = 1;
    return gdn::launch_norm_rope_fwd(a, bf, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  }
  if (!all_given(dwq, dwk) || (a.BT > 0 && !all_given(q, k))) return GDN_ERR_INVALID_ARG;
  const size_t need = align_up(static_cast<size_t>(a.blocks) * 2 * a.D * sizeof(float));
  if (need > ws_bytes || (need > 0 && !ws)) return GDN_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws)) return GDN_ERR_INVALID_ARG;
  const Range out[] = {{dq, z.q}, {dk, z.k}, {ws, need}};
  const Range in[] = {{q, z.qs}, {k, z.ks}, {dyq, z.q}, {dyk, z.k}, {wq, z.w}, {wk, z.w}, {rope, z.rope},
                      {pos, z.pos * A}, {axis, static_cast<size_t>(a.R / 2)}};
  // (the weights' gradients are written when all inputs are read)
  const Range dw[] = {{dwq, z.w}, {dwk, z.w}};
  if (overlaps(out, in) || overlaps(dw, out)) return GDN_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.dyq = dyq;
  a.dyk = dyk;
  a.part = static_cast<float*>(ws);
  a.dwq = dwq;
  a.dwk = dwk;
  return gdn::launch_norm_rope_bwd(a, bf, st) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
