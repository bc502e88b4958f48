// New tokens of a batch of sequences: queries and keys with the RMS norm and the
// rotation of gdn_norm_rope.hip, keys and values to their places in a paged cache,
// in one pass.
//
// A wave takes a run of a token's head groups (queries, keys, values), as the norm's
// kernels do, and finds the token's sequence, its place (past + number in the call)
// and the place's page itself, while the rows that it goes through first are on
// their way.
#include "gdn_paged.h"
#include "gdn_rows.h"

namespace gdn {
namespace {

// Groups of 64 / LPH heads of q, then of k, then of v; runs of them.
struct Work {
  int gq, gk;
  int run, runs;
};
constexpr int64_t kBlocks = 1 << 22;  // workgroups in x, of 2^30 threads; more go on in y

// The sequence of a token (wave-uniform): the last s with cu[s] <= token, by sixty-four
// of its candidates at a time; -1 before the first, S behind the last.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int S, int64_t token) {
  int lo = -1, n = S + 1;  // candidates lo + 1 .. lo + n; cu[lo] <= token
  const int lane = threadIdx.x & 63;
  while (n > 0) {
    const int step = (n + 63) / 64, i = lo + (lane + 1) * step;
    const bool in = (lane + 1) * step <= n;
    const int c = __popcll(__ballot(in && cu[in ? i : 0] <= token));
    // the answer is in lo + c step .. lo + (c + 1) step - 1
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  return lo;
}

template <typename T, int LPH, bool INTER>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs a, Work wk) {
  constexpr int RPW = 64 / LPH;
  const Lane<LPH, INTER> ln(a);
  const int64_t item = (static_cast<int64_t>(blockIdx.y) * kBlocks + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t token = item / wk.runs;
  if (token >= a.BT) return;
  int s;
  int64_t i;
  if (a.cu) {
    s = find_sequence(a.cu, a.S, token);
    if (s < 0 || s >= a.S) return;
    i = token - a.cu[s];
  } else {
    s = static_cast<int>(token / a.per);
    i = token % a.per;
  }
  const int64_t place = a.past[s] + i, in_row = place >> a.pool.shift;
  const bool room = place >= 0 && in_row < a.width;
  const int page = room ? a.table[s * a.width + in_row] : -1;
  const bool write = page >= 0 && page < a.pool.pages;
  const int64_t at = write ? page * a.pool.ps + (place & ((1 << a.pool.shift) - 1)) * a.pool.ts : 0;
  const int g0 = static_cast<int>(item % wk.runs) * wk.run, g1 = min(g0 + wk.run, wk.gq + 2 * wk.gk);
  const int sub_row = (threadIdx.x & 63) / LPH;
  Turn tn;
  if (g0 < wk.gq + wk.gk) ln.template load<true>(a, token, a.first + place, tn, false);
  const float inv = 1.f / static_cast<float>(a.D);
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lo = max(g0, part ? wk.gq : 0), hi = min(g1, part ? wk.gq + wk.gk : wk.gq);
    if (lo >= hi || (part && !write)) continue;
    const float* wp = part ? a.wk : a.wq;
    float wt[8], wo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[j] = !ln.on ? 0.f : wp ? wp[ln.c0 + j] + a.w_offset : 1.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) wo[j] = __shfl(wt[j], ln.other);
    const int H = part ? a.Hk : a.Hq, base = part ? wk.gq : 0;
    const T* src = static_cast<const T*>(part ? a.k : a.q) + token * (part ? a.ks : a.qs);
    char* dst = part ? static_cast<char*>(a.kp) + at : static_cast<char*>(a.oq) + token * H * a.D * static_cast<int64_t>(sizeof(T));
    const int64_t step = part ? a.pool.hs : a.D * static_cast<int64_t>(sizeof(T));
    for (int g = lo; g < hi; ++g) {
      const int head = (g - base) * RPW + sub_row;
      const bool on = ln.on && head < H;
      Raw<T> x;
      x.zero();
      if (on) x.load(src + head * a.D + ln.c0);
      float v[8], o[8];
      x.unpack(v);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
      const float r = wp ? 1.f / sqrtf(row_sum<LPH>(ss) * inv + a.eps) : 1.f;
      if constexpr (!INTER) {
        x.from_lane(ln.other).unpack(o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= r * wo[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= r * wt[j];
      ln.turn(v, o, tn);
      if (on) Raw<T>::store(reinterpret_cast<T*>(dst + head * step) + ln.c0, v);
    }
  }
  if (!write) return;
  for (int g = max(g0, wk.gq + wk.gk); g < g1; ++g) {
    const int head = (g - wk.gq - wk.gk) * RPW + sub_row;
    if (!ln.on || head >= a.Hk) continue;
    Raw<T> x;
    x.load(static_cast<const T*>(a.v) + token * a.vs + head * a.D + ln.c0);
    x.put(reinterpret_cast<T*>(static_cast<char*>(a.vp) + at + head * a.pool.hs) + ln.c0);
  }
}

template <typename T, int LPH> hipError_t launch_lph(const AppendArgs& a, hipStream_t st) {
  constexpr int RPW = 64 / LPH;
  Work w;
  w.gq = (a.Hq + RPW - 1) / RPW;
  w.gk = (a.Hk + RPW - 1) / RPW;
  // a token's heads go to as many waves as it takes to have 8192 of them
  const int groups = w.gq + 2 * w.gk;
  int64_t runs = (8192 + a.BT - 1) / a.BT;
  if (runs > groups) runs = groups;
  w.run = static_cast<int>((groups + runs - 1) / runs);
  w.runs = (groups + w.run - 1) / w.run;
  const int64_t n = (a.BT * w.runs + 3) / 4;
  const dim3 grid(static_cast<unsigned>(n < kBlocks ? n : kBlocks), static_cast<unsigned>((n + kBlocks - 1) / kBlocks));
  if (a.interleaved) append_kernel<T, LPH, true><<<grid, 256, 0, st>>>(a, w);
  else append_kernel<T, LPH, false><<<grid, 256, 0, st>>>(a, w);
  return hipGetLastError();
}

template <typename T> hipError_t launch_any(const AppendArgs& a, hipStream_t st) {
  switch (lanes_for(a.D)) {
    case 1: return launch_lph<T, 1>(a, st);
    case 2: return launch_lph<T, 2>(a, st);
    case 4: return launch_lph<T, 4>(a, st);
    case 8: return launch_lph<T, 8>(a, st);
    case 16: return launch_lph<T, 16>(a, st);
    default: return launch_lph<T, 32>(a, st);
  }
}

}  // namespace

hipError_t launch_append(const AppendArgs& a, bool bf, hipStream_t st) {
  if (a.BT == 0) return hipSuccess;
  return bf ? launch_any<bf16>(a, st) : launch_any<float>(a, st);
}

}  // namespace gdn
