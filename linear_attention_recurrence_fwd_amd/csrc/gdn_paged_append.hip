// New tokens of a batch of sequences: queries and keys with the RMS norm and the
// rotation of gdn_norm_rope.hip, keys and values to their places in a paged cache,
// in one pass.
//
// A wave takes a run of a token's head groups (queries, keys, values), as the norm's
// kernels do, and finds the token's sequence, its place (past + number in the call)
// and the place's page itself, while the rows that it goes through first are on
// their way.
//
// Bound by memory where tokens are many: 12 prompts of 33 to 1500 tokens, 32 + 8 + 8 heads
// of 128, bf16, 257 MB in 62 us, 4.1 TB/s (a large copy: 5.15).  The rows' writes go to
// pages of 32 tokens.  One token of each of 64 sequences: 4 us, a launch and two trips to
// memory, one behind the other (the page's number, the row).
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
  const Lane<LPH, INTER> ln(a);
  const int64_t item = (static_cast<int64_t>(blockIdx.y) * kBlocks + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t token = item / wk.runs;
  if (token >= a.BT) return;
  const int g0 = static_cast<int>(item % wk.runs) * wk.run, g1 = min(g0 + wk.run, wk.gq + 2 * wk.gk);
  const T* const src[3] = {static_cast<const T*>(a.q) + token * a.qs, static_cast<const T*>(a.k) + token * a.ks,
                           static_cast<const T*>(a.v) + token * a.vs};
  turn_rows<T, LPH, INTER, true, 3>(a, ln, token, g0, g1, wk.gq, wk.gk, src, [&](Turn& tn, char* (&dst)[3], int64_t (&step)[3]) {
    dst[0] = dst[1] = dst[2] = nullptr;
    step[0] = a.D * static_cast<int64_t>(sizeof(T));
    step[1] = step[2] = a.pool.hs;
    int s;
    int64_t i;
    if (a.cu) {
      s = find_sequence(a.cu, a.S, token);
      if (s < 0 || s >= a.S) return;  // (the rows are read, and not written)
      i = token - a.cu[s];
    } else {
      s = static_cast<int>(token / a.per);
      i = token % a.per;
    }
    const int64_t place = a.past[s] + i, in_row = place >> a.pool.shift;
    const int page = place >= 0 && in_row < a.width ? a.table[s * a.width + in_row] : -1;
    if (g0 < wk.gq + wk.gk) ln.template load<true>(a, token, a.first + place, tn, false);
    dst[0] = static_cast<char*>(a.oq) + token * a.Hq * step[0];
    if (page < 0 || page >= a.pool.pages) return;
    const int64_t at = page * a.pool.ps + (place & ((1 << a.pool.shift) - 1)) * a.pool.ts;
    dst[1] = static_cast<char*>(a.kp) + at;
    dst[2] = static_cast<char*>(a.vp) + at;
  });
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
