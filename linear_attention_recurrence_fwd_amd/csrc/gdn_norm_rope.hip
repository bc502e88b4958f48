// RMS norm of every query and key head with a learned weight, and the rotation
// of its first R channels by the token's position, in one pass; and its VJP.
//
//   h = x (mean(x^2) + eps)^-1/2,  u = h (w + w_offset),  y = rotate(u)
//   e = rotate^-1(dy),  dw = sum over rows of e h,  a = e (w + w_offset),
//   dx = (mean(x^2) + eps)^-1/2 (a - h mean(a h))
//
// rotate turns the pairs (i, i + R/2) -- or (2i, 2i + 1) when interleaved --
// by the angle of pair i at the token's position (cos and sin from a table).
//
// Both directions are streams over the rows (2 and 3 row sizes of traffic).
// A row is held by LPH lanes, eight channels each (16 bytes of bf16), so a wave
// takes 64 / LPH rows of one token at a time and goes through a run of the
// token's heads with the cos and sin of its channels in registers: read once for
// the token instead of once for each head.  The other channel of a pair lies
// eight or more channels away in another lane of the row (or in the same lane
// when interleaved) and comes by a lane move of the raw storage.
//
// Bound by memory: 4096 tokens, 32 + 16 heads of 128, bf16: forward 103 MB in 21.5 us,
// 4.8 TB/s (a large copy: 5.1); backward 153 MB in 29.4 us, 5.2 TB/s, and 4 us for
// dw's parts; fp32 201 MB in 41 us, 4.9 TB/s, and 302 MB in 51 us, 5.9 TB/s, a part of
// it still cached.  64 tokens of 16 + 2 heads of 256, bf16 or fp32: 4 us, a launch and
// a trip to memory.
#include "gdn_dev.h"
#include "gdn_decay.h"

namespace gdn {
namespace {

template <typename T> struct Raw;  // eight channels as they are stored
template <> struct Raw<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(float* v) const { Vec16<bf16>::unpack(u, v); }
  __device__ __forceinline__ Raw from_lane(int src) const {
    Raw o;
    o.u = make_uint4(__shfl(u.x, src), __shfl(u.y, src), __shfl(u.z, src), __shfl(u.w, src));
    return o;
  }
  __device__ __forceinline__ static void store(bf16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
  }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void unpack(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ Raw from_lane(int src) const {
    Raw o;
    o.a = make_float4(__shfl(a.x, src), __shfl(a.y, src), __shfl(a.z, src), __shfl(a.w, src));
    o.b = make_float4(__shfl(b.x, src), __shfl(b.y, src), __shfl(b.z, src), __shfl(b.w, src));
    return o;
  }
  __device__ __forceinline__ static void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Sum over the LPH lanes of a row; every lane gets the same bits.
template <int LPH> __device__ __forceinline__ float row_sum(float v) {
  if constexpr (LPH >= 2) v += dpp<kQuadXor1>(v);
  if constexpr (LPH >= 4) v += dpp<kQuadXor2>(v);
  if constexpr (LPH >= 8) v += dpp<kRowHalfMirror>(v);
  if constexpr (LPH >= 16) v += dpp<kRowMirror>(v);
  if constexpr (LPH >= 32) v += __shfl_xor(v, 16);
  if constexpr (LPH >= 64) v += __shfl_xor(v, 32);
  return v;
}

// What a lane keeps for a token: cos and sin of its channels' pairs.  A pair's
// outputs are y1 = u1 cos - u2 sin, y2 = u2 cos + u1 sin, so a channel's is
// its own u times cos plus the other's times -sin or sin.
struct Turn {
  float c[8], s[8];
};

template <int LPH, bool INTER> struct Lane {
  int sub, c0, other;  // lane in the row, its first channel, the lane of the other channels
  bool on, turned;
  float sign;
  __device__ __forceinline__ Lane(const NormRopeArgs& a) {
    const int l = threadIdx.x & 63;
    sub = l % LPH;
    c0 = 8 * sub;
    on = c0 < a.D;
    turned = c0 < a.R;
    const int half = a.R / 16;  // lanes of the first channels of the pairs
    const int to = INTER || !turned ? sub : sub < half ? sub + half : sub - half;
    other = (l - sub) + to;
    sign = sub < half ? -1.f : 1.f;
  }
  // cos and sin at position pos (NaN where the table has no such row); back: of
  // the inverse rotation
  __device__ __forceinline__ void load(const NormRopeArgs& a, int64_t token, Turn& tn, bool back) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tn.c[i] = 1.f;
      tn.s[i] = 0.f;
    }
    if (!turned) return;
    const int64_t pos = a.pos ? a.pos[token] : token % a.T;
    const float flip = back ? -1.f : 1.f;
    if (pos < 0 || pos >= a.P) {
#pragma unroll
      for (int i = 0; i < 8; ++i) tn.c[i] = tn.s[i] = __builtin_nanf("");
      return;
    }
    const float* row = a.rope + pos * a.R;
    if constexpr (INTER) {
      const float4 c = *reinterpret_cast<const float4*>(row + c0 / 2);
      const float4 s = *reinterpret_cast<const float4*>(row + a.R / 2 + c0 / 2);
      const float cs[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        tn.c[i] = cs[i / 2];
        tn.s[i] = (i & 1 ? flip : -flip) * ss[i / 2];
      }
    } else {
      const int p0 = c0 < a.R / 2 ? c0 : c0 - a.R / 2;
      Raw<float> c, s;
      c.load(row + p0);
      s.load(row + a.R / 2 + p0);
      c.unpack(tn.c);
      s.unpack(tn.s);
#pragma unroll
      for (int i = 0; i < 8; ++i) tn.s[i] *= flip * sign;
    }
  }
  // v turned, given the other channels' values (unused when interleaved)
  __device__ __forceinline__ void turn(float* v, const float* o, const Turn& tn) const {
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float x = v[i], y = v[i + 1];
        v[i] = turned ? x * tn.c[i] + y * tn.s[i] : x;
        v[i + 1] = turned ? y * tn.c[i + 1] + x * tn.s[i + 1] : y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = turned ? v[i] * tn.c[i] + o[i] * tn.s[i] : v[i];
    }
  }
};

__device__ __forceinline__ void load_w(const float* w, const NormRopeArgs& a, int c0, bool on, float* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = on ? w[c0 + i] + a.w_offset : 0.f;
}

// A wave's work: token and run of head groups (a group: 64 / LPH heads); the
// query heads' groups come first, then the key heads'.
struct Work {
  int gq, gk;      // groups of query and key heads
  int run, runs;   // groups of one run, runs of one token
};

// Workgroups of a forward launch in x, of 2^30 threads: a launch's threads are
// counted in 32 bits in each direction.  More go on in y.
constexpr int64_t kFwdBlocks = 1 << 22;

template <typename T, int LPH, bool INTER>
__global__ void __launch_bounds__(256) fwd_kernel(NormRopeArgs a, Work wk) {
  constexpr int RPW = 64 / LPH;
  const Lane<LPH, INTER> ln(a);
  const int64_t item = (static_cast<int64_t>(blockIdx.y) * kFwdBlocks + blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t token = item / wk.runs;
  if (token >= a.BT) return;
  const int g0 = static_cast<int>(item % wk.runs) * wk.run, g1 = min(g0 + wk.run, wk.gq + wk.gk);
  const int sub_row = (threadIdx.x & 63) / LPH;
  Turn tn;
  ln.load(a, token, tn, false);
  const float inv = 1.f / static_cast<float>(a.D);
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lo = max(g0, part ? wk.gq : 0), hi = min(g1, part ? wk.gq + wk.gk : wk.gq);
    if (lo >= hi) continue;
    float wt[8], wo[8];
    const float* wp = part ? a.wk : a.wq;
    load_w(wp, a, ln.c0, ln.on, wt);
#pragma unroll
    for (int i = 0; i < 8; ++i) wo[i] = __shfl(wt[i], ln.other);
    const int H = part ? a.Hk : a.Hq, base = part ? wk.gq : 0;
    const T* src = static_cast<const T*>(part ? a.k : a.q) + token * (part ? a.ks : a.qs);
    T* dst = static_cast<T*>(part ? a.ok : a.oq) + token * H * a.D;
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
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
      const float r = 1.f / sqrtf(row_sum<LPH>(ss) * inv + a.eps);
      if constexpr (!INTER) {
        x.from_lane(ln.other).unpack(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= r * wo[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= r * wt[i];
      ln.turn(v, o, tn);
      if (on) Raw<T>::store(dst + head * a.D + ln.c0, v);
    }
  }
}

// The backward's blocks each take a run of tokens and leave their rows' part of
// dw in the workspace, [block][2][D]: lanes sum over their rows, then the rows of
// a wave, then the waves, all in a fixed order.
template <typename T, int LPH, bool INTER>
__global__ void __launch_bounds__(256) bwd_kernel(NormRopeArgs a, Work wk) {
  constexpr int RPW = 64 / LPH;
  const Lane<LPH, INTER> ln(a);
  const int w = threadIdx.x >> 6, sub_row = (threadIdx.x & 63) / LPH;
  const float inv = 1.f / static_cast<float>(a.D);
  __shared__ float red[4][2][8 * LPH];
  float wt[2][8], dw[2][8];
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    load_w(part ? a.wk : a.wq, a, ln.c0, ln.on, wt[part]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[part][i] = 0.f;
  }
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + w; item < a.BT * wk.runs;
       item += static_cast<int64_t>(gridDim.x) * 4) {
    const int64_t token = item / wk.runs;
    const int g0 = static_cast<int>(item % wk.runs) * wk.run, g1 = min(g0 + wk.run, wk.gq + wk.gk);
    Turn tn;
    ln.load(a, token, tn, true);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int lo = max(g0, part ? wk.gq : 0), hi = min(g1, part ? wk.gq + wk.gk : wk.gq);
      const int H = part ? a.Hk : a.Hq, base = part ? wk.gq : 0;
      const T* src = static_cast<const T*>(part ? a.k : a.q) + token * (part ? a.ks : a.qs);
      const T* dyp = static_cast<const T*>(part ? a.dyk : a.dyq) + token * H * a.D;
      T* dst = static_cast<T*>(part ? a.ok : a.oq) + token * H * a.D;
      for (int g = lo; g < hi; ++g) {
        const int head = (g - base) * RPW + sub_row;
        const bool on = ln.on && head < H;
        Raw<T> x, y;
        x.zero();
        y.zero();
        if (on) {
          x.load(src + head * a.D + ln.c0);
          y.load(dyp + head * a.D + ln.c0);
        }
        float v[8], e[8], o[8];
        x.unpack(v);
        y.unpack(e);
        if constexpr (!INTER) y.from_lane(ln.other).unpack(o);
        ln.turn(e, o, tn);
        float ss = 0.f, ah = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(v[i], v[i], ss);
          ah = fmaf(v[i], e[i] * wt[part][i], ah);
        }
        const float r = 1.f / sqrtf(row_sum<LPH>(ss) * inv + a.eps);
        const float m = row_sum<LPH>(ah) * r * r * inv;  // mean(a h) r
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (on) dw[part][i] = fmaf(e[i], v[i] * r, dw[part][i]);
          v[i] = r * (e[i] * wt[part][i]) - v[i] * r * m;
        }
        if (on) Raw<T>::store(dst + head * a.D + ln.c0, v);
      }
    }
  }
#pragma unroll
  for (int part = 0; part < 2; ++part)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = dw[part][i];
#pragma unroll
      for (int m = LPH; m < 64; m <<= 1) s += __shfl_xor(s, m);
      if (sub_row == 0) red[w][part][ln.c0 + i] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += 256) {
    const int part = i / a.D, c = i % a.D;
    a.part[static_cast<size_t>(blockIdx.x) * 2 * a.D + i] =
        (red[0][part][c] + red[1][part][c]) + (red[2][part][c] + red[3][part][c]);
  }
}

// dw: the blocks' parts summed in a fixed order, one workgroup for 8 of the 2 D
// sums, each by 128 lanes whose loads are independent.
__global__ void __launch_bounds__(1024) dw_kernel(NormRopeArgs a) {
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), row = threadIdx.x >> 3;
  float s = 0.f;
  if (c < 2 * a.D) {
#pragma unroll 4
    for (int b = row; b < a.blocks; b += 128) s += a.part[static_cast<size_t>(b) * 2 * a.D + c];
  }
  __shared__ float red[128][9];
  red[row][threadIdx.x & 7] = s;
  __syncthreads();
  for (int m = 64; m >= 1; m >>= 1) {
    if (row < m) red[row][threadIdx.x & 7] += red[row + m][threadIdx.x & 7];
    __syncthreads();
  }
  if (row == 0 && c < 2 * a.D) (c < a.D ? a.dwq : a.dwk)[c % a.D] = red[0][threadIdx.x & 7];
}

int lanes_for(int D) {
  int n = 1;
  while (8 * n < D) n *= 2;
  return n;
}

Work work_of(const NormRopeArgs& a, int64_t waves) {
  const int rpw = 64 / lanes_for(a.D);
  Work w;
  w.gq = (a.Hq + rpw - 1) / rpw;
  w.gk = (a.Hk + rpw - 1) / rpw;
  // a token's heads go to as many waves as it takes to have `waves` of them
  const int groups = w.gq + w.gk;
  int64_t runs = a.BT > 0 ? (waves + a.BT - 1) / a.BT : 1;
  if (runs > groups) runs = groups;
  w.run = static_cast<int>((groups + runs - 1) / runs);
  w.runs = (groups + w.run - 1) / w.run;
  return w;
}

template <typename T, int LPH>
hipError_t launch_lph(const NormRopeArgs& a, bool bwd, hipStream_t st) {
  if (!bwd) {
    const Work w = work_of(a, 8192);
    const int64_t n = (a.BT * w.runs + 3) / 4;
    const dim3 grid(static_cast<unsigned>(n < kFwdBlocks ? n : kFwdBlocks),
                    static_cast<unsigned>((n + kFwdBlocks - 1) / kFwdBlocks));
    if (a.interleaved) fwd_kernel<T, LPH, true><<<grid, 256, 0, st>>>(a, w);
    else fwd_kernel<T, LPH, false><<<grid, 256, 0, st>>>(a, w);
    return hipGetLastError();
  }
  if (a.blocks > 0) {
    const Work w = work_of(a, 8192);
    if (a.interleaved) bwd_kernel<T, LPH, true><<<a.blocks, 256, 0, st>>>(a, w);
    else bwd_kernel<T, LPH, false><<<a.blocks, 256, 0, st>>>(a, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  dw_kernel<<<a.D / 4, 1024, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T> hipError_t launch_any(const NormRopeArgs& a, bool bwd, hipStream_t st) {
  switch (lanes_for(a.D)) {
    case 1: return launch_lph<T, 1>(a, bwd, st);
    case 2: return launch_lph<T, 2>(a, bwd, st);
    case 4: return launch_lph<T, 4>(a, bwd, st);
    case 8: return launch_lph<T, 8>(a, bwd, st);
    case 16: return launch_lph<T, 16>(a, bwd, st);
    case 32: return launch_lph<T, 32>(a, bwd, st);
    default: return launch_lph<T, 64>(a, bwd, st);
  }
}

}  // namespace

int norm_rope_blocks(int64_t BT, int Hq, int Hk, int D, bool) {
  const int rpw = 64 / lanes_for(D);
  const int64_t groups = (Hq + rpw - 1) / rpw + (Hk + rpw - 1) / rpw;
  const int64_t n = (BT * groups + 3) / 4;
  return static_cast<int>(n < 1024 ? n : 1024);
}

hipError_t launch_norm_rope_fwd(const NormRopeArgs& a, bool bf, hipStream_t st) {
  if (a.BT == 0) return hipSuccess;
  return bf ? launch_any<gdn::bf16>(a, false, st) : launch_any<float>(a, false, st);
}
hipError_t launch_norm_rope_bwd(const NormRopeArgs& a, bool bf, hipStream_t st) {
  return bf ? launch_any<gdn::bf16>(a, true, st) : launch_any<float>(a, true, st);
}

}  // namespace gdn
