// Rows of heads as the norm, rotation and cache kernels hold them: eight channels
// to a lane (16 bytes of bf16), LPH lanes to a row, the angles of a token's
// channels in registers for all of its heads.
#pragma once

#include "gdn_dev.h"

namespace gdn {

template <typename T> struct Raw;  // eight channels as they are stored
template <> struct Raw<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void put(bf16* p) const { *reinterpret_cast<uint4*>(p) = u; }
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
  __device__ __forceinline__ void put(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
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

// Args: the rotation's part of a launch's arguments (D, R, P, rope, pos; with AXES
// also A, axis and the tokens BT).
template <int LPH, bool INTER> struct Lane {
  int sub, c0, other;  // lane in the row, its first channel, the lane of the other channels
  bool on, turned;
  float sign;
  template <typename Args> __device__ __forceinline__ Lane(const Args& a) {
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
  // cos and sin at the token's position (dflt without positions; NaN where the table
  // has no such row); back: of the inverse rotation
  template <bool AXES, typename Args>
  __device__ __forceinline__ void load(const Args& a, int64_t token, int64_t dflt, Turn& tn, bool back) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tn.c[i] = 1.f;
      tn.s[i] = 0.f;
    }
    if (!turned) return;
    const float flip = back ? -1.f : 1.f;
    if constexpr (AXES) {
      if (a.axis) {
        load_axes(a, token, dflt, tn, flip);
        return;
      }
    }
    const int64_t pos = a.pos ? a.pos[token] : dflt;
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
  // The same with an axis to each pair: a lane's pairs may lie on any of them, so each
  // pair's cos and sin is a load of its own (sixteen, as many as whole rows of four
  // axes would take), once for all heads of the token.
  template <typename Args>
  __device__ __forceinline__ void load_axes(const Args& a, int64_t token, int64_t dflt, Turn& tn, float flip) const {
    constexpr int NP = INTER ? 4 : 8;
    const int p0 = INTER ? c0 / 2 : c0 < a.R / 2 ? c0 : c0 - a.R / 2;
    int64_t at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) at[x] = !a.pos ? dflt : x < a.A ? a.pos[x * a.BT + token] : -1;
    int axis[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) axis[i] = a.axis[p0 + i];
    float c[NP], s[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int64_t pos = axis[i] == 0 ? at[0] : axis[i] == 1 ? at[1] : axis[i] == 2 ? at[2] : at[3];
      const bool ok = axis[i] < a.A && pos >= 0 && pos < a.P;
      const float* row = a.rope + (ok ? pos : 0) * a.R;
      c[i] = s[i] = __builtin_nanf("");
      if (ok) {
        c[i] = row[p0 + i];
        s[i] = row[a.R / 2 + p0 + i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tn.c[i] = c[INTER ? i / 2 : i];
      tn.s[i] = INTER ? (i & 1 ? flip : -flip) * s[i / 2] : flip * sign * s[i];
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


// The smallest power of two of lanes that holds a row.
inline int lanes_for(int D) {
  int n = 1;
  while (8 * n < D) n *= 2;
  return n;
}

}  // namespace gdn
