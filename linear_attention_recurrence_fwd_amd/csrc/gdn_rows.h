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
    // (all loads are unconditional, from clamped places: under a condition each waits
    // for the one before it)
    int at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) at[x] = dflt < 0 || dflt >= a.P ? -1 : static_cast<int>(dflt);
    if (a.pos) {
#pragma unroll
      for (int x = 0; x < 4; ++x) at[x] = a.pos[min(x, a.A - 1) * a.BT + token];
    }
    int axis[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) axis[i] = a.axis[p0 + i];
    float c[NP], s[NP];
    int at_i[NP];
    bool ok[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      at_i[i] = axis[i] == 0 ? at[0] : axis[i] == 1 ? at[1] : axis[i] == 2 ? at[2] : at[3];
      ok[i] = axis[i] < a.A && at_i[i] >= 0 && at_i[i] < a.P;
      c[i] = s[i] = 0.f;
    }
    if (a.P > 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float* row = a.rope + static_cast<int64_t>(ok[i] ? at_i[i] : 0) * a.R + p0 + i;
        c[i] = row[0];
        s[i] = row[a.R / 2];
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      c[i] = ok[i] ? c[i] : __builtin_nanf("");
      s[i] = ok[i] ? s[i] : __builtin_nanf("");
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tn.c[i] = c[INTER ? i / 2 : i];
      tn.s[i] = INTER ? (i & 1 ? flip : -flip) * s[i / 2] : flip * sign * s[i];
    }
  }
  // v turned, given the other channels' values (unused when interleaved).  Which of the
  // two products is rounded is said here and not left to the compiler, so that every
  // kernel that turns rows gives the same bits: the own one forward, the other one back.
  template <bool BACK> __device__ __forceinline__ void turn(float* v, const float* o, const Turn& tn) const {
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float x = v[i], y = v[i + 1];
        v[i] = turned ? fmaf(x, tn.c[i], y * tn.s[i]) : x;
        v[i + 1] = turned ? fmaf(y, tn.c[i + 1], x * tn.s[i + 1]) : y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = BACK ? fmaf(v[i], tn.c[i], o[i] * tn.s[i]) : fmaf(o[i], tn.s[i], v[i] * tn.c[i]);
        v[i] = turned ? t : v[i];
      }
    }
  }
};


// A wave's run of a token's head groups (64 / LPH heads each): the groups of the
// query heads, then the key heads', then (PARTS = 3) the value heads', from g0 to g1.
// Queries and keys are normed (where they have weights) and turned; values are copied.
// A batch of rows is on its way while the one before it is worked on (rows one by one
// left the wave waiting for each: 8192 tokens of 32 + 8 heads of 128, bf16, several
// axes, 47 us against 38).  bf16 rows with one axis go one by one ahead, and the weights
// are fetched where a part begins: that takes 76 registers and not 126, and twice as many
// waves are there to wait for each other (4096 tokens of 16 + 2 heads of 256: 17.3 us, in
// batches of four 20.1; 32 + 16 heads of 192, interleaved, 31.4 and 35.8).  With several
// axes, whose angles are sixteen loads for each token, batches of four stay ahead (42 us
// against 44).  find is called once, behind the first batch's loads: it gives the token's
// angles, and where each part's rows go (null: nowhere) and from one head to the next, in
// bytes.
template <typename T, int LPH, bool INTER, bool AXES, int PARTS, typename Args, typename Find>
__device__ __forceinline__ void turn_rows(const Args& a, const Lane<LPH, INTER>& ln, int64_t token, int g0, int g1,
                                          int gq, int gk, const T* const (&src)[PARTS], Find find) {
  constexpr bool LEAN = sizeof(T) == 2 && !AXES;
  constexpr int RPW = 64 / LPH, U = LEAN ? 1 : sizeof(T) == 2 ? 4 : 2;
  const int sub_row = (threadIdx.x & 63) / LPH;
  const int begin[4] = {0, gq, gq + gk, gq + 2 * gk};
  auto part_of = [&](int g) { return g < begin[1] ? 0 : PARTS == 2 || g < begin[2] ? 1 : 2; };
  auto pick = [&](int part, auto x, auto y, auto z) { return part == 0 ? x : PARTS == 2 || part == 1 ? y : z; };
  auto last = [&](int part) { return min(g1, pick(part, begin[1], begin[2], begin[3])); };  // the part's end in the run
  auto fetch = [&](int g, Raw<T>(&x)[U]) {
    const int part = part_of(g), end = last(part), base = pick(part, begin[0], begin[1], begin[2]);
    const T* from = pick(part, src[0], src[1], src[PARTS - 1]);
    const int H = part ? a.Hk : a.Hq;
    // (from clamped places: a load under a condition waits for the one before it)
    const int c0 = ln.on ? ln.c0 : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(from + min((min(g + u, end - 1) - base) * RPW + sub_row, H - 1) * a.D + c0);
  };
  if (g0 >= g1) return;
  Raw<T> x[U];
  fetch(g0, x);
  Raw<float> raw[2];
  auto fetch_w = [&](int part, Raw<float>& x) {
    const float* wp = part ? a.wk : a.wq;
    x.zero();
    if (wp) x.load(wp + (ln.on ? ln.c0 : 0));
  };
  if constexpr (!LEAN) {
    fetch_w(0, raw[0]);
    fetch_w(1, raw[1]);
  }
  Turn tn;
  char* dst[3];
  int64_t step[3];
  find(tn, dst, step);
  const float inv = 1.f / static_cast<float>(a.D);
  float wt[8], wo[8];
  int now = -1;
#pragma unroll 1
  for (int g = g0; g < g1;) {
    const int part = part_of(g), end = last(part), next = min(g + U, end);
    Raw<T> y[U];
    if (next < g1) fetch(next, y);
    const bool normed = !AXES || (part ? a.wk : a.wq) != nullptr;
    if (part != now && part < 2) {
      float w0[8], w1[8];
      if constexpr (LEAN) {
        fetch_w(part, raw[0]);
        raw[1] = raw[0];
      }
      raw[0].unpack(w0);
      raw[1].unpack(w1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wt[i] = normed ? (part ? w1[i] : w0[i]) + a.w_offset : 1.f;
        wo[i] = __shfl(wt[i], ln.other);
      }
    }
    now = part;
    const int H = part ? a.Hk : a.Hq, base = pick(part, begin[0], begin[1], begin[2]);
    char* to = pick(part, dst[0], dst[1], dst[PARTS - 1]);
    const int64_t hop = pick(part, step[0], step[1], step[PARTS - 1]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g + u >= end) break;
      const int head = (g + u - base) * RPW + sub_row;
      const bool on = ln.on && head < H && to;
      T* out = reinterpret_cast<T*>(to + head * hop) + ln.c0;
      if (PARTS == 3 && part == 2) {
        if (on) x[u].put(out);
        continue;
      }
      float v[8], o[8];
      if (!ln.on) x[u].zero();
      x[u].unpack(v);
      float r = 1.f;
      if (normed) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
        r = 1.f / sqrtf(row_sum<LPH>(ss) * inv + a.eps);
      }
      if constexpr (!INTER) {
        x[u].from_lane(ln.other).unpack(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= r * wo[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= r * wt[i];
      ln.template turn<false>(v, o, tn);
      if (on) Raw<T>::store(out, v);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = y[u];
    g = next;
  }
}

// The smallest power of two of lanes that holds a row.
inline int lanes_for(int D) {
  int n = 1;
  while (8 * n < D) n *= 2;
  return n;
}

}  // namespace gdn
