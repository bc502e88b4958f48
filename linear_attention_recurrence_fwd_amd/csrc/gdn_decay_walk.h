// The walk kernel of the decay operator (see DecayWalk in gdn_decay.h).
//
// A workgroup owns one segment of one (batch, value head) and goes through its
// chunks of CH steps with the whole state in registers: wave w holds columns
// 32 w .. 32 w + 31 of all KD channels, fp32, in the accumulator layout of the
// matrix cores.  With c_i the valid steps of the chunk up to step i (counted in
// walk order; up to and with i forward in time, before i backward), L its valid
// steps, and g = e^lg:
//   P_ij = [j <= i] g^(c_i - c_j) (x_i . y_j)
//   w_i  = g^c_i S^T x_i + sum_j P_ij z_j
//   S   <- g^L S + sum_j y_j (g^(L - c_j) z_j)^T
// Masked steps take no part because their rows are read as zeros (y and z
// forward, x backward); their own decay is one because c does not grow there.
//
// The products run on bf16 matrix cores with fp32 sums for bf16 tensors, on
// the fp32 ones for fp32 tensors.  Where bf16 operands are not tensors as they
// were given, they are rounded as follows:
//   - g^(L - c_j) z_j, which the state sums: as three bf16 parts (24 bits), so
//     the state keeps fp32 precision over any number of steps;
//   - the state against x: one bf16 part, as the result is rounded to bf16 (a
//     relative error of at most 2^-8 for each product, independent between the
//     products); three parts where the result also enters the fp32 sums for dlg;
//   - P: one bf16 part, as the result is rounded to bf16.
#pragma once

#include "gdn_dev.h"
#include "gdn_decay.h"

namespace gdn {
namespace decay {

constexpr float kLog2e = 1.44269504088896340736f;

// log2 of the decay of one step; -inf (a state that is dropped at every step)
// becomes a finite value that still gives 0 for one step and 1 for none.
__device__ __forceinline__ float log2_decay(float lg) { return (lg < -1e30f ? -1e30f : lg) * kLog2e; }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Eight floats as bf16 parts: hi + mid + lo holds 24 bits of each.
__device__ __forceinline__ bf16x8 pack8(const float* v) {
  return as_bf16x8(make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]),
                              pack2_bf16(v[6], v[7])));
}
__device__ __forceinline__ void minus8(float* v, const bf16x8& p) {
  const uint4 u = __builtin_bit_cast(uint4, p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] -= __uint_as_float(w[i] << 16);
    v[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int N> __device__ __forceinline__ void split8(float* v, bf16x8 (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = pack8(v);
    if (i + 1 < N) minus8(v, part[i]);
  }
}

// Workgroups are dealt to the 8 XCDs in turn: this order gives each XCD a run
// of neighbouring work items, so the value heads that share a key head's rows
// find them in one L2.  Items past n stay idle.
__device__ __forceinline__ int xcd_order(int blk, int n) {
  const int per = (n + 7) / 8;
  return (blk & 7) * per + (blk >> 3);
}

template <typename T> struct Cfg;
template <> struct Cfg<bf16> {
  static constexpr int CH = 64, EPP = 8;
};
template <> struct Cfg<float> {
  static constexpr int CH = 32, EPP = 4;
};

template <typename T, int KD, int NW, bool OUT, bool DOTS>
struct Smem {
  static constexpr int CH = Cfg<T>::CH, EPP = Cfg<T>::EPP;
  static constexpr int PX = KD / EPP, PZ = 32 * NW / EPP;
  uint4 x[OUT ? CH * PX : 1];
  uint4 y[CH * PX];
  uint4 z[CH * PZ];
  uint4 e[DOTS ? CH * PZ : 1];
  uint4 p[OUT ? CH * CH / EPP : 1];
  float c[CH], rf[CH], sw[CH];
};

// Tiles in LDS: row-major 16-byte pieces, piece p of row r at p ^ (r & 7).
template <int PPR> __device__ __forceinline__ int piece(int r, int p) { return r * PPR + (p ^ (r & 7)); }
// 8-byte unit u of row r.
template <int PPR> __device__ __forceinline__ const uint2* unit(const uint4* t, int r, int u) {
  return reinterpret_cast<const uint2*>(t + piece<PPR>(r, u >> 1)) + (u & 1);
}

template <typename T, int PPR, int NT>
__device__ __forceinline__ void load_tile(uint4* dst, const DecayRows& s, size_t bT, int Tn, int h, int t0, bool rev,
                                          const uint8_t* zero_at) {
  constexpr int CH = Cfg<T>::CH, EPP = Cfg<T>::EPP;
  const T* base = static_cast<const T*>(s.p) + static_cast<size_t>(h / s.group) * s.D;
  const size_t rs = static_cast<size_t>(s.H) * s.D;
#pragma unroll 4
  for (int i = threadIdx.x; i < CH * PPR; i += NT) {
    const int r = i / PPR, p = i % PPR, t = rev ? t0 + CH - 1 - r : t0 + r;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < Tn && p * EPP < s.D && (zero_at == nullptr || zero_at[t] != 0))
      v = *reinterpret_cast<const uint4*>(base + (bT + t) * rs + p * EPP);
    dst[piece<PPR>(r, p)] = v;
  }
}

__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum16(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// SPS: bf16 parts of the state in the products with x.
template <typename T, int KD, int NW, bool OUT, bool DOTS, int SPS>
__global__ void __launch_bounds__(64 * NW) walk_kernel(DecayWalkArgs a) {
  using M = Smem<T, KD, NW, OUT, DOTS>;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int CH = M::CH, EPP = M::EPP, PX = M::PX, PZ = M::PZ, PP = CH / EPP, MT = CH / 16, KT = KD / 16;
  constexpr int NT = 64 * NW;
  __shared__ M sm;
  const DecayDims& d = a.d;
  const int BH = d.B * d.Hv, per_walk = BH * a.nseg;
  const int id = xcd_order(blockIdx.x, per_walk * a.nwalk);
  if (id >= per_walk * a.nwalk) return;
  const DecayWalk& wk = a.walk[id / per_walk];
  // value heads fastest: the heads of a group run side by side
  const int it = id % per_walk, h = it % d.Hv, sg = (it / d.Hv) % a.nseg, b = it / (d.Hv * a.nseg);
  const int bh = b * d.Hv + h;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, lr = l & 15, g = l >> 4;
  const bool rev = wk.reverse != 0;
  const size_t bT = static_cast<size_t>(b) * d.T;
  const uint8_t* mrow = a.mask ? a.mask + bT : nullptr;
  const float lg2 = log2_decay(a.lg[h]);

  // state tile i, register r of lane (lr, g): channel 32 (i/2) + 8 g + 4 (i%2)
  // + r for bf16 (two tiles together then are the B operand of a 32-deep
  // product as they stand), 16 i + 4 g + r for fp32; column 32 w + 16 n + lr
  auto chan = [&](int i, int r) { return BF ? 32 * (i / 2) + 8 * g + 4 * (i % 2) + r : 16 * i + 4 * g + r; };
  f32x4 S[KT][2];
  {
    const bool first = rev ? sg == a.nseg - 1 : sg == 0;
    const size_t hs = static_cast<size_t>(d.Dk) * d.Dv;
    const float* src = nullptr;
    if (OUT) {
      if (wk.seg_start) src = wk.seg_start + (static_cast<size_t>(sg) * BH + bh) * hs;
      else if (first && wk.start) src = wk.start + bh * hs;
    }
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ch = chan(i, r), col = 32 * w + 16 * n + lr;
          S[i][n][r] = src && ch < wk.KD && col < wk.N
                           ? src[static_cast<size_t>(ch) * wk.sr + static_cast<size_t>(col) * wk.sc] : 0.f;
        }
  }

  const int t_lo = sg * a.seg * kDecayChunk;
  const int t_hi = min(d.T, t_lo + a.seg * kDecayChunk);
  const int nch = t_hi > t_lo ? (t_hi - t_lo + CH - 1) / CH : 0;
  const size_t nstat = (static_cast<size_t>(d.T) + CH - 1) / CH;
  for (int ci = 0; ci < nch; ++ci) {
    const int cc = rev ? nch - 1 - ci : ci;
    const int t0 = t_lo + cc * CH;
    __syncthreads();  // the tiles of the chunk before are read
    if constexpr (OUT) load_tile<T, PX, NT>(sm.x, wk.x, bT, d.T, h, t0, rev, rev ? mrow : nullptr);
    load_tile<T, PX, NT>(sm.y, wk.y, bT, d.T, h, t0, rev, rev ? nullptr : mrow);
    load_tile<T, PZ, NT>(sm.z, wk.z, bT, d.T, h, t0, rev, rev ? nullptr : mrow);
    if constexpr (DOTS) load_tile<T, PZ, NT>(sm.e, wk.e, bT, d.T, h, t0, rev, rev ? mrow : nullptr);
    // the valid steps, in walk order
    const int tl = rev ? t0 + CH - 1 - l : t0 + l;
    const bool live = l < CH && tl < d.T && (mrow == nullptr || mrow[tl] != 0);
    const unsigned long long bal = __ballot(live);
    const int L = __popcll(bal);
    if (w == 0 && l < CH) {
      const float c = static_cast<float>(__popcll(bal & ((rev ? 1ull : 2ull) << l) - 1ull));
      sm.c[l] = c;
      sm.rf[l] = wk.scale_i * exp2_fast(lg2 * c);
      sm.sw[l] = wk.scale_u * exp2_fast(lg2 * (static_cast<float>(L) - c));
    }
    __syncthreads();

    f32x4 acc[MT][2];
    if constexpr (OUT) {
      // ---- P, transposed tiles (rows j, columns i): lower ones, and zeros
      // where a 32-deep product reaches past the diagonal
      float intra = 0.f;
      // (BF: MT (MT + 1) / 2 lower tiles, then tiles (0, 1) and (2, 3))
      constexpr int LOW = MT * (MT + 1) / 2, TILES = LOW + (BF ? MT / 2 : 0);
      for (int tile = w; tile < TILES; tile += NW) {
        int mt, nt;
        if (tile >= LOW) {
          mt = 2 * (tile - LOW);
          nt = mt + 1;
        } else {
          mt = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0;
          nt = tile - mt * (mt + 1) / 2;
        }
        {
          f32x4 t = f4zero();
          if (nt <= mt) {
            f32x4 u = f4zero();
            if constexpr (BF) {
#pragma unroll
              for (int ks = 0; ks < KD / 32; ++ks)
                t = mfma16(load_bf16x8(&sm.y[piece<PX>(16 * nt + lr, 4 * ks + g)]),
                           load_bf16x8(&sm.x[piece<PX>(16 * mt + lr, 4 * ks + g)]), t);
              if constexpr (DOTS) {
#pragma unroll
                for (int ks = 0; ks < NW; ++ks)
                  u = mfma16(load_bf16x8(&sm.z[piece<PZ>(16 * nt + lr, 4 * ks + g)]),
                             load_bf16x8(&sm.e[piece<PZ>(16 * mt + lr, 4 * ks + g)]), u);
              }
            } else {
#pragma unroll
              for (int ks = 0; ks < KD / 16; ++ks) {
                const float4 yv = *reinterpret_cast<const float4*>(&sm.y[piece<PX>(16 * nt + lr, 4 * ks + g)]);
                const float4 xv = *reinterpret_cast<const float4*>(&sm.x[piece<PX>(16 * mt + lr, 4 * ks + g)]);
                t = mfma16f(yv.x, xv.x, t);
                t = mfma16f(yv.y, xv.y, t);
                t = mfma16f(yv.z, xv.z, t);
                t = mfma16f(yv.w, xv.w, t);
              }
              if constexpr (DOTS) {
#pragma unroll
                for (int ks = 0; ks < 2 * NW; ++ks) {
                  const float4 zv = *reinterpret_cast<const float4*>(&sm.z[piece<PZ>(16 * nt + lr, 4 * ks + g)]);
                  const float4 ev = *reinterpret_cast<const float4*>(&sm.e[piece<PZ>(16 * mt + lr, 4 * ks + g)]);
                  u = mfma16f(zv.x, ev.x, u);
                  u = mfma16f(zv.y, ev.y, u);
                  u = mfma16f(zv.z, ev.z, u);
                  u = mfma16f(zv.w, ev.w, u);
                }
              }
            }
            const float ci_ = sm.c[16 * mt + lr];
            const float4 cj = *reinterpret_cast<const float4*>(&sm.c[16 * nt + 4 * g]);
            const float cjs[4] = {cj.x, cj.y, cj.z, cj.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float dn = ci_ - cjs[r];
              const bool in = 16 * nt + 4 * g + r <= 16 * mt + lr;
              t[r] = in ? t[r] * exp2_fast(lg2 * dn) * wk.scale_p : 0.f;
              if constexpr (DOTS) intra += in ? dn * t[r] * u[r] : 0.f;
            }
          }
          if constexpr (BF)
            reinterpret_cast<uint2*>(&sm.p[piece<PP>(16 * mt + lr, 2 * nt + (g >> 1))])[g & 1] =
                pack4_bf16(t[0], t[1], t[2], t[3]);
          else
            *reinterpret_cast<f32x4*>(&sm.p[piece<PP>(16 * mt + lr, 4 * nt + g)]) = t;
        }
      }
      // ---- S^T x
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[mt][0] = acc[mt][1] = f4zero();
      if constexpr (BF) {
#pragma unroll
        for (int ks = 0; ks < KD / 32; ++ks) {
          bf16x8 xa[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) xa[mt] = load_bf16x8(&sm.x[piece<PX>(16 * mt + lr, 4 * ks + g)]);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              v[r] = S[2 * ks][n][r];
              v[4 + r] = S[2 * ks + 1][n][r];
            }
            bf16x8 part[SPS];
            split8<SPS>(v, part);
#pragma unroll
            for (int s = 0; s < SPS; ++s)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) acc[mt][n] = mfma16(xa[mt], part[s], acc[mt][n]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float4 xv = *reinterpret_cast<const float4*>(&sm.x[piece<PX>(16 * mt + lr, 4 * i + g)]);
            const float xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int n = 0; n < 2; ++n) acc[mt][n] = mfma16f(xs[r], S[i][n][r], acc[mt][n]);
          }
      }
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float4 rf = *reinterpret_cast<const float4*>(&sm.rf[16 * mt + 4 * g]);
        const float rfs[4] = {rf.x, rf.y, rf.z, rf.w};
        float ct[4];
        if constexpr (DOTS) {
          const float4 c4 = *reinterpret_cast<const float4*>(&sm.c[16 * mt + 4 * g]);
          ct[0] = c4.x; ct[1] = c4.y; ct[2] = c4.z; ct[3] = c4.w;
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float ev[4];
          if constexpr (DOTS) {
            if constexpr (BF) {
              const uint2 u = lds_read_tr16(unit<PZ>(sm.e, 16 * mt + 4 * g + (lr >> 2), 4 * (2 * w + n) + (lr & 3)));
              ev[0] = __uint_as_float(u.x << 16);
              ev[1] = __uint_as_float(u.x & 0xffff0000u);
              ev[2] = __uint_as_float(u.y << 16);
              ev[3] = __uint_as_float(u.y & 0xffff0000u);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                ev[r] = reinterpret_cast<const float*>(
                    &sm.e[piece<PZ>(16 * mt + 4 * g + r, 4 * (2 * w + n) + (lr >> 2))])[lr & 3];
            }
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc[mt][n][r] *= rfs[r];
            if constexpr (DOTS) {
              const float f = acc[mt][n][r] * ev[r];
              s0 += f;
              s1 = fmaf(ct[r], f, s1);
            }
          }
        }
      }
      if constexpr (DOTS) {
        s0 = wave_sum(s0);
        s1 = wave_sum(s1);
        intra = wave_sum(intra);
        if (l == 0) {
          const size_t at = (static_cast<size_t>(bh) * nstat + t0 / CH) * NW + w;
          if (rev) {
            wk.dots[at * kDecayKStats] = s0;
            wk.dots[at * kDecayKStats + 1] = s1;
            wk.dots[at * kDecayKStats + 2] = static_cast<float>(L);
          } else {
            wk.dots[at * kDecayQStats] = s0;
            wk.dots[at * kDecayQStats + 1] = s1;
            wk.dots[at * kDecayQStats + 2] = intra;
          }
        }
      }
      __syncthreads();  // P is whole
    }

    // ---- products with z: P z, and the state's update
    const float gL = exp2_fast(lg2 * static_cast<float>(L));
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i][n][r] *= gL;
    if constexpr (BF) {
#pragma unroll
      for (int kt = 0; kt < CH / 32; ++kt) {
        const int r0 = 32 * kt + 8 * g + (lr >> 2);
        float sw[8];
        *reinterpret_cast<float4*>(sw) = *reinterpret_cast<const float4*>(&sm.sw[32 * kt + 8 * g]);
        *reinterpret_cast<float4*>(sw + 4) = *reinterpret_cast<const float4*>(&sm.sw[32 * kt + 8 * g + 4]);
        bf16x8 zp[2][3];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int u = 4 * (2 * w + n) + (lr & 3);
          const uint2 z0 = lds_read_tr16(unit<PZ>(sm.z, r0, u)), z1 = lds_read_tr16(unit<PZ>(sm.z, r0 + 4, u));
          const uint4 zu = make_uint4(z0.x, z0.y, z1.x, z1.y);
          if constexpr (OUT) {
            const bf16x8 zf = as_bf16x8(zu);
#pragma unroll
            for (int mt = 2 * kt; mt < MT; ++mt)
              acc[mt][n] = mfma16(load_bf16x8(&sm.p[piece<PP>(16 * mt + lr, 4 * kt + g)]), zf, acc[mt][n]);
          }
          float v[8];
          Vec16<bf16>::unpack(zu, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] *= sw[k];
          split8<3>(v, zp[n]);
        }
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int u = 8 * (i / 2) + 2 * (lr & 3) + (i & 1);
          const uint2 y0 = lds_read_tr16(unit<PX>(sm.y, r0, u)), y1 = lds_read_tr16(unit<PX>(sm.y, r0 + 4, u));
          const bf16x8 ya = as_bf16x8(make_uint4(y0.x, y0.y, y1.x, y1.y));
#pragma unroll
          for (int s = 2; s >= 0; --s)
#pragma unroll
            for (int n = 0; n < 2; ++n) S[i][n] = mfma16(ya, zp[n][s], S[i][n]);
        }
      }
    } else {
#pragma unroll
      for (int bq = 0; bq < CH / 16; ++bq) {
        float zv[2][4], sw[4];
        *reinterpret_cast<float4*>(sw) = *reinterpret_cast<const float4*>(&sm.sw[16 * bq + 4 * g]);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            zv[n][r] = reinterpret_cast<const float*>(
                &sm.z[piece<PZ>(16 * bq + 4 * g + r, 4 * (2 * w + n) + (lr >> 2))])[lr & 3];
        if constexpr (OUT) {
#pragma unroll
          for (int mt = bq; mt < MT; ++mt) {
            const float4 pv = *reinterpret_cast<const float4*>(&sm.p[piece<PP>(16 * mt + lr, 4 * bq + g)]);
            const float ps[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int n = 0; n < 2; ++n) acc[mt][n] = mfma16f(ps[r], zv[n][r], acc[mt][n]);
          }
        }
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float yv = reinterpret_cast<const float*>(
                &sm.y[piece<PX>(16 * bq + 4 * g + r, 4 * i + (lr >> 2))])[lr & 3];
#pragma unroll
            for (int n = 0; n < 2; ++n) S[i][n] = mfma16f(yv, zv[n][r] * sw[r], S[i][n]);
          }
      }
    }

    if constexpr (OUT) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * mt + 4 * g + r, t = rev ? t0 + CH - 1 - row : t0 + row;
          if (t >= d.T) continue;
          const size_t at = ((bT + t) * d.Hv + h) * wk.N;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int col = 32 * w + 16 * n + lr;
            if (col >= wk.N) continue;
            if (wk.w32) static_cast<float*>(wk.w)[at + col] = acc[mt][n][r];
            else static_cast<T*>(wk.w)[at + col] = from_f32<T>(acc[mt][n][r]);
          }
        }
    }
  }

  // ---- the state behind the segment
  const size_t hs = static_cast<size_t>(d.Dk) * d.Dv;
  float* dst = nullptr;
  const float* crs = nullptr;
  if constexpr (OUT) {
    if (sg == (rev ? 0 : a.nseg - 1) && wk.end) dst = wk.end + bh * hs;
    if (wk.seg_cross) crs = wk.seg_cross + (static_cast<size_t>(sg) * BH + bh) * hs;
    else if (wk.cross) crs = wk.cross + bh * hs;
  } else {
    dst = wk.seg_sum + (static_cast<size_t>(sg) * BH + bh) * hs;
  }
  float dot = 0.f;
  if (dst || crs) {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int ch = chan(i, r), col = 32 * w + 16 * n + lr;
          if (ch >= wk.KD || col >= wk.N) continue;
          const size_t at = static_cast<size_t>(ch) * wk.sr + static_cast<size_t>(col) * wk.sc;
          if (dst) dst[at] = S[i][n][r];
          if (crs) dot = fmaf(S[i][n][r], crs[at], dot);
        }
  }
  if constexpr (OUT && !DOTS) {
    if (wk.dots) {
      dot = wave_sum(dot);
      if (l == 0) wk.dots[(static_cast<size_t>(bh) * a.nseg + sg) * NW + w] = dot;
    }
  }
}

template <typename T, int KD, int NW>
hipError_t launch_nw(const DecayWalkArgs& a, hipStream_t st) {
  const int n = a.d.B * a.d.Hv * a.nseg * a.nwalk, grid = (n + 7) / 8 * 8;
  const DecayWalk& w = a.walk[0];
  if (w.seg_sum) walk_kernel<T, KD, NW, false, false, 1><<<grid, 64 * NW, 0, st>>>(a);
  else if (w.e.p) walk_kernel<T, KD, NW, true, true, 3><<<grid, 64 * NW, 0, st>>>(a);
  else walk_kernel<T, KD, NW, true, false, 1><<<grid, 64 * NW, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int KD> hipError_t launch_kd(const DecayWalkArgs& a, hipStream_t st) {
  switch (decay_waves(a.walk[0].N)) {
    case 2: return launch_nw<T, KD, 2>(a, st);
    case 4: return launch_nw<T, KD, 4>(a, st);
    case 6: return launch_nw<T, KD, 6>(a, st);
    default: return launch_nw<T, KD, 8>(a, st);
  }
}

}  // namespace decay

// One translation unit per (type, channel class): gdn_decay_walk_*.hip.
hipError_t decay_walk_bf16_64(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_bf16_128(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_bf16_192(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_bf16_256(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_64(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_128(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_192(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_256(const DecayWalkArgs& a, hipStream_t st);

}  // namespace gdn
