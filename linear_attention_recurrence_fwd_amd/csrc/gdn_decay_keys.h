// dq and dk of a key head (bf16): the walks over the value heads that share it,
// together.  See DecayKeysArgs in gdn_decay.h and the walk kernel
// (gdn_decay_walk.h), whose parts this one is made of:
//   dq: x = dO, y = v,  z = k, e = q, forward in time;  w summed over the heads
//   dk: x = v,  y = dO, z = q, backward in time
// dq carries the states' derivatives in lg beside them (E, see the walk kernel), with
// all products that reach dlg in three bf16 parts; dk's state and sums reach bf16
// results only (one part against x, two in its update).
//
// A workgroup of four waves owns 64 columns of GH value heads' transposed states
// [Dv, Dk], all in registers (wave w: 16 columns of every head's), and for each
// chunk goes through the heads.  The sum over the heads then stays in registers,
// where one workgroup to a head would write fp32 rows for another kernel to sum
// (at 4 heads to a key head, 9/4 of the bytes that q, k, v, dO, dq, dk and dv have
// together), and what depends on the key head alone is made once a chunk: z as an
// operand, e at the places of the results, and e . z for dlg.  After the first
// head's P is made neither tile is read again, so the next chunk's come in while
// the heads are gone through.  Two workgroups fit a compute unit for Dv <= 128, and
// one's products fill the other's waits.  The blocks of 64 columns repeat P, a tenth
// of the products.
//
// dq's bound are vector instructions (half of its cycles; matrix products a third):
// of some 1000 a wave and chunk, 560 cut the two states and what they sum into bf16
// parts.  Two parts for dlg would save a third of them and leave errors of 2^-17 in
// each product, which a dlg of cancelling terms shows.  dk is bound like the walks.
#pragma once

#include "gdn_decay_walk.h"

namespace gdn {
namespace decay {

template <int KD> struct KeysLds {
  static constexpr int CH = 64, PX = KD / 8, PZ = 8, PP = 8;
  static constexpr int XB = CH * PX * 16, ZB = CH * PZ * 16;
  static constexpr int Y = 0, X = 2 * XB, Z = X + XB, E = Z + ZB, P = E + ZB, F = P + CH * PP * 16;
  static constexpr int TOTAL = F + 2 * 4 * CH * 4;
};

// Workgroup `block` of one direction's.
template <int KD, int GH, bool DQ>
__device__ __forceinline__ void keys_walk(const DecayKeysArgs& a, int block, char* sm) {
  using M = KeysLds<KD>;
  constexpr int CH = M::CH, PX = M::PX, PZ = M::PZ, PP = M::PP, MT = 4, KT = KD / 16, NW = 4;
  const int Hv = a.d.Hv, Hk = a.d.Hk, Tn = a.d.T, Dk = a.d.Dk, Dv = a.d.Dv, nseg = a.nseg, parts = a.d.G() / GH;
  const int ncb = (Dk + 63) / 64, n_items = a.d.B * nseg * Hk * parts * ncb;
  const int it = xcd_order(block, n_items);
  if (it >= n_items) return;
  // blocks of columns fastest, then a key head's parts: they share rows
  const int cb = it % ncb * 64, hp = it / ncb % (Hk * parts), sg = it / (ncb * Hk * parts) % nseg;
  const int b = it / (ncb * Hk * parts * nseg), hk = hp / parts, h0 = hp * GH;
  constexpr bool rev = !DQ;
  constexpr int SP = DQ ? 3 : 1, SU = DQ ? 3 : 2;  // bf16 parts of the state, of what it sums
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, lr = l & 15, g = l >> 4;
  const size_t bT = static_cast<size_t>(b) * Tn;
  const uint8_t* mrow = a.mask ? a.mask + bT : nullptr;
  const bool masked = mrow != nullptr;
  const uint32_t lds0 = lds_addr(sm);
  const bf16 *xp = static_cast<const bf16*>(rev ? a.v : a.dO), *yp = static_cast<const bf16*>(rev ? a.dO : a.v);
  const bf16 *zp_ = static_cast<const bf16*>(rev ? a.q : a.k), *ep = static_cast<const bf16*>(a.q);
  // scale on P, on the product with the state, on the state's update
  const float scale_p = a.scale, scale_i = rev ? 1.f : a.scale, scale_u = rev ? a.scale : 1.f;
  float lg2[GH];
#pragma unroll
  for (int q = 0; q < GH; ++q) lg2[q] = log2_decay(a.lg[h0 + q]);

  const int col = cb + 16 * w + lr;
  f32x4 S[GH][KT], E[DQ ? GH : 1][KT];
  double grad[GH];

  const int t_lo = sg * a.seg * kDecayChunk, t_hi = min(Tn, t_lo + a.seg * kDecayChunk);
  const int nch = t_hi > t_lo ? (t_hi - t_lo + CH - 1) / CH : 0;
  auto chunk_start = [&](int ci) { return t_lo + (rev ? nch - 1 - ci : ci) * CH; };
  auto mask_byte = [&](int ci) -> int {
    if (!masked || ci >= nch) return 1;
    return mrow[max(0, min(chunk_start(ci) + (rev ? CH - 1 - l : l), Tn - 1))];
  };
  auto live_of = [&](int ci, int byte) -> unsigned long long {
    return __ballot(chunk_start(ci) + (rev ? CH - 1 - l : l) < Tn && byte != 0);
  };

  Loader<CH, PX, 8, NW> lx;
  Loader<CH, PZ, 8, NW> lz;
  lx.init(w, l, static_cast<uint32_t>(Hv) * Dv * 2, Dv, rev);
  lz.init(w, l, static_cast<uint32_t>(Hk) * Dk * 2, Dk - cb, rev);
  auto rows = [&](const bf16* p, int H, int head, int D, int t0, int c0) {
    const int n = min(Tn - t0, CH);
    const uint64_t at = reinterpret_cast<uint64_t>(p + ((bT + t0) * H + head) * D + c0);
    return i32x4{static_cast<int>(at), static_cast<int>(at >> 32) & 0xffff, ((n - 1) * H * D + D - c0) * 2, 0x00020000};
  };
  auto issue_x = [&](int ci, int q, unsigned long long live) {
    const i32x4 dx = rows(xp, Hv, h0 + q, Dv, chunk_start(ci), 0);
    if (masked && rev) lx.load_live(dx, lds0 + M::X, w, l, live);
    else lx.load(dx, lds0 + M::X, w, l);
  };
  auto issue_y = [&](int ci, int q, int slot, unsigned long long live) {
    const i32x4 dy = rows(yp, Hv, h0 + q, Dv, chunk_start(ci), 0);
    if (masked && !rev) lx.load_live(dy, lds0 + M::Y + slot * M::XB, w, l, live);
    else lx.load(dy, lds0 + M::Y + slot * M::XB, w, l);
  };
  auto issue_ze = [&](int ci, unsigned long long live) {
    const i32x4 dz = rows(zp_, Hk, hk, Dk, chunk_start(ci), cb);
    if (masked && !rev) lz.load_live(dz, lds0 + M::Z, w, l, live);
    else lz.load(dz, lds0 + M::Z, w, l);
    if constexpr (DQ) lz.load(rows(ep, Hk, hk, Dk, chunk_start(ci), cb), lds0 + M::E, w, l);
  };
  // c, row factors, source weights, and these times the steps left, for head q
  auto factors = [&](int set, float lg2q, unsigned long long live) {
    float* f = reinterpret_cast<float*>(sm + M::F) + set * 4 * CH + l;
    const float c = static_cast<float>(__popcll(live & (((rev ? 1ull : 2ull) << l) - 1ull)));
    const float left = static_cast<float>(__popcll(live)) - c;
    f[0] = c;
    f[CH] = scale_i * exp2_fast(lg2q * c);
    f[2 * CH] = scale_u * exp2_fast(lg2q * left);
    f[3 * CH] = left * f[2 * CH];
  };

  // operand places, as in the walk kernel; piece 4 e further is 64 e in the place's
  // exclusive or, made at each use to save registers (opaque() keeps it there)
  constexpr int QX = PX % 16 == 0 ? 4 : 2;
  uint32_t rx = static_cast<uint32_t>(lr * PX + (g ^ key<PX>(lr))) * 16u, rz[2], ty[2], tz[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    rz[q] = static_cast<uint32_t>(lr * PZ + ((4 * q + g) ^ key<PZ>(lr))) * 16u;
    const int row = 8 * g + (lr >> 2) + 4 * q, c = 16 * w + 4 * (lr & 3);
    ty[q] = static_cast<uint32_t>(row * PX + ((lr & 3) ^ key<PX>(row))) * 16u;
    tz[q] = static_cast<uint32_t>(row * PZ + ((c >> 3) ^ key<PZ>(row))) * 16u + (c & 4) * 2;
  }
  // (a row of 8 or 24 pieces starts at a multiple of 8 pieces: bit 6 is the piece's)
  auto at_x = [&](int tile, int ks) { return (rx ^ (ks % QX * 64u)) + tile * 16 * PX * 16 + (ks / QX) * QX * 64; };
  auto opaque = [](uint32_t& v) { asm volatile("" : "+v"(v)); };
  // P's tiles of this wave: w, w + 4, w + 8 of the ten on and below the diagonal
  constexpr int TP = 3;
  auto tile_of = [&](int k, int& mt, int& nt) {
    const int t = w + 4 * k;
    mt = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
    nt = t - mt * (mt + 1) / 2;
    return t < 10;
  };

  unsigned long long live = 0, live_next = 0;
  int byte_next = 1;
  if (nch > 0) {
    live = live_of(0, mask_byte(0));
    byte_next = mask_byte(1);
    issue_ze(0, live);
    issue_y(0, 0, 0, live);
    issue_x(0, 0, live);
    if (w == 0) factors(0, lg2[0], live);
    // the tiles above the diagonal that 32-deep products reach
    if (threadIdx.x < 128) {
      const int t = threadIdx.x >> 6, row = 32 * t + (l >> 2), p = 2 * (2 * t + 1) + (l & 1);
      reinterpret_cast<uint2*>(sm + M::P + (row * PP + (p ^ key<PP>(row))) * 16)[(l >> 1) & 1] = make_uint2(0, 0);
    }
  }
  // ---- start states (behind the first tiles' loads), element (channel c of Dv, column k of Dk) at k Dv + c
#pragma unroll
  for (int q = 0; q < GH; ++q) {
    const size_t hs = static_cast<size_t>(Dk) * Dv, bh = static_cast<size_t>(b) * Hv + h0 + q;
    const float* src = nseg > 1 ? (rev ? a.R : a.S) + (static_cast<size_t>(sg) * a.d.B * Hv + bh) * hs
                                : (rev ? a.dS : a.state0);
    if (nseg == 1 && src) src += bh * hs;
    const rsrc_t rs = make_rsrc(src, src ? hs * 4 : 0);
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      const int ch = 32 * (i / 2) + 8 * g + 4 * (i % 2);
      const float4 v = buf_f4(rs, ch < Dv && col < Dk ? 4u * static_cast<uint32_t>(col * Dv + ch) : kOff);
      S[q][i] = f32x4{v.x, v.y, v.z, v.w};
      if constexpr (DQ) E[q][i] = f4zero();
    }
    grad[q] = 0.0;
  }
  for (int ci = 0; ci < nch; ++ci) {
    const int t0 = chunk_start(ci), L = __popcll(live);
    f32x4 acc[MT], pu[DQ ? TP : 1];
    uint2 ev[DQ ? MT : 1];
    uint4 zu[2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f4zero();
#pragma unroll
    for (int q = 0; q < GH; ++q) {
      const int set = GH % 2 == 0 ? q & 1 : (ci * GH + q) & 1;
      const uint32_t ytile = M::Y + set * M::XB;
      const float *fc = reinterpret_cast<const float*>(sm + M::F) + set * 4 * CH, *frf = fc + CH, *fsw = fc + 2 * CH;
      // (the stores of the last chunk's results are asked for behind the loads)
      if (q == 0 && ci > 0) wait_vm<MT>();
      else wait_vm<0>();
      lds_barrier();
      opaque(rx);
      opaque(ty[0]);
      opaque(ty[1]);
      if (q == 0 && ci + 1 < nch) {
        live_next = live_of(ci + 1, byte_next);
        byte_next = mask_byte(ci + 2);
      }
      const bool more = q + 1 < GH || ci + 1 < nch;
      const int cn = q + 1 < GH ? ci : ci + 1;
      constexpr int kLast = GH - 1;
      const int qn = q == kLast ? 0 : q + 1;
      const unsigned long long ln = q == kLast ? live_next : live;
      if (more) {
        issue_y(cn, qn, set ^ 1, ln);
        if (w == 3) factors(set ^ 1, lg2[qn], ln);
      }

      // ---- what the heads share: e . z tiles, e at the results' places, z
      if (q == 0) {
        if constexpr (DQ) {
#pragma unroll
          for (int k = 0; k < TP; ++k) {
            int mt, nt;
            pu[k] = f4zero();
            if (tile_of(k, mt, nt)) {
#pragma unroll
              for (int ks = 0; ks < 2; ++ks)
                pu[k] = mfma16(load_bf16x8(sm + M::Z + rz[ks] + nt * 16 * PZ * 16),
                               load_bf16x8(sm + M::E + rz[ks] + mt * 16 * PZ * 16), pu[k]);
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int row = 16 * mt + lr, p = 2 * w + (g >> 1);
            ev[mt] = reinterpret_cast<const uint2*>(sm + M::E + (row * PZ + (p ^ key<PZ>(lr))) * 16)[g & 1];
          }
        }
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          const uint2 z0 = lds_read_tr16(sm + M::Z + kt * 32 * PZ * 16 + tz[0]);
          const uint2 z1 = lds_read_tr16(sm + M::Z + kt * 32 * PZ * 16 + tz[1]);
          zu[kt] = make_uint4(z0.x, z0.y, z1.x, z1.y);
        }
      }

      // ---- P, transposed tiles
      float intra = 0.f;
#pragma unroll
      for (int k = 0; k < TP; ++k) {
        int mt, nt;
        if (!tile_of(k, mt, nt)) continue;
        f32x4 t = f4zero();
        const uint32_t py = ytile + nt * 16 * PX * 16, px = M::X + mt * 16 * PX * 16;
#pragma unroll
        for (int ks = 0; ks < KD / 32; ++ks) t = mfma16(load_bf16x8(sm + (py + at_x(0, ks))), load_bf16x8(sm + (px + at_x(0, ks))), t);
        const float c_i = fc[16 * mt + lr];
        const f32x4 c_j = *reinterpret_cast<const f32x4*>(fc + 16 * nt + 4 * g);
        float dn[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          dn[r] = c_i - c_j[r];
          t[r] *= exp2_fast(lg2[q] * dn[r]) * scale_p;
        }
        if (nt == mt) {
#pragma unroll
          for (int r = 0; r < 4; ++r) t[r] = 4 * g + r <= lr ? t[r] : 0.f;
        }
        if constexpr (DQ) {
#pragma unroll
          for (int r = 0; r < 4; ++r) intra = fmaf(dn[r] * t[r], nt < mt || 4 * g + r <= lr ? pu[k][r] : 0.f, intra);
        }
        reinterpret_cast<uint2*>(sm + M::P + ((16 * mt + lr) * PP + ((2 * nt + (g >> 1)) ^ key<PP>(lr))) * 16)[g & 1] =
            pack4_bf16(t[0], t[1], t[2], t[3]);
      }
      // ---- S^T x into the sum over the heads, and with E^T x against e
      f32x4 ai[MT], ae[DQ ? MT : 1];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        ai[mt] = f4zero();
        if constexpr (DQ) ae[mt] = f4zero();
      }
      auto operand = [](const f32x4& s, const f32x4& t, bf16x8 (&part)[SP]) {
        float v[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = s[r];
          v[4 + r] = t[r];
        }
        split8<SP>(v, part);
      };
#pragma unroll
      for (int ks = 0; ks < KD / 32; ++ks) {
        bf16x8 xa[MT], part[SP];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) xa[mt] = load_bf16x8(sm + M::X + at_x(mt, ks));
        operand(S[q][2 * ks], S[q][2 * ks + 1], part);
#pragma unroll
        for (int s = 0; s < SP; ++s)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) ai[mt] = mfma16(part[s], xa[mt], ai[mt]);
        if constexpr (DQ) {
          operand(E[q][2 * ks], E[q][2 * ks + 1], part);
#pragma unroll
          for (int s = 0; s < SP; ++s)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) ae[mt] = mfma16(part[s], xa[mt], ae[mt]);
        }
      }
      float sum = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float rf = frf[16 * mt + lr];
        if constexpr (DQ) {
          const float ct = fc[16 * mt + lr];
          const float e[4] = {__uint_as_float(ev[mt].x << 16), __uint_as_float(ev[mt].x & 0xffff0000u),
                              __uint_as_float(ev[mt].y << 16), __uint_as_float(ev[mt].y & 0xffff0000u)};
          float f = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) f = fmaf(fmaf(ct, ai[mt][r], ae[mt][r]), e[r], f);
          sum = fmaf(rf, f, sum);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[mt][r] = fmaf(ai[mt][r], rf, acc[mt][r]);
      }
      if constexpr (DQ) grad[q] += static_cast<double>(sum) + static_cast<double>(intra);
      lds_barrier();  // P is whole; x, and by the first head z and e, are read
      if (more) issue_x(cn, qn, ln);
      if (q == 0 && ci + 1 < nch) issue_ze(ci + 1, live_next);

      // ---- the state's update, and P z
      const float gL = exp2_fast(lg2[q] * static_cast<float>(L));
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (DQ) E[q][i][r] = gL * fmaf(static_cast<float>(L), S[q][i][r], E[q][i][r]);
          S[q][i][r] *= gL;
        }
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        constexpr int YH = DQ ? 2 : 4;  // y tiles held at a time
        bf16x8 part[SU], pe[DQ ? SU : 1], ya[YH];
        auto weighted = [&](const float* f, bf16x8 (&p)[SU]) {
          float sw[8], v[8];
          *reinterpret_cast<f32x4*>(sw) = *reinterpret_cast<const f32x4*>(f + 32 * kt + 8 * g);
          *reinterpret_cast<f32x4*>(sw + 4) = *reinterpret_cast<const f32x4*>(f + 32 * kt + 8 * g + 4);
          Vec16<bf16>::unpack(zu[kt], v);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] *= sw[k];
          split8<SU>(v, p);
        };
        weighted(fsw, part);
        if constexpr (DQ) weighted(fsw + CH, pe);
#pragma unroll
        for (int i0 = 0; i0 < KT; i0 += YH) {
#pragma unroll
          for (int i = 0; i < YH; ++i) {
            const int ks = (i0 + i) / 2;
            const uint32_t yt = ytile + kt * 32 * PX * 16 + (ks / QX) * QX * 64 + (i & 1) * 8;
            const uint2 y0 = lds_read_tr16(sm + (yt + (ty[0] ^ (ks % QX * 64u))));
            const uint2 y1 = lds_read_tr16(sm + (yt + (ty[1] ^ (ks % QX * 64u))));
            ya[i] = as_bf16x8(make_uint4(y0.x, y0.y, y1.x, y1.y));
          }
#pragma unroll
          for (int s = 0; s < SU; ++s)
#pragma unroll
            for (int i = 0; i < YH; ++i) {
              S[q][i0 + i] = mfma16(ya[i], part[s], S[q][i0 + i]);
              if constexpr (DQ) E[q][i0 + i] = mfma16(ya[i], pe[s], E[q][i0 + i]);
            }
        }
#pragma unroll
        for (int mt = 2 * kt; mt < MT; ++mt)
          acc[mt] = mfma16(as_bf16x8(zu[kt]),
                           load_bf16x8(sm + M::P + ((16 * mt + lr) * PP + ((4 * kt + g) ^ key<PP>(lr))) * 16), acc[mt]);
      }
    }

    // ---- rows of the chunk: dq / dk, or this part of the heads in fp32
    {
      const int es = parts > 1 ? 4 : 2, H = Hk * parts, c = cb + 16 * w + 4 * g;
      char* base = parts > 1 ? reinterpret_cast<char*>(rev ? a.pk : a.pq) : static_cast<char*>(rev ? a.dk : a.dq);
      const rsrc_t rw = make_rsrc(base + ((bT + t0) * H + hp) * Dk * es,
                                  (static_cast<size_t>(min(Tn - t0, CH) - 1) * H * Dk + Dk) * es);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = 16 * mt + lr;
        if (masked && rev && !((live >> row) & 1)) acc[mt] = f4zero();  // a masked step's, whatever its factors are
        const uint32_t o = c < Dk ? (static_cast<uint32_t>(rev ? CH - 1 - row : row) * H * Dk + c) * es : kOff;
        if (es == 4) buf_store_u4(rw, o, __builtin_bit_cast(uint4, acc[mt]));
        else buf_store_u2(rw, o, pack4_bf16(acc[mt][0], acc[mt][1], acc[mt][2], acc[mt][3]));
      }
    }
    live = live_next;
  }
  wait_vm<0>();  // no load to LDS outlives the workgroup
  if constexpr (DQ) {  // the derivative of the state behind the segment, against the loss's
#pragma unroll
    for (int q = 0; q < GH; ++q) {
      const size_t hs = static_cast<size_t>(Dk) * Dv, bh = static_cast<size_t>(b) * Hv + h0 + q;
      const float* R = nseg > 1 ? a.R + (static_cast<size_t>(sg) * a.d.B * Hv + bh) * hs : a.dS ? a.dS + bh * hs : nullptr;
      const rsrc_t rc = make_rsrc(R, R ? hs * 4 : 0);
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const int ch = 32 * (i / 2) + 8 * g + 4 * (i % 2);
        const float4 v = buf_f4(rc, ch < Dv && col < Dk ? 4u * static_cast<uint32_t>(col * Dv + ch) : kOff);
        grad[q] += static_cast<double>(fmaf(E[q][i][3], v.w, fmaf(E[q][i][2], v.z, fmaf(E[q][i][1], v.y, E[q][i][0] * v.x))));
      }
      const double t = wave_sum_f64_dpp(grad[q]);
      if (l == 0) a.grad[(bh * nseg + sg) * (4 * ncb) + (cb >> 4) + w] = t;
    }
  }
}

// Both directions in one launch, the longer walks (dq) first, so that dk's fill the
// compute units that dq's last round leaves idle.  At 16 key heads of 192, 64 value
// heads of 128 and 2048 steps: 172 to 189 us, one after the other 126 + 70 us.
template <int KD, int GH>
__global__ void __launch_bounds__(256, KD <= 128 ? 2 : 1) keys_kernel(DecayKeysArgs a, int n_dq) {
  __shared__ __attribute__((aligned(16))) char sm[KeysLds<KD>::TOTAL];
  const int block = blockIdx.x;
  if (block < n_dq) keys_walk<KD, 1, true>(a, block, sm);
  else keys_walk<KD, GH, false>(a, block - n_dq, sm);
}

template <int KD> hipError_t launch_keys(const DecayKeysArgs& a, hipStream_t st) {
  const int gh = decay_heads_together(a.d.G());
  const auto blocks = [&](int heads) { return (a.d.B * a.nseg * (a.d.Hv / heads) * ((a.d.Dk + 63) / 64) + 7) / 8 * 8; };
  const int n = blocks(1), grid = n + blocks(gh);
  if (gh == 2) keys_kernel<KD, 2><<<grid, 256, 0, st>>>(a, n);
  else keys_kernel<KD, 1><<<grid, 256, 0, st>>>(a, n);
  return hipGetLastError();
}

}  // namespace decay
}  // namespace gdn
