// The walk kernel of the decay operator (see DecayWalk in gdn_decay.h).
//
// A workgroup owns one segment of one (batch, value head) and goes through its
// chunks of CH steps with the whole state beside it: wave w holds columns
// 16 NTL w .. of all KD channels, fp32, in the accumulator layout of the matrix
// cores.  These are registers for the narrower heads; the wider classes keep a part
// in scratch (see below).  With c_i the valid steps of the chunk up to step i
// (counted in walk order; up to and with i forward in time, before i backward), L
// its valid steps, and g = e^lg:
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
//     the state keeps fp32 precision; two parts (16 bits) where only bf16 results
//     are read from this state;
//   - the state against x: one bf16 part, as the result is rounded to bf16 (a
//     relative error of at most 2^-8 for each product, independent between the
//     products);
//   - P: one bf16 part, as the result is rounded to bf16.
//
// dlg (DOTS; the fp32 dq walk, whose e is q).  The loss's derivative in lg, taken
// forward: beside the state goes its derivative since the segment's start, E = dS /
// d lg,
//   E <- g^L (E + L S) + sum_j y_j ((L - c_j) g^(L - c_j) z_j)^T,
// and with the segment's share of the loss in what it reads,
//   dlg += sum_i g^c_i e_i . (c_i S + E)^T x_i + sum_ij (c_i - c_j) P_ij (e_i . z_j),
// in the final state or later segments' reading through R, the loss's derivative in
// the state behind the segment: dlg += <E, R>.  All of these are sums of products
// with the distances as weights.  (From dq and dk the same sum would follow as
// sum_i n_i q_i . dq_i - sum_j n_j k_j . dk_j, a difference of terms up to T times
// larger: chunk by chunk that was off by 5e-4 in single heads, this by 1e-7.)
//
// Tiles go to LDS by direct loads into a second set, where two sets fit, while the
// chunk's own are used; x and e, which are read first, into their only set otherwise
// as soon as they are.  With two sets of all, loads stand between the products one
// at a time: asked for in a row they hold up every wave, as a compute unit takes
// one (1 KB) in about 25 cycles; and the only product that needs the other waves'
// P comes last, behind the state's update.  The descriptors end behind the sequence's last row of the chunk and masked
// or padding pieces get an offset past them, so all of these read as zeros.
// Results in bf16 go to LDS and from there to memory a chunk later, as whole
// rows: a wave's own columns would be 32 bytes of a row at a time, which costs the
// memory pipeline four times the cycles.
//
// Measured, bf16: 64 value heads of 192 x 128, 2048 steps in 4 segments of 8 chunks
// (one workgroup of 8 waves to a compute unit): the sums 24 us, the output walks 45
// to 52 us, with 101 MB of rows 1.4 TB/s together.  4 heads of 128 x 128, 32768 steps
// in 64 segments: 20 and 33 us, 1.6 TB/s with the chain's 10 us.  A chunk costs 1.4 us
// as a sum and 2.3 us as outputs (128 x 128), a launch with its first tiles and its
// states' way in and out 9 to 15 us.  Of a walk's cycles matrix products take 29%,
// vector instructions 34%, LDS reads 39%: the bound is their order inside a chunk (P
// before P z, the old state before the new one, barriers between), with too few
// registers for a second workgroup beside the state.
//
// One workgroup takes all columns of a head, whatever KD is, so wide heads do not
// fit the registers.  Scratch of the output walks, bytes a lane, by classes KD x N:
//   bf16          128 x 192 / 256   32 / 84;   192 x 192 / 256   84 / 384;
//                 256 x 128 / 192 / 256   16 / 344 / 1168
//   fp32          128 x 192 / 256  100 / 160;  192 x 128 / 192 / 256   120 / 552 / 976;
//                 256 x 128 / 192 / 256  272 / 736 / 1504
//   fp32 dq, dk   64 x 192 / 256   180 / 300;  128 x 128 / 192 / 256   88 / 576 / 1056;
//                 192 x 128 / 192 / 256  668 / 1328 / 2424;  256 x 128 / 192 / 256
//                 1016 / 1864 / 3284
// (fp32 sums of 192 x 192 and wider 48 to 120; all else none.)  What it costs: 32 heads,
// 2048 steps, forward and backward in us, 128 x 128, 192 x 192 and 256 x 256: bf16 49 and
// 125, 86 and 288, 355 and 518; fp32 104 and 296, 403 and 1652, 760 and 3172, where
// the products alone are 4 times those of 128 x 128.
//
// The decay of a chunk, g^L, is one fp32 number, and its rounding is the same for
// every full chunk, or every call of L steps: a state that remembers n steps is off by
// n / L times 2^-24 of it at most (1e-5 at lg = -1e-4 for chunks of 64, where the
// roundings of its sums come to 1e-6).
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

template <int N> struct Int {
  static constexpr int v = N;
};

template <typename T> struct Cfg;
template <> struct Cfg<bf16> {
  static constexpr int CH = 64, EPP = 8;
};
template <> struct Cfg<float> {
  static constexpr int CH = 32, EPP = 4;
};

// Place of piece p of row r in a tile's row of PPR pieces: p ^ key(r).  LDS serves
// 256 bytes (16 pieces) a cycle from 64 banks, over all 64 lanes of a read (measured:
// a read takes as many cycles as distinct rows meet on its busiest bank).  With
// these keys 16 rows' pieces of one number lie on all 16 places: a 16-byte read of 16
// rows by 4 pieces takes 4 cycles, the least.  (Rows of 8 or 24 pieces start on the
// other half of the places in turn, which stands for the key's fourth bit.)  A
// transposing read of four neighbouring half pieces of 16 rows takes 4 cycles (2 if
// it took lower and upper halves in turn, but then x had to be read in the same
// order, eight bytes at a time, and put together again).
template <int PPR> __device__ __forceinline__ int key(int r) {
  return PPR % 16 == 0 ? ((r & 1) << 3) | ((r >> 1) & 7) : (r >> 1) & 7;
}

constexpr uint32_t kOff = 0x80000000u;  // an offset past every descriptor here

// LDS, in bytes: tiles of y and z and of x and e (one or two sets each), P, the
// results to store, and the chunk's per-step factors (two sets).  Tiles are row-major
// 16-byte pieces, piece p of row r at place p ^ key(r).
template <typename T, int KD, int NW, int NTL, bool OUT, bool DOTS>
struct Lds {
  static constexpr int CH = Cfg<T>::CH, EPP = Cfg<T>::EPP, MAX = 160 * 1024;
  static constexpr int COLS = 16 * NW * NTL, NF = DOTS ? 4 : 3;
  static constexpr int PX = KD / EPP, PZ = COLS / EPP, PP = CH / EPP;  // pieces per row
  static constexpr int XB = CH * PX * 16, ZB = CH * PZ * 16;
  static constexpr int SET = XB + ZB, Y = 0, Z = XB;
  static constexpr int XE = (OUT ? XB : 0) + (DOTS ? ZB : 0);
  static constexpr int REST = (OUT ? CH * PP * 16 : 0) + 2 * NF * CH * 4;
  static constexpr int SLOTS = 2 * SET + XE + REST <= MAX ? 2 : 1;
  static constexpr bool STAGE = OUT && sizeof(T) == 2 && SLOTS * SET + XE + REST + ZB <= MAX;
  static constexpr bool XE2 = OUT && SLOTS == 2 && 2 * (SET + XE) + REST + (STAGE ? ZB : 0) <= MAX;
  static constexpr int X = SLOTS * SET, E = X + XB, P = X + (XE2 ? 2 : 1) * XE, O = P + (OUT ? CH * PP * 16 : 0);
  static constexpr int F = O + (STAGE ? ZB : 0), TOTAL = F + 2 * NF * CH * 4;
};

// dma16 to an LDS address; and for a place that nothing reads before the next
// barrier, without the clobber that would keep LDS reads from moving past it.
__device__ __forceinline__ void dma16_to(const i32x4& r, uint32_t lds, uint32_t off) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(r), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void dma16_ahead(const i32x4& r, uint32_t lds, uint32_t off) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(r), "{m0}"(lds));
}

// Loads of one tile by this wave: 64 pieces at a time.
template <int CH, int PPR, int EPP, int NW> struct Loader {
  static constexpr int N = CH * PPR / 64, PER = (N + NW - 1) / NW;
  uint32_t off[PER];
  // row_bytes: from one step's row to the next; D: channels in a row
  __device__ __forceinline__ void init(int w, int l, uint32_t row_bytes, int D, bool rev) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int s = (k * NW + w) * 64 + l, r = s / PPR, p = (s % PPR) ^ key<PPR>(r);
      off[k] = p * EPP < D ? (rev ? CH - 1 - r : r) * row_bytes + p * 16 : kOff;
    }
  }
  // where rows whose bit in live is clear read as zeros
  __device__ __forceinline__ uint32_t live_off(int k, int w, int l, unsigned long long live) const {
    const int r = ((k * NW + w) * 64 + l) / PPR;
    return (live >> r) & 1 ? off[k] : kOff;
  }
  // dst: the tile's LDS address
  __device__ __forceinline__ void load(const i32x4& desc, uint32_t dst, int w, int l) const {
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (N % NW == 0 || k * NW + w < N) dma16_to(desc, dst + (k * NW + w) * 1024, off[k]);
  }
  __device__ __forceinline__ void load_live(const i32x4& desc, uint32_t dst, int w, int l, unsigned long long live) const {
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (N % NW == 0 || k * NW + w < N) dma16_to(desc, dst + (k * NW + w) * 1024, live_off(k, w, l, live));
  }
};

// Workgroup `block` of walk wk; SPU: bf16 parts of the weighted z that the state sums.
template <typename T, int KD, int NW, int NTL, bool OUT, bool DOTS, int SPU>
__device__ __forceinline__ void walk(const DecayWalkArgs& a, const DecayWalk& wk, int block, char* sm) {
  using M = Lds<T, KD, NW, NTL, OUT, DOTS>;
  constexpr bool BF = sizeof(T) == 2;
  static_assert(!(BF && DOTS), "bf16 dq rows come from keys_kernel");
  constexpr int CH = M::CH, EPP = M::EPP, PX = M::PX, PZ = M::PZ, PP = M::PP, MT = CH / 16, KT = KD / 16;
  const int Hv = a.d.Hv, Tn = a.d.T, BH = a.d.B * Hv, nseg = a.nseg, n_items = BH * nseg;
  const int it = xcd_order(block, n_items);
  if (it >= n_items) return;
  // value heads fastest: the heads of a group run side by side
  const int h = it % Hv, sg = (it / Hv) % nseg, b = it / (Hv * nseg), bh = b * Hv + h;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, lr = l & 15, g = l >> 4;
  const bool rev = wk.reverse != 0;
  const int N = wk.N, KDr = wk.KD;
  const size_t bT = static_cast<size_t>(b) * Tn;
  const uint8_t* mrow = a.mask ? a.mask + bT : nullptr;
  const float lg2 = log2_decay(a.lg[h]);
  const float scale_p = wk.scale_p, scale_i = wk.scale_i, scale_u = wk.scale_u;

  // state tile (i, n), register r of lane (lr, g): channel 32 (i/2) + 8 g + 4
  // (i%2) + r for bf16 (two tiles together then are an operand of a 32-deep
  // product as they stand), 16 i + 4 g + r for fp32.  Column of place idx of
  // tile n: two tiles together hold runs of eight columns for each g.
  auto chan = [&](int i) { return BF ? 32 * (i / 2) + 8 * g + 4 * (i % 2) : 16 * i + 4 * g; };
  const int col0 = 16 * NTL * w;
  auto column = [&](int n, int idx) {
    return n < NTL / 2 * 2 ? col0 + 32 * (n / 2) + 8 * (idx >> 2) + 4 * (n & 1) + (idx & 3) : col0 + 16 * n + idx;
  };
  const size_t hs = static_cast<size_t>(a.d.Dk) * a.d.Dv;
  const uint32_t hbytes = static_cast<uint32_t>(hs * 4);
  const int sr = wk.sr, sc = wk.sc;
  auto state_off = [&](int i, int n) {
    const int ch = chan(i), col = column(n, lr);
    return ch < KDr && col < N ? 4u * static_cast<uint32_t>(ch * sr + col * sc) : kOff;
  };

  // Segment sums that only walks of this kind read lie in the order of the
  // registers: [KT NTL tiles][wave][lane][4].
  const size_t native = static_cast<size_t>(KT) * NTL * NW * 256;
  auto native_of = [&](int s) {
    return wk.seg_sum + (static_cast<size_t>(s) * BH + bh) * native + (w * 64 + l) * 4;
  };
  f32x4 S[KT][NTL], E[DOTS ? KT : 1][NTL];
  double grad = 0.0;  // this lane's part of dlg
  const float* src = nullptr;
  const bool prefix = OUT && wk.seg_sum != nullptr;  // starts from the sums before it
  if (OUT) {
    if (wk.seg_start) src = wk.seg_start + (static_cast<size_t>(sg) * BH + bh) * hs;
    else if (wk.start) src = wk.start + bh * hs;
  }
  auto load_start = [&]() {
    const rsrc_t rs = make_rsrc(src, src ? hbytes : 0);
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < NTL; ++n) {
        const uint32_t o = state_off(i, n);
        if (sr == 1) {
          const float4 v = buf_f4(rs, o);
          S[i][n] = f32x4{v.x, v.y, v.z, v.w};
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) S[i][n][r] = buf_f1(rs, o + 4u * static_cast<uint32_t>(r * sr));
        }
      }
  };
  auto store_state = [&](float* dst) {
    const rsrc_t rd = make_rsrc(dst, hbytes);
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < NTL; ++n) {
        const uint32_t o = state_off(i, n);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][n][r]), rd, o + 4u * static_cast<uint32_t>(r * sr), 0, 0);
      }
  };
  // S <- (S g^N0 + U0) g^N1 + U1 ... over the first `count` sums, in walk order
  // (forward); two sums' loads are in flight at a time
  auto add_sums = [&](int count) {
    for (int s = 0; s < count; s += 2) {
      f32x4 U[2][KT][NTL];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (s + q < count) {
          const float* u = native_of(s + q);
#pragma unroll
          for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int n = 0; n < NTL; ++n)
              U[q][i][n] = *reinterpret_cast<const f32x4*>(u + static_cast<size_t>(i * NTL + n) * NW * 256);
        }
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (s + q < count) {
          const float f = exp2_fast(lg2 * wk.seg_steps[b * nseg + s + q]);
#pragma unroll
          for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int n = 0; n < NTL; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) S[i][n][r] = fmaf(f, S[i][n][r], U[q][i][n][r]);
        }
    }
  };

  const int t_lo = sg * a.seg * kDecayChunk, t_hi = min(Tn, t_lo + a.seg * kDecayChunk);
  const int nch = t_hi > t_lo ? (t_hi - t_lo + CH - 1) / CH : 0;
  // (sums go through the chunks from the walk's end, so that the steps behind a
  // chunk are counted when its weights are made and the state needs no decay)
  auto chunk_start = [&](int ci) { return t_lo + (rev == OUT ? nch - 1 - ci : ci) * CH; };
  // the mask byte of this lane's step of a chunk (walk order; any where there is
  // no such step), and the live steps
  auto mask_byte = [&](int ci) -> int {
    if (mrow == nullptr || ci >= nch) return 1;
    const int t = chunk_start(ci) + (rev ? CH - 1 - l : l);
    return mrow[max(0, min(t, Tn - 1))];
  };
  auto live_of = [&](int ci, int byte) -> unsigned long long {
    const int t = chunk_start(ci) + (rev ? CH - 1 - l : l);
    return __ballot(l < CH && t < Tn && byte != 0);
  };

  const int xH = wk.x.H, xg = wk.x.group, yH = wk.y.H, yg = wk.y.group, zH = wk.z.H, zg = wk.z.group;
  Loader<CH, PX, EPP, NW> ly;
  Loader<CH, PZ, EPP, NW> lz;
  ly.init(w, l, static_cast<uint32_t>(yH) * KDr * sizeof(T), KDr, rev);
  lz.init(w, l, static_cast<uint32_t>(zH) * N * sizeof(T), N, rev);
  // a chunk's rows of one head: from its first step to the sequence's end
  // (all of this is the same in every lane, so the words stay in scalar registers)
  auto rows = [&](const void* p, int H, int head, int D, int t0) {
    const int n = min(Tn - t0, CH);
    const uint64_t at = reinterpret_cast<uint64_t>(static_cast<const T*>(p) + ((bT + t0) * H + head) * D);
    return i32x4{static_cast<int>(at), static_cast<int>(at >> 32) & 0xffff,
                 ((n - 1) * H * D + D) * static_cast<int>(sizeof(T)), 0x00020000};
  };
  const int xh = h / xg, yh = h / yg, zh = h / zg;
  const bool masked = mrow != nullptr;
  const uint32_t lds0 = lds_addr(sm);
  auto issue_yz = [&](int ci, int slot, unsigned long long live) {
    const uint32_t s = lds0 + slot * M::SET;
    const int t0 = chunk_start(ci);
    const i32x4 dy = rows(wk.y.p, yH, yh, KDr, t0), dz = rows(wk.z.p, zH, zh, N, t0);
    if (masked && !rev) {
      ly.load_live(dy, s + M::Y, w, l, live);
      lz.load_live(dz, s + M::Z, w, l, live);
    } else {
      ly.load(dy, s + M::Y, w, l);
      lz.load(dz, s + M::Z, w, l);
    }
  };
  auto issue_xe = [&](int ci, int slot, unsigned long long live) {  // x has y's row length, e has z's
    const uint32_t s = lds0 + (M::XE2 ? slot * M::XE : 0);
    const int t0 = chunk_start(ci);
    if constexpr (OUT) {
      const i32x4 dx = rows(wk.x.p, xH, xh, KDr, t0);
      if (masked && rev) ly.load_live(dx, s + M::X, w, l, live);
      else ly.load(dx, s + M::X, w, l);
    }
    if constexpr (DOTS) {
      const i32x4 de = rows(wk.e.p, zH, zh, N, t0);
      if (masked && rev) lz.load_live(de, s + M::E, w, l, live);
      else lz.load(de, s + M::E, w, l);
    }
  };
  // results of a chunk: rows behind the sequence and columns past N lie past the
  // descriptor
  constexpr int es = sizeof(T);
  auto out_rows = [&](int t0) {
    return make_rsrc(static_cast<char*>(wk.w) + ((bT + t0) * Hv + h) * N * es,
                     (static_cast<size_t>(min(Tn - t0, CH) - 1) * Hv * N + N) * es);
  };
  auto store_staged = [&](int ci) {
    if constexpr (M::STAGE) {
      const rsrc_t rw = out_rows(chunk_start(ci));
      constexpr int NS = CH * PZ / 64;
#pragma unroll
      for (int k = 0; k < (NS + NW - 1) / NW; ++k) {
        if (NS % NW != 0 && k * NW + w >= NS) continue;
        const int s = (k * NW + w) * 64 + l, r = s / PZ, p = s % PZ;
        const uint4 v = *reinterpret_cast<const uint4*>(sm + M::O + (r * PZ + (p ^ key<PZ>(r))) * 16);
        buf_store_u4(rw, p * 8 < N ? (static_cast<uint32_t>(rev ? CH - 1 - r : r) * Hv * N + p * 8) * 2u : kOff, v);
      }
    }
  };

  // byte offsets of this lane's operand pieces in a tile: row lr (a 16-row tile
  // further is a constant further), piece 4 ks + g for ks = 0 .. 3 (0, 1 where
  // keys have three bits; further ks are a constant further)
  constexpr int QX = PX % 16 == 0 ? 4 : 2, QZ = PZ % 16 == 0 ? 4 : 2;
  uint32_t rx[QX], rz[QZ];
#pragma unroll
  for (int q = 0; q < QX; ++q) rx[q] = static_cast<uint32_t>(lr * PX + ((4 * q + g) ^ key<PX>(lr))) * 16u;
#pragma unroll
  for (int q = 0; q < QZ; ++q) rz[q] = static_cast<uint32_t>(lr * PZ + ((4 * q + g) ^ key<PZ>(lr))) * 16u;
  auto at_x = [&](int tile, int ks) { return rx[ks % QX] + tile * 16 * PX * 16 + (ks / QX) * QX * 64; };
  auto at_z = [&](int tile, int ks) { return rz[ks % QZ] + tile * 16 * PZ * 16 + (ks / QZ) * QZ * 64; };
  // transposing reads (bf16): lane (lr, g) addresses row 8 g + lr/4 (+ 4 for the
  // second half), and of two 16-channel tiles together piece lr%4, half i%2
  const int tr = 8 * g + (lr >> 2);
  uint32_t ty[QX][2], tz[NTL][2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = tr + 4 * q;
#pragma unroll
    for (int e = 0; e < QX; ++e)
      ty[e][q] = static_cast<uint32_t>(row * PX + ((4 * e + (lr & 3)) ^ key<PX>(row))) * 16u;
#pragma unroll
    for (int n = 0; n < NTL; ++n) {
      const int c = column(n, 4 * (lr & 3));  // four columns from here
      tz[n][q] = static_cast<uint32_t>(row * PZ + ((c >> 3) ^ key<PZ>(row))) * 16u + (c & 4) * 2;
    }
  }

  unsigned long long live = 0, live_next = 0;
  int counted = 0;  // valid steps of the segment
  // a chunk's c, row factors, source weights, and these times the steps left
  auto factors = [&](int ci, unsigned long long live, int behind) {
    if (l >= CH) return;
    float* f = reinterpret_cast<float*>(sm + M::F) + (ci & 1) * M::NF * CH + l;
    const float c = static_cast<float>(__popcll(live & (((rev ? 1ull : 2ull) << l) - 1ull)));
    f[0] = c;
    f[CH] = scale_i * exp2_fast(lg2 * c);
    const float left = static_cast<float>(behind + __popcll(live)) - c;
    f[2 * CH] = scale_u * exp2_fast(lg2 * left);
    if constexpr (DOTS) f[3 * CH] = left * f[2 * CH];
  };
  // loads that stand between products: those of a set that every wave takes an
  // equal share of
  constexpr bool SPREAD = M::XE2 && !DOTS && decltype(ly)::N % NW == 0 && decltype(lz)::N % NW == 0;
  constexpr int NY = decltype(ly)::PER, NZ = decltype(lz)::PER;
  int byte_next = 1;
  if (nch > 0) {
    live = live_of(0, mask_byte(0));
    byte_next = mask_byte(1);
    if (w == 0) factors(0, live, 0);
    if constexpr (M::SLOTS == 2) issue_yz(0, 0, live);
    issue_xe(0, 0, live);
  }
  // (the state's loads behind those of the first tiles)
  if constexpr (OUT) {
    load_start();
    if constexpr (!DOTS)
      if (prefix) add_sums(sg);
    if constexpr (DOTS) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int n = 0; n < NTL; ++n) E[i][n] = f4zero();
    }
  } else {
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < NTL; ++n) S[i][n] = f4zero();
  }
  for (int ci = 0; ci < nch; ++ci) {
    const int t0 = chunk_start(ci), slot = M::SLOTS == 2 ? ci & 1 : 0;
    const bool more = ci + 1 < nch;
    char* tile = sm + slot * M::SET;
    char* xe = sm + (M::XE2 ? slot * M::XE : 0);
    const float* fc = reinterpret_cast<const float*>(sm + M::F) + (ci & 1) * M::NF * CH;
    const float *frf = fc + CH, *fsw = fc + 2 * CH;
    if constexpr (M::SLOTS == 1) {
      lds_barrier();  // the chunk before is read
      issue_yz(ci, 0, live);
    }
    const int L = __popcll(live);
    counted += L;
    // this wave's part of the tiles has arrived (what it stored after asking for
    // them, MT stores at least, may be on the way still)
    if (OUT && M::SLOTS == 2 && !M::STAGE && ci > 0) wait_vm<MT>();
    else wait_vm<0>();
    lds_barrier();
    if (more) {
      live_next = live_of(ci + 1, byte_next);
      byte_next = mask_byte(ci + 2);
      if (w == NW - 1) factors(ci + 1, live_next, OUT ? 0 : counted);
    }
    i32x4 dny, dnz, dnx;
    uint32_t ony[NY], onz[NZ], onx[NY];
    if constexpr (SPREAD) {
      const int tn = chunk_start(more ? ci + 1 : ci);
      dny = rows(wk.y.p, yH, yh, KDr, tn);
      dnz = rows(wk.z.p, zH, zh, N, tn);
      dnx = rows(wk.x.p, xH, xh, KDr, tn);
      if (!more) dny[2] = dnz[2] = dnx[2] = 0;  // (nothing is read)
#pragma unroll
      for (int k = 0; k < NY; ++k) ony[k] = onx[k] = ly.off[k];
#pragma unroll
      for (int k = 0; k < NZ; ++k) onz[k] = lz.off[k];
      if (masked) {
#pragma unroll
        for (int k = 0; k < NY; ++k) {
          const uint32_t o = ly.live_off(k, w, l, live_next);
          ony[k] = rev ? ony[k] : o;
          onx[k] = rev ? o : onx[k];
        }
#pragma unroll
        for (int k = 0; k < NZ; ++k) onz[k] = rev ? onz[k] : lz.live_off(k, w, l, live_next);
      }
    } else if (more) {
      if constexpr (M::SLOTS == 2) issue_yz(ci + 1, slot ^ 1, live_next);
      if constexpr (M::XE2) issue_xe(ci + 1, slot ^ 1, live_next);
    }
    const uint32_t next_tile = lds0 + (slot ^ 1) * M::SET, next_xe = lds0 + (slot ^ 1) * M::XE;
    auto spread_yz = [&](int k) {
      if constexpr (SPREAD) {
        if (k < NY) dma16_ahead(dny, next_tile + M::Y + (k * NW + w) * 1024, ony[k < NY ? k : 0]);
        else if (k < NY + NZ)
          dma16_ahead(dnz, next_tile + M::Z + ((k - NY) * NW + w) * 1024, onz[k < NY + NZ && k >= NY ? k - NY : 0]);
      }
    };
    auto spread_x = [&](int k) {
      if constexpr (SPREAD)
        if (k < NY) dma16_ahead(dnx, next_xe + M::X + (k * NW + w) * 1024, onx[k < NY ? k : 0]);
    };
    if (M::STAGE && ci > 0) store_staged(ci - 1);

    f32x4 acc[MT][NTL];
    if constexpr (OUT) {
      // ---- P, transposed tiles (rows j, columns i).  Needed are the lower ones
      // and, for 32-deep products with z, those up to the next even tile: runs of
      // TW tiles of one row, one run to a wave at a time.
      float intra = 0.f;
      constexpr int TW = BF && NW < 12 ? 2 : 1, RUNS = BF ? 12 / TW : 3;
      f32x4 pt[TW], pu[TW];
      auto run_rows = [&](int run, int& mt, int& nt0) {
        if constexpr (!BF) {
          mt = run > 0;
          nt0 = run - mt;
        } else if constexpr (TW == 2) {
          mt = run < 2 ? run : 1 + run / 2;
          nt0 = run < 2 ? 0 : 2 * (run & 1);
        } else {
          mt = run < 4 ? run >> 1 : 2 + ((run - 4) >> 2);
          nt0 = run < 4 ? run & 1 : (run - 4) & 3;
        }
      };
      auto p_products = [&](int run) {
        int mt, nt0;
        run_rows(run, mt, nt0);
#pragma unroll
        for (int q = 0; q < TW; ++q) pt[q] = pu[q] = f4zero();
        const char *py = tile + M::Y + nt0 * 16 * PX * 16, *px = xe + M::X + mt * 16 * PX * 16;
        const char *pz = tile + M::Z + nt0 * 16 * PZ * 16, *pe = xe + M::E + mt * 16 * PZ * 16;
        if constexpr (BF) {
#pragma unroll
          for (int ks = 0; ks < KD / 32; ++ks) {
            const bf16x8 xa = load_bf16x8(px + at_x(0, ks));
#pragma unroll
            for (int q = 0; q < TW; ++q) pt[q] = mfma16(load_bf16x8(py + at_x(q, ks)), xa, pt[q]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KD / 16; ++ks) {
            const f32x4 yv = *reinterpret_cast<const f32x4*>(py + at_x(0, ks));
            const f32x4 xv = *reinterpret_cast<const f32x4*>(px + at_x(0, ks));
#pragma unroll
            for (int r = 0; r < 4; ++r) pt[0] = mfma16f(yv[r], xv[r], pt[0]);
          }
          if constexpr (DOTS) {
#pragma unroll
            for (int ks = 0; ks < M::COLS / 16; ++ks) {
              const f32x4 zv = *reinterpret_cast<const f32x4*>(pz + at_z(0, ks));
              const f32x4 ev = *reinterpret_cast<const f32x4*>(pe + at_z(0, ks));
#pragma unroll
              for (int r = 0; r < 4; ++r) pu[0] = mfma16f(zv[r], ev[r], pu[0]);
            }
          }
        }
      };
      auto p_write = [&](int run, bool mine) {
        int mt, nt0;
        run_rows(run, mt, nt0);
        const float c_i = fc[16 * mt + lr];
        char* pp = sm + M::P + (16 * mt + lr) * PP * 16;
#pragma unroll
        for (int q = 0; q < TW; ++q) {
          const int nt = nt0 + q;
          const f32x4 c_j = *reinterpret_cast<const f32x4*>(fc + 16 * nt + 4 * g);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float dn = c_i - c_j[r];
            const bool in = 16 * nt + 4 * g + r <= 16 * mt + lr;
            pt[q][r] = in ? pt[q][r] * exp2_fast(lg2 * dn) * scale_p : 0.f;
            if constexpr (DOTS) intra += in ? dn * pt[q][r] * pu[q][r] : 0.f;
          }
          if (!mine) continue;
          if constexpr (BF)
            *reinterpret_cast<uint2*>(pp + (((2 * nt + (g >> 1)) ^ key<PP>(lr)) * 16 + (g & 1) * 8)) =
                pack4_bf16(pt[q][0], pt[q][1], pt[q][2], pt[q][3]);
          else
            *reinterpret_cast<f32x4*>(pp + ((4 * nt + g) ^ key<PP>(lr)) * 16) = pt[q];
        }
      };
      // Where there is a wave for every run, P's products go ahead of those with
      // the state and the rest of its making behind them, in one stretch of code
      // (a wave without a run repeats the last one's products).
      constexpr bool ONE = BF && NW >= RUNS;
      if constexpr (ONE) {
        p_products(min(w, RUNS - 1));
      } else {
        for (int run = w; run < RUNS; run += NW) {
          p_products(run);
          p_write(run, true);
        }
      }
      // ---- S^T x, transposed tiles (rows are columns of w, columns are steps)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < NTL; ++n) acc[mt][n] = f4zero();
      f32x4 ae[DOTS ? MT : 1][NTL];
      if constexpr (DOTS) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < NTL; ++n) ae[mt][n] = f4zero();
      }
      if constexpr (BF) {
#pragma unroll
        for (int ks = 0; ks < KD / 32; ++ks) {
          bf16x8 xa[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) xa[mt] = load_bf16x8(xe + M::X + at_x(mt, ks));
          spread_yz(ks);
#pragma unroll
          for (int n = 0; n < NTL; ++n) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              v[r] = S[2 * ks][n][r];
              v[4 + r] = S[2 * ks + 1][n][r];
            }
            bf16x8 part[1];
            split8<1>(v, part);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[mt][n] = mfma16(part[0], xa[mt], acc[mt][n]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const f32x4 xv = *reinterpret_cast<const f32x4*>(xe + M::X + at_x(mt, i));
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int n = 0; n < NTL; ++n) {
                acc[mt][n] = mfma16f(S[i][n][r], xv[r], acc[mt][n]);
                if constexpr (DOTS) ae[mt][n] = mfma16f(E[i][n][r], xv[r], ae[mt][n]);
              }
          }
      }
#pragma unroll
      for (int k = BF ? KD / 32 : 0; k < NY + NZ; ++k) spread_yz(k);
      if constexpr (ONE) p_write(min(w, RUNS - 1), w < RUNS);
      float s = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float rf = frf[16 * mt + lr], ct = fc[16 * mt + lr];
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          if constexpr (DOTS) {
            const int c = column(n, 4 * g), row = 16 * mt + lr;  // four columns from here
            const f32x4 ev = *reinterpret_cast<const f32x4*>(xe + M::E + (row * PZ + ((c >> 2) ^ key<PZ>(lr))) * 16);
            float f = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) f = fmaf(fmaf(ct, acc[mt][n][r], ae[mt][n][r]), ev[r], f);
            s = fmaf(rf, f, s);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[mt][n][r] *= rf;
        }
      }
      if constexpr (DOTS) grad += static_cast<double>(s) + static_cast<double>(intra);
    }
    if constexpr (OUT && !M::XE2) {
      lds_barrier();  // P is whole, x and e are read
      if (more) issue_xe(ci + 1, 0, live_next);
    }

    // ---- the state's update
    const float gL = OUT ? exp2_fast(lg2 * static_cast<float>(L)) : 1.f;
    if constexpr (OUT && BF) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int n = 0; n < NTL; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[i][n][r] *= gL;
    }
    uint4 zu[BF ? CH / 32 : 1][NTL];  // z as operands
    float zv[BF ? 1 : CH / 16][NTL][4];
    if constexpr (BF) {
      constexpr int YH = NW >= 12 ? 4 : KT > 8 ? KT / 2 : KT;  // y tiles held at a time
#pragma unroll
      for (int kt = 0; kt < CH / 32; ++kt) {
        // y's reads ahead of the splitting of z; then products on different state
        // tiles in turn
        bf16x8 zp[NTL][SPU], ya[YH];
        auto load_y = [&](int i) {
          const int ks = i / 2;
          const char* yt = tile + M::Y + kt * 32 * PX * 16 + (ks / QX) * QX * 64 + (i & 1) * 8;
          const uint2 y0 = lds_read_tr16(yt + ty[ks % QX][0]);
          const uint2 y1 = lds_read_tr16(yt + ty[ks % QX][1]);
          return as_bf16x8(make_uint4(y0.x, y0.y, y1.x, y1.y));
        };
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          const char* zt = tile + M::Z + kt * 32 * PZ * 16;
          const uint2 z0 = lds_read_tr16(zt + tz[n][0]), z1 = lds_read_tr16(zt + tz[n][1]);
          zu[kt][n] = make_uint4(z0.x, z0.y, z1.x, z1.y);
        }
        float sw[8];
        *reinterpret_cast<f32x4*>(sw) = *reinterpret_cast<const f32x4*>(fsw + 32 * kt + 8 * g);
        *reinterpret_cast<f32x4*>(sw + 4) = *reinterpret_cast<const f32x4*>(fsw + 32 * kt + 8 * g + 4);
#pragma unroll
        for (int i = 0; i < YH; ++i) ya[i] = load_y(i);
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          float v[8];
          Vec16<bf16>::unpack(zu[kt][n], v);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] *= sw[k];
          split8<SPU>(v, zp[n]);
        }
        spread_x(2 * kt);
#pragma unroll
        for (int i0 = 0; i0 < KT; i0 += YH) {
          if (i0 > 0) {
#pragma unroll
            for (int i = 0; i < YH; ++i) ya[i] = load_y(i0 + i);
          }
#pragma unroll
          for (int s = 0; s < SPU; ++s)
#pragma unroll
            for (int i = 0; i < YH; ++i)
#pragma unroll
              for (int n = 0; n < NTL; ++n) S[i0 + i][n] = mfma16(ya[i], zp[n][s], S[i0 + i][n]);
        }
        spread_x(2 * kt + 1);
      }
    } else {
      // The chunk's own sum is made from zero and added to the state once: added
      // product by product, every rounding would be one of the state's size, and
      // dlg, a sum of both signs over all states, was off by up to three times as much.
      float zs[CH / 16][NTL][4], ze[DOTS ? CH / 16 : 1][NTL][4];
#pragma unroll
      for (int bq = 0; bq < CH / 16; ++bq) {
        const f32x4 sw = *reinterpret_cast<const f32x4*>(fsw + 16 * bq + 4 * g);
        const f32x4 se = DOTS ? *reinterpret_cast<const f32x4*>(fsw + CH + 16 * bq + 4 * g) : f4zero();
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          const int c = column(n, lr);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * bq + 4 * g + r;
            zv[bq][n][r] =
                *reinterpret_cast<const float*>(tile + M::Z + (row * PZ + ((c >> 2) ^ key<PZ>(row))) * 16 + (c & 3) * 4);
            zs[bq][n][r] = zv[bq][n][r] * sw[r];
            if constexpr (DOTS) ze[bq][n][r] = zv[bq][n][r] * se[r];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        f32x4 U[NTL], UE[DOTS ? NTL : 1];
#pragma unroll
        for (int n = 0; n < NTL; ++n) {
          U[n] = f4zero();
          if constexpr (DOTS) UE[n] = f4zero();
        }
#pragma unroll
        for (int bq = 0; bq < CH / 16; ++bq)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * bq + 4 * g + r;
            const float yv = *reinterpret_cast<const float*>(
                tile + M::Y + (row * PX + ((4 * i + (lr >> 2)) ^ key<PX>(row))) * 16 + (lr & 3) * 4);
#pragma unroll
            for (int n = 0; n < NTL; ++n) {
              U[n] = mfma16f(yv, zs[bq][n][r], U[n]);
              if constexpr (DOTS) UE[n] = mfma16f(yv, ze[bq][n][r], UE[n]);
            }
          }
#pragma unroll
        for (int n = 0; n < NTL; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if constexpr (DOTS) E[i][n][r] = fmaf(gL, fmaf(static_cast<float>(L), S[i][n][r], E[i][n][r]), UE[n][r]);
            S[i][n][r] = OUT ? fmaf(gL, S[i][n][r], U[n][r]) : S[i][n][r] + U[n][r];
          }
      }
    }
#pragma unroll
    for (int k = BF ? 2 * (CH / 32) : 0; k < NY; ++k) spread_x(k);

    // ---- P z
    if constexpr (OUT) {
      if constexpr (M::XE2) lds_barrier();  // P is whole
      if constexpr (BF) {
#pragma unroll
        for (int kt = 0; kt < CH / 32; ++kt)
#pragma unroll
          for (int mt = 2 * kt; mt < MT; ++mt) {
            const bf16x8 pa = load_bf16x8(sm + M::P + ((16 * mt + lr) * PP + ((4 * kt + g) ^ key<PP>(lr))) * 16);
#pragma unroll
            for (int n = 0; n < NTL; ++n) acc[mt][n] = mfma16(as_bf16x8(zu[kt][n]), pa, acc[mt][n]);
          }
      } else {
#pragma unroll
        for (int bq = 0; bq < CH / 16; ++bq)
#pragma unroll
          for (int mt = bq; mt < MT; ++mt) {
            const f32x4 pv =
                *reinterpret_cast<const f32x4*>(sm + M::P + ((16 * mt + lr) * PP + ((4 * bq + g) ^ key<PP>(lr))) * 16);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int n = 0; n < NTL; ++n) acc[mt][n] = mfma16f(zv[bq][n][r], pv[r], acc[mt][n]);
          }
      }
    }

    if constexpr (OUT) {
      if (masked && rev) {  // masked steps give zeros, whatever their factors are
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < NTL; ++n)
            if (!((live >> (16 * mt + lr)) & 1)) acc[mt][n] = f4zero();
      }
      if constexpr (M::STAGE) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < NTL; ++n) {
            const int c = column(n, 4 * g), row = 16 * mt + lr;
            *reinterpret_cast<uint2*>(sm + M::O + (row * PZ + ((c >> 3) ^ key<PZ>(lr))) * 16 + (c & 4) * 2) =
                pack4_bf16(acc[mt][n][0], acc[mt][n][1], acc[mt][n][2], acc[mt][n][3]);
          }
      } else {
        const rsrc_t rw = out_rows(t0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int row = 16 * mt + lr;
          const uint32_t ro = static_cast<uint32_t>(rev ? CH - 1 - row : row) * static_cast<uint32_t>(Hv * N);
#pragma unroll
          for (int n = 0; n < NTL; ++n) {
            const int c = column(n, 4 * g);
            if constexpr (!BF) buf_store_u4(rw, c < N ? (ro + c) * 4u : kOff, __builtin_bit_cast(uint4, acc[mt][n]));
            else
              buf_store_u2(rw, c < N ? (ro + c) * 2u : kOff,
                           pack4_bf16(acc[mt][n][0], acc[mt][n][1], acc[mt][n][2], acc[mt][n][3]));
          }
        }
      }
    }
    live = live_next;
  }

  if (M::STAGE && nch > 0) {
    lds_barrier();
    store_staged(nch - 1);
  }
  wait_vm<0>();  // no load to LDS outlives the workgroup

  // ---- the state behind the segment
  float* dst = nullptr;
  if constexpr (OUT) {
    if (wk.end && !prefix) dst = wk.end + bh * hs;  // (one segment)
  } else {
    if (wk.seg_native) {
      float* o = native_of(sg);
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int n = 0; n < NTL; ++n)
          *reinterpret_cast<f32x4*>(o + static_cast<size_t>(i * NTL + n) * NW * 256) = S[i][n];
    } else {
      dst = wk.seg_sum + (static_cast<size_t>(sg) * BH + bh) * hs;
    }
    if (wk.seg_steps && h == 0 && threadIdx.x == 0) wk.seg_steps[b * nseg + sg] = static_cast<float>(counted);
  }
  if (dst) store_state(dst);
  if constexpr (OUT && !DOTS) {
    if (prefix && wk.end && sg == 0) {  // the final state, by the walk that had no sums to add
      load_start();
      add_sums(nseg);
      store_state(wk.end + bh * hs);
    }
  }
  if constexpr (DOTS) {
    const float* R = wk.seg_R ? wk.seg_R + (static_cast<size_t>(sg) * BH + bh) * hs : wk.R ? wk.R + bh * hs : nullptr;
    const rsrc_t rc = make_rsrc(R, R ? hbytes : 0);
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
      for (int n = 0; n < NTL; ++n) {
        const float4 v = buf_f4(rc, state_off(i, n));  // (sr is 1 in these walks)
        grad += static_cast<double>(fmaf(E[i][n][3], v.w, fmaf(E[i][n][2], v.z, fmaf(E[i][n][1], v.y, E[i][n][0] * v.x))));
      }
    grad = wave_sum_f64_dpp(grad);
    if (l == 0) wk.grad[(static_cast<size_t>(bh) * nseg + sg) * NW + w] = grad;
  }
}

template <typename T, int KD, int NW, int NTL, bool OUT, int SPU>
__global__ void __launch_bounds__(64 * NW) walk_kernel(DecayWalkArgs a) {
  __shared__ __attribute__((aligned(16))) char sm[Lds<T, KD, NW, NTL, OUT, false>::TOTAL];
  walk<T, KD, NW, NTL, OUT, false, SPU>(a, a.walk[blockIdx.y], blockIdx.x, sm);
}

// dq (walk 0) and dk of fp32 tensors in one launch, dq's longer walks first: a few
// heads' walks fill a part of the chip each (8 heads of 64 x 96, 515 steps, 72
// workgroups a walk: 20 us, one after the other 20 + 14 us).
template <int KD, int NW, int NTL> __global__ void __launch_bounds__(64 * NW) pair_kernel(DecayWalkArgs a) {
  // (dk's may be the larger one: two sets of its tiles fit where one of dq's does)
  constexpr int DQ = Lds<float, KD, NW, NTL, true, true>::TOTAL, DK = Lds<float, KD, NW, NTL, true, false>::TOTAL;
  __shared__ __attribute__((aligned(16))) char sm[DQ > DK ? DQ : DK];
  if (blockIdx.y == 0) walk<float, KD, NW, NTL, true, true, 3>(a, a.walk[0], blockIdx.x, sm);
  else walk<float, KD, NW, NTL, true, false, 3>(a, a.walk[1], blockIdx.x, sm);
}

template <typename T, int KD, int NW, int NTL>
hipError_t launch_nw(const DecayWalkArgs& a, hipStream_t st) {
  const int n = a.d.B * a.d.Hv * a.nseg;
  const dim3 grid((n + 7) / 8 * 8, a.nwalk);
  const DecayWalk& w = a.walk[0];
  constexpr int SPU = sizeof(T) == 2 ? 2 : 3;  // where only the tensors' type is read from the state
  if (w.e.p) {
    if constexpr (sizeof(T) == 4) pair_kernel<KD, NW, NTL><<<grid, 64 * NW, 0, st>>>(a);
    else return hipErrorInvalidValue;  // (keys_kernel's)
  } else if (w.end && !w.seg_sum) walk_kernel<T, KD, NW, NTL, true, 3><<<grid, 64 * NW, 0, st>>>(a);
  else walk_kernel<T, KD, NW, NTL, true, SPU><<<grid, 64 * NW, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int KD> hipError_t launch_kd(const DecayWalkArgs& a, hipStream_t st) {
  const int N = a.walk[0].N;
  if (N <= 64) return launch_nw<T, KD, 4, 1>(a, st);
  if (N <= 128) return launch_nw<T, KD, 8, 1>(a, st);
  if (N <= 192) return launch_nw<T, KD, 12, 1>(a, st);
  return launch_nw<T, KD, 8, 2>(a, st);
}

template <typename T, int KD> hipError_t launch_sum_kd(const DecayWalkArgs& a, hipStream_t st) {
  const int n = a.d.B * a.d.Hv * a.nseg, N = a.walk[0].N;
  const dim3 grid((n + 7) / 8 * 8, a.nwalk);
  auto go = [&](auto nw, auto ntl) {
    walk_kernel<T, KD, decltype(nw)::v, decltype(ntl)::v, false, 3><<<grid, 64 * decltype(nw)::v, 0, st>>>(a);
  };
  if (N <= 64) go(Int<4>{}, Int<1>{});
  else if (N <= 128) go(Int<8>{}, Int<1>{});
  else if (N <= 192) go(Int<12>{}, Int<1>{});
  else go(Int<8>{}, Int<2>{});
  return hipGetLastError();
}

}  // namespace decay

// One translation unit per (type, channel class): gdn_decay_walk_*.hip.
hipError_t decay_walk_bf16_64(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_bf16_64(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_bf16_128(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_bf16_128(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_bf16_192(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_bf16_192(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_bf16_256(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_bf16_256(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_64(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_f32_64(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_128(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_f32_128(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_192(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_f32_192(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_walk_f32_256(const DecayWalkArgs& a, hipStream_t st);
hipError_t decay_sum_f32_256(const DecayWalkArgs& a, hipStream_t st);

}  // namespace gdn
