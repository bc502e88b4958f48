// The attention of gdn_prefix_attn.hip for many rows (bf16): the four waves of a
// workgroup, 32 rows each, share every tile of keys, so that a key that was brought to
// LDS serves 128 rows.
//
// 32x32x16 products: scores transposed, keys by rows, so that a lane holds sixteen
// keys of one query.  In the product with the values the order in which keys take the
// places of the inner index is free as long as both operands agree: the weights are
// taken as the scores' product left them (places 8 (e / 4) + 4 half + e % 4), and the
// values' transposing reads follow, so no weight changes its lane.
//
// A 32x32x16 product takes 32 cycles of a SIMD and one operand of 1 KB from LDS, 4
// cycles of the compute unit's one LDS: four SIMDs busy with products alone would keep
// the LDS busy for half of the time.  What bounds the kernel is the issue of
// instructions: two waves to a SIMD, each of which starts one in about four cycles, have
// reads, exponentials, packing and waits to start beside each product.  Measured: 16
// prompts of 20 to 290 tokens over 8192 shared keys, 32 heads of 128 on 8 key heads, 404
// us of this kernel, 850 TFLOP/s (a large product of matrices reaches 1233 here), the
// matrix units busy 46% of the time and the LDS 25%; 64 single tokens over 32768 shared
// keys, 16 heads of 256 on 2, 54 us, 640 TFLOP/s, 35% and 22%.
#include "gdn_prefix_attn.h"

#include <type_traits>

namespace gdn {
namespace attn {
namespace {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;

constexpr float kLarge = 1048576.f;  // references beyond this do not hold the lift in fp32

template <int DC> struct Many {
  static constexpr int W = 4, PR = DC / 8;                  // waves; pieces of 16 bytes of a row
  static constexpr int BN = DC <= 128 ? 64 : 32;            // keys of a tile
  static constexpr int XN = BN / 32;                        // blocks of 32 keys of a tile
  static constexpr int TILE = BN * PR * 16;                 // bytes of a tile of keys or values
  static constexpr int ST = 2;                              // tiles in LDS
  static constexpr int RW = BN / W;                         // rows that a wave loads
  static constexpr int NL = TILE / 1024 / W;                // load instructions of a wave for a tile
  static constexpr int AHEAD_K = DC == 64 ? 4 : DC == 128 ? 8 : DC == 192 ? 4 : 3;  // operands read ahead: what
  static constexpr int AHEAD_V = DC == 64 ? 4 : DC == 128 ? 4 : DC == 192 ? 3 : 2;  // registers are there for
  static constexpr int STAGE = 32 * 68 * 4;                 // a wave's 64 channels of its rows
  static constexpr int PAGES = 2 * TILE * ST > W * STAGE ? 2 * TILE * ST : W * STAGE, LDS = PAGES + W * 256;
  static_assert(NL * 1024 * W == TILE && LDS <= 80 * 1024, "whole loads, two workgroups to a compute unit");
};

__device__ __forceinline__ f32x16 mfma32(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Reads at an LDS address and a constant number of bytes from it.
__device__ __forceinline__ bf16x8 read16(uint32_t at, int off) {
  typedef __attribute__((address_space(3))) const bf16x8 lds_t;
  return *reinterpret_cast<lds_t*>(at + off);
}
__device__ __forceinline__ uint2 read_tr(uint32_t at, int off) {
  typedef __attribute__((address_space(3))) i16x4 lds_t;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_t*>(at + off)));
}

// Has the compiler read the operands (READS to a product) of AHEAD products before the
// first of N, and then each product's AHEAD ahead: left to itself it reads each operand
// when it is wanted, and every product of the chain waits for the LDS.
template <int N, int READS, int AHEAD> __device__ __forceinline__ void operands_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, READS * AHEAD, READS);  // LDS reads
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, READS);  // products
    __builtin_amdgcn_sched_group_barrier(0x100, READS, READS);
  }
  __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, READS);
}

template <int DC> __global__ void __launch_bounds__(256, 2) many_kernel(AttnArgs a) {
  using F = Many<DC>;
  constexpr int PR = F::PR, ST = F::ST, NL = F::NL, RW = F::RW, BN = F::BN, XN = F::XN, NQ = DC / 16, ND = DC / 32;
  __shared__ __align__(256) char lds[F::LDS];
  auto swz = [](int row) { return swizzle<PR, 4>(row); };
  constexpr int SW = PR % 16 == 0 ? 16 : 8;  // pieces among which the swizzle moves one
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, lr = l & 31, half = l >> 5;
  const Item it = find_item(a);
  if (it.empty) return;
  const int cnt = it.k1 > it.k0 ? (it.k1 - it.k0 + BN - 1) / BN : 0;  // tiles
  const uint32_t lds_at = lds_of(lds);

  const int G = a.G, nrows = it.n * G, row_w = it.row0 + 32 * w, row = row_w + lr;
  const bool on = row < nrows && !it.bad;
  const int lim = it.seen + row / G;                                  // keys that the row sees,
  const int lim_first = it.seen + row_w / G;                          // and the wave's first row
  bf16x8 q[NQ];
  {
    const int r = on ? row : it.row0;
    const bf16* src = static_cast<const bf16*>(a.q) + (static_cast<int64_t>(it.t0 + (it.bad ? 0 : r / G)) * a.Hq + it.hk * G + r % G) * a.D;
#pragma unroll
    for (int st = 0; st < NQ; ++st) {
      const int c = 16 * st + 8 * half;
      q[st] = load_bf16x8(src + (c < a.D ? c : 0));
      if (!on || c >= a.D || a.scale == 0.f) q[st] = zero8();
    }
  }
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -__builtin_inff(), sum = 0.f;

  const char *kb = static_cast<const char*>(a.kp) + it.hk * a.pool.hs, *vb = static_cast<const char*>(a.vp) + it.hk * a.pool.hs;
  const int in_page = (1 << a.pool.shift) - 1;
  const int lw = w * RW + l % RW;  // the row of a tile whose page this lane knows
  const int32_t* pages = reinterpret_cast<const int32_t*>(lds + F::PAGES) + w * 64;
  auto load_page = [&](int t) {
    load_lds4(it.list + (min(it.k0 + BN * min(t, cnt - 1) + lw, it.k1 - 1) >> a.pool.shift), lds_at + F::PAGES + w * 256);
  };
  // The rows that a wave loads of a full tile lie in one page where pages hold them all:
  // one address for the wave, and each lane's constant distance from it.  Channels that
  // there are not are not loaded (their places hold zeros from the start).
  const bool one_page = (1 << a.pool.shift) >= RW && a.pool.ts < (1 << 19);
  // At 256 channels, whose sums and queries fill the registers, the distances are worked
  // out each time from the first load's: held, some of them lay in scratch memory, and
  // reading one back waited for all loads under way (64 single tokens over 32768 shared
  // keys: 112 us, worked out 59; at 128 channels 16 prompts over 8192 keys take 410 us
  // with them held, 436 worked out).  76 bytes a lane lie there still at 256 channels.
  constexpr int RL = 64 / PR;  // whole rows of a load
  constexpr bool WHOLE = DC == 256;
  const int place = ((l % PR) ^ swz(w * RW + l / PR)) * 16, first_at = l / PR * a.pool.ts, step = RL * a.pool.ts;
  uint32_t from_first[WHOLE ? 1 : NL];
  if constexpr (!WHOLE) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = (i * 64 + l) / PR;
      from_first[i] = r * static_cast<uint32_t>(a.pool.ts) + (((i * 64 + l) % PR) ^ swz(w * RW + r)) * 16;
    }
  }
  auto load_tile = [&](int t) {
    const int page = pages[l];
    int place_ = place, first_ = first_at;
    if constexpr (WHOLE) asm volatile("" : "+v"(place_), "+v"(first_));  // (not before the loop)
    const uint32_t to = lds_at + (t & (ST - 1)) * 2 * F::TILE + w * NL * 1024;
    const int key_w = it.k0 + BN * t + w * RW, page_w = __builtin_amdgcn_readfirstlane(page);
    if (one_page && key_w + RW <= it.k1 && page_w >= 0 && page_w < a.pool.pages) {
      const int64_t off = page_w * a.pool.ps + static_cast<uint32_t>((key_w & in_page) * static_cast<uint32_t>(a.pool.ts));
      const char *kr = kb + off, *vr = vb + off;
      auto rows = [&](auto whole) {
#pragma unroll
        for (int x = 0; x < 2 * NL; ++x) {
          const int i = x % NL;
          const uint32_t into = to + x / NL * F::TILE + i * 1024;
          if constexpr (WHOLE) {
            const int at = place_ ^ (swz(i * RL) * 16);
            if (whole || at < a.D * 2) load_lds16(x < NL ? kr : vr, at + first_ + i * step, into);
          } else {
            const int piece = ((i * 64 + l) % PR) ^ swz(w * RW + (i * 64 + l) / PR);
            if (whole || piece * 16 < a.D * 2) load_lds16(x < NL ? kr : vr, from_first[i], into);
          }
        }
      };
      if (a.D == DC) rows(std::true_type{});
      else rows(std::false_type{});
      return;
    }
    const int key = key_w + l % RW;
    int64_t off = page * a.pool.ps + (key & in_page) * a.pool.ts;
    if (page < 0 || page >= a.pool.pages) off = -2;
    if (key >= it.k1) off = -1;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = (i * 64 + l) / PR;
      const int at = WHOLE ? place_ ^ (swz(i * RL) * 16) : (((i * 64 + l) % PR) ^ swz(w * RW + r)) * 16;
      const int64_t from = (static_cast<int64_t>(__shfl(static_cast<int>(off >> 32), r)) << 32) |
                           static_cast<uint32_t>(__shfl(static_cast<int>(off), r));
      const bool fill = from < 0 || at >= a.D * 2;
      const void* none = &kFill[from == -2 ? 1 : 0];
      load_lds16(fill ? none : kb + (from + at), to + i * 1024);
      load_lds16(fill ? none : vb + (from + at), to + F::TILE + i * 1024);
    }
  };

  // Where the products' operands lie in a tile.  A piece further along a row is its
  // number XORed into the address below the swizzle's range, and a constant beyond it.
  uint32_t ka, va[2];
  {
    const int sl = l & 15, r = 4 * half + (sl >> 2), col = 2 * ((l >> 4) & 1) + ((sl & 3) >> 1);
    ka = lds_at + lr * PR * 16 + (half ^ swz(lr)) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) va[i] = lds_at + F::TILE + (r + 8 * i) * PR * 16 + (col ^ swz(r + 8 * i)) * 16 + (sl & 1) * 8;
  }

  // A block's products of queries and keys; what the scale makes -inf for keys that the
  // row does not see.  (With a scale of 0 the queries were taken as zeros.)
  const float scale = a.scale == 0.f ? 1.f : a.scale, hide = scale < 0.f ? __builtin_inff() : -__builtin_inff();
  const int every = min(it.k1, lim_first);  // keys that all rows of the wave see
  auto products = [&](uint32_t at, int key0, f32x16& s) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
    uint32_t k_at = ka + at;
    asm volatile("" : "+v"(k_at));  // (not taken apart: the constants would be held in registers)
#pragma unroll
    for (int st = 0; st < NQ; ++st) s = mfma32(read16(k_at ^ (2 * st % SW * 16), 2 * st / SW * SW * 16), q[st], s);
    operands_ahead<NQ, 1, F::AHEAD_K>();
    if (key0 + 32 > every) {
      const int see = min(it.k1, lim) - key0 - 4 * half;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + i % 4 < see ? s[i] : hide;
    }
  };
  // A block's weights, in place, and their sum (before they are rounded: lse is the
  // statistics' in 32 bits).  ref is m + lift, which m is chosen to have exactly.
  float ref = 0.f;
  bool large = false, wide = false;
  auto weights = [&](f32x16& s, bool all_small) {
    if (all_small) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], scale, -ref));
    } else {
      // Of scores as large as this the product with the scale, in one step with the
      // difference, may exceed the reference (which is rounded) by any amount: there
      // the product is rounded as well, and the lift, which the reference cannot hold
      // beside them, is a product of its own.
#pragma unroll
      for (int i = 0; i < 16; ++i) {
#pragma clang fp contract(off)
        const float y = s[i] * scale, d = fmaf(s[i], scale, -ref);
        s[i] = __builtin_amdgcn_exp2f(large ? y - ref : d) * (large ? a.unit : 1.f);
      }
    }
    return (((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]))) +
                       (((s[8] + s[9]) + (s[10] + s[11])) + ((s[12] + s[13]) + (s[14] + s[15])));
  };
  // A block with the reference as it is; false, and nothing changed, where its weights
  // exceed their bound (which a block that is `sure` is not asked).
  const float most = kMost * a.unit;
  auto block = [&](uint32_t at, int key0, bool sure) {
    f32x16 s;
    products(at, key0, s);
    const float part = weights(s, !wide);
    if (!sure && __any(part > most)) return false;
    sum += part;
    // (the weights rounded to bf16, for which the matrix cores take values of bf16 as they
    // lie: up to 2^-8 of each weight, where fp32 products would take eight times as long)
    bf16x8 p[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      p[j] = as_bf16x8(make_uint4(pack2_bf16(s[8 * j], s[8 * j + 1]), pack2_bf16(s[8 * j + 2], s[8 * j + 3]),
                                  pack2_bf16(s[8 * j + 4], s[8 * j + 5]), pack2_bf16(s[8 * j + 6], s[8 * j + 7])));
    uint32_t v0_at = va[0] + at, v1_at = va[1] + at;
    asm volatile("" : "+v"(v0_at), "+v"(v1_at));
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int off = 4 * d / SW * SW * 16 + 16 * j * PR * 16;
        const uint2 v0 = read_tr(v0_at ^ (4 * d % SW * 16), off), v1 = read_tr(v1_at ^ (4 * d % SW * 16), off);
        o[d] = mfma32(as_bf16x8(make_uint4(v0.x, v0.y, v1.x, v1.y)), p[j], o[d]);
      }
    operands_ahead<NQ, 2, F::AHEAD_V>();
    return true;
  };

  if (cnt > 0) {
    if (a.D != DC) {  // the places of channels that there are not
      for (int i = threadIdx.x; i < 2 * F::TILE * ST / 16; i += 256) reinterpret_cast<uint4*>(lds)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    load_page(0);
    wait_vm<0>();
    load_tile(0);
    load_page(1);
    int t = -1, x = 0;
    auto next_tile = [&]() {
      ++t;
      // this wave's part of tile t has come; behind the barrier everyone's has, and
      // everyone is done with tile t - 1, whose place tile t + 1 takes
      wait_vm<0>();
      lds_barrier();
      if (t + 1 < cnt) {
        load_tile(t + 1);
        load_page(t + 2);
      }
    };
    next_tile();
#pragma unroll 1
    while (true) {
      // The reference is moved to the block's maximum: at the first block, and where the
      // weights exceed their bound.  Outside the loop over the tiles, so that in it the
      // result stays in its registers (scaled under a condition there, or with a way
      // round the products, it was held, and copied, twice).
      bool again;
      {
        f32x16 s;
        products((t & (ST - 1)) * 2 * F::TILE + x * 32 * PR * 16, it.k0 + BN * t + 32 * x, s);
        float top = s[0] * scale;
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i] * scale);
        // (only of the rows that ask for it, by the very sum that `block` asks for: a row's
        // bits are its own, whatever lies beside it)
        const float part = weights(s, false);  // (the same bits)
        const bool need = (part > most) | (__shfl_xor(part, 32) > most) | (m == -__builtin_inff());
        top = fmaxf(top, __shfl_xor(top, 32));
        if (fabsf(top) <= kLarge) top = (top + a.lift) - a.lift;
        const float to = need ? fmaxf(top, m) : m, f = to == m ? 1.f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        sum *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= f;
        large = fabsf(m) > kLarge && m != -__builtin_inff();
        ref = m == -__builtin_inff() ? 0.f : large ? m : m + a.lift;
        wide = __any(large);
        // a row that has seen no key yet: its first sets the reference (one whose scores are
        // NaN has a NaN sum, and nothing to wait for: it had its wave go this way for every
        // block, queries of NaN behind the last sequence among them: 4 prompts of 1500 tokens in
        // 2048 rows over 8192 shared keys, 32 heads of 128 on 8, 428 us, now 295)
        again = __any(m == -__builtin_inff() && sum == sum);
      }
      // that block (which is not tried twice, whatever it holds), and the tile's others
      bool ok = true, sure = true;
#pragma unroll 1
      do {
        ok = block((t & (ST - 1)) * 2 * F::TILE + x * 32 * PR * 16, it.k0 + BN * t + 32 * x, sure);
        sure = false;
        x += ok ? 1 : 0;
      } while (ok && !again && x < XN);
      if (x < XN) continue;
      x = 0;
      // whole tiles
#pragma unroll 1
      while (!again && ok && t + 1 < cnt) {
        next_tile();
        const uint32_t at = (t & (ST - 1)) * 2 * F::TILE;
        const int key0 = it.k0 + BN * t;
        ok = block(at, key0, false);
        if (XN == 1 || !ok) continue;
        ok = block(at + 32 * PR * 16, key0 + 32, false);
        x = ok ? 0 : 1;
      }
      if (ok) {
        if (t + 1 >= cnt) break;
        next_tile();  // (again)
      }
    }
  }

  // The waves of a row's keys join, then rows go out 64 channels at a time through LDS,
  // whole lines of them.
  sum += __shfl_xor(sum, 32);
  const float inv = it.bad ? __builtin_nanf("") : sum == 0.f ? 0.f : 1.f / sum;
  const bool first = half == 0 && row < nrows;
  const int64_t out_row = static_cast<int64_t>(it.t0 + row / G) * a.Hq + it.hk * G + row % G;
  if (a.together) {
    if (first && a.lse) a.lse[out_row] = it.bad ? inv : (m + log2f(sum * a.whole)) * kLn2;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] *= inv;
  } else if (first) {
    a.ml[static_cast<int64_t>(it.slot) * a.N * a.Hq + out_row] = make_float2(m, sum);
  }
  float* mine = reinterpret_cast<float*>(lds + w * F::STAGE);
  __syncthreads();  // (the ring is read no more)
#pragma unroll
  for (int c = 0; c < ND / 2; ++c) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const f32x16& z = o[2 * c + x / 4];
      *reinterpret_cast<float4*>(mine + lr * 68 + 32 * (x / 4) + 8 * (x & 3) + 4 * half) =
          make_float4(z[4 * (x & 3)], z[4 * (x & 3) + 1], z[4 * (x & 3) + 2], z[4 * (x & 3) + 3]);
    }
    wave_lds_sync();
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int r = 4 * x + (l >> 4), ch = 64 * c + 4 * (l & 15), gr = row_w + r;
      const float4 y = *reinterpret_cast<const float4*>(mine + r * 68 + 4 * (l & 15));
      if (gr >= nrows || ch >= a.D) continue;
      const int64_t to = static_cast<int64_t>(it.t0 + gr / G) * a.Hq + it.hk * G + gr % G;
      if (a.together) *reinterpret_cast<uint2*>(static_cast<bf16*>(a.o) + to * a.D + ch) = pack4_bf16(y.x, y.y, y.z, y.w);
      else *reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(it.slot) * a.N * a.Hq + to) * a.D + ch) = y;
    }
    wave_lds_sync();
  }
  if (a.together) bad_rows<bf16>(a, it, nrows, 256);
}

template <int DC> hipError_t launch(const AttnArgs& a, unsigned items, hipStream_t st) {
  many_kernel<DC><<<items, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_many(const AttnArgs& a, unsigned items, hipStream_t st) {
  if (a.D <= 64) return launch<64>(a, items, st);
  if (a.D <= 128) return launch<128>(a, items, st);
  if (a.D <= 192) return launch<192>(a, items, st);
  return launch<256>(a, items, st);
}

}  // namespace attn
}  // namespace gdn
