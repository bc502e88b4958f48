// The attention of gdn_prefix_attn.hip for many rows (bf16): eight waves share each
// tile of 64 keys, so that a key that was brought to LDS serves 32 QW rows.
//
// QW waves of 32 rows each by KW waves that share out a tile's keys, 32 at a time.
// 32x32x16 products: scores transposed, keys by rows, so that a lane holds sixteen
// keys of one query.  In the product with the values the order in which keys take the
// places of the inner index is free as long as both operands agree: the weights are
// taken as the scores' product left them (places 8 (e / 4) + 4 half + e % 4), and the
// values' transposing reads follow, so no weight changes its lane.
//
// A 32x32x16 product takes 32 cycles of a SIMD and one operand of 1 KB from LDS, 8
// cycles of the compute unit's one LDS: with four SIMDs both are full at once.  Two
// waves on a SIMD let one's exponentials run beside the other's products.
#include "gdn_prefix_attn.h"

namespace gdn {
namespace attn {
namespace {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;

template <int DC, int QW, int KW> struct Many {
  static constexpr int W = QW * KW, BN = 64, PR = DC / 8;   // pieces of 16 bytes of a row
  static constexpr int TILE = BN * PR * 16;                 // bytes of a tile of keys or values
  static constexpr int ST = DC <= 128 ? 4 : DC == 192 ? 3 : 2;
  static constexpr int RW = BN / W;                         // rows that a wave loads
  static constexpr int NL = TILE / 1024 / W;                // load instructions of a wave for a tile
  static constexpr int TS = 2 * ST;                         // tiles whose pages are held
  static constexpr int STAGE = 32 * 68 * 4;                 // a wave's 64 channels of its rows
  static constexpr int RING = 2 * TILE * ST > W * STAGE ? 2 * TILE * ST : W * STAGE;
  static constexpr int LDS = RING + W * TS * RW * 4 + QW * KW * 32 * 8;
  static_assert(LDS <= 160 * 1024, "LDS");
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

template <int DC, int QW, int KW>
__global__ void __launch_bounds__(64 * QW * KW, 2) many_kernel(AttnArgs a) {
  using F = Many<DC, QW, KW>;
  constexpr int PR = F::PR, ST = F::ST, NL = F::NL, TS = F::TS, RW = F::RW, BN = F::BN, NQ = DC / 16, ND = DC / 32;
  __shared__ __align__(16) char lds[F::LDS];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, lr = l & 31, half = l >> 5;
  const int qw = w % QW, kw = w / QW;
  const Item it = find_item(a);
  if (it.empty) return;
  const int cnt = it.k1 > it.k0 ? (it.k1 - it.k0 + BN - 1) / BN : 0;  // tiles
  int32_t* pages = reinterpret_cast<int32_t*>(lds + F::RING) + w * TS * RW;
  const uint32_t lds_at = lds_of(lds), pages_at = lds_at + F::RING + w * TS * RW * 4;
  float2* stats = reinterpret_cast<float2*>(lds + F::RING + F::W * TS * RW * 4);

  const int G = a.G, nrows = it.n * G, row_w = it.row0 + 32 * qw, row = row_w + lr;
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
  const int in_page = (1 << a.pool.shift) - 1, lw = w * RW + (l % RW);
  auto page_of = [&](int t) {
    const int key = min(it.k0 + BN * (t < cnt ? t : cnt - 1) + lw, it.k1 - 1);
    return it.list + (key >> a.pool.shift);
  };
  // The rows that a wave loads of a full tile lie in one page where pages hold them all:
  // one address for the wave, and each lane's constant distance from it.
  const bool one_page = (1 << a.pool.shift) >= RW && a.D == DC && a.pool.ts < (1 << 26);
  uint32_t from_first[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int r = (i * 64 + l) / PR, piece = ((i * 64 + l) % PR) ^ swizzle(w * RW + r);
    from_first[i] = r * static_cast<uint32_t>(a.pool.ts) + piece * 16;
  }
  auto load_tile = [&](int t) {
    const int page = pages[(t % TS) * RW + l % RW];
    const uint32_t kt = lds_at + (t % ST) * 2 * F::TILE + w * NL * 1024;
    const int key_w = it.k0 + BN * t + w * RW, page_w = __builtin_amdgcn_readfirstlane(page);
    if (one_page && key_w + RW <= it.k1 && page_w >= 0 && page_w < a.pool.pages) {
      const int64_t off = page_w * a.pool.ps + (key_w & in_page) * a.pool.ts;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        load_lds16(kb + off, from_first[i], kt + i * 1024);
        load_lds16(vb + off, from_first[i], kt + F::TILE + i * 1024);
      }
      return;
    }
    const int key = key_w + l % RW;
    int64_t off = page * a.pool.ps + (key & in_page) * a.pool.ts;
    if (page < 0 || page >= a.pool.pages) off = -2;
    if (key >= it.k1) off = -1;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int r = (i * 64 + l) / PR, piece = ((i * 64 + l) % PR) ^ swizzle(w * RW + r);
      const int64_t from = (static_cast<int64_t>(__shfl(static_cast<int>(off >> 32), r)) << 32) |
                           static_cast<uint32_t>(__shfl(static_cast<int>(off), r));
      const bool fill = from < 0 || piece * 16 >= a.D * 2;
      const void* none = &kFill[from == -2 ? 1 : 0];
      load_lds16(fill ? none : kb + from + piece * 16, kt + i * 1024);
      load_lds16(fill ? none : vb + from + piece * 16, kt + F::TILE + i * 1024);
    }
  };
  auto load_pages = [&](int t) {
    if (l < RW) load_lds4(page_of(t), pages_at + (t % TS) * RW * 4);
  };

  // Where the products' operands lie in a tile: the swizzle moves a piece among the
  // eight of its 128 bytes, so channels 64 further (and rows 8 further) are a constant
  // number of bytes away.
  uint32_t ka[4], va[2];
  {
    const int sl = l & 15, r = 4 * half + (sl >> 2), col = 2 * ((l >> 4) & 1) + ((sl & 3) >> 1), x0 = KW == 2 ? 32 * kw : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) ka[i] = lds_at + ((x0 + lr) * PR + ((2 * i + half) ^ swizzle(lr))) * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) va[i] = lds_at + F::TILE + ((x0 + r) * PR + ((4 * i + col) ^ swizzle(r))) * 16 + (sl & 1) * 8;
  }

  if (cnt > 0) {
    if (l < RW)
      for (int t = 0; t < ST - 1; ++t) pages[t * RW + l] = *page_of(t);
    wave_lds_sync();
#pragma unroll 1
    for (int t = 0; t < ST - 1; ++t) {
      load_pages(t + ST - 1);
      if (t < cnt) load_tile(t);
    }
  }
  // The wave's blocks of 32 keys, one after the other.  Where it is: tile t, block x of
  // it, the block's first key, the bytes to its tile, and how many of its keys every row
  // of the wave sees.
  constexpr int XN = 2 / KW;
  int t = -1, x = XN - 1, key0 = 0, all_see = 0;
  uint32_t at = 0;
  auto next_block = [&]() {
    if (x + 1 < XN) {
      ++x;
      key0 += 32;
      all_see -= 32;
      at += 32 * PR * 16;
      return;
    }
    ++t;
    x = 0;
    // this wave's part of tile t has come; behind the barrier everyone's has, and
    // everyone is done with tile t - 1, whose place tile t + ST - 1 takes
    if (t + ST - 1 <= cnt) wait_vm<(ST - 2) * (2 * NL + 1)>();
    else wait_vm<0>();
    lds_barrier();
    if (t + ST - 1 < cnt) {
      load_pages(t + 2 * (ST - 1));
      load_tile(t + ST - 1);
    }
    at = (t % ST) * 2 * F::TILE;
    key0 = it.k0 + BN * t + (KW == 2 ? 32 * kw : 0);
    all_see = min(it.k1, lim_first) - key0;
  };
  // The block's products of queries and keys; what the scale makes -inf for keys that
  // the row does not see.  (With a scale of 0 the queries were taken as zeros.)
  const float scale = a.scale == 0.f ? 1.f : a.scale, hide = scale < 0.f ? __builtin_inff() : -__builtin_inff();
  auto products = [&](f32x16& s) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int st = 0; st < NQ; ++st) s = mfma32(read16(ka[st & 3] + at, (st >> 2) * 128), q[st], s);
    if (all_see < 32) {
      const int see = min(it.k1, lim) - key0 - 4 * half;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + i % 4 < see ? s[i] : hide;
    }
  };
  int left = cnt * XN;
  if (left > 0) next_block();
#pragma unroll 1
  while (left > 0) {
    // The reference is moved to the block's maximum: at the first block, and where the
    // weights exceed their bound.  Outside the loop over the blocks, so that in it the
    // result stays in its registers (scaled under a condition there, it was held, and
    // copied, twice).
    {
      f32x16 s;
      products(s);
      float top = s[0] * scale;
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i] * scale);
      top = fmaxf(top, __shfl_xor(top, 32));
      top = fmaxf(top, m);
      const float f = top == m ? 1.f : __builtin_amdgcn_exp2f(m - top);
      m = top;
      sum *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] *= f;
    }
    const float ref = m == -__builtin_inff() ? 0.f : m;
    const bool again = __any(m == -__builtin_inff());  // a row that has seen no key yet: its first sets the reference
#pragma unroll 1
    while (true) {
      f32x16 s;
      products(s);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], scale, -ref));
      // (the sum before the weights are rounded: lse is the statistics' in 32 bits)
      const float part = (((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]))) +
                         (((s[8] + s[9]) + (s[10] + s[11])) + ((s[12] + s[13]) + (s[14] + s[15])));
      if (__any(part > kMost)) break;
      sum += part;
      bf16x8 p[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        p[j] = as_bf16x8(make_uint4(pack2_bf16(s[8 * j], s[8 * j + 1]), pack2_bf16(s[8 * j + 2], s[8 * j + 3]),
                                    pack2_bf16(s[8 * j + 4], s[8 * j + 5]), pack2_bf16(s[8 * j + 6], s[8 * j + 7])));
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int off = (d >> 1) * 128 + 16 * j * PR * 16;
          const uint2 v0 = read_tr(va[d & 1] + at, off), v1 = read_tr(va[d & 1] + at, off + 8 * PR * 16);
          o[d] = mfma32(as_bf16x8(make_uint4(v0.x, v0.y, v1.x, v1.y)), p[j], o[d]);
        }
      if (--left == 0) break;
      next_block();
      if (again) break;
    }
  }

  // The waves of a row's keys join, then rows go out 64 channels at a time through LDS,
  // whole lines of them.
  sum += __shfl_xor(sum, 32);
  if constexpr (KW == 2) {
    if (half == 0) stats[(kw * QW + qw) * 32 + lr] = make_float2(m, sum);
    __syncthreads();
    const float2 other = stats[((1 - kw) * QW + qw) * 32 + lr];
    const float top = fmaxf(m, other.x), ref = top == -__builtin_inff() ? 0.f : top;
    const float f = __builtin_amdgcn_exp2f(m - ref);
    sum = f * sum + __builtin_amdgcn_exp2f(other.x - ref) * other.y;
    m = top;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] *= f;
  }
  const float inv = it.bad ? __builtin_nanf("") : sum == 0.f ? 0.f : 1.f / sum;
  const bool first = kw == 0 && half == 0 && row < nrows;
  const int64_t out_row = static_cast<int64_t>(it.t0 + row / G) * a.Hq + it.hk * G + row % G;
  if (a.together) {
    if (first && a.lse) a.lse[out_row] = it.bad ? inv : (m + log2f(sum)) * kLn2;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] *= inv;
  } else if (first) {
    a.ml[static_cast<int64_t>(it.slot) * a.N * a.Hq + out_row] = make_float2(m, sum);
  }
  float* mine = reinterpret_cast<float*>(lds + w * F::STAGE);
  const float4* theirs = reinterpret_cast<const float4*>(lds + ((1 - kw) * QW + qw) * F::STAGE);
#pragma unroll
  for (int c = 0; c < ND / 2; ++c) {
    const bool writer = KW == 1 || kw == (c & 1);
    if (KW == 2) {
      __syncthreads();
      if (!writer) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const f32x16& y = o[2 * c + x / 4];
          reinterpret_cast<float4*>(mine)[x * 64 + l] = make_float4(y[4 * (x & 3)], y[4 * (x & 3) + 1], y[4 * (x & 3) + 2], y[4 * (x & 3) + 3]);
        }
      }
      __syncthreads();
    } else if (c == 0) {
      __syncthreads();  // (the ring is read no more)
    }
    if (writer) {
      float4 y[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const f32x16& z = o[2 * c + x / 4];
        y[x] = make_float4(z[4 * (x & 3)], z[4 * (x & 3) + 1], z[4 * (x & 3) + 2], z[4 * (x & 3) + 3]);
        if (KW == 2) {
          const float4 t = theirs[x * 64 + l];
          y[x].x += t.x;
          y[x].y += t.y;
          y[x].z += t.z;
          y[x].w += t.w;
        }
      }
      wave_lds_sync();
#pragma unroll
      for (int x = 0; x < 8; ++x) *reinterpret_cast<float4*>(mine + lr * 68 + 32 * (x / 4) + 8 * (x & 3) + 4 * half) = y[x];
      wave_lds_sync();
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int r = 4 * x + (l >> 4), ch = 64 * c + 4 * (l & 15), gr = row_w + r;
        const float4 y4 = *reinterpret_cast<const float4*>(mine + r * 68 + 4 * (l & 15));
        if (gr >= nrows || ch >= a.D) continue;
        const int64_t to = static_cast<int64_t>(it.t0 + gr / G) * a.Hq + it.hk * G + gr % G;
        if (a.together) *reinterpret_cast<uint2*>(static_cast<bf16*>(a.o) + to * a.D + ch) = pack4_bf16(y4.x, y4.y, y4.z, y4.w);
        else *reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(it.slot) * a.N * a.Hq + to) * a.D + ch) = y4;
      }
      wave_lds_sync();
    }
  }
  if (a.together) bad_rows<bf16>(a, it, nrows, 64 * F::W);
}

template <int DC, int QW, int KW> hipError_t launch(const AttnArgs& a, unsigned items, hipStream_t st) {
  many_kernel<DC, QW, KW><<<items, 64 * QW * KW, 0, st>>>(a);
  return hipGetLastError();
}
template <int DC> hipError_t launch_rows(const AttnArgs& a, int rows, unsigned items, hipStream_t st) {
  return rows == 128 ? launch<DC, 4, 2>(a, items, st) : launch<DC, 8, 1>(a, items, st);
}

}  // namespace

hipError_t launch_many(const AttnArgs& a, int rows, unsigned items, hipStream_t st) {
  if (a.D <= 64) return launch_rows<64>(a, rows, items, st);
  if (a.D <= 128) return launch_rows<128>(a, rows, items, st);
  if (a.D <= 192) return launch_rows<192>(a, rows, items, st);
  return launch_rows<256>(a, rows, items, st);
}

}  // namespace attn
}  // namespace gdn
