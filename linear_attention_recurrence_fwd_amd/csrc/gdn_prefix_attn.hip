// Softmax attention of a batch's new tokens over a prefix that all sequences share
// and over their own keys, in pages.
//
//   o_i = sum_j e^(s_ij - m_i) v_j / l_i,  s_ij = scale q_i . k_j,  l_i = sum_j e^(s_ij - m_i)
//
// in one pass over the keys with a running reference m and sum l (all weights times
// 2^-lift, gdn_prefix_attn.h); parts over
// disjoint keys join by o = sum o_x e^(m_x - m), l = sum l_x e^(m_x - m).
//
// The rows of a key head's G query heads go together, and over the prefix those of
// all sequences: the prefix's keys are read once for the batch (once for each tile
// of rows), not once for each sequence.
//
// The kernel for few rows is bound by the keys and values that it reads once: the own
// keys of 64 sequences, 100 to 2000 each, 2 heads of 256, bf16, 137 MB in 38 us, 3.6 TB/s
// (a large copy: 5.15).  Eight single tokens over 1000 shared keys and a few hundred own
// ones are latency: 9 us for the keys, 4 for the parts.
#include "gdn_prefix_attn.h"
namespace gdn {
namespace attn {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

// ---- few rows: 16 QB rows of queries, NW waves that share out the keys
//
// Each wave takes every NW-th tile of 16 keys and brings it to its own part of LDS by
// direct loads, ST tiles ahead: no barriers, and 128 KB of keys and values on their way
// to a compute unit.  Scores are formed transposed, keys by rows: a lane holds four
// keys of one query, which is as the second product takes the weights, from
// registers; the values' other operand comes by transposing reads (bf16) or single
// words (fp32).  At the end the waves' results are joined through LDS.
template <typename T, int DC, int QB, int NW> struct Few {
  static constexpr int E = sizeof(T), KT = 16;
  static constexpr int PR = DC * E / 16;                    // pieces of 16 bytes of a row
  static constexpr int TILE = KT * PR * 16;                 // bytes of a tile of keys or values
  // two workgroups to a compute unit, so that one's begin and end lie beside the other's
  // middle (fp32 of wide heads: one)
  static constexpr int ST = (NW == 4 ? 16384 : sizeof(T) == 4 && DC > 128 ? 65536 : 32768) / (2 * TILE);
  static constexpr int NL = TILE / 1024;                    // load instructions of a tile
  static constexpr int RING = 2 * TILE * ST;
  static constexpr int TS = 4 * ST;                         // tiles whose pages are held
  static constexpr int ROW = DC + 4;                        // floats of a result's row in LDS
  static constexpr int OUT = 16 * QB * ROW * 4;
  static constexpr int WAVE = (RING > OUT ? RING : OUT);
  static constexpr int LDS = NW * (WAVE + TS * KT * 4 + 16 * QB * 8);
  static_assert(ST >= 2 && (ST - 1) * (2 * NL + 1) < 64, "waits count up to 63 loads");
  static_assert(LDS <= (sizeof(T) == 4 && DC > 128 ? 160 : 80) * 1024, "LDS");
};


template <typename T, int DC, int QB, int NW>
__global__ void __launch_bounds__(64 * NW, NW == 4 ? 2 : 1) few_kernel(AttnArgs a) {
  using F = Few<T, DC, QB, NW>;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int KT = F::KT, PR = F::PR, ST = F::ST, NL = F::NL, TS = F::TS, NS = DC / 16;
  __shared__ __align__(256) char lds[F::LDS];
  auto swz = [](int row) { return swizzle<PR, BF ? 2 : 0>(row); };
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, lr = l & 15, lg = l >> 4;
  const Item it = find_item(a);
  if (it.empty) return;
  const int tiles = it.k1 > it.k0 ? (it.k1 - it.k0 + KT - 1) / KT : 0;
  char* ring = lds + w * F::WAVE;
  const uint32_t ring_at = lds_of(lds) + w * F::WAVE;
  int32_t* pages = reinterpret_cast<int32_t*>(lds + NW * F::WAVE) + w * TS * KT;
  const uint32_t pages_at = lds_of(lds) + NW * F::WAVE + w * TS * KT * 4;
  float2* stats = reinterpret_cast<float2*>(lds + NW * (F::WAVE + TS * KT * 4));

  // Queries, as the products take them: bf16 channels 32 st + 8 lg .. + 7 of row lr;
  // fp32 channels 16 st + 4 lg .. + 3.
  const int G = a.G, nrows = it.n * G;
  uint4 q[QB][BF ? NS / 2 : NS];
  int lim[QB];  // keys that the row sees
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int r = it.row0 + 16 * b + lr, tok = r / G;
    const bool on = r < nrows && !it.bad;
    lim[b] = it.seen + tok;
    const T* row = static_cast<const T*>(a.q) + (static_cast<int64_t>(it.t0 + (on ? tok : 0)) * a.Hq + it.hk * G + (on ? r % G : 0)) * a.D;
#pragma unroll
    for (int st = 0; st < (BF ? NS / 2 : NS); ++st) {
      const int c = BF ? 32 * st + 8 * lg : 16 * st + 4 * lg;
      q[b][st] = make_uint4(0, 0, 0, 0);
      if (on && c < a.D) q[b][st] = *reinterpret_cast<const uint4*>(row + c);
    }
  }

  f32x4 o[QB][NS];
  float m[QB], sum[QB];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    m[b] = -__builtin_inff();
    sum[b] = 0.f;
#pragma unroll
    for (int d = 0; d < NS; ++d) o[b][d] = f4zero();
  }

  const int cnt = tiles > w ? (tiles - w + NW - 1) / NW : 0;  // this wave's tiles: w, w + NW, ...
  const char *kb = static_cast<const char*>(a.kp) + it.hk * a.pool.hs, *vb = static_cast<const char*>(a.vp) + it.hk * a.pool.hs;
  const int in_page = (1 << a.pool.shift) - 1;
  auto page_of = [&](int x) {  // where the page of key lr of the wave's tile x is told
    const int key = min(it.k0 + KT * (w + NW * (x < cnt ? x : cnt - 1)) + lr, it.k1 - 1);
    return it.list + (key >> a.pool.shift);
  };
  auto load_pages = [&](int x) {
    if (l < KT) load_lds4(page_of(x), pages_at + (x % TS) * KT * 4);
  };
  // A full tile lies in one page where pages hold it: one address for the wave, and each
  // lane's constant distance from it.  (Row by row, the addresses cost as much as the
  // tile's products.)  Heads of other sizes than 64, 128, 192 and 256 go row by row: the
  // places of the channels that there are not have to be filled.
  const bool one_page = (1 << a.pool.shift) >= KT && a.D == DC && a.pool.ts < (1 << 26);
  uint32_t from_first[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int row = (i * 64 + l) / PR, piece = ((i * 64 + l) % PR) ^ swz(row);
    from_first[i] = row * static_cast<uint32_t>(a.pool.ts) + piece * 16;
  }
  auto load_tile = [&](int x) {
    const int key0 = it.k0 + KT * (w + NW * x), end = it.k1;
    const int page = pages[(x % TS) * KT + lr], page_w = __builtin_amdgcn_readfirstlane(page);
    const uint32_t kt = ring_at + (x % ST) * 2 * F::TILE;
    if (one_page && key0 + KT <= end && page_w >= 0 && page_w < a.pool.pages) {
      const int64_t off = page_w * a.pool.ps + (key0 & in_page) * a.pool.ts;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        load_lds16(kb + off, from_first[i], kt + i * 1024);
        load_lds16(vb + off, from_first[i], kt + F::TILE + i * 1024);
      }
      return;
    }
    // offset of key lr's row; -1: behind the end, -2: no such page
    const int key = key0 + lr;
    int64_t off = page * a.pool.ps + (key & in_page) * a.pool.ts;
    if (page < 0 || page >= a.pool.pages) off = -2;
    if (key >= end) off = -1;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int row = (i * 64 + l) / PR, piece = ((i * 64 + l) % PR) ^ swz(row);
      const int64_t from = (static_cast<int64_t>(__shfl(static_cast<int>(off >> 32), row)) << 32) |
                           static_cast<uint32_t>(__shfl(static_cast<int>(off), row));
      const bool fill = from < 0 || piece * 16 >= a.D * F::E;
      const int64_t at = from + piece * 16;
      const void* none = &kFill[from == -2 ? 1 : 0];
      load_lds16(fill ? none : kb + at, kt + i * 1024);
      load_lds16(fill ? none : vb + at, kt + F::TILE + i * 1024);
    }
  };

  if (cnt > 0) {
    for (int x = l; x < ST * KT; x += 64) {
      const int t = x / KT, key = min(it.k0 + KT * (w + NW * (t < cnt ? t : cnt - 1)) + x % KT, it.k1 - 1);
      pages[x] = it.list[key >> a.pool.shift];
    }
    wave_lds_sync();
#pragma unroll 1
    for (int x = 0; x < ST; ++x) {
      load_pages(ST + x);
      if (x < cnt) load_tile(x);
    }
  }
#pragma unroll 1
  for (int x = 0; x < cnt; ++x) {
    // everything issued up to tile x's loads
    if (x + ST <= cnt) wait_vm<(ST - 1) * (2 * NL + 1)>();
    else wait_vm<0>();
    const int key0 = it.k0 + KT * (w + NW * x);
    const char *kt = ring + (x % ST) * 2 * F::TILE, *vt = kt + F::TILE;
    f32x4 s[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) s[b] = f4zero();
    if constexpr (BF) {
#pragma unroll
      for (int st = 0; st < NS / 2; ++st) {
        const bf16x8 k = load_bf16x8(kt + (lr * PR + ((4 * st + lg) ^ swz(lr))) * 16);
#pragma unroll
        for (int b = 0; b < QB; ++b) s[b] = mfma16(k, as_bf16x8(q[b][st]), s[b]);
      }
    } else {
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        const float4 k = *reinterpret_cast<const float4*>(kt + (lr * PR + ((4 * st + lg) ^ swz(lr))) * 16);
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          s[b] = mfma16f(k.x, __uint_as_float(q[b][st].x), s[b]);
          s[b] = mfma16f(k.y, __uint_as_float(q[b][st].y), s[b]);
          s[b] = mfma16f(k.z, __uint_as_float(q[b][st].z), s[b]);
          s[b] = mfma16f(k.w, __uint_as_float(q[b][st].w), s[b]);
        }
      }
    }
    bool move = false;
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const int see = min(it.k1, lim[b]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[b][r] = key0 + 4 * lg + r < see ? s[b][r] * a.scale : -__builtin_inff();
        move |= s[b][r] - m[b] > kSlack;
      }
    }
    if (__any(move)) {
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        float top = fmaxf(fmaxf(s[b][0], s[b][1]), fmaxf(s[b][2], s[b][3]));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        // (only of the rows that ask for it: a row's bits are its own, whatever lies beside it)
        const float to = top - m[b] > kSlack ? top : m[b], f = to == m[b] ? 1.f : __builtin_amdgcn_exp2f(m[b] - to);
        m[b] = to;
        sum[b] *= f;
#pragma unroll
        for (int d = 0; d < NS; ++d) o[b][d] *= f;
      }
    }
    f32x4 p[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const float ref = m[b] == -__builtin_inff() ? 0.f : m[b];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        p[b][r] = __builtin_amdgcn_exp2f(s[b][r] - ref) * a.unit;
        sum[b] += p[b][r];  // (bf16: before they are rounded, so that lse is exact to 32 bits)
      }
    }
    if constexpr (BF) {
      // (the weights rounded to bf16: up to 2^-8 of each, as the products of bf16 take them)
      s16x4 pb[QB];
#pragma unroll
      for (int b = 0; b < QB; ++b) pb[b] = __builtin_bit_cast(s16x4, pack4_bf16(p[b][0], p[b][1], p[b][2], p[b][3]));
      const int row = 4 * lg + (lr >> 2), in = (lr & 1) * 8;
#pragma unroll
      for (int d = 0; d < NS; ++d) {
        const uint2 v = lds_read_tr16(vt + (row * PR + ((2 * d + ((lr & 3) >> 1)) ^ swz(row))) * 16 + in);
#pragma unroll
        for (int b = 0; b < QB; ++b)
          o[b][d] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, v), pb[b], o[b][d], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int d = 0; d < NS; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 4 * lg + r;
          const float v = *reinterpret_cast<const float*>(vt + (row * PR + ((4 * d + (lr >> 2)) ^ swz(row))) * 16 + (lr & 3) * 4);
#pragma unroll
          for (int b = 0; b < QB; ++b) o[b][d] = mfma16f(v, p[b][r], o[b][d]);
        }
    }
    wave_lds_sync();  // what was read of this tile's place is in registers
    if (x + ST < cnt) {
      load_pages(x + 2 * ST);
      load_tile(x + ST);
    }
  }

  // Join the waves' results: row-major in LDS, then every thread a few channels.
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    float t = sum[b];
    t += __shfl_xor(t, 16);
    t += __shfl_xor(t, 32);
    if (lg == 0) stats[w * 16 * QB + 16 * b + lr] = make_float2(m[b], t);
#pragma unroll
    for (int d = 0; d < NS; ++d)
      *reinterpret_cast<float4*>(mine + (16 * b + lr) * F::ROW + 16 * d + 4 * lg) = make_float4(o[b][d][0], o[b][d][1], o[b][d][2], o[b][d][3]);
  }
  __syncthreads();
  const int cols = a.D / 4, rows = min(16 * QB, nrows - it.row0);
  for (int i = threadIdx.x; i < rows * cols; i += 64 * NW) {
    const int r = i / cols, c = 4 * (i % cols);
    float top = -__builtin_inff();
#pragma unroll
    for (int x = 0; x < NW; ++x) top = fmaxf(top, stats[x * 16 * QB + r].x);
    const float ref = top == -__builtin_inff() ? 0.f : top;
    float t = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      const float2 ms = stats[x * 16 * QB + r];
      const float f = __builtin_amdgcn_exp2f(ms.x - ref);
      const float4 z = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(lds + x * F::WAVE) + r * F::ROW + c);
      t += f * ms.y;
      y.x += f * z.x;
      y.y += f * z.y;
      y.z += f * z.z;
      y.w += f * z.w;
    }
    const int tok = (it.row0 + r) / G;
    const int64_t row = static_cast<int64_t>(it.t0 + tok) * a.Hq + it.hk * G + (it.row0 + r) % G;
    if (a.together) {
      const float f = it.bad ? __builtin_nanf("") : t == 0.f ? 0.f : 1.f / t;
      T* dst = static_cast<T*>(a.o) + row * a.D + c;
      if constexpr (BF) *reinterpret_cast<uint2*>(dst) = pack4_bf16(y.x * f, y.y * f, y.z * f, y.w * f);
      else *reinterpret_cast<float4*>(dst) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
      if (a.lse && c == 0) a.lse[row] = it.bad ? f : (top + log2f(t * a.whole)) * kLn2;
    } else {
      const int64_t at = static_cast<int64_t>(it.slot) * a.N * a.Hq + row;
      *reinterpret_cast<float4*>(a.part + at * a.D + c) = y;
      if (c == 0) a.ml[at] = make_float2(top, t);
    }
  }
  if (a.together) bad_rows<T>(a, it, nrows, 64 * NW);
}

// ---- the join of the parts
//
// LPR lanes to a row, four channels each.  The row's parts are the prefix's splits and
// those of its own keys that it sees.  WPR waves share them out, where there are few rows.
template <typename T, int LPR, int WPR>
__global__ void __launch_bounds__(256) join_kernel(AttnArgs a) {
  constexpr int RB = 256 / LPR / WPR;  // rows of a workgroup
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int which = WPR == 1 ? 0 : wave, slot = WPR == 1 ? threadIdx.x / LPR : lane / LPR;
  const int64_t all = static_cast<int64_t>(a.N) * a.Hq, row_ = static_cast<int64_t>(blockIdx.x) * RB + slot;
  const int64_t row = row_ < all ? row_ : all - 1;
  const int c = 4 * (threadIdx.x % LPR);
  const int tok = static_cast<int>(row / a.Hq);
  int s, i, n;
  if (a.cu) {
    // the last sequence that begins at or before the token
    int lo = -1, hi = a.S;
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (a.cu[mid] <= tok) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    const bool in = s >= 0 && s < a.S;
    i = in ? tok - a.cu[s] : 0;
    n = in ? a.cu[s + 1] - a.cu[s] : 0;
  } else {
    s = tok / a.per;
    i = tok % a.per;
    n = a.per;
  }
  const bool mine = row_ < all && c < a.D && s >= 0 && s < a.S;
  const int len = mine ? a.lens[s] : 0;
  const bool bad = len < 0 || len > a.max_len || n > a.max_q;
  const int see = len - n + 1 + i;
  const int parts = !mine ? 0 : a.p_split + (bad || see <= 0 ? 0 : min(a.o_split, (see + a.o_chunk - 1) / a.o_chunk));
  float m = -__builtin_inff();
#pragma unroll 4
  for (int x = which; x < parts; x += WPR) m = fmaxf(m, a.ml[x * all + row].x);
  float ref = m == -__builtin_inff() ? 0.f : m, t = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int x = which; x < parts; x += WPR) {
    const float2 ms = a.ml[x * all + row];
    const float f = __builtin_amdgcn_exp2f(ms.x - ref);
    const float4 z = *reinterpret_cast<const float4*>(a.part + (x * all + row) * a.D + c);
    t += f * ms.y;
    y.x += f * z.x;
    y.y += f * z.y;
    y.z += f * z.z;
    y.w += f * z.w;
  }
  if constexpr (WPR > 1) {
    __shared__ float4 ys[WPR][64];
    __shared__ float2 ms[WPR][64];
    ys[wave][lane] = y;
    ms[wave][lane] = make_float2(m, t);
    __syncthreads();
    if (wave > 0) return;
    m = -__builtin_inff();
#pragma unroll
    for (int x = 0; x < WPR; ++x) m = fmaxf(m, ms[x][lane].x);
    ref = m == -__builtin_inff() ? 0.f : m;
    t = 0.f;
    y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < WPR; ++x) {
      const float f = __builtin_amdgcn_exp2f(ms[x][lane].x - ref);
      const float4 z = ys[x][lane];
      t += f * ms[x][lane].y;
      y.x += f * z.x;
      y.y += f * z.y;
      y.z += f * z.z;
      y.w += f * z.w;
    }
  }
  if (!mine) return;
  const float f = bad ? __builtin_nanf("") : t == 0.f ? 0.f : 1.f / t;
  T* dst = static_cast<T*>(a.o) + row * a.D + c;
  if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(dst) = pack4_bf16(y.x * f, y.y * f, y.z * f, y.w * f);
  else *reinterpret_cast<float4*>(dst) = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
  if (a.lse && c == 0) a.lse[row] = bad ? f : (m + log2f(t * a.whole)) * kLn2;
}

template <typename T, int LPR> hipError_t launch_join(const AttnArgs& a, hipStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.N) * a.Hq;
  if (rows * LPR >= 65536 * 8) join_kernel<T, LPR, 1><<<static_cast<unsigned>((rows + 256 / LPR - 1) / (256 / LPR)), 256, 0, st>>>(a);
  else join_kernel<T, LPR, 4><<<static_cast<unsigned>((rows + 64 / LPR - 1) / (64 / LPR)), 256, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int DC, int QB, int NW> hipError_t launch_few(const AttnArgs& a, unsigned items, hipStream_t st) {
  few_kernel<T, DC, QB, NW><<<items, 64 * NW, 0, st>>>(a);
  return hipGetLastError();
}
template <typename T, int DC> hipError_t launch_qb(const AttnArgs& a, int rows, unsigned items, hipStream_t st) {
  constexpr int NW = DC * sizeof(T) <= 256 ? 4 : 2;
  return rows == 16 ? launch_few<T, DC, 1, NW>(a, items, st) : launch_few<T, DC, 2, NW>(a, items, st);
}
// The items of a launch (which of them: a.which), all of the same number of rows.
template <typename T> hipError_t launch_items(AttnArgs a, int which, hipStream_t st) {
  a.which = which;
  const unsigned items = static_cast<unsigned>((which & 1 ? prefix_items(a) : 0) + (which & 2 ? own_items(a) : 0));
  const int rows = which & 2 ? a.o_rows : a.p_rows;
  if (items == 0) return hipSuccess;
  if (rows > 32) return launch_many(a, items, st);  // (bf16 only)
  if (a.D <= 64) return launch_qb<T, 64>(a, rows, items, st);
  if (a.D <= 128) return launch_qb<T, 128>(a, rows, items, st);
  if (a.D <= 192) return launch_qb<T, 192>(a, rows, items, st);
  return launch_qb<T, 256>(a, rows, items, st);
}
template <typename T> hipError_t launch_any(const AttnArgs& a, hipStream_t st) {
  hipError_t e;
  if (a.together) return launch_items<T>(a, 2, st);
  if (a.p_rows == a.o_rows) {
    e = launch_items<T>(a, 3, st);
  } else {
    e = launch_items<T>(a, 1, st);
    if (e == hipSuccess) e = launch_items<T>(a, 2, st);
  }
  if (e != hipSuccess) return e;
  if (a.D <= 64) return launch_join<T, 16>(a, st);
  if (a.D <= 128) return launch_join<T, 32>(a, st);
  return launch_join<T, 64>(a, st);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn(const AttnArgs& a, bool bf, hipStream_t st) {
  if (a.N == 0) return hipSuccess;
  return bf ? attn::launch_any<bf16>(a, st) : attn::launch_any<float>(a, st);
}

}  // namespace gdn
