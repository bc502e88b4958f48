// Kernels of the decay operator beside the walks (gdn_decay_walk.h): the chain
// over segment states, the reductions of the backward, and the single steps.
#include "gdn_decay_walk.h"

namespace gdn {

size_t decay_sum_floats(int KD, int N) {
  auto up = [](int n) { return static_cast<size_t>(n <= 64 ? 64 : n <= 128 ? 128 : n <= 192 ? 192 : 256); };
  return up(KD) * up(N);
}

int decay_waves(int N) { return N <= 64 ? 4 : N <= 128 ? 8 : N <= 192 ? 12 : 8; }

hipError_t launch_decay_walk(const DecayWalkArgs& a, bool sum, bool bf, hipStream_t st) {
  const int KD = a.walk[0].KD;
  if (sum) {
    if (KD <= 64) return bf ? decay_sum_bf16_64(a, st) : decay_sum_f32_64(a, st);
    if (KD <= 128) return bf ? decay_sum_bf16_128(a, st) : decay_sum_f32_128(a, st);
    if (KD <= 192) return bf ? decay_sum_bf16_192(a, st) : decay_sum_f32_192(a, st);
    return bf ? decay_sum_bf16_256(a, st) : decay_sum_f32_256(a, st);
  }
  if (KD <= 64) return bf ? decay_walk_bf16_64(a, st) : decay_walk_f32_64(a, st);
  if (KD <= 128) return bf ? decay_walk_bf16_128(a, st) : decay_walk_f32_128(a, st);
  if (KD <= 192) return bf ? decay_walk_bf16_192(a, st) : decay_walk_f32_192(a, st);
  return bf ? decay_walk_bf16_256(a, st) : decay_walk_f32_256(a, st);
}

hipError_t decay_keys_64(const DecayKeysArgs& a, hipStream_t st);
hipError_t decay_keys_128(const DecayKeysArgs& a, hipStream_t st);
hipError_t decay_keys_192(const DecayKeysArgs& a, hipStream_t st);
hipError_t decay_keys_256(const DecayKeysArgs& a, hipStream_t st);

hipError_t launch_decay_keys(const DecayKeysArgs& a, hipStream_t st) {
  if (a.d.Dv <= 64) return decay_keys_64(a, st);
  if (a.d.Dv <= 128) return decay_keys_128(a, st);
  if (a.d.Dv <= 192) return decay_keys_192(a, st);
  return decay_keys_256(a, st);
}

namespace {

using decay::exp2_fast;
using decay::log2_decay;

// ---- chain: the segment sums U_s of one direction become the states before
// each segment, start_{s+1} = g^{N_s} start_s + U_s with N_s the segment's valid
// steps.  One thread per four elements of one (b, h) goes through the segments
// (in walk order), a wave to a workgroup so that few heads still reach every
// compute unit; the loads of the next eight segments are in flight while the last
// eight are summed.  All of it is traffic: both directions of 64 heads of 192 x 128
// with 4 segments, 101 MB in 18 us, 5.6 TB/s; 4 heads of 128 x 128 with 64 segments,
// 34 MB in 10 us, 3.2 TB/s (256 waves, eight loads of 16 bytes a lane each).
struct ChainArgs {
  DecayChainArgs c[2];
};

__global__ void __launch_bounds__(64) chain_kernel(ChainArgs aa) {
  const DecayChainArgs& a = aa.c[blockIdx.z];
  const DecayDims& d = a.d;
  const int bh = blockIdx.x, b = bh / d.Hv, h = bh % d.Hv, BH = d.B * d.Hv, l = threadIdx.x, nseg = a.nseg;
  __shared__ float dec[kDecayMaxSeg];  // g^{N_s}, in walk order
  const float lg2 = log2_decay(a.lg[h]);
  for (int s = l; s < nseg; s += 64)
    dec[s] = exp2_fast(lg2 * a.seg_steps[static_cast<size_t>(b) * nseg + (a.reverse ? nseg - 1 - s : s)]);
  __syncthreads();
  const size_t hs = static_cast<size_t>(d.Dk) * d.Dv;
  const size_t e = (static_cast<size_t>(blockIdx.y) * 64 + l) * 4;
  if (e >= hs) return;
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.start) run = *reinterpret_cast<const float4*>(a.start + bh * hs + e);
  const size_t step = static_cast<size_t>(BH) * hs;
  float* p = a.states + bh * hs + e;
  auto at = [&](int s) { return reinterpret_cast<float4*>(p + (a.reverse ? nseg - 1 - s : s) * step); };
  constexpr int N = 8;
  float4 u[2][N];
#pragma unroll
  for (int k = 0; k < N; ++k) u[0][k] = *at(min(k, nseg - 1));
  for (int s0 = 0; s0 < nseg; s0 += 2 * N) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int s1 = s0 + half * N;
      if (s1 >= nseg) break;
      if (s1 + N < nseg) {
#pragma unroll
        for (int k = 0; k < N; ++k) u[half ^ 1][k] = *at(min(s1 + N + k, nseg - 1));
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (s1 + k >= nseg) break;
        *at(s1 + k) = run;
        const float f = dec[s1 + k];
        const float4 v = u[half][k];
        run.x = fmaf(f, run.x, v.x);
        run.y = fmaf(f, run.y, v.y);
        run.z = fmaf(f, run.z, v.z);
        run.w = fmaf(f, run.w, v.w);
      }
    }
  }
  if (a.end) *reinterpret_cast<float4*>(a.end + bh * hs + e) = run;
}

// ---- dlg of one head: its parts summed in a fixed order.
__global__ void __launch_bounds__(256) reduce_kernel(DecayReduceArgs a) {
  const int h = blockIdx.x, tid = threadIdx.x;
  __shared__ double part[256];
  double total = 0.0;
  for (int b = 0; b < a.d.B; ++b) {
    const double* p = a.grad + (static_cast<size_t>(b) * a.d.Hv + h) * a.n;
    for (int i = tid; i < a.n; i += 256) total += p[i];
  }
  part[tid] = total;
  __syncthreads();
  for (int m = 128; m >= 1; m >>= 1) {
    if (tid < m) part[tid] += part[tid + m];
    __syncthreads();
  }
  if (tid == 0) a.dlg[h] = static_cast<float>(part[0]);
}

// ---- dq / dk of the key heads: their value heads' rows summed in fp32, in
// head order, and rounded once.  All of it is traffic: 16 key heads of 192 with four
// (dq) and two (dk) parts, 2048 steps: 176 MB in 26 us, 6.8 TB/s, partly still cached.
template <typename T>
__global__ void __launch_bounds__(256) group_kernel(DecayGroupArgs a, size_t n) {
  const DecayDims& d = a.d;
  const int G = a.parts[blockIdx.y];
  if (G == 1) return;
  const float* src = blockIdx.y ? a.pk : a.pq;
  T* dst = static_cast<T*>(blockIdx.y ? a.dk : a.dq);
  for (size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < n;
       i += static_cast<size_t>(gridDim.x) * 1024) {
    const size_t row = i / d.Dk, c = i % d.Dk;  // (token, key head), channel
    const float* p = src + row * G * d.Dk + c;
    float4 s = *reinterpret_cast<const float4*>(p);
    for (int g = 1; g < G; ++g) {
      const float4 v = *reinterpret_cast<const float4*>(p + static_cast<size_t>(g) * d.Dk);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(dst + i) = pack4_bf16(s.x, s.y, s.z, s.w);
    else *reinterpret_cast<float4*>(dst + i) = s;
  }
}

// ---- single steps, S <- g S + k v^T, o = scale S^T q, T of them in turn.  The
// state is the whole traffic of a single step, read and written once (64 sequences
// of 32 heads of 128 x 128: 268 MB in 43 us, 6.2 TB/s, part of it still cached;
// one of them: 4 MB in 4.4 us, a launch and two trips to memory).  One wave per 32
// columns of one (b, h): lane 8 rg + cq holds rows rg RL .. + RL - 1 of columns 4 cq
// .. + 3, so eight lanes cover 128 contiguous bytes of a row.  The next step's q, k
// and v are asked for ahead of the step's own sums, as whole pieces of a row (element
// by element the 64 sequences take 56 us).

// N consecutive values (from a place that can be read); zeros where in is false.
template <typename T, int N> __device__ __forceinline__ void load_row(const T* p, bool in, float* out) {
  constexpr int B = N * static_cast<int>(sizeof(T));
  if constexpr (B >= 16) {
    constexpr int E = Vec16<T>::N;
#pragma unroll
    for (int i = 0; i < N / E; ++i) Vec16<T>::unpack(reinterpret_cast<const uint4*>(p)[i], out + i * E);
  } else {
    uint32_t u[B / 4];
    if constexpr (B == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      u[0] = v.x;
      u[1] = v.y;
    } else {
      u[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4) out[i] = __uint_as_float(u[i]);
      else out[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = in ? out[i] : 0.f;
}

// f x + t in x's place.  (The compiler makes the sum in t's and moves it back, a move
// to each element: 7.9 us instead of 7.5 for 4 steps of 32 heads of 128 x 128.)
__device__ __forceinline__ void times_plus(float& x, float f, float t) {
  asm("v_fma_f32 %0, %1, %0, %2" : "+v"(x) : "v"(f), "v"(t));
}

template <typename T, int DK>
__global__ void __launch_bounds__(64) step_kernel(DecayStepArgs p, int slices) {
  constexpr int RL = DK / 8;
  const DecayDims& d = p.d;
  const int bh = blockIdx.x / slices, w = blockIdx.x % slices, b = bh / d.Hv, h = bh % d.Hv, j = h / d.G();
  const int l = threadIdx.x, rg = l >> 3, cq = l & 7, col = 32 * w + 4 * cq;
  const size_t hs = static_cast<size_t>(d.Dk) * d.Dv;
  const uint32_t bytes = static_cast<uint32_t>(hs * 4);
  // Dk and Dv are multiples of 8, so P rows of a lane, and its columns, are all
  // there or none.  State entries that are not there are sent past the descriptor's
  // size; the values of q, k and v are read from the head's start and dropped.
  constexpr int P = RL < 8 ? RL : 8;
  const bool on = col < d.Dv;
  uint32_t off[RL];
#pragma unroll
  for (int r = 0; r < RL; ++r)
    off[r] = on && rg * RL + r < d.Dk ? 4u * ((rg * RL + r) * d.Dv + col) : 0xfffffff0u;
  const rsrc_t rs0 = make_rsrc(p.state0 ? static_cast<const void*>(p.state0 + bh * hs) : p.state_out, p.state0 ? bytes : 0);
  float4 s[RL];
#pragma unroll
  for (int r = 0; r < RL; ++r) s[r] = buf_f4(rs0, off[r]);
  // The decay of a step in two parts, gate + rest: one fp32 number below one is off by
  // up to 2^-25, the same at every step.  At lg = -3e-4 that left a state of thousands
  // of steps 7e-5 off; with rest it is 1e-6, what the roundings of its sums come to.
  // (Below -1/2 a state forgets within a few steps, and rest is of no use.)  A third
  // product to each element: 4 steps of 32 heads of 128 x 128 take 7.5 us, without
  // 6.9; single steps, which wait for memory, the same.
  const float lg = p.lg[h], m = expm1f(lg);
  const bool slow = fabsf(lg) < 0.5f;
  const float gate = slow ? 1.f + m : exp2_fast(log2_decay(lg)), rest = slow ? (1.f - gate) + m : 0.f;
  const size_t qs = static_cast<size_t>(d.Hk) * d.Dk, vs = static_cast<size_t>(d.Hv) * d.Dv;
  const size_t bt0 = static_cast<size_t>(b) * d.T;
  const T* qr = static_cast<const T*>(p.q) + bt0 * qs + static_cast<size_t>(j) * d.Dk;
  const T* kr = static_cast<const T*>(p.k) + bt0 * qs + static_cast<size_t>(j) * d.Dk;
  const T* vr = static_cast<const T*>(p.v) + bt0 * vs + static_cast<size_t>(h) * d.Dv + (on ? col : 0);
  float q[RL], k[RL], v[4];
  int live = 1;
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < RL; i += P) {
      const bool in = rg * RL + i < d.Dk;
      const int at = in ? rg * RL + i : 0;
      load_row<T, P>(qr + t * qs + at, in, q + i);
      load_row<T, P>(kr + t * qs + at, in, k + i);
    }
    load_row<T, 4>(vr + t * vs, on, v);
    live = p.mask == nullptr ? 1 : p.mask[bt0 + t];
  };
  if (d.T > 0) load(0);
  for (int t = 0; t < d.T; ++t) {
    float qt[RL], kt[RL], vt[4];
#pragma unroll
    for (int r = 0; r < RL; ++r) {
      qt[r] = q[r] * p.scale;
      kt[r] = k[r];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) vt[c] = v[c];
    const bool valid = live != 0;
    if (t + 1 < d.T) load(t + 1);
    if (valid) {
#pragma unroll
      for (int r = 0; r < RL; ++r) {
        times_plus(s[r].x, gate, fmaf(rest, s[r].x, kt[r] * vt[0]));
        times_plus(s[r].y, gate, fmaf(rest, s[r].y, kt[r] * vt[1]));
        times_plus(s[r].z, gate, fmaf(rest, s[r].z, kt[r] * vt[2]));
        times_plus(s[r].w, gate, fmaf(rest, s[r].w, kt[r] * vt[3]));
      }
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < RL; ++r) {
      o.x = fmaf(qt[r], s[r].x, o.x);
      o.y = fmaf(qt[r], s[r].y, o.y);
      o.z = fmaf(qt[r], s[r].z, o.z);
      o.w = fmaf(qt[r], s[r].w, o.w);
    }
#pragma unroll
    for (int m = 8; m <= 32; m <<= 1) {
      o.x += __shfl_xor(o.x, m);
      o.y += __shfl_xor(o.y, m);
      o.z += __shfl_xor(o.z, m);
      o.w += __shfl_xor(o.w, m);
    }
    if (rg == 0 && on) {
      T* orow = static_cast<T*>(p.o) + (bt0 + t) * vs + static_cast<size_t>(h) * d.Dv + col;
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(orow) = pack4_bf16(o.x, o.y, o.z, o.w);
      else *reinterpret_cast<float4*>(orow) = o;
    }
  }
  const rsrc_t rs1 = make_rsrc(p.state_out + bh * hs, bytes);
#pragma unroll
  for (int r = 0; r < RL; ++r)
    buf_store_u4(rs1, off[r], make_uint4(__float_as_uint(s[r].x), __float_as_uint(s[r].y), __float_as_uint(s[r].z),
                                         __float_as_uint(s[r].w)));
}

template <typename T>
hipError_t launch_step(const DecayStepArgs& a, hipStream_t st) {
  const int slices = (a.d.Dv + 31) / 32, n = a.d.B * a.d.Hv * slices;
  if (a.d.Dk <= 16) step_kernel<T, 16><<<n, 64, 0, st>>>(a, slices);
  else if (a.d.Dk <= 32) step_kernel<T, 32><<<n, 64, 0, st>>>(a, slices);
  else if (a.d.Dk <= 64) step_kernel<T, 64><<<n, 64, 0, st>>>(a, slices);
  else if (a.d.Dk <= 128) step_kernel<T, 128><<<n, 64, 0, st>>>(a, slices);
  else if (a.d.Dk <= 192) step_kernel<T, 192><<<n, 64, 0, st>>>(a, slices);
  else step_kernel<T, 256><<<n, 64, 0, st>>>(a, slices);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_decay_chain(const DecayChainArgs* a, int n, hipStream_t st) {
  ChainArgs c;
  for (int i = 0; i < 2; ++i) c.c[i] = a[i < n ? i : 0];
  const DecayDims& d = a[0].d;
  const size_t hs = static_cast<size_t>(d.Dk) * d.Dv;
  chain_kernel<<<dim3(d.B * d.Hv, static_cast<unsigned>((hs + 255) / 256), n), 64, 0, st>>>(c);
  return hipGetLastError();
}

hipError_t launch_decay_reduce(const DecayReduceArgs& a, hipStream_t st) {
  reduce_kernel<<<a.d.Hv, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_decay_group(const DecayGroupArgs& a, bool bf, hipStream_t st) {
  const size_t n = static_cast<size_t>(a.d.B) * a.d.T * a.d.Hk * a.d.Dk;
  const size_t blocks = (n + 1023) / 1024;
  const dim3 grid(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 2);
  if (bf) group_kernel<gdn::bf16><<<grid, 256, 0, st>>>(a, n);
  else group_kernel<float><<<grid, 256, 0, st>>>(a, n);
  return hipGetLastError();
}

hipError_t launch_decay_step(const DecayStepArgs& a, bool bf, hipStream_t st) {
  return bf ? launch_step<gdn::bf16>(a, st) : launch_step<float>(a, st);
}

}  // namespace gdn
