// Host-side interfaces of the decay operator (linear attention with a decay
// for each head) and of the query/key norm with rotation: between their entry
// points (gdn_decay_api.hip) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

constexpr int kDecayChunk = 64;   // steps per chunk; segments are whole chunks
constexpr int kDecayMaxSeg = 256;      // segments of one sequence: one to a compute unit at most
constexpr int kDecayMaxT = 1 << 30;    // steps of one sequence
constexpr int kDecayMaxPairs = (1 << 21) - 64;  // (b, h) pairs

struct DecayDims {
  int B, T, Hk, Hv, Dk, Dv;
  __host__ __device__ int G() const { return Hv / Hk; }
  __host__ __device__ int nchunk() const { return (T + kDecayChunk - 1) / kDecayChunk; }
};

// One [B, T, H, D] tensor as a walk reads it: the head of value head h is
// h / group.
struct DecayRows {
  const void* p;
  int H, D, group;
};

// A walk over the chunks of one segment for each (b, value head): with a state
// S [KD, N] (KD channels of x and y, N columns of z and w),
//   w_i = rs (S_i^T x_i) with S_i = sum_j<=i decay y_j z_j^T + decay S_start.
// The four sums of the operator and its backward are walks:
//   o : x = q,  y = k,  z = v,  forward in time, start state0
//   dq: x = dO, y = v,  z = k,  forward in time, start state0 transposed
//   dk: x = v,  y = dO, z = q,  backward in time, start dS_final transposed
//   dv: x = k,  y = q,  z = dO, backward in time, start dS_final
struct DecayWalk {
  DecayRows x, y, z, e;   // e: what the outputs are dotted with (dlg), [.., N]
  void* w;                // [B, T, Hv, N], of the tensors' type
  int KD, N;              // channels and columns
  int reverse;            // backward in time
  float scale_p;          // on the products x . y
  float scale_i;          // on the products with the state
  float scale_u;          // on the state update
  // states [Dk, Dv] fp32 per (b, h): element (channel, column) at
  // channel * sr + column * sc
  int sr, sc;
  const float* start;       // [B*Hv] states the sequence starts from (null: zeros)
  const float* seg_start;   // [nseg, B*Hv] start states (null: one segment)
  float* end;               // state behind the sequence (null: not written)
  // A sum (the walk that only sums its segments' updates) writes [nseg, B*Hv]
  // states here, in the order of the kernel's registers if seg_native (then
  // decay_sum_floats() each), and its segments' valid steps into [B, nseg] (if not
  // null).  A walk with seg_sum starts from start and the native sums before its
  // segment, and the first segment's writes end from all of them.
  float* seg_sum;
  float* seg_steps;
  int seg_native;
  // the dq walk: its part of dlg, fp64 [B*Hv, nseg, waves], from what e gives and
  // the loss's derivative in the state behind the segment (R; [nseg, B*Hv] seg_R)
  double* grad;
  const float *R, *seg_R;
};

struct DecayWalkArgs {
  DecayDims d;
  const float* lg;          // [Hv]
  const uint8_t* mask;      // may be null
  int nseg, seg;            // segments, chunks per segment
  int nwalk;
  DecayWalk walk[2];        // walks of one launch, with the same KD, N class
};

// dlg of a head: the sum of its walks' parts, n of them for each b.
struct DecayReduceArgs {
  DecayDims d;
  int n;
  const double* grad;       // [B*Hv, n]
  float* dlg;               // [Hv]
};

// dq and dk of the key heads (bf16), and the parts of dlg ([B*Hv, nseg, 4 waves to
// each block of 64 columns]).
struct DecayKeysArgs {
  DecayDims d;
  const float* lg;
  float scale;
  const uint8_t* mask;
  int nseg, seg;
  const void *q, *k, *v, *dO;
  const float *state0, *dS;   // one segment: start states (may be null)
  const float *S, *R;         // else [nseg, B*Hv] start states of both directions
  void *dq, *dk;              // [B, T, Hk, Dk]
  float *pq, *pk;             // or, where a key head's value heads go in parts, [B, T, Hk*parts, Dk] fp32
  double* grad;
};
// Value heads of a key head that one workgroup goes through for dk.  Two: four
// states of 128 channels leave too few registers (9B layer, 2048 steps: 75 us with
// two, 113 us with four).  For dq, which carries as many derivatives, one.
inline int decay_heads_together(int G) { return G % 2 == 0 ? 2 : 1; }

struct DecayChainArgs {
  DecayDims d;
  const float* lg;
  const float* seg_steps;   // [B, nseg] valid steps of the segments
  int nseg;
  float* states;            // [nseg, B*Hv, Dk*Dv]: segment sums in, start states out
  const float* start;       // may be null
  float* end;               // state behind the last segment walked (may alias start; null: not written)
  int reverse;
};

// dq / dk of a key head: the sum of its value heads' (or parts of them) rows,
// rounded once.
struct DecayGroupArgs {
  DecayDims d;
  int parts[2];             // of a key head, for dq and for dk (1: nothing to do)
  const float *pq, *pk;     // [B, T, Hk*parts, Dk] fp32
  void *dq, *dk;            // [B, T, Hk, Dk]
};

struct DecayStepArgs {
  DecayDims d;
  const void *q, *k, *v;
  const float* lg;
  float scale;
  const float* state0;
  const uint8_t* mask;
  void* o;
  float* state_out;
};

int decay_waves(int N);     // waves of a walk with N columns

size_t decay_sum_floats(int KD, int N);
hipError_t launch_decay_walk(const DecayWalkArgs& a, bool sum, bool bf16, hipStream_t st);
hipError_t launch_decay_keys(const DecayKeysArgs& a, hipStream_t st);
hipError_t launch_decay_chain(const DecayChainArgs* a, int n, hipStream_t st);
hipError_t launch_decay_reduce(const DecayReduceArgs& a, hipStream_t st);
hipError_t launch_decay_group(const DecayGroupArgs& a, bool bf16, hipStream_t st);
hipError_t launch_decay_step(const DecayStepArgs& a, bool bf16, hipStream_t st);

// ---- norm of queries and keys with rotation

struct NormRopeArgs {
  int64_t BT;               // tokens
  int Hq, Hk, D, R, P;
  int64_t qs, ks;           // elements from one token's rows to the next one's
  int T;                    // positions when pos is null: token % T
  int interleaved;
  float eps, w_offset;
  const void *q, *k;
  const float *wq, *wk;     // [D]
  const float* rope;        // [P, R]
  const int32_t* pos;       // [BT], may be null
  void *oq, *ok;            // forward: outputs
  const void *dyq, *dyk;    // backward: cotangents
  float* part;              // backward: [blocks, 2, D]
  float *dwq, *dwk;
  int blocks;
  // rotation with several axes (A of them; 0: the operator with one)
  int A;
  const uint8_t* axis;      // [R/2], may be null: all pairs on the first; pos is [A, BT]
  int bare;                 // no norm and no weights
  int back;                 // forward kernel: the inverse rotation (the VJP without norm)
};
int norm_rope_blocks(int64_t BT, int Hq, int Hk, int D, bool bf16);
hipError_t launch_norm_rope_fwd(const NormRopeArgs& a, bool bf16, hipStream_t st);
hipError_t launch_norm_rope_bwd(const NormRopeArgs& a, bool bf16, hipStream_t st);

}  // namespace gdn
