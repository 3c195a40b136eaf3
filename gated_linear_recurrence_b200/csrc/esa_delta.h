// esa_delta.h -- host-side interface between the gated delta rule's C ABI and
// its kernels.  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace esa {

// Shape and element strides of a call: row (b, t) of q and k starts at
// (b T + t) ld_qk, of v at (b T + t) ld_v, of a and b at (b T + t) ld_g.
struct DeltaShape {
  int B, T, H, D;
  long long ld_qk, ld_v, ld_g;
  float scale;
};

// One token-by-token sweep (see esa_delta_sweep.cuh for the four kinds).
struct SweepArgs {
  DeltaShape s;
  const void *q, *k, *v, *dy, *a, *b;   // I/O type
  const float *S_in;                    // state (or its gradient) before the first token visited; NULL = zeros
  float *S_out;                         // after the last one; NULL = not written
  void *y;                              // forward sweep's output, I/O type
  float *u, *du, *dk, *dk2, *dq;        // float32 scratch, [B,T,H,D]; dk2: what the last sweep adds to dk
  float *S_ck, *dS_ck;                  // [B,H,nc,D,D] state entering, gradient leaving each chunk of 64 tokens
  float *end;                           // [B,H,nc,D*D/1024] parts of their inner product at the chunk's end
  int nc;
  bool cut;                             // forward and Du sweeps start every chunk from S_ck, dS_ck, which are given
  float *wt, *u0, *fac;                 // [B,H,nc,64,D] W, U0 (then Z0) and [B,H,nc,3,64] factors of esa_delta_wy.cu
};

// Kinds of sweep.
enum { kSweepFwd = 0, kSweepDu = 1, kSweepDk = 2, kSweepDq = 3 };

int launch_sweep(int kind, int dtype, const SweepArgs &a, cudaStream_t st);   // kSweepDk: that and kSweepDq
// The states between chunks, float32: S_ck from S_in, also wt, fac; backward dS_ck from S_in = dS_final. And S_out.
int launch_delta_states(bool bwd, const SweepArgs &a, cudaStream_t st);
int launch_delta_step(int dtype, const SweepArgs &a, cudaStream_t st);   // one token, S_in = S_out

struct FinishArgs {
  DeltaShape s;
  const void *q, *k, *v, *a, *b, *dy;
  const float *u, *du, *dkf, *dk2, *dqf, *end, *S_ck, *dS_ck;
  int nc;
  float *gain;   // [B,H,T]
  void *dq, *dk, *dv, *da, *db;
};
int launch_delta_finish(int dtype, const FinishArgs &a, cudaStream_t st);   // dq, dk, dv, db, gain
int launch_delta_gate(int dtype, const FinishArgs &a, cudaStream_t st);     // da

}  // namespace esa
