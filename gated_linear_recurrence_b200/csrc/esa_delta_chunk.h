// esa_delta_chunk.h -- the chunked gated delta rule: its arrays in the
// workspace and the launches.  Internal to the library.
//
// A head's sequence is cut into chunks of 64 tokens (the last one padded with
// tokens that neither write nor forget).  Chunk c = head * nc + n, head =
// b H + h, has a record of ChunkRecord<D>::bytes bytes, written by the first
// kernel in the order and with the swizzle in which later kernels hold it in
// shared memory, so that a copy of it is linear:
//   tok    [kTokRows][64] float32  per-token factors (rows below)
//   fac    [8] float32             the chunk's factors, `Fac` below
//   k, q   [64][D] float16         keys and queries, each tile scaled by a power of two (exact)
//   th, tl 10 blocks 16 x 16       two float16 terms of T = (1 + M)^-1 (lower triangle), scaled likewise
//   ph, pl 10 blocks 16 x 16       two float16 terms of P_ij = e^{Gi-Gj} q_i.k_j (j <= i), scaled likewise
//   g      [2][64] float32         running sums of log alpha, two terms
// and, kept for the backward or written by it,
//   u16, r16   [64][D] float16     u and du (token rows), one power of two per 16 channels
//   u16l, r16l [64][D] float16     their second terms (float16 tensors)
//   s16, ds16  [D][D] float16      state entering the chunk and gradient of the state leaving it
//                                  (row: value channel), one power of two per 16 rows
//   slice      [4][8] float32      inverses of those powers of two (0 for a group of zeros, NaN for one that is not finite)
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>

#include "esa_delta.h"

namespace esa {

constexpr int kChunk = 64;
enum { kTokBeta = 0, kTokX = 1, kTokL = 2, kTokY = 3, kTokRows = 4 };
//   kTokBeta  beta (0 where the key or gate is not finite)
//   kTokX     beta e^G          (what the state's prediction K S is multiplied by; 0 where the key is not finite)
//   kTokL     e^{G_last - G}    (what u is multiplied by before it is added to the state; the same)
//   kTokY     e^G               (what the state's output Q S is multiplied by; NaN where the query is not finite)
// The keys' and queries' scales are not multiplied into the factors: a product
// of three scales can leave float32's range where the value itself does not.

// The factors of a chunk: e^{G_last}, 1/scale of T, 1/scale of P, first token
// whose key or gate is not finite (or 64), 1/scale of the keys, of the queries, scale of P,
// and 1/scale of T again for the backward, NaN where a key, query or gate of the chunk is not finite.
enum { kFacLast = 0, kFacK = 4, kFacQ = 5 };
struct Fac {
  float last, t, p, first, k, q, ps, tb;
};
__device__ __forceinline__ Fac load_fac(const void *at) {
  const float4 a = static_cast<const float4 *>(at)[0], b = static_cast<const float4 *>(at)[1];
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

constexpr int kTriangle = 10 * 512;   // bytes of a triangle (kTriBytes of esa_mma.cuh)

template <int D>
struct ChunkRecord {
  static constexpr int tok = 0, fac = kTokRows * 64 * 4, k = fac + 128, q = k + 64 * D * 2, th = q + 64 * D * 2,
                       tl = th + kTriangle, ph = tl + kTriangle, pl = ph + kTriangle, g = pl + kTriangle,
                       bytes = g + 512;
};

enum { kSliceU = 0, kSliceR = 8, kSliceS = 16, kSliceDs = 24 };   // rows of `slice`

struct ChunkArrays {
  unsigned char *rec;
  __half *u16, *r16, *u16l, *r16l, *s16, *ds16;
  float *slice;
  int nc;
};

struct ChunkArgs {
  DeltaShape s;
  ChunkArrays w;
  const void *q, *k, *v, *a, *b, *dy;
  void *y, *dq, *dk, *dv, *da, *db;
  const float *S_in;   // S_init, or dS_final for the backward chain
  float *S_out;        // S_final, or dS_init
  bool keep;
  float least, iscale;   // of the scale: the least unit of an output (see output_unit), its inverse
};

// A power of two of 2^-120 / min(|scale|, 1) to twice that, 1 at most: its product with the scale keeps its digits too.
inline float least_output_unit(float scale) {
  int e = 0;
  if (scale != 0.0f && fabsf(scale) < 1.0f) frexpf(scale, &e);   // 2^(e - 1) <= |scale| < 2^e
  return ldexpf(1.0f, e > -119 ? -119 - e : 0);
}

int launch_chunk_prep(int dtype, const ChunkArgs &a, cudaStream_t st);
int launch_chunk_fwd(int dtype, const ChunkArgs &a, cudaStream_t st);
int launch_chunk_bwd(int dtype, const ChunkArgs &a, cudaStream_t st);    // dv, dS_init, du
int launch_chunk_grad(int dtype, const ChunkArgs &a, cudaStream_t st);   // dq, dk, da, db

// The chains with a slice of 16 value channels shared by four warps (D = 64, 128).
int launch_split_fwd(int dtype, const ChunkArgs &a, cudaStream_t st);
int launch_split_bwd(int dtype, const ChunkArgs &a, cudaStream_t st);

// How the chains spread a head over the device.
enum ChainPlan { kChainWhole, kChainHalves, kChainSplit };
ChainPlan chain_plan(int heads, int D);

}  // namespace esa
