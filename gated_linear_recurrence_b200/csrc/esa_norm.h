// esa_norm.h -- host-side interface between the layer norm's C ABI and its
// kernel units (one per I/O type).  Internal to the library.
#pragma once

#include <cuda_runtime.h>

namespace esa {

constexpr int kNormMaxN = 16384;    // the widest row: 1024 threads of 16 elements
constexpr int kNormFwdElems = 32;   // most elements a thread, forward and backward
constexpr int kNormBwdElems = 16;

// Threads of a row and vectors of a thread.
struct NormRow {
  int tpr, nv;
};

// A row of `nvec` vectors: part of a warp with one vector a thread while it
// fits, a warp with up to `most`, then as few threads as hold it with `most`.
inline NormRow norm_row(int nvec, int most) {
  int tpr = 4, nv = 1;
  while (tpr < 32 && tpr < nvec) tpr <<= 1;
  while (tpr >= 32 && tpr * most < nvec) tpr <<= 1;
  while (nv * tpr < nvec) nv <<= 1;
  return {tpr, tpr > 32 ? most : nv};
}

struct NormFwdArgs {
  const void *x, *res, *w, *c;
  void *y, *h;
  float2 *stats;
  long long rows, ld_x, ld_res;
  int N;
  float eps, n;   // n = N: sums are divided by it, so that a row of equal values has exactly their mean
};

struct NormBwdArgs {
  const void *dy, *h, *w, *dh;
  void *dx;
  const float2 *stats;
  void *dweight, *dbias;
  float *part;   // [gridDim.x][2][N]: dweight and dbias of each block's rows
  long long rows, ld_dy, ld_h, ld_dh;
  int N;
  float n;
};

// wide: the weight, the bias and their gradients are float32 (else the I/O
// type).  vec: elements per vector: 16 or 8 bytes' worth, or 1.
int norm_fwd_f32(int vec, const NormFwdArgs &a, cudaStream_t st);
int norm_fwd_f16(int vec, bool wide, const NormFwdArgs &a, cudaStream_t st);
int norm_fwd_bf16(int vec, bool wide, const NormFwdArgs &a, cudaStream_t st);
int norm_bwd_f32(int vec, const NormBwdArgs &a, int most, cudaStream_t st);
int norm_bwd_f16(int vec, bool wide, const NormBwdArgs &a, int most, cudaStream_t st);
int norm_bwd_bf16(int vec, bool wide, const NormBwdArgs &a, int most, cudaStream_t st);

}  // namespace esa
