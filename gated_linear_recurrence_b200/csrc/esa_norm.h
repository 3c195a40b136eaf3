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
// type).  vec: elements per vector: 16, 8, 4 or 2 bytes' worth.
int norm_fwd_f32(int vec, NormRow s, const NormFwdArgs &a, cudaStream_t st);
int norm_fwd_f16(int vec, NormRow s, bool wide, const NormFwdArgs &a, cudaStream_t st);
int norm_fwd_bf16(int vec, NormRow s, bool wide, const NormFwdArgs &a, cudaStream_t st);
int norm_bwd_f32(int vec, NormRow s, const NormBwdArgs &a, int most, cudaStream_t st);
int norm_bwd_f16(int vec, NormRow s, bool wide, const NormBwdArgs &a, int most, cudaStream_t st);
int norm_bwd_bf16(int vec, NormRow s, bool wide, const NormBwdArgs &a, int most, cudaStream_t st);

}  // namespace esa
