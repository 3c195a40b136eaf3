// esa_norm.cuh -- kernels of the layer norm over the last axis, with the
// residual addition before it, forward and backward (sm_100a).
//
//   h = x + residual (rounded to the I/O type: it is the new residual stream)
//   y = n w + c,  n = (h - mean) rstd,  rstd = 1 / sqrt(mean((h - mean)^2) + eps)
//   dx = rstd (g - mean(g) - n mean(g n)) + dh,  g = dy w
//   dw = sum_rows dy n,  dc = sum_rows dy
//
// Both directions are bound by memory traffic: each tensor is read once and
// written once, so a row lives in registers from its load to its store.  A
// row is shared by TPR threads (a power of two: part of a warp, a warp, or
// several warps), each holding NV vectors of VEC elements; the smallest TPR
// that keeps a thread at one to two 16-byte vectors wins for short rows
// (more rows in flight), and longer rows take more threads.  The mean and
// the variance are two passes over the registers (the sum of squares of the
// differences, not of the values: a row far from zero keeps its variance),
// all in float32.
//
// The weight and bias gradients are sums over all rows: a thread owns the
// same columns of every row it visits and adds them up in float32 registers;
// the row groups of a block are joined in shared memory, each block writes
// one partial row, and a second kernel adds the partial rows in a fixed
// order, so the result does not change from run to run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstddef>

#include "esa.h"
#include "esa_host.h"
#include "esa_norm.h"

namespace esa {
namespace {

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

// A vector of the weight (or bias): WT elements, `VEC` of them; their own
// alignment is VEC elements of WT only where VEC sizeof(WT) <= 16, so a
// float32 weight next to 8 16-bit elements is read as two vectors.
template <typename WT, int VEC>
__device__ __forceinline__ void load_w(const WT *p, float (&x)[VEC], float fill) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = fill;
    return;
  }
  constexpr int PER = VEC * sizeof(WT) > 16 ? 16 / sizeof(WT) : VEC;
#pragma unroll
  for (int i = 0; i < VEC; i += PER) {
    const Pack<WT, PER> u = *reinterpret_cast<const Pack<WT, PER> *>(p + i);
#pragma unroll
    for (int j = 0; j < PER; ++j) x[i + j] = to_f(u.v[j]);
  }
}

// Sum over the TPR threads of a row.  Rows of more than a warp go through
// `red` (two slots of 32 floats, used in turn so that one barrier per sum is
// enough).
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float (*red)[32], int &slot) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    float *r = red[slot];
    slot ^= 1;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) s += r[i];
  }
  return s;
}

template <int TPR>
constexpr int norm_block() { return TPR > 256 ? TPR : 256; }

template <typename T, typename WT, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(norm_block<TPR>()) norm_fwd_kernel(NormFwdArgs p) {
  constexpr int BLOCK = norm_block<TPR>();
  constexpr int GROUPS = TPR > 32 ? 1 : BLOCK / TPR;   // rows of a block at a time (TPR > 32: BLOCK == TPR)
  static_assert(TPR <= 32 || BLOCK == TPR, "a row of several warps takes the whole block");
  __shared__ float red[2][32];
  using V = Pack<T, VEC>;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.res);
  T *y = static_cast<T *>(p.y), *h = static_cast<T *>(p.h);
  const long long row = static_cast<long long>(blockIdx.x) * GROUPS + group;
  const bool live = row < p.rows;
  int slot = 0;
  float f[NV][VEC];
  V vx[NV], vr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * VEC;
    if (live && col < p.N) {
      vx[i] = *reinterpret_cast<const V *>(x + row * p.ld_x + col);
      if (res) vr[i] = *reinterpret_cast<const V *>(res + row * p.ld_res + col);
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * VEC;
    const bool on = live && col < p.N;
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[i][j] = on ? to_f(vx[i].v[j]) : 0.0f;
    if (res && on) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        vx[i].v[j] = from_f<T>(f[i][j] + to_f(vr[i].v[j]));
        f[i][j] = to_f(vx[i].v[j]);
      }
      *reinterpret_cast<V *>(h + row * p.N + col) = vx[i];
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += f[i][j];
  }
  const float mean = row_sum<TPR>(s, red, slot) / p.n;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool on = (i * TPR + lane) * VEC < p.N;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      f[i][j] -= mean;
      if (on) s = fmaf(f[i][j], f[i][j], s);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(s, red, slot) / p.n + p.eps);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * VEC;
    if (col < p.N) {
      float w[VEC], c[VEC];
      load_w<WT, VEC>(p.w ? static_cast<const WT *>(p.w) + col : nullptr, w, 1.0f);
      load_w<WT, VEC>(p.c ? static_cast<const WT *>(p.c) + col : nullptr, c, 0.0f);
      V o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) o.v[j] = from_f<T>(fmaf(f[i][j] * rstd, w[j], c[j]));
      *reinterpret_cast<V *>(y + row * p.N + col) = o;
    }
  }
  if (p.stats && lane == 0) p.stats[row] = make_float2(mean, rstd);
}

template <typename T, typename WT, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(norm_block<TPR>()) norm_bwd_kernel(NormBwdArgs p) {
  constexpr int BLOCK = norm_block<TPR>();
  constexpr int GROUPS = TPR > 32 ? 1 : BLOCK / TPR;
  __shared__ float red[2][32];
  __shared__ float join[TPR > 32 ? 1 : BLOCK * VEC];
  using V = Pack<T, VEC>;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const T *dy = static_cast<const T *>(p.dy), *h = static_cast<const T *>(p.h), *dh = static_cast<const T *>(p.dh);
  T *dx = static_cast<T *>(p.dx);
  int slot = 0;
  float aw[NV][VEC], ac[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[i][j] = ac[i][j] = 0.0f;
  const long long stride = static_cast<long long>(gridDim.x) * GROUPS;
  // Every thread of a block makes the same number of turns (the row sums of
  // TPR > 32 are barriers; those of TPR <= 32 are whole-warp shuffles).
  for (long long base = static_cast<long long>(blockIdx.x) * GROUPS; base < p.rows; base += stride) {
    const long long row = base + group;
    const bool live = row < p.rows;
    V vh[NV], vy[NV], vd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + lane) * VEC;
      if (live && col < p.N) {
        vh[i] = *reinterpret_cast<const V *>(h + row * p.ld_h + col);
        vy[i] = *reinterpret_cast<const V *>(dy + row * p.ld_dy + col);
        if (dh) vd[i] = *reinterpret_cast<const V *>(dh + row * p.ld_dh + col);
      }
    }
    const float2 st = live ? p.stats[row] : make_float2(0.0f, 0.0f);
    float s1 = 0.0f, s2 = 0.0f;
    float g[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + lane) * VEC;
      if (live && col < p.N) {
        float w[VEC];
        load_w<WT, VEC>(p.w ? static_cast<const WT *>(p.w) + col : nullptr, w, 1.0f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = to_f(vy[i].v[j]), n = (to_f(vh[i].v[j]) - st.x) * st.y;
          aw[i][j] = fmaf(d, n, aw[i][j]);
          ac[i][j] += d;
          g[i][j] = d * w[j];
          s1 += g[i][j];
          s2 = fmaf(g[i][j], n, s2);
        }
      }
    }
    s1 = row_sum<TPR>(s1, red, slot) / p.n;
    s2 = row_sum<TPR>(s2, red, slot) / p.n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + lane) * VEC;
      if (live && col < p.N) {
        V o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float n = (to_f(vh[i].v[j]) - st.x) * st.y;
          float v = st.y * (g[i][j] - s1 - n * s2);
          if (dh) v += to_f(vd[i].v[j]);
          o.v[j] = from_f<T>(v);
        }
        *reinterpret_cast<V *>(dx + row * p.N + col) = o;
      }
    }
  }
  if (p.part == nullptr) return;
  float *pw = p.part + static_cast<long long>(blockIdx.x) * 2 * p.N, *pc = pw + p.N;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * VEC;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float *out = which ? pc : pw;
      float(&acc)[VEC] = which ? ac[i] : aw[i];
      if constexpr (GROUPS > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) join[(group * TPR + lane) * VEC + j] = acc[j];
        __syncthreads();
        // columns of this vector index: TPR * VEC of them, summed over the groups in order
        for (int k = threadIdx.x; k < TPR * VEC; k += BLOCK) {
          const int c = i * TPR * VEC + k;
          float s = 0.0f;
          for (int gr = 0; gr < GROUPS; ++gr) s += join[gr * TPR * VEC + k];
          if (c < p.N) out[c] = s;
        }
      } else if (col < p.N) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) out[col + j] = acc[j];
      }
    }
  }
}

// Sum of the partial rows, columns of dweight then of dbias: a block takes 32
// columns, its 32 warps every 32nd partial row each, then the 32 sums of a
// column are added in order.
template <typename WT>
__global__ void __launch_bounds__(1024) norm_fold_kernel(const float *part, int nparts, int N, WT *dw, WT *dc) {
  __shared__ float s[32][33];
  const int cx = threadIdx.x & 31, wy = threadIdx.x >> 5;
  const long long col = static_cast<long long>(blockIdx.x) * 32 + cx, two_n = 2ll * N;
  float acc = 0.0f;
  if (col < two_n)
    for (int r = wy; r < nparts; r += 32) acc += part[r * two_n + col];
  s[wy][cx] = acc;
  __syncthreads();
  if (wy == 0 && col < two_n) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][cx];
    if (col < N) {
      if (dw) dw[col] = from_f<WT>(t);
    } else if (dc) {
      dc[col - N] = from_f<WT>(t);
    }
  }
}

// ---- dispatch of one I/O type ----------------------------------------------
template <typename T, typename WT, int VEC>
struct RunFwd {
  const NormFwdArgs &a;
  cudaStream_t st;
  template <int NV, int TPR>
  int run() const {
    constexpr int GROUPS = TPR > 32 ? 1 : norm_block<TPR>() / TPR;
    const long long blocks = (a.rows + GROUPS - 1) / GROUPS;
    norm_fwd_kernel<T, WT, VEC, NV, TPR><<<static_cast<unsigned>(blocks), norm_block<TPR>(), 0, st>>>(a);
    return runtime_status(cudaGetLastError());
  }
};

template <typename T, typename WT, int VEC>
struct RunBwd {
  const NormBwdArgs &a;
  int grid;
  cudaStream_t st;
  template <int NV, int TPR>
  int run() const {
    norm_bwd_kernel<T, WT, VEC, NV, TPR><<<grid, norm_block<TPR>(), 0, st>>>(a);
    return runtime_status(cudaGetLastError());
  }
};

// The instantiation for a row's shape; shapes that no row of at most
// kNormMaxN elements of this vector width takes are not compiled.
template <int VEC, int NV, int TPR, typename F>
int run_if(const F &f) {
  if constexpr (NV == 1 || TPR * VEC * NV / 2 < kNormMaxN) return f.template run<NV, TPR>();
  return ESA_ERR_UNSUPPORTED;
}
template <int VEC, typename F>
int by_shape(NormRow s, const F &f) {
  switch (s.tpr * 32 + s.nv) {
    case 4 * 32 + 1: return run_if<VEC, 1, 4>(f);
    case 8 * 32 + 1: return run_if<VEC, 1, 8>(f);
    case 16 * 32 + 1: return run_if<VEC, 1, 16>(f);
    case 32 * 32 + 1: return run_if<VEC, 1, 32>(f);
    case 32 * 32 + 2: return run_if<VEC, 2, 32>(f);
    case 32 * 32 + 4: return run_if<VEC, 4, 32>(f);
    case 256 * 32 + 1: return run_if<VEC, 1, 256>(f);
    case 256 * 32 + 2: return run_if<VEC, 2, 256>(f);
    case 512 * 32 + 2: return run_if<VEC, 2, 512>(f);
    case 1024 * 32 + 2: return run_if<VEC, 2, 1024>(f);
    case 1024 * 32 + 4: return run_if<VEC, 4, 1024>(f);
    case 1024 * 32 + 8: return run_if<VEC, 8, 1024>(f);
    case 1024 * 32 + 16: return run_if<VEC, 16, 1024>(f);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

template <typename T, typename WT>
int norm_fwd_typed(int vec, NormRow s, const NormFwdArgs &a, cudaStream_t st) {
  if (vec == 16 / static_cast<int>(sizeof(T))) return by_shape<16 / sizeof(T)>(s, RunFwd<T, WT, 16 / sizeof(T)>{a, st});
  if constexpr (sizeof(T) == 2)
    if (vec == 2) return by_shape<2>(s, RunFwd<T, WT, 2>{a, st});
  return by_shape<1>(s, RunFwd<T, WT, 1>{a, st});
}

template <typename T, typename WT>
int norm_bwd_typed(int vec, NormRow s, const NormBwdArgs &a, int grid, cudaStream_t st) {
  int rc;
  if (vec == 16 / static_cast<int>(sizeof(T))) rc = by_shape<16 / sizeof(T)>(s, RunBwd<T, WT, 16 / sizeof(T)>{a, grid, st});
  else if (sizeof(T) == 2 && vec == 2) rc = by_shape<2>(s, RunBwd<T, WT, 2>{a, grid, st});
  else rc = by_shape<1>(s, RunBwd<T, WT, 1>{a, grid, st});
  if (rc || a.part == nullptr) return rc;
  norm_fold_kernel<WT><<<(2 * a.N + 31) / 32, 1024, 0, st>>>(a.part, grid, a.N, static_cast<WT *>(a.dweight),
                                                             static_cast<WT *>(a.dbias));
  return runtime_status(cudaGetLastError());
}

}  // namespace
}  // namespace esa
