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
// row is shared by TPR threads (part of a warp, a warp, or a block of its
// own), each holding NV vectors of VEC elements: up to 32 elements a thread
// forward and 16 backward, where the column sums take as many registers
// again.  Few threads a row and many rows under way beat the opposite: what
// counts is the bytes in flight while other rows are being reduced.  The mean
// and the variance are two passes over the registers (the sum of squares of
// the differences, not of the values: a row far from zero keeps its variance),
// all in float32.
//
// The weight and bias gradients are sums over all rows: a thread owns the
// same columns of every row it visits and adds them up in float32 registers;
// the row groups of a block are joined in shared memory, each block writes
// one partial row, and a second kernel adds the partial rows in a fixed
// order, so the result does not change from run to run.
//
// Measured (B200, copy rate 6.53 TB/s), forward and backward, with a residual:
// 262144 x 128 float16 46 us (5.8 TB/s) and 46 (5.9); 65536 x 512 bfloat16 with
// float32 weights 43 (6.2) and 49 (5.5); 16384 x 2048 bfloat16 43 and 63.  The
// backward keeps its columns' weights in registers: read anew for every row it
// took 50 and 53.  Rows that start on 8 bytes only: 4099 x 5002 float32 38 and
// 63.  Rows that start anywhere: esa_norm_ragged.cuh.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

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

// A vector of the weight (or bias): WT elements, `VEC` of them, `fill` where
// there is no tensor.  Their own alignment is VEC elements of WT only where
// VEC sizeof(WT) <= 16, so a float32 weight next to 8 16-bit elements is read
// as two vectors.  Read-only loads: the compiler may issue them ahead of the
// row's stores (with plain loads a row's vectors waited for one another:
// 8000 x 4100 took 173 us forward).
template <typename P>
__device__ __forceinline__ P load_readonly(const P *p) {
  P v;
  if constexpr (sizeof(P) == 16) *reinterpret_cast<uint4 *>(&v) = __ldg(reinterpret_cast<const uint4 *>(p));
  else if constexpr (sizeof(P) == 8) *reinterpret_cast<uint2 *>(&v) = __ldg(reinterpret_cast<const uint2 *>(p));
  else if constexpr (sizeof(P) == 4) *reinterpret_cast<unsigned *>(&v) = __ldg(reinterpret_cast<const unsigned *>(p));
  else *reinterpret_cast<unsigned short *>(&v) = __ldg(reinterpret_cast<const unsigned short *>(p));
  return v;
}
template <typename WT, int VEC>
__device__ __forceinline__ void load_w(const void *base, int col, float (&x)[VEC], float fill) {
  const WT *p = static_cast<const WT *>(base) + col;
  constexpr int PER = VEC * sizeof(WT) > 16 ? 16 / sizeof(WT) : VEC;
#pragma unroll
  for (int i = 0; i < VEC; i += PER) {
    Pack<WT, PER> u;
    if (base != nullptr) u = load_readonly(reinterpret_cast<const Pack<WT, PER> *>(p + i));
#pragma unroll
    for (int j = 0; j < PER; ++j) x[i + j] = base != nullptr ? to_f(u.v[j]) : fill;
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

// Two sums with one exchange.
template <int TPR>
__device__ __forceinline__ void row_sum2(float &a, float &b, float2 (*red)[32], int &slot) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR > 32) {
    float2 *r = red[slot];
    slot ^= 1;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      a += r[i].x;
      b += r[i].y;
    }
  }
}

template <int TPR>
constexpr int norm_block() { return TPR > 32 ? TPR : 256; }

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
  const bool live = TPR > 32 || row < p.rows;   // a block of its own has a row
  int slot = 0;
  float f[NV][VEC];
  V vx[NV], vr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * VEC;
    if (live && col < p.N) {
      vx[i] = *reinterpret_cast<const V *>(x + row * p.ld_x + col);
      if (NV <= 2 && res) vr[i] = *reinterpret_cast<const V *>(res + row * p.ld_res + col);
    }
  }
  float s = 0.0f;
  if constexpr (NV <= 2) {
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
  } else {   // all loads first, no branch between them (30000 x 1000: 39 us, in the form above 49)
    if (res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * VEC;
        if (live && col < p.N) vr[i] = *reinterpret_cast<const V *>(res + row * p.ld_res + col);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) vx[i].v[j] = from_f<T>(to_f(vx[i].v[j]) + to_f(vr[i].v[j]));
        if (live && col < p.N) *reinterpret_cast<V *>(h + row * p.N + col) = vx[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = live && (i * TPR + lane) * VEC < p.N;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        f[i][j] = on ? to_f(vx[i].v[j]) : 0.0f;
        s += f[i][j];
      }
    }
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
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * VEC;
    if (live && col < p.N) {
      float w[VEC], c[VEC];
      load_w<WT, VEC>(p.w, col, w, 1.0f);
      load_w<WT, VEC>(p.c, col, c, 0.0f);
      V o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) o.v[j] = from_f<T>(fmaf(f[i][j] * rstd, w[j], c[j]));
      *reinterpret_cast<V *>(y + row * p.N + col) = o;
    }
  }
  if (p.stats && live && lane == 0) p.stats[row] = make_float2(mean, rstd);
}

// A thread's vectors of the rows under way, in shared memory that no other
// thread touches: [stage][h, dy, dh][NV][thread].  Single elements are loaded
// into registers instead, one row at a time: a copy instruction for each costs
// more than it hides (4099 x 5001 float32: 142 us staged, 90 in registers).
template <typename V>
constexpr bool norm_staged() { return sizeof(V) >= 8; }
template <typename V, int NV, int BLOCK>
constexpr int norm_stage_bytes() { return norm_staged<V>() ? 3 * NV * BLOCK * static_cast<int>(sizeof(V)) : 0; }
// Rows under way: two, one where two do not fit in shared memory.
template <typename V, int NV, int BLOCK>
constexpr int norm_stages() { return 2 * norm_stage_bytes<V, NV, BLOCK>() <= 200 * 1024 ? 2 : 1; }

template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
}

template <typename T, typename WT, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(norm_block<TPR>()) norm_bwd_kernel(NormBwdArgs p) {
  constexpr int BLOCK = norm_block<TPR>();
  constexpr int GROUPS = TPR > 32 ? 1 : BLOCK / TPR;
  using V = Pack<T, VEC>;
  constexpr bool kStaged = norm_staged<V>();
  constexpr int kStages = kStaged ? norm_stages<V, NV, BLOCK>() : 1;
  extern __shared__ __align__(16) unsigned char stage_bytes[];
  __shared__ float2 red[2][32];
  V *stage = reinterpret_cast<V *>(stage_bytes) + threadIdx.x;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const T *dy = static_cast<const T *>(p.dy), *h = static_cast<const T *>(p.h), *dh = static_cast<const T *>(p.dh);
  T *dx = static_cast<T *>(p.dx);
  int slot = 0;
  float aw[NV][VEC], ac[NV][VEC], w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * VEC;
    if (col < p.N) load_w<WT, VEC>(p.w, col, w[i], 1.0f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[i][j] = ac[i][j] = 0.0f;
  }
  const long long stride = static_cast<long long>(gridDim.x) * GROUPS;
  float2 stats[kStages];
  V rh[kStaged ? 1 : NV], ry[kStaged ? 1 : NV];
  auto fetch = [&](long long row, int k) {
    stats[k] = make_float2(0.0f, 0.0f);
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * VEC;
        if constexpr (!kStaged) {
          if (col < p.N) {
            rh[i] = *reinterpret_cast<const V *>(h + row * p.ld_h + col);
            ry[i] = *reinterpret_cast<const V *>(dy + row * p.ld_dy + col);
          }
        } else if (col < p.N) {
          V *s = stage + (k * 3 * NV + i) * BLOCK;
          copy_async<sizeof(V)>(s, h + row * p.ld_h + col);
          copy_async<sizeof(V)>(s + NV * BLOCK, dy + row * p.ld_dy + col);
          if (dh) copy_async<sizeof(V)>(s + 2 * NV * BLOCK, dh + row * p.ld_dh + col);
        }
      }
      stats[k] = p.stats[row];
    }
    if constexpr (kStaged) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  long long row = static_cast<long long>(blockIdx.x) * GROUPS + group;
#pragma unroll
  for (int k = 0; k < kStages; ++k) fetch(row + k * stride, k);
  // Every thread of a block makes the same number of turns (the row sums of
  // TPR > 32 are barriers; those of TPR <= 32 are whole-warp shuffles).
  for (long long base = static_cast<long long>(blockIdx.x) * GROUPS; base < p.rows;) {
#pragma unroll
    for (int k = 0; k < kStages; ++k, base += stride, row += stride) {
      if (base >= p.rows) break;
      const bool live = row < p.rows;
      if constexpr (kStaged) asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      const float2 st = stats[k];
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * VEC;
        if (live && col < p.N) {
          const V *s = stage + (k * 3 * NV + i) * BLOCK;
          V vh, vy;
          if constexpr (kStaged) {
            vh = s[0];
            vy = s[NV * BLOCK];
          } else {
            vh = rh[i];
            vy = ry[i];
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float d = to_f(vy.v[j]), n = (to_f(vh.v[j]) - st.x) * st.y, g = d * w[i][j];
            aw[i][j] = fmaf(d, n, aw[i][j]);
            ac[i][j] += d;
            s1 += g;
            s2 = fmaf(g, n, s2);
          }
        }
      }
      row_sum2<TPR>(s1, s2, red, slot);
      s1 /= p.n;
      s2 /= p.n;
      // the products again, from the row as it was read: cheaper than the registers to keep them
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * TPR + lane) * VEC;
        if (live && col < p.N) {
          const V *s = stage + (k * 3 * NV + i) * BLOCK;
          V vh, vy, vd, o;
          if constexpr (kStaged) {
            vh = s[0];
            vy = s[NV * BLOCK];
            if (dh) vd = s[2 * NV * BLOCK];
          } else {
            vh = rh[i];
            vy = ry[i];
            if (dh) vd = *reinterpret_cast<const V *>(dh + row * p.ld_dh + col);
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float n = (to_f(vh.v[j]) - st.x) * st.y;
            float v = st.y * (to_f(vy.v[j]) * w[i][j] - s1 - n * s2);
            if (dh) v += to_f(vd.v[j]);
            o.v[j] = from_f<T>(v);
          }
          *reinterpret_cast<V *>(dx + row * p.N + col) = o;
        }
      }
      fetch(row + kStages * stride, k);
    }
  }
  if constexpr (kStaged) asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (p.part == nullptr) return;
  float *join = reinterpret_cast<float *>(stage_bytes);   // BLOCK * VEC floats, once the rows are done
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
  static constexpr int kMost = kNormFwdElems / VEC;
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

// Blocks of the backward: as many as the device holds at once, never more than
// there are rows to share out, nor than the workspace has partial rows for.
template <typename T, typename WT, int VEC>
struct RunBwd {
  static constexpr int kMost = kNormBwdElems / VEC;
  const NormBwdArgs &a;
  int most;
  int *grid;
  cudaStream_t st;
  template <int NV, int TPR>
  int run() const {
    constexpr int BLOCK = norm_block<TPR>(), GROUPS = BLOCK / TPR;
    constexpr int rows = norm_stages<Pack<T, VEC>, NV, BLOCK>() * norm_stage_bytes<Pack<T, VEC>, NV, BLOCK>(), sums = GROUPS > 1 ? BLOCK * VEC * 4 : 0;
    constexpr int smem = rows > sums ? rows : sums;
    auto kern = norm_bwd_kernel<T, WT, VEC, NV, TPR>;
    static std::atomic<int> resident{0};   // blocks an SM holds: the same on every device the library runs on
    int per = resident.load(std::memory_order_relaxed);
    if (smem > 40 * 1024) {   // 48 KB with the static part
      const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
      if (rc) return rc;
    }
    if (per == 0) {
      const int rc = runtime_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, BLOCK, smem));
      if (rc) return rc;
      resident.store(per = per > 0 ? per : 1, std::memory_order_relaxed);
    }
    const long long need = (a.rows + GROUPS - 1) / GROUPS;
    long long full = static_cast<long long>(sm_count()) * per;
    if (full > most) full = most;
    *grid = static_cast<int>(need < full ? need : full);
    kern<<<*grid, BLOCK, smem, st>>>(a);
    return runtime_status(cudaGetLastError());
  }
};

// The instantiation for a row's shape (norm_row): a warp or less has any
// number of vectors a thread up to the most, more threads only the most.
template <int VEC, int NV, int TPR, typename F>
int run_if(const F &f) {
  if constexpr (NV <= F::kMost && (TPR <= 32 || (NV == F::kMost && TPR * VEC * NV / 2 < kNormMaxN)))
    return f.template run<NV, TPR>();
  return ESA_ERR_UNSUPPORTED;
}
template <int VEC, int TPR, typename F>
int by_nv(int nv, const F &f) {
  switch (nv) {
    case 1: return run_if<VEC, 1, TPR>(f);
    case 2: return run_if<VEC, 2, TPR>(f);
    case 4: return run_if<VEC, 4, TPR>(f);
    case 8: return run_if<VEC, 8, TPR>(f);
    case 16: return run_if<VEC, 16, TPR>(f);
    case 32: return run_if<VEC, 32, TPR>(f);
    default: return ESA_ERR_UNSUPPORTED;
  }
}
template <int VEC, typename F>
int by_shape(NormRow s, const F &f) {
  switch (s.tpr) {
    case 4: return run_if<VEC, 1, 4>(f);
    case 8: return run_if<VEC, 1, 8>(f);
    case 16: return run_if<VEC, 1, 16>(f);
    case 32: return by_nv<VEC, 32>(s.nv, f);
    case 64: return by_nv<VEC, 64>(s.nv, f);
    case 128: return by_nv<VEC, 128>(s.nv, f);
    case 256: return by_nv<VEC, 256>(s.nv, f);
    case 512: return by_nv<VEC, 512>(s.nv, f);
    case 1024: return by_nv<VEC, 1024>(s.nv, f);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace
}  // namespace esa
