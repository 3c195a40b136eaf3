// esa_norm_ragged.cuh -- the layer norm of rows that do not all start on 16
// bytes (odd widths, offset views), sm_100a.
//
// The mathematics is esa_norm.cuh's.  Rows are read and written in the 16-byte
// units of memory all the same: a thread's unit i begins at column
// (i TPR + lane) VEC - off, off elements being the distance of the row's first
// element from a unit.  The first and the last unit of a row hold elements of
// its neighbours, which are set to zero on arrival and not written; units that
// would reach over the ends of the tensor are loaded by element.  off depends
// on the row only through row * ld mod VEC, and the rows of a thread are a
// multiple of VEC apart: a thread has the same columns in every row it visits,
// so it keeps their weights in registers and adds up their gradients there.
// Rows are staged ahead in shared memory, each thread's units its own.
//
// Measured: 4099 x 5001 float32 50 us forward (3.3 TB/s), 55 backward (4.5);
// 3000 x 8001 float16 46 and 75; 200000 x 129 float16 75 and 97.  Element by
// element (the kernels of esa_norm.cuh with VEC = 1): 60 and 90, 115 and 224,
// 71 and 96.  With whole rows copied through shared memory, elements dealt to
// threads there: 68 and 115, bound by some 70 instructions an element.  The
// forward without staging, a block a row, weights read anew: 61, 88, 108.
// Half the elements a thread: 56 and 68, 49 and 71.
#pragma once

#include <climits>
#include <initializer_list>

#include "esa_norm.cuh"

namespace esa {
namespace {

// Unit of VEC elements at element `at` of a tensor of `end` elements, column
// `col` of its row, into a thread's own place in shared memory.
template <typename V, typename T, int VEC>
__device__ __forceinline__ void unit_fetch(V *s, const T *base, long long at, bool inside, int col, int N) {
  if (inside || (col >= 0 && col + VEC <= N)) {
    copy_async<16>(s, base + at);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (col + j >= 0 && col + j < N) s->v[j] = base[at + j];
  }
}
template <typename V, typename T, int VEC>
__device__ __forceinline__ void unit_mask(V &v, int col, int N) {
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (col + j < 0 || col + j >= N) v.v[j] = from_f<T>(0.0f);
}
template <typename V, typename T, int VEC>
__device__ __forceinline__ void unit_store(T *dst, const V &v, int col, int N) {
  if (col >= 0 && col + VEC <= N) {
    *reinterpret_cast<V *>(dst) = v;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (col + j >= 0 && col + j < N) dst[j] = v.v[j];
  }
}

// Sums over the threads of a row; of more than a warp each warp adds the
// warps' sums for itself (with 16 warps and more, cheaper than every thread
// adding all of them).
template <int TPR>
__device__ __forceinline__ float ragged_sum(float a, float (*red)[32], int &slot) {
  a = row_sum<(TPR < 32 ? TPR : 32)>(a, red, slot);
  if constexpr (TPR > 32) {
    float *r = red[slot];
    slot ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) r[threadIdx.x >> 5] = a;
    __syncthreads();
    a = row_sum<TPR / 32>(r[lane & (TPR / 32 - 1)], red, slot);
  }
  return a;
}
template <int TPR>
__device__ __forceinline__ void ragged_sum2(float &a, float &b, float2 (*red)[32], int &slot) {
  row_sum2<(TPR < 32 ? TPR : 32)>(a, b, red, slot);
  if constexpr (TPR > 32) {
    float2 *r = red[slot];
    slot ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) r[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 v = r[lane & (TPR / 32 - 1)];
    a = v.x;
    b = v.y;
    row_sum2<TPR / 32>(a, b, red, slot);
  }
}

template <typename T, typename WT, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(norm_block<TPR>()) norm_fwd_ragged_kernel(NormFwdArgs p, int stages) {
  constexpr int BLOCK = norm_block<TPR>(), GROUPS = BLOCK / TPR;
  using V = Pack<T, VEC>;
  extern __shared__ __align__(16) unsigned char stage_bytes[];
  __shared__ float red[2][32];
  V *stage = reinterpret_cast<V *>(stage_bytes) + threadIdx.x;   // [stage][x, residual][NV][thread]
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR, ins = p.res ? 2 : 1;
  const T *x = static_cast<const T *>(p.x), *res = static_cast<const T *>(p.res);
  T *y = static_cast<T *>(p.y), *h = static_cast<T *>(p.h);
  const long long stride = static_cast<long long>(gridDim.x) * GROUPS;
  long long row = static_cast<long long>(blockIdx.x) * GROUPS + group;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x + row * p.ld_x) & 15) / static_cast<int>(sizeof(T));
  auto col_of = [&](int i) { return (i * TPR + lane) * VEC - off; };
  auto used = [&](int col) { return col + VEC > 0 && col < p.N; };
  auto whole = [&](int col) { return col >= 0 && col + VEC <= p.N; };
  float w[NV][VEC], c[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int col = col_of(i) + j;
      const bool on = col >= 0 && col < p.N;
      w[i][j] = on && p.w ? to_f(load_readonly(static_cast<const WT *>(p.w) + col)) : 1.0f;
      c[i][j] = on && p.c ? to_f(load_readonly(static_cast<const WT *>(p.c) + col)) : 0.0f;
    }
  const int edge = (VEC + p.N - 1) / p.N;   // rows, at least N apart, that hold a unit
  auto fetch = [&](long long r, int k) {
    if (r < p.rows) {
      const bool inside = r >= edge && r < p.rows - edge;   // units that reach into other rows stay in the tensor
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = col_of(i);
        V *s = stage + (k * ins * NV + i) * BLOCK;
        if (used(col)) {
          unit_fetch<V, T, VEC>(s, x, r * p.ld_x + col, inside, col, p.N);
          if (res) unit_fetch<V, T, VEC>(s + NV * BLOCK, res, r * p.ld_res + col, inside, col, p.N);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int slot = 0, k = 0;
  for (int j = 0; j < stages; ++j) fetch(row + j * stride, j);
  // Every thread of a block makes the same number of turns (see norm_bwd_kernel).
  for (long long base = static_cast<long long>(blockIdx.x) * GROUPS; base < p.rows; base += stride, row += stride) {
    const bool live = row < p.rows;
    if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    float f[NV][VEC], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col_of(i);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i][j] = 0.0f;
      if (live && used(col)) {
        const V *at = stage + (k * ins * NV + i) * BLOCK;
        V v = at[0];
        if (res) {
          const V r = at[NV * BLOCK];
#pragma unroll
          for (int j = 0; j < VEC; ++j) v.v[j] = from_f<T>(to_f(v.v[j]) + to_f(r.v[j]));
          unit_store<V, T, VEC>(h + row * p.N + col, v, col, p.N);
        }
        if (!whole(col)) unit_mask<V, T, VEC>(v, col, p.N);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          f[i][j] = to_f(v.v[j]);
          s += f[i][j];
        }
      }
    }
    fetch(row + stages * stride, k);
    k = k + 1 == stages ? 0 : k + 1;
    const float mean = ragged_sum<TPR>(s, red, slot) / p.n;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col_of(i);
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[i][j] -= mean;
      if (whole(col)) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) s = fmaf(f[i][j], f[i][j], s);
      } else if (used(col)) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (col + j >= 0 && col + j < p.N) s = fmaf(f[i][j], f[i][j], s);
      }
    }
    const float rstd = 1.0f / sqrtf(ragged_sum<TPR>(s, red, slot) / p.n + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col_of(i);
      if (live && used(col)) {
        V o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.v[j] = from_f<T>(fmaf(f[i][j] * rstd, w[i][j], c[i][j]));
        unit_store<V, T, VEC>(y + row * p.N + col, o, col, p.N);
      }
    }
    if (p.stats && live && lane == 0) p.stats[row] = make_float2(mean, rstd);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, typename WT, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(norm_block<TPR>()) norm_bwd_ragged_kernel(NormBwdArgs p, int stages) {
  constexpr int BLOCK = norm_block<TPR>(), GROUPS = BLOCK / TPR;
  using V = Pack<T, VEC>;
  extern __shared__ __align__(16) unsigned char stage_bytes[];
  __shared__ float2 red[2][32];
  V *stage = reinterpret_cast<V *>(stage_bytes) + threadIdx.x;   // [stage][h, dy, dh][NV][thread]
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR, ins = p.dh ? 3 : 2;
  const T *h = static_cast<const T *>(p.h), *dy = static_cast<const T *>(p.dy), *dh = static_cast<const T *>(p.dh);
  T *dx = static_cast<T *>(p.dx);
  const long long stride = static_cast<long long>(gridDim.x) * GROUPS;
  long long row = static_cast<long long>(blockIdx.x) * GROUPS + group;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(h + row * p.ld_h) & 15) / static_cast<int>(sizeof(T));
  auto col_of = [&](int i) { return (i * TPR + lane) * VEC - off; };
  auto used = [&](int col) { return col + VEC > 0 && col < p.N; };
  float w[NV][VEC], aw[NV][VEC], ac[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int col = col_of(i) + j;
      w[i][j] = col >= 0 && col < p.N && p.w ? to_f(load_readonly(static_cast<const WT *>(p.w) + col)) : 1.0f;
      aw[i][j] = ac[i][j] = 0.0f;
    }
  const int edge = (VEC + p.N - 1) / p.N;   // rows, at least N apart, that hold a unit
  auto fetch = [&](long long r, int k) {
    if (r < p.rows) {
      const bool inside = r >= edge && r < p.rows - edge;   // units that reach into other rows stay in the tensor
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = col_of(i);
        V *s = stage + (k * ins * NV + i) * BLOCK;
        if (used(col)) {
          unit_fetch<V, T, VEC>(s, h, r * p.ld_h + col, inside, col, p.N);
          unit_fetch<V, T, VEC>(s + NV * BLOCK, dy, r * p.ld_dy + col, inside, col, p.N);
          if (dh) unit_fetch<V, T, VEC>(s + 2 * NV * BLOCK, dh, r * p.ld_dh + col, inside, col, p.N);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int slot = 0, k = 0;
  float2 next;
  for (int j = 0; j < stages; ++j) fetch(row + j * stride, j);
  next = row < p.rows ? p.stats[row] : make_float2(0.0f, 0.0f);
  for (long long base = static_cast<long long>(blockIdx.x) * GROUPS; base < p.rows; base += stride, row += stride) {
    const bool live = row < p.rows;
    const float2 st = next;
    next = row + stride < p.rows ? p.stats[row + stride] : make_float2(0.0f, 0.0f);
    if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col_of(i);
      if (live && used(col)) {
        V *s = stage + (k * ins * NV + i) * BLOCK;
        V vh = s[0], vy = s[NV * BLOCK];
        if (col < 0 || col + VEC > p.N) {
          unit_mask<V, T, VEC>(vh, col, p.N);
          unit_mask<V, T, VEC>(vy, col, p.N);
          s[0] = vh;
          s[NV * BLOCK] = vy;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = to_f(vy.v[j]), n = (to_f(vh.v[j]) - st.x) * st.y, g = __fmul_rn(d, w[i][j]);
          aw[i][j] = fmaf(d, n, aw[i][j]);
          ac[i][j] += d;
          s1 += g;
          s2 = fmaf(g, n, s2);
        }
      }
    }
    ragged_sum2<TPR>(s1, s2, red, slot);
    s1 /= p.n;
    s2 /= p.n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col_of(i);
      if (live && used(col)) {
        const V *s = stage + (k * ins * NV + i) * BLOCK;
        const V vh = s[0], vy = s[NV * BLOCK];
        V o;
        // g rounded as above: what is equal cancels exactly (a row of one element has dx = dh)
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          v[j] = st.y * (__fmul_rn(to_f(vy.v[j]), w[i][j]) - s1 - (to_f(vh.v[j]) - st.x) * st.y * s2);
        if (dh) {
          const V vd = s[2 * NV * BLOCK];
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[j] += to_f(vd.v[j]);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) o.v[j] = from_f<T>(v[j]);
        unit_store<V, T, VEC>(dx + row * p.N + col, o, col, p.N);
      }
    }
    fetch(row + stages * stride, k);
    k = k + 1 == stages ? 0 : k + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (p.part == nullptr) return;
  float *join = reinterpret_cast<float *>(stage_bytes);   // [group][column], once the rows are done
  float *pw = p.part + static_cast<long long>(blockIdx.x) * 2 * p.N, *pc = pw + p.N;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float *dst = which ? pc : pw;
    if constexpr (GROUPS > 1) {
      __syncthreads();
      dst = join + group * p.N;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int col = col_of(i) + j;
        if (col >= 0 && col < p.N) dst[col] = which ? ac[i][j] : aw[i][j];
      }
    if constexpr (GROUPS > 1) {   // the groups of a block in order
      __syncthreads();
      for (int col = threadIdx.x; col < p.N; col += BLOCK) {
        float s = 0.0f;
        for (int g = 0; g < GROUPS; ++g) s += join[g * p.N + col];
        (which ? pc : pw)[col] = s;
      }
    }
  }
}

// ---- launches ---------------------------------------------------------------
constexpr int kRaggedMost = 200 * 1024;   // shared memory of a block
constexpr int kRaggedElems = 16;          // elements a thread: as many weights and sums again are in registers

// Threads of a row and its units, wherever it starts.
template <typename T>
NormRow ragged_row(int N) {
  constexpr int VEC = 16 / sizeof(T);
  return norm_row((N + 2 * (VEC - 1)) / VEC, kRaggedElems / VEC);
}

// `tile`: bytes of a stage; `resident`: blocks an SM holds, kept for the next
// call (the same on every device the library runs on).
template <typename K, typename A>
int ragged_launch(K kern, const A &a, int block, int groups, int step, int tile, int most, int *grid,
                  std::atomic<int> *resident, cudaStream_t st) {
  int rc, per = resident->load(std::memory_order_relaxed);
  const int stages = 2 * tile <= kRaggedMost ? 2 : 1, smem = stages * tile;
  if (smem > 40 * 1024 &&   // 48 KB with the static part
      (rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRaggedMost))))
    return rc;
  if (per == 0) {
    if ((rc = runtime_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, block, smem)))) return rc;
    resident->store(per = per > 0 ? per : 1, std::memory_order_relaxed);
  }
  const long long need = (a.rows + groups - 1) / groups;
  long long full = static_cast<long long>(sm_count()) * per;
  if (full > most) full = most;
  full -= full % step;   // a thread's rows are a multiple of VEC apart
  *grid = static_cast<int>(need < full ? need : full);
  kern<<<*grid, block, smem, st>>>(a, stages);
  return runtime_status(cudaGetLastError());
}

template <typename T, typename WT>
struct RaggedFwd {
  static constexpr int VEC = 16 / sizeof(T), kMost = kRaggedElems / VEC;
  const NormFwdArgs &a;
  cudaStream_t st;
  template <int NV, int TPR>
  int run() const {
    constexpr int BLOCK = norm_block<TPR>(), GROUPS = BLOCK / TPR;
    static std::atomic<int> resident[2]{};
    int grid;
    return ragged_launch(norm_fwd_ragged_kernel<T, WT, VEC, NV, TPR>, a, BLOCK, GROUPS, GROUPS >= VEC ? 1 : VEC,
                         (a.res ? 2 : 1) * NV * BLOCK * 16, INT_MAX, &grid, &resident[a.res != nullptr], st);
  }
};
template <typename T, typename WT>
struct RaggedBwd {
  static constexpr int VEC = 16 / sizeof(T), kMost = kRaggedElems / VEC;
  const NormBwdArgs &a;
  int most, *grid;
  cudaStream_t st;
  template <int NV, int TPR>
  int run() const {
    constexpr int BLOCK = norm_block<TPR>(), GROUPS = BLOCK / TPR;
    static std::atomic<int> resident[2]{};
    // the sums of a block's groups, GROUPS N floats, fit in a stage: N <= TPR NV VEC, and it has two tensors at least
    return ragged_launch(norm_bwd_ragged_kernel<T, WT, VEC, NV, TPR>, a, BLOCK, GROUPS, GROUPS >= VEC ? 1 : VEC,
                         (a.dh ? 3 : 2) * NV * BLOCK * 16, most, grid, &resident[a.dh != nullptr], st);
  }
};

// Whether the rows of all tensors lie alike relative to 16 bytes, and a block holds one.
template <typename T>
bool ragged_alike(int N, std::initializer_list<const void *> ts, std::initializer_list<long long> lds) {
  constexpr int VEC = 16 / sizeof(T);
  for (const void *t : ts)
    if (t && (reinterpret_cast<uintptr_t>(t) - reinterpret_cast<uintptr_t>(*ts.begin())) % 16) return false;
  for (long long ld : lds)
    if ((ld - N) % VEC) return false;
  return N + 2 * (VEC - 1) <= kNormMaxN;
}
// ---- dispatch of one I/O type: units of 16 or 8 bytes where every row and the
// weights start on one; else the kernels above; single elements where the
// tensors' rows lie differently, or are the widest.
template <typename T, typename WT>
int norm_fwd_typed(int vec, const NormFwdArgs &a, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  if (vec == VEC) return by_shape<VEC>(norm_row(a.N / VEC, kNormFwdElems / VEC), RunFwd<T, WT, VEC>{a, st});
  if (vec == VEC / 2)
    return by_shape<VEC / 2>(norm_row(a.N / vec, kNormFwdElems / vec), RunFwd<T, WT, VEC / 2>{a, st});
  if (ragged_alike<T>(a.N, {a.x, a.res, a.y, a.h}, {a.ld_x, a.res ? a.ld_res : a.N}))
    return by_shape<VEC>(ragged_row<T>(a.N), RaggedFwd<T, WT>{a, st});
  return by_shape<1>(norm_row(a.N, kNormFwdElems), RunFwd<T, WT, 1>{a, st});
}

template <typename T, typename WT>
int norm_bwd_typed(int vec, const NormBwdArgs &a, int most, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  int rc, grid = 0;
  if (vec == VEC)
    rc = by_shape<VEC>(norm_row(a.N / VEC, kNormBwdElems / VEC), RunBwd<T, WT, VEC>{a, most, &grid, st});
  else if (vec == VEC / 2)
    rc = by_shape<VEC / 2>(norm_row(a.N / vec, kNormBwdElems / vec), RunBwd<T, WT, VEC / 2>{a, most, &grid, st});
  else if (ragged_alike<T>(a.N, {a.h, a.dy, a.dh, a.dx}, {a.ld_h, a.ld_dy, a.dh ? a.ld_dh : a.N}))
    rc = by_shape<VEC>(ragged_row<T>(a.N), RaggedBwd<T, WT>{a, most, &grid, st});
  else
    rc = by_shape<1>(norm_row(a.N, kNormBwdElems), RunBwd<T, WT, 1>{a, most, &grid, st});
  if (rc || a.part == nullptr) return rc;
  norm_fold_kernel<WT><<<(2 * a.N + 31) / 32, 1024, 0, st>>>(a.part, grid, a.N, static_cast<WT *>(a.dweight),
                                                             static_cast<WT *>(a.dbias));
  return runtime_status(cudaGetLastError());
}

}  // namespace
}  // namespace esa
