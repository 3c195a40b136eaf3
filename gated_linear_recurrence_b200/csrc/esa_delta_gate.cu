// esa_delta_gate.cu -- the gradient of the forget gate after the token sweeps
// of the gated delta rule (sm_100a).
//
//   da_t = (1 - alpha_t) f_t,   f_t = <gradient of S_{t-1} from the tokens t .., S_{t-1}>.
// f_t differs from f_{t+1} by q.dq - beta v.du of token t, so a chunk's f are
// running sums of that from <dS, S> at its end.  They cancel to alpha_t of
// their terms: right to some 2^-22 / alpha_t.  Where every gate of a chunk
// keeps a quarter or more that is what is done, by one warp.  Else f_t is summed
// from the terms that have the factor alpha_t,
//   f_t = sum_{j < t <= s} W_sj + sum_{s >= t} A_s + sum_{j < t} B_j + e^{G_last} <dS, S>,
//   W_sj = e^{Gs - Gj} (scale (q_s.k_j)(dy_s.u_j) - beta_s (k_s.k_j)(du_s.u_j)),
//   A_s = e^{Gs} (scale q_s S dy_s - beta_s k_s S du_s),   B_j = e^{G_last - Gj} k_j dS u_j,
// with S the state entering the chunk and dS the gradient of the one leaving
// it: seven products of 64 rows in float32 multiply-adds, by a block a chunk.
// Training with long memory does not pay for them: 8 heads of D = 64, T = 4096,
// 646 us with the backward at logits around 4 and 698 around 0; 256 heads of
// D = 32, T = 512, 393 and 528.
#include "esa_delta_sweep.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

using sweep::decay;
using sweep::Place;
constexpr int C = sweep::CHUNK, kThreads = 256, kTri = C + 4;
constexpr float kForgets = 0.25f;

template <int D>
struct GateSmem {   // in floats
  static constexpr int x = 0, y = C * (D + 4), w = 2 * y, g = w + C * kTri, beta = g + 2 * C, as = beta + C, bs = as + C,
                       fq = bs + C, fk = fq + C, fb = fk + C, part = fb + C, total = part + 8;
};

template <typename T>
__device__ __forceinline__ float4 widen4(const T *p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4 *>(p);
  } else {
    const uint2 raw = *reinterpret_cast<const uint2 *>(p);
    const T *e = reinterpret_cast<const T *>(&raw);
    return make_float4(sweep::widen(e[0]), sweep::widen(e[1]), sweep::widen(e[2]), sweep::widen(e[3]));
  }
}

// Rows [0, n) of D elements, `ld` apart; zeros behind them up to 64.
template <typename T, int D>
__device__ __forceinline__ void rows_in(float *dst, const T *src, long long ld, int n) {
  for (int i = threadIdx.x; i < C * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    *reinterpret_cast<float4 *>(dst + r * (D + 4) + c) = r < n ? widen4(src + r * ld + c) : make_float4(0, 0, 0, 0);
  }
}

// out[s] += f[s] sum_k x_s[k] (sum_v M[k][v] X_s[v]), s < len: X in shared memory, x and M in global memory, Y scratch.
// Begins and ends with a barrier.
template <typename T, int D>
__device__ __forceinline__ void state_dots(float *out, const float *f, const float *X, float *Y, const float *M, const T *x,
                                           long long ld, int len) {
  const int ti = threadIdx.x >> 4, tj = threadIdx.x & 15;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = 0; k0 < D; k0 += C) {
    __syncthreads();
    rows_in<float, D>(Y, M + k0 * D, D, min(C, D - k0));
    __syncthreads();
    float acc[4][4];
    sweep::dots<D>(X, Y, ti, tj, acc);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int s = ti + 16 * r, k = k0 + tj + 16 * c;
        if (s < len && k < D) sum[r] = fmaf(acc[r][c], sweep::widen(x[s * ld + k]), sum[r]);
      }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float z = sum[r];
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (tj == 0) out[ti + 16 * r] = fmaf(f[ti + 16 * r], z, out[ti + 16 * r]);
  }
  __syncthreads();
}

// Two tokens a lane: the logits, and whether a gate of the chunk forgets.
template <typename T>
__device__ __forceinline__ bool read_logits(const FinishArgs &p, const Place &a, float (&logit)[2]) {
  const T *ga = static_cast<const T *>(p.a) + a.row * p.s.ld_g + a.h;
  bool forgets = false;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * (threadIdx.x & 31) + e;
    logit[e] = i < a.len ? sweep::clamp(sweep::widen(ga[i * p.s.ld_g])) : 80.0f;
    forgets = forgets || !(sweep::gate(logit[e]) >= kForgets);
  }
  return __any_sync(0xffffffffu, forgets);
}

template <typename T>
__device__ __forceinline__ void write_da(const FinishArgs &p, const Place &a, const float (&f)[2], const float (&logit)[2]) {
  T *da = static_cast<T *>(p.da) + a.row * p.s.H + a.h;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * (threadIdx.x & 31) + e;
    if (i < a.len) da[static_cast<long long>(i) * p.s.H] = sweep::narrow<T>(f[e] / (1.0f + expf(logit[e])));   // 1 - alpha = 1 / (1 + e^a)
  }
}

// The running sums, by one warp.
template <typename T, int D>
__device__ __forceinline__ void light_chunk(const FinishArgs &p, const Place &a, const float (&logit)[2]) {
  constexpr int kParts = D * D / 1024;   // of <dS, S> at the chunk's end
  const int lane = threadIdx.x & 31;
  const float *gain = p.gain + (static_cast<long long>(a.b) * p.s.H + a.h) * p.s.T + a.t0;
  float end = 0.0f, f[2];
  for (int i = 0; i < kParts; ++i) end += p.end[a.chunk * kParts + i];
  const float x0 = 2 * lane < a.len ? gain[2 * lane] : 0.0f, x1 = 2 * lane + 1 < a.len ? gain[2 * lane + 1] : 0.0f;
  float sum = x0 + x1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_down_sync(0xffffffffu, sum, o);
    if (lane + o < 32) sum += y;
  }
  const float after = __shfl_down_sync(0xffffffffu, sum, 1);
  f[1] = end + (lane < 31 ? after : 0.0f) + x1;
  f[0] = f[1] + x0;
  write_da<T>(p, a, f, logit);
}

// The terms that have the factor alpha, by the block.
template <typename T, int D>
__device__ __forceinline__ void heavy_chunk(const FinishArgs &p, const Place &a, float *sm) {
  using L = GateSmem<D>;
  const int tid = threadIdx.x, lane = tid & 31;
  float *X = sm + L::x, *Y = sm + L::y, *W = sm + L::w, *beta = sm + L::beta, *as = sm + L::as, *bs = sm + L::bs,
        *fq = sm + L::fq, *fk = sm + L::fk, *fb = sm + L::fb, *part = sm + L::part;
  float2 *G = reinterpret_cast<float2 *>(sm + L::g);
  const long long ldc = static_cast<long long>(p.s.H) * D, own = a.row * ldc + a.h * D;
  const T *q = static_cast<const T *>(p.q) + a.row * p.s.ld_qk + a.h * D, *k = static_cast<const T *>(p.k) + a.row * p.s.ld_qk + a.h * D;
  const T *dy = static_cast<const T *>(p.dy) + own;
  const float *S = p.S_ck + a.chunk * (D * D), *dS = p.dS_ck + a.chunk * (D * D);
  const int ti = tid >> 4, tj = tid & 15;
  sweep::gates_of<T>(p.s, p.a, p.b, a, G, beta);
  rows_in<T, D>(X, q, p.s.ld_qk, a.len);
  rows_in<T, D>(Y, k, p.s.ld_qk, a.len);
  __syncthreads();
  if (tid < C) {
    const float2 zero = make_float2(0.0f, 0.0f);
    const float into = decay(G[tid], zero);
    as[tid] = bs[tid] = 0.0f;
    fq[tid] = p.s.scale * into;
    fk[tid] = -beta[tid] * into;
    fb[tid] = decay(G[C - 1], G[tid]);
  }
  float qk[4][4], kk[4][4], z[4][4];
  sweep::dots<D>(X, Y, ti, tj, qk);
  sweep::dots<D>(Y, Y, ti, tj, kk);
  __syncthreads();
  rows_in<T, D>(X, dy, ldc, a.len);
  rows_in<float, D>(Y, p.u + own, ldc, a.len);
  __syncthreads();
  sweep::dots<D>(X, Y, ti, tj, z);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) qk[r][c] *= p.s.scale * z[r][c];
  __syncthreads();
  rows_in<float, D>(X, p.du + own, ldc, a.len);
  __syncthreads();
  sweep::dots<D>(X, Y, ti, tj, z);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int i = ti + 16 * r, j = tj + 16 * c;
      W[i * kTri + j] = j < i ? decay(G[i], G[j]) * fmaf(-beta[i] * kk[r][c], z[r][c], qk[r][c]) : 0.0f;
    }
  state_dots<T, D>(as, fk, X, Y, S, k, p.s.ld_qk, a.len);   // X: du
  rows_in<T, D>(X, dy, ldc, a.len);
  state_dots<T, D>(as, fq, X, Y, S, q, p.s.ld_qk, a.len);
  rows_in<float, D>(X, p.u + own, ldc, a.len);
  state_dots<T, D>(bs, fb, X, Y, dS, k, p.s.ld_qk, a.len);
  float c = 0.0f;
  for (int i = tid * 4; i < D * D; i += kThreads * 4) {
    const float4 s4 = *reinterpret_cast<const float4 *>(S + i), d4 = *reinterpret_cast<const float4 *>(dS + i);
    c = fmaf(s4.x, d4.x, fmaf(s4.y, d4.y, fmaf(s4.z, d4.z, fmaf(s4.w, d4.w, c))));
  }
  c = head_sum<32>(c);
  if (lane == 0) part[tid >> 5] = c;
  if (tid < C) {   // column j of W: the sum over s >= i in the place of row i, for the rectangles with j < i
    float x = 0.0f;
    for (int i = C - 1; i > tid; --i) W[i * kTri + tid] = x += W[i * kTri + tid];
  }
  __syncthreads();
  if (tid < 32) {
    float A[2], B[2], F[2], cc = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) cc += part[i];
    cc *= decay(G[C - 1], make_float2(0.0f, 0.0f));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      const float *w = W + i * kTri;
      A[e] = as[i];
      B[e] = bs[i];
      float2 x = make_float2(0.0f, 0.0f);
      for (int j = 0; j < C; j += 4) {   // zeros from the diagonal on
        const float4 v = *reinterpret_cast<const float4 *>(w + j);
        x = add2(x, add2(make_float2(v.x, v.y), make_float2(v.z, v.w)));
      }
      F[e] = x.x + x.y;
    }
    float later = A[0] + A[1], earlier = B[0] + B[1];   // over this lane's tokens and those behind (before) them
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, later, o), z2 = __shfl_up_sync(0xffffffffu, earlier, o);
      if (lane + o < 32) later += y;
      if (lane >= o) earlier += z2;
    }
    const float behind = __shfl_down_sync(0xffffffffu, later, 1), before = __shfl_up_sync(0xffffffffu, earlier, 1);
    const float b0 = lane > 0 ? before : 0.0f, a1 = (lane < 31 ? behind : 0.0f) + A[1];
    float logit[2];
    read_logits<T>(p, a, logit);
    const float f[2] = {F[0] + (later + b0 + cc), F[1] + (a1 + (b0 + B[0]) + cc)};
    write_da<T>(p, a, f, logit);
  }
}

// Each warp looks at one of the block's `group` chunks; those with a gate that
// forgets are left to the whole block, one after another.  4096 chunks of long
// memory take 7.5 us so, 25 with a block a chunk; with 2048 that all forget a
// whole pass takes 528 us, 509 with a block a chunk.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) delta_gate_kernel(FinishArgs p, int chunks, int group) {
  extern __shared__ __align__(16) float sm[];
  __shared__ unsigned heavy;
  const int warp = threadIdx.x >> 5, first = blockIdx.x * group;
  if (threadIdx.x == 0) heavy = 0;
  __syncthreads();
  if (warp < group && first + warp < chunks) {
    const int head = (first + warp) / p.nc;
    const Place a = sweep::place_of(p.s, p.nc, head, first + warp - head * p.nc);
    float logit[2];
    if (!read_logits<T>(p, a, logit)) light_chunk<T, D>(p, a, logit);
    else if ((threadIdx.x & 31) == 0) atomicOr(&heavy, 1u << warp);
  }
  __syncthreads();
  for (unsigned left = heavy; left != 0; left &= left - 1) {
    const int c = first + __ffs(left) - 1, head = c / p.nc;
    heavy_chunk<T, D>(p, sweep::place_of(p.s, p.nc, head, c - head * p.nc), sm);
    __syncthreads();
  }
}

template <typename T, int D>
int run(const FinishArgs &a, cudaStream_t st) {
  auto kern = delta_gate_kernel<T, D>;
  constexpr int bytes = GateSmem<D>::total * 4;
  if (bytes > 47 * 1024) {   // 48 KB with the static part
    const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (rc) return rc;
  }
  const int chunks = a.s.B * a.s.H * a.nc;
  int group = chunks / (4 * sm_count());   // four blocks an SM at least, where there are as many chunks
  group = group < 1 ? 1 : group > kThreads / 32 ? kThreads / 32 : group;
  kern<<<(chunks + group - 1) / group, kThreads, bytes, st>>>(a, chunks, group);
  return runtime_status(cudaGetLastError());
}

template <typename T>
int by_d(const FinishArgs &a, cudaStream_t st) {
  switch (a.s.D) {
    case 32: return run<T, 32>(a, st);
    case 64: return run<T, 64>(a, st);
    case 128: return run<T, 128>(a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace

int launch_delta_gate(int dtype, const FinishArgs &a, cudaStream_t st) {
  switch (dtype) {
    case ESA_F32: return by_d<float>(a, st);
    case ESA_F16: return by_d<__half>(a, st);
    case ESA_BF16: return by_d<__nv_bfloat16>(a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace esa
