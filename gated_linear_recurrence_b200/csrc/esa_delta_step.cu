// esa_delta_step.cu -- one token of the gated delta rule (sm_100a):
//   u = beta (v - alpha S^T k),  y = scale (alpha S^T q + (k.q) u),  S <- alpha S + k u^T.
//
// The state is read once and written once (8 D^2 bytes a head against 7 D^2
// operations), so memory traffic bounds it.  A block takes 32 value channels
// of a head: a thread has a float4 of four of them, and the block's threads go
// down the key channels, so that every access is a whole 128-byte line and all
// loads of a thread are under way at once (8 of 16 bytes at D = 128); the two
// sums over the key channels meet once in shared memory.  At B = 64, H = 8,
// D = 128 it takes 12.3 us (5.5 TB/s of the state's traffic), at B = 1 2.5.
// Blocks of 256 threads with whole heads took 15.1 and 3.8 (fewer blocks, whose
// loads, sums and stores take turns), with 64 channels 13.8 and 3.1; 64 threads
// 13.6 and 2.9; the token sweep's tiles, 32-byte pieces of a row, 22.
#include "esa_delta_sweep.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

constexpr int kThreads = 128, kWidth = 32;   // of a block: threads, value channels

__device__ __forceinline__ float4 fma4(float s, float4 a, float4 c) {
  const float2 x = fma2(splat(s), make_float2(a.x, a.y), make_float2(c.x, c.y));
  const float2 y = fma2(splat(s), make_float2(a.z, a.w), make_float2(c.z, c.w));
  return make_float4(x.x, x.y, y.x, y.y);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(SweepArgs p) {
  constexpr int C = D / kWidth;   // blocks of a head
  constexpr int LPR = kWidth / 4, ROWS = kThreads / LPR, NP = D / ROWS;   // threads a row, rows a pass, passes
  __shared__ __align__(16) float k[D], q[D], v[kWidth];
  __shared__ __align__(16) float4 part[2][kThreads / 32][LPR];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c4 = tid % LPR, r0 = tid / LPR;
  const long long head = blockIdx.x / C;
  const int v0 = blockIdx.x % C * kWidth;
  const int bat = static_cast<int>(head) / p.s.H, h = static_cast<int>(head) - bat * p.s.H;
  const long long qk = bat * p.s.ld_qk + h * D, vo = bat * p.s.ld_v + h * D, g = bat * p.s.ld_g + h;
  const float4 *S = reinterpret_cast<const float4 *>(p.S_in + head * D * D + v0) + r0 * (D / 4) + c4;
  float4 m[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) m[i] = S[i * ROWS * (D / 4)];
  if (tid < D) {   // D <= kThreads
    k[tid] = sweep::widen(static_cast<const T *>(p.k)[qk + tid]);
    q[tid] = sweep::widen(static_cast<const T *>(p.q)[qk + tid]);
    if (tid < kWidth) v[tid] = sweep::widen(static_cast<const T *>(p.v)[vo + v0 + tid]);
  }
  const float alpha = sweep::gate(sweep::widen(static_cast<const T *>(p.a)[g]));
  const float beta = sweep::gate(sweep::widen(static_cast<const T *>(p.b)[g]));
  __syncthreads();
  float4 P = make_float4(0, 0, 0, 0), Q = P;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    P = fma4(k[r0 + i * ROWS], m[i], P);
    Q = fma4(q[r0 + i * ROWS], m[i], Q);
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {   // rows of one warp
    P.x += __shfl_xor_sync(0xffffffffu, P.x, o);
    P.y += __shfl_xor_sync(0xffffffffu, P.y, o);
    P.z += __shfl_xor_sync(0xffffffffu, P.z, o);
    P.w += __shfl_xor_sync(0xffffffffu, P.w, o);
    Q.x += __shfl_xor_sync(0xffffffffu, Q.x, o);
    Q.y += __shfl_xor_sync(0xffffffffu, Q.y, o);
    Q.z += __shfl_xor_sync(0xffffffffu, Q.z, o);
    Q.w += __shfl_xor_sync(0xffffffffu, Q.w, o);
  }
  if (lane < LPR) {
    part[0][warp][c4] = P;
    part[1][warp][c4] = Q;
  }
  float kq = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) kq = fmaf(k[32 * i + lane], q[32 * i + lane], kq);
  kq = head_sum<32>(kq);
  __syncthreads();
  P = part[0][0][c4];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) P = fma4(1.0f, part[0][w][c4], P);
  const float4 vv = reinterpret_cast<const float4 *>(v)[c4];
  const float4 u = make_float4(beta * fmaf(-alpha, P.x, vv.x), beta * fmaf(-alpha, P.y, vv.y),
                               beta * fmaf(-alpha, P.z, vv.z), beta * fmaf(-alpha, P.w, vv.w));
  float4 *So = reinterpret_cast<float4 *>(p.S_out + head * D * D + v0) + r0 * (D / 4) + c4;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float4 a = make_float4(alpha * m[i].x, alpha * m[i].y, alpha * m[i].z, alpha * m[i].w);
    So[i * ROWS * (D / 4)] = fma4(k[r0 + i * ROWS], u, a);
  }
  if (tid < LPR) {
    Q = part[1][0][c4];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) Q = fma4(1.0f, part[1][w][c4], Q);
    T *y = static_cast<T *>(p.y) + head * D + v0 + 4 * c4;
    y[0] = sweep::narrow<T>(p.s.scale * fmaf(alpha, Q.x, kq * u.x));
    y[1] = sweep::narrow<T>(p.s.scale * fmaf(alpha, Q.y, kq * u.y));
    y[2] = sweep::narrow<T>(p.s.scale * fmaf(alpha, Q.z, kq * u.z));
    y[3] = sweep::narrow<T>(p.s.scale * fmaf(alpha, Q.w, kq * u.w));
  }
}

template <typename T>
int run(const SweepArgs &a, cudaStream_t st) {
  const unsigned heads = static_cast<unsigned>(a.s.B) * a.s.H;
  switch (a.s.D) {
    case 32: delta_step_kernel<T, 32><<<heads * (32 / kWidth), kThreads, 0, st>>>(a); break;
    case 64: delta_step_kernel<T, 64><<<heads * (64 / kWidth), kThreads, 0, st>>>(a); break;
    case 128: delta_step_kernel<T, 128><<<heads * (128 / kWidth), kThreads, 0, st>>>(a); break;
    default: return ESA_ERR_UNSUPPORTED;
  }
  return runtime_status(cudaGetLastError());
}

}  // namespace

int launch_delta_step(int dtype, const SweepArgs &a, cudaStream_t st) {
  switch (dtype) {
    case ESA_F32: return run<float>(a, st);
    case ESA_F16: return run<__half>(a, st);
    case ESA_BF16: return run<__nv_bfloat16>(a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace esa
