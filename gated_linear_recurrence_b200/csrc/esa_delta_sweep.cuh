// esa_delta_sweep.cuh -- the gated delta rule token by token (sm_100a).
//
//   alpha = sigmoid(a), beta = sigmoid(b) (logits clamped at -80 below),
//   u_t = beta_t (v_t - alpha_t S_{t-1}^T k_t),  S_t = alpha_t S_{t-1} + k_t u_t^T,
//   y_t = scale S_t^T q_t,      S [D key channels][D value channels], float32.
//
// A sweep keeps a matrix M in registers and visits the tokens in order.  M has
// a split axis (its D entries are shared by 8 lanes, which sum their parts of
// each dot product by shuffles) and an independent axis (4 entries a thread,
// 16 a warp, no communication).  The forward is split over the key channels:
// every value channel is a recurrence of its own.  The gradients need both
// orientations, so the backward is three more sweeps, each with two dot
// products or one and one or two rank-one updates per token:
//   kSweepFwd  forward,  M = S,  split = key:   u (kept for the backward), y, S_T
//   kSweepDu   backward, M = dS, split = key:   du_t = dS_t^T k_t with dS_t += scale q_t dy_t^T first,
//                                               then dS <- alpha_t (dS - beta_t k_t du_t^T);  dS_init
//   kSweepDk   backward, M = dS^T, split = value: dk_t = dS_t u_t
//   kSweepDq   forward,  M = S^T, split = value:  dk_t -= alpha_t beta_t S_{t-1} du_t, dq_t = scale S_t dy_t,
//                                               and <S_T, dS_final>
// All arithmetic is float32, as the state is; this is the path of float32
// tensors, of short sequences (a decode step is a sweep of one token) and of
// D = 32.  It is bound by float32 issue: 8 D^2 multiply-adds (packed in pairs)
// a token forward, so at D = 128 about 1.4 ns a token and head with every SM
// busy, and by the latency of one token (a dot product, three shuffles, a
// broadcast) when there are few heads.  More warps per block share the
// staged rows; fewer give more blocks: see sweep_warps().
//
// Rows are staged 16 tokens at a time: cp.async into a double buffer in the
// tensors' own type, then widened once to float32 for all warps of the block.
#pragma once

#include "esa_common.cuh"
#include "esa_delta.h"

namespace esa {
namespace sweep {

constexpr int TC = 16;      // tokens staged at a time
constexpr int SPLIT = 8;    // lanes that share the split axis
constexpr int PER = 4;      // independent entries a thread
constexpr int COLS = 16;    // independent entries a warp

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow(float v) { return v; }
template <> __device__ __forceinline__ __half narrow(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float gate(float x) { return 1.0f / (1.0f + expf(-fmaxf(x, -80.0f))); }

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Copy rows [0, n) of `width` elements (a whole number of 16-byte units),
// `ld` elements apart, into dst[row * width].
template <typename E>
__device__ __forceinline__ void stage(E *dst, const E *src, long long ld, int n, int width) {
  constexpr int V = 16 / sizeof(E);
  const int per = width / V;
  for (int i = threadIdx.x; i < n * per; i += blockDim.x) {
    const int r = i / per, c = (i - r * per) * V;
    cp_async16(dst + r * width + c, src + r * ld + c);
  }
}

template <typename E>
__device__ __forceinline__ void widen_rows(float *dst, const E *src, int count) {
  constexpr int V = 16 / sizeof(E);
  for (int i = threadIdx.x * V; i < count; i += blockDim.x * V) {
    const uint4 raw = *reinterpret_cast<const uint4 *>(src + i);
    const E *e = reinterpret_cast<const E *>(&raw);
#pragma unroll
    for (int j = 0; j < V; j += 4)
      *reinterpret_cast<float4 *>(dst + i + j) = make_float4(widen(e[j]), widen(e[j + 1]), widen(e[j + 2]), widen(e[j + 3]));
  }
}

// The staged rows of a kind: three along the split axis (X0, X1 of type T or
// float, X2 float), two along the independent axis.
template <typename T, int KIND> struct Rows;
template <typename T> struct Rows<T, kSweepFwd> { static constexpr bool x0f = false, x2 = false, y1 = false; };
template <typename T> struct Rows<T, kSweepDu> { static constexpr bool x0f = false, x2 = false, y1 = false; };
template <typename T> struct Rows<T, kSweepDk> { static constexpr bool x0f = true, x2 = true, y1 = true; };
template <typename T> struct Rows<T, kSweepDq> { static constexpr bool x0f = true, x2 = true, y1 = false; };

// Shared memory, in floats and bytes, for W warps.
template <typename T, int D, int KIND>
struct Layout {
  using R = Rows<T, KIND>;
  static constexpr bool kWide = sizeof(T) == 4;
  int cols;
  size_t x0, x1, x2, y0, y1, raw;    // raw buffer (one stage): byte offsets
  size_t fx0, fx1, fy0, fy1, tok;    // widened rows and per-token scalars: byte offsets from the start
  size_t total;
  __host__ __device__ explicit Layout(int W) {
    cols = COLS * W;
    size_t o = 0;
    x0 = o; o += static_cast<size_t>(TC) * D * (R::x0f ? 4 : sizeof(T));
    x1 = o; o += static_cast<size_t>(TC) * D * sizeof(T);
    x2 = o; o += R::x2 ? static_cast<size_t>(TC) * D * 4 : 0;
    y0 = o; o += static_cast<size_t>(TC) * cols * sizeof(T);
    y1 = o; o += R::y1 ? static_cast<size_t>(TC) * cols * sizeof(T) : 0;
    raw = o;
    o = 2 * raw;
    fx0 = o; o += kWide || R::x0f ? 0 : static_cast<size_t>(TC) * D * 4;
    fx1 = o; o += kWide ? 0 : static_cast<size_t>(TC) * D * 4;
    fy0 = o; o += kWide ? 0 : static_cast<size_t>(TC) * cols * 4;
    fy1 = o; o += kWide || !R::y1 ? 0 : static_cast<size_t>(TC) * cols * 4;
    tok = o; o += 3 * TC * sizeof(float);
    total = o;
  }
};

template <typename T, int D, int KIND>
__global__ void __launch_bounds__(D * 2) delta_sweep_kernel(SweepArgs p) {
  constexpr bool kReverse = KIND == kSweepDu || KIND == kSweepDk;
  constexpr bool kCols = KIND == kSweepFwd || KIND == kSweepDu;   // split over the key channels
  constexpr int RPT = D / SPLIT;                                  // split entries a thread
  constexpr int M4 = RPT / 4;
  using R = Rows<T, KIND>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int W = blockDim.x >> 5;
  const Layout<T, D, KIND> lo(W);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane & 7, cg = lane >> 3;
  const int slices = D / lo.cols;
  const int slice = blockIdx.x % slices;
  const int head = blockIdx.x / slices;                // b H + h
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int c_blk = slice * lo.cols;                   // first independent entry of the block
  const int c_thr = c_blk + warp * COLS + cg * PER;    // and of this thread
  const int T_ = p.s.T;
  const long long tok0 = static_cast<long long>(b) * T_;
  const long long ldc = static_cast<long long>(p.s.H) * D;   // contiguous rows (dy, y, scratch)

  // M in registers: entry (split i, independent j) at m[j][i / 2], pairs along the split axis;
  // this lane's split entries are 32 g + 4 r + 0..3.
  float2 m[PER][RPT / 2];
  const float *Sin = p.S_in ? p.S_in + static_cast<long long>(head) * D * D : nullptr;
#pragma unroll
  for (int g = 0; g < M4; ++g) {
    const int i0 = 32 * g + 4 * r;
    if (Sin == nullptr) {
#pragma unroll
      for (int j = 0; j < PER; ++j) m[j][2 * g] = m[j][2 * g + 1] = make_float2(0.0f, 0.0f);
    } else if (kCols) {
      float4 row[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) row[e] = *reinterpret_cast<const float4 *>(Sin + (i0 + e) * D + c_thr);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[0][2 * g + e] = make_float2(row[2 * e].x, row[2 * e + 1].x);
        m[1][2 * g + e] = make_float2(row[2 * e].y, row[2 * e + 1].y);
        m[2][2 * g + e] = make_float2(row[2 * e].z, row[2 * e + 1].z);
        m[3][2 * g + e] = make_float2(row[2 * e].w, row[2 * e + 1].w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const float4 x = *reinterpret_cast<const float4 *>(Sin + (c_thr + j) * D + i0);
        m[j][2 * g] = make_float2(x.x, x.y);
        m[j][2 * g + 1] = make_float2(x.z, x.w);
      }
    }
  }

  const T *q = static_cast<const T *>(p.q) + h * D, *k = static_cast<const T *>(p.k) + h * D;
  const T *v = static_cast<const T *>(p.v), *dy = static_cast<const T *>(p.dy);
  const T *ga = static_cast<const T *>(p.a), *gb = static_cast<const T *>(p.b);
  const int nch = (T_ + TC - 1) / TC;

  auto fetch = [&](int c, int buf) {
    const int t0 = c * TC, n = min(TC, T_ - t0);
    const long long row = tok0 + t0;
    unsigned char *s = smem + buf * lo.raw;
    if constexpr (KIND == kSweepFwd || KIND == kSweepDu) {
      stage(reinterpret_cast<T *>(s + lo.x0), k + row * p.s.ld_qk, p.s.ld_qk, n, D);
      stage(reinterpret_cast<T *>(s + lo.x1), q + row * p.s.ld_qk, p.s.ld_qk, n, D);
      if constexpr (KIND == kSweepFwd)
        stage(reinterpret_cast<T *>(s + lo.y0), v + row * p.s.ld_v + h * D + c_blk, p.s.ld_v, n, lo.cols);
      else
        stage(reinterpret_cast<T *>(s + lo.y0), dy + row * ldc + h * D + c_blk, ldc, n, lo.cols);
    } else {
      const float *f0 = KIND == kSweepDk ? p.u : p.du, *f2 = KIND == kSweepDk ? p.du : p.u;
      stage(reinterpret_cast<float *>(s + lo.x0), f0 + row * ldc + h * D, ldc, n, D);
      stage(reinterpret_cast<T *>(s + lo.x1), dy + row * ldc + h * D, ldc, n, D);
      stage(reinterpret_cast<float *>(s + lo.x2), f2 + row * ldc + h * D, ldc, n, D);
      const T *i0 = KIND == kSweepDk ? q : k;
      stage(reinterpret_cast<T *>(s + lo.y0), i0 + row * p.s.ld_qk + c_blk, p.s.ld_qk, n, lo.cols);
      if constexpr (KIND == kSweepDk)
        stage(reinterpret_cast<T *>(s + lo.y1), k + row * p.s.ld_qk + c_blk, p.s.ld_qk, n, lo.cols);
    }
    cp_async_commit();
  };
  float ga_next = 0.0f, gb_next = 0.0f;
  auto fetch_gates = [&](int c) {
    const int t = c * TC + threadIdx.x;
    if (threadIdx.x < TC && t < T_) {
      ga_next = widen(ga[(tok0 + t) * p.s.ld_g + h]);
      gb_next = widen(gb[(tok0 + t) * p.s.ld_g + h]);
    }
  };

  float *tok = reinterpret_cast<float *>(smem + lo.tok);   // alpha, beta, dot, TC each
  if (nch > 0) {
    fetch(kReverse ? nch - 1 : 0, 0);
    fetch_gates(kReverse ? nch - 1 : 0);
  }
  for (int it = 0; it < nch; ++it) {
    const int c = kReverse ? nch - 1 - it : it, buf = it & 1;
    const int t0 = c * TC, n = min(TC, T_ - t0);
    if (threadIdx.x < TC) {
      tok[threadIdx.x] = gate(ga_next);
      tok[TC + threadIdx.x] = gate(gb_next);
    }
    if (it + 1 < nch) {
      const int cn = kReverse ? c - 1 : c + 1;
      fetch(cn, buf ^ 1);
      fetch_gates(cn);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    unsigned char *s = smem + buf * lo.raw;
    const float *X0, *X1, *X2 = nullptr, *Y0, *Y1 = nullptr;
    if constexpr (sizeof(T) == 4) {
      X0 = reinterpret_cast<const float *>(s + lo.x0);
      X1 = reinterpret_cast<const float *>(s + lo.x1);
      Y0 = reinterpret_cast<const float *>(s + lo.y0);
      Y1 = reinterpret_cast<const float *>(s + lo.y1);
    } else {
      float *w;
      if constexpr (R::x0f) {
        X0 = reinterpret_cast<const float *>(s + lo.x0);
      } else {
        widen_rows(w = reinterpret_cast<float *>(smem + lo.fx0), reinterpret_cast<const T *>(s + lo.x0), n * D);
        X0 = w;
      }
      widen_rows(w = reinterpret_cast<float *>(smem + lo.fx1), reinterpret_cast<const T *>(s + lo.x1), n * D);
      X1 = w;
      widen_rows(w = reinterpret_cast<float *>(smem + lo.fy0), reinterpret_cast<const T *>(s + lo.y0), n * lo.cols);
      Y0 = w;
      if constexpr (R::y1) {
        widen_rows(w = reinterpret_cast<float *>(smem + lo.fy1), reinterpret_cast<const T *>(s + lo.y1), n * lo.cols);
        Y1 = w;
      }
      __syncthreads();
    }
    if constexpr (R::x2) X2 = reinterpret_cast<const float *>(s + lo.x2);
    // k.q (sweeps over columns) or u.dy (sweeps over rows) of each token
    {
      const float *d0 = KIND == kSweepDq ? X2 : X0;   // k, k, u, u
      for (int t = warp; t < n; t += W) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x = fmaf(d0[t * D + 32 * i + lane], X1[t * D + 32 * i + lane], x);
        x = head_sum<32>(x);
        if (lane == 0) tok[2 * TC + t] = x;
      }
    }
    __syncthreads();

    for (int e = 0; e < n; ++e) {
      const int t = kReverse ? n - 1 - e : e;
      const float alpha = tok[t], beta = tok[TC + t], dot = tok[2 * TC + t];
      const float4 *x0 = reinterpret_cast<const float4 *>(X0 + t * D) + r;
      const float4 *x1 = reinterpret_cast<const float4 *>(X1 + t * D) + r;
      float4 a0[M4], a1[M4];
#pragma unroll
      for (int g = 0; g < M4; ++g) {
        a0[g] = x0[8 * g];
        a1[g] = x1[8 * g];
      }
      const float4 in0 = *reinterpret_cast<const float4 *>(Y0 + t * lo.cols + warp * COLS + cg * PER);
      const float i0[4] = {in0.x, in0.y, in0.z, in0.w};
      const long long out = (tok0 + t0 + t) * ldc + h * D + c_thr;
      // P_j = sum_i x0_i m_ij; Q_j = sum_i x1_i m_ij (forward kinds only)
      float P[PER], Q[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        float2 s0 = make_float2(0.0f, 0.0f), s1 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int g = 0; g < M4; ++g) {
          s0 = fma2(make_float2(a0[g].x, a0[g].y), m[j][2 * g], s0);
          s0 = fma2(make_float2(a0[g].z, a0[g].w), m[j][2 * g + 1], s0);
          if constexpr (!kReverse) {
            s1 = fma2(make_float2(a1[g].x, a1[g].y), m[j][2 * g], s1);
            s1 = fma2(make_float2(a1[g].z, a1[g].w), m[j][2 * g + 1], s1);
          }
        }
        P[j] = s0.x + s0.y;
        Q[j] = s1.x + s1.y;
      }
      // Sum over the 8 lanes of a column group by halving: a lane gives away
      // the half of its values that its partner keeps.  After it lane r holds
      // column r & 3 of P (r < 4) or of Q (r >= 4); the backward kinds have no
      // Q and add the two halves instead, so both halves hold P.
      float mine;
      {
        const bool hi = r & 4;
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (!kReverse) {
            const float keep = hi ? Q[j] : P[j], give = hi ? P[j] : Q[j];
            x[j] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
          } else {
            x[j] = P[j] + __shfl_xor_sync(0xffffffffu, P[j], 4);
          }
        }
        const bool h2 = r & 2, h1 = r & 1;
        const float k0 = h2 ? x[2] : x[0], k1 = h2 ? x[3] : x[1], g0 = h2 ? x[0] : x[2], g1 = h2 ? x[1] : x[3];
        const float z0 = k0 + __shfl_xor_sync(0xffffffffu, g0, 2), z1 = k1 + __shfl_xor_sync(0xffffffffu, g1, 2);
        mine = (h1 ? z1 : z0) + __shfl_xor_sync(0xffffffffu, h1 ? z0 : z1, 1);
      }
      const int jj = r & 3;                                           // the column (of this thread's 4) that `mine` is of
      const float mi0 = jj < 2 ? (jj == 0 ? i0[0] : i0[1]) : (jj == 2 ? i0[2] : i0[3]);
      if constexpr (KIND == kSweepFwd) {
        // lanes 0-3: u; lanes 4-7: y = scale (alpha S^T q + (k.q) u)
        float u = beta * fmaf(-alpha, mine, mi0);
        const float u_other = __shfl_xor_sync(0xffffffffu, u, 4);
        if (r >= 4)
          static_cast<T *>(p.y)[out + jj] = narrow<T>(p.s.scale * fmaf(alpha, mine, dot * u_other));
        else if (p.u != nullptr)
          p.u[out + jj] = u;
        float uu[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) uu[j] = __shfl_sync(0xffffffffu, u, (lane & 24) | j);
        const float2 al = splat(alpha);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const float2 us = splat(uu[j]);
#pragma unroll
          for (int g = 0; g < M4; ++g) {
            m[j][2 * g] = fma2(make_float2(a0[g].x, a0[g].y), us, mul2(al, m[j][2 * g]));
            m[j][2 * g + 1] = fma2(make_float2(a0[g].z, a0[g].w), us, mul2(al, m[j][2 * g + 1]));
          }
        }
      } else if constexpr (KIND == kSweepDu) {
        const float du = fmaf(p.s.scale * dot, mi0, mine);
        if (r < 4) p.du[out + jj] = du;
        float uu[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) uu[j] = __shfl_sync(0xffffffffu, du, (lane & 24) | j);
        const float2 al = splat(alpha);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const float2 ks = splat(-beta * uu[j]), qs = splat(p.s.scale * i0[j]);
#pragma unroll
          for (int g = 0; g < M4; ++g) {
            m[j][2 * g] = mul2(al, fma2(make_float2(a0[g].x, a0[g].y), ks,
                                        fma2(make_float2(a1[g].x, a1[g].y), qs, m[j][2 * g])));
            m[j][2 * g + 1] = mul2(al, fma2(make_float2(a0[g].z, a0[g].w), ks,
                                            fma2(make_float2(a1[g].z, a1[g].w), qs, m[j][2 * g + 1])));
          }
        }
      } else if constexpr (KIND == kSweepDk) {
        // x0 = u, x1 = dy, x2 = du; independent: q, k.  dk_i = sum_j dS_ij u_j + scale q_i (u.dy)
        if (r < 4) p.dk[out + jj] = fmaf(p.s.scale * dot, mi0, mine);
        const float4 in1 = *reinterpret_cast<const float4 *>(Y1 + t * lo.cols + warp * COLS + cg * PER);
        const float i1[4] = {in1.x, in1.y, in1.z, in1.w};
        const float4 *x2 = reinterpret_cast<const float4 *>(X2 + t * D) + r;
        const float2 al = splat(alpha);
#pragma unroll
        for (int g = 0; g < M4; ++g) {
          const float4 a2 = x2[8 * g];
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            const float2 ks = splat(-beta * i1[j]), qs = splat(p.s.scale * i0[j]);
            m[j][2 * g] = mul2(al, fma2(make_float2(a2.x, a2.y), ks,
                                        fma2(make_float2(a1[g].x, a1[g].y), qs, m[j][2 * g])));
            m[j][2 * g + 1] = mul2(al, fma2(make_float2(a2.z, a2.w), ks,
                                            fma2(make_float2(a1[g].z, a1[g].w), qs, m[j][2 * g + 1])));
          }
        }
      } else {
        // x0 = du, x1 = dy, x2 = u; independent: k.  lanes 0-3: S_{t-1} du, lanes 4-7: S_{t-1} dy
        if (r < 4)
          p.dk[out + jj] = fmaf(-alpha * beta, mine, p.dk[out + jj]);
        else
          p.dq[out + jj] = p.s.scale * fmaf(alpha, mine, dot * mi0);
        const float4 *x2 = reinterpret_cast<const float4 *>(X2 + t * D) + r;
        const float2 al = splat(alpha);
#pragma unroll
        for (int g = 0; g < M4; ++g) {
          const float4 a2 = x2[8 * g];
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            const float2 ks = splat(i0[j]);
            m[j][2 * g] = fma2(make_float2(a2.x, a2.y), ks, mul2(al, m[j][2 * g]));
            m[j][2 * g + 1] = fma2(make_float2(a2.z, a2.w), ks, mul2(al, m[j][2 * g + 1]));
          }
        }
      }
    }
    __syncthreads();   // the next turn overwrites the widened rows and the other raw buffer
  }

  if constexpr (KIND == kSweepDq) {   // <S_T, dS_final> over this warp's 16 rows
    if (p.end != nullptr) {
      float x = 0.0f;
      if (p.dS_final != nullptr) {
        const float *d = p.dS_final + static_cast<long long>(head) * D * D;
#pragma unroll
        for (int g = 0; g < M4; ++g)
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            const float4 f = *reinterpret_cast<const float4 *>(d + (c_thr + j) * D + 32 * g + 4 * r);
            x = fmaf(f.x, m[j][2 * g].x, fmaf(f.y, m[j][2 * g].y, fmaf(f.z, m[j][2 * g + 1].x, fmaf(f.w, m[j][2 * g + 1].y, x))));
          }
      }
      x = head_sum<32>(x);
      if (lane == 0) p.end[static_cast<long long>(head) * (D / COLS) + slice * W + warp] = x;
    }
  }
  if constexpr (kCols) {
    if (p.S_out != nullptr) {
      float *So = p.S_out + static_cast<long long>(head) * D * D;
#pragma unroll
      for (int g = 0; g < M4; ++g) {
        const int i0 = 32 * g + 4 * r;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          *reinterpret_cast<float4 *>(So + (i0 + 2 * e) * D + c_thr) =
              make_float4(m[0][2 * g + e].x, m[1][2 * g + e].x, m[2][2 * g + e].x, m[3][2 * g + e].x);
          *reinterpret_cast<float4 *>(So + (i0 + 2 * e + 1) * D + c_thr) =
              make_float4(m[0][2 * g + e].y, m[1][2 * g + e].y, m[2][2 * g + e].y, m[3][2 * g + e].y);
        }
      }
    }
  }
}

// One warp per token and head: round dq, dk, dv; db = (u.du)(1 - beta);
// gain = q.dq - beta v.du, the summand of dlog alpha.
template <typename T, int D>
__global__ void __launch_bounds__(256) delta_finish_kernel(FinishArgs p) {
  const long long id = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(p.s.B) * p.s.T * p.s.H;
  if (id >= rows) return;
  const int h = static_cast<int>(id % p.s.H);
  const long long bt = id / p.s.H;
  const long long o = id * D;
  const T *q = static_cast<const T *>(p.q) + bt * p.s.ld_qk + h * D, *v = static_cast<const T *>(p.v) + bt * p.s.ld_v + h * D;
  const float beta = gate(widen(static_cast<const T *>(p.b)[bt * p.s.ld_g + h]));
  float g = 0.0f, ub = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int c = 32 * i + lane;
    const float du = p.du[o + c], dq = p.dqf[o + c];
    static_cast<T *>(p.dq)[o + c] = narrow<T>(dq);
    static_cast<T *>(p.dk)[o + c] = narrow<T>(p.dkf[o + c]);
    static_cast<T *>(p.dv)[o + c] = narrow<T>(beta * du);
    g = fmaf(widen(q[c]), dq, fmaf(-beta * du, widen(v[c]), g));
    ub = fmaf(p.u[o + c], du, ub);
  }
  g = head_sum<32>(g);
  ub = head_sum<32>(ub);
  if (lane == 0) {
    const float x = fmaxf(widen(static_cast<const T *>(p.b)[bt * p.s.ld_g + h]), -80.0f);
    static_cast<T *>(p.db)[id] = narrow<T>(ub / (1.0f + expf(x)));   // 1 - beta = 1 / (1 + e^b)
    const long long b = bt / p.s.T, t = bt - b * p.s.T;
    p.gain[(b * p.s.H + h) * p.s.T + t] = g;
  }
}

// da_t = (1 - alpha_t) (sum_{s >= t} gain_s + <S_T, dS_final>), one block per
// head, from the last token back.  The running sum is float64: it passes over
// the whole sequence without the decay that would forget its roundings.
template <typename T>
__global__ void __launch_bounds__(256) delta_da_kernel(FinishArgs p, int slices) {
  __shared__ double part[8];
  const int head = blockIdx.x, b = head / p.s.H, h = head - b * p.s.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float *gain = p.gain + static_cast<long long>(head) * p.s.T;
  double carry = 0.0;
  for (int i = 0; i < slices; ++i) carry += p.end[static_cast<long long>(head) * slices + i];
  for (int last = p.s.T; last > 0; last -= 256) {
    const int t = last - 1 - static_cast<int>(threadIdx.x);
    double x = t >= 0 ? static_cast<double>(gain[t]) : 0.0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    double before = carry, all = carry;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < warp) before += part[i];
      all += part[i];
    }
    if (t >= 0) {
      const long long bt = static_cast<long long>(b) * p.s.T + t;
      const float a = fmaxf(widen(static_cast<const T *>(p.a)[bt * p.s.ld_g + h]), -80.0f);
      static_cast<T *>(p.da)[bt * p.s.H + h] = narrow<T>(static_cast<float>(before + x) / (1.0f + expf(a)));
    }
    carry = all;
    __syncthreads();
  }
}

}  // namespace sweep
}  // namespace esa
