// esa_delta_sweep.cuh -- the gated delta rule token by token (sm_100a).
//
//   alpha = sigmoid(a), beta = sigmoid(b) (logits clamped at -80 below),
//   u_t = beta_t (v_t - alpha_t S_{t-1}^T k_t),  S_t = alpha_t S_{t-1} + k_t u_t^T,
//   y_t = scale S_t^T q_t,      S [D key channels][D value channels], float32.
//
// A sweep keeps a matrix M in registers and visits the tokens in order.  D / 32
// neighbouring lanes share one entry of M's independent axis, 32 entries of
// the other, the split axis, each; a dot product over the split axis is 32
// multiply-adds a lane and log2(D / 32) shuffles, and the update needs no
// other thread.  The forward has M = S with its value channels independent:
// each is a recurrence of its own.  The gradients need both orientations:
//   kSweepFwd  forward,  M = S:    u (kept for the backward), y, S_T; the state entering each chunk of 64 tokens
//   kSweepDu   backward, M = dS:   du_t = dS_t^T k_t with dS_t += scale q_t dy_t^T first, then
//                                  dS <- alpha_t (dS - beta_t k_t du_t^T); dS_init; the gradient leaving each chunk
//   kSweepDk   backward, M = dS^T: dk_t = dS_t u_t
//   kSweepDq   forward,  M = S^T:  dk_t's other part -alpha_t beta_t S_{t-1} du_t, dq_t = scale S_t dy_t, <dS, S> at each chunk's end
// The first two pass over the whole sequence, or start every chunk from the
// states of esa_delta_wy.cu and take all chunks at once; the last two always do.
//
// All arithmetic is float32, as the state is; this is the path of float32
// tensors and of short sequences.
// With few heads it is bound by the latency of a token (load k, dot, shuffles,
// update), with many by the issue of some 200 instructions a token, warp and
// 32 x 32 of the state.  Measured a token, few heads: 174 ns at D = 32, 205
// at 64, 302 at 128.  (Columns shared by 8 lanes whatever D: 390, 450,
// 600; a whole column a thread: 312, 448, 924, since one warp then issues all
// of it.)  More warps per block share the staged rows; fewer give more blocks:
// see sweep_warps().
//
// Rows are staged 16 or 32 tokens at a time: cp.async into a double buffer in
// the tensors' own type, then widened once to float32 for the block's warps.
#pragma once

#include "esa_common.cuh"
#include "esa_delta.h"

namespace esa {
namespace sweep {

constexpr int CHUNK = 64;    // tokens between the states that are kept
template <int D> constexpr int lanes() { return D / 32; }         // that share the split axis
template <int D> constexpr int columns() { return 32 / lanes<D>(); }   // independent entries a warp
template <int D> constexpr int tokens() { return D == 128 ? 16 : 32; }   // staged at a time

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow(float v) { return v; }
template <> __device__ __forceinline__ __half narrow(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 narrow(float v) { return __float2bfloat16_rn(v); }

// Logits are clamped at -80 below; a NaN stays one, as everything after it.
__device__ __forceinline__ float clamp(float x) { return x < -80.0f ? -80.0f : x; }
__device__ __forceinline__ float gate(float x) { return 1.0f / (1.0f + expf(-clamp(x))); }

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

// Shared memory, byte offsets, for W warps.
template <typename T, int D, int KIND>
struct Layout {
  using R = Rows<T, KIND>;
  static constexpr bool kWide = sizeof(T) == 4;
  static constexpr int TC = tokens<D>();
  int cols;
  size_t x0, x1, x2, y0, y1, raw;    // raw buffer (one stage)
  size_t fx0, fx1, fy0, fy1, tok;    // widened rows and per-token scalars, from the start
  size_t total;
  __host__ __device__ explicit Layout(int W) {
    cols = columns<D>() * W;
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
    tok = o; o += 2 * TC * sizeof(float);
    total = o;
  }
};

template <typename T, int D, int KIND>
__device__ __forceinline__ void sweep_body(const SweepArgs &p) {
  constexpr bool kReverse = KIND == kSweepDu || KIND == kSweepDk;
  constexpr bool kCols = KIND == kSweepFwd || KIND == kSweepDu;   // whole sequences, value channels independent
  constexpr int TC = tokens<D>(), SP = lanes<D>();
  using R = Rows<T, KIND>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int W = blockDim.x >> 5;
  const Layout<T, D, KIND> lo(W);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sl = threadIdx.x % SP, jj = threadIdx.x / SP;
  const int slices = D / lo.cols;
  const int slice = blockIdx.x % slices;
  int head = blockIdx.x / slices, chunk = 0;           // head = b H + h
  const bool cut = !kCols || p.cut;                    // a chunk a block, else the sequence
  if (cut) {
    chunk = head % p.nc;
    head /= p.nc;
  }
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int c_blk = slice * lo.cols, j = c_blk + jj;   // first independent entry of the block, this thread's
  const int t_begin = cut ? chunk * CHUNK : 0, t_end = cut ? min(p.s.T, t_begin + CHUNK) : p.s.T;
  const long long tok0 = static_cast<long long>(b) * p.s.T;
  const long long ldc = static_cast<long long>(p.s.H) * D;   // contiguous rows (dy, y, scratch)
  const long long state0 = static_cast<long long>(head) * D * D;

  // This lane's split entries: 4 (SP i + sl) + 0..3 at m[2 i], m[2 i + 1]
  float2 m[16];
  if constexpr (kCols) {
    const float *Sin = p.S_in ? p.S_in + state0 + 4 * sl * D + j : nullptr;
    if (cut)
      Sin = (KIND == kSweepDu ? p.dS_ck : p.S_ck) + (static_cast<long long>(head) * p.nc + chunk) * D * D + 4 * sl * D + j;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 4 * SP * (i >> 1) + 2 * (i & 1);
      m[i] = Sin ? make_float2(Sin[r * D], Sin[(r + 1) * D]) : make_float2(0.0f, 0.0f);
    }
  } else {
    const float4 *Sin = reinterpret_cast<const float4 *>(
        (KIND == kSweepDk ? p.dS_ck : p.S_ck) + (static_cast<long long>(head) * p.nc + chunk) * D * D + j * D) + sl;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 x = Sin[SP * i];
      m[2 * i] = make_float2(x.x, x.y);
      m[2 * i + 1] = make_float2(x.z, x.w);
    }
  }
  // M to [D][D] memory: the final state, and what enters (leaves) a chunk
  auto keep = [&](float *base) {
    float *o = base + 4 * sl * D + j;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 4 * SP * (i >> 1) + 2 * (i & 1);
      o[r * D] = m[i].x;
      o[(r + 1) * D] = m[i].y;
    }
  };

  const T *q = static_cast<const T *>(p.q) + h * D, *k = static_cast<const T *>(p.k) + h * D;
  const T *v = static_cast<const T *>(p.v), *dy = static_cast<const T *>(p.dy);
  const T *ga = static_cast<const T *>(p.a), *gb = static_cast<const T *>(p.b);
  const int nch = (t_end - t_begin + TC - 1) / TC;

  auto fetch = [&](int c, int buf) {
    const int t0 = t_begin + c * TC, n = min(TC, t_end - t0);
    const long long row = tok0 + t0;
    unsigned char *s = smem + buf * lo.raw;
    if constexpr (kCols) {
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
    const int t = t_begin + c * TC + threadIdx.x;
    if (threadIdx.x < TC && t < t_end) {
      ga_next = widen(ga[(tok0 + t) * p.s.ld_g + h]);
      gb_next = widen(gb[(tok0 + t) * p.s.ld_g + h]);
    }
  };

  float *tok = reinterpret_cast<float *>(smem + lo.tok);   // alpha, beta, TC each
  if (nch > 0) {
    fetch(kReverse ? nch - 1 : 0, 0);
    fetch_gates(kReverse ? nch - 1 : 0);
  }
  for (int it = 0; it < nch; ++it) {
    const int c = kReverse ? nch - 1 - it : it, buf = it & 1;
    const int t0 = t_begin + c * TC, n = min(TC, t_end - t0);
    if constexpr (KIND == kSweepFwd)
      if (p.S_ck != nullptr && !cut && t0 % CHUNK == 0) keep(p.S_ck + (static_cast<long long>(head) * p.nc + t0 / CHUNK) * D * D);
    if constexpr (KIND == kSweepDu)
      if (!cut && (t0 + n == t_end || (t0 + n) % CHUNK == 0)) keep(p.dS_ck + (static_cast<long long>(head) * p.nc + (t0 + n - 1) / CHUNK) * D * D);
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

    const int step = kReverse ? -1 : 1;
    int t = kReverse ? n - 1 : 0;
    // the first operand of the coming token is loaded while this one is finished
    float4 x[8];
    float alpha, beta, in;
    auto load = [&](const float *rows, int at) {
      const float4 *r = reinterpret_cast<const float4 *>(rows + at * D) + sl;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = r[SP * i];
      alpha = tok[at];
      beta = tok[TC + at];
      in = Y0[at * lo.cols + jj];
    };
    // sum over the lanes of an entry
    auto total = [&](float2 a, float2 b, float2 c, float2 d) {
      const float2 z = add2(add2(a, b), add2(c, d));
      float f = z.x + z.y;
#pragma unroll
      for (int o = 1; o < SP; o <<= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
      return f;
    };
    load(KIND == kSweepDq ? X0 : KIND == kSweepDk ? X1 : KIND == kSweepDu ? X1 : X0, t);
#pragma unroll 1
    for (int e = 0; e < n; ++e, t += step) {
      const long long out = (tok0 + t0 + t) * ldc + h * D + j;
      const float2 al = splat(alpha);
      const int next = e + 1 < n ? t + step : t;
      float2 P[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) P[i] = make_float2(0.0f, 0.0f);
      if constexpr (kReverse) {
        // M += scale x1 in^T (dO, q or the other way round), then P = sum x0 M (k or u), then
        // M <- alpha (M - beta k du^T).  x holds x1.
        const float2 qs = splat(p.s.scale * in);
        const float4 *x0 = reinterpret_cast<const float4 *>(X0 + t * D) + sl;
        const float4 *x2 = reinterpret_cast<const float4 *>(KIND == kSweepDk ? X2 + t * D : X0 + t * D) + sl;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 a0 = x0[SP * i];
          m[2 * i] = fma2(make_float2(x[i].x, x[i].y), qs, m[2 * i]);
          m[2 * i + 1] = fma2(make_float2(x[i].z, x[i].w), qs, m[2 * i + 1]);
          P[(2 * i) & 3] = fma2(make_float2(a0.x, a0.y), m[2 * i], P[(2 * i) & 3]);
          P[(2 * i + 1) & 3] = fma2(make_float2(a0.z, a0.w), m[2 * i + 1], P[(2 * i + 1) & 3]);
        }
        const float dp = total(P[0], P[1], P[2], P[3]);
        const float ks = KIND == kSweepDk ? -beta * Y1[t * lo.cols + jj] : -beta * dp;
        if (sl == 0) (KIND == kSweepDk ? p.dk : p.du)[out] = dp;
        load(X1, next);
        const float2 k2 = splat(ks);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 a2 = x2[SP * i];
          m[2 * i] = mul2(al, fma2(make_float2(a2.x, a2.y), k2, m[2 * i]));
          m[2 * i + 1] = mul2(al, fma2(make_float2(a2.z, a2.w), k2, m[2 * i + 1]));
        }
      } else {
        // P = sum x0 M (k or du), M <- alpha M + x2 w^T, then sum x1 M (q or dy).  x holds x0.
        float2 Q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) Q[i] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          P[(2 * i) & 3] = fma2(make_float2(x[i].x, x[i].y), m[2 * i], P[(2 * i) & 3]);
          P[(2 * i + 1) & 3] = fma2(make_float2(x[i].z, x[i].w), m[2 * i + 1], P[(2 * i + 1) & 3]);
        }
        const float4 *x1 = reinterpret_cast<const float4 *>(X1 + t * D) + sl;
        const float4 *x2 = reinterpret_cast<const float4 *>(KIND == kSweepDq ? X2 + t * D : X0 + t * D) + sl;
        const float dp = total(P[0], P[1], P[2], P[3]);
        float w;
        if constexpr (KIND == kSweepFwd) {
          w = beta * fmaf(-alpha, dp, in);
          if (p.u != nullptr && sl == 0) p.u[out] = w;
        } else {
          w = in;
          if (sl == 0) p.dk2[out] = -alpha * beta * dp;
        }
        const float2 ws = splat(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float4 a2;
          if constexpr (KIND == kSweepDq) a2 = x2[SP * i];
          else a2 = x[i];
          const float4 a1 = x1[SP * i];
          m[2 * i] = fma2(make_float2(a2.x, a2.y), ws, mul2(al, m[2 * i]));
          m[2 * i + 1] = fma2(make_float2(a2.z, a2.w), ws, mul2(al, m[2 * i + 1]));
          Q[(2 * i) & 3] = fma2(make_float2(a1.x, a1.y), m[2 * i], Q[(2 * i) & 3]);
          Q[(2 * i + 1) & 3] = fma2(make_float2(a1.z, a1.w), m[2 * i + 1], Q[(2 * i + 1) & 3]);
        }
        load(X0, next);
        const float dq = p.s.scale * total(Q[0], Q[1], Q[2], Q[3]);
        if (sl == 0) {
          if constexpr (KIND == kSweepFwd) static_cast<T *>(p.y)[out] = narrow<T>(dq);
          else p.dq[out] = dq;
        }
      }
    }
    __syncthreads();   // the next turn overwrites the widened rows and the other raw buffer
  }

  if constexpr (KIND == kSweepDq) {   // <dS, S> at the chunk's end over this warp's rows
    const float4 *g = reinterpret_cast<const float4 *>(p.dS_ck + (static_cast<long long>(head) * p.nc + chunk) * D * D + j * D) + sl;
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 f = g[SP * i];
      x = fmaf(f.x, m[2 * i].x, fmaf(f.y, m[2 * i].y, fmaf(f.z, m[2 * i + 1].x, fmaf(f.w, m[2 * i + 1].y, x))));
    }
    x = head_sum<32>(x);
    if (lane == 0) p.end[(static_cast<long long>(head) * p.nc + chunk) * (D / columns<D>()) + slice * W + warp] = x;
  }
  if constexpr (kCols) {
    if (p.S_out != nullptr && !cut) keep(p.S_out + state0);
  }
}

template <typename T, int D, int KIND>
__global__ void __launch_bounds__(D * lanes<D>()) delta_sweep_kernel(SweepArgs p) {
  sweep_body<T, D, KIND>(p);
}

// The two sweeps over key channels, which do not need one another, in one
// launch: with few chunks both fit on the device (48 chunks of D = 32: 15 us,
// one behind the other 14 + 16), with many they share it evenly (4096 chunks:
// 195 and 99 + 180).
template <typename T, int D>
__global__ void __launch_bounds__(D * lanes<D>()) delta_keys_kernel(SweepArgs p) {
  if (blockIdx.y == 0) sweep_body<T, D, kSweepDk>(p);
  else sweep_body<T, D, kSweepDq>(p);
}

// One warp per token and head: round dq, dk, dv; db = (u.du)(1 - beta);
// gain = q.dq - beta v.du, the summand of dlog alpha (esa_delta_gate.cu).
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
    static_cast<T *>(p.dk)[o + c] = narrow<T>(p.dkf[o + c] + p.dk2[o + c]);
    static_cast<T *>(p.dv)[o + c] = narrow<T>(beta * du);
    g = fmaf(widen(q[c]), dq, fmaf(-beta * du, widen(v[c]), g));
    ub = fmaf(p.u[o + c], du, ub);
  }
  g = head_sum<32>(g);
  ub = head_sum<32>(ub);
  if (lane == 0) {
    const float x = clamp(widen(static_cast<const T *>(p.b)[bt * p.s.ld_g + h]));
    static_cast<T *>(p.db)[id] = narrow<T>(ub / (1.0f + expf(x)));   // 1 - beta = 1 / (1 + e^b)
    const long long b = bt / p.s.T, t = bt - b * p.s.T;
    p.gain[(b * p.s.H + h) * p.s.T + t] = g;
  }
}

// ---- chunk by chunk (esa_delta_wy.cu, esa_delta_gate.cu) ----------------------
struct Place {
  int b, h, t0, len;      // batch entry, head, first token, tokens
  long long row, chunk;   // first token's row, index of the chunk
};
// Chunk n of a head.
__device__ __forceinline__ Place place_of(const DeltaShape &s, int nc, int head, int n) {
  Place a;
  a.b = head / s.H;
  a.h = head - a.b * s.H;
  a.t0 = n * CHUNK;
  a.len = min(CHUNK, s.T - a.t0);
  a.row = static_cast<long long>(a.b) * s.T + a.t0;
  a.chunk = static_cast<long long>(head) * nc + n;
  return a;
}

// G in two terms (differences of sums that may reach thousands are
// exponentiated) and beta, by the first warp; alpha = 1, beta = 0 behind the end.
template <typename T>
__device__ __forceinline__ void gates_of(const DeltaShape &s, const void *a_, const void *b_, const Place &a, float2 *G, float *beta) {
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  const T *ga = static_cast<const T *>(a_), *gb = static_cast<const T *>(b_);
  double la[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    la[e] = 0.0;
    float be = 0.0f;
    if (i < a.len) {
      la[e] = -log1pf(expf(-clamp(widen(ga[(a.row + i) * s.ld_g + a.h]))));
      be = gate(widen(gb[(a.row + i) * s.ld_g + a.h]));
    }
    beta[i] = be;
  }
  double x = la[0] + la[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const double before = __shfl_up_sync(0xffffffffu, x, 1), first = (lane > 0 ? before : 0.0) + la[0];
  const float f0 = static_cast<float>(first), f1 = static_cast<float>(x);
  G[2 * lane] = make_float2(f0, static_cast<float>(first - f0));
  G[2 * lane + 1] = make_float2(f1, static_cast<float>(x - f1));
}
__device__ __forceinline__ float decay(float2 i, float2 j) { return expf((i.x - j.x) + (i.y - j.y)); }

// X Y^T of two [64][D] tiles: rows ti + 16 r, columns tj + 16 c.
template <int D>
__device__ __forceinline__ void dots(const float *X, const float *Y, int ti, int tj, float (&acc)[4][4]) {
  constexpr int P = D + 4;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[r][c] = 0.0f;
#pragma unroll 2
  for (int d = 0; d < D; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = *reinterpret_cast<const float4 *>(X + (ti + 16 * r) * P + d);
      y[r] = *reinterpret_cast<const float4 *>(Y + (tj + 16 * r) * P + d);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        acc[r][c] = fmaf(x[r].x, y[c].x, fmaf(x[r].y, y[c].y, fmaf(x[r].z, y[c].z, fmaf(x[r].w, y[c].w, acc[r][c]))));
  }
}

}  // namespace sweep
}  // namespace esa
