// esa_delta_wy.cu -- the states between chunks of 64 tokens of the gated delta
// rule in float32 (sm_100a), so that long float32 sequences of few heads need
// not be swept token by token from end to end.
//
// With G the running sum of log alpha in the chunk, M_ij = beta_i e^{Gi - Gj}
// k_i.k_j (j < i) and T = (1 + M)^-1, a chunk takes the state S that enters it to
//   S' = e^{G_last} S + K^T L (U0 - W S),   W = T (beta e^G K), U0 = T (beta V), L = e^{G_last - G},
// and the gradient dS' of the state leaving it to
//   dS = e^{G_last} dS' + (scale e^G Q)^T dO - W^T (Z0 + L K dS'),   Z0 = P^T dO,
//   P_ij = scale e^{Gi - Gj} q_i.k_j (j <= i).
// W, U0 and Z0 are formed for all chunks at once (delta_wy_kernel, a thread a
// column of the triangular solve; delta_wz_kernel); the states then take two
// products of 64 D^2 / 16 a chunk and 16 value channels (delta_state_kernel);
// the token sweeps start every chunk from its state.  Everything is float32
// multiply-adds, and within a chunk the results are the sweeps', values that
// are not finite included.
//
// The chain of states is bound by its latency, two products, their sums over
// lanes and three barriers a chunk, and by shared memory: forward 1.8 us a
// chunk at D = 32, 2.5 at 64, 4.0 at 128 (backward 2.3, 3.4, 5.2), against 64
// tokens of a sweep, 11, 13 and 18.5 us.
#include "esa_delta_sweep.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

using sweep::decay;
using sweep::dots;
using sweep::Place;
constexpr int C = sweep::CHUNK, kThreads = 256, kCols = 16;   // tokens, threads, value channels of a state block

__device__ __forceinline__ void copy_or_zero(float *dst, const float *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// Rows [0, len) of `width` floats, `ld` apart, into rows of `pitch`; zeros behind them.
__device__ __forceinline__ void rows_in(float *dst, int pitch, const float *src, long long ld, int len, int width) {
  const int per = width / 4;
  for (int i = threadIdx.x; i < C * per; i += kThreads) {
    const int r = i / per, c = (i - r * per) * 4;
    copy_or_zero(dst + r * pitch + c, src + (r < len ? r * ld : 0) + c, r < len);
  }
}

constexpr int kTri = C + 4;   // pitch of a [64][64] matrix
template <int D> constexpr int wy_floats() { return C * (D + 4) + C * kTri + C * 2 * D + 4 * C; }

template <int D>
__global__ void __launch_bounds__(kThreads) delta_wy_kernel(SweepArgs p) {
  extern __shared__ __align__(16) unsigned char smem[];
  float *K = reinterpret_cast<float *>(smem), *M = K + C * (D + 4), *X = M + C * kTri;
  float2 *G = reinterpret_cast<float2 *>(X + C * 2 * D);
  float *beta = reinterpret_cast<float *>(G + C), *into_beta = beta + C;
  const Place a = sweep::place_of(p.s, p.nc, blockIdx.x / p.nc, blockIdx.x % p.nc);
  const int tid = threadIdx.x;
  rows_in(K, D + 4, static_cast<const float *>(p.k) + a.row * p.s.ld_qk + a.h * D, p.s.ld_qk, a.len, D);
  rows_in(X + D, 2 * D, static_cast<const float *>(p.v) + a.row * p.s.ld_v + a.h * D, p.s.ld_v, a.len, D);
  sweep::cp_async_commit();
  sweep::gates_of<float>(p.s, p.a, p.b, a, G, beta);
  sweep::cp_async_wait<0>();
  __syncthreads();
  {
    const int ti = tid >> 4, tj = tid & 15;
    float acc[4][4];
    dots<D>(K, K, ti, tj, acc);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = ti + 16 * r, j = tj + 16 * c;
        M[i * kTri + j] = j < i ? beta[i] * decay(G[i], G[j]) * acc[r][c] : 0.0f;
      }
  }
  if (tid < C) {
    float *fac = p.fac + a.chunk * 3 * C;
    const float2 zero = make_float2(0.0f, 0.0f);
    const float into = decay(G[tid], zero);
    into_beta[tid] = beta[tid] * into;
    fac[tid] = decay(G[C - 1], G[tid]);
    fac[C + tid] = p.s.scale * into;
    fac[2 * C + tid] = decay(G[C - 1], zero);
  }
  __syncthreads();
  for (int i = tid; i < C * (D / 4); i += kThreads) {   // the right sides: beta e^G K, beta V
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const float4 x = *reinterpret_cast<const float4 *>(K + r * (D + 4) + c);
    float4 *o = reinterpret_cast<float4 *>(X + r * 2 * D + c);
    const float f = into_beta[r], be = beta[r];
    *o = make_float4(f * x.x, f * x.y, f * x.z, f * x.w);
    const float4 y = o[D / 4];   // V, copied there
    o[D / 4] = make_float4(be * y.x, be * y.y, be * y.z, be * y.w);
  }
  __syncthreads();
  // a thread a column of W and U0: substitution in blocks of 16 tokens.  Rolled
  // where that costs little: with few chunks the time is that of fetching the
  // code (all of it unrolled, 21 us for any number up to 100 of them).
  if (tid < 2 * D) {
    float *x = X + tid;
#pragma unroll 1
    for (int blk = 0; blk < C / 16; ++blk) {
      const float *Mb = M + 16 * blk * kTri;
      float acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = x[(16 * blk + i) * 2 * D];
#pragma unroll 1
      for (int j = 0; j < 16 * blk; j += 4) {
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = x[(j + e) * 2 * D];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 m = *reinterpret_cast<const float4 *>(Mb + i * kTri + j);
          acc[i] = fmaf(-m.x, z[0], fmaf(-m.y, z[1], fmaf(-m.z, z[2], fmaf(-m.w, z[3], acc[i]))));
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int j = 0; j < i; j += 4) {
          const float4 m = *reinterpret_cast<const float4 *>(Mb + i * kTri + 16 * blk + j);
          acc[i] = fmaf(-m.x, acc[j], acc[i]);
          if (j + 1 < i) acc[i] = fmaf(-m.y, acc[j + 1], acc[i]);
          if (j + 2 < i) acc[i] = fmaf(-m.z, acc[j + 2], acc[i]);
          if (j + 3 < i) acc[i] = fmaf(-m.w, acc[j + 3], acc[i]);
        }
        x[(16 * blk + i) * 2 * D] = acc[i];
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < C * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const float4 *o = reinterpret_cast<const float4 *>(X + r * 2 * D + c);
    const long long at = a.chunk * (C * D) + r * D + c;
    *reinterpret_cast<float4 *>(p.wt + at) = o[0];
    *reinterpret_cast<float4 *>(p.u0 + at) = o[D / 4];
  }
}

template <int D> constexpr int wz_floats() { return 2 * C * (D + 4) + C * kTri + C * D + 3 * C; }

// Z0 = P^T dO (in the place of U0, which only the forward's states needed)
template <int D>
__global__ void __launch_bounds__(kThreads) delta_wz_kernel(SweepArgs p) {
  extern __shared__ __align__(16) unsigned char smem[];
  float *K = reinterpret_cast<float *>(smem), *Q = K + C * (D + 4), *P = Q + C * (D + 4), *O = P + C * kTri;
  float2 *G = reinterpret_cast<float2 *>(O + C * D);
  float *beta = reinterpret_cast<float *>(G + C);
  const Place a = sweep::place_of(p.s, p.nc, blockIdx.x / p.nc, blockIdx.x % p.nc);
  const int tid = threadIdx.x;
  const long long ldc = static_cast<long long>(p.s.H) * D;
  rows_in(K, D + 4, static_cast<const float *>(p.k) + a.row * p.s.ld_qk + a.h * D, p.s.ld_qk, a.len, D);
  rows_in(Q, D + 4, static_cast<const float *>(p.q) + a.row * p.s.ld_qk + a.h * D, p.s.ld_qk, a.len, D);
  rows_in(O, D, static_cast<const float *>(p.dy) + a.row * ldc + a.h * D, ldc, a.len, D);
  sweep::cp_async_commit();
  sweep::gates_of<float>(p.s, p.a, p.b, a, G, beta);
  sweep::cp_async_wait<0>();
  __syncthreads();
  {
    const int ti = tid >> 4, tj = tid & 15;
    float acc[4][4];
    dots<D>(Q, K, ti, tj, acc);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = ti + 16 * r, j = tj + 16 * c;
        P[i * kTri + j] = j <= i ? p.s.scale * decay(G[i], G[j]) * acc[r][c] : 0.0f;
      }
  }
  __syncthreads();
#pragma unroll 1
  for (int tile = tid; tile < (C / 4) * (D / 4); tile += kThreads) {
    const int j = tile / (D / 4) * 4, c = tile % (D / 4) * 4;
    float z[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[r][e] = 0.0f;
#pragma unroll 4
    for (int i = j; i < C; ++i) {
      const float4 w = *reinterpret_cast<const float4 *>(P + i * kTri + j), o = *reinterpret_cast<const float4 *>(O + i * D + c);
      const float ws[4] = {w.x, w.y, w.z, w.w}, os[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[r][e] = fmaf(ws[r], os[e], z[r][e]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<float4 *>(p.u0 + a.chunk * (C * D) + (j + r) * D + c) = make_float4(z[r][0], z[r][1], z[r][2], z[r][3]);
  }
}

template <int D, bool BWD>
struct StateSmem {   // in floats
  static constexpr int pitch = BWD && D == 128 ? D : D + 4, mat = C * pitch, sp = kCols + 4;
  static constexpr int yp = D == 32 ? 20 : D == 64 ? 24 : 16;   // rows of Y and dO: no bank conflicts between `SPL` rows
  static constexpr int first = 0, second = mat, third = 2 * mat;        // factor of the state; K (W); Q
  static constexpr int add = (BWD ? 3 : 2) * mat, dout = add + C * kCols;  // U0 (Z0) slice, dO slice
  static constexpr int fac = dout + (BWD ? C * yp : 0), stage = fac + 3 * C;
  static constexpr int S = 2 * stage, Y = S + D * sp, total = Y + C * yp;
};

// Float4 `cg` of row d of the state: rows 4, 8 and 12 apart, which the four
// quarters of a product read together, lie in different banks.
__device__ __forceinline__ int state_at(int d, int cg) { return d * (kCols + 4) + 4 * (cg ^ ((d >> 3 & 1) << 1)); }

// The state (its gradient) from chunk to chunk: a block carries 16 value channels of a head.
template <int D, bool BWD>
__global__ void __launch_bounds__(kThreads) delta_state_kernel(SweepArgs p) {
  using L = StateSmem<D, BWD>;
  constexpr int slices = D / kCols, SPL = kThreads / D;   // threads that share a tile of the state
  extern __shared__ __align__(16) unsigned char smem[];
  float *sm = reinterpret_cast<float *>(smem), *S = sm + L::S, *Y = sm + L::Y;
  const int tid = threadIdx.x, head = blockIdx.x / slices, c0 = blockIdx.x % slices * kCols;
  const long long ldc = static_cast<long long>(p.s.H) * D, state0 = static_cast<long long>(head) * D * D;
  const float *k = static_cast<const float *>(p.k), *q = static_cast<const float *>(p.q), *dy = static_cast<const float *>(p.dy);
  auto fetch = [&](int it, int buf) {
    if (it < p.nc) {
      const Place a = sweep::place_of(p.s, p.nc, head, BWD ? p.nc - 1 - it : it);
      float *s = sm + buf * L::stage;
      const float *w = p.wt + a.chunk * (C * D);
      rows_in(s + (BWD ? L::second : L::first), L::pitch, w, D, C, D);
      rows_in(s + (BWD ? L::first : L::second), L::pitch, k + a.row * p.s.ld_qk + a.h * D, p.s.ld_qk, a.len, D);
      rows_in(s + L::add, kCols, p.u0 + a.chunk * (C * D) + c0, D, C, kCols);
      if constexpr (BWD) {
        rows_in(s + L::third, L::pitch, q + a.row * p.s.ld_qk + a.h * D, p.s.ld_qk, a.len, D);
        rows_in(s + L::dout, L::yp, dy + a.row * ldc + a.h * D + c0, ldc, a.len, kCols);
      }
      if (tid < 3 * C / 4) copy_or_zero(s + L::fac + 4 * tid, p.fac + a.chunk * 3 * C + 4 * tid, true);
    }
    sweep::cp_async_commit();
  };
  fetch(0, 0);
  for (int i = tid; i < D * (kCols / 4); i += kThreads) {
    const int d = i / (kCols / 4), c = i % (kCols / 4) * 4;
    float4 x = make_float4(0, 0, 0, 0);
    if (p.S_in) x = *reinterpret_cast<const float4 *>(p.S_in + state0 + d * D + c0 + c);
    *reinterpret_cast<float4 *>(S + state_at(d, c / 4)) = x;
  }
  auto keep = [&](float *base) {   // the state of this moment
    for (int i = tid; i < D * (kCols / 4); i += kThreads) {
      const int d = i / (kCols / 4), c = i % (kCols / 4) * 4;
      *reinterpret_cast<float4 *>(base + d * D + c0 + c) = *reinterpret_cast<const float4 *>(S + state_at(d, c / 4));
    }
  };
  for (int it = 0; it < p.nc; ++it) {
    const float *s = sm + (it & 1) * L::stage, *fac = s + L::fac;
    fetch(it + 1, (it + 1) & 1);
    sweep::cp_async_wait<1>();
    __syncthreads();
    keep((BWD ? p.dS_ck : p.S_ck) + (static_cast<long long>(head) * p.nc + (BWD ? p.nc - 1 - it : it)) * D * D);
    {   // Y = L (U0 - W S), backward Z0 + L K dS: rows rg + 16 r, columns 4 cg, a quarter of the channels
      const int sq = tid & 3, cg = (tid >> 2) & 3, rg = tid >> 4;
      float acc[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = 0.0f;
#pragma unroll 2
      for (int d = 4 * sq; d < D; d += 16) {
        float4 x[4], y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = *reinterpret_cast<const float4 *>(s + L::first + (rg + 16 * r) * L::pitch + d);
          y[r] = *reinterpret_cast<const float4 *>(S + state_at(d + r, cg));
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float xs[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[r][0] = fmaf(xs[e], y[e].x, acc[r][0]);
            acc[r][1] = fmaf(xs[e], y[e].y, acc[r][1]);
            acc[r][2] = fmaf(xs[e], y[e].z, acc[r][2]);
            acc[r][3] = fmaf(xs[e], y[e].w, acc[r][3]);
          }
        }
      }
      float mine[4];   // row rg + 16 sq
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = acc[r][e];
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          if (r == sq) mine[e] = x;
        }
      const int row = rg + 16 * sq;
      const float4 u = *reinterpret_cast<const float4 *>(s + L::add + row * kCols + 4 * cg);
      const float f = fac[row];
      float4 o;
      if constexpr (BWD)
        o = make_float4(-fmaf(f, mine[0], u.x), -fmaf(f, mine[1], u.y), -fmaf(f, mine[2], u.z), -fmaf(f, mine[3], u.w));
      else
        o = make_float4(f * (u.x - mine[0]), f * (u.y - mine[1]), f * (u.z - mine[2]), f * (u.w - mine[3]));
      *reinterpret_cast<float4 *>(Y + row * L::yp + 4 * cg) = o;
    }
    __syncthreads();
    {   // S <- e^{G_last} S + K^T Y, backward - W^T Y + Q^T (scale e^G dO)
      const int ss = tid % SPL, cg = tid / SPL % 4, dg = tid / (4 * SPL);
      float acc[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = 0.0f;
      auto rank = [&](const float *A, int i, float4 y) {
        const float4 x = *reinterpret_cast<const float4 *>(A + i * L::pitch + 4 * dg);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][e] = fmaf(xs[r], ys[e], acc[r][e]);
      };
#pragma unroll 4
      for (int i = ss; i < C; i += SPL) {
        rank(s + L::second, i, *reinterpret_cast<const float4 *>(Y + i * L::yp + 4 * cg));
        if constexpr (BWD) {
          const float4 o = *reinterpret_cast<const float4 *>(s + L::dout + i * L::yp + 4 * cg);
          const float f = fac[C + i];
          rank(s + L::third, i, make_float4(f * o.x, f * o.y, f * o.z, f * o.w));
        }
      }
#pragma unroll
      for (int o = 1; o < SPL; o <<= 1)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][e] += __shfl_xor_sync(0xffffffffu, acc[r][e], o);
      if (ss == 0) {
        const float g = fac[2 * C];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float4 *o = reinterpret_cast<float4 *>(S + state_at(4 * dg + r, cg));
          const float4 x = *o;
          *o = make_float4(fmaf(g, x.x, acc[r][0]), fmaf(g, x.y, acc[r][1]), fmaf(g, x.z, acc[r][2]), fmaf(g, x.w, acc[r][3]));
        }
      }
    }
    __syncthreads();
  }
  if (p.S_out) keep(p.S_out + state0);
}

template <typename K>
int launch(K kern, long long blocks, int floats, const SweepArgs &a, cudaStream_t st) {
  const int bytes = floats * 4;
  if (bytes > 48 * 1024) {
    const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (rc) return rc;
  }
  kern<<<static_cast<unsigned>(blocks), kThreads, bytes, st>>>(a);
  return runtime_status(cudaGetLastError());
}

template <int D>
int run(bool bwd, const SweepArgs &a, cudaStream_t st) {
  const long long heads = static_cast<long long>(a.s.B) * a.s.H, chunks = heads * a.nc;
  int rc = bwd ? launch(delta_wz_kernel<D>, chunks, wz_floats<D>(), a, st)
               : launch(delta_wy_kernel<D>, chunks, wy_floats<D>(), a, st);
  if (rc) return rc;
  return bwd ? launch(delta_state_kernel<D, true>, heads * (D / kCols), StateSmem<D, true>::total, a, st)
             : launch(delta_state_kernel<D, false>, heads * (D / kCols), StateSmem<D, false>::total, a, st);
}

}  // namespace

int launch_delta_states(bool bwd, const SweepArgs &a, cudaStream_t st) {
  switch (a.s.D) {
    case 32: return run<32>(bwd, a, st);
    case 64: return run<64>(bwd, a, st);
    case 128: return run<128>(bwd, a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace esa
