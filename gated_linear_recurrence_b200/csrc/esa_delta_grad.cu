// esa_delta_grad.cu -- the backward of the chunked gated delta rule, second
// kernel: the gradients that each chunk forms by itself (sm_100a).
//
// With S the state entering the chunk, dS the gradient of the state leaving
// it, U and du the chunk's rows of u and of its gradient, and
// D_ij = e^{Gi - Gj} (j <= i):
//   dP_ij = scale D_ij dO_i.U_j (j <= i),   N_ij = -beta_i D_ij du_i.U_j (j < i),
//   dQ = scale e^G dO S^T + dP K,
//   dK = e^{G_last - G} U dS^T - beta e^G du S^T + dP^T Q + N K + N^T K,
//   db = (du.u)(1 - beta),
//   da_i = (1 - alpha_i)(c + sum_{s >= i} (q_s.dq_s - beta_s v_s.du_s)),
//   c = <dS, S leaving> = e^{G_last} <dS, S> + sum_j k_j.(e^{G_last - G_j} u_j dS^T).
// Sums of the gate's gradient start anew in every chunk, from c.
//
// These are outputs in 16 bits: S, dS, U, du, dP and N are operands in one
// float16 term each (2^-12 of a value on average, against 2^-9 for a bfloat16
// output and 2^-12 for a float16 one).  Tiles whose rows or channel groups
// have powers of two of their own are brought to one per tile first.
//
// One block of 8 warps per chunk and head: warp (m, half) has 16 tokens and
// half of the channels.  About 2,500 mma at D = 128 against 190 KB read and
// written, so memory traffic and mma bound it alike.
#include "esa_delta_chunk.h"
#include "esa_delta_sweep.cuh"
#include "esa_mma.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

constexpr int kThreads = 256;

template <int D>
struct GradSmem {
  static constexpr int row = 64 * D * 2, mat = D * D * 2;
  static constexpr int k = 0, q = row, u = 2 * row, r = 3 * row, o = 4 * row, s = 5 * row, ds = s + mat, dp = ds + mat,
                       n = dp + 8192, vec = n + 8192, total = vec + 13 * 64 * 4 + 128;
};

// Rows of 16-byte units of a plain [rows][D] float16 array into a swizzled tile.
template <int D>
__device__ __forceinline__ void fetch_tile(uint32_t dst, const __half *src, int rows) {
  constexpr int U = D / 8;
  for (int i = threadIdx.x; i < rows * U; i += kThreads) cp_async16_s(dst + tile_off<D * 2>(i / U, i % U), src + i * 8);
}

// Multiply unit (row, unit) of a tile by f, a power of two of at most 1.
__device__ __forceinline__ void scale_unit(unsigned char *p, float f) {
  uint4 v = *reinterpret_cast<uint4 *>(p);
  __half2 *h = reinterpret_cast<__half2 *>(&v);
  const __half2 s = __float2half2_rn(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __hmul2(h[i], s);
  *reinterpret_cast<uint4 *>(p) = v;
}

// Largest of n (<= 64) positive factors, seen by every thread.
__device__ __forceinline__ float factor_top(const float *f, int n) {
  float x = 0.0f;
  for (int i = threadIdx.x & 31; i < n; i += 32) x = fmaxf(x, f[i]);
  x = warp_max(x);
  return x > 0.0f ? x : 1.0f;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) delta_grad_kernel(ChunkArgs p) {
  using L = GradSmem<D>;
  using R = ChunkRecord<D>;
  constexpr int NH = D / 16;      // accumulator tiles of half the channels
  constexpr int SLC = D / 16;     // channel groups
  extern __shared__ __align__(128) unsigned char smem[];
  float *vec = reinterpret_cast<float *>(smem + L::vec);
  float *G = vec, *Gl = vec + 64, *beta = vec + 128, *kf = vec + 192, *qf = vec + 256, *oinv = vec + 320;
  float *qdq = vec + 384, *wk = vec + 512, *vdu = vec + 640, *udu = vec + 704, *red = vec + 768;   // qdq, wk: two halves
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const long long c = blockIdx.x;
  const int head = static_cast<int>(c / p.w.nc), n = static_cast<int>(c - static_cast<long long>(head) * p.w.nc);
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int t0 = n * kChunk, len = min(kChunk, p.s.T - t0);
  const long long row = static_cast<long long>(b) * p.s.T + t0, ldc = static_cast<long long>(p.s.H) * D;
  const unsigned char *rec = p.w.rec + c * R::bytes;
  const uint32_t s0 = smem_u32(smem);
  const float *tokg = reinterpret_cast<const float *>(rec + R::tok);

  copy_linear<2 * L::row, kThreads>(s0 + L::k, rec + R::k);   // keys and queries, swizzled already
  fetch_tile<D>(s0 + L::u, p.w.u16 + c * (64 * D), 64);
  fetch_tile<D>(s0 + L::r, p.w.r16 + c * (64 * D), 64);
  sweep::cp_async_commit();
  fetch_tile<D>(s0 + L::s, p.w.s16 + c * (D * D), D);
  sweep::cp_async_commit();
  fetch_tile<D>(s0 + L::ds, p.w.ds16 + c * (D * D), D);
  sweep::cp_async_commit();

  const float *su = p.w.su + c * SLC, *sr = p.w.sr + c * SLC, *ss = p.w.ss + c * SLC, *sds = p.w.sds + c * SLC;
  const float uinv = factor_top(su, SLC), rinv = factor_top(sr, SLC), sinv = factor_top(ss, SLC), dsinv = factor_top(sds, SLC);
  const float ktop = factor_top(tokg + kTokK * 64, 64), qtop = factor_top(tokg + kTokQ * 64, 64);
  const float last = *reinterpret_cast<const float *>(rec + R::fac);
  if (tid < 64) {
    const float *gg = reinterpret_cast<const float *>(rec + R::g);
    G[tid] = gg[tid];
    Gl[tid] = gg[64 + tid];
    beta[tid] = tokg[kTokBeta * 64 + tid];
    kf[tid] = tokg[kTokK * 64 + tid];
    qf[tid] = tokg[kTokQ * 64 + tid];
  }
  {   // dO, each row to float16 with its own power of two; 8 rows a warp
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const int sub = lane % LPR;
    const T *dy = static_cast<const T *>(p.dy) + row * ldc + h * D + sub * 8;
#pragma unroll
    for (int i = 0; i < 8 / RPI + (RPI > 8); ++i) {
      const int rr = 8 * warp + i * RPI + lane / LPR;
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (rr < len) raw = *reinterpret_cast<const uint4 *>(dy + rr * ldc);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(&raw);
      float2 x[4];
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = unpack_io<T>(w[j]);
        top = fmaxf(top, fmaxf(fabsf(x[j].x), fabsf(x[j].y)));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const Pow2 ps = pow2_scale(top);
      uint4 ov;
      uint32_t *ow = reinterpret_cast<uint32_t *>(&ov);
#pragma unroll
      for (int j = 0; j < 4; ++j) ow[j] = pack2(mul2(x[j], splat(ps.s)));
      *reinterpret_cast<uint4 *>(smem + L::o + tile_off<D * 2>(rr, sub)) = ov;
      if (sub == 0) oinv[rr] = ps.inv;
    }
  }
  sweep::cp_async_wait<2>();
  __syncthreads();
  {   // one power of two per tile
    constexpr int U = D / 8;
    for (int i = tid; i < 64 * U; i += kThreads) {
      const int rr = i / U, uu = i % U;
      const uint32_t o = tile_off<D * 2>(rr, uu);
      scale_unit(smem + L::k + o, kf[rr] / ktop);
      scale_unit(smem + L::q + o, qf[rr] / qtop);
      scale_unit(smem + L::u + o, su[uu >> 1] / uinv);
      scale_unit(smem + L::r + o, sr[uu >> 1] / rinv);
    }
  }
  __syncthreads();

  const int m = warp & 3, half = warp >> 2;
  const LaneOff<D * 2> ofd(lane, s0);
  const LaneOff<128> of64(lane, s0);
  const int i0 = 16 * m + g;   // this thread's token rows: i0, i0 + 8
  {   // dP and N: columns 32 half .. 32 half + 31
    float P[4][4], N[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) P[i][e] = N[i][e] = 0.0f;
    if (2 * half <= m) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t ao[4], ar[4];
        ldsm4(ao, ofd.at(0, ks) + L::o + 16 * m * D * 2);
        ldsm4(ar, ofd.at(0, ks) + L::r + 16 * m * D * 2);
#pragma unroll
        for (int np = 0; np < 2; ++np) {
          if (2 * half + np > m) continue;
          uint32_t bu[4];
          ldsm4(bu, ofd.at(np, ks) + L::u + 32 * half * D * 2);
          mma_f16(P[2 * np], ao, bu[0], bu[2]);
          mma_f16(P[2 * np + 1], ao, bu[1], bu[3]);
          mma_f16(N[2 * np], ar, bu[0], bu[2]);
          mma_f16(N[2 * np + 1], ar, bu[1], bu[3]);
        }
      }
    }
    // in the factors under which both enter dK: dP qtop, N ktop
    float top = 0.0f;
    float fp[2], fn[2], gi[2], gli[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      fp[e] = p.s.scale * oinv[i0 + 8 * e] * uinv * qtop;
      fn[e] = -beta[i0 + 8 * e] * rinv * uinv * ktop;
      gi[e] = G[i0 + 8 * e];
      gli[e] = Gl[i0 + 8 * e];
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + (e >> 1) * 8, j = 32 * half + 8 * nt + 2 * t4 + (e & 1);
        float d = 0.0f;
        if (j <= i) d = expf((gi[e >> 1] - G[j]) + (gli[e >> 1] - Gl[j]));
        P[nt][e] = j <= i ? P[nt][e] * (d * fp[e >> 1]) : 0.0f;
        N[nt][e] = j < i ? N[nt][e] * (d * fn[e >> 1]) : 0.0f;
        top = fmaxf(top, fmaxf(fabsf(P[nt][e]), fabsf(N[nt][e])));
      }
    top = warp_max(top);
    if (lane == 0) red[warp] = top;
    __syncthreads();
    top = red[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, red[i]);
    const Pow2 pp = pow2_scale(top);
    if (tid == 0) red[8] = pp.inv;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint32_t o = tile_off<128>(i0 + (e >> 1) * 8, 4 * half + nt) + 4 * t4;
        *reinterpret_cast<uint32_t *>(smem + L::dp + o) = pack_h2(P[nt][e] * pp.s, P[nt][e + 1] * pp.s);
        *reinterpret_cast<uint32_t *>(smem + L::n + o) = pack_h2(N[nt][e] * pp.s, N[nt][e + 1] * pp.s);
      }
  }
  // v.du and du.u of each token, four threads a row
  {
    const int rr = tid >> 2, part = tid & 3;
    const T *v = static_cast<const T *>(p.v) + (row + rr) * p.s.ld_v + h * D;
    float a = 0.0f, bb = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int uu = part + 4 * i;
      const uint32_t o = tile_off<D * 2>(rr, uu);
      const uint4 du = *reinterpret_cast<const uint4 *>(smem + L::r + o), uv = *reinterpret_cast<const uint4 *>(smem + L::u + o);
      uint4 vv = make_uint4(0, 0, 0, 0);
      if (rr < len) vv = *reinterpret_cast<const uint4 *>(v + uu * 8);
      const uint32_t *x = reinterpret_cast<const uint32_t *>(&du), *y = reinterpret_cast<const uint32_t *>(&uv),
                     *z = reinterpret_cast<const uint32_t *>(&vv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 d2 = unpack_h2(x[j]), u2 = unpack_h2(y[j]), v2 = unpack_io<T>(z[j]);
        a = fmaf(d2.x, v2.x, fmaf(d2.y, v2.y, a));
        bb = fmaf(d2.x, u2.x, fmaf(d2.y, u2.y, bb));
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      bb += __shfl_xor_sync(0xffffffffu, bb, o);
    }
    if (part == 0) {
      vdu[rr] = a * rinv * beta[rr];
      udu[rr] = bb * rinv * uinv;
    }
  }
  sweep::cp_async_wait<0>();
  __syncthreads();
  float inner = 0.0f;   // <dS, S>, this thread's share
  {
    constexpr int U = D / 8;
    for (int i = tid; i < D * U; i += kThreads) {
      const int rr = i / U, uu = i % U;
      const uint32_t o = tile_off<D * 2>(rr, uu);
      scale_unit(smem + L::s + o, ss[rr >> 4] / sinv);
      scale_unit(smem + L::ds + o, sds[rr >> 4] / dsinv);
      const uint4 x = *reinterpret_cast<const uint4 *>(smem + L::s + o), y = *reinterpret_cast<const uint4 *>(smem + L::ds + o);
      const uint32_t *xw = reinterpret_cast<const uint32_t *>(&x), *yw = reinterpret_cast<const uint32_t *>(&y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = unpack_h2(xw[j]), bb = unpack_h2(yw[j]);
        inner = fmaf(a.x, bb.x, fmaf(a.y, bb.y, inner));
      }
    }
  }
  inner = head_sum<32>(inner);
  if (lane == 0) red[16 + warp] = inner;
  __syncthreads();

  float Qa[NH][4], Ka[NH][4], X[NH][4];
  const uint32_t cofs = D >= 128 ? 128 * half : 0;             // first column of this half, in swizzled units of 64 columns
  const int cj = D >= 128 ? 0 : half * (D / 32);               // or as a 16-column block index
  auto zero = [&] {
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) X[i][e] = 0.0f;
  };
  // X = A B^T with A the token rows of a tile and B stored [value channel][key channel]
  auto rows_by_state = [&](int a_tile, int s_tile) {
    zero();
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      ldsm4(a, ofd.at(0, ks) + a_tile + 16 * m * D * 2);
#pragma unroll
      for (int np = 0; np < NH / 2; ++np) {
        uint32_t bs[4];
        if constexpr (D >= 128) ldsm4t(bs, ofd.at(ks, np) + s_tile + cofs);
        else ldsm4t(bs, (cj == 0 ? ofd.at(ks, np) : ofd.at(ks, np + D / 32)) + s_tile);
        mma_f16(X[2 * np], a, bs[0], bs[1]);
        mma_f16(X[2 * np + 1], a, bs[2], bs[3]);
      }
    }
  };
  // X += A B with A a 64 x 64 tile's rows (or its transpose's) and B the token rows of a tile
  auto mat_by_rows = [&](int a_tile, bool transposed, int b_tile) {
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      if (transposed ? kb < m : kb > m) continue;
      uint32_t a[4];
      if (!transposed) {
        ldsm4(a, of64.at(0, kb) + a_tile + 16 * m * 128);
      } else {
        uint32_t r[4];
        ldsm4t(r, s0 + a_tile + tile_off<128>(16 * kb + (lane & 15), 2 * m + (lane >> 4)));
        a[0] = r[0]; a[1] = r[2]; a[2] = r[1]; a[3] = r[3];
      }
#pragma unroll
      for (int np = 0; np < NH / 2; ++np) {
        uint32_t bs[4];
        if constexpr (D >= 128) ldsm4t(bs, ofd.at(kb, np) + b_tile + cofs);
        else ldsm4t(bs, (cj == 0 ? ofd.at(kb, np) : ofd.at(kb, np + D / 32)) + b_tile);
        mma_f16(X[2 * np], a, bs[0], bs[1]);
        mma_f16(X[2 * np + 1], a, bs[2], bs[3]);
      }
    }
  };
  const float e0 = expf(G[i0] + Gl[i0]), e1 = expf(G[i0 + 8] + Gl[i0 + 8]);
  const float l0 = expf((G[63] - G[i0]) + (Gl[63] - Gl[i0])), l1 = expf((G[63] - G[i0 + 8]) + (Gl[63] - Gl[i0 + 8]));
  // scale e^G dO S^T
  rows_by_state(L::o, L::s);
  {
    const float f0 = p.s.scale * e0 * oinv[i0] * sinv, f1 = p.s.scale * e1 * oinv[i0 + 8] * sinv;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      Qa[i][0] = X[i][0] * f0; Qa[i][1] = X[i][1] * f0; Qa[i][2] = X[i][2] * f1; Qa[i][3] = X[i][3] * f1;
    }
  }
  // -beta e^G du S^T
  rows_by_state(L::r, L::s);
  {
    const float f0 = -beta[i0] * e0 * rinv * sinv, f1 = -beta[i0 + 8] * e1 * rinv * sinv;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      Ka[i][0] = X[i][0] * f0; Ka[i][1] = X[i][1] * f0; Ka[i][2] = X[i][2] * f1; Ka[i][3] = X[i][3] * f1;
    }
  }
  // e^{G_last - G} U dS^T, and its product with the key
  rows_by_state(L::u, L::ds);
  {
    const float f0 = l0 * uinv * dsinv, f1 = l1 * uinv * dsinv;
    float w0 = 0.0f, w1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const int unit = half * NH + i;
      const float2 k0 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::k + tile_off<D * 2>(i0, unit) + 4 * t4));
      const float2 k1 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::k + tile_off<D * 2>(i0 + 8, unit) + 4 * t4));
      w0 = fmaf(X[i][0], k0.x, fmaf(X[i][1], k0.y, w0));
      w1 = fmaf(X[i][2], k1.x, fmaf(X[i][3], k1.y, w1));
      Ka[i][0] = fmaf(X[i][0], f0, Ka[i][0]);
      Ka[i][1] = fmaf(X[i][1], f0, Ka[i][1]);
      Ka[i][2] = fmaf(X[i][2], f1, Ka[i][2]);
      Ka[i][3] = fmaf(X[i][3], f1, Ka[i][3]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      w0 += __shfl_xor_sync(0xffffffffu, w0, o);
      w1 += __shfl_xor_sync(0xffffffffu, w1, o);
    }
    if (t4 == 0) {
      wk[half * 64 + i0] = w0 * f0 * ktop;
      wk[half * 64 + i0 + 8] = w1 * f1 * ktop;
    }
  }
  const float pinv = red[8];
  T *dq = static_cast<T *>(p.dq) + row * ldc + h * D + half * (D / 2) + 2 * t4;
  T *dk = static_cast<T *>(p.dk) + row * ldc + h * D + half * (D / 2) + 2 * t4;
  // dP K
  zero();
  mat_by_rows(L::dp, false, L::k);
  {
    const float f = pinv * (ktop / qtop);
    float w0 = 0.0f, w1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) Qa[i][e] = fmaf(X[i][e], f, Qa[i][e]);
      const int unit = half * NH + i;
      const float2 q0 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::q + tile_off<D * 2>(i0, unit) + 4 * t4));
      const float2 q1 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::q + tile_off<D * 2>(i0 + 8, unit) + 4 * t4));
      w0 = fmaf(Qa[i][0], q0.x, fmaf(Qa[i][1], q0.y, w0));
      w1 = fmaf(Qa[i][2], q1.x, fmaf(Qa[i][3], q1.y, w1));
      if (i0 < len) *reinterpret_cast<uint32_t *>(dq + i0 * ldc + 8 * i) = pack_io<T>(Qa[i][0], Qa[i][1]);
      if (i0 + 8 < len) *reinterpret_cast<uint32_t *>(dq + (i0 + 8) * ldc + 8 * i) = pack_io<T>(Qa[i][2], Qa[i][3]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      w0 += __shfl_xor_sync(0xffffffffu, w0, o);
      w1 += __shfl_xor_sync(0xffffffffu, w1, o);
    }
    if (t4 == 0) {
      qdq[half * 64 + i0] = w0 * qtop;
      qdq[half * 64 + i0 + 8] = w1 * qtop;
    }
  }
  // dP^T Q + N K + N^T K
  zero();
  mat_by_rows(L::dp, true, L::q);
  mat_by_rows(L::n, false, L::k);
  mat_by_rows(L::n, true, L::k);
#pragma unroll
  for (int i = 0; i < NH; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) Ka[i][e] = fmaf(X[i][e], pinv, Ka[i][e]);
    if (i0 < len) *reinterpret_cast<uint32_t *>(dk + i0 * ldc + 8 * i) = pack_io<T>(Ka[i][0], Ka[i][1]);
    if (i0 + 8 < len) *reinterpret_cast<uint32_t *>(dk + (i0 + 8) * ldc + 8 * i) = pack_io<T>(Ka[i][2], Ka[i][3]);
  }
  __syncthreads();
  if (warp == 0) {   // the gates' gradients: two tokens a lane, later tokens first
    float in = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) in += red[16 + i];
    float w = wk[2 * lane] + wk[2 * lane + 1] + wk[64 + 2 * lane] + wk[64 + 2 * lane + 1];
    w = head_sum<32>(w);
    const float cc = fmaf(last * sinv * dsinv, in, w);
    const float x1 = qdq[2 * lane + 1] + qdq[64 + 2 * lane + 1] - vdu[2 * lane + 1];
    const float x0 = qdq[2 * lane] + qdq[64 + 2 * lane] - vdu[2 * lane];
    const float own = x0 + x1;
    float sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, sum, o);
      if (lane + o < 32) sum += y;
    }
    const float after = cc + (sum - own);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      if (i < len) {
        const float a = fmaxf(sweep::widen(static_cast<const T *>(p.a)[(row + i) * p.s.ld_g + h]), -80.0f);
        const float bb = fmaxf(sweep::widen(static_cast<const T *>(p.b)[(row + i) * p.s.ld_g + h]), -80.0f);
        const float dl = after + x1 + (e == 0 ? x0 : 0.0f);
        static_cast<T *>(p.da)[(row + i) * p.s.H + h] = sweep::narrow<T>(dl / (1.0f + expf(a)));
        static_cast<T *>(p.db)[(row + i) * p.s.H + h] = sweep::narrow<T>(udu[i] / (1.0f + expf(bb)));
      }
    }
  }
}

template <typename T, int D>
int run(const ChunkArgs &a, cudaStream_t st) {
  auto kern = delta_grad_kernel<T, D>;
  const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GradSmem<D>::total));
  if (rc) return rc;
  kern<<<static_cast<unsigned>(a.s.B) * a.s.H * a.w.nc, kThreads, GradSmem<D>::total, st>>>(a);
  return runtime_status(cudaGetLastError());
}

template <typename T>
int by_d(const ChunkArgs &a, cudaStream_t st) {
  switch (a.s.D) {
    case 32: return run<T, 32>(a, st);
    case 64: return run<T, 64>(a, st);
    case 128: return run<T, 128>(a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace

int launch_chunk_grad(int dtype, const ChunkArgs &a, cudaStream_t st) {
  return dtype == ESA_F16 ? by_d<__half>(a, st) : by_d<__nv_bfloat16>(a, st);
}

}  // namespace esa
