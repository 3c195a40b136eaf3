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
//   da_i = (1 - alpha_i) (sum_{j < i <= s} W_sj + sum_{s >= i} A_s + sum_{j < i} B_j + e^{G_last} <dS, S>),
//   W_sj = dP_sj q_s.k_j + N_sj k_s.k_j,   B_j = k_j.(e^{G_last - G_j} u_j dS^T),
//   A_s = q_s.(scale e^G dO S^T)_s - k_s.(beta e^G du S^T)_s.
// da's sum is over every decay factor that token i has a part in: between two
// tokens, from the state to a later token, from an earlier token or the state
// to the chunk's end.  Each has the factor alpha_i, so that a gate that forgets
// keeps the digits of its gradient.  (The same sum as the differences of
// q.dq - beta v.du of later tokens cancels to alpha of its terms: with float16
// operands da was off by 0.3% at logits near 0, 8% at -4, 50% at -6.)  The
// rectangles of W are summed in blocks of 16 by shuffles: a diagonal block its
// 16 rectangles, another its rows from each token on and its columns up to
// each.  <dS, S> is the diagonal of dS S^T, 16 rows at a time, on the tensor
// cores too.
//
// These are outputs in 16 bits: S, dS, U, du, dP and N are operands in one
// float16 term each (2^-12 of a value on average) where the output is bfloat16
// (2^-9).  For a float16 output (2^-12) U, du, dP and N are in two, so that of
// each product's operands one is rounded, S or dS, at most: with one term each
// dq, dk and db were 3.7e-4 off in the 2-norm, where the output's rounding alone
// is 2.1e-4; now dq and dk are at 2.4e-4 and db at 2.1e-4, for 25% more time of
// this kernel.  (S and dS in two as well would be 64 KB more a chunk at D = 128.)
//
// A persistent block takes chunk after chunk.  Warp (m, cw) has 16 tokens and
// a share of the channels.  U, du and dO of the next chunk are copied while
// this one is computed (two buffers), its S and dS as soon as this one's have
// been used, then its K and Q; so copies of 190 KB a chunk (D = 128) run under
// 3,300 mma.  With two terms U, du and dO have one buffer at D >= 64 and are
// copied with S and dS.
#include <type_traits>

#include "esa_delta_chunk.h"
#include "esa_delta_sweep.cuh"
#include "esa_mma.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

// TWO: U, du, dP and N in two terms.  Then a chunk's rows have one buffer where
// two of them do not fit (D = 128) or keep a second block off the SM (D = 64).
template <int D, bool TWO>
struct GradShape {
  static constexpr int threads = D == 128 ? 512 : 256;
  static constexpr int CW = threads / 128;          // shares of the channels
  static constexpr int row = 64 * D * 2, mat = D * D * 2;
  static constexpr int hdr = ChunkRecord<D>::k + 512 + 128;   // per-token factors, running sums, slice scales
  static constexpr int stages = TWO && D >= 64 ? 1 : 2;
  static constexpr int k = 0, q = row, s = 2 * row, ds = s + mat, dp = ds + mat, n = dp + 8192, lo = 16384,   // lo: from a tile to its second term
                       h = n + 8192 + (TWO ? lo : 0), buf = h + 2 * hdr,
                       u = 0, r = row, o = 2 * row, ul = 3 * row, rl = 4 * row, stage = (TWO ? 5 : 3) * row, vec = buf + stages * stage,
                       total = vec + (64 + 64 + 2 * CW * 64 + 9 * 64 + 64) * 4;
  static_assert(hdr % 128 == 0 && total <= 227 * 1024, "headers between tiles; a block's shared memory");
};

__device__ __forceinline__ void scale_frag(uint32_t (&a)[4], float f) {
  const __half2 s = __float2half2_rn(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&a[i]), s);
    a[i] = *reinterpret_cast<const uint32_t *>(&x);
  }
}

// x a b of two units, whose product may leave float32's range where that with x does not.
__device__ __forceinline__ float mul3(float x, float a, float b) {
  const float ab = a * b;
  return ab >= 1.17549435e-38f && ab <= 8.507059173023462e37f ? x * ab : x * a * b;   // 2^-126, 2^126
}

// Two neighbouring accumulator tiles times f, rounded, as 8-byte stores: lanes
// exchange as in store_block.  `o` is the thread's first element of a pair.
template <typename T>
__device__ __forceinline__ void store_pair(T *o, long long ld, int col, const float (&c0)[4], const float (&c1)[4], float f,
                                           bool on0, bool on1, int lane) {
  const bool odd = lane & 1;
  const uint32_t a0 = pack_io<T>(c0[0] * f, c0[1] * f), a1 = pack_io<T>(c0[2] * f, c0[3] * f);
  const uint32_t b0 = pack_io<T>(c1[0] * f, c1[1] * f), b1 = pack_io<T>(c1[2] * f, c1[3] * f);
  const uint32_t x0 = __shfl_xor_sync(0xffffffffu, odd ? a0 : b0, 1), x1 = __shfl_xor_sync(0xffffffffu, odd ? a1 : b1, 1);
  if (on0) *reinterpret_cast<uint2 *>(o + col) = odd ? make_uint2(x0, b0) : make_uint2(a0, x0);
  if (on1) *reinterpret_cast<uint2 *>(o + 8 * ld + col) = odd ? make_uint2(x1, b1) : make_uint2(a1, x1);
}

// Sum over a row's four threads; over the eight rows of a half of a block, of
// this row and those behind it.
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float rows_from(float x, int g) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float y = __shfl_down_sync(0xffffffffu, x, 4 * o);
    if (g + o < 8) x += y;
  }
  return x;
}

// A 16 x 16 block of W (rows s, columns j), as an accumulator pair.  On the
// diagonal: diag[r] = sum of s >= r, j < r.  Else rows[r] = sum of s >= r over
// all j, cols[r] = sum of j < r over all s.
__device__ __forceinline__ void diagonal_sums(const float (&w)[2][4], float *diag, int lane) {
  const int g = lane >> 2, t4 = lane & 3;
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 8 * nt + 2 * t4 + e;
      const float b = rows_from(w[nt][e + 2], g), a = rows_from(w[nt][e], g) + __shfl_sync(0xffffffffu, b, t4);
      if (col < g) lo += a;
      if (col < g + 8) hi += b;
    }
  lo = quad_sum(lo);
  hi = quad_sum(hi);
  if (t4 == 0) {
    diag[g] = lo;
    diag[g + 8] = hi;
  }
}
__device__ __forceinline__ void edge_sums(const float (&w)[2][4], float *rows, float *cols, int lane) {
  const int g = lane >> 2, t4 = lane & 3;
  const float hi = rows_from(quad_sum((w[0][2] + w[0][3]) + (w[1][2] + w[1][3])), g);
  const float lo = rows_from(quad_sum((w[0][0] + w[0][1]) + (w[1][0] + w[1][1])), g) + __shfl_sync(0xffffffffu, hi, t4);
  if (t4 == 0) {
    rows[g] = lo;
    rows[g + 8] = hi;
  }
  float before = 0.0f;   // columns of the first half, then of both
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    float c0 = w[nt][0] + w[nt][2], c1 = w[nt][1] + w[nt][3];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      c0 += __shfl_xor_sync(0xffffffffu, c0, o);
      c1 += __shfl_xor_sync(0xffffffffu, c1, o);
    }
    float to = c0 + c1;   // up to this pair
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, to, o, 4);
      if (t4 >= o) to += y;
    }
    float from = __shfl_up_sync(0xffffffffu, to, 1, 4);
    from = before + (t4 > 0 ? from : 0.0f);
    if (g == 0) {
      cols[8 * nt + 2 * t4] = from;
      cols[8 * nt + 2 * t4 + 1] = from + c0;
    }
    before += __shfl_sync(0xffffffffu, to, 3, 4);
  }
}

template <typename T>
constexpr bool two_terms() { return std::is_same<T, __half>::value; }

template <typename T, int D>
__global__ void __launch_bounds__(GradShape<D, two_terms<T>()>::threads, D == 128 ? 1 : 2) delta_grad_kernel(ChunkArgs p, int chunks) {
  constexpr bool kTwo = two_terms<T>();
  using L = GradShape<D, kTwo>;
  using R = ChunkRecord<D>;
  constexpr int kThreads = L::threads, CW = L::CW;
  constexpr int NH = D / (8 * CW);   // accumulator tiles of a share of the channels
  constexpr int NPA = 4 / CW;        // 16-column blocks of dP and N a warp forms
  constexpr int KS = D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  float *vec = reinterpret_cast<float *>(smem + L::vec);
  // per token: scale of dO, u.du, A, B; rows[4][64], cols[4][64], diag[64] of W's blocks; maxima and <dS, S>
  float *oinv = vec, *udu = vec + 64, *as = vec + 128, *bs = as + CW * 64, *wrows = bs + CW * 64, *wcols = wrows + 256,
        *wdiag = wcols + 256, *red = wdiag + 64;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int m = warp & 3, cw = warp >> 2;
  const long long ldc = static_cast<long long>(p.s.H) * D;
  const uint32_t s0 = smem_u32(smem);

  auto place = [&](int c, int &b, int &h, int &t0) {
    const int head = c / p.w.nc;
    b = head / p.s.H;
    h = head - b * p.s.H;
    t0 = (c - head * p.w.nc) * kChunk;
  };
  int nb = 0, nh = 0, nt0 = 0;              // place of the chunk whose rows were fetched last
  auto fetch_rows = [&](int c, int buf) {   // U, du, dO and the header
    if (c < chunks) {
      const uint32_t st = s0 + L::buf + (L::stages == 2 ? buf : 0) * L::stage, hd = s0 + L::h + buf * L::hdr;
      if constexpr (kTwo) {
        copy_rows<D * 2, 64, kThreads>(st + L::ul, p.w.u16l + static_cast<long long>(c) * (64 * D));
        copy_rows<D * 2, 64, kThreads>(st + L::rl, p.w.r16l + static_cast<long long>(c) * (64 * D));
      }
      copy_rows<D * 2, 64, kThreads>(st + L::u, p.w.u16 + static_cast<long long>(c) * (64 * D));
      copy_rows<D * 2, 64, kThreads>(st + L::r, p.w.r16 + static_cast<long long>(c) * (64 * D));
      place(c, nb, nh, nt0);
      const int b = nb, h = nh, t0 = nt0;
      constexpr int U = D / 8, STEP = kThreads / U;
      const int r = tid / U, u = tid % U, len = min(kChunk, p.s.T - t0);
      const T *dy = static_cast<const T *>(p.dy) + (static_cast<long long>(b) * p.s.T + t0) * ldc + h * D + u * 8;
#pragma unroll
      for (int i = 0; i < (64 + STEP - 1) / STEP; ++i) {
        const int rr = r + i * STEP;
        if (STEP <= 64 || rr < 64)
          cp_async16_zfill(st + L::o + tile_off<D * 2>(rr, u), rr < len ? dy + rr * ldc : static_cast<const T *>(p.dy), rr < len);
      }
      const unsigned char *rec = p.w.rec + static_cast<long long>(c) * R::bytes;
      if (tid < R::k / 16) cp_async16_s(hd + tid * 16, rec + tid * 16);
      else if (tid >= 128 && tid < 160) cp_async16_s(hd + R::k + (tid - 128) * 16, rec + R::g + (tid - 128) * 16);
      else if (tid >= 160 && tid < 168)
        cp_async16_s(hd + R::k + 512 + (tid - 160) * 16, p.w.slice + static_cast<long long>(c) * 32 + (tid - 160) * 4);
    }
    sweep::cp_async_commit();
  };
  auto fetch_states = [&](int c) {
    if (c < chunks) {
      copy_rows<D * 2, D, kThreads>(s0 + L::s, p.w.s16 + static_cast<long long>(c) * (D * D));
      copy_rows<D * 2, D, kThreads>(s0 + L::ds, p.w.ds16 + static_cast<long long>(c) * (D * D));
    }
    sweep::cp_async_commit();
  };
  auto fetch_keys = [&](int c) {
    if (c < chunks) copy_linear<2 * L::row, kThreads>(s0 + L::k, p.w.rec + static_cast<long long>(c) * R::bytes + R::k);
    sweep::cp_async_commit();
  };

  const LaneOff<D * 2> ofd(lane, s0);
  const LaneOffB<D * 2> ofb(lane, s0);
  const LaneOff<128> of64(lane, s0);
  const int i0 = 16 * m + g;   // this thread's token rows: i0, i0 + 8
  int it = 0;
  fetch_rows(blockIdx.x, 0);
  fetch_states(blockIdx.x);
  fetch_keys(blockIdx.x);
#pragma unroll 1
  for (int c = blockIdx.x; c < chunks; c += gridDim.x, ++it) {
    const int buf = it & 1, next = c + gridDim.x;
    const int b = nb, h = nh, t0 = nt0;
    const int len = min(kChunk, p.s.T - t0);
    const long long row = static_cast<long long>(b) * p.s.T + t0;
    const uint32_t bo = L::buf + (L::stages == 2 ? buf : 0) * L::stage;
    unsigned char *sb = smem + bo;
    const unsigned char *hd = smem + L::h + buf * L::hdr;
    const float *tok = reinterpret_cast<const float *>(hd);
    const float *G = reinterpret_cast<const float *>(hd + R::k), *Gl = G + 64;
    sweep::cp_async_wait<2>();   // rows of this chunk
    __syncthreads();
    if constexpr (L::stages == 2) fetch_rows(next, buf ^ 1);
    T la[2], lb[2];              // warp 0: the gates' logits, for the end
    la[0] = la[1] = lb[0] = lb[1] = sweep::narrow<T>(0.0f);
    if (warp == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * lane + e < len) {
          la[e] = static_cast<const T *>(p.a)[(row + 2 * lane + e) * p.s.ld_g + h];
          lb[e] = static_cast<const T *>(p.b)[(row + 2 * lane + e) * p.s.ld_g + h];
        }
    }
    // dO, each row to float16 with its own power of two
    {
      constexpr int U = D / 8;
#pragma unroll
      for (int i = 0; i < 64 * U / kThreads; ++i) {
        const int e = tid + i * kThreads, rr = e / U;
        unsigned char *at = sb + L::o + tile_off<D * 2>(rr, e % U);
        uint4 raw = *reinterpret_cast<const uint4 *>(at);
        uint32_t *w = reinterpret_cast<uint32_t *>(&raw);
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack_io<T>(w[j]);
          top = fmaxf(fmaxf(top, fabsf(x.x)), fabsf(x.y));
        }
#pragma unroll
        for (int o = U / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const Pow2 ps = pow2_scale(top);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack2(mul2(unpack_io<T>(w[j]), splat(ps.s)));
        *reinterpret_cast<uint4 *>(at) = raw;
        if (e % U == 0) oinv[rr] = top > 0.0f ? ps.inv : 0.0f;
      }
    }
    // slice scales: the largest of each kind, and what each slice has of it (1 almost always)
    float part, uinv, rinv, sinv, dsinv;   // 0 for zeros
    bool flat;
    {
      float v = (lane & 7) < KS ? reinterpret_cast<const float *>(hd + R::k + 512)[lane] : 0.0f;
      float t = v;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
      if (__any_sync(0xffffffffu, v != v)) t = v = __int_as_float(0x7fc00000);   // a channel of the chunk is not finite
      part = v > 0.0f && v != t ? v / t : 1.0f;
      flat = __all_sync(0xffffffffu, part == 1.0f);
      uinv = __shfl_sync(0xffffffffu, t, kSliceU);
      rinv = __shfl_sync(0xffffffffu, t, kSliceR);
      sinv = __shfl_sync(0xffffffffu, t, kSliceS);
      dsinv = __shfl_sync(0xffffffffu, t, kSliceDs);
    }
    const float *fac = reinterpret_cast<const float *>(hd + R::fac);
    const float last = fac[kFacLast], kinv = fac[kFacK], qinv = fac[kFacQ];
    __syncthreads();

    const float be0 = tok[kTokBeta * 64 + i0], be1 = tok[kTokBeta * 64 + i0 + 8];
    float uq, uk, fpk, fpq, fnk;   // units of dQ's and dK's sums; of dP in dQ, dP^T in dK, N in dK
    {   // dP and N: 16-column blocks NPA cw ..
      float P[2 * NPA][4], N[2 * NPA][4];
#pragma unroll
      for (int i = 0; i < 2 * NPA; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) P[i][e] = N[i][e] = 0.0f;
      if (NPA * cw <= m) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t ao[4], ar[4], al[4];
          ldsm4(ao, ofd.at(0, ks) + bo + L::o + 16 * m * D * 2);
          ldsm4(ar, ofd.at(0, ks) + bo + L::r + 16 * m * D * 2);
          if constexpr (kTwo) ldsm4(al, ofd.at(0, ks) + bo + L::rl + 16 * m * D * 2);
          if (!flat) {
            const float fu = __shfl_sync(0xffffffffu, part, kSliceU + ks), fr = fu * __shfl_sync(0xffffffffu, part, kSliceR + ks);
            scale_frag(ao, fu);
            scale_frag(ar, fr);
            if constexpr (kTwo) scale_frag(al, fr);
          }
#pragma unroll
          for (int np = 0; np < NPA; ++np) {
            if (NPA * cw + np > m) continue;
            uint32_t bu[4];
            ldsm4(bu, ofb.at(np, ks) + bo + L::u + 16 * NPA * cw * D * 2);
            mma_f16(P[2 * np], ao, bu[0], bu[1]);
            mma_f16(P[2 * np + 1], ao, bu[2], bu[3]);
            mma_f16(N[2 * np], ar, bu[0], bu[1]);
            mma_f16(N[2 * np + 1], ar, bu[2], bu[3]);
            if constexpr (kTwo) {
              mma_f16(N[2 * np], al, bu[0], bu[1]);
              mma_f16(N[2 * np + 1], al, bu[2], bu[3]);
              ldsm4(bu, ofb.at(np, ks) + bo + L::ul + 16 * NPA * cw * D * 2);
              mma_f16(P[2 * np], ao, bu[0], bu[1]);
              mma_f16(P[2 * np + 1], ao, bu[2], bu[3]);
              mma_f16(N[2 * np], ar, bu[0], bu[1]);
              mma_f16(N[2 * np + 1], ar, bu[2], bu[3]);
            }
          }
        }
      }
      float topp = 0.0f, topn = 0.0f;
      const float ru = rinv * uinv;
      float fp[2], fn[2], gi[2], gli[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fp[e] = mul3(p.s.scale, oinv[i0 + 8 * e], uinv);
        fn[e] = -mul3(e ? be1 : be0, rinv, uinv);
        gi[e] = G[i0 + 8 * e];
        gli[e] = Gl[i0 + 8 * e];
      }
#pragma unroll
      for (int nt = 0; nt < 2 * NPA; ++nt) {
        const int j0 = 16 * NPA * cw + 8 * nt + 2 * t4;
        const float2 gj = *reinterpret_cast<const float2 *>(G + j0), glj = *reinterpret_cast<const float2 *>(Gl + j0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + (e >> 1) * 8, j = j0 + (e & 1);
          // 16-bit results: the exponential's error of a few 2^-23 times the exponent does not show
          const float d = __expf((gi[e >> 1] - (e & 1 ? gj.y : gj.x)) + (gli[e >> 1] - (e & 1 ? glj.y : glj.x)));
          if (i == j) udu[i] = N[nt][e] * ru;
          P[nt][e] = j <= i ? P[nt][e] * (d * fp[e >> 1]) : 0.0f;
          N[nt][e] = j < i ? N[nt][e] * (d * fn[e >> 1]) : 0.0f;
        }
        topp = max_tile(P[nt], topp);
        topn = max_tile(N[nt], topn);
      }
      topp = warp_max(topp);
      topn = warp_max(topn);
      if (lane == 0) {
        red[warp] = topp;
        red[32 + warp] = topn;
      }
      sweep::cp_async_wait<L::stages - 1>();   // S, dS, K and Q
      __syncthreads();
#pragma unroll
      for (int np = 0; np < NPA; ++np) {   // W, from Q K^T and K K^T
        const int blk = NPA * cw + np;
        if (blk > m) continue;
        float w[2][4], z[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) w[i][e] = z[i][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t aq[4], ak[4], bk[4];
          ldsm4(aq, ofd.at(0, ks) + L::q + 16 * m * D * 2);
          ldsm4(ak, ofd.at(0, ks) + L::k + 16 * m * D * 2);
          ldsm4(bk, ofb.at(np, ks) + L::k + 16 * NPA * cw * D * 2);
          mma_f16(w[0], aq, bk[0], bk[1]);
          mma_f16(w[1], aq, bk[2], bk[3]);
          mma_f16(z[0], ak, bk[0], bk[1]);
          mma_f16(z[1], ak, bk[2], bk[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = w[i][e] * qinv * (kinv * P[2 * np + i][e]);
            w[i][e] = fmaf(z[i][e] * kinv, kinv * N[2 * np + i][e], p);
            if (blk == m && 8 * i + 2 * t4 + (e & 1) >= g + (e >> 1) * 8) w[i][e] = 0.0f;
          }
        if (blk == m) diagonal_sums(w, wdiag + 16 * m, lane);
        else edge_sums(w, wrows + 64 * blk + 16 * m, wcols + 64 * m + 16 * blk, lane);
      }
      topp = warp_max(red[lane & (kThreads / 32 - 1)]);
      topn = warp_max(red[32 + (lane & (kThreads / 32 - 1))]);
      const Pow2 pp = pow2_scale(topp), pn = pow2_scale(topn);
      // Units of the sums of dQ and dK: the largest of their addends' (0 for addends of zeros), dP K, N K and dP^T Q
      // here; those of the states' share, sums below 2^33 of the products of factors, need 2^-77 of theirs (see
      // kLeastShare).  Fragments of a smaller unit are brought to it as they are read.
      const float omax = warp_max(fmaxf(oinv[lane], oinv[32 + lane]));
      const float bmax = warp_max(fmaxf(tok[kTokBeta * 64 + lane], tok[kTokBeta * 64 + 32 + lane]));
      const float pk = topp > 0.0f ? pp.inv * kinv : 0.0f, pq = topp > 0.0f ? pp.inv * qinv : 0.0f, nk = topn > 0.0f ? pn.inv * kinv : 0.0f;
      uq = fmaxf(fmaxf(pk, kLeastUnit), mul3(fabsf(p.s.scale), omax, sinv) * (1024.0f * kLeastShare));
      uk = fmaxf(fmaxf(fmaxf(nk, pq), kLeastUnit), mul3(bmax, rinv, sinv) * (1024.0f * kLeastShare));
      fpk = pk / uq;
      fpq = pq / uk;
      fnk = nk / uk;
#pragma unroll
      for (int nt = 0; nt < 2 * NPA; ++nt)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const uint32_t o = tile_off<128>(i0 + (e >> 1) * 8, 2 * NPA * cw + nt) + 4 * t4;
          const float2 x = mul2(make_float2(P[nt][e], P[nt][e + 1]), splat(pp.s)), y = mul2(make_float2(N[nt][e], N[nt][e + 1]), splat(pn.s));
          if constexpr (kTwo) {
            split2(x, *reinterpret_cast<uint32_t *>(smem + L::dp + o), *reinterpret_cast<uint32_t *>(smem + L::dp + L::lo + o));
            split2(y, *reinterpret_cast<uint32_t *>(smem + L::n + o), *reinterpret_cast<uint32_t *>(smem + L::n + L::lo + o));
          } else {
            *reinterpret_cast<uint32_t *>(smem + L::dp + o) = pack2(x);
            *reinterpret_cast<uint32_t *>(smem + L::n + o) = pack2(y);
          }
        }
    }
    __syncthreads();

    float Q[NH][4], K[NH][4], X[NH][4];
#pragma unroll
    for (int i = 0; i < NH; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) Q[i][e] = K[i][e] = X[i][e] = 0.0f;
    // Block index of this warp's channels: NH / 2 blocks from b0 on.  The
    // offsets of LaneOff repeat every four blocks, so with a share of two
    // blocks the warp's parity of pairs picks which of them it uses.
    const bool odd = (NH / 2 == 2) && (cw & 1);
    const uint32_t far = D == 128 ? (cw >> 1) * 128u : 0u;
    auto cols = [&](int kb, int np) -> uint32_t {
      if constexpr (NH / 2 == 2) return (odd ? ofd.at(kb, 2 + np) : ofd.at(kb, np)) + far;
      else return cw ? ofd.at(kb, 1) : ofd.at(kb, 0);   // D = 32: one block a share
    };
    // dO S^T, du S^T and U dS^T; S and dS are stored [value channel][key channel]
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t ao[4], ar[4], au[4], rl[4], ul[4];
      ldsm4(ao, ofd.at(0, ks) + bo + L::o + 16 * m * D * 2);
      ldsm4(ar, ofd.at(0, ks) + bo + L::r + 16 * m * D * 2);
      ldsm4(au, ofd.at(0, ks) + bo + L::u + 16 * m * D * 2);
      if constexpr (kTwo) {
        ldsm4(rl, ofd.at(0, ks) + bo + L::rl + 16 * m * D * 2);
        ldsm4(ul, ofd.at(0, ks) + bo + L::ul + 16 * m * D * 2);
      }
      if (!flat) {
        const float fs = __shfl_sync(0xffffffffu, part, kSliceS + ks), fr = fs * __shfl_sync(0xffffffffu, part, kSliceR + ks);
        const float fu = __shfl_sync(0xffffffffu, part, kSliceU + ks) * __shfl_sync(0xffffffffu, part, kSliceDs + ks);
        scale_frag(ao, fs);
        scale_frag(ar, fr);
        scale_frag(au, fu);
        if constexpr (kTwo) {
          scale_frag(rl, fr);
          scale_frag(ul, fu);
        }
      }
#pragma unroll
      for (int np = 0; np < NH / 2; ++np) {
        uint32_t bs[4], bd[4];
        ldsm4t(bs, cols(ks, np) + L::s);
        ldsm4t(bd, cols(ks, np) + L::ds);
        mma_f16(Q[2 * np], ao, bs[0], bs[1]);
        mma_f16(Q[2 * np + 1], ao, bs[2], bs[3]);
        mma_f16(K[2 * np], ar, bs[0], bs[1]);
        mma_f16(K[2 * np + 1], ar, bs[2], bs[3]);
        mma_f16(X[2 * np], au, bd[0], bd[1]);
        mma_f16(X[2 * np + 1], au, bd[2], bd[3]);
        if constexpr (kTwo) {
          mma_f16(K[2 * np], rl, bs[0], bs[1]);
          mma_f16(K[2 * np + 1], rl, bs[2], bs[3]);
          mma_f16(X[2 * np], ul, bd[0], bd[1]);
          mma_f16(X[2 * np + 1], ul, bd[2], bd[3]);
        }
      }
    }
    if (warp < KS) {   // <dS, S> of 16 rows: the diagonal of dS S^T
      float d[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][e] = 0.0f;
#pragma unroll
      for (int kb = 0; kb < KS; ++kb) {
        uint32_t a[4], bs[4];
        ldsm4(a, ofd.at(0, kb) + L::ds + 16 * warp * D * 2);
        ldsm4(bs, ofb.at(0, kb) + L::s + 16 * warp * D * 2);
        mma_f16(d[0], a, bs[0], bs[1]);
        mma_f16(d[1], a, bs[2], bs[3]);
      }
      float x = 0.0f;
      if (2 * t4 == g) x = d[0][0] + d[1][2];
      if (2 * t4 + 1 == g) x = d[0][1] + d[1][3];
      x = head_sum<32>(x);
      if (!flat) x *= __shfl_sync(0xffffffffu, part, kSliceS + warp) * __shfl_sync(0xffffffffu, part, kSliceDs + warp);
      if (lane == 0) red[16 + warp] = x;
    }
    __syncthreads();             // S and dS have been used, and U, du and dO
    if constexpr (L::stages == 1) fetch_rows(next, buf ^ 1);
    fetch_states(next);
    {   // the sums so far, in the units of what joins them
      const float e0 = expf(G[i0] + Gl[i0]), e1 = expf(G[i0 + 8] + Gl[i0 + 8]);
      const float iq = 1.0f / uq, ik = 1.0f / uk;
      const float q0 = mul3(p.s.scale, oinv[i0], sinv) * iq * e0, q1 = mul3(p.s.scale, oinv[i0 + 8], sinv) * iq * e1;
      const float k0 = -mul3(be0, rinv, sinv) * ik * e0, k1 = -mul3(be1, rinv, sinv) * ik * e1;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        set_lo(Q[i], mul2(row_lo(Q[i]), splat(q0)));
        set_hi(Q[i], mul2(row_hi(Q[i]), splat(q1)));
        set_lo(K[i], mul2(row_lo(K[i]), splat(k0)));
        set_hi(K[i], mul2(row_hi(K[i]), splat(k1)));
      }
    }
    {   // A and B: dots of the states' share with the key and the query
      const float l0 = expf((G[63] - G[i0]) + (Gl[63] - Gl[i0])) * uinv * dsinv;
      const float l1 = expf((G[63] - G[i0 + 8]) + (Gl[63] - Gl[i0 + 8])) * uinv * dsinv;
      float2 z0 = make_float2(0, 0), z1 = z0, w0 = z0, w1 = z0, y0 = z0, y1 = z0;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const uint32_t o = tile_off<D * 2>(i0, cw * NH + i) + 4 * t4;
        const float2 k0 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::k + o));
        const float2 k1 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::k + o + 8 * D * 2));
        const float2 q0 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::q + o));
        const float2 q1 = unpack_h2(*reinterpret_cast<const uint32_t *>(smem + L::q + o + 8 * D * 2));
        z0 = fma2(row_lo(K[i]), k0, z0);
        z1 = fma2(row_hi(K[i]), k1, z1);
        w0 = fma2(row_lo(X[i]), k0, w0);
        w1 = fma2(row_hi(X[i]), k1, w1);
        y0 = fma2(row_lo(Q[i]), q0, y0);
        y1 = fma2(row_hi(Q[i]), q1, y1);
        set_lo(X[i], mul2(row_lo(X[i]), splat(l0)));
        set_hi(X[i], mul2(row_hi(X[i]), splat(l1)));
      }
      float r[6] = {z0.x + z0.y, z1.x + z1.y, w0.x + w0.y, w1.x + w1.y, y0.x + y0.y, y1.x + y1.y};
#pragma unroll
      for (int i = 0; i < 6; ++i) r[i] = quad_sum(r[i]);
      if (t4 == 0) {
        // unit by unit: a product of two may be below float32's range
        as[cw * 64 + i0] = fmaf(r[4] * uq, qinv, r[0] * uk * kinv);
        as[cw * 64 + i0 + 8] = fmaf(r[5] * uq, qinv, r[1] * uk * kinv);
        bs[cw * 64 + i0] = r[2] * l0 * kinv;
        bs[cw * 64 + i0 + 8] = r[3] * l1 * kinv;
      }
    }
    // Q += dP K, K += N K
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      if (kb > m) continue;
      uint32_t ap[4], an[4];
      ldsm4(ap, of64.at(0, kb) + L::dp + 16 * m * 128);
      ldsm4(an, of64.at(0, kb) + L::n + 16 * m * 128);
      if (fpk != 1.0f) scale_frag(ap, fpk);
      if (fnk != 1.0f) scale_frag(an, fnk);
      uint32_t pl[4], nl[4];
      if constexpr (kTwo) {
        ldsm4(pl, of64.at(0, kb) + L::dp + L::lo + 16 * m * 128);
        ldsm4(nl, of64.at(0, kb) + L::n + L::lo + 16 * m * 128);
        if (fpk != 1.0f) scale_frag(pl, fpk);
        if (fnk != 1.0f) scale_frag(nl, fnk);
      }
#pragma unroll
      for (int np = 0; np < NH / 2; ++np) {
        uint32_t bk[4];
        ldsm4t(bk, cols(kb, np) + L::k);
        mma_f16(Q[2 * np], ap, bk[0], bk[1]);
        mma_f16(Q[2 * np + 1], ap, bk[2], bk[3]);
        mma_f16(K[2 * np], an, bk[0], bk[1]);
        mma_f16(K[2 * np + 1], an, bk[2], bk[3]);
        if constexpr (kTwo) {
          mma_f16(Q[2 * np], pl, bk[0], bk[1]);
          mma_f16(Q[2 * np + 1], pl, bk[2], bk[3]);
          mma_f16(K[2 * np], nl, bk[0], bk[1]);
          mma_f16(K[2 * np + 1], nl, bk[2], bk[3]);
        }
      }
    }
    const int col0 = cw * NH * 8 + (lane & 1 ? 8 : 0) + 2 * (t4 & 2);   // this thread's first channel in a pair of tiles
    T *dq = static_cast<T *>(p.dq) + (row + i0) * ldc + h * D + col0;
    T *dk = static_cast<T *>(p.dk) + (row + i0) * ldc + h * D + col0;
    const bool on0 = i0 < len, on1 = i0 + 8 < len;
#pragma unroll
    for (int i = 0; i < NH; i += 2) store_pair<T>(dq, ldc, 8 * i, Q[i], Q[i + 1], uq, on0, on1, lane);
    // K += N^T K + dP^T Q
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      if (kb < m) continue;
      const uint32_t at = s0 + tile_off<128>(16 * kb + (lane & 15), 2 * m + (lane >> 4));
      uint32_t ap[2][4], an[2][4];   // terms
#pragma unroll
      for (int x = 0; x < (kTwo ? 2 : 1); ++x) {
        uint32_t rp[4], rn[4];
        ldsm4t(rp, at + L::dp + x * L::lo);
        ldsm4t(rn, at + L::n + x * L::lo);
        ap[x][0] = rp[0]; ap[x][1] = rp[2]; ap[x][2] = rp[1]; ap[x][3] = rp[3];
        an[x][0] = rn[0]; an[x][1] = rn[2]; an[x][2] = rn[1]; an[x][3] = rn[3];
        if (fpq != 1.0f) scale_frag(ap[x], fpq);
        if (fnk != 1.0f) scale_frag(an[x], fnk);
      }
#pragma unroll
      for (int np = 0; np < NH / 2; ++np) {
        uint32_t bk[4], bq[4];
        ldsm4t(bk, cols(kb, np) + L::k);
        ldsm4t(bq, cols(kb, np) + L::q);
#pragma unroll
        for (int x = 0; x < (kTwo ? 2 : 1); ++x) {
          mma_f16(K[2 * np], an[x], bk[0], bk[1]);
          mma_f16(K[2 * np + 1], an[x], bk[2], bk[3]);
          mma_f16(K[2 * np], ap[x], bq[0], bq[1]);
          mma_f16(K[2 * np + 1], ap[x], bq[2], bq[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      set_lo(K[i], fma2(row_lo(K[i]), splat(uk), row_lo(X[i])));
      set_hi(K[i], fma2(row_hi(K[i]), splat(uk), row_hi(X[i])));
    }
#pragma unroll
    for (int i = 0; i < NH; i += 2) store_pair<T>(dk, ldc, 8 * i, K[i], K[i + 1], 1.0f, on0, on1, lane);
    __syncthreads();   // K, Q, dP, N have been used, the dots are written
    fetch_keys(next);
    if (warp == 0) {   // the gates' gradients, two tokens a lane
      float A[2], B[2], F[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e, blk = i >> 4;
        A[e] = B[e] = 0.0f;
#pragma unroll
        for (int j = 0; j < CW; ++j) {
          A[e] += as[j * 64 + i];
          B[e] += bs[j * 64 + i];
        }
        F[e] = wdiag[i];   // the rectangle of W: the diagonal block's, the block row's, the block column's, whole blocks
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (j < blk) F[e] += wrows[j * 64 + i];
#pragma unroll
        for (int j = 1; j < 4; ++j)
          if (j > blk) F[e] += wcols[j * 64 + i];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int l = 2; l < 4; ++l)
            if (j < blk && blk < l) F[e] += wrows[j * 64 + 16 * l];
      }
      const float cc = head_sum<32>(lane < KS ? red[16 + lane] : 0.0f) * sinv * (last * dsinv);
      float later = A[0] + A[1], earlier = B[0] + B[1];   // over this lane's tokens and those behind (before) them
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, later, o), z = __shfl_up_sync(0xffffffffu, earlier, o);
        if (lane + o < 32) later += y;
        if (lane >= o) earlier += z;
      }
      const float behind = __shfl_down_sync(0xffffffffu, later, 1), before = __shfl_up_sync(0xffffffffu, earlier, 1);
      const float b0 = lane > 0 ? before : 0.0f, a1 = (lane < 31 ? behind : 0.0f) + A[1];
      const float dl[2] = {F[0] + (later + b0 + cc), F[1] + (a1 + (b0 + B[0]) + cc)};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        if (i < len) {
          const float a = sweep::clamp(sweep::widen(la[e])), bb = sweep::clamp(sweep::widen(lb[e]));
          static_cast<T *>(p.da)[(row + i) * p.s.H + h] = sweep::narrow<T>(dl[e] / (1.0f + expf(a)));
          static_cast<T *>(p.db)[(row + i) * p.s.H + h] = sweep::narrow<T>(udu[i] / (1.0f + expf(bb)));
        }
      }
    }
  }
  sweep::cp_async_wait<0>();
}

template <typename T, int D>
int run(const ChunkArgs &a, cudaStream_t st) {
  using L = GradShape<D, two_terms<T>()>;
  auto kern = delta_grad_kernel<T, D>;
  int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total));
  if (rc) return rc;
  int per_sm = 0;
  if ((rc = runtime_status(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, L::threads, L::total)))) return rc;
  const long long chunks = static_cast<long long>(a.s.B) * a.s.H * a.w.nc, full = static_cast<long long>(sm_count()) * (per_sm > 0 ? per_sm : 1);
  kern<<<static_cast<unsigned>(chunks < full ? chunks : full), L::threads, L::total, st>>>(a, static_cast<int>(chunks));
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
