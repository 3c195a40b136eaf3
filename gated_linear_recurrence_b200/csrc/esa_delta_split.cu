// esa_delta_split.cu -- the two chain kernels of the chunked gated delta rule
// for few heads: four warps, one per SM quarter, share 16 value channels
// (sm_100a).
//
// The mathematics, the scales and the roundings are those of
// esa_delta_chain.cu and esa_delta_chain_bwd.cu.  There a warp carries 16
// value channels alone; with few heads most SMs are idle while each chunk
// waits for one warp's 400 to 484 mma and the conversions between them.  Here
// the state's key channels are split over the block's four warps (a quarter of
// S^T each), and each warp forms the chunk's rows for 16 of the 64 tokens:
//   1. every warp multiplies its quarter of S^T by K^T (and Q^T) for all
//      tokens; the partial sums meet in shared memory, where each warp adds
//      those of its own tokens and forms R (dU) for them;
//   2. all of R meets in shared memory; each warp solves for its tokens' U;
//   3. all of U meets; each warp adds to its quarter of the state, and
//      finishes the outputs of its tokens.
// Four barriers a chunk.  At 16 heads of D = 128 a chunk takes 2.5 us forward
// (with what the backward reads) against 4.9 with a warp a slice, 2.7 against
// 4.8 backward.
#include <type_traits>

#include "esa_delta_chunk.h"
#include "esa_delta_sweep.cuh"
#include "esa_mma.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

constexpr int kThreads = 128;
constexpr int kTileF = 32 * 16;   // bytes of an accumulator tile of a warp: a float4 a lane

template <int D, bool BWD, bool TWO>   // TWO: the forward's with the second term of P
struct SplitSmem {
  using R = ChunkRecord<D>;
  static constexpr int rows = BWD ? R::bytes : TWO ? R::g : R::pl;   // v (dy) rows, 32 bytes each
  static constexpr int stage = rows + 64 * 32;
  static constexpr int part = 2 * stage;                        // [warp][tile] partial sums
  static constexpr int party = part + 32 * kTileF;              // the output's (forward)
  static constexpr int mid = party + (BWD ? 0 : 32 * kTileF);   // R (dU) of all tokens, then U (du) in `fin`
  static constexpr int fin = mid + 8 * kTileF;
  static constexpr int top = fin + 8 * kTileF;                  // [4][row][warp] maxima
  static constexpr int total = top + 4 * 4 * 16 * 4;
};

__device__ __forceinline__ void put_tile(unsigned char *p, const float (&c)[4], int lane) {
  reinterpret_cast<float4 *>(p)[lane] = make_float4(c[0], c[1], c[2], c[3]);
}
__device__ __forceinline__ void get_tile(const unsigned char *p, float (&c)[4], int lane) {
  const float4 v = reinterpret_cast<const float4 *>(p)[lane];
  c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
}
__device__ __forceinline__ void add_tile(const unsigned char *p, float (&c)[4], int lane) {
  const float4 v = reinterpret_cast<const float4 *>(p)[lane];
  set_lo(c, add2(row_lo(c), make_float2(v.x, v.y)));
  set_hi(c, add2(row_hi(c), make_float2(v.z, v.w)));
}
// The largest of each row (value channel): each warp's, from its threads', and that of the four warps.
__device__ __forceinline__ void put_top(float *t, int w, float2 x, int lane) {
  x = quad_max(x);
  if ((lane & 3) == 0) {
    t[lane + w] = x.x;
    t[32 + lane + w] = x.y;
  }
}
__device__ __forceinline__ float2 get_top(const float *t, int g) {
  const float4 a = reinterpret_cast<const float4 *>(t)[g], b = reinterpret_cast<const float4 *>(t)[8 + g];
  return make_float2(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
}
template <int N>
__device__ __forceinline__ void zero_tiles(float (&c)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[i][e] = 0.0f;
}

// State rows dvw .. + 15 and this warp's key channels, to and from [D][D] float32.
template <int D>
__device__ __forceinline__ void load_state(float (&S)[D / 32][4], const float *s, int row0, int dk0, int g, int t4) {
#pragma unroll
  for (int nt = 0; nt < D / 32; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[nt][e] = s ? s[(dk0 + 8 * nt + 2 * t4 + (e & 1)) * D + row0 + g + (e >> 1) * 8] : 0.0f;
}
template <int D>
__device__ __forceinline__ void store_state(const float (&S)[D / 32][4], float2 f, float *s, int row0, int dk0, int g, int t4) {
#pragma unroll
  for (int nt = 0; nt < D / 32; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[(dk0 + 8 * nt + 2 * t4 + (e & 1)) * D + row0 + g + (e >> 1) * 8] = S[nt][e] * (e < 2 ? f.x : f.y);
}

template <typename T, int D, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1) delta_split_fwd_kernel(ChunkArgs p) {
  constexpr bool kTwo = std::is_same<T, __half>::value;
  using L = SplitSmem<D, false, kTwo>;
  using R = ChunkRecord<D>;
  constexpr int KQ = D / 64, NQ = D / 32;   // k-steps and accumulator tiles of a quarter of the key channels
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int head = blockIdx.x / (D / 16), slice = blockIdx.x % (D / 16), dvw = 16 * slice;
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int nc = p.w.nc;
  const long long c0 = static_cast<long long>(head) * nc, row0 = static_cast<long long>(b) * p.s.T;
  const T *v = static_cast<const T *>(p.v) + h * D + dvw + (threadIdx.x & 1) * 8;
  const long long ldy = static_cast<long long>(p.s.H) * D;
  T *y = static_cast<T *>(p.y) + h * D + dvw + 8 * (lane & 1);
  const uint32_t s0 = smem_u32(smem);
  float *tops_ = reinterpret_cast<float *>(smem + L::top);   // rows: state, R, U, U decayed

  auto fetch = [&](int n, int buf) {
    const uint32_t s = s0 + buf * L::stage;
    copy_linear<L::rows, kThreads>(s, p.w.rec + (c0 + n) * R::bytes);
    const int len = min(kChunk, p.s.T - n * kChunk), r = threadIdx.x >> 1;   // 64 rows of two units
    cp_async16_zfill(s + L::rows + tile_off<32>(r, threadIdx.x & 1),
                     r < len ? v + (row0 + n * kChunk + r) * p.s.ld_v : v, r < len);
    sweep::cp_async_commit();
  };

  float S[NQ][4];
  float2 sinv = splat(1.0f);
  load_state<D>(S, p.S_in ? p.S_in + static_cast<long long>(head) * D * D : nullptr, dvw, w * (D / 4), g, t4);
  fetch(0, 0);
#pragma unroll 1
  for (int n = 0; n < nc; ++n) {
    const int buf = n & 1;
    {
      float2 top = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < NQ; ++i) top = max_rows(S[i], top);
      put_top(tops_, w, top, lane);
    }
    if (n + 1 < nc) {
      fetch(n + 1, buf ^ 1);
      sweep::cp_async_wait<1>();
    } else {
      sweep::cp_async_wait<0>();
    }
    __syncthreads();
    const uint32_t st = s0 + buf * L::stage;
    unsigned char *sb = smem + buf * L::stage;
    const LaneOff<D * 2> ofd(lane, st);
    const LaneOffB<D * 2> ofb(lane, st);
    const uint32_t tri0 = LaneOffB<32>(lane, st).o[0];
    const float *tok = reinterpret_cast<const float *>(sb + R::tok) + 2 * t4;
    const Fac fac = load_fac(sb + R::fac);
    const long long c = c0 + n;
    // The quarter's block columns: D = 128 has two a warp, D = 64 one.
    auto colb = [&](int np, int j) -> uint32_t {   // [token][channel] B blocks
      if constexpr (D == 128) return ((w & 1) ? ofb.at(np, 2 + j) : ofb.at(np, j)) + (w >> 1) * 128u;
      else return (w & 1 ? (w & 2 ? ofb.at(np, 3) : ofb.at(np, 1)) : (w & 2 ? ofb.at(np, 2) : ofb.at(np, 0)));
    };
    auto cold = [&](int kb, int j) -> uint32_t {   // the same, loaded with .trans
      if constexpr (D == 128) return ((w & 1) ? ofd.at(kb, 2 + j) : ofd.at(kb, j)) + (w >> 1) * 128u;
      else return (w & 1 ? (w & 2 ? ofd.at(kb, 3) : ofd.at(kb, 1)) : (w & 2 ? ofd.at(kb, 2) : ofd.at(kb, 0)));
    };

    // 1. partial X = S^T K^T and S^T Q^T
    float Xo[2][4], Yo[2][4];   // this warp's tokens
    const float2 tops = get_top(tops_, g);
    const RowPow2 ps = pow2_scale(tops);
    const float2 sunit = mul2(ps.inv, sinv), xinv = unit_or_zero(tops, sunit);
    float2 sf;
    if constexpr (KEEP) {
      const float all = warp_max(fmaxf(tops.x * sinv.x, tops.y * sinv.y));
      const Pow2 pss = store_scale(all);
      sf = mul2(splat(pss.s), xinv);
      if (threadIdx.x == 0) p.w.slice[c * 32 + kSliceS + slice] = slice_unit(all, pss);
    }
    {
      float X[8][4], Y[8][4];
      zero_tiles(X);
      zero_tiles(Y);
#pragma unroll
      for (int ks = 0; ks < KQ; ++ks) {
        uint32_t hi[4], lo[4];
        split_rows(S[2 * ks], S[2 * ks + 1], ps.s, hi, lo);
        if constexpr (KEEP) {
          uint32_t x[4] = {hi[0], hi[1], hi[2], hi[3]};
          if (sf.x != 1.0f || sf.y != 1.0f) scale_h2(x, sf);
          store_block(p.w.s16 + c * (D * D) + dvw * D + w * (D / 4) + 16 * ks, D, x, lane);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t bk[4], bq[4];
          ldsm4(bk, colb(np, ks) + R::k);
          ldsm4(bq, colb(np, ks) + R::q);
          mma_f16(X[2 * np], hi, bk[0], bk[1]);
          mma_f16(X[2 * np + 1], hi, bk[2], bk[3]);
          mma_f16(Y[2 * np], hi, bq[0], bq[1]);
          mma_f16(Y[2 * np + 1], hi, bq[2], bq[3]);
          mma_f16(X[2 * np], lo, bk[0], bk[1]);
          mma_f16(X[2 * np + 1], lo, bk[2], bk[3]);
          if constexpr (kTwo) {
            mma_f16(Y[2 * np], lo, bq[0], bq[1]);
            mma_f16(Y[2 * np + 1], lo, bq[2], bq[3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        put_tile(smem + L::part + (w * 8 + i) * kTileF, X[i], lane);
        put_tile(smem + L::party + (w * 8 + i) * kTileF, Y[i], lane);
      }
    }
    __syncthreads();
    // R = beta V^T - (beta e^G) X for this warp's tokens, 16 w ..
    {
      zero_tiles(Xo);
      zero_tiles(Yo);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          add_tile(smem + L::part + (j * 8 + 2 * w + i) * kTileF, Xo[i], lane);
          add_tile(smem + L::party + (j * 8 + 2 * w + i) * kTileF, Yo[i], lane);
        }
      uint32_t vv[4];
      ldsm4t(vv, st + L::rows + tile_off<32>(16 * w + (lane & 15), lane >> 4));
      const float2 xk = mul2(xinv, splat(-fac.k));
      float2 top = make_float2(0.0f, 0.0f), chk0 = top, chk1 = top;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 be = *reinterpret_cast<const float2 *>(tok + kTokBeta * 64 + 16 * w + 8 * i);
        const float2 tx = *reinterpret_cast<const float2 *>(tok + kTokX * 64 + 16 * w + 8 * i);
        set_lo(Xo[i], fma2(mul2(tx, splat(xk.x)), row_lo(Xo[i]), mul2(be, unpack_io<T>(vv[i]))));
        set_hi(Xo[i], fma2(mul2(tx, splat(xk.y)), row_hi(Xo[i]), mul2(be, unpack_io<T>(vv[2 + i]))));
        chk0 = fma2(row_lo(Xo[i]), splat(0.0f), chk0);
        chk1 = fma2(row_hi(Xo[i]), splat(0.0f), chk1);
        top = max_rows(Xo[i], top);
        put_tile(smem + L::mid + (2 * w + i) * kTileF, Xo[i], lane);
      }
      // an entry that is not finite is announced as its row's infinite maximum
      if (!(chk0.x + chk0.y == 0.0f)) top.x = __int_as_float(0x7f800000);
      if (!(chk1.x + chk1.y == 0.0f)) top.y = __int_as_float(0x7f800000);
      put_top(tops_ + 64, w, top, lane);
    }
    __syncthreads();
    // 2. U = R T^T for this warp's tokens: all of R up to them
    float2 topr = get_top(tops_ + 64, g);
    const bool cut = __any_sync(0xffffffffu, fmaxf(topr.x, topr.y) == __int_as_float(0x7f800000)) || fac.first < 64.0f;
    int first[2] = {static_cast<int>(fac.first), static_cast<int>(fac.first)};   // first token from which a row is not finite
    if (cut) {
      topr = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (int i = 7; i >= 0; --i) {
        float r[4];
        get_tile(smem + L::mid + i * kTileF, r, lane);
#pragma unroll
        for (int e = 3; e >= 0; --e)
          if (!(fabsf(r[e]) <= 3.4028235e38f)) first[e >> 1] = min(first[e >> 1], 8 * i + 2 * t4 + (e & 1));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        first[r] = min(first[r], __shfl_xor_sync(0xffffffffu, first[r], 1));
        first[r] = min(first[r], __shfl_xor_sync(0xffffffffu, first[r], 2));
      }
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        float r[4];
        get_tile(smem + L::mid + i * kTileF, r, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * i + 2 * t4 + (e & 1) >= first[e >> 1]) r[e] = 0.0f;
        topr = max_rows(r, topr);
      }
      topr = quad_max(topr);
    }
    const RowPow2 pr = pow2_scale(topr);
    float Uo[2][4];
    {
      float A[3][2][4];   // the three products of the two terms, summed apart: shorter chains
#pragma unroll
      for (int i = 0; i < 3; ++i) zero_tiles(A[i]);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb > w) continue;
        float r0[4], r1[4];
        get_tile(smem + L::mid + (2 * kb) * kTileF, r0, lane);
        get_tile(smem + L::mid + (2 * kb + 1) * kTileF, r1, lane);
        if (cut) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (16 * kb + 2 * t4 + (e & 1) >= first[e >> 1]) r0[e] = 0.0f;
            if (16 * kb + 8 + 2 * t4 + (e & 1) >= first[e >> 1]) r1[e] = 0.0f;
          }
        }
        uint32_t hi[4], lo[4], bh[4], bl[4];
        split_rows(r0, r1, pr.s, hi, lo);
        const uint32_t at = tri0 + (w * (w + 1) / 2 + kb) * 512;
        ldsm4(bh, at + R::th);
        ldsm4(bl, at + R::tl);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma_f16(A[0][i], hi, bh[2 * i], bh[2 * i + 1]);
          mma_f16(A[1][i], lo, bh[2 * i], bh[2 * i + 1]);
          mma_f16(A[2][i], hi, bl[2 * i], bl[2 * i + 1]);
        }
      }
      const float2 uf = mul2(pr.inv, splat(fac.t));
      float2 top = make_float2(0.0f, 0.0f), topl = top;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 tl = *reinterpret_cast<const float2 *>(tok + kTokL * 64 + 16 * w + 8 * i);
        set_lo(Uo[i], mul2(add2(row_lo(A[0][i]), add2(row_lo(A[1][i]), row_lo(A[2][i]))), splat(uf.x)));
        set_hi(Uo[i], mul2(add2(row_hi(A[0][i]), add2(row_hi(A[1][i]), row_hi(A[2][i]))), splat(uf.y)));
        top = max_rows(Uo[i], top);
        float x[4];
        set_lo(x, mul2(row_lo(Uo[i]), tl));
        set_hi(x, mul2(row_hi(Uo[i]), tl));
        topl = max_rows(x, topl);
        put_tile(smem + L::fin + (2 * w + i) * kTileF, Uo[i], lane);
      }
      put_top(tops_ + 128, w, top, lane);
      put_top(tops_ + 192, w, topl, lane);
    }
    __syncthreads();
    // 3. the state's quarter, and the outputs of this warp's tokens
    const float2 topu = get_top(tops_ + 128, g);
    const RowPow2 pu = pow2_scale(topu);
    const float2 asc = update_scale(mul2(get_top(tops_ + 192, g), splat(fac.k)), tops, sunit, fac.last);
    {
      const float2 sc = mul2(mul2(asc, splat(fac.last)), sinv);
#pragma unroll
      for (int i = 0; i < NQ; ++i) scale_rows(S[i], sc);
      sinv = make_float2(pow2_inverse(asc.x), pow2_inverse(asc.y));
    }
    const float2 xs = mul2(asc, splat(fac.k));
    const OutputUnit ou0 = output_unit(xinv.x * fac.q, pu.inv.x, fac.p, fac.ps, p.least),
                     ou1 = output_unit(xinv.y * fac.q, pu.inv.y, fac.p, fac.ps, p.least);
    const float2 us = make_float2(ou0.us, ou1.us), yf = mul2(make_float2(ou0.unit, ou1.unit), splat(p.s.scale));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 ty = *reinterpret_cast<const float2 *>(tok + kTokY * 64 + 16 * w + 8 * i);
      set_lo(Yo[i], mul2(row_lo(Yo[i]), mul2(ty, splat(ou0.r))));
      set_hi(Yo[i], mul2(row_hi(Yo[i]), mul2(ty, splat(ou1.r))));
    }
    uint32_t own[4];
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      float u0[4], u1[4];
      get_tile(smem + L::fin + (2 * kb) * kTileF, u0, lane);
      get_tile(smem + L::fin + (2 * kb + 1) * kTileF, u1, lane);
      uint32_t hi[4], lo[4];
      const float2 l0 = *reinterpret_cast<const float2 *>(tok + kTokL * 64 + 16 * kb);
      const float2 l1 = *reinterpret_cast<const float2 *>(tok + kTokL * 64 + 16 * kb + 8);
      split_grid(u0, u1, l0, l1, xs, hi, lo);
#pragma unroll
      for (int j = 0; j < NQ / 2; ++j) {
        uint32_t bk[4];
        ldsm4t(bk, cold(kb, j) + R::k);
        mma_f16(S[2 * j], hi, bk[0], bk[1]);
        mma_f16(S[2 * j + 1], hi, bk[2], bk[3]);
        mma_f16(S[2 * j], lo, bk[0], bk[1]);
        mma_f16(S[2 * j + 1], lo, bk[2], bk[3]);
      }
      if (kb <= w) {
        uint32_t uh[4], ul[4], bp[4];
        if constexpr (kTwo) split_rows(u0, u1, us, uh, ul);
        else single_rows(u0, u1, us, uh);
        ldsm4(bp, tri0 + (w * (w + 1) / 2 + kb) * 512 + R::ph);
        mma_f16(Yo[0], uh, bp[0], bp[1]);
        mma_f16(Yo[1], uh, bp[2], bp[3]);
        if constexpr (kTwo) {
          mma_f16(Yo[0], ul, bp[0], bp[1]);
          mma_f16(Yo[1], ul, bp[2], bp[3]);
          ldsm4(bp, tri0 + (w * (w + 1) / 2 + kb) * 512 + R::pl);
          mma_f16(Yo[0], uh, bp[0], bp[1]);
          mma_f16(Yo[1], uh, bp[2], bp[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) own[e] = uh[e];   // the last one is this warp's own tokens
      }
    }
    if (cut) {
      const float nan = __int_as_float(0x7fc00000);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * w + 8 * i + 2 * t4 + (e & 1) >= first[e >> 1]) Yo[i][e] = nan;
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (first[e >> 1] < 64) S[i][e] = nan;
    }
    const int len = min(kChunk, p.s.T - n * kChunk), r = 16 * w + (lane >> 1);
    const uint32_t vw = st + L::rows + tile_off<32>(16 * w + (lane & 15), lane >> 4);
    const unsigned char *vr = sb + L::rows + tile_off<32>(r, lane & 1);
    {   // this warp's 16 rows of the value tile were read before the second barrier
      const float2 a = mul2(row_lo(Yo[0]), splat(yf.x)), bb = mul2(row_lo(Yo[1]), splat(yf.x));
      const float2 cc = mul2(row_hi(Yo[0]), splat(yf.y)), d = mul2(row_hi(Yo[1]), splat(yf.y));
      const uint32_t o[4] = {pack_io<T>(a.x, a.y), pack_io<T>(bb.x, bb.y), pack_io<T>(cc.x, cc.y), pack_io<T>(d.x, d.y)};
      stsm4t(vw, o);
      __syncwarp();
      if (r < len) *reinterpret_cast<uint4 *>(y + (row0 + n * kChunk + r) * ldy) = *reinterpret_cast<const uint4 *>(vr);
      if constexpr (KEEP) {
        __syncwarp();
        const float all = warp_max(fmaxf(topu.x, topu.y));
        const Pow2 pus = store_scale(all);
        if (pus.s != us.x || pus.s != us.y) single_rows(Uo[0], Uo[1], splat(pus.s), own);
        const uint32_t u[4] = {own[0], own[2], own[1], own[3]};
        stsm4t(vw, u);
        __syncwarp();
        *reinterpret_cast<uint4 *>(p.w.u16 + (c * 64 + r) * D + dvw + 8 * (lane & 1)) = *reinterpret_cast<const uint4 *>(vr);
        if constexpr (kTwo) {   // and the second term
          uint32_t hi[4], lo[4];
          split_rows(Uo[0], Uo[1], splat(pus.s), hi, lo);
          const uint32_t ul[4] = {lo[0], lo[2], lo[1], lo[3]};
          __syncwarp();
          stsm4t(vw, ul);
          __syncwarp();
          *reinterpret_cast<uint4 *>(p.w.u16l + (c * 64 + r) * D + dvw + 8 * (lane & 1)) = *reinterpret_cast<const uint4 *>(vr);
        }
        if (threadIdx.x == 0) p.w.slice[c * 32 + kSliceU + slice] = cut ? __int_as_float(0x7fc00000) : slice_unit(all, pus);
      }
    }
    __syncthreads();
  }
  if (p.S_out != nullptr) store_state<D>(S, sinv, p.S_out + static_cast<long long>(head) * D * D, dvw, w * (D / 4), g, t4);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) delta_split_bwd_kernel(ChunkArgs p) {
  using L = SplitSmem<D, true, false>;
  using R = ChunkRecord<D>;
  constexpr int KQ = D / 64, NQ = D / 32;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int head = blockIdx.x / (D / 16), slice = blockIdx.x % (D / 16), dvw = 16 * slice;
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int nc = p.w.nc;
  const long long c0 = static_cast<long long>(head) * nc, row0 = static_cast<long long>(b) * p.s.T;
  const long long ldc = static_cast<long long>(p.s.H) * D;
  const T *dy = static_cast<const T *>(p.dy) + h * D + dvw + (threadIdx.x & 1) * 8;
  T *dv = static_cast<T *>(p.dv) + h * D + dvw + 8 * (lane & 1);
  const uint32_t s0 = smem_u32(smem);
  float *tops_ = reinterpret_cast<float *>(smem + L::top);   // rows: state, dU, du, du decayed

  auto fetch = [&](int n, int buf) {
    const uint32_t s = s0 + buf * L::stage;
    copy_linear<R::bytes, kThreads>(s, p.w.rec + (c0 + n) * R::bytes);
    const int len = min(kChunk, p.s.T - n * kChunk), r = threadIdx.x >> 1;
    cp_async16_zfill(s + L::rows + tile_off<32>(r, threadIdx.x & 1), r < len ? dy + (row0 + n * kChunk + r) * ldc : dy, r < len);
    sweep::cp_async_commit();
  };

  float S[NQ][4];
  float2 sinv = splat(1.0f);
  load_state<D>(S, p.S_in ? p.S_in + static_cast<long long>(head) * D * D : nullptr, dvw, w * (D / 4), g, t4);
  fetch(nc - 1, 0);
#pragma unroll 1
  for (int it = 0; it < nc; ++it) {
    const int n = nc - 1 - it, buf = it & 1;
    {
      float2 top = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < NQ; ++i) top = max_rows(S[i], top);
      put_top(tops_, w, top, lane);
    }
    if (n > 0) {
      fetch(n - 1, buf ^ 1);
      sweep::cp_async_wait<1>();
    } else {
      sweep::cp_async_wait<0>();
    }
    __syncthreads();
    const uint32_t st = s0 + buf * L::stage;
    unsigned char *sb = smem + buf * L::stage;
    const LaneOff<D * 2> ofd(lane, st);
    const LaneOffB<D * 2> ofb(lane, st);
    const uint32_t tri0 = LaneOff<32>(lane, st).o[0];
    const float *tok = reinterpret_cast<const float *>(sb + R::tok) + 2 * t4;
    const Fac fac = load_fac(sb + R::fac);
    const long long c = c0 + n;
    auto colb = [&](int np, int j) -> uint32_t {
      if constexpr (D == 128) return ((w & 1) ? ofb.at(np, 2 + j) : ofb.at(np, j)) + (w >> 1) * 128u;
      else return (w & 1 ? (w & 2 ? ofb.at(np, 3) : ofb.at(np, 1)) : (w & 2 ? ofb.at(np, 2) : ofb.at(np, 0)));
    };
    auto cold = [&](int kb, int j) -> uint32_t {
      if constexpr (D == 128) return ((w & 1) ? ofd.at(kb, 2 + j) : ofd.at(kb, j)) + (w >> 1) * 128u;
      else return (w & 1 ? (w & 2 ? ofd.at(kb, 3) : ofd.at(kb, 1)) : (w & 2 ? ofd.at(kb, 2) : ofd.at(kb, 0)));
    };

    // 1. partial dS^T K^T; dO^T as an A operand (every warp needs all of it)
    const float2 tops = get_top(tops_, g);
    const RowPow2 ps = pow2_scale(tops);
    const float2 sunit = mul2(ps.inv, sinv), xinv = unit_or_zero(tops, sunit);
    const float alls = warp_max(fmaxf(tops.x * sinv.x, tops.y * sinv.y));
    const Pow2 pss = store_scale(alls);
    const float2 sf = mul2(splat(pss.s), xinv);
    if (threadIdx.x == 0) p.w.slice[c * 32 + kSliceDs + slice] = slice_unit(alls, pss);
    {
      float X[8][4];
      zero_tiles(X);
#pragma unroll
      for (int ks = 0; ks < KQ; ++ks) {
        uint32_t hi[4], lo[4];
        split_rows(S[2 * ks], S[2 * ks + 1], ps.s, hi, lo);
        uint32_t x[4] = {hi[0], hi[1], hi[2], hi[3]};
        if (sf.x != 1.0f || sf.y != 1.0f) scale_h2(x, sf);
        store_block(p.w.ds16 + c * (D * D) + dvw * D + w * (D / 4) + 16 * ks, D, x, lane);
#pragma unroll
        for (int np = 0; np < 4; np += 2) {
          uint32_t b0[4], b1[4];
          ldsm4(b0, colb(np, ks) + R::k);
          ldsm4(b1, colb(np + 1, ks) + R::k);
          mma_f16(X[2 * np], hi, b0[0], b0[1]);
          mma_f16(X[2 * np + 1], hi, b0[2], b0[3]);
          mma_f16(X[2 * np + 2], hi, b1[0], b1[1]);
          mma_f16(X[2 * np + 3], hi, b1[2], b1[3]);
          mma_f16(X[2 * np], lo, b0[0], b0[1]);
          mma_f16(X[2 * np + 1], lo, b0[2], b0[3]);
          mma_f16(X[2 * np + 2], lo, b1[0], b1[1]);
          mma_f16(X[2 * np + 3], lo, b1[2], b1[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) put_tile(smem + L::part + (w * 8 + i) * kTileF, X[i], lane);
    }
    uint32_t od[4][4];   // registers 0 and 2 of a block are row g
    float2 topd = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t r[4];
      ldsm4t(r, st + L::rows + tile_off<32>(16 * kb + (lane & 15), lane >> 4));
      od[kb][0] = r[0]; od[kb][1] = r[2]; od[kb][2] = r[1]; od[kb][3] = r[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = unpack_io<T>(od[kb][e]);
        float &t = e & 1 ? topd.y : topd.x;
        t = fmaxf(fmaxf(t, fabsf(x.x)), fabsf(x.y));
      }
    }
    // the unit of the output gradient's share of dU^T (see kLeastShare); without a share (scale 0) P is left out
    const bool with = p.s.scale != 0.0f;
    const float2 xk = mul2(xinv, splat(fac.k));
    const RowPow2 pd = pow2_scale(quad_max(topd)), pz = with ? least_unit(pd, xk, fabsf(p.iscale), fac.ps) : pd;
    const float2 low = mul2(pd.inv, pz.s);   // what the product with P takes of dO: 1 unless its unit is too small
    const float2 zf = with ? make_float2(mul_pow2(p.s.scale, fac.p, pz.inv.x), mul_pow2(p.s.scale, fac.p, pz.inv.y)) : splat(1.0f);
    const float2 yd = mul2(pd.inv, splat(p.s.scale));
    // xk / zf; 1 / zf is at most 2^120
    const float2 xr = with ? mul2(xk, make_float2(mul_pow2(p.iscale, pz.s.x, fac.ps), mul_pow2(p.iscale, pz.s.y, fac.ps))) : xk;
    float2 topo = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = mul2(unpack_io<T>(od[kb][e]), splat(e & 1 ? pd.s.y : pd.s.x));
        od[kb][e] = pack2(x);
        const float2 z = mul2(x, mul2(*reinterpret_cast<const float2 *>(tok + kTokY * 64 + 16 * kb + 8 * (e >> 1)), splat(e & 1 ? yd.y : yd.x)));
        float &t = e & 1 ? topo.y : topo.x;
        t = fmaxf(fmaxf(t, fabsf(z.x)), fabsf(z.y));
      }
    topo = quad_max(topo);
    __syncthreads();
    // dU^T = zf (X r + dO^T P) for this warp's tokens, 16 w ..
    {
      float X[2][4];
      zero_tiles(X);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) add_tile(smem + L::part + (j * 8 + 2 * w + i) * kTileF, X[i], lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 tl = *reinterpret_cast<const float2 *>(tok + kTokL * 64 + 16 * w + 8 * i);
        set_lo(X[i], mul2(row_lo(X[i]), mul2(tl, splat(xr.x))));
        set_hi(X[i], mul2(row_hi(X[i]), mul2(tl, splat(xr.y))));
      }
      if (with) {
        float Z[2][4];
        zero_tiles(Z);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          if (kb < w) continue;
          uint32_t bh[4], bl[4];
          const uint32_t at = tri0 + kb * (kb + 1) / 2 * 512 + w * 512;
          ldsm4t(bh, at + R::ph);
          ldsm4t(bl, at + R::pl);
          uint32_t o[4] = {od[kb][0], od[kb][1], od[kb][2], od[kb][3]};
          if (low.x != 1.0f || low.y != 1.0f) scale_h2(o, low);
          mma_f16(X[0], o, bh[0], bh[1]);
          mma_f16(X[1], o, bh[2], bh[3]);
          mma_f16(Z[0], o, bl[0], bl[1]);
          mma_f16(Z[1], o, bl[2], bl[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          set_lo(X[i], add2(row_lo(X[i]), row_lo(Z[i])));
          set_hi(X[i], add2(row_hi(X[i]), row_hi(Z[i])));
        }
      }
      float2 top = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top = max_rows(X[i], top);
        put_tile(smem + L::mid + (2 * w + i) * kTileF, X[i], lane);
      }
      put_top(tops_ + 64, w, top, lane);
    }
    __syncthreads();
    // 2. du^T = dU^T T for this warp's tokens: all of dU from them on
    const RowPow2 pr = pow2_scale(get_top(tops_ + 64, g));
    const float2 rf = mul2(mul2(pr.inv, zf), splat(fac.tb));
    float Uo[2][4];
    {
      float A[3][2][4];
#pragma unroll
      for (int i = 0; i < 3; ++i) zero_tiles(A[i]);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb < w) continue;
        float r0[4], r1[4];
        get_tile(smem + L::mid + (2 * kb) * kTileF, r0, lane);
        get_tile(smem + L::mid + (2 * kb + 1) * kTileF, r1, lane);
        uint32_t hi[4], lo[4], bh[4], bl[4];
        split_rows(r0, r1, pr.s, hi, lo);
        const uint32_t at = tri0 + kb * (kb + 1) / 2 * 512 + w * 512;
        ldsm4t(bh, at + R::th);
        ldsm4t(bl, at + R::tl);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma_f16(A[0][i], hi, bh[2 * i], bh[2 * i + 1]);
          mma_f16(A[1][i], lo, bh[2 * i], bh[2 * i + 1]);
          mma_f16(A[2][i], hi, bl[2 * i], bl[2 * i + 1]);
        }
      }
      float2 top = make_float2(0.0f, 0.0f), topx = top;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 tx = *reinterpret_cast<const float2 *>(tok + kTokX * 64 + 16 * w + 8 * i);
        set_lo(Uo[i], mul2(add2(row_lo(A[0][i]), add2(row_lo(A[1][i]), row_lo(A[2][i]))), splat(rf.x)));
        set_hi(Uo[i], mul2(add2(row_hi(A[0][i]), add2(row_hi(A[1][i]), row_hi(A[2][i]))), splat(rf.y)));
        top = max_rows(Uo[i], top);
        float x[4];
        set_lo(x, mul2(row_lo(Uo[i]), tx));
        set_hi(x, mul2(row_hi(Uo[i]), tx));
        topx = max_rows(x, topx);
        put_tile(smem + L::fin + (2 * w + i) * kTileF, Uo[i], lane);
      }
      put_top(tops_ + 128, w, top, lane);
      put_top(tops_ + 192, w, topx, lane);
    }
    __syncthreads();
    // 3. the quarter of dS^T, dv and du of this warp's tokens
    const float2 topu = get_top(tops_ + 128, g), topx = get_top(tops_ + 192, g);
    const float allu = warp_max(fmaxf(topu.x, topu.y));
    const Pow2 pus = store_scale(allu);
    const float2 upd = make_float2(fmaxf(topx.x * fac.k, topo.x * fac.q), fmaxf(topx.y * fac.k, topo.y * fac.q));
    const float2 asc = update_scale(upd, tops, sunit, fac.last);
    {
      const float2 sc = mul2(mul2(asc, splat(fac.last)), sinv);
#pragma unroll
      for (int i = 0; i < NQ; ++i) scale_rows(S[i], sc);
      sinv = make_float2(pow2_inverse(asc.x), pow2_inverse(asc.y));
    }
    const float2 os = mul2(yd, mul2(asc, splat(fac.q))), xs = mul2(asc, splat(-fac.k));
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      float u0[4], u1[4];
      get_tile(smem + L::fin + (2 * kb) * kTileF, u0, lane);
      get_tile(smem + L::fin + (2 * kb + 1) * kTileF, u1, lane);
      uint32_t hi[4], lo[4], qh[4], ql[4];
      const float2 x0 = *reinterpret_cast<const float2 *>(tok + kTokX * 64 + 16 * kb);
      const float2 x1 = *reinterpret_cast<const float2 *>(tok + kTokX * 64 + 16 * kb + 8);
      split_grid(u0, u1, x0, x1, xs, hi, lo);
      const float2 y0 = *reinterpret_cast<const float2 *>(tok + kTokY * 64 + 16 * kb);
      const float2 y1 = *reinterpret_cast<const float2 *>(tok + kTokY * 64 + 16 * kb + 8);
      split2(mul2(unpack_h2(od[kb][0]), mul2(y0, splat(os.x))), qh[0], ql[0]);
      split2(mul2(unpack_h2(od[kb][1]), mul2(y0, splat(os.y))), qh[1], ql[1]);
      split2(mul2(unpack_h2(od[kb][2]), mul2(y1, splat(os.x))), qh[2], ql[2]);
      split2(mul2(unpack_h2(od[kb][3]), mul2(y1, splat(os.y))), qh[3], ql[3]);
#pragma unroll
      for (int j = 0; j < NQ / 2; ++j) {
        uint32_t bk[4], bq[4];
        ldsm4t(bk, cold(kb, j) + R::k);
        ldsm4t(bq, cold(kb, j) + R::q);
        mma_f16(S[2 * j], hi, bk[0], bk[1]);
        mma_f16(S[2 * j + 1], hi, bk[2], bk[3]);
        mma_f16(S[2 * j], lo, bk[0], bk[1]);
        mma_f16(S[2 * j + 1], lo, bk[2], bk[3]);
        mma_f16(S[2 * j], qh, bq[0], bq[1]);
        mma_f16(S[2 * j + 1], qh, bq[2], bq[3]);
        mma_f16(S[2 * j], ql, bq[0], bq[1]);
        mma_f16(S[2 * j + 1], ql, bq[2], bq[3]);
      }
    }
    // every warp has read all of the dy tile (before the second barrier); this one's rows take dv, then du
    const int len = min(kChunk, p.s.T - n * kChunk), r = 16 * w + (lane >> 1);
    const uint32_t vw = st + L::rows + tile_off<32>(16 * w + (lane & 15), lane >> 4);
    const unsigned char *vr = sb + L::rows + tile_off<32>(r, lane & 1);
    {
      const float2 b0 = *reinterpret_cast<const float2 *>(tok + kTokBeta * 64 + 16 * w);
      const float2 b1 = *reinterpret_cast<const float2 *>(tok + kTokBeta * 64 + 16 * w + 8);
      const float2 a = mul2(row_lo(Uo[0]), b0), bb = mul2(row_lo(Uo[1]), b1);
      const float2 cc = mul2(row_hi(Uo[0]), b0), d = mul2(row_hi(Uo[1]), b1);
      const uint32_t o[4] = {pack_io<T>(a.x, a.y), pack_io<T>(bb.x, bb.y), pack_io<T>(cc.x, cc.y), pack_io<T>(d.x, d.y)};
      stsm4t(vw, o);
      __syncwarp();
      if (r < len) *reinterpret_cast<uint4 *>(dv + (row0 + n * kChunk + r) * ldc) = *reinterpret_cast<const uint4 *>(vr);
      __syncwarp();
      uint32_t x[4];
      single_rows(Uo[0], Uo[1], splat(pus.s), x);
      const uint32_t u[4] = {x[0], x[2], x[1], x[3]};
      stsm4t(vw, u);
      __syncwarp();
      *reinterpret_cast<uint4 *>(p.w.r16 + (c * 64 + r) * D + dvw + 8 * (lane & 1)) = *reinterpret_cast<const uint4 *>(vr);
      if constexpr (std::is_same<T, __half>::value) {   // and the second term
        uint32_t hi[4], lo[4];
        split_rows(Uo[0], Uo[1], splat(pus.s), hi, lo);
        const uint32_t ul[4] = {lo[0], lo[2], lo[1], lo[3]};
        __syncwarp();
        stsm4t(vw, ul);
        __syncwarp();
        *reinterpret_cast<uint4 *>(p.w.r16l + (c * 64 + r) * D + dvw + 8 * (lane & 1)) = *reinterpret_cast<const uint4 *>(vr);
      }
      if (threadIdx.x == 0) p.w.slice[c * 32 + kSliceR + slice] = slice_unit(allu, pus);
    }
    __syncthreads();
  }
  if (p.S_out != nullptr) store_state<D>(S, sinv, p.S_out + static_cast<long long>(head) * D * D, dvw, w * (D / 4), g, t4);
}

template <typename K>
int launch(K kern, int smem, const ChunkArgs &a, cudaStream_t st) {
  const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (rc) return rc;
  kern<<<static_cast<unsigned>(a.s.B) * a.s.H * (a.s.D / 16), kThreads, smem, st>>>(a);
  return runtime_status(cudaGetLastError());
}

template <typename T, int D>
int fwd(const ChunkArgs &a, cudaStream_t st) {
  constexpr int smem = SplitSmem<D, false, std::is_same<T, __half>::value>::total;
  return a.keep ? launch(delta_split_fwd_kernel<T, D, true>, smem, a, st) : launch(delta_split_fwd_kernel<T, D, false>, smem, a, st);
}
template <typename T, int D>
int bwd(const ChunkArgs &a, cudaStream_t st) {
  return launch(delta_split_bwd_kernel<T, D>, SplitSmem<D, true, false>::total, a, st);
}

}  // namespace

int launch_split_fwd(int dtype, const ChunkArgs &a, cudaStream_t st) {
  if (a.s.D == 128) return dtype == ESA_F16 ? fwd<__half, 128>(a, st) : fwd<__nv_bfloat16, 128>(a, st);
  return dtype == ESA_F16 ? fwd<__half, 64>(a, st) : fwd<__nv_bfloat16, 64>(a, st);
}
int launch_split_bwd(int dtype, const ChunkArgs &a, cudaStream_t st) {
  if (a.s.D == 128) return dtype == ESA_F16 ? bwd<__half, 128>(a, st) : bwd<__nv_bfloat16, 128>(a, st);
  return dtype == ESA_F16 ? bwd<__half, 64>(a, st) : bwd<__nv_bfloat16, 64>(a, st);
}

}  // namespace esa
