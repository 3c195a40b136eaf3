// esa_delta_chain.cu -- second kernel of the chunked gated delta rule: the
// state carried from chunk to chunk, and the outputs (sm_100a).
//
// Value channels do not mix, so a warp carries 16 of them through the whole
// sequence by itself: S^T (16 value channels x D key channels) stays in its
// registers as float32 accumulators, and every product of a chunk has the
// warp's 16 channels as its 16 rows, so that the accumulators of one product
// are the A operand of the next (esa_mma.cuh) and no shared memory, tensor
// memory round trip or barrier lies on the chain
//     X = S^T K^T,   R = beta (V^T - e^G X),   U = R T^T,   S^T <- e^{G_last} S^T + (e^{G_last - G} U) K.
// The B operands -- K, Q, T, P of the chunk -- are the same for all warps of a
// head; they are copied to shared memory one chunk ahead (cp.async, two
// buffers).  The output is Y^T = scale (e^G S^T Q^T + U P^T) from the same
// fragments.
//
// Rounding.  What enters the state keeps float32 accuracy: S, R, U and T are
// operands in two float16 terms each (22 bits, esa_mma.cuh), K is exact, sums
// are float32.  The output's own product takes S, U and P in one float16 term
// (2^-12 of a value on average) when the output is bfloat16 (2^-9), and in two
// when it is float16 (y 2.1e-4 off in the 2-norm, as its rounding alone; with P
// in one term 2.8e-4).
//
// Scales.  A row, a value channel, has its own powers of two (RowPow2): what is
// kept of an entry depends on its own channel alone, within the chunk.
//
// A chunk costs a warp 400 mma at D = 128 (130 of them off the chain).  The
// issue rate of mma.sync (8 clocks per m16n8k16 and SM quarter, measured 550
// TFLOP/s) bounds it with two warps per quarter, the latency of the dependent
// steps with one.  With few heads (the usual case of a long prompt) 16-row warps
// spread a head over eight SMs.  tcgen05 takes 128 rows, a whole head at D = 128:
// where heads fill their blocks anyway its rate would pay, at the price of the
// state's conversion through tensor memory three times a chunk; not tried.
#include <type_traits>

#include "esa_delta_chunk.h"
#include "esa_delta_sweep.cuh"
#include "esa_mma.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

template <int D, int W, bool TWO>   // TWO: with the second term of P
struct ChainSmem {
  using R = ChunkRecord<D>;
  static constexpr int kRow = 32 * W;   // bytes of a value row of the block
  static constexpr int v = TWO ? R::g : R::pl, stage = v + 64 * kRow;
  static constexpr int total = 2 * stage;
};

// A warp's 16 value channels (columns `unit`, `unit` + 1 of the tile) hold an
// entry that is not finite, or a key of the chunk does (from token `key` on).
// Entries that are not finite become zero, so that they cannot reach earlier
// tokens of the chunk through the zeros above the diagonals of T and P;
// first[r] is the token from which this thread's channels g and g + 8 are to
// be NaN.
template <typename T, int RB>
__device__ __noinline__ void cut_values(unsigned char *tile, int unit, int key, int *first) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  first[0] = first[1] = key;
  for (int r = 63; r >= 0; --r)
    for (int e = 0; e < 2; ++e) {
      const T *v = reinterpret_cast<const T *>(tile + tile_off<RB>(r, unit + e)) + g;
      if (!(fabsf(sweep::widen(*v)) <= 3.4028235e38f)) first[e] = min(first[e], r);
    }
  __syncwarp();
  for (int r = lane; r < 64; r += 32)
    for (int e = 0; e < 16; ++e) {
      T *v = reinterpret_cast<T *>(tile + tile_off<RB>(r, unit + (e >> 3))) + (e & 7);
      if (!(fabsf(sweep::widen(*v)) <= 3.4028235e38f)) *v = sweep::narrow<T>(0.0f);
    }
  __syncwarp();
}

// NaN into the staged output rows (32 bytes a token) of those channels.
template <typename T, int RB>
__device__ __noinline__ void poison_rows(unsigned char *tile, int unit, int first0, int first1) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  const T nan = sweep::narrow<T>(__int_as_float(0x7fc00000));
  if ((lane & 3) == 0)
    for (int r = 0; r < 64; ++r) {
      if (r >= first0) reinterpret_cast<T *>(tile + tile_off<RB>(r, unit))[g] = nan;
      if (r >= first1) reinterpret_cast<T *>(tile + tile_off<RB>(r, unit + 1))[g] = nan;
    }
  __syncwarp();
}

template <typename T, int D, int W, bool KEEP>
__global__ void __launch_bounds__(W * 32, 1) delta_chain_fwd_kernel(ChunkArgs p) {
  constexpr bool kTwo = std::is_same<T, __half>::value;    // two terms in the output's product
  using L = ChainSmem<D, W, kTwo>;
  using R = ChunkRecord<D>;
  constexpr int NT = D / 8;                                // accumulator tiles of the state
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  constexpr int SL = D / (16 * W);
  const int head = blockIdx.x / SL, slice = blockIdx.x - head * SL;
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int dv0 = slice * 16 * W;             // first value channel of the block
  const int dvw = dv0 + 16 * warp;            // and of this warp
  const int nc = p.w.nc;
  const long long c0 = static_cast<long long>(head) * nc;
  const long long row0 = static_cast<long long>(b) * p.s.T;
  const T *v = static_cast<const T *>(p.v) + h * D + dv0;
  T *y = static_cast<T *>(p.y) + h * D + dvw + 8 * (lane & 1);
  const long long ldy = static_cast<long long>(p.s.H) * D;
  const uint32_t s0 = smem_u32(smem);
  const uint32_t vofs = tile_off<L::kRow>(lane & 15, 2 * warp + (lane >> 4));          // this warp's columns, fragments
  const uint32_t vrow = tile_off<L::kRow>(lane >> 1, 2 * warp + (lane & 1));           // the same, 32-byte rows

  auto fetch = [&](int n, int buf) {
    const uint32_t s = s0 + buf * L::stage;
    copy_linear<L::v, W * 32>(s, p.w.rec + (c0 + n) * R::bytes);
    const int len = min(kChunk, p.s.T - n * kChunk);
    const T *src = v + (row0 + n * kChunk) * p.s.ld_v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // 64 rows of 2 W units, W 32 threads
      const int e = threadIdx.x + i * W * 32, r = e / (2 * W), u = e % (2 * W);
      const bool on = r < len;
      cp_async16_zfill(s + L::v + tile_off<L::kRow>(r, u), on ? src + r * p.s.ld_v + u * 8 : v, on);
    }
    sweep::cp_async_commit();
  };

  // S^T, each row times a power of two, 1 / sinv: each chunk leaves it in the
  // scale in which it added to it.
  float S[NT][4];
  float2 sinv = splat(1.0f);
  if (p.S_in != nullptr) {
    const float *Si = p.S_in + static_cast<long long>(head) * D * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[nt][e] = Si[(8 * nt + 2 * t4 + (e & 1)) * D + dvw + g + (e >> 1) * 8];
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[nt][e] = 0.0f;
  }

  bool dead0 = false, dead1 = false;   // channels g and g + 8 are NaN from an earlier token on
  fetch(0, 0);
#pragma unroll 1
  for (int n = 0; n < nc; ++n) {
    const int buf = n & 1;
    if (n + 1 < nc) {
      fetch(n + 1, buf ^ 1);
      sweep::cp_async_wait<1>();
    } else {
      sweep::cp_async_wait<0>();
    }
    __syncthreads();
    const uint32_t st = s0 + buf * L::stage;
    const LaneOff<D * 2> ofd(lane, st);        // tiles of keys and queries
    const LaneOffB<D * 2> ofb(lane, st);       // the same as [token][channel] B operands
    const uint32_t tri0 = LaneOffB<32>(lane, st).o[0];   // blocks of T and P
    const unsigned char *sb = smem + buf * L::stage;
    const float *tok = reinterpret_cast<const float *>(sb + R::tok) + 2 * t4;
    const Fac fac = load_fac(sb + R::fac);
    const long long c = c0 + n;
    int first0 = 64, first1 = 64;
    bool cut;
    {
      uint32_t top = fac.first < 64.0f ? 0x7f800000u : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = max(top, unit_top<T>(*reinterpret_cast<const uint4 *>(sb + L::v + vrow + 16 * i * L::kRow)));
      cut = __reduce_max_sync(0xffffffffu, top) >= 0x7f800000u;
      if (cut) {
        int first[2];
        cut_values<T, L::kRow>(smem + buf * L::stage + L::v, 2 * warp, static_cast<int>(fac.first), first);
        first0 = first[0];
        first1 = first[1];
      }
      if (dead0) first0 = 0;
      if (dead1) first1 = 0;
      dead0 = first0 < 64;
      dead1 = first1 < 64;
      cut = __any_sync(0xffffffffu, dead0 || dead1);
    }

    // X = S^T K^T and the output's S^T Q^T
    float X[8][4], Y[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) X[i][e] = Y[i][e] = 0.0f;
    float2 top = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) top = max_rows(S[nt], top);
    const float2 tops = quad_max(top);
    const RowPow2 ps = pow2_scale(tops);
    const float2 sunit = mul2(ps.inv, sinv), xinv = unit_or_zero(tops, sunit);
    // what the backward keeps of the state has one scale for the 16 channels
    float2 sf;
    if constexpr (KEEP) {
      const float all = warp_max(fmaxf(tops.x * sinv.x, tops.y * sinv.y));
      const Pow2 pss = store_scale(all);
      sf = mul2(splat(pss.s), xinv);
      if (lane == 0)
        p.w.slice[c * 32 + kSliceS + (dvw >> 4)] = cut ? __int_as_float(0x7fc00000) : slice_unit(all, pss);
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t hi[4], lo[4];
      split_rows(S[2 * ks], S[2 * ks + 1], ps.s, hi, lo);
      if constexpr (KEEP) {
        uint32_t x[4] = {hi[0], hi[1], hi[2], hi[3]};
        if (sf.x != 1.0f || sf.y != 1.0f) scale_h2(x, sf);
        store_block(p.w.s16 + c * (D * D) + dvw * D + 16 * ks, D, x, lane);
      }
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t bk[4], bq[4];
        ldsm4(bk, ofb.at(np, ks) + R::k);
        ldsm4(bq, ofb.at(np, ks) + R::q);
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
    // R = beta V^T - (beta e^G) X, in place of X
    top = make_float2(0.0f, 0.0f);
    const float2 xk = mul2(xinv, splat(-fac.k));
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t vv[4];
      ldsm4t(vv, st + L::v + vofs + 16 * np * L::kRow);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int nt = 2 * np + half;
        const float2 be = *reinterpret_cast<const float2 *>(tok + kTokBeta * 64 + 8 * nt);
        const float2 tx = *reinterpret_cast<const float2 *>(tok + kTokX * 64 + 8 * nt);
        const float2 r0 = fma2(mul2(tx, splat(xk.x)), row_lo(X[nt]), mul2(be, unpack_io<T>(vv[half])));
        const float2 r1 = fma2(mul2(tx, splat(xk.y)), row_hi(X[nt]), mul2(be, unpack_io<T>(vv[2 + half])));
        set_lo(X[nt], r0);
        set_hi(X[nt], r1);
        top = max_rows(X[nt], top);
      }
    }
    const RowPow2 pr = pow2_scale(quad_max(top));
    // U = R T^T: T_ij = 0 for j > i, in blocks of 16
    float U[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) U[i][e] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t hi[4], lo[4];
      split_rows(X[2 * kb], X[2 * kb + 1], pr.s, hi, lo);
      uint32_t bh[4][4], bl[4];
#pragma unroll
      for (int np = kb; np < 4; ++np) {
        ldsm4(bh[np], tri0 + tri(np, kb) + R::th);
        mma_f16(U[2 * np], hi, bh[np][0], bh[np][1]);
        mma_f16(U[2 * np + 1], hi, bh[np][2], bh[np][3]);
      }
#pragma unroll
      for (int np = kb; np < 4; ++np) {
        mma_f16(U[2 * np], lo, bh[np][0], bh[np][1]);
        mma_f16(U[2 * np + 1], lo, bh[np][2], bh[np][3]);
      }
#pragma unroll
      for (int np = kb; np < 4; ++np) {
        ldsm4(bl, tri0 + tri(np, kb) + R::tl);
        mma_f16(U[2 * np], hi, bl[0], bl[1]);
        mma_f16(U[2 * np + 1], hi, bl[2], bl[3]);
      }
    }
    // U itself, and U e^{G_last - G} into X
    const float2 uf = mul2(pr.inv, splat(fac.t));
    top = make_float2(0.0f, 0.0f);
    float2 topl = top;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      scale_rows(U[nt], uf);
      const float2 tl = *reinterpret_cast<const float2 *>(tok + kTokL * 64 + 8 * nt);
      top = max_rows(U[nt], top);
      set_lo(X[nt], mul2(row_lo(U[nt]), tl));
      set_hi(X[nt], mul2(row_hi(U[nt]), tl));
      topl = max_rows(X[nt], topl);
    }
    top = quad_max(top);
    const RowPow2 pu = pow2_scale(top);
    // S^T <- e^{G_last} S^T + X K in the scale that suits X
    const float2 asc = update_scale(mul2(quad_max(topl), splat(fac.k)), tops, sunit, fac.last);
    {
      const float2 sc = mul2(mul2(asc, splat(fac.last)), sinv);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) scale_rows(S[nt], sc);
      sinv = make_float2(pow2_inverse(asc.x), pow2_inverse(asc.y));
    }
    const float2 xs = mul2(asc, splat(fac.k));
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t hi[4], lo[4];
      split_rows(X[2 * kb], X[2 * kb + 1], xs, hi, lo);
      // two blocks at a time: an accumulator's second product comes four mma
      // (32 clocks) after its first, which takes 25
#pragma unroll
      for (int np = 0; np < D / 16; np += 2) {
        uint32_t b0[4], b1[4];
        ldsm4t(b0, ofd.at(kb, np) + R::k);
        ldsm4t(b1, ofd.at(kb, np + 1) + R::k);
        mma_f16(S[2 * np], hi, b0[0], b0[1]);
        mma_f16(S[2 * np + 1], hi, b0[2], b0[3]);
        mma_f16(S[2 * np + 2], hi, b1[0], b1[1]);
        mma_f16(S[2 * np + 3], hi, b1[2], b1[3]);
        mma_f16(S[2 * np], lo, b0[0], b0[1]);
        mma_f16(S[2 * np + 1], lo, b0[2], b0[3]);
        mma_f16(S[2 * np + 2], lo, b1[0], b1[1]);
        mma_f16(S[2 * np + 3], lo, b1[2], b1[3]);
      }
    }
    // Y = scale (e^G S^T Q^T + U P^T); the first product joins the second's
    // sum, in its unit zu (see kLeastShare)
    const OutputUnit ou0 = output_unit(xinv.x * fac.q, pu.inv.x, fac.p, fac.ps, p.least),
                     ou1 = output_unit(xinv.y * fac.q, pu.inv.y, fac.p, fac.ps, p.least);
    const float2 us = make_float2(ou0.us, ou1.us), yf = mul2(make_float2(ou0.unit, ou1.unit), splat(p.s.scale));
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      const float2 ty = *reinterpret_cast<const float2 *>(tok + kTokY * 64 + 8 * nt);
      set_lo(Y[nt], mul2(row_lo(Y[nt]), mul2(ty, splat(ou0.r))));
      set_hi(Y[nt], mul2(row_hi(Y[nt]), mul2(ty, splat(ou1.r))));
    }
    Pow2 pus;
    if constexpr (KEEP) {
      const float all = warp_max(fmaxf(top.x, top.y));
      pus = store_scale(all);
      if (lane == 0)
        p.w.slice[c * 32 + kSliceU + (dvw >> 4)] = cut ? __int_as_float(0x7fc00000) : slice_unit(all, pus);
    }
    uint32_t uh[4][4];
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t ul[4];
      if constexpr (kTwo) split_rows(U[2 * kb], U[2 * kb + 1], us, uh[kb], ul);
      else single_rows(U[2 * kb], U[2 * kb + 1], us, uh[kb]);
#pragma unroll
      for (int np = kb; np < 4; ++np) {
        uint32_t bp[4];
        ldsm4(bp, tri0 + tri(np, kb) + R::ph);
        mma_f16(Y[2 * np], uh[kb], bp[0], bp[1]);
        mma_f16(Y[2 * np + 1], uh[kb], bp[2], bp[3]);
        if constexpr (kTwo) {
          mma_f16(Y[2 * np], ul, bp[0], bp[1]);
          mma_f16(Y[2 * np + 1], ul, bp[2], bp[3]);
          ldsm4(bp, tri0 + tri(np, kb) + R::pl);
          mma_f16(Y[2 * np], uh[kb], bp[0], bp[1]);
          mma_f16(Y[2 * np + 1], uh[kb], bp[2], bp[3]);
        }
      }
    }
    // Transpose through this warp's own columns of the value tile (read above) and store rows of 32 bytes.
    const int len = min(kChunk, p.s.T - n * kChunk);
    const uint32_t vw = st + L::v + vofs;
    const unsigned char *vr = sb + L::v + vrow;
    __syncwarp();
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      const float2 a = mul2(row_lo(Y[2 * np]), splat(yf.x)), bb = mul2(row_lo(Y[2 * np + 1]), splat(yf.x));
      const float2 cc = mul2(row_hi(Y[2 * np]), splat(yf.y)), d = mul2(row_hi(Y[2 * np + 1]), splat(yf.y));
      const uint32_t o[4] = {pack_io<T>(a.x, a.y), pack_io<T>(bb.x, bb.y), pack_io<T>(cc.x, cc.y), pack_io<T>(d.x, d.y)};
      stsm4t(vw + 16 * np * L::kRow, o);
    }
    __syncwarp();
    if (cut) poison_rows<T, L::kRow>(smem + buf * L::stage + L::v, 2 * warp, first0, first1);
    T *yr = y + (row0 + n * kChunk + (lane >> 1)) * ldy;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (16 * i + (lane >> 1) < len)
        *reinterpret_cast<uint4 *>(yr + 16 * i * ldy) = *reinterpret_cast<const uint4 *>(vr + 16 * i * L::kRow);
    if constexpr (KEEP) {
      __syncwarp();
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (pus.s != us.x || pus.s != us.y) single_rows(U[2 * kb], U[2 * kb + 1], splat(pus.s), uh[kb]);
        const uint32_t o[4] = {uh[kb][0], uh[kb][2], uh[kb][1], uh[kb][3]};
        stsm4t(vw + 16 * kb * L::kRow, o);
      }
      __syncwarp();
      const long long ur = (c * 64 + (lane >> 1)) * D + dvw + 8 * (lane & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(p.w.u16 + ur + 16 * i * D) = *reinterpret_cast<const uint4 *>(vr + 16 * i * L::kRow);
      if constexpr (kTwo) {   // and the second term
        __syncwarp();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          uint32_t hi[4], lo[4];
          split_rows(U[2 * kb], U[2 * kb + 1], splat(pus.s), hi, lo);
          const uint32_t o[4] = {lo[0], lo[2], lo[1], lo[3]};
          stsm4t(vw + 16 * kb * L::kRow, o);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4 *>(p.w.u16l + ur + 16 * i * D) = *reinterpret_cast<const uint4 *>(vr + 16 * i * L::kRow);
      }
    }
    __syncthreads();   // the next turn's copies overwrite this buffer
  }
  if (p.S_out != nullptr) {
    float *So = p.S_out + static_cast<long long>(head) * D * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) 
        So[(8 * nt + 2 * t4 + (e & 1)) * D + dvw + g + (e >> 1) * 8] =
            (e < 2 ? dead0 : dead1) ? __int_as_float(0x7fc00000) : S[nt][e] * (e < 2 ? sinv.x : sinv.y);
  }
}

template <typename T, int D, int W, bool KEEP>
int run(const ChunkArgs &a, cudaStream_t st) {
  using L = ChainSmem<D, W, std::is_same<T, __half>::value>;
  auto kern = delta_chain_fwd_kernel<T, D, W, KEEP>;
  const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total));
  if (rc) return rc;
  kern<<<static_cast<unsigned>(a.s.B) * a.s.H * (D / (16 * W)), W * 32, L::total, st>>>(a);
  return runtime_status(cudaGetLastError());
}

template <typename T, int D, int W>
int by_keep(const ChunkArgs &a, cudaStream_t st) {
  return a.keep ? run<T, D, W, true>(a, st) : run<T, D, W, false>(a, st);
}

template <typename T, int D>
int by_warps(const ChunkArgs &a, cudaStream_t st) {
  if constexpr (D == 128)
    if (chain_plan(a.s.B * a.s.H, D) == kChainHalves) return by_keep<T, D, 4>(a, st);
  return by_keep<T, D, D / 16>(a, st);
}

template <typename T>
int by_d(const ChunkArgs &a, cudaStream_t st) {
  switch (a.s.D) {
    case 32: return by_warps<T, 32>(a, st);
    case 64: return by_warps<T, 64>(a, st);
    case 128: return by_warps<T, 128>(a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace

// Four warps a slice while every slice's block has an SM to itself; else whole
// heads, of which a block takes eight warps at D = 128 once four warps a block
// would put more than one block on an SM (32 chunks with what the backward
// reads, in halves and whole: 16 heads 157 and 221 us, backward 155 and 248; 128
// heads 236 and 232, 311 and 252).
ChainPlan chain_plan(int heads, int D) {
  if (D >= 64 && static_cast<long long>(heads) * (D / 16) <= sm_count()) return kChainSplit;
  return D == 128 && 2ll * heads <= sm_count() ? kChainHalves : kChainWhole;
}

int launch_chunk_fwd(int dtype, const ChunkArgs &a, cudaStream_t st) {
  if (chain_plan(a.s.B * a.s.H, a.s.D) == kChainSplit) return launch_split_fwd(dtype, a, st);
  return dtype == ESA_F16 ? by_d<__half>(a, st) : by_d<__nv_bfloat16>(a, st);
}

}  // namespace esa
