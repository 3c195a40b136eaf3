// esa_delta_chain_bwd.cu -- the backward of the chunked gated delta rule, first
// kernel: the gradient of the state carried from the last chunk to the first
// (sm_100a).
//
// As in the forward chain (esa_delta_chain.cu) a warp carries 16 value
// channels, here of dS^T, in its registers.  For a chunk, with dS the gradient
// of the state leaving it and P, T as in the first kernel,
//   dU^T = e^{G_last - G} (dS^T K^T) + scale dO^T P,
//   du^T = dU^T T                                  (the gradient of u: T^T is applied to dU),
//   dS^T <- e^{G_last} dS^T - (beta e^G du^T) K + scale (e^G dO^T) Q,
// and dv = beta du.  What enters dS keeps float32 accuracy (two float16 terms,
// K, Q and dO exact), because dS_init is float32.  dS and du are left for the
// second kernel (esa_delta_grad.cu) in float16, one power of two per 16
// channels; du of float16 tensors in two terms.
//
// A key or query that is not finite makes du of its chunk NaN, and with it all
// that the chunk adds to dS.
//
// 484 mma a chunk and warp at D = 128, bound as the forward chain is.
#include <type_traits>

#include "esa_delta_chunk.h"
#include "esa_delta_sweep.cuh"
#include "esa_mma.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

template <int D, int W>
struct ChainBwdSmem {
  using R = ChunkRecord<D>;
  static constexpr int kRow = 32 * W;
  static constexpr int dy = R::bytes, stage = dy + 64 * kRow, total = 2 * stage;
};

template <typename T, int D, int W>
__global__ void __launch_bounds__(W * 32, 1) delta_chain_bwd_kernel(ChunkArgs p) {
  using L = ChainBwdSmem<D, W>;
  using R = ChunkRecord<D>;
  constexpr int NT = D / 8;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  constexpr int SL = D / (16 * W);
  const int head = blockIdx.x / SL, slice = blockIdx.x - head * SL;
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int dv0 = slice * 16 * W, dvw = dv0 + 16 * warp;
  const int nc = p.w.nc;
  const long long c0 = static_cast<long long>(head) * nc;
  const long long row0 = static_cast<long long>(b) * p.s.T;
  const long long ldc = static_cast<long long>(p.s.H) * D;
  const T *dy = static_cast<const T *>(p.dy) + h * D + dv0;
  T *dv = static_cast<T *>(p.dv) + h * D + dvw + 8 * (lane & 1);
  const uint32_t s0 = smem_u32(smem);
  const uint32_t vofs = tile_off<L::kRow>(lane & 15, 2 * warp + (lane >> 4));
  const uint32_t vrow = tile_off<L::kRow>(lane >> 1, 2 * warp + (lane & 1));

  auto fetch = [&](int n, int buf) {
    const uint32_t s = s0 + buf * L::stage;
    copy_linear<R::bytes, W * 32>(s, p.w.rec + (c0 + n) * R::bytes);
    const int len = min(kChunk, p.s.T - n * kChunk);
    const T *src = dy + (row0 + n * kChunk) * ldc;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = threadIdx.x + i * W * 32, r = e / (2 * W), u = e % (2 * W);
      const bool on = r < len;
      cp_async16_zfill(s + L::dy + tile_off<L::kRow>(r, u), on ? src + r * ldc + u * 8 : dy, on);
    }
    sweep::cp_async_commit();
  };

  float S[NT][4];   // dS^T, each row over its sinv
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

  fetch(nc - 1, 0);
#pragma unroll 1
  for (int it = 0; it < nc; ++it) {
    const int n = nc - 1 - it, buf = it & 1;
    if (n > 0) {
      fetch(n - 1, buf ^ 1);
      sweep::cp_async_wait<1>();
    } else {
      sweep::cp_async_wait<0>();
    }
    __syncthreads();
    const uint32_t st = s0 + buf * L::stage;
    const LaneOff<D * 2> ofd(lane, st);
    const LaneOffB<D * 2> ofb(lane, st);
    const uint32_t tri0 = LaneOff<32>(lane, st).o[0];   // blocks of T and P
    const unsigned char *sb = smem + buf * L::stage;
    const float *tok = reinterpret_cast<const float *>(sb + R::tok) + 2 * t4;
    const Fac fac = load_fac(sb + R::fac);
    const long long c = c0 + n;

    // X = dS^T K^T
    float X[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) X[i][e] = 0.0f;
    float2 top = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) top = max_rows(S[nt], top);
    const float2 tops = quad_max(top);
    const RowPow2 ps = pow2_scale(tops);
    const float2 sunit = mul2(ps.inv, sinv), xinv = unit_or_zero(tops, sunit);
    const float alls = warp_max(fmaxf(tops.x * sinv.x, tops.y * sinv.y));
    const Pow2 pss = store_scale(alls);
    const float2 sf = mul2(splat(pss.s), xinv);
    if (lane == 0) p.w.slice[c * 32 + kSliceDs + (dvw >> 4)] = slice_unit(alls, pss);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t hi[4], lo[4];
      split_rows(S[2 * ks], S[2 * ks + 1], ps.s, hi, lo);
      uint32_t x[4] = {hi[0], hi[1], hi[2], hi[3]};
      if (sf.x != 1.0f || sf.y != 1.0f) scale_h2(x, sf);
      store_block(p.w.ds16 + c * (D * D) + dvw * D + 16 * ks, D, x, lane);
#pragma unroll
      for (int np = 0; np < 4; np += 2) {   // an accumulator's second product four mma after its first
        uint32_t b0[4], b1[4];
        ldsm4(b0, ofb.at(np, ks) + R::k);
        ldsm4(b1, ofb.at(np + 1, ks) + R::k);
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
    // dO^T as an A operand, scaled to float16
    uint32_t od[4][4];   // registers 0 and 2 of a block are row g
    top = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t r[4];
      ldsm4t(r, st + L::dy + vofs + 16 * kb * L::kRow);
      od[kb][0] = r[0]; od[kb][1] = r[2]; od[kb][2] = r[1]; od[kb][3] = r[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = unpack_io<T>(od[kb][e]);
        float &t = e & 1 ? top.y : top.x;
        t = fmaxf(t, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
    }
    // dU^T = zf (X r + dO^T P) (see kLeastShare); without an output gradient's share (scale 0) P is left out
    const bool with = p.s.scale != 0.0f;
    const float2 xk = mul2(xinv, splat(fac.k));
    const RowPow2 pd = pow2_scale(quad_max(top)), pz = with ? least_unit(pd, xk, fabsf(p.iscale), fac.ps) : pd;
    const float2 low = mul2(pd.inv, pz.s);   // what the product with P takes of dO: 1 unless its unit is too small
    const float2 zf = with ? make_float2(mul_pow2(p.s.scale, fac.p, pz.inv.x), mul_pow2(p.s.scale, fac.p, pz.inv.y)) : splat(1.0f);
    const float2 yd = mul2(pd.inv, splat(p.s.scale));
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) od[kb][e] = pack2(mul2(unpack_io<T>(od[kb][e]), splat(e & 1 ? pd.s.y : pd.s.x)));
    {
      // xk / zf; 1 / zf is at most 2^120
      const float2 r = with ? mul2(xk, make_float2(mul_pow2(p.iscale, pz.s.x, fac.ps), mul_pow2(p.iscale, pz.s.y, fac.ps))) : xk;
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const float2 tl = *reinterpret_cast<const float2 *>(tok + kTokL * 64 + 8 * nt);
        set_lo(X[nt], mul2(row_lo(X[nt]), mul2(tl, splat(r.x))));
        set_hi(X[nt], mul2(row_hi(X[nt]), mul2(tl, splat(r.y))));
      }
    }
    if (with) {
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        uint32_t o[4] = {od[kb][0], od[kb][1], od[kb][2], od[kb][3]};
        if (low.x != 1.0f || low.y != 1.0f) scale_h2(o, low);
#pragma unroll
        for (int np = 0; np <= kb; ++np) {
          uint32_t bh[4];
          ldsm4t(bh, tri0 + tri(kb, np) + R::ph);
          mma_f16(X[2 * np], o, bh[0], bh[1]);
          mma_f16(X[2 * np + 1], o, bh[2], bh[3]);
        }
#pragma unroll
        for (int np = 0; np <= kb; ++np) {
          uint32_t bl[4];
          ldsm4t(bl, tri0 + tri(kb, np) + R::pl);
          mma_f16(X[2 * np], o, bl[0], bl[1]);
          mma_f16(X[2 * np + 1], o, bl[2], bl[3]);
        }
      }
    }
    // du^T = dU^T T
    top = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) top = max_rows(X[nt], top);
    const RowPow2 pr = pow2_scale(quad_max(top));
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
      for (int np = 0; np <= kb; ++np) {
        ldsm4t(bh[np], tri0 + tri(kb, np) + R::th);
        mma_f16(U[2 * np], hi, bh[np][0], bh[np][1]);
        mma_f16(U[2 * np + 1], hi, bh[np][2], bh[np][3]);
      }
#pragma unroll
      for (int np = 0; np <= kb; ++np) {
        mma_f16(U[2 * np], lo, bh[np][0], bh[np][1]);
        mma_f16(U[2 * np + 1], lo, bh[np][2], bh[np][3]);
      }
#pragma unroll
      for (int np = 0; np <= kb; ++np) {
        ldsm4t(bl, tri0 + tri(kb, np) + R::tl);
        mma_f16(U[2 * np], hi, bl[0], bl[1]);
        mma_f16(U[2 * np + 1], hi, bl[2], bl[3]);
      }
    }
    // du itself, -beta e^G du into X; the largest of that and of scale e^G dO
    const float2 rf = mul2(mul2(pr.inv, zf), splat(fac.tb));
    top = make_float2(0.0f, 0.0f);
    float2 topx = top, topo = top;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      scale_rows(U[nt], rf);
      const float2 tx = mul2(*reinterpret_cast<const float2 *>(tok + kTokX * 64 + 8 * nt), splat(-1.0f));
      top = max_rows(U[nt], top);
      set_lo(X[nt], mul2(row_lo(U[nt]), tx));
      set_hi(X[nt], mul2(row_hi(U[nt]), tx));
      topx = max_rows(X[nt], topx);
    }
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = mul2(unpack_h2(od[kb][e]), mul2(*reinterpret_cast<const float2 *>(tok + kTokY * 64 + 16 * kb + 8 * (e >> 1)), splat(e & 1 ? yd.y : yd.x)));
        float &t = e & 1 ? topo.y : topo.x;
        t = fmaxf(t, fmaxf(fabsf(x.x), fabsf(x.y)));
      }
    const float allu = warp_max(fmaxf(top.x, top.y));
    const Pow2 pus = store_scale(allu);
    const float2 upd = make_float2(fmaxf(topx.x * fac.k, topo.x * fac.q), fmaxf(topx.y * fac.k, topo.y * fac.q));
    const float2 asc = update_scale(quad_max(upd), tops, sunit, fac.last);
    const float2 xs = mul2(asc, splat(fac.k)), os = mul2(yd, mul2(asc, splat(fac.q)));
    {
      const float2 sc = mul2(mul2(asc, splat(fac.last)), sinv);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) scale_rows(S[nt], sc);
      sinv = make_float2(pow2_inverse(asc.x), pow2_inverse(asc.y));
    }
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      uint32_t hi[4], lo[4], qh[4], ql[4];
      split_rows(X[2 * kb], X[2 * kb + 1], xs, hi, lo);
      const float2 y0 = *reinterpret_cast<const float2 *>(tok + kTokY * 64 + 16 * kb);
      const float2 y1 = *reinterpret_cast<const float2 *>(tok + kTokY * 64 + 16 * kb + 8);
      split2(mul2(unpack_h2(od[kb][0]), mul2(y0, splat(os.x))), qh[0], ql[0]);
      split2(mul2(unpack_h2(od[kb][1]), mul2(y0, splat(os.y))), qh[1], ql[1]);
      split2(mul2(unpack_h2(od[kb][2]), mul2(y1, splat(os.x))), qh[2], ql[2]);
      split2(mul2(unpack_h2(od[kb][3]), mul2(y1, splat(os.y))), qh[3], ql[3]);
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
        ldsm4t(b0, ofd.at(kb, np) + R::q);
        ldsm4t(b1, ofd.at(kb, np + 1) + R::q);
        mma_f16(S[2 * np], qh, b0[0], b0[1]);
        mma_f16(S[2 * np + 1], qh, b0[2], b0[3]);
        mma_f16(S[2 * np + 2], qh, b1[0], b1[1]);
        mma_f16(S[2 * np + 3], qh, b1[2], b1[3]);
        mma_f16(S[2 * np], ql, b0[0], b0[1]);
        mma_f16(S[2 * np + 1], ql, b0[2], b0[3]);
        mma_f16(S[2 * np + 2], ql, b1[0], b1[1]);
        mma_f16(S[2 * np + 3], ql, b1[2], b1[3]);
      }
    }
    // dv = beta du, and du itself, through this warp's own columns of the dy tile
    const int len = min(kChunk, p.s.T - n * kChunk);
    const uint32_t vw = st + L::dy + vofs;
    const unsigned char *vr = sb + L::dy + vrow;
    __syncwarp();
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      const float2 b0 = *reinterpret_cast<const float2 *>(tok + kTokBeta * 64 + 16 * np);
      const float2 b1 = *reinterpret_cast<const float2 *>(tok + kTokBeta * 64 + 16 * np + 8);
      const float2 a = mul2(row_lo(U[2 * np]), b0), bb = mul2(row_lo(U[2 * np + 1]), b1);
      const float2 cc = mul2(row_hi(U[2 * np]), b0), d = mul2(row_hi(U[2 * np + 1]), b1);
      const uint32_t o[4] = {pack_io<T>(a.x, a.y), pack_io<T>(bb.x, bb.y), pack_io<T>(cc.x, cc.y), pack_io<T>(d.x, d.y)};
      stsm4t(vw + 16 * np * L::kRow, o);
    }
    __syncwarp();
    T *dr = dv + (row0 + n * kChunk + (lane >> 1)) * ldc;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (16 * i + (lane >> 1) < len)
        *reinterpret_cast<uint4 *>(dr + 16 * i * ldc) = *reinterpret_cast<const uint4 *>(vr + 16 * i * L::kRow);
    __syncwarp();
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t r[4];
      single_rows(U[2 * np], U[2 * np + 1], splat(pus.s), r);
      const uint32_t o[4] = {r[0], r[2], r[1], r[3]};
      stsm4t(vw + 16 * np * L::kRow, o);
    }
    __syncwarp();
    const long long ur = (c * 64 + (lane >> 1)) * D + dvw + 8 * (lane & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4 *>(p.w.r16 + ur + 16 * i * D) = *reinterpret_cast<const uint4 *>(vr + 16 * i * L::kRow);
    if constexpr (std::is_same<T, __half>::value) {   // and the second term
      __syncwarp();
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t hi[4], lo[4];
        split_rows(U[2 * np], U[2 * np + 1], splat(pus.s), hi, lo);
        const uint32_t o[4] = {lo[0], lo[2], lo[1], lo[3]};
        stsm4t(vw + 16 * np * L::kRow, o);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(p.w.r16l + ur + 16 * i * D) = *reinterpret_cast<const uint4 *>(vr + 16 * i * L::kRow);
    }
    if (lane == 0) p.w.slice[c * 32 + kSliceR + (dvw >> 4)] = slice_unit(allu, pus);
    __syncthreads();
  }
  if (p.S_out != nullptr) {
    float *So = p.S_out + static_cast<long long>(head) * D * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) So[(8 * nt + 2 * t4 + (e & 1)) * D + dvw + g + (e >> 1) * 8] = S[nt][e] * (e < 2 ? sinv.x : sinv.y);
  }
}

template <typename T, int D, int W>
int run(const ChunkArgs &a, cudaStream_t st) {
  using L = ChainBwdSmem<D, W>;
  auto kern = delta_chain_bwd_kernel<T, D, W>;
  const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total));
  if (rc) return rc;
  kern<<<static_cast<unsigned>(a.s.B) * a.s.H * (D / (16 * W)), W * 32, L::total, st>>>(a);
  return runtime_status(cudaGetLastError());
}

template <typename T>
int by_d(const ChunkArgs &a, cudaStream_t st) {
  switch (a.s.D) {
    case 32: return run<T, 32, 2>(a, st);
    case 64: return run<T, 64, 4>(a, st);
    case 128: return chain_plan(a.s.B * a.s.H, 128) == kChainHalves ? run<T, 128, 4>(a, st) : run<T, 128, 8>(a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace

int launch_chunk_bwd(int dtype, const ChunkArgs &a, cudaStream_t st) {
  if (chain_plan(a.s.B * a.s.H, a.s.D) == kChainSplit) return launch_split_bwd(dtype, a, st);
  return dtype == ESA_F16 ? by_d<__half>(a, st) : by_d<__nv_bfloat16>(a, st);
}

}  // namespace esa
