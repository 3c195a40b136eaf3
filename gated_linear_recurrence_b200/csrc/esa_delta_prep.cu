// esa_delta_prep.cu -- first kernel of the chunked gated delta rule: what each
// chunk of 64 tokens needs and no other chunk changes (sm_100a).
//
// With G_i the running sum of log alpha in the chunk, the recurrence over its
// tokens is the triangular system
//   (1 + M) U = beta (V - e^G K S),   M_ij = beta_i e^{Gi - Gj} k_i.k_j  (j < i),
// where S is the state entering the chunk.  This kernel forms M from K K^T and
// P_ij = e^{Gi - Gj} q_i.k_j (j <= i) from Q K^T on the tensor cores, and
// T = (1 + M)^-1 in blocks of 16: the diagonal blocks D_i by substitution in
// float32 (one column a thread), the blocks below by
//   T_ij = -D_i sum_{j <= l < i} M_il T_lj,
// a block column a warp, on the tensor cores with two float16 terms per
// operand (22 bits).  A warp works on the transposes, so that each block it
// has formed is, as it lies in its registers, the next product's A operand:
// a column takes no barrier.  (In float32 multiply-adds with barriers between
// the block levels this kernel took 182 us instead of 124 at 4096 chunks of
// D = 128.)
//
// G is kept in two float32 terms: its differences are exponentiated, and a
// token that forgets everything (G falls by 80) must not cost its successors
// their digits.  A gate that is NaN is treated as a key that is not finite: the
// head is NaN from its token on.  Below the diagonal blocks e^{Gi - Gj} is e^{Gi - Gr} e^{Gr - Gj}
// with r the row block's first token: two factors of at most 1, one
// exponential per row and one per column instead of one per element.
//
// Keys and queries are brought to float16 with one power of two per tile
// (exact for bfloat16 and float16 elements down to 2^-19 of the tile's
// largest, then off by at most 2^-30 of it), so that bfloat16 tensors take the
// same products as float16 ones and the split terms keep 22 bits.
//
// The record (esa_delta_chunk.h) is put together in shared memory and leaves
// in one bulk copy.
#include <type_traits>

#include "esa_delta_chunk.h"
#include "esa_delta_sweep.cuh"
#include "esa_mma.cuh"
#include "esa_umma.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

constexpr int kThreads = 256;
constexpr int kDiag = 16 * 20;   // floats of a 16 x 16 block, rows of 20 (float4 rows, spread over the banks)
constexpr unsigned kInf = 0x7f800000u;
static_assert(kTriangle == kTriBytes, "one layout of a triangle");

template <int D>
struct PrepSmem {
  using R = ChunkRecord<D>;
  static constexpr int mh = R::th, ml = R::tl;                  // M's terms, until T's take their place
  static constexpr int md = (R::bytes + 127) / 128 * 128;       // M's diagonal blocks, float32
  static constexpr int dd = md + 4 * kDiag * 4;                 // their inverses D, float32
  static constexpr int dh = dd + 4 * kDiag * 4, dl = dh + 2048; // and in two terms
  static constexpr int vec = dl + 2048, red = vec + (2 + 8) * 64 * 4, total = red + 160;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(ChunkArgs p) {
  using L = PrepSmem<D>;
  using R = ChunkRecord<D>;
  constexpr int LPR = D / 8, RPI = 32 / LPR, NV = 16 / RPI;   // lanes of a row, rows of a load, loads of a warp's 16 rows
  extern __shared__ __align__(128) unsigned char smem[];
  float *Md = reinterpret_cast<float *>(smem + L::md), *Dd = reinterpret_cast<float *>(smem + L::dd);
  float *vec = reinterpret_cast<float *>(smem + L::vec), *red = reinterpret_cast<float *>(smem + L::red);
  uint32_t *redu = reinterpret_cast<uint32_t *>(red);
  // bad: tokens whose key (1), query (2) or gate (4) is not finite
  float *beta = vec, *bad = vec + 64;
  float *G = reinterpret_cast<float *>(smem + R::g), *Gl = G + 64;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int mw = warp & 3;
  const long long c = blockIdx.x;
  const int head = static_cast<int>(c / p.w.nc), n = static_cast<int>(c - static_cast<long long>(head) * p.w.nc);
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int t0 = n * kChunk, len = min(kChunk, p.s.T - t0);
  const long long row = static_cast<long long>(b) * p.s.T + t0;

  // K rows (warps 0-3) and Q rows (warps 4-7), 16 a warp
  uint4 raw[NV];
  const int sub = lane % LPR, r0 = 16 * mw + lane / LPR;
  {
    const T *src = static_cast<const T *>(warp < 4 ? p.k : p.q) + (row + r0) * p.s.ld_qk + h * D + sub * 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (r0 + i * RPI < len) raw[i] = *reinterpret_cast<const uint4 *>(src + i * RPI * p.s.ld_qk);
    }
  }
  if (warp == 0) {   // gates and their running sum, two tokens a lane
    const T *ga = static_cast<const T *>(p.a), *gb = static_cast<const T *>(p.b);
    float la[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      float be = 0.0f, lost = 0.0f;
      if (i < len) {
        const float xa = sweep::widen(ga[(row + i) * p.s.ld_g + h]), xb = sweep::widen(gb[(row + i) * p.s.ld_g + h]);
        if (xa == xa && xb == xb) {
          la[e] = -log1pf(expf(-sweep::clamp(xa)));
          be = sweep::gate(xb);
        } else {
          lost = 4.0f;
        }
      }
      beta[i] = be;
      bad[i] = lost;
    }
    double x = static_cast<double>(la[0]) + la[1];
    const double own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const double first = x - own + la[0];
    const float f0 = static_cast<float>(first), f1 = static_cast<float>(x);
    *reinterpret_cast<float2 *>(G + 2 * lane) = make_float2(f0, f1);
    *reinterpret_cast<float2 *>(Gl + 2 * lane) = make_float2(static_cast<float>(first - f0), static_cast<float>(x - f1));
  }
  {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) top = max(top, unit_top<T>(raw[i]));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) redu[warp] = top;
  }
  __syncthreads();
  uint32_t topk = max(max(redu[0], redu[1]), max(redu[2], redu[3])), topq = max(max(redu[4], redu[5]), max(redu[6], redu[7]));
  if (max(topk, topq) >= kInf) {   // rows that are not finite become zero and are marked
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t bits = unit_top<T>(raw[i]);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
      if (bits >= kInf) {
        raw[i] = make_uint4(0, 0, 0, 0);
        if (sub == 0) atomicAdd(bad + r0 + i * RPI, warp < 4 ? 1.0f : 2.0f);
      } else {
        top = max(top, bits);
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if (lane == 0) redu[warp] = top;
    __syncthreads();
    topk = max(max(redu[0], redu[1]), max(redu[2], redu[3]));
    topq = max(max(redu[4], redu[5]), max(redu[6], redu[7]));
  }
  const Pow2 sk = pow2_scale(__uint_as_float(topk)), sq = pow2_scale(__uint_as_float(topq));
  {
    unsigned char *tile = smem + (warp < 4 ? R::k : R::q) + tile_off<D * 2>(r0, sub);
    const float2 s = splat(warp < 4 ? sk.s : sq.s);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t *w = reinterpret_cast<uint32_t *>(&raw[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack2(mul2(unpack_io<T>(w[j]), s));
      if constexpr (RPI == 8) *reinterpret_cast<uint4 *>(tile + i * RPI * D * 2) = raw[i];
      else *reinterpret_cast<uint4 *>(smem + (warp < 4 ? R::k : R::q) + tile_off<D * 2>(r0 + i * RPI, sub)) = raw[i];
    }
  }
  __syncthreads();
  if (tid < 64) {
    const int i = tid, flag = static_cast<int>(bad[i]);
    const float into = expf(G[i] + Gl[i]), out = expf((G[63] - G[i]) + (Gl[63] - Gl[i]));
    const float nan = __int_as_float(0x7fc00000), be = beta[i];
    float *tok = reinterpret_cast<float *>(smem + R::tok);
    tok[kTokBeta * 64 + i] = flag & 5 ? 0.0f : be;
    tok[kTokX * 64 + i] = flag & 5 ? 0.0f : be * into;
    tok[kTokL * 64 + i] = flag & 5 ? 0.0f : out;
    tok[kTokY * 64 + i] = flag & 2 ? nan : into;
  }
  // K K^T (warps 0-3) and Q K^T (warps 4-7): 16 rows a warp, tiles on and below the diagonal
  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  {
    const LaneOff<D * 2> off(lane, smem_u32(smem + R::k));
    const LaneOffB<D * 2> ofb(lane, smem_u32(smem + R::k));
    const uint32_t ao = (warp < 4 ? 0 : R::q - R::k) + 16 * mw * D * 2;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      ldsm4(a, off.at(0, ks) + ao);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if (np > mw) continue;
        uint32_t bk[4];
        ldsm4(bk, ofb.at(np, ks));
        mma_f16(acc[2 * np], a, bk[0], bk[1]);
        mma_f16(acc[2 * np + 1], a, bk[2], bk[3]);
      }
    }
  }
  float top = 0.0f;
  {
    const int r = 16 * mw, i0 = r + g;
    const float gr = G[r], grl = Gl[r];
    float *cf = vec + 128 + 64 * warp;   // this warp's column factors
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = lane + 32 * e;
      if (j < r) cf[j] = expf((gr - G[j]) + (grl - Gl[j]));
    }
    const float f = sk.inv * (warp < 4 ? sk.inv : sq.inv);
    float fr[2], gi[2], gli[2], fe[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      fr[e] = warp < 4 ? f * beta[i0 + 8 * e] : f;
      gi[e] = G[i0 + 8 * e];
      gli[e] = Gl[i0 + 8 * e];
      fe[e] = fr[e] * expf((gi[e] - gr) + (gli[e] - grl));
    }
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt > 2 * mw + 1) continue;
      if (nt < 2 * mw) {
        const float2 c2 = *reinterpret_cast<const float2 *>(cf + 8 * nt + 2 * t4);
        set_lo(acc[nt], mul2(row_lo(acc[nt]), mul2(c2, splat(fe[0]))));
        set_hi(acc[nt], mul2(row_hi(acc[nt]), mul2(c2, splat(fe[1]))));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + (e >> 1) * 8, j = 8 * nt + 2 * t4 + (e & 1);
          float x = 0.0f;
          if (j < i || (j == i && warp >= 4))
            x = expf((gi[e >> 1] - G[j]) + (gli[e >> 1] - Gl[j])) * fr[e >> 1] * acc[nt][e];
          acc[nt][e] = x;
        }
        if (warp < 4) {
          float *o = Md + mw * kDiag + 8 * (nt & 1) + 2 * t4;
          *reinterpret_cast<float2 *>(o + g * 20) = row_lo(acc[nt]);
          *reinterpret_cast<float2 *>(o + (g + 8) * 20) = row_hi(acc[nt]);
        }
      }
      top = max_tile(acc[nt], top);
    }
  }
  top = warp_max(top);
  if (lane == 0) red[8 + warp] = top;
  __syncthreads();
  const Pow2 sm = pow2_scale(fmaxf(fmaxf(red[8], red[9]), fmaxf(red[10], red[11])));
  const Pow2 sp = pow2_scale(fmaxf(fmaxf(red[12], red[13]), fmaxf(red[14], red[15])));
  {   // P with its diagonal blocks, M without
    const float2 s = splat(warp < 4 ? sm.s : sp.s);
    unsigned char *th = smem + (warp < 4 ? L::mh : R::ph), *tl = smem + (warp < 4 ? L::ml : R::pl);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      if (nt > 2 * mw + 1 || (warp < 4 && nt >= 2 * mw)) continue;
      const uint32_t o = tri(mw, nt >> 1) + tile_off<32>(g, nt & 1) + 4 * t4;   // rows g and g + 8: the same swizzle
      uint32_t hi, lo;
      split2(mul2(row_lo(acc[nt]), s), hi, lo);
      *reinterpret_cast<uint32_t *>(th + o) = hi;
      *reinterpret_cast<uint32_t *>(tl + o) = lo;
      split2(mul2(row_hi(acc[nt]), s), hi, lo);
      *reinterpret_cast<uint32_t *>(th + o + 256) = hi;
      *reinterpret_cast<uint32_t *>(tl + o + 256) = lo;
    }
  }
  if (warp < 2) {   // D_blk: column `col` a thread
    const int blk = tid >> 4, col = tid & 15;
    const float *Mb = Md + blk * kDiag;
    float *Db = Dd + blk * kDiag;
    float x[16], dt = 1.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(Mb + i * 20 + l);
        s[0] = fmaf(m.x, x[l], s[0]);
        if (l + 1 < i) s[1] = fmaf(m.y, x[l + 1], s[1]);
        if (l + 2 < i) s[2] = fmaf(m.z, x[l + 2], s[2]);
        if (l + 3 < i) s[3] = fmaf(m.w, x[l + 3], s[3]);
      }
      const float sum = (s[0] + s[1]) + (s[2] + s[3]);
      x[i] = i == col ? 1.0f : (i > col ? -sum : 0.0f);
      dt = fmaxf(dt, fabsf(x[i]));
      Db[i * 20 + col] = x[i];
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) dt = fmaxf(dt, __shfl_xor_sync(0xffffffffu, dt, o));
    if (col == 0) red[16 + blk] = dt;
    const Pow2 sd = pow2_scale(dt);
    __half *dh = reinterpret_cast<__half *>(smem + L::dh + blk * 512), *dl = reinterpret_cast<__half *>(smem + L::dl + blk * 512);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t o = tile_off<32>(i, col >> 3) / 2 + (col & 7);
      const float v = x[i] * sd.s;
      const __half hi = __float2half_rn(v);
      dh[o] = hi;
      dl[o] = __float2half_rn(v - __half2float(hi));
    }
  }
  __syncthreads();
  // Block column j = warp of T, blocks (i, j) with i > j, as transposes
  float Tt[3][2][4];
  float tt = 0.0f;
  if (warp < 3) {
    const uint32_t trib = LaneOffB<32>(lane, smem_u32(smem)).o[0];
    float Dj[2][4];
    {
      const float *o = Dd + warp * kDiag;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 8 * e + 2 * t4;   // row of D, column of the transpose
        Dj[e][0] = o[i * 20 + g];
        Dj[e][1] = o[(i + 1) * 20 + g];
        Dj[e][2] = o[i * 20 + g + 8];
        Dj[e][3] = o[(i + 1) * 20 + g + 8];
      }
    }
    float run = red[16 + warp];   // largest entry of the column so far
#pragma unroll
    for (int d = 0; d < 3; ++d) {   // i = warp + 1 + d
      const int i = warp + 1 + d;
      if (i > 3) continue;
      float Z[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) Z[0][e] = Z[1][e] = 0.0f;
      const Pow2 st = pow2_scale(run);
#pragma unroll
      for (int l = 0; l <= d; ++l) {   // block row warp + l
        uint32_t hi[4], lo[4], bh[4], bl[4];
        if (l == 0) split_a(Dj[0], Dj[1], splat(st.s), splat(st.s), hi, lo);
        else split_a(Tt[l > 0 ? l - 1 : 0][0], Tt[l > 0 ? l - 1 : 0][1], splat(st.s), splat(st.s), hi, lo);
        const uint32_t at = trib + (i * (i + 1) / 2 + warp + l) * 512;
        ldsm4(bh, at + L::mh);
        ldsm4(bl, at + L::ml);
        mma_f16(Z[0], hi, bh[0], bh[1]);
        mma_f16(Z[1], hi, bh[2], bh[3]);
        mma_f16(Z[0], lo, bh[0], bh[1]);
        mma_f16(Z[1], lo, bh[2], bh[3]);
        mma_f16(Z[0], hi, bl[0], bl[1]);
        mma_f16(Z[1], hi, bl[2], bl[3]);
      }
      const Pow2 sz = pow2_scale(warp_max(max_tile(Z[0], max_tile(Z[1], 0.0f))));
      uint32_t hi[4], lo[4], bh[4], bl[4];
      split_a(Z[0], Z[1], splat(sz.s), splat(sz.s), hi, lo);
      ldsm4(bh, trib + L::dh + i * 512);
      ldsm4(bl, trib + L::dl + i * 512);
      float Y[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) Y[0][e] = Y[1][e] = 0.0f;
      mma_f16(Y[0], hi, bh[0], bh[1]);
      mma_f16(Y[1], hi, bh[2], bh[3]);
      mma_f16(Y[0], lo, bh[0], bh[1]);
      mma_f16(Y[1], lo, bh[2], bh[3]);
      mma_f16(Y[0], hi, bl[0], bl[1]);
      mma_f16(Y[1], hi, bl[2], bl[3]);
      const float f = -(sz.inv * st.inv) * (sm.inv * pow2_scale(red[16 + i]).inv);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        scale_tile(Y[e], splat(f));
#pragma unroll
        for (int k = 0; k < 4; ++k) Tt[d][e][k] = Y[e][k];
      }
      run = fmaxf(run, warp_max(max_tile(Y[0], max_tile(Y[1], 0.0f))));
    }
    tt = run;
    if (lane == 0) red[20 + warp] = tt;
  }
  __syncthreads();
  const Pow2 st = pow2_scale(fmaxf(fmaxf(red[20], red[21]), fmaxf(red[22], red[19])));
  if (warp < 3) {
    const uint32_t tria = LaneOff<32>(lane, smem_u32(smem)).o[0];
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      const int i = warp + 1 + d;
      if (i > 3) continue;
      uint32_t hi[4], lo[4];
      split_a(Tt[d][0], Tt[d][1], splat(st.s), splat(st.s), hi, lo);
      const uint32_t at = tria + (i * (i + 1) / 2 + warp) * 512;
      const uint32_t oh[4] = {hi[0], hi[2], hi[1], hi[3]}, ol[4] = {lo[0], lo[2], lo[1], lo[3]};
      stsm4t(at + R::th, oh);
      stsm4t(at + R::tl, ol);
    }
  } else if (warp >= 4) {   // diagonal blocks: half a row a lane
    const int blk = warp - 4, i = lane >> 1, u = lane & 1;
    const float *o = Dd + blk * kDiag + i * 20 + 8 * u;
    uint4 hi, lo;
    uint32_t *hw = reinterpret_cast<uint32_t *>(&hi), *lw = reinterpret_cast<uint32_t *>(&lo);
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(mul2(*reinterpret_cast<const float2 *>(o + 2 * e), splat(st.s)), hw[e], lw[e]);
    const uint32_t at = (blk * (blk + 1) / 2 + blk) * 512 + tile_off<32>(i, u);
    *reinterpret_cast<uint4 *>(smem + R::th + at) = hi;
    *reinterpret_cast<uint4 *>(smem + R::tl + at) = lo;
  } else {   // warp 3
    const int f0 = static_cast<int>(bad[lane]), f1 = static_cast<int>(bad[32 + lane]);
    const unsigned lost0 = __ballot_sync(0xffffffffu, f0 & 5), lost1 = __ballot_sync(0xffffffffu, f1 & 5);
    const bool any = __any_sync(0xffffffffu, f0 | f1);
    if (lane == 0) {
      const int first = lost0 ? __ffs(lost0) - 1 : lost1 ? 31 + __ffs(lost1) : 64;
      float4 *fac = reinterpret_cast<float4 *>(smem + R::fac);
      fac[0] = make_float4(expf(G[63] + Gl[63]), st.inv, sp.inv, static_cast<float>(first));
      fac[1] = make_float4(sk.inv, sq.inv, sp.s, any ? __int_as_float(0x7fc00000) : st.inv);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p.w.rec + c * R::bytes),
                 "r"(smem_u32(smem)), "r"(p.keep ? R::bytes : std::is_same<T, __half>::value ? R::g : R::pl)   // what the forward reads
                 : "memory");
    bulk_commit();
    bulk_wait_read0();
  }
}

template <typename T, int D>
int run(const ChunkArgs &a, cudaStream_t st) {
  auto kern = delta_prep_kernel<T, D>;
  const int rc = runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepSmem<D>::total));
  if (rc) return rc;
  kern<<<static_cast<unsigned>(a.s.B) * a.s.H * a.w.nc, kThreads, PrepSmem<D>::total, st>>>(a);
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

int launch_chunk_prep(int dtype, const ChunkArgs &a, cudaStream_t st) {
  return dtype == ESA_F16 ? by_d<__half>(a, st) : by_d<__nv_bfloat16>(a, st);
}

}  // namespace esa
