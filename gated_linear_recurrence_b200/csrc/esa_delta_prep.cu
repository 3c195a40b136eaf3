// esa_delta_prep.cu -- first kernel of the chunked gated delta rule: what each
// chunk of 64 tokens needs and no other chunk changes (sm_100a).
//
// With G_i the running sum of log alpha in the chunk, the recurrence over its
// tokens is the triangular system
//   (1 + M) U = beta (V - e^G K S),   M_ij = beta_i e^{Gi - Gj} k_i.k_j  (j < i),
// where S is the state entering the chunk.  This kernel forms M from K K^T and
// P_ij = e^{Gi - Gj} q_i.k_j (j <= i) from Q K^T on the tensor cores, and
// T = (1 + M)^-1 in float32: four 16 x 16 diagonal blocks by substitution (one
// column a thread), then the blocks below the diagonal, first of 16, then of
// 32, as T21 = -T22 M21 T11.  G is kept in two float32 terms: its differences
// are exponentiated, and a token that forgets everything (G falls by 80) must
// not cost its successors their digits.
//
// Keys and queries are brought to float16 with a power of two of their own per
// row (exact for bfloat16 and float16 rows up to elements 2^-26 of the row's
// largest), so that bfloat16 tensors take the same products as float16 ones
// and the split terms of T and P keep 22 bits.
//
// The record (esa_delta_chunk.h) is put together in shared memory and leaves
// in one bulk copy.
#include "esa_delta_chunk.h"
#include "esa_delta_sweep.cuh"
#include "esa_mma.cuh"
#include "esa_umma.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

constexpr int kThreads = 256;
constexpr int LDT = 68;   // floats per row of T in shared memory

template <int D>
struct PrepSmem {
  using R = ChunkRecord<D>;
  static constexpr int m = R::th;                               // M [64][64] float32, until T's terms take its place
  static constexpr int t = (R::bytes + 127) / 128 * 128;        // T [64][LDT] float32
  static constexpr int tmp = t + 64 * LDT * 4, vec = tmp + 32 * 36 * 4, red = vec + 11 * 64 * 4, total = red + 64;
};
static_assert(ChunkRecord<64>::ph - ChunkRecord<64>::th == 64 * 64 * 4, "M takes the place of T's terms");

// M's element (i, j): columns permuted by fours so that a column's rows fall into different banks.
__device__ __forceinline__ int m_at(int i, int j) { return i * 64 + (j ^ ((i & 7) << 2)); }

// Bits of the largest magnitude of a 16-byte unit of 16-bit elements, as a
// float32 (exact): NaN and infinity compare above every finite value.
template <typename T>
__device__ __forceinline__ float unit_top(uint4 v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  const uint32_t top = max(m & 0xffffu, m >> 16);
  return unpack_io<T>(top).x;
}

// Scale 64 rows to float16 with the threads of four warps; 1 / scale of each
// row into `inv` (0 for a row of zeros; NaN marks a row that is not finite,
// which becomes zero).
template <typename T, int D>
__device__ __forceinline__ void stage_rows(const T *src, long long ld, int n, int warp, unsigned char *tile, float *inv) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPR, r0 = 16 * warp + lane / LPR;
  src += r0 * ld + sub * 8;
  uint4 raw[16 / RPI];
#pragma unroll
  for (int i = 0; i < 16 / RPI; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (r0 + i * RPI < n) raw[i] = *reinterpret_cast<const uint4 *>(src + i * RPI * ld);
  }
#pragma unroll
  for (int i = 0; i < 16 / RPI; ++i) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&raw[i]);
    uint32_t bits = __float_as_uint(unit_top<T>(raw[i]));   // not negative: orders as an integer, NaN on top
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
    const bool fine = bits < 0x7f800000u;
    const Pow2 p = pow2_scale(__uint_as_float(fine ? bits : 0u));
    const float s = fine ? p.s : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack2(mul2(unpack_io<T>(w[j]), splat(s)));
    if (!fine) raw[i] = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4 *>(tile + tile_off<D * 2>(r0 + i * RPI, sub)) = raw[i];
    if (sub == 0) inv[r0 + i * RPI] = fine ? (bits ? p.inv : 0.0f) : __int_as_float(0x7fc00000);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) delta_prep_kernel(ChunkArgs p) {
  using L = PrepSmem<D>;
  using R = ChunkRecord<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  float *M = reinterpret_cast<float *>(smem + L::m), *Ti = reinterpret_cast<float *>(smem + L::t);
  float *tmp = reinterpret_cast<float *>(smem + L::tmp), *red = reinterpret_cast<float *>(smem + L::red);
  float *vec = reinterpret_cast<float *>(smem + L::vec);
  float *kinv = vec, *qinv = vec + 64, *beta = vec + 128;
  float *G = reinterpret_cast<float *>(smem + R::g), *Gl = G + 64;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const long long c = blockIdx.x;
  const int head = static_cast<int>(c / p.w.nc), n = static_cast<int>(c - static_cast<long long>(head) * p.w.nc);
  const int b = head / p.s.H, h = head - b * p.s.H;
  const int t0 = n * kChunk, len = min(kChunk, p.s.T - t0);
  const long long row = static_cast<long long>(b) * p.s.T + t0;

  float la[2] = {0.0f, 0.0f};
  if (warp == 0) {   // two tokens a lane
    const T *ga = static_cast<const T *>(p.a), *gb = static_cast<const T *>(p.b);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      float be = 0.0f;
      if (i < len) {
        la[e] = -log1pf(expf(-fmaxf(sweep::widen(ga[(row + i) * p.s.ld_g + h]), -80.0f)));
        be = sweep::gate(sweep::widen(gb[(row + i) * p.s.ld_g + h]));
      }
      beta[i] = be;
    }
  }
  if (warp < 4)
    stage_rows<T, D>(static_cast<const T *>(p.k) + row * p.s.ld_qk + h * D, p.s.ld_qk, len, warp, smem + R::k, kinv);
  else
    stage_rows<T, D>(static_cast<const T *>(p.q) + row * p.s.ld_qk + h * D, p.s.ld_qk, len, warp - 4, smem + R::q, qinv);
  if (warp == 0) {   // running sum, in two terms
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
  __syncthreads();
  if (tid < 64) {
    const int i = tid;
    const float into = expf(G[i] + Gl[i]), out = expf((G[63] - G[i]) + (Gl[63] - Gl[i]));
    const float ki = kinv[i], qi = qinv[i], be = beta[i];
    const float kf = ki == ki ? ki : 0.0f, qf = qi == qi ? qi : 0.0f;
    float *tok = reinterpret_cast<float *>(smem + R::tok);
    tok[kTokBeta * 64 + i] = ki == ki ? be : ki;
    tok[kTokX * 64 + i] = be * into * kf;
    tok[kTokL * 64 + i] = out * kf;
    tok[kTokY * 64 + i] = p.s.scale * into * qi;
    tok[kTokK * 64 + i] = kf;
    tok[kTokQ * 64 + i] = qf;
  }
  // K K^T (warps 0-3) and Q K^T (warps 4-7): 16 rows a warp, tiles on and below the diagonal
  const int mw = warp & 3;
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
  // times e^{Gi - Gj}.  Below the diagonal block that is e^{Gi - Gr} e^{Gr - Gj}
  // with r the block's first row: two factors of at most 1, one exponential
  // per row and one per column instead of one per element.
  float top = 0.0f;
  {
    const float *rinv = warp < 4 ? kinv : qinv;
    const int r = 16 * mw, i0 = r + g;
    const float gr = G[r], grl = Gl[r];
    float *cf = vec + 192 + 64 * warp;   // this warp's column factors
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = lane + 32 * e;
      const float kj = kinv[j];
      if (j < r) cf[j] = expf((gr - G[j]) + (grl - Gl[j])) * (kj == kj ? kj : 0.0f);
    }
    float f[2], gi[2], gli[2], fe[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float ri = rinv[i0 + 8 * e];
      f[e] = ri == ri ? ri : 0.0f;
      if (warp < 4) f[e] *= beta[i0 + 8 * e];
      gi[e] = G[i0 + 8 * e];
      gli[e] = Gl[i0 + 8 * e];
      fe[e] = f[e] * expf((gi[e] - gr) + (gli[e] - grl));
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
          const float kj = kinv[j];
          float x = 0.0f;
          if (j < i || (j == i && warp >= 4))
            x = expf((gi[e >> 1] - G[j]) + (gli[e >> 1] - Gl[j])) * (kj == kj ? kj : 0.0f) * f[e >> 1] * acc[nt][e];
          acc[nt][e] = x;
        }
      }
      top = max_tile(acc[nt], top);
      if (warp < 4) {
        *reinterpret_cast<float2 *>(M + m_at(i0, 8 * nt + 2 * t4)) = row_lo(acc[nt]);
        *reinterpret_cast<float2 *>(M + m_at(i0 + 8, 8 * nt + 2 * t4)) = row_hi(acc[nt]);
      }
    }
  }
  top = warp_max(top);
  if (lane == 0) red[warp] = top;
  __syncthreads();
  const Pow2 sp = pow2_scale(fmaxf(fmaxf(red[4], red[5]), fmaxf(red[6], red[7])));
  if (warp >= 4) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int i = 16 * mw + g + (e >> 1) * 8;
        uint32_t hi = 0, lo = 0;
        if (nt <= 2 * mw + 1) split2(make_float2(acc[nt][e] * sp.s, acc[nt][e + 1] * sp.s), hi, lo);
        const uint32_t o = tile_off<128>(i, nt) + 4 * t4;
        *reinterpret_cast<uint32_t *>(smem + R::ph + o) = hi;
        *reinterpret_cast<uint32_t *>(smem + R::pl + o) = lo;
      }
  }
  // T = (1 + M)^-1
  if (tid < 64) {   // column `col` of the 16 x 16 block at r0
    const int r0 = tid & 48, col = tid & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(M + m_at(r0 + i, r0 + l));
        s[0] = fmaf(m.x, x[l], s[0]);
        if (l + 1 < i) s[1] = fmaf(m.y, x[l + 1], s[1]);
        if (l + 2 < i) s[2] = fmaf(m.z, x[l + 2], s[2]);
        if (l + 3 < i) s[3] = fmaf(m.w, x[l + 3], s[3]);
      }
      const float sum = (s[0] + s[1]) + (s[2] + s[3]);
      x[i] = i == col ? 1.0f : (i > col ? -sum : 0.0f);
      Ti[(r0 + i) * LDT + r0 + col] = x[i];
    }
  }
  __syncthreads();
  {   // blocks (1,0) and (3,2): 128 threads each, 2 columns of a row a thread
    const int pr = tid >> 7, i = (tid & 127) >> 3, j = (tid & 7) * 2, r0 = 32 * pr;
    float2 s = make_float2(0, 0);
#pragma unroll
    for (int l = 0; l < 16; ++l)
      s = fma2(splat(M[m_at(r0 + 16 + i, r0 + l)]), *reinterpret_cast<const float2 *>(Ti + (r0 + l) * LDT + r0 + j), s);
    *reinterpret_cast<float2 *>(tmp + (16 * pr + i) * 36 + j) = s;
    __syncthreads();
    s = make_float2(0, 0);
#pragma unroll
    for (int l = 0; l < 16; ++l)
      s = fma2(splat(-Ti[(r0 + 16 + i) * LDT + r0 + 16 + l]), *reinterpret_cast<const float2 *>(tmp + (16 * pr + l) * 36 + j), s);
    *reinterpret_cast<float2 *>(Ti + (r0 + 16 + i) * LDT + r0 + j) = s;
    *reinterpret_cast<float2 *>(Ti + (r0 + i) * LDT + r0 + 16 + j) = make_float2(0, 0);   // above the diagonal
  }
  __syncthreads();
  {   // rows 32-63, columns 0-31: 4 columns of a row a thread
    const int i = tid >> 3, j = (tid & 7) * 4;
    float2 s0 = make_float2(0, 0), s1 = s0;
#pragma unroll 16
    for (int l = 0; l < 32; ++l) {
      const float2 m = splat(M[m_at(32 + i, l)]);
      const float4 x = *reinterpret_cast<const float4 *>(Ti + l * LDT + j);
      s0 = fma2(m, make_float2(x.x, x.y), s0);
      s1 = fma2(m, make_float2(x.z, x.w), s1);
    }
    *reinterpret_cast<float4 *>(tmp + i * 36 + j) = make_float4(s0.x, s0.y, s1.x, s1.y);
    __syncthreads();
    s0 = s1 = make_float2(0, 0);
#pragma unroll 16
    for (int l = 0; l < 32; ++l) {
      const float2 m = splat(-Ti[(32 + i) * LDT + 32 + l]);
      const float4 x = *reinterpret_cast<const float4 *>(tmp + l * 36 + j);
      s0 = fma2(m, make_float2(x.x, x.y), s0);
      s1 = fma2(m, make_float2(x.z, x.w), s1);
    }
    *reinterpret_cast<float4 *>(Ti + (32 + i) * LDT + j) = make_float4(s0.x, s0.y, s1.x, s1.y);
    *reinterpret_cast<float4 *>(Ti + i * LDT + 32 + j) = make_float4(0, 0, 0, 0);
  }
  __syncthreads();
  const int ti = tid >> 2, tu = (tid & 3) * 2;   // a row's 16-byte units tu and tu + 1 (16 columns) a thread
  float x[16];
  top = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    const float4 v = *reinterpret_cast<const float4 *>(Ti + ti * LDT + 8 * tu + j);
    x[j] = v.x; x[j + 1] = v.y; x[j + 2] = v.z; x[j + 3] = v.w;
    top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
  top = warp_max(top);
  if (lane == 0) red[8 + warp] = top;
  __syncthreads();
  top = red[8];
#pragma unroll
  for (int w = 1; w < 8; ++w) top = fmaxf(top, red[8 + w]);
  const Pow2 stt = pow2_scale(top);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint4 hi, lo;
    uint32_t *hw = reinterpret_cast<uint32_t *>(&hi), *lw = reinterpret_cast<uint32_t *>(&lo);
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(mul2(make_float2(x[8 * u + 2 * e], x[8 * u + 2 * e + 1]), splat(stt.s)), hw[e], lw[e]);
    *reinterpret_cast<uint4 *>(smem + R::th + tile_off<128>(ti, tu + u)) = hi;   // M has been read
    *reinterpret_cast<uint4 *>(smem + R::tl + tile_off<128>(ti, tu + u)) = lo;
  }
  if (tid == 0)
    *reinterpret_cast<float4 *>(smem + R::fac) = make_float4(expf(G[63] + Gl[63]), stt.inv, sp.inv, 0.0f);
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p.w.rec + c * R::bytes),
                 "r"(smem_u32(smem)), "r"(p.keep ? R::bytes : R::pl)
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
