// esa_mma.cuh -- warp-level helpers of the chunked gated delta rule: matrix
// fragments in registers, swizzled shared-memory tiles, and the splitting of
// float32 values into scaled float16 terms (sm_100a).
//
// Fragments are those of mma.m16n8k16: with g = lane / 4 and t = lane % 4, an
// accumulator holds (row g, columns 2t, 2t+1) and (row g + 8, the same); an A
// operand holds rows g and g + 8 of columns 2t, 2t+1 and 2t+8, 2t+9.  So two
// neighbouring accumulators are the A operand of the next product without any
// exchange between lanes.
//
// A float32 value x is kept as two float16 terms of x s, with s a power of two
// that brings the largest |x| of its row to [2^5, 2^13): hi = fp16(x s),
// lo = fp16(x s - hi).  The two carry 22 bits (an absolute error of at most
// 2^-30 of the row's largest value for its small elements), and a product
// with an exact float16 operand is two mma with one accumulator.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "esa_common.cuh"

namespace esa {

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// Byte offset of 16-byte unit `c` of row `row` in a tile of RB-byte rows.  The
// units are permuted so that the 8 rows of one matrix of an ldmatrix fall
// into different banks.
template <int RB>
__device__ __forceinline__ uint32_t tile_off(int row, int c) {
  if constexpr (RB >= 128) return row * RB + ((c ^ (row & 7)) << 4);
  else if constexpr (RB == 64) return row * RB + ((c ^ ((row >> 1) & 3)) << 4);
  else return row * RB + ((c ^ ((row >> 2) & 1)) << 4);
}

__device__ __forceinline__ float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ uint32_t pack_h2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Pair of I/O elements packed in 32 bits -> floats, and back.
template <typename T> __device__ __forceinline__ float2 unpack_io(uint32_t v);
template <> __device__ __forceinline__ float2 unpack_io<__half>(uint32_t v) { return unpack_h2(v); }
template <> __device__ __forceinline__ float2 unpack_io<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}
template <typename T> __device__ __forceinline__ uint32_t pack_io(float x, float y);
template <> __device__ __forceinline__ uint32_t pack_io<__half>(float x, float y) { return pack_h2(x, y); }
template <> __device__ __forceinline__ uint32_t pack_io<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Bits of the largest magnitude of a 16-byte unit of 16-bit elements, as a
// float32 (exact): NaN and infinity compare above every finite value.
template <typename T>
__device__ __forceinline__ uint32_t unit_top(uint4 v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return __float_as_uint(unpack_io<T>(max(m & 0xffffu, m >> 16)).x);
}

// Power of two, of an exponent divisible by 8, that brings `top` (>= 0) to
// [2^5, 2^13), and its inverse; 1 for zero.  Steps of 2^8 let the groups of a
// tile have the same scale almost always; float16 has the room.  A product of
// two of them may have no reciprocal in float32: none is formed.
struct Pow2 {
  float s, inv;
};
__device__ __forceinline__ Pow2 pow2_scale(float top) {
  int e = ((static_cast<int>(__float_as_uint(top) >> 23) - 132) >> 3) * 8;   // floor((exponent - 5) / 8) * 8
  e = top > 0.0f ? max(-120, min(e, 120)) : 0;
  return {__uint_as_float(static_cast<uint32_t>(127 - e) << 23), __uint_as_float(static_cast<uint32_t>(127 + e) << 23)};
}

// 1 / x of a normal power of two.
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

// Scale of a group that another kernel reads as one float16 term: 2^8 for any
// largest value in [2^-9, 2^7), so that the groups of a tile agree and need not
// be brought together there; else that of pow2_scale.
__device__ __forceinline__ Pow2 store_scale(float top) {
  if (top >= 0.001953125f && top < 128.0f) return {256.0f, 0.00390625f};
  return pow2_scale(top);
}

// What is kept of that scale beside the group: its inverse, 0 for a group of
// zeros, NaN for one that is not finite.
__device__ __forceinline__ float slice_unit(float top, Pow2 s) {
  return top <= 3.4028235e38f ? (top > 0.0f ? s.inv : 0.0f) : __int_as_float(0x7fc00000);
}

// A sum whose addends have different units (powers of two) is formed in one of
// them, which must not be so much smaller than another that this one overflows:
// where all write gates of a chunk are closed (beta = e^-80), the products of
// its own values are 2^-115 of those with the state.  So a unit is at least
// 2^-87 of that of sums below 2^33, and at least 2^-120; what the smaller
// addends then lose is below 2^-80 of the larger.  (The unit of a state of
// zeros is zero here.)
constexpr float kLeastShare = 6.462348535570529e-27f;   // 2^-87
constexpr float kLeastUnit = 7.52316384526264e-37f;     // 2^-120

// Scale of the state after a chunk: the one that suits its update, whose
// largest value is `upd` (2^126 below 2^-113, so that updates of 2^-120 keep 22
// bits), unless that would lift the state, of largest value `top` and unit
// `unit` and decaying by `decay`, by more than 2^36 over its own scale.
__device__ __forceinline__ float update_scale(float upd, float top, float unit, float decay) {
  const int s = upd > 0.0f && upd < 9.62964972193618e-35f ? 253 : static_cast<int>(__float_as_uint(pow2_scale(upd).s) >> 23);
  const int most = 127 + 36 + 127 + 127 - static_cast<int>(__float_as_uint(unit) >> 23) - static_cast<int>(__float_as_uint(decay) >> 23);
  return __uint_as_float(static_cast<uint32_t>(top > 0.0f ? min(s, most) : s) << 23);
}
__device__ __forceinline__ float2 update_scale(float2 upd, float2 top, float2 unit, float decay) {
  return make_float2(update_scale(upd.x, top.x, unit.x, decay), update_scale(upd.y, top.y, unit.y, decay));
}

// The scale of an output gradient, `own`, such that the unit of its product, its
// inverse times 1 / (a b), is no smaller than kLeastShare allows beside a product
// of unit `other`; a power of two.
__device__ __forceinline__ Pow2 least_unit(Pow2 own, float other, float a, float b) {
  const float least = fminf(fmaxf(other * kLeastShare, kLeastUnit) * a * b, 2.5961484292674138e33f);   // 2^111
  if (!(least > own.inv)) return own;
  const float inv = __uint_as_float((__float_as_uint(least) & 0x7f800000u) + 0x00800000u);   // the next power of two
  return {pow2_inverse(inv), inv};
}

// x a b for powers of two a and b whose product alone may leave float32's range.
__device__ __forceinline__ float mul_pow2(float x, float a, float b) {
  const int e = static_cast<int>(__float_as_uint(a) >> 23) + static_cast<int>(__float_as_uint(b) >> 23) - 254, h = e >> 1;
  return x * __uint_as_float(static_cast<uint32_t>(127 + h) << 23) * __uint_as_float(static_cast<uint32_t>(127 + e - h) << 23);
}

// Y = scale (e^G S^T Q^T + U P^T), formed as unit scale (r e^G (S^T Q^T) + (us U) P^T):
// `xq` is the unit of S^T Q^T, `uinv` that of U by its own size, `p` that of P
// (`ps` its inverse), `least` the least of `unit` (ChunkArgs::least).
struct OutputUnit {
  float us, unit, r;
};
__device__ __forceinline__ OutputUnit output_unit(float xq, float uinv, float p, float ps, float least) {
  uinv = fmaxf(uinv, fmaxf(xq * kLeastShare, least) * ps);
  const float unit = p * uinv;
  return {pow2_inverse(uinv), unit, xq * pow2_inverse(unit)};
}

// ---- factors of the two rows (g and g + 8) that a thread has of a tile --------
// The chains' rows are value channels, which do not mix: each has scales of its
// own, or a large (or infinite) channel would take its neighbours' digits.
struct RowPow2 {
  float2 s, inv;
};
__device__ __forceinline__ RowPow2 pow2_scale(float2 top) {
  const Pow2 a = pow2_scale(top.x), b = pow2_scale(top.y);
  return {make_float2(a.s, b.s), make_float2(a.inv, b.inv)};
}
__device__ __forceinline__ RowPow2 least_unit(RowPow2 own, float2 other, float a, float b) {
  const Pow2 x = least_unit(Pow2{own.s.x, own.inv.x}, other.x, a, b), y = least_unit(Pow2{own.s.y, own.inv.y}, other.y, a, b);
  return {make_float2(x.s, y.s), make_float2(x.inv, y.inv)};
}
// A state's unit, zero for a state of zeros (see kLeastShare).
__device__ __forceinline__ float2 unit_or_zero(float2 top, float2 unit) {
  return make_float2(top.x > 0.0f ? unit.x : 0.0f, top.y > 0.0f ? unit.y : 0.0f);
}
// The largest of a row from the largest of each of the four threads that share it (a NaN is passed over).
__device__ __forceinline__ float2 quad_max(float2 t) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    t.x = fmaxf(t.x, __shfl_xor_sync(0xffffffffu, t.x, o));
    t.y = fmaxf(t.y, __shfl_xor_sync(0xffffffffu, t.y, o));
  }
  return t;
}
__device__ __forceinline__ float2 max_rows(const float (&c)[4], float2 t) {
  return make_float2(fmaxf(fmaxf(t.x, fabsf(c[0])), fabsf(c[1])), fmaxf(fmaxf(t.y, fabsf(c[2])), fabsf(c[3])));
}

// An A operand's rows times f (registers 0 and 2 hold row g).
__device__ __forceinline__ void scale_h2(uint32_t (&r)[4], float2 f) {
  const __half2 s[2] = {__float2half2_rn(f.x), __float2half2_rn(f.y)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&r[i]), s[i & 1]);
    r[i] = *reinterpret_cast<const uint32_t *>(&x);
  }
}

// Store a 16 x 16 float16 block held as an A operand, rows `ld` elements apart.
// Neighbouring lanes exchange one register of each row's two, so that four
// lanes write the 32 bytes of a row (a whole sector) with 8-byte stores.
__device__ __forceinline__ void store_block(__half *p, int ld, const uint32_t (&a)[4], int lane) {
  const bool odd = lane & 1;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t x0 = __shfl_xor_sync(0xffffffffu, odd ? a[0] : a[2], 1);
  const uint32_t x1 = __shfl_xor_sync(0xffffffffu, odd ? a[1] : a[3], 1);
  __half *o = p + g * ld + (odd ? 8 : 0) + 2 * (t4 & 2);
  *reinterpret_cast<uint2 *>(o) = odd ? make_uint2(x0, a[2]) : make_uint2(a[0], x0);
  *reinterpret_cast<uint2 *>(o + 8 * ld) = odd ? make_uint2(x1, a[3]) : make_uint2(a[1], x1);
}

// Largest |x| of the warp (a NaN is passed over unless all are).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// hi and lo terms of an already scaled pair; x - hi is one mixed-precision
// multiply-add (exact).
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
  hi = pack_h2(x.x, x.y);
  unsigned short h0, h1;
  float d0, d1;
  asm("mov.b32 {%0, %1}, %2;" : "=h"(h0), "=h"(h1) : "r"(hi));
  const unsigned short minus_one = 0xBC00;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d0) : "h"(h0), "h"(minus_one), "f"(x.x));
  asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d1) : "h"(h1), "h"(minus_one), "f"(x.y));
  lo = pack_h2(d0, d1);
}

// An accumulator tile's two rows, as pairs.
__device__ __forceinline__ float2 row_lo(const float (&c)[4]) { return make_float2(c[0], c[1]); }
__device__ __forceinline__ float2 row_hi(const float (&c)[4]) { return make_float2(c[2], c[3]); }
__device__ __forceinline__ void set_lo(float (&c)[4], float2 x) { c[0] = x.x; c[1] = x.y; }
__device__ __forceinline__ void set_hi(float (&c)[4], float2 x) { c[2] = x.x; c[3] = x.y; }
__device__ __forceinline__ void scale_tile(float (&c)[4], float2 s) {
  set_lo(c, mul2(row_lo(c), s));
  set_hi(c, mul2(row_hi(c), s));
}
__device__ __forceinline__ float max_tile(const float (&c)[4], float top) {
  top = fmaxf(fmaxf(top, fabsf(c[0])), fabsf(c[1]));
  return fmaxf(fmaxf(top, fabsf(c[2])), fabsf(c[3]));
}

__device__ __forceinline__ void scale_rows(float (&c)[4], float2 s) {
  set_lo(c, mul2(row_lo(c), splat(s.x)));
  set_hi(c, mul2(row_hi(c), splat(s.y)));
}

// A operand (hi and lo terms, or hi alone) of columns 16 k .. 16 k + 15 from
// the accumulators of tiles 2 k and 2 k + 1, whose columns are multiplied by
// s0 and s1 first, or whose rows are by s, or both.
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4], float2 s0, float2 s1,
                                        uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(mul2(row_lo(c0), s0), hi[0], lo[0]);
  split2(mul2(row_hi(c0), s0), hi[1], lo[1]);
  split2(mul2(row_lo(c1), s1), hi[2], lo[2]);
  split2(mul2(row_hi(c1), s1), hi[3], lo[3]);
}
__device__ __forceinline__ uint32_t pack2(float2 x) { return pack_h2(x.x, x.y); }
__device__ __forceinline__ void split_rows(const float (&c0)[4], const float (&c1)[4], float2 s, uint32_t (&hi)[4],
                                           uint32_t (&lo)[4]) {
  split2(mul2(row_lo(c0), splat(s.x)), hi[0], lo[0]);
  split2(mul2(row_hi(c0), splat(s.y)), hi[1], lo[1]);
  split2(mul2(row_lo(c1), splat(s.x)), hi[2], lo[2]);
  split2(mul2(row_hi(c1), splat(s.y)), hi[3], lo[3]);
}
__device__ __forceinline__ void split_grid(const float (&c0)[4], const float (&c1)[4], float2 s0, float2 s1, float2 s,
                                           uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split2(mul2(row_lo(c0), mul2(s0, splat(s.x))), hi[0], lo[0]);
  split2(mul2(row_hi(c0), mul2(s0, splat(s.y))), hi[1], lo[1]);
  split2(mul2(row_lo(c1), mul2(s1, splat(s.x))), hi[2], lo[2]);
  split2(mul2(row_hi(c1), mul2(s1, splat(s.y))), hi[3], lo[3]);
}
__device__ __forceinline__ void single_rows(const float (&c0)[4], const float (&c1)[4], float2 s, uint32_t (&hi)[4]) {
  hi[0] = pack2(mul2(row_lo(c0), splat(s.x)));
  hi[1] = pack2(mul2(row_hi(c0), splat(s.y)));
  hi[2] = pack2(mul2(row_lo(c1), splat(s.x)));
  hi[3] = pack2(mul2(row_hi(c1), splat(s.y)));
}

// A lane's offsets for ldmatrix.x4 of 16 x 16 blocks of a tile of RB-byte
// rows: block (16 i, 16 j) is at off[j % 4] + 128 (j / 4) + 16 i RB, so a whole
// chunk's fragment loads are a few registers and immediate offsets.  The
// matrices come in the order (rows 0-7, columns 0-7), (rows 8-15, 0-7), (rows
// 0-7, 8-15), (rows 8-15, 8-15): that of an A operand, and with .trans and
// read as [0, 2, 1, 3] that of its transpose.
template <int RB>
struct LaneOff {
  static constexpr int N = RB >= 128 ? 4 : RB / 32;
  uint32_t o[N];
  __device__ __forceinline__ explicit LaneOff(int lane, uint32_t base = 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = base + tile_off<RB>(lane & 15, 2 * j + (lane >> 4));
  }
  __device__ __forceinline__ uint32_t at(int i, int j) const { return o[j % N] + 128 * (j / N) + 16 * i * RB; }
};

// The same for B operands stored [column n][k] and loaded without .trans: the
// matrices come in the order (n 0-7: k 0-7, k 8-15), (n 8-15: k 0-7, k 8-15),
// so that each mma's two registers are neighbours (the hardware wants an
// aligned pair; in the order above every fragment cost two moves).  With
// LaneOff and .trans the blocks of B stored [k][n] come in that order too.
template <int RB>
struct LaneOffB {
  static constexpr int N = LaneOff<RB>::N;
  uint32_t o[N];
  __device__ __forceinline__ explicit LaneOffB(int lane, uint32_t base = 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = base + tile_off<RB>((lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1));
  }
  __device__ __forceinline__ uint32_t at(int i, int j) const { return o[j % N] + 128 * (j / N) + 16 * i * RB; }
};

// Lower triangle of a 64 x 64 float16 matrix as ten 16 x 16 blocks of 512
// bytes, rows of 32 bytes: byte offset of block (i, j), j <= i.
constexpr int kTriBytes = 10 * 512;
__host__ __device__ constexpr int tri(int i, int j) { return (i * (i + 1) / 2 + j) * 512; }

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16_s(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Copy BYTES contiguous bytes to shared memory with all THREADS threads.
template <int BYTES, int THREADS>
__device__ __forceinline__ void copy_linear(uint32_t dst, const unsigned char *src) {
  constexpr int U = BYTES / 16;
  const uint32_t d = dst + threadIdx.x * 16;
  const unsigned char *s = src + threadIdx.x * 16;
#pragma unroll
  for (int i = 0; i < U / THREADS; ++i) cp_async16_s(d + i * THREADS * 16, s + i * THREADS * 16);
  if constexpr (U % THREADS != 0)
    if (threadIdx.x < U % THREADS) cp_async16_s(d + U / THREADS * THREADS * 16, s + U / THREADS * THREADS * 16);
}

// Copy ROWS plain rows of RB bytes into a swizzled tile with all THREADS
// threads; a thread's units lie a whole number of 8 rows apart, so its place
// in the swizzle does not change.
template <int RB, int ROWS, int THREADS>
__device__ __forceinline__ void copy_rows(uint32_t dst, const void *src) {
  constexpr int U = RB / 16, STEP = THREADS / U;
  static_assert(THREADS % U == 0 && STEP % 8 == 0, "whole groups of 8 rows");
  const int r = threadIdx.x / U;
  const uint32_t d = dst + tile_off<RB>(r, threadIdx.x % U);
  const unsigned char *s = static_cast<const unsigned char *>(src) + threadIdx.x * 16;
#pragma unroll
  for (int i = 0; i < (ROWS + STEP - 1) / STEP; ++i)
    if (ROWS % STEP == 0 || r + i * STEP < ROWS) cp_async16_s(d + i * STEP * RB, s + i * THREADS * 16);
}

}  // namespace esa
