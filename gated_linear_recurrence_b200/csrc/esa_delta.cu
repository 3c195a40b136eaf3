// esa_delta.cu -- C ABI of the gated delta rule (declared in include/esa.h):
// argument checks, the workspace, and the order of the kernels.
#include "esa_delta.h"
#include "esa_delta_chunk.h"

#include <climits>
#include <cmath>

#include "esa.h"
#include "esa_host.h"

using namespace esa;

namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Sequences of 16-bit types of at least this many tokens go through the
// chunked kernels, shorter ones and float32 token by token.  A chunk costs the
// same however few its tokens, a sweep goes by the token, and the gradients
// have four sweeps.  Forward alone (us, chunked / token by token):
//             8 heads                         64 heads             512 heads
//   D =  32   9.9 / 7.8 at T = 32, 9.9 / 9.9 at 40   10.2 / 9.9 at 40     16.2 / 10.4 at 40, 26.9 / 27.3 at 128
//   D =  64   10.5 / 8.9 at 32, 10.4 / 11.3 at 40    11.4 / 11.4 at 40    21.7 / 20.8 at 32, 21.9 / 26.0 at 40
//   D = 128   11.8 / 10.8 at 24, 11.9 / 13.3 at 32   13.8 / 14.0 at 24    48.2 / 55.6 at 16, 49.6 / 80.6 at 24
// and with the backward:
//   D =  32   21.0 / 19.4 at 12, 20.9 / 21.4 at 16   21.7 / 22.0 at 16    39.8 / 30.5 at 16, 40.0 / 37.7 at 24
//   D =  64   22.6 / 19.2 at 8, 22.5 / 21.9 at 12    25.3 / 27.1 at 12    55.8 / 41.9 at 8, 56.0 / 50.7 at 12
//   D = 128   28.0 / 23.4 at 8, 28.1 / 26.6 at 12    33.5 / 34.2 at 8     133 / 114 at 4, 134 / 162 at 8
int chunk_min(int D, bool keep) { return keep ? (D == 32 ? 16 : D == 64 ? 12 : 8) : D == 128 ? 24 : 40; }
bool chunked(const DeltaShape &s, int dtype, bool keep) { return dtype != ESA_F32 && s.T >= chunk_min(s.D, keep); }

// Long float32 sequences of few heads: the states between chunks first, then
// the sweeps of all chunks at once.  Forward (us, states first / one sweep): 8
// heads at T = 128 27 / 24 (D = 32), 34 / 27 (64), 48 / 39 (128); at T = 333
// 35 / 59, 43 / 69, 69 / 98; at T = 4096 143 / 707, 226 / 833, 508 / 1183, and
// with the backward 361 / 1422, 605 / 1948, 1565 / 3327.  64 heads at T = 1024
// 80 / 178, 197 / 214, 758 / 416; 32 heads of D = 128 410 / 321: one sweep
// keeps the device busy there.
constexpr int kCutMinT = 192, kCutMostHeads = 64, kCutMostState = 1 << 18;   // floats of all heads' states
bool cut_sweeps(const DeltaShape &s, int dtype) {
  const long long heads = static_cast<long long>(s.B) * s.H;
  return dtype == ESA_F32 && s.T >= kCutMinT && heads <= kCutMostHeads && heads * s.D * s.D <= kCutMostState;
}

// Token by token: what the forward keeps for the backward (u, the state at
// each chunk), then the backward's scratch.
struct DeltaLayout {
  int nc = 0;
  bool cut = false;
  size_t u = 0, S_ck = 0, dS_ck = 0, du = 0, dk = 0, dq = 0, gain = 0, end = 0, dk2 = 0, wt = 0, u0 = 0, fac = 0, total = 0;
};
// The chunk arrays, laid out from `base`; `*total` gets their size.
ChunkArrays chunk_arrays(unsigned char *base, const DeltaShape &s, int dtype, bool keep, size_t *total) {
  ChunkArrays w{};
  w.nc = (s.T + kChunk - 1) / kChunk;
  const size_t n = static_cast<size_t>(s.B) * s.H * w.nc;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    unsigned char *p = base + o;
    o += up256(bytes);
    return p;
  };
  const size_t rec = s.D == 32 ? ChunkRecord<32>::bytes : s.D == 64 ? ChunkRecord<64>::bytes : ChunkRecord<128>::bytes;
  w.rec = take(n * rec);
  if (keep) {
    const size_t D = s.D;
    w.u16 = reinterpret_cast<__half *>(take(n * 64 * D * 2));
    w.r16 = reinterpret_cast<__half *>(take(n * 64 * D * 2));
    if (dtype == ESA_F16) {
      w.u16l = reinterpret_cast<__half *>(take(n * 64 * D * 2));
      w.r16l = reinterpret_cast<__half *>(take(n * 64 * D * 2));
    }
    w.s16 = reinterpret_cast<__half *>(take(n * D * D * 2));
    w.ds16 = reinterpret_cast<__half *>(take(n * D * D * 2));
    w.slice = reinterpret_cast<float *>(take(n * 32 * sizeof(float)));
  }
  *total = o;
  return w;
}

DeltaLayout delta_layout(const DeltaShape &s, int dtype, bool keep) {
  DeltaLayout lo;
  lo.nc = (s.T + 63) / 64;
  lo.cut = cut_sweeps(s, dtype);
  const size_t n = static_cast<size_t>(s.B) * s.T * s.H, chunks = static_cast<size_t>(s.B) * s.H * lo.nc;
  size_t o = 0;
  const size_t rows = up256(n * s.D * sizeof(float)), states = up256(chunks * s.D * s.D * sizeof(float));
  if (keep || lo.cut) {
    lo.S_ck = o; o += states;
  }
  if (lo.cut) {
    lo.wt = o; o += up256(chunks * 64 * s.D * sizeof(float));
    lo.u0 = o; o += up256(chunks * 64 * s.D * sizeof(float));
    lo.fac = o; o += up256(chunks * 3 * 64 * sizeof(float));
  }
  if (keep) {
    lo.u = o; o += rows;
    lo.dS_ck = o; o += states;
    lo.du = o; o += rows;
    lo.dk = o; o += rows;
    lo.dk2 = o; o += rows;
    lo.dq = o; o += rows;
    lo.gain = o; o += up256(n * sizeof(float));
    lo.end = o; o += up256(chunks * (s.D * s.D / 1024) * sizeof(float));
  }
  lo.total = o;
  return lo;
}

void between(SweepArgs *p, const DeltaLayout &lo, unsigned char *base) {
  p->cut = true;
  p->wt = reinterpret_cast<float *>(base + lo.wt);
  p->u0 = reinterpret_cast<float *>(base + lo.u0);
  p->fac = reinterpret_cast<float *>(base + lo.fac);
}

int elem(int dtype) { return dtype == ESA_F32 ? 4 : 2; }

int check_shape(int B, int T, int H, int D, int dtype) {
  if (B < 0 || T < 0 || H < 1 || D < 1) return ESA_ERR_ARG;
  if (T > INT_MAX - 64) return ESA_ERR_ARG;                                    // tokens up to a chunk's end
  if (dtype < ESA_F32 || dtype > ESA_E4M3) return ESA_ERR_ARG;
  if (dtype == ESA_E4M3 || (D != 32 && D != 64 && D != 128)) return ESA_ERR_UNSUPPORTED;
  if (static_cast<long long>(H) * D > INT_MAX / 2) return ESA_ERR_ARG;
  if (static_cast<long long>(B) * H > INT_MAX / 8) return ESA_ERR_ARG;         // blocks of a launch
  if (static_cast<long long>(B) * T > (1ll << 33) / H) return ESA_ERR_ARG;     // eight rows a block
  return ESA_OK;
}

int check_rows(long long ld, long long least, int dtype) {
  if (ld < least || ld > INT_MAX) return ESA_ERR_ARG;
  return (ld * elem(dtype)) % 16 ? ESA_ERR_ALIGN : ESA_OK;
}

// A scale below the normal range has no inverse in float32: it counts as zero.
float normal(float s) { return fabsf(s) < 1.17549435e-38f ? 0.0f : s; }

int check_scale(float s) { return s == s && s < 3.0e38f && s > -3.0e38f ? ESA_OK : ESA_ERR_ARG; }

// Shape, strides and the five inputs of a sequence call.
int check_inputs(const DeltaShape &s, int dtype, const void *q, const void *k, const void *v, const void *a,
                 const void *b) {
  int rc = check_shape(s.B, s.T, s.H, s.D, dtype);
  if (rc) return rc;
  if ((rc = check_scale(s.scale))) return rc;
  const long long C = static_cast<long long>(s.H) * s.D;
  if ((rc = check_rows(s.ld_qk, C, dtype)) || (rc = check_rows(s.ld_v, C, dtype))) return rc;
  if (s.ld_g < s.H || s.ld_g > INT_MAX) return ESA_ERR_ARG;
  if (s.B > 0 && s.T > 0 && (!q || !k || !v || !a || !b)) return ESA_ERR_ARG;
  for (const void *p : {q, k, v})
    if (p && !aligned_to(p, 16)) return ESA_ERR_ALIGN;
  for (const void *p : {a, b})
    if (p && !aligned_to(p, elem(dtype))) return ESA_ERR_ALIGN;
  return ESA_OK;
}

size_t state_bytes(const DeltaShape &s) { return static_cast<size_t>(s.B) * s.H * s.D * s.D * sizeof(float); }

// The state (or its gradient) of no tokens.
int copy_state(float *out, const float *in, const DeltaShape &s, cudaStream_t st) {
  if (!out || out == in) return ESA_OK;
  return in ? runtime_status(cudaMemcpyAsync(out, in, state_bytes(s), cudaMemcpyDeviceToDevice, st))
            : runtime_status(cudaMemsetAsync(out, 0, state_bytes(s), st));
}

}  // namespace

extern "C" {

size_t esa_delta_workspace_size(int B, int T, int H, int D, int dtype, int keep) {
  if (check_shape(B, T, H, D, dtype) != ESA_OK || (keep != 0 && keep != 1)) return 0;
  const DeltaShape s{B, T, H, D, 0, 0, 0, 1.0f};
  size_t total = 0;
  if (chunked(s, dtype, keep != 0)) {
    chunk_arrays(nullptr, s, dtype, keep != 0, &total);
    return total + 256;
  }
  return delta_layout(s, dtype, keep != 0).total + 256;
}

int esa_delta_fwd(const void *q, const void *k, long long ld_qk, const void *v, long long ld_v, const void *a,
                  const void *b, long long ld_g, void *y, float *S_final, int B, int T, int H, int D, float scale,
                  const float *S_init, int dtype, int keep, void *workspace, size_t workspace_bytes, void *stream) {
  const DeltaShape s{B, T, H, D, ld_qk, ld_v, ld_g, normal(scale)};
  int rc = check_inputs(s, dtype, q, k, v, a, b);
  if (rc) return rc;
  if (keep != 0 && keep != 1) return ESA_ERR_ARG;
  if (B > 0 && T > 0 && !y) return ESA_ERR_ARG;
  for (const void *p : {static_cast<const void *>(y), static_cast<const void *>(S_final),
                        static_cast<const void *>(S_init), static_cast<const void *>(workspace)})
    if (p && !aligned_to(p, 16)) return ESA_ERR_ALIGN;
  if (!workspace || workspace_bytes < esa_delta_workspace_size(B, T, H, D, dtype, keep)) return ESA_ERR_WORKSPACE;
  if ((rc = check_current_device())) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B == 0) return ESA_OK;
  if (T == 0) return copy_state(S_final, S_init, s, st);
  if (chunked(s, dtype, keep != 0)) {
    ChunkArgs c{};
    size_t total;
    c.s = s;
    c.w = chunk_arrays(static_cast<unsigned char *>(workspace), s, dtype, keep != 0, &total);
    c.q = q; c.k = k; c.v = v; c.a = a; c.b = b;
    c.y = y;
    c.S_in = S_init;
    c.S_out = S_final;
    c.keep = keep != 0;
    c.least = least_output_unit(s.scale);
    if ((rc = launch_chunk_prep(dtype, c, st))) return rc;
    return launch_chunk_fwd(dtype, c, st);
  }
  const DeltaLayout lo = delta_layout(s, dtype, keep != 0);
  unsigned char *base = static_cast<unsigned char *>(workspace);
  SweepArgs p{};
  p.s = s;
  p.q = q; p.k = k; p.v = v; p.a = a; p.b = b;
  p.S_in = S_init;
  p.S_out = S_final;
  p.y = y;
  p.nc = lo.nc;
  if (keep) p.u = reinterpret_cast<float *>(base + lo.u);
  if (keep || lo.cut) p.S_ck = reinterpret_cast<float *>(base + lo.S_ck);
  if (lo.cut) {
    between(&p, lo, base);
    if ((rc = launch_delta_states(false, p, st))) return rc;
  }
  return launch_sweep(kSweepFwd, dtype, p, st);
}

int esa_delta_bwd(const void *q, const void *k, long long ld_qk, const void *v, long long ld_v, const void *a,
                  const void *b, long long ld_g, const void *dy, const float *dS_final, void *dq, void *dk, void *dv,
                  void *da, void *db, float *dS_init, int B, int T, int H, int D, float scale, const float *S_init,
                  int dtype, void *workspace, size_t workspace_bytes, void *stream) {
  const DeltaShape s{B, T, H, D, ld_qk, ld_v, ld_g, normal(scale)};
  int rc = check_inputs(s, dtype, q, k, v, a, b);
  if (rc) return rc;
  if (B > 0 && T > 0 && (!dy || !dq || !dk || !dv || !da || !db)) return ESA_ERR_ARG;
  for (const void *p : {dy, static_cast<const void *>(dS_final), static_cast<const void *>(dq),
                        static_cast<const void *>(dk), static_cast<const void *>(dv),
                        static_cast<const void *>(dS_init), static_cast<const void *>(S_init),
                        static_cast<const void *>(workspace)})
    if (p && !aligned_to(p, 16)) return ESA_ERR_ALIGN;
  for (const void *p : {static_cast<const void *>(da), static_cast<const void *>(db)})
    if (p && !aligned_to(p, elem(dtype))) return ESA_ERR_ALIGN;
  if (!workspace || workspace_bytes < esa_delta_workspace_size(B, T, H, D, dtype, 1)) return ESA_ERR_WORKSPACE;
  if ((rc = check_current_device())) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B == 0) return ESA_OK;
  if (T == 0) return copy_state(dS_init, dS_final, s, st);
  unsigned char *base = static_cast<unsigned char *>(workspace);
  if (chunked(s, dtype, true)) {
    ChunkArgs c{};
    size_t total;
    c.s = s;
    c.w = chunk_arrays(base, s, dtype, true, &total);
    c.q = q; c.k = k; c.v = v; c.a = a; c.b = b; c.dy = dy;
    c.dq = dq; c.dk = dk; c.dv = dv; c.da = da; c.db = db;
    c.S_in = dS_final;
    c.S_out = dS_init;
    c.keep = true;
    c.iscale = 1.0f / s.scale;   // not used where the scale is zero
    if ((rc = launch_chunk_bwd(dtype, c, st))) return rc;
    return launch_chunk_grad(dtype, c, st);
  }
  const DeltaLayout lo = delta_layout(s, dtype, true);
  SweepArgs p{};
  p.s = s;
  p.q = q; p.k = k; p.v = v; p.dy = dy; p.a = a; p.b = b;
  p.u = reinterpret_cast<float *>(base + lo.u);
  p.du = reinterpret_cast<float *>(base + lo.du);
  p.dk = reinterpret_cast<float *>(base + lo.dk);
  p.dk2 = reinterpret_cast<float *>(base + lo.dk2);
  p.dq = reinterpret_cast<float *>(base + lo.dq);
  p.end = reinterpret_cast<float *>(base + lo.end);
  p.S_ck = reinterpret_cast<float *>(base + lo.S_ck);
  p.dS_ck = reinterpret_cast<float *>(base + lo.dS_ck);
  p.nc = lo.nc;
  p.S_in = dS_final;
  p.S_out = dS_init;
  if (lo.cut) {
    between(&p, lo, base);
    if ((rc = launch_delta_states(true, p, st))) return rc;
  }
  if ((rc = launch_sweep(kSweepDu, dtype, p, st))) return rc;
  if ((rc = launch_sweep(kSweepDk, dtype, p, st))) return rc;
  FinishArgs f{};
  f.s = s;
  f.nc = lo.nc;
  f.q = q; f.k = k; f.v = v; f.a = a; f.b = b; f.dy = dy;
  f.u = p.u; f.du = p.du; f.dkf = p.dk; f.dk2 = p.dk2; f.dqf = p.dq; f.end = p.end;
  f.S_ck = p.S_ck; f.dS_ck = p.dS_ck;
  f.gain = reinterpret_cast<float *>(base + lo.gain);
  f.dq = dq; f.dk = dk; f.dv = dv; f.da = da; f.db = db;
  if ((rc = launch_delta_finish(dtype, f, st))) return rc;
  return launch_delta_gate(dtype, f, st);
}

int esa_delta_step(const void *q_t, const void *k_t, long long ld_qk, const void *v_t, long long ld_v,
                   const void *a_t, const void *b_t, long long ld_g, float *S, void *y_t, int B, int H, int D,
                   float scale, int dtype, void *stream) {
  const DeltaShape s{B, 1, H, D, ld_qk, ld_v, ld_g, normal(scale)};
  int rc = check_inputs(s, dtype, q_t, k_t, v_t, a_t, b_t);
  if (rc) return rc;
  if (B > 0 && (!S || !y_t)) return ESA_ERR_ARG;
  for (const void *p : {static_cast<const void *>(S), static_cast<const void *>(y_t)})
    if (p && !aligned_to(p, 16)) return ESA_ERR_ALIGN;
  if ((rc = check_current_device())) return rc;
  if (B == 0) return ESA_OK;
  SweepArgs p{};
  p.s = s;
  p.q = q_t; p.k = k_t; p.v = v_t; p.a = a_t; p.b = b_t;
  p.S_in = S;
  p.S_out = S;
  p.y = y_t;
  return launch_delta_step(dtype, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
