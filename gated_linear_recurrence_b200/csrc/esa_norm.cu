// esa_norm.cu -- C ABI of the layer norm (declared in include/esa.h): checks,
// the vector width and the threads of a row, dispatch on the I/O type.
#include <climits>
#include <cstddef>
#include <initializer_list>

#include "esa.h"
#include "esa_host.h"
#include "esa_norm.h"

namespace esa {
namespace {

int elem(int dtype) { return dtype == ESA_F32 ? 4 : 2; }

// Elements per vector: 16 or 8 bytes of the I/O type if that divides N and every
// row stride and suits every pointer's alignment, else one element.
int pick_vec(int dtype, int wdtype, int N, std::initializer_list<long long> lds, std::initializer_list<const void *> io,
             std::initializer_list<const void *> wt) {
  for (int bytes = 16; bytes >= 8; bytes >>= 1) {
    const int vec = bytes / elem(dtype);
    bool ok = N % vec == 0;
    for (long long ld : lds) ok = ok && ld % vec == 0;
    for (const void *p : io) ok = ok && (p == nullptr || aligned_to(p, bytes));
    const int wbytes = vec * elem(wdtype) > 16 ? 16 : vec * elem(wdtype);
    for (const void *p : wt) ok = ok && (p == nullptr || aligned_to(p, wbytes));
    if (ok) return vec;
  }
  return 1;
}

int check_norm(long long rows, int N, int dtype, int wdtype) {
  if (rows < 0 || N < 1) return ESA_ERR_ARG;
  if (dtype < ESA_F32 || dtype > ESA_E4M3 || wdtype < ESA_F32 || wdtype > ESA_E4M3) return ESA_ERR_ARG;
  if (dtype == ESA_E4M3 || wdtype == ESA_E4M3) return ESA_ERR_UNSUPPORTED;
  if (wdtype != ESA_F32 && wdtype != dtype) return ESA_ERR_UNSUPPORTED;
  if (N > kNormMaxN) return ESA_ERR_UNSUPPORTED;
  if (rows > (1ll << 40) / N) return ESA_ERR_ARG;
  if (rows > INT_MAX) return ESA_ERR_ARG;   // one block, or a share of one, per row
  return ESA_OK;
}

bool bad_ld(long long ld, int N) { return ld < N || ld > INT_MAX; }

// Partial rows of the column sums.
int max_blocks(int N) { return N <= 1024 ? 2368 : 1184; }

}  // namespace
}  // namespace esa

using namespace esa;

extern "C" {

size_t esa_norm_workspace_size(long long rows, int N, int dtype, int wdtype) {
  if (check_norm(rows, N, dtype, wdtype) != ESA_OK) return 0;
  const long long most = max_blocks(N), blocks = rows < most ? (rows > 0 ? rows : 1) : most;
  return static_cast<size_t>(blocks) * 2 * N * sizeof(float);
}

int esa_norm_fwd(const void *x, long long ld_x, const void *residual, long long ld_res, const void *weight,
                 const void *bias, void *y, void *h, float *stats, long long rows, int N, float eps, int dtype,
                 int wdtype, void *stream) {
  int rc = check_norm(rows, N, dtype, wdtype);
  if (rc) return rc;
  if (!(eps >= 0.0f) || eps > 1.0e30f) return ESA_ERR_ARG;
  if (bad_ld(ld_x, N) || (residual && bad_ld(ld_res, N))) return ESA_ERR_ARG;
  if (rows > 0 && (!x || !y || (residual && !h))) return ESA_ERR_ARG;
  const unsigned es = elem(dtype), ws = elem(wdtype);
  for (const void *p : {x, residual, static_cast<const void *>(y), static_cast<const void *>(h)})
    if (p && !aligned_to(p, es)) return ESA_ERR_ALIGN;
  for (const void *p : {weight, bias})
    if (p && !aligned_to(p, ws)) return ESA_ERR_ALIGN;
  if (stats && !aligned_to(stats, 8)) return ESA_ERR_ALIGN;
  if ((rc = check_current_device())) return rc;
  if (rows == 0) return ESA_OK;
  const int vec = pick_vec(dtype, wdtype, N, {ld_x, residual ? ld_res : 0}, {x, residual, y, residual ? h : nullptr},
                           {weight, bias});
  NormFwdArgs a{x, residual, weight, bias, y, h, reinterpret_cast<float2 *>(stats), rows, ld_x, ld_res, N, eps,
                static_cast<float>(N)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool wide = wdtype == ESA_F32;
  if (dtype == ESA_F32) return norm_fwd_f32(vec, a, st);
  return dtype == ESA_F16 ? norm_fwd_f16(vec, wide, a, st) : norm_fwd_bf16(vec, wide, a, st);
}

int esa_norm_bwd(const void *dy, long long ld_dy, const void *h, long long ld_h, const void *weight,
                 const float *stats, const void *dh, long long ld_dh, void *dx, void *dweight, void *dbias,
                 long long rows, int N, int dtype, int wdtype, void *workspace, size_t workspace_bytes,
                 void *stream) {
  int rc = check_norm(rows, N, dtype, wdtype);
  if (rc) return rc;
  if (bad_ld(ld_dy, N) || bad_ld(ld_h, N) || (dh && bad_ld(ld_dh, N))) return ESA_ERR_ARG;
  if (rows > 0 && (!dy || !h || !stats || !dx)) return ESA_ERR_ARG;
  const unsigned es = elem(dtype), ws = elem(wdtype);
  for (const void *p : {dy, h, dh, static_cast<const void *>(dx)})
    if (p && !aligned_to(p, es)) return ESA_ERR_ALIGN;
  for (const void *p : {weight, static_cast<const void *>(dweight), static_cast<const void *>(dbias)})
    if (p && !aligned_to(p, ws)) return ESA_ERR_ALIGN;
  if (stats && !aligned_to(stats, 8)) return ESA_ERR_ALIGN;
  const bool sums = dweight || dbias;
  if (sums && workspace && !aligned_to(workspace, 16)) return ESA_ERR_ALIGN;
  if (sums && rows > 0 && (!workspace || workspace_bytes < esa_norm_workspace_size(rows, N, dtype, wdtype)))
    return ESA_ERR_WORKSPACE;
  if ((rc = check_current_device())) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // sums over no rows
    if (dweight && (rc = runtime_status(cudaMemsetAsync(dweight, 0, static_cast<size_t>(N) * ws, st)))) return rc;
    return dbias ? runtime_status(cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * ws, st)) : ESA_OK;
  }
  const int vec = pick_vec(dtype, wdtype, N, {ld_dy, ld_h, dh ? ld_dh : 0}, {dy, h, dh, dx}, {weight});
  const int most = max_blocks(N);
  NormBwdArgs a{dy, h, weight, dh, dx, reinterpret_cast<const float2 *>(stats), dweight, dbias,
                sums ? static_cast<float *>(workspace) : nullptr, rows, ld_dy, ld_h, ld_dh, N,
                static_cast<float>(N)};
  const bool wide = wdtype == ESA_F32;
  if (dtype == ESA_F32) return norm_bwd_f32(vec, a, most, st);
  return dtype == ESA_F16 ? norm_bwd_f16(vec, wide, a, most, st) : norm_bwd_bf16(vec, wide, a, most, st);
}

}  // extern "C"
