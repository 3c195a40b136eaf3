// esa_delta_sweep.cu -- instantiations and launchers of the token-by-token
// gated delta rule kernels.
#include "esa_delta_sweep.cuh"

#include "esa.h"
#include "esa_host.h"

namespace esa {
namespace {

// Warps per block: all of a head's when whole heads (or chunks of them) give
// every SM two blocks, else fewer, so that a small batch still spreads over
// the device.
int sweep_warps(long long units, int most) {
  int W = most;
  while (W > 1 && units * (most / W) < 2 * sm_count()) W >>= 1;
  return W;
}

template <typename T, int D, int KIND>
int run(const SweepArgs &a, cudaStream_t st) {
  const long long heads = static_cast<long long>(a.s.B) * a.s.H;
  const long long units = a.cut ? heads * a.nc : heads;
  const int W = sweep_warps(units, D / sweep::columns<D>());
  const sweep::Layout<T, D, KIND> lo(W);
  auto kern = sweep::delta_sweep_kernel<T, D, KIND>;
  if (lo.total > 48 * 1024) {
    const int rc = runtime_status(
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lo.total)));
    if (rc) return rc;
  }
  kern<<<static_cast<unsigned>(units * (D / lo.cols)), W * 32, lo.total, st>>>(a);
  return runtime_status(cudaGetLastError());
}

template <typename T, int D>
int run_keys(const SweepArgs &a, cudaStream_t st) {
  const long long units = static_cast<long long>(a.s.B) * a.s.H * a.nc;
  const int W = sweep_warps(units, D / sweep::columns<D>());
  const sweep::Layout<T, D, kSweepDk> lo(W);
  const size_t other = sweep::Layout<T, D, kSweepDq>(W).total, bytes = lo.total > other ? lo.total : other;
  auto kern = sweep::delta_keys_kernel<T, D>;
  if (bytes > 48 * 1024) {
    const int rc =
        runtime_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)));
    if (rc) return rc;
  }
  kern<<<dim3(static_cast<unsigned>(units * (D / lo.cols)), 2), W * 32, bytes, st>>>(a);
  return runtime_status(cudaGetLastError());
}

template <typename T, int D>
int by_kind(int kind, const SweepArgs &a, cudaStream_t st) {
  switch (kind) {
    case kSweepFwd: return run<T, D, kSweepFwd>(a, st);
    case kSweepDu: return run<T, D, kSweepDu>(a, st);
    default: return run_keys<T, D>(a, st);
  }
}

template <typename T>
int by_d(int kind, const SweepArgs &a, cudaStream_t st) {
  switch (a.s.D) {
    case 32: return by_kind<T, 32>(kind, a, st);
    case 64: return by_kind<T, 64>(kind, a, st);
    case 128: return by_kind<T, 128>(kind, a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

template <typename T>
int finish(const FinishArgs &a, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.s.B) * a.s.T * a.s.H;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  switch (a.s.D) {
    case 32: sweep::delta_finish_kernel<T, 32><<<grid, 256, 0, st>>>(a); break;
    case 64: sweep::delta_finish_kernel<T, 64><<<grid, 256, 0, st>>>(a); break;
    case 128: sweep::delta_finish_kernel<T, 128><<<grid, 256, 0, st>>>(a); break;
    default: return ESA_ERR_UNSUPPORTED;
  }
  return runtime_status(cudaGetLastError());
}

}  // namespace

int launch_sweep(int kind, int dtype, const SweepArgs &a, cudaStream_t st) {
  switch (dtype) {
    case ESA_F32: return by_d<float>(kind, a, st);
    case ESA_F16: return by_d<__half>(kind, a, st);
    case ESA_BF16: return by_d<__nv_bfloat16>(kind, a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

int launch_delta_finish(int dtype, const FinishArgs &a, cudaStream_t st) {
  switch (dtype) {
    case ESA_F32: return finish<float>(a, st);
    case ESA_F16: return finish<__half>(a, st);
    case ESA_BF16: return finish<__nv_bfloat16>(a, st);
    default: return ESA_ERR_UNSUPPORTED;
  }
}

}  // namespace esa
