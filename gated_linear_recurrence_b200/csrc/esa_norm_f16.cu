// esa_norm_f16.cu -- layer norm instantiations for f16 rows.
#include "esa_norm_ragged.cuh"

namespace esa {
int norm_fwd_f16(int vec, bool wide, const NormFwdArgs &a, cudaStream_t st) {
  return wide ? norm_fwd_typed<__half, float>(vec, a, st) : norm_fwd_typed<__half, __half>(vec, a, st);
}
int norm_bwd_f16(int vec, bool wide, const NormBwdArgs &a, int most, cudaStream_t st) {
  return wide ? norm_bwd_typed<__half, float>(vec, a, most, st) : norm_bwd_typed<__half, __half>(vec, a, most, st);
}
}  // namespace esa
