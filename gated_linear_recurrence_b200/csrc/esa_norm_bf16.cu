// esa_norm_bf16.cu -- layer norm instantiations for bf16 rows.
#include "esa_norm_ragged.cuh"

namespace esa {
int norm_fwd_bf16(int vec, bool wide, const NormFwdArgs &a, cudaStream_t st) {
  return wide ? norm_fwd_typed<__nv_bfloat16, float>(vec, a, st) : norm_fwd_typed<__nv_bfloat16, __nv_bfloat16>(vec, a, st);
}
int norm_bwd_bf16(int vec, bool wide, const NormBwdArgs &a, int most, cudaStream_t st) {
  return wide ? norm_bwd_typed<__nv_bfloat16, float>(vec, a, most, st) : norm_bwd_typed<__nv_bfloat16, __nv_bfloat16>(vec, a, most, st);
}
}  // namespace esa
