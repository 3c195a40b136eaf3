// esa_norm_f32.cu -- layer norm instantiations for float32 rows.
#include "esa_norm_ragged.cuh"

namespace esa {
int norm_fwd_f32(int vec, const NormFwdArgs &a, cudaStream_t st) {
  return norm_fwd_typed<float, float>(vec, a, st);
}
int norm_bwd_f32(int vec, const NormBwdArgs &a, int most, cudaStream_t st) {
  return norm_bwd_typed<float, float>(vec, a, most, st);
}
}  // namespace esa
