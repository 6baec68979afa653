// layernorm_f32.cu -- layer norm of inputs in 32 bits, to 16 bits.
#include "layernorm_body.cuh"

namespace atlas {
namespace layernorm {
template <>
int precise<float>(const Args& a, cudaStream_t st);  // layernorm_precise_f32.cu
}  // namespace layernorm
int layernorm_run_f32(const LayerNormArgs& a, cudaStream_t st) {
  const bool to16 = a.ot == ATLAS_BF16 || a.ot == ATLAS_F16;
  return to16 ? layernorm::forward<float, false>(a, st) : layernorm::precise<float>(a, st);
}
}  // namespace atlas
