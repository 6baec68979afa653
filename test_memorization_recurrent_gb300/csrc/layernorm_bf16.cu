// layernorm_bf16.cu -- layer norm of inputs in bf16, to 16 bits.
#include "layernorm_body.cuh"

namespace atlas {
namespace layernorm {
template <>
int precise<__nv_bfloat16>(const Args& a, cudaStream_t st);  // layernorm_precise_bf16.cu
}  // namespace layernorm
int layernorm_run_bf16(const LayerNormArgs& a, cudaStream_t st) {
  const bool to16 = a.ot == ATLAS_BF16 || a.ot == ATLAS_F16;
  return to16 ? layernorm::forward<__nv_bfloat16, false>(a, st) : layernorm::precise<__nv_bfloat16>(a, st);
}
}  // namespace atlas
