// layernorm_f16.cu -- layer norm of inputs in fp16, to 16 bits.
#include "layernorm_body.cuh"

namespace atlas {
namespace layernorm {
template <>
int precise<__half>(const Args& a, cudaStream_t st);  // layernorm_precise_f16.cu
}  // namespace layernorm
int layernorm_run_f16(const LayerNormArgs& a, cudaStream_t st) {
  const bool to16 = a.ot == ATLAS_BF16 || a.ot == ATLAS_F16;
  return to16 ? layernorm::forward<__half, false>(a, st) : layernorm::precise<__half>(a, st);
}
}  // namespace atlas
