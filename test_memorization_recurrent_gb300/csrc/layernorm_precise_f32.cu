// layernorm_precise_f32.cu -- layer norm of inputs in 32 bits: outputs in 32 and 8 bits, and rows straight from memory.
#include "layernorm_body.cuh"

namespace atlas {
namespace layernorm {
template <>
int precise<float>(const Args& a, cudaStream_t st) {
  return forward<float, true>(a, st);
}
}  // namespace layernorm
}  // namespace atlas
