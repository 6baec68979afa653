// layernorm_precise_bf16.cu -- layer norm of inputs in bf16: outputs in 32 and 8 bits, and rows straight from memory.
#include "layernorm_body.cuh"

namespace atlas {
namespace layernorm {
template <>
int precise<__nv_bfloat16>(const Args& a, cudaStream_t st) {
  return forward<__nv_bfloat16, true>(a, st);
}
}  // namespace layernorm
}  // namespace atlas
