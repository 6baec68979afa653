// layernorm_precise_f16.cu -- layer norm of inputs in fp16: outputs in 32 and 8 bits, and rows straight from memory.
#include "layernorm_body.cuh"

namespace atlas {
namespace layernorm {
template <>
int precise<__half>(const Args& a, cudaStream_t st) {
  return forward<__half, true>(a, st);
}
}  // namespace layernorm
}  // namespace atlas
