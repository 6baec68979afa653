// layernorm_f16.cu -- layer norm of rows in fp16.
#include "layernorm_body.cuh"

namespace atlas {
int layernorm_run_f16(const LayerNormArgs& a, cudaStream_t st) { return layernorm::forward<__half>(a, st); }
}  // namespace atlas
