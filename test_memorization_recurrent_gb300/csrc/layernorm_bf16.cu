// layernorm_bf16.cu -- layer norm of rows in bf16.
#include "layernorm_body.cuh"

namespace atlas {
int layernorm_run_bf16(const LayerNormArgs& a, cudaStream_t st) { return layernorm::forward<__nv_bfloat16>(a, st); }
}  // namespace atlas
