// layernorm_f32.cu -- layer norm of rows in fp32.
#include "layernorm_body.cuh"

namespace atlas {
int layernorm_run_f32(const LayerNormArgs& a, cudaStream_t st) { return layernorm::forward<float>(a, st); }
}  // namespace atlas
