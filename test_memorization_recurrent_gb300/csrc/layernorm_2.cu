// layernorm_2.cu -- layer norm of rows in 16 bits.
#include "layernorm_body.cuh"

namespace atlas {
int layernorm_run_2(const LayerNormArgs& a, cudaStream_t st) { return layernorm::forward<2>(a, st); }
}  // namespace atlas
