// layernorm_4.cu -- layer norm of rows in 32 bits.
#include "layernorm_body.cuh"

namespace atlas {
int layernorm_run_4(const LayerNormArgs& a, cudaStream_t st) { return layernorm::forward<4>(a, st); }
}  // namespace atlas
