// conv_bf16.cu -- the short convolution's kernels for bf16 elements.
#include "conv_body.cuh"

namespace atlas {
int conv_run_bf16(const ConvArgs& a, bool back, cudaStream_t st) {
  return a.wide ? conv::run<__nv_bfloat16, 4>(a, back, st) : conv::run<__nv_bfloat16, 1>(a, back, st);
}
}  // namespace atlas
