// conv_f32.cu -- the short convolution's kernels for f32 elements.
#include "conv_body.cuh"

namespace atlas {
int conv_run_f32(const ConvArgs& a, bool back, cudaStream_t st) {
  return a.wide ? conv::run<float, 4>(a, back, st) : conv::run<float, 1>(a, back, st);
}
}  // namespace atlas
