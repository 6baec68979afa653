// conv_f16.cu -- the short convolution's kernels for f16 elements.
#include "conv_body.cuh"

namespace atlas {
int conv_run_f16(const ConvArgs& a, bool back, cudaStream_t st) {
  return a.wide ? conv::run<__half, 4>(a, back, st) : conv::run<__half, 1>(a, back, st);
}
}  // namespace atlas
