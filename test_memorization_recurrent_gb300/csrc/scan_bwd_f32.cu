// scan_bwd_f32.cu -- the selective scan's backward kernels for f32 elements.
#include "scan_bwd_body.cuh"

namespace atlas {
int scan_back_f32(const ScanArgs& a, cudaStream_t st) {
  return a.wide ? scan::backward_n<float, 4>(a, st) : scan::backward_n<float, 1>(a, st);
}
}  // namespace atlas
