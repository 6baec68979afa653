// scan_bwd_f16.cu -- the selective scan's backward kernels for f16 elements.
#include "scan_bwd_body.cuh"

namespace atlas {
int scan_back_f16(const ScanArgs& a, cudaStream_t st) {
  return a.wide ? scan::backward_n<__half, 8>(a, st) : scan::backward_n<__half, 1>(a, st);
}
}  // namespace atlas
