// scan_f32.cu -- the selective scan's forward kernels for f32 elements.
#include "scan_body.cuh"

namespace atlas {
int scan_run_f32(const ScanArgs& a, cudaStream_t st) {
  return a.wide ? scan::forward_n<float, 4>(a, st) : scan::forward_n<float, 1>(a, st);
}
}  // namespace atlas
