// scan_f16.cu -- the selective scan's forward kernels for f16 elements.
#include "scan_body.cuh"

namespace atlas {
int scan_run_f16(const ScanArgs& a, cudaStream_t st) {
  return a.wide ? scan::forward_n<__half, 8>(a, st) : scan::forward_n<__half, 1>(a, st);
}
}  // namespace atlas
