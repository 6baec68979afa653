// scan_bf16.cu -- the selective scan's forward kernels for bf16 elements.
#include "scan_body.cuh"

namespace atlas {
int scan_run_bf16(const ScanArgs& a, cudaStream_t st) {
  return a.wide ? scan::forward_n<__nv_bfloat16, 8>(a, st) : scan::forward_n<__nv_bfloat16, 1>(a, st);
}
}  // namespace atlas
