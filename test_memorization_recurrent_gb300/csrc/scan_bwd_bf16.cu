// scan_bwd_bf16.cu -- the selective scan's backward kernels for bf16 elements.
#include "scan_bwd_body.cuh"

namespace atlas {
int scan_back_bf16(const ScanArgs& a, cudaStream_t st) {
  return a.wide ? scan::backward_n<__nv_bfloat16, 8>(a, st) : scan::backward_n<__nv_bfloat16, 1>(a, st);
}
}  // namespace atlas
