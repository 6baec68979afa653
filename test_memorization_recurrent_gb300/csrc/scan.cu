// scan.cu -- the selective scan: choice of the element type's kernels and workspace.
#include "scan_bwd_body.cuh"

namespace atlas {

int scan_run_f32(const ScanArgs& a, cudaStream_t st);
int scan_run_bf16(const ScanArgs& a, cudaStream_t st);
int scan_run_f16(const ScanArgs& a, cudaStream_t st);
int scan_back_f32(const ScanArgs& a, cudaStream_t st);
int scan_back_bf16(const ScanArgs& a, cudaStream_t st);
int scan_back_f16(const ScanArgs& a, cudaStream_t st);

int scan_forward_launch(const ScanArgs& a, cudaStream_t st) {
  if (a.type == ATLAS_BF16) return scan_run_bf16(a, st);
  if (a.type == ATLAS_F16) return scan_run_f16(a, st);
  return scan_run_f32(a, st);
}

int scan_backward_launch(const ScanArgs& a, cudaStream_t st) {
  if (a.type == ATLAS_BF16) return scan_back_bf16(a, st);
  if (a.type == ATLAS_F16) return scan_back_f16(a, st);
  return scan_back_f32(a, st);
}

size_t scan_workspace(const ScanArgs& a) {
  if (!a.s.start && a.s.L == 1) return 0;
  if (a.N <= 8) return scan::workspace<2>(a);
  if (a.N <= 16) return scan::workspace<4>(a);
  if (a.N <= 32) return scan::workspace<8>(a);
  if (a.N <= 64) return scan::workspace<16>(a);
  return scan::workspace<32>(a);
}

size_t scan_backward_workspace(const ScanArgs& a) {
  if (a.N <= 8) return scan::Back<2>(a, nullptr).bytes;
  if (a.N <= 16) return scan::Back<4>(a, nullptr).bytes;
  if (a.N <= 32) return scan::Back<8>(a, nullptr).bytes;
  if (a.N <= 64) return scan::Back<16>(a, nullptr).bytes;
  return scan::Back<32>(a, nullptr).bytes;
}

}  // namespace atlas
