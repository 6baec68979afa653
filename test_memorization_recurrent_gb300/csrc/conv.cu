// conv.cu -- the short convolution: choice of the element type's kernels and workspace.
#include "conv_body.cuh"

namespace atlas {

int conv_run_f32(const ConvArgs& a, bool back, cudaStream_t st);
int conv_run_bf16(const ConvArgs& a, bool back, cudaStream_t st);
int conv_run_f16(const ConvArgs& a, bool back, cudaStream_t st);

static int conv_run(const ConvArgs& a, bool back, cudaStream_t st) {
  if (a.dt == ATLAS_BF16) return conv_run_bf16(a, back, st);
  if (a.dt == ATLAS_F16) return conv_run_f16(a, back, st);
  return conv_run_f32(a, back, st);
}

int conv_forward_launch(const ConvArgs& a, cudaStream_t st) { return conv_run(a, false, st); }
int conv_backward_launch(const ConvArgs& a, cudaStream_t st) { return conv_run(a, true, st); }

// States' gradients, then the partial sums of dw and db; whether the wide kernels run is
// known at the call, so the larger of both counts.
size_t conv_backward_workspace(const ConvArgs& a) {
  size_t most = 0;
  for (int V : {1, 4}) {
    const long share = seq_share(a.s, conv::workers(a, V, conv::kBackWarps), 1);
    const size_t n = (size_t)conv::blocks_of(a, share) * (a.W + 1) * a.C;
    most = n > most ? n : most;
  }
  return (most + (size_t)a.s.B * (a.W - 1) * a.C) * 4;
}

}  // namespace atlas
