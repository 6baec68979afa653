// glr.cu -- the gated linear recurrence: choice of the element type's kernels and workspace.
#include "glr_body.cuh"

namespace atlas {

int glr_run_f32(const GlrArgs& a, bool back, cudaStream_t st);
int glr_run_bf16(const GlrArgs& a, bool back, cudaStream_t st);
int glr_run_f16(const GlrArgs& a, bool back, cudaStream_t st);

static int glr_run(const GlrArgs& a, bool back, cudaStream_t st) {
  if (a.type == ATLAS_BF16) return glr_run_bf16(a, back, st);
  if (a.type == ATLAS_F16) return glr_run_f16(a, back, st);
  return glr_run_f32(a, back, st);
}

int glr_forward_launch(const GlrArgs& a, cudaStream_t st) { return glr_run(a, false, st); }
int glr_backward_launch(const GlrArgs& a, cudaStream_t st) { return glr_run(a, true, st); }

// Tickets and words' places are 32-bit.
bool glr_covered(const GlrArgs& a) {
  return a.s.B <= 65535 && glr::tiles_of(a) + 1 <= 0x7FFFFFFFL / glr::groups_of(a);
}
size_t glr_workspace(const GlrArgs& a) {
  if (!a.s.start && a.s.L == 1) return 0;
  return glr::space(a, false, false).bytes;
}
// (Whether the forward's states come with the call is known at the call.)
size_t glr_backward_workspace(const GlrArgs& a) { return glr::space(a, true, true).bytes; }
size_t glr_kept(const GlrArgs& a) { return (size_t)glr::tiles_of(a) * a.D * 4; }

}  // namespace atlas
