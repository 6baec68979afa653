// glr_f32.cu -- the gated linear recurrence for fp32 elements.
#include "glr_body.cuh"

namespace atlas {
int glr_run_f32(const GlrArgs& a, bool back, cudaStream_t st) { return glr::run<float>(a, back, st); }
}  // namespace atlas
