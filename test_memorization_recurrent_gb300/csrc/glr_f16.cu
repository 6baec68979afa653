// glr_f16.cu -- the gated linear recurrence for fp16 elements.
#include "glr_body.cuh"

namespace atlas {
int glr_run_f16(const GlrArgs& a, bool back, cudaStream_t st) { return glr::run<__half>(a, back, st); }
}  // namespace atlas
