// glr_bf16.cu -- the gated linear recurrence for bf16 elements.
#include "glr_body.cuh"

namespace atlas {
int glr_run_bf16(const GlrArgs& a, bool back, cudaStream_t st) { return glr::run<__nv_bfloat16>(a, back, st); }
}  // namespace atlas
