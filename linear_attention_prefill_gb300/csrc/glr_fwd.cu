// glr_fwd.cu - the gated linear recurrence in bf16, and the choice of the type.
#include "glr_fwd.cuh"

namespace gdn {

cudaError_t launch_glr(const GlrParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_glr_f32(p, false, stream) : launch_type<__nv_bfloat16>(p, false, stream);
}
cudaError_t launch_glr_step(const GlrParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_glr_f32(p, true, stream) : launch_type<__nv_bfloat16>(p, true, stream);
}

}  // namespace gdn
