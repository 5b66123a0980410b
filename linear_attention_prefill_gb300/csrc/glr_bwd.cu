// glr_bwd.cu - the gated linear recurrence's gradient in bf16, and the choice of the type.
#include "glr_bwd.cuh"

namespace gdn {

cudaError_t launch_glr_bwd(const GlrParams& p, bool f32, cudaStream_t stream) {
  return f32 ? launch_glr_bwd_f32(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
