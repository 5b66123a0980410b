// glr_bwd_f32.cu - the gated linear recurrence's gradient in fp32.
#include "glr_bwd.cuh"

namespace gdn {

cudaError_t launch_glr_bwd_f32(const GlrParams& p, cudaStream_t stream) {
  return launch_type<float>(p, stream);
}

}  // namespace gdn
