// glr_fwd_f32.cu - the gated linear recurrence in fp32.
#include "glr_fwd.cuh"

namespace gdn {

cudaError_t launch_glr_f32(const GlrParams& p, bool step, cudaStream_t stream) {
  return launch_type<float>(p, step, stream);
}

}  // namespace gdn
