// glr_bwd.cu - the gated linear recurrence's gradient in bf16, and the choice of the type.
#include "glr_bwd.cuh"

namespace gdn {

cudaError_t launch_glr_bwd(GlrParams p, bool f32, cudaStream_t stream) {
  const cudaError_t e = p.cluster > 1 ? device_error_word(&p.err) : cudaSuccess;
  if (e != cudaSuccess) return e;
  return f32 ? launch_glr_bwd_f32(p, stream) : launch_type<__nv_bfloat16>(p, stream);
}

}  // namespace gdn
