// s6_scan_f32.cu - the S6 scan on fp32 inputs (s6_scan.cuh).
#include "s6_scan.cuh"

namespace gdn {

cudaError_t launch_s6_f32(const S6Params& p, cudaStream_t stream) {
  return launch_scan<float>(p, stream);
}

}  // namespace gdn
