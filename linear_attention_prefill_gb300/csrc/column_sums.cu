// column_sums.cu - the sums of partial sums by columns, in a fixed order: the end of a
// parameter's gradient (the recurrence's rate, layer norm's weight and bias).
#include "gdn_common.cuh"
#include "layer_internal.h"

namespace gdn {
namespace {

// 32 columns a block of 32 warps; a warp adds every thirty-second row, then the warps' sums are added
// in order.  Launched as a dependent of the kernel that leaves the partial sums.
constexpr int kWarps = 32;
__global__ void __launch_bounds__(32 * kWarps) column_sums_kernel(const float* in, float* a, float* b, int rows,
                                                                  int D, int all) {
  __shared__ float s[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + lane;
  griddep_wait();
  float sum = 0.f;
  if (c < all) {
#pragma unroll 8
    for (int r = warp; r < rows; r += kWarps) sum += in[(long long)r * all + c];
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < all) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += s[w][lane];
    (c < D ? a + c : b + (c - D))[0] = sum;
  }
}

}  // namespace

cudaError_t launch_column_sums(const float* in, float* a, float* b, int rows, int D, cudaStream_t stream) {
  const int all = b ? 2 * D : D;
  return launch_after(column_sums_kernel, (unsigned)((all - 1) / 32 + 1), 32 * kWarps, 0, stream, in, a, b, rows, D,
                      all);
}

}  // namespace gdn
