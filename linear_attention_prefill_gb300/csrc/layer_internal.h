// layer_internal.h - launch parameters of the layer operators (short convolution, S6 scan,
// RMS norm), shared by their C ABI layer (layer_abi.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Short causal convolution over tokens, one filter per channel.
struct ConvParams {
  const void* x;      // rows of D channels, x_stride elements from token to token
  const float* w;     // [D, W]
  const float* bias;  // [D] or nullptr
  const void* s0;     // [N, W - 1, D] or nullptr (zeros)
  void* y;            // [tokens, D]
  void* sT;           // [N, W - 1, D] or nullptr
  const int32_t* cu;  // [N + 1] or nullptr (N rows of T tokens)
  long long x_stride;
  int N, T, D, W;
  int silu;
  int vec;            // every 8-channel access is 16-byte aligned and D is a multiple of 8
};
cudaError_t launch_conv(const ConvParams& p, bool f32, cudaStream_t stream);
// One token per sequence: s0 == sT, updated in place; T = 1, cu = nullptr.
cudaError_t launch_conv_step(const ConvParams& p, bool f32, cudaStream_t stream);

// Selective state space scan, prompt or one token.
struct S6Params {
  const void *x, *dt, *B, *C, *z;   // x, dt, z: D channels; B, C: Ns states; z may be nullptr
  const float *A, *D, *dt_bias;     // [D, Ns], [D] or nullptr, [D] or nullptr
  const float* h0;                  // [N, D, Ns] or nullptr (zeros)
  void* y;                          // [tokens, D]
  float* hT;                        // [N, D, Ns] or nullptr
  const int32_t* cu;                // [N + 1] or nullptr (N rows of T tokens)
  long long x_stride, dt_stride, b_stride, c_stride, z_stride;  // elements from token to token
  int N, T, dim, Ns;
  int softplus;
  int vec2;                         // channel pairs of x, dt, z, y are aligned, dim is even
  int vec_bc;                       // four states of B and of C are aligned, Ns % 4 == 0
  // the split over time: chunks of `chunk` tokens (a multiple of 32) per sequence, their
  // summaries in the workspace; chunk = 0: whole sequences
  int chunk;
  int slots;                        // chunk slots (chunk > 0)
  float* ws_sum;                    // [slots, dim]: the chunk's sum of steps
  float* ws_h;                      // [slots, dim, Ns]: the state after it, from zero (first: from h0)
  float* ws_h0;                     // [N, dim, Ns]: h0 kept for the scan when hT == h0, else nullptr
};
// Chunk length the scan takes for these sizes (0: no split), and the slots it has then.
int s6_chunk(int N, int T, int dim, int Ns, bool packed);
long long s6_slots(int N, int T, int chunk, bool packed);
// Workspace bytes of that split, the copy of h0 included; 0 without one.
size_t s6_ws_bytes(int N, int T, int dim, int Ns, bool packed);
cudaError_t launch_s6(const S6Params& p, bool f32, cudaStream_t stream);
cudaError_t launch_s6_step(const S6Params& p, bool f32, cudaStream_t stream);

// RMS norm of rows, optional residual addition, output gate and e4m3 output.
struct NormParams {
  const void *x, *residual, *gate;  // residual, gate: nullptr for none
  const float* w;                   // [D]
  void *y, *residual_out;           // residual_out: nullptr without a residual
  float* scales;                    // e4m3 output only: [tokens * heads, ceil(D / group)]
  long long rows;                   // tokens * heads
  long long x_stride, gate_stride;  // elements from token to token
  int heads, D;
  int group;                        // columns per scale; D for one scale a row
  float eps;
  int vec;                          // every 8-column access is aligned and D is a multiple of 8
};
constexpr int kNormMaxD = 32768;
cudaError_t launch_norm(const NormParams& p, bool f32, bool fp8, cudaStream_t stream);

}  // namespace gdn
