// layer_internal.h - launch parameters of the layer operators (short convolution, S6 scan,
// RMS norm), shared by their C ABI layer (layer_abi.cu) and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

constexpr int kSms = 152;

// Address of the device error word on the current device (gdn_abi.cu).
cudaError_t device_error_word(unsigned** out);

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
  int vec;            // 4-channel pieces are aligned (8 bytes of bf16, 16 of fp32), D % 4 == 0
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
  int copy;                         // x, dt, z rows: 16-byte pieces, 4-byte words or 2-byte elements
  int copy_bc;                      // four states of B and of C: 16 (fp32) or 8 bytes, words, elements
  int vec2;                         // channel pairs of y are aligned, dim is even
  int vec_bc;                       // four states of B and of C are aligned, Ns % 4 == 0
  int lone;                         // the variant for one CTA an SM (s6_split)
  // the split over time (s6_split): channels from 32 * whole on run in chunks of `chunk`
  // tokens per sequence, with summaries in the workspace; chunk = 0: no channel does
  int whole, chunk, slots;
  float* ws_sum;                    // [slots, split channels]: the chunk's sum of steps
  float* ws_h;                      // [slots, split channels, Ns]: the state after it, from zero
                                    // (a first chunk: from h0)
  float* ws_h0;                     // [N, split channels, Ns]: h0 kept where hT == h0, else nullptr
};
// How the scan runs for these sizes: 32-channel tiles that walk whole sequences, and the
// chunks, slots and workspace (256-byte aligned pieces) of the others; chunk = 0 without.
struct S6Split {
  int whole, chunk, lone;
  long long slots;
  size_t sum_floats, h_floats, ws_bytes;
};
S6Split s6_split(int N, int T, int dim, int Ns, bool packed);
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
  int group, groups;                // columns per scale (D: one scale a row), scales a row
  int group_log;                    // log2 of a group below D
  float eps, inv_d;                 // inv_d: 1 / D
  int by;                           // columns of an access (8, 4, 2, 1): D is a multiple, all are aligned
  unsigned* err;                    // device error word: bounded waits record a timeout here (set
                                    // by the launch that has them)
};
constexpr int kNormMaxD = 32768;
cudaError_t launch_norm(const NormParams& p, bool f32, bool fp8, cudaStream_t stream);

}  // namespace gdn
