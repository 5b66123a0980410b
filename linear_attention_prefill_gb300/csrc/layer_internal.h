// layer_internal.h - launch parameters of the layer operators (short convolution, S6 scan,
// RMS norm, gated linear recurrence, layer norm, rotary positions), shared by their C ABI layer
// (layer_abi.cu, glr_abi.cu, layer_norm_abi.cu, rotary_abi.cu) and the kernels.
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

// Gated linear recurrence: prompt, its gradient, or one token (h0 == hT, T = 1).
enum { GLR_LOG = 0, GLR_SIGMOID = 1, GLR_RATE = 2 };    // as GDN_GLR_GATE_*
enum { GLR_NONE = 0, GLR_LINEAR = 1, GLR_SQRT = 2 };    // as GDN_GLR_INPUT_*
constexpr int kGlrChunk = 64;                           // tokens between the states that are kept
constexpr int kGlrFwdRun = 16, kGlrFwdWarps = 4, kGlrFwdBlocks = 4;  // tokens of a thread, warps of a block,
constexpr int kGlrBwdRun = 16, kGlrBwdWarps = 4, kGlrBwdBlocks = 3;   // blocks an SM (bf16; one of fp32)
constexpr int kGlrMaxCluster = 16;
struct GlrParams {
  const void *x, *g, *dy;           // rows of D channels; dy: gradient only
  const float *rate;                // [D], GLR_RATE only
  const float *h0, *dhT, *kept;     // [N, D] or nullptr; kept: the forward's states, gradient only
  void *y, *dx, *dg;                // [tokens, D]
  float *hT, *states, *dh0;         // [N, D], [rows, chunks, D], [N, D]; nullptr for none
  float *drate, *partial;           // [D] and [rows * cluster, D]: the rate's gradient, its blocks' sums
  const int32_t* cu;                // [N + 1] or nullptr (N rows of T tokens)
  long long x_stride, g_stride, dy_stride;  // elements from token to token
  long long chunks;                 // 64-token chunks of a row, the last one partial
  int N, T, D;
  int gate, norm;
  int vec;                          // channel pairs are aligned in every tensor, D is even
  int piece;                        // rows are made of, and aligned to, 16, 4 or 2 bytes
  unsigned* err;                    // device error word: bounded waits record a timeout here (set
                                    // by the launch that has them)
  int tiles;                        // of 64 channels
  int cluster;                      // blocks of a cluster: successive tokens (set by the launch)
};
inline long long glr_units(const GlrParams& p) { return (p.cu ? 1ll : p.N) * p.tiles; }
// at most so many blocks a cluster
inline int glr_most_blocks(const GlrParams& p) {
  const int span = kGlrBwdRun * kGlrBwdWarps;
  return p.T <= span ? 1 : p.T > span * (kGlrMaxCluster - 1) ? kGlrMaxCluster : (p.T - 1) / span + 1;
}
inline unsigned glr_grid(const GlrParams& p) { return (unsigned)(glr_units(p) * p.cluster); }
cudaError_t launch_glr_f32(const GlrParams& p, bool step, cudaStream_t stream);
cudaError_t launch_glr_bwd_f32(const GlrParams& p, cudaStream_t stream);
cudaError_t launch_glr(const GlrParams& p, bool f32, cudaStream_t stream);
cudaError_t launch_glr_bwd(const GlrParams& p, bool f32, cudaStream_t stream);
cudaError_t launch_glr_step(const GlrParams& p, bool f32, cudaStream_t stream);
// The sums over the rows of in [rows, D] into a, or of in [rows, 2, D] into a and b; in a fixed order.
cudaError_t launch_column_sums(const float* in, float* a, float* b, int rows, int D, cudaStream_t stream);

// Layer norm of rows, or its gradient (dy; residual: the gradient added to dx; y: dx).
struct LnParams {
  const void *x, *dy, *residual;    // residual: nullptr for none
  const float *w, *b;               // [D]; nullptr for ones and zeros
  void *y, *residual_out;
  float *dw, *db;                   // [D], both or neither
  float* partial;                   // [blocks, 2, D], with dw: ln_partials(D) of them are enough
  long long rows, x_stride, dy_stride;
  int D;
  int blocks, slice;                // blocks of a row (1, 2 or 4), columns of each
  int whole;                        // vectors of 8 columns: D is a multiple, all are 16 bytes aligned
  float eps, inv_d;
  unsigned* err;                    // device error word: bounded waits record a timeout here (set
                                    // by the launch that has them)
};
constexpr int kLnMaxD = 32768, kLnMaxThreads = 1024, kLnSlice = 8 * kLnMaxThreads;
inline int ln_partials(int D) { return (D <= 2560 ? 8 : 2) * kSms; }
cudaError_t launch_layer_norm(const LnParams& p, bool f32, cudaStream_t stream);
cudaError_t launch_layer_norm_bwd(const LnParams& p, bool f32, cudaStream_t stream);

// Rotary positions of q and k (k: nullptr and Hk = 0 for none).
struct RotaryParams {
  const void *q, *k;                // tokens of Hq, Hk heads of D columns
  void *q_out, *k_out;
  const unsigned long long* turns;  // [R / 2]: 2^64 is a whole turn
  const int32_t *positions;         // [tokens], or nullptr: counted from a sequence's first token
  const int32_t *offsets, *cu;      // [N] or nullptr (zeros), [N + 1] or nullptr (N rows of T)
  long long q_stride, k_stride, q_out_stride, k_out_stride, tokens;  // elements from token to token
  int N, T, Hq, Hk, D, R;
  int interleaved, backward;
  int by;                           // elements of an access (16 bytes at most): they divide R / 2 and D - R, and
                                    // are aligned everywhere
  int q_same, k_same;               // the output is the input
  int block_tokens;                 // set by the launch
  float magnitude;
};
constexpr int kRotaryMaxD = 1024;
cudaError_t launch_rotary(const RotaryParams& p, bool f32, cudaStream_t stream);

}  // namespace gdn
