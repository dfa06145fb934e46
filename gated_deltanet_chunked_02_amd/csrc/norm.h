// Host-side views of the group norm and of the convolution's backward, shared by the C ABI
// (api_ssm.cpp) and the launchers (group_norm.hip, conv1d_bwd.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

struct NormProblem {
  int N, P, C, G, cpg;  // samples, positions a sample, channels, groups, channels a group
  bool f32, silu;
  bool wide;            // weight and bias are 16-byte aligned (set by the launchers)
  float eps;
  const void* x;
  const float* weight;  // [C] or null (ones)
  const float* bias;    // [C] or null (zeros)
  const void* gate;     // x's shape, or null
  void* y;
  float* mean;          // [N, G]; the forward's may be null
  float* rstd;          // [N, G]; the forward's may be null
  // backward
  const void* dy;
  void* dx;
  void* dgate;          // null without gate
  float* dweight;       // [C] or null
  float* dbias;         // [C] or null
  float* ws;            // workspace, norm_workspace() bytes
};
// Bytes of workspace at p.ws, whatever the alignment of the pointers.
size_t norm_workspace(const NormProblem& p, bool backward);
hipError_t launch_norm_fwd(const NormProblem& p, hipStream_t st);
hipError_t launch_norm_bwd(const NormProblem& p, hipStream_t st);
// The statistics of no positions: NaN.
hipError_t launch_norm_no_stats(const NormProblem& p, hipStream_t st);
// The parameters' gradients of no data: zeros.
hipError_t launch_norm_no_params(const NormProblem& p, hipStream_t st);

struct ConvBwdProblem {
  int T, Ttot, N, C, W;
  bool f32, silu;
  const void* x;
  const float* weight;  // [C, W]
  const float* bias;    // [C] or null
  const void* init;     // [N, W - 1, C] the inputs before each sequence, or null (zeros)
  const int32_t* cu;
  const void* dy;
  const void* dfinal;   // [N, W - 1, C] gradient of the last inputs, or null (zeros)
  void* dx;
  float* dweight;       // [C, W] or null
  float* dbias;         // [C] or null
  void* dinit;          // [N, W - 1, C] or null
  float* part;          // workspace: [blocks, W + 1, C] partial sums
  int blocks, tokens;   // token blocks and their length
};
hipError_t launch_conv1d_bwd(const ConvBwdProblem& p, hipStream_t st);

}  // namespace gdn
