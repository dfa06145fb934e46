// Host-side view of the block norm, shared by the C ABI (api_block_norm.cpp) and the launchers
// (block_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

struct BlockNormProblem {
  int rows, C;
  bool f32, residual_f32;  // of h, gate, y; of x and x'
  bool post, silu;
  float eps, residual_scale;
  int64_t sh, sg;          // elements from one row of h (gate) to the next
  const void* x;           // [rows, C]
  const void* h;           // or null
  const void* gate;        // or null
  const float* w1;         // [C] post_weight, or null (ones)
  const float* scale;      // [C] or null (ones)
  const float* w2;         // [C] weight, or null (ones)
  void* xo;                // x', with h; may be x
  void* y;                 // or null
  float* rstd1;            // [rows] of h, or null; read by the backward
  float* rstd2;            // [rows] of x', or null; read by the backward
  // backward
  const void* dxo;         // or null (zero)
  const void* dy;          // or null (no pre-norm)
  void* dx;
  void* dh;
  void* dgate;
  float* dw1;              // or null, as the two below
  float* dscale;
  float* dw2;
  float* part;             // workspace: block_norm_parts() rows of [3, C]
};
// Rows of partial sums that the backward needs.
int block_norm_parts(const BlockNormProblem& p);
hipError_t launch_block_norm_fwd(const BlockNormProblem& p, hipStream_t st);
hipError_t launch_block_norm_bwd(const BlockNormProblem& p, hipStream_t st);

}  // namespace gdn
