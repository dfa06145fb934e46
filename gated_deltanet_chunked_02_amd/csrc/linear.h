// Host-side views of the linear attention calls, shared by the C ABI (api_linear.cpp) and the
// launchers (linear.hip, linear_bwd.hip, linear_step.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

constexpr int kLinearChunk = 64;     // tokens of a chunk in bf16
constexpr int kLinearChunkF32 = 32;  // in fp32, whose tiles take twice the LDS
constexpr int kLinearSlab = 128;     // value columns of a workgroup, at most
// Chunks from one state kept for the gradient to the next, at most.  A head's own decay gathers what the
// differences between them are off by over all tokens, so it has twice as many.
constexpr int kLinearAnchor = 8, kLinearAnchorHead = 4;

// Segments are chunks of Lc tokens (a multiple of the tile chunk, or kScanNoSplit for whole
// sequences) with the slots of ScanProblem (ssm.h); tile chunks have slots of the same form with the
// chunk length in place of Lc.
struct LinearProblem {
  int T, Ttot, N;      // tokens a sequence (dense), all tokens, sequences
  int H, Hg, Dk, Dv;   // value heads, q/k heads, head sizes
  int Lc, slots;       // segment length, segment slots
  int group;           // workgroups in a row that share q and k rows (set by the launchers)
  bool f32, head_decay;
  float scale;
  int64_t sq, sk, sv;  // elements from one token's row to the next
  const void* q;
  const void* k;
  const void* v;
  const float* g;      // [H] with head_decay, [B, T, H] without
  const float* h0;     // [N, H, Dk, Dv] or null
  const int32_t* cu;   // [N + 1] or null
  void* o;
  float* ht;           // [N, H, Dk, Dv] or null
  float* states;       // workspace: [slots, H, Dk, Dv], each segment's own end state, then its start
  bool direct;         // first segments start from h0 itself: no other reads it after ht is written
  bool join;           // segments make their start states from the own ones of those before them
  float* sums;         // workspace: [slots, H], each segment's sum of log2 decays
};

hipError_t launch_linear_fwd(const LinearProblem& p, hipStream_t st);

struct LinearBwd {
  const void* dout;    // [B, T, H, Dv]
  const float* dht;    // [N, H, Dk, Dv] or null
  void* dq;
  void* dk;
  void* dv;
  float* dg;           // [H] or [B, T, H], or null
  float* dh0;          // or null
  float* grads;        // workspace: [slots, H, Dk, Dv], as states but from the ends
  bool direct;         // last segments end with dht itself, likewise
  float* anchors;      // workspace: the state at every `every`-th chunk's end, in the kernels' tile order
  double* a;           // workspace: [Ttot, H] what q . dq takes from before the chunk
  int every;
  float* part;         // workspace: [2, Ttot, H, Dk] dq and dk of every value head (shared q/k heads)
  double* dgp;         // workspace: [slots, H] sums of dg (head_decay)
};

// A pass over segments that makes states only: sums of x_t y_t^T.
struct LinearPass {
  const void* x;       // k; back: q
  const void* y;       // v; back: dout
  int64_t sx, sy;
  float* own;          // [slots, H, Dk, Dv] every segment's own sum
};
// The segments' start states (p.states) and, with b, the gradients at their ends (b->grads).
hipError_t launch_linear_states(const LinearProblem& p, const LinearBwd* b, hipStream_t st);

// The tensors of one pass of the recurrence: the forward's own, or those that make dq (linear.hip).
// Heads: q and k rows have those of h / qrep, v (and x) rows those of h / vrep.
struct LinearRun {
  const void* q;
  const void* k;
  const void* v;
  const void* x;
  int64_t sq, sk, sv, sx;
  int Dk, Dv, qrep, vrep;
  void* out;           // [B, T, H, Dv]
  double* a;
  float* anchors;
  int every;
};
// dq (or every value head's share of it), a and the anchors.
hipError_t launch_linear_dq(const LinearProblem& p, const LinearBwd& b, hipStream_t st);

// Tile sizes of the backward: 64 or 128 for head sizes up to that.
inline int linear_tile(int D) { return D <= 64 ? 64 : 128; }
inline int linear_anchor(const LinearProblem& p) {
  return p.head_decay ? kLinearAnchorHead : kLinearAnchor;
}
inline int linear_chunk(bool f32) { return f32 ? kLinearChunkF32 : kLinearChunk; }
hipError_t launch_linear_bwd(const LinearProblem& p, const LinearBwd& b, hipStream_t st);

struct LinearStepProblem {
  int B, H, Hg, Dk, Dv, lines;
  bool f32, head_decay;
  float scale;
  int64_t sq, sk, sv;
  float* state;           // [lines, H, Dk, Dv]
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const int32_t* read;    // [B] or null (line b)
  const int32_t* write;   // [B] or null (the line read)
  void* o;
};
hipError_t launch_linear_step(const LinearStepProblem& p, hipStream_t st);

}  // namespace gdn
