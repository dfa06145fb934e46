// Host-side views of the selective state-space calls, shared by the C ABI (api_ssm.cpp) and
// the launchers (scan.hip, scan_bwd.hip, scan_step.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

constexpr int kScanTile = 16;      // tokens a workgroup takes through LDS at a time
constexpr int kScanLanes = 64;     // channels of a workgroup: one per lane
constexpr int kScanNoSplit = 1 << 30;  // chunk length that leaves every sequence whole

// Chunk slots: sequence n's chunk i (of Lc tokens, the last one shorter; one chunk, of no
// tokens, for an empty sequence) has slot first(n) + i, with first(n) = n ceil(T / Lc) for a
// dense batch and floor(cu[n] / Lc) + n for a packed one.  The packed form needs no prefix sum
// over the sequences, and slots do not collide because ceil(len / Lc) is at most
// floor((cu + len) / Lc) - floor(cu / Lc) + 1; a slot that no chunk has stays unused.
struct ScanProblem {
  int T, Ttot, N;      // tokens a sequence (dense), all tokens, sequences
  int C, G, S;         // channels, groups of B and C, states a channel
  int per, nblk;       // channels a group, 64-channel blocks a group
  int Sp;              // states of a padded fp32 row of B or C (ns * nw)
  int ns, nw;          // states a lane, waves a workgroup
  int reach;           // tokens whose rows lie within 2 GiB of the first one's
  int Lc, slots;       // chunk length (kScanNoSplit: whole sequences), chunk slots
  bool f32, softplus;
  const void* x;
  const void* dt;
  const void* z;       // or null
  const void* Bm;
  const void* Cm;
  const float* A;      // [C, S]
  const float* D;      // [C] or null
  const float* bias;   // [C] or null
  const float* h0;     // [N, C, S] or null
  const int32_t* cu;   // [N + 1] or null
  int64_t sx, sdt, sz, sb, sc;  // elements from one token's row to the next
  float* bc;           // workspace: [G, Sp / ns, Ttot, 2, ns], B and C in fp32, padded with zeros
  float* hst;          // workspace: [slots, S, C], each chunk's own end state, then its start
  float* dsum;         // workspace: [slots, C], each chunk's sum of steps
  void* y;
  float* ht;           // [N, C, S] or null
};

hipError_t launch_scan_fwd(const ScanProblem& p, hipStream_t st);
// B and C as padded fp32 rows (p.bc).
hipError_t launch_scan_pack(const ScanProblem& p, hipStream_t st);

// Backward: the same problem at chunks of up to kBwdChunk tokens, nw waves of 4 states (blocks of 32
// states one after another when there are more), plus the gradients.
constexpr int kBwdChunk = 64;
struct ScanBwd {
  const void* dy;
  const float* dht;  // or null
  float* gst;        // workspace, as the kernels' arguments
  float* bcp;
  float* dAp;
  float* dvp;
  void* dx;
  void* ddt;
  void* dz;          // null without z
  void* dB;
  void* dC;
  float* dA;
  float* dD;         // or null
  float* dbias;      // or null
  float* dh0;        // or null
};
hipError_t launch_scan_bwd(const ScanProblem& p, const ScanBwd& b, hipStream_t st);

struct ScanStepProblem {
  int B, C, G, S, per, lines;
  bool f32, softplus;
  bool vec4;  // a channel's states and A come 16 bytes at a time
  bool wide;  // and so may four values of B and C rows
  float* state;  // [lines, C, S]
  const void* x;
  const void* dt;
  const void* z;
  const void* Bm;
  const void* Cm;
  const float* A;
  const float* D;
  const float* bias;
  const int32_t* read;   // [B] or null (line b)
  const int32_t* write;  // [B] or null (the line read)
  int64_t sx, sdt, sz, sb, sc;
  void* y;
};
hipError_t launch_scan_step(const ScanStepProblem& p, hipStream_t st);

}  // namespace gdn
