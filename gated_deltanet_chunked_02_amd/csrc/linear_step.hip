// Linear attention's step for single tokens: for a sequence's value head, its state line H [Dk, Dv]
// from the pool,
//
//   H <- e^g H + k v^T,    o = scale H^T q
//
// The line read and written once bounds it (64 KB each way for a head of 128 x 128; q, k, v and o are
// a hundredth of that).  A workgroup has 4 LPR columns of one head, four a lane, its row groups a row
// each in turn; every load of the line is issued before the first is used.  Sums over rows are
// joined in a fixed order: lanes, then waves.
//
// Measured: 256 sequences of 32 heads of 128 x 128 204 us (5.3 TB/s), one sequence 4.3.
#include "linear_device.h"

namespace gdn {

namespace {

constexpr int kStepThreads = 256;

template <typename E, int LPR, int RPT>
__global__ __launch_bounds__(kStepThreads) void k_linear_step(LinearStepProblem p) {
  constexpr int RG = kStepThreads / LPR;
  __shared__ __align__(16) f32x4 part[kStepThreads / 64][LPR];
  const int slabs = (p.Dv + 4 * LPR - 1) / (4 * LPR);
  const int slab = blockIdx.x % slabs, bh = blockIdx.x / slabs, n = bh / p.H, h = bh - n * p.H;
  const int cl = threadIdx.x % LPR, rg = threadIdx.x / LPR, col = slab * 4 * LPR + 4 * cl;
  const bool live = col < p.Dv;
  const int from = p.read ? p.read[n] : n, to = p.write ? p.write[n] : from;
  const long cell = (long)p.Dk * p.Dv;
  const float* src = p.state + ((long)from * p.H + h) * cell + col;
  float* dst = p.state + ((long)to * p.H + h) * cell + col;
  const bool reads = live && from >= 0 && from < p.lines;
  const bool writes = live && to >= 0 && to < p.lines;

  f32x4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RG * i;
    s[i] = reads && r < p.Dk ? *reinterpret_cast<const f32x4*>(src + (long)r * p.Dv) : zero4();
  }
  const int hk = h / (p.H / p.Hg);
  const E* qp = static_cast<const E*>(p.q) + n * p.sq + (long)hk * p.Dk;
  const E* kp = static_cast<const E*>(p.k) + n * p.sk + (long)hk * p.Dk;
  float q[RPT], k[RPT], v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RG * i;
    q[i] = r < p.Dk ? (float)qp[r] : 0.f;
    k[i] = r < p.Dk ? (float)kp[r] : 0.f;
  }
  if (live) {
    const E* vp = static_cast<const E*>(p.v) + n * p.sv + (long)h * p.Dv + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)vp[e];
  }
  const float keep = exp2_f32(p.g[p.head_decay ? h : (long)n * p.H + h] * kLog2e);
  f32x4 o = zero4();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + RG * i;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = fmaf(keep, s[i][e], k[i] * v[e]);
      o[e] = fmaf(q[i], s[i][e], o[e]);
    }
    if (writes && r < p.Dk)
      __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(dst + (long)r * p.Dv));
  }
#pragma unroll
  for (int d = LPR; d < 64; d *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], d);
  if (lane_id() < LPR) part[wave_id()][cl] = o;
  __syncthreads();
  if (threadIdx.x < LPR && live) {
    o = part[0][cl];
#pragma unroll
    for (int w = 1; w < kStepThreads / 64; ++w) o += part[w][cl];
    o *= p.scale;
    E* op = static_cast<E*>(p.o) + (long)bh * p.Dv + col;
    if constexpr (sizeof(E) == 2)
      *reinterpret_cast<bf16x4*>(op) = __builtin_convertvector(o, bf16x4);
    else
      *reinterpret_cast<f32x4*>(op) = o;
  }
}

template <typename E>
hipError_t launch_e(const LinearStepProblem& p, hipStream_t st) {
  constexpr int LPR = 8;
  const unsigned blocks = (unsigned)p.B * p.H * ((p.Dv + 4 * LPR - 1) / (4 * LPR));
  if (p.Dk <= 64)
    k_linear_step<E, LPR, 2><<<blocks, kStepThreads, 0, st>>>(p);
  else if (p.Dk <= 128)
    k_linear_step<E, LPR, 4><<<blocks, kStepThreads, 0, st>>>(p);
  else
    k_linear_step<E, LPR, 8><<<blocks, kStepThreads, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_step(const LinearStepProblem& p, hipStream_t st) {
  return p.f32 ? launch_e<float>(p, st) : launch_e<bf16>(p, st);
}

}  // namespace gdn
