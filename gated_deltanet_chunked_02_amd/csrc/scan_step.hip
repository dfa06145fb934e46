// The selective scan for one token of each sequence, its states in a pool of lines: the decode
// step.  Per (sequence, channel) the S states are read, decayed, fed and written once:
//
//   h' = exp(step A) h + step x B,   y = (sum_s C h' + D x) silu(z)
//
// so the pool's bytes bound it.  LPC lanes share a channel and read VEC states each (16 bytes
// when S is a multiple of 4 and the pool and A are aligned to that), so a wave's loads of the pool
// and of A are contiguous; y is summed over the LPC lanes.  A workgroup keeps to its channels for
// `seqs` sequences, so A is loaded once for them, and every sequence's loads are issued before the
// one before it computes.  256 sequences of 4096 channels and 16 states (143 MB) take 26 us when the
// last pool is still in the last-level cache and 34 us from HBM (4.2 TB/s; a copy takes 28); one
// sequence takes 3.6 us.
#include "ssm_device.h"

namespace gdn {

namespace {

// VEC values of B or C (WIDE: their rows are aligned to VEC values).
template <typename E, int VEC, bool WIDE>
__device__ __forceinline__ void load_bc(const E* p, float* v) {
  if constexpr (WIDE && VEC == 4) {
    typedef E vec __attribute__((ext_vector_type(4)));
    const vec r = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = (float)r[k];
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = (float)p[k];
  }
}

template <int VEC>
__device__ __forceinline__ void load_states(const float* p, float* v) {
  if constexpr (VEC == 4) {
    const f32x4 r = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = r[k];
  } else {
    v[0] = p[0];
  }
}

// NV: vectors of states a lane holds (LPC VEC NV >= S).
template <typename E, int VEC, int LPC, int NV, bool WIDE>
__global__ __launch_bounds__(256) void k_scan_step(ScanStepProblem p, int seqs) {
  constexpr int CPB = 256 / LPC;  // channels of a workgroup
  const int blocks = (p.C + CPB - 1) / CPB;
  const int group = blockIdx.x / blocks;  // of sequences
  const int c = (blockIdx.x - group * blocks) * CPB + (int)threadIdx.x / LPC;
  const int l = threadIdx.x % LPC;
  if (c >= p.C) return;  // LPC divides 64: a channel's lanes leave together
  const int g = c / p.per;
  float A2[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int s = (j * LPC + l) * VEC;
    if (s < p.S) load_states<VEC>(p.A + (long)c * p.S + s, A2[j]);
#pragma unroll
    for (int k = 0; k < VEC; ++k) A2[j][k] = s < p.S ? A2[j][k] * kLog2e : 0.f;
  }
  const float bias = p.bias ? p.bias[c] : 0.f, Dc = p.D ? p.D[c] : 0.f;

  struct In {
    float h[NV][VEC], b[NV][VEC], c[NV][VEC], x, dt, z;
    float* to;
  };
  auto load = [&](int b, In& in) {
    const int rl = p.read ? p.read[b] : b;
    const int wl = p.write ? p.write[b] : rl;
    const float* from =
        rl >= 0 && rl < p.lines ? p.state + ((long)rl * p.C + c) * p.S : nullptr;
    in.to = wl >= 0 && wl < p.lines ? p.state + ((long)wl * p.C + c) * p.S : nullptr;
    const E* Bm = static_cast<const E*>(p.Bm) + b * p.sb + (long)g * p.S;
    const E* Cm = static_cast<const E*>(p.Cm) + b * p.sc + (long)g * p.S;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int s = (j * LPC + l) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) in.h[j][k] = in.b[j][k] = in.c[j][k] = 0.f;
      if (s < p.S) {
        if (from) load_states<VEC>(from + s, in.h[j]);
        load_bc<E, VEC, WIDE>(Bm + s, in.b[j]);
        load_bc<E, VEC, WIDE>(Cm + s, in.c[j]);
      }
    }
    in.x = (float)static_cast<const E*>(p.x)[b * p.sx + c];
    in.dt = (float)static_cast<const E*>(p.dt)[b * p.sdt + c];
    in.z = p.z ? (float)static_cast<const E*>(p.z)[b * p.sz + c] : 0.f;
  };
  const int first = group * seqs, end = min(first + seqs, p.B);
  In in;
  load(first, in);
  for (int b = first; b < end; ++b) {
    In next;
    if (b + 1 < end) load(b + 1, next);
    float step = in.dt + bias;
    if (p.softplus) step = softplus_f32(step);
    const float dx = step * in.x;
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int s = (j * LPC + l) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        in.h[j][k] = fmaf(__builtin_amdgcn_exp2f(step * A2[j][k]), in.h[j][k], dx * in.b[j][k]);
        if (s < p.S) y = fmaf(in.c[j][k], in.h[j][k], y);
      }
      if (in.to && s < p.S) {
        if constexpr (VEC == 4)
          // past the caches: a layer's states are not read again before every other layer's
          __builtin_nontemporal_store(
              (f32x4{in.h[j][0], in.h[j][1], in.h[j][2], in.h[j][3]}),
              reinterpret_cast<f32x4*>(in.to + s));
        else
          in.to[s] = in.h[j][0];
      }
    }
#pragma unroll
    for (int o = LPC / 2; o > 0; o >>= 1) y += __shfl_xor(y, o);
    if (l == 0) {
      y = fmaf(Dc, in.x, y);
      if (p.z) y *= in.z * sigmoid_f32(in.z);
      static_cast<E*>(p.y)[(long)b * p.C + c] = (E)y;
    }
    in = next;
  }
}

template <typename E, int VEC, int LPC, int NV, bool WIDE>
hipError_t launch_cfg(const ScanStepProblem& p, hipStream_t st) {
  const int blocks = (p.C + 256 / LPC - 1) / (256 / LPC);
  // sequences that share a workgroup's A, where that leaves eight workgroups a CU: 256 sequences of
  // 4096 channels with their states in HBM take 44 us at 1, 38 at 4, 37 at 8 (33 with the stores
  // that pass the caches)
  const int seqs = (long)blocks * p.B >= 8 * 2048 ? 8 : (long)blocks * p.B >= 4 * 2048 ? 4 : 1;
  k_scan_step<E, VEC, LPC, NV, WIDE>
      <<<(unsigned)blocks * ((p.B + seqs - 1) / seqs), 256, 0, st>>>(p, seqs);
  return hipGetLastError();
}

template <typename E, int VEC, bool WIDE>
hipError_t launch_vec(const ScanStepProblem& p, hipStream_t st) {
  // lanes a channel: the smallest power of two that holds the vectors, at most 16
  const int q = (p.S + VEC - 1) / VEC;
  if (q <= 1) return launch_cfg<E, VEC, 1, 1, WIDE>(p, st);
  if (q <= 2) return launch_cfg<E, VEC, 2, 1, WIDE>(p, st);
  if (q <= 4) return launch_cfg<E, VEC, 4, 1, WIDE>(p, st);
  if (q <= 8) return launch_cfg<E, VEC, 8, 1, WIDE>(p, st);
  if (q <= 16) return launch_cfg<E, VEC, 16, 1, WIDE>(p, st);
  if (q <= 32) return launch_cfg<E, VEC, 16, 2, WIDE>(p, st);
  if (VEC == 4 || q <= 64) return launch_cfg<E, VEC, 16, 4, WIDE>(p, st);  // dstate <= 256
  if constexpr (VEC == 1) return launch_cfg<E, 1, 16, 16, false>(p, st);
  return hipErrorInvalidValue;
}

template <typename E>
hipError_t launch_e(const ScanStepProblem& p, hipStream_t st) {
  if (!p.vec4) return launch_vec<E, 1, false>(p, st);
  return p.wide ? launch_vec<E, 4, true>(p, st) : launch_vec<E, 4, false>(p, st);
}

}  // namespace

hipError_t launch_scan_step(const ScanStepProblem& p, hipStream_t st) {
  return p.f32 ? launch_e<float>(p, st) : launch_e<bf16>(p, st);
}

}  // namespace gdn
