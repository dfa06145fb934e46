// The selective scan for one token of each sequence, its states in a pool of lines: the decode
// step.  Per (sequence, channel) the S states are read, decayed, fed and written once:
//
//   h' = exp(step A) h + step x B,   y = (sum_s C h' + D x) silu(z)
//
// so the pool's bytes bound it.  LPC lanes share a channel and read VEC states each (16 bytes
// when S is a multiple of 4 and the pool and A are aligned to that), so a wave's loads of the pool and of A are contiguous; y is summed
// over the LPC lanes.
#include "ssm_device.h"

namespace gdn {

namespace {

template <typename E, int VEC, int LPC>
__global__ __launch_bounds__(256) void k_scan_step(ScanStepProblem p) {
  constexpr int CPB = 256 / LPC;  // channels of a workgroup
  const int b = blockIdx.y + gridDim.y * blockIdx.z;
  if (b >= p.B) return;
  const int c = blockIdx.x * CPB + (int)threadIdx.x / LPC;
  const int l = threadIdx.x % LPC;
  if (c >= p.C) return;  // LPC divides 64: a channel's lanes leave together
  const int g = c / p.per;
  const int rl = p.read ? p.read[b] : b;
  const int wl = p.write ? p.write[b] : rl;
  const float* hin = rl >= 0 && rl < p.lines ? p.state + ((long)rl * p.C + c) * p.S : nullptr;
  float* hout = wl >= 0 && wl < p.lines ? p.state + ((long)wl * p.C + c) * p.S : nullptr;
  const E* Bm = static_cast<const E*>(p.Bm) + b * p.sb + (long)g * p.S;
  const E* Cm = static_cast<const E*>(p.Cm) + b * p.sc + (long)g * p.S;
  const float* A = p.A + (long)c * p.S;
  const float x = (float)static_cast<const E*>(p.x)[b * p.sx + c];
  float step = (float)static_cast<const E*>(p.dt)[b * p.sdt + c] + (p.bias ? p.bias[c] : 0.f);
  if (p.softplus) step = softplus_f32(step);
  const float dx = step * x;
  float y = 0.f;
  for (int s = l * VEC; s < p.S; s += LPC * VEC) {
    float h[VEC], av[VEC];
    if constexpr (VEC == 4) {
      const float4 a4 = *reinterpret_cast<const float4*>(A + s);
      const float4 h4 = hin ? *reinterpret_cast<const float4*>(hin + s) : make_float4(0, 0, 0, 0);
      av[0] = a4.x; av[1] = a4.y; av[2] = a4.z; av[3] = a4.w;
      h[0] = h4.x; h[1] = h4.y; h[2] = h4.z; h[3] = h4.w;
    } else {
      av[0] = A[s];
      h[0] = hin ? hin[s] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      h[k] = fmaf(__builtin_amdgcn_exp2f(step * (av[k] * kLog2e)), h[k], dx * (float)Bm[s + k]);
      y = fmaf((float)Cm[s + k], h[k], y);
    }
    if (hout) {
      if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(hout + s) = make_float4(h[0], h[1], h[2], h[3]);
      else
        hout[s] = h[0];
    }
  }
#pragma unroll
  for (int o = LPC / 2; o > 0; o >>= 1) y += __shfl_xor(y, o);
  if (l == 0) {
    if (p.D) y = fmaf(p.D[c], x, y);
    if (p.z) {
      const float z = (float)static_cast<const E*>(p.z)[b * p.sz + c];
      y *= z * sigmoid_f32(z);
    }
    static_cast<E*>(p.y)[(long)b * p.C + c] = (E)y;
  }
}

template <typename E, int VEC, int LPC>
hipError_t launch_cfg(const ScanStepProblem& p, hipStream_t st) {
  const int by = p.B < 32768 ? p.B : 32768;
  const dim3 grid((p.C + 256 / LPC - 1) / (256 / LPC), by, (p.B + by - 1) / by);
  k_scan_step<E, VEC, LPC><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

template <typename E, int VEC>
hipError_t launch_vec(const ScanStepProblem& p, hipStream_t st) {
  const int q = p.S / VEC;  // the largest power of two of lanes that all have states
  if (q >= 16) return launch_cfg<E, VEC, 16>(p, st);
  if (q >= 8) return launch_cfg<E, VEC, 8>(p, st);
  if (q >= 4) return launch_cfg<E, VEC, 4>(p, st);
  if (q >= 2) return launch_cfg<E, VEC, 2>(p, st);
  return launch_cfg<E, VEC, 1>(p, st);
}

}  // namespace

hipError_t launch_scan_step(const ScanStepProblem& p, hipStream_t st) {
  if (p.vec4)
    return p.f32 ? launch_vec<float, 4>(p, st) : launch_vec<bf16, 4>(p, st);
  return p.f32 ? launch_vec<float, 1>(p, st) : launch_vec<bf16, 1>(p, st);
}

}  // namespace gdn
