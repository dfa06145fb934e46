// Device-side pieces shared by the selective scan's kernels and the norms.
#pragma once

#include "gdn_device.h"
#include "ssm.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|), with log1p(e) = 2 atanh(s), s = e / (2 + e), by the
// odd series of atanh: s <= 1/3, so the first term left out, s^17 / 17, is 5e-10 of the sum.
// (A log of 1 + e would lose e's low bits: steps of 0.001 are the usual ones here.)
__device__ __forceinline__ float softplus_f32(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float q = s * s;
  float p = 1.f / 15.f;
  p = fmaf(p, q, 1.f / 13.f);
  p = fmaf(p, q, 1.f / 11.f);
  p = fmaf(p, q, 1.f / 9.f);
  p = fmaf(p, q, 1.f / 7.f);
  p = fmaf(p, q, 1.f / 5.f);
  p = fmaf(p, q, 1.f / 3.f);
  p = fmaf(p, q, 1.f);
  return fmaf(2.f * s, p, fmaxf(v, 0.f));  // a NaN comes through s
}

// A wave-uniform row of fp32 values read through the scalar cache: the address space tells the
// compiler that nothing in the kernel writes it.
typedef const float __attribute__((address_space(4))) * scalar_row;
__device__ __forceinline__ scalar_row as_scalar(const float* p) {
  return (scalar_row)(uintptr_t)p;
}

// The chunk of a slot (see ScanProblem).
struct Chunk {
  int n, i, count;     // sequence, chunk of the sequence, chunks of the sequence
  int bos, t0, len;    // the sequence's first token, the chunk's, the chunk's length
  bool ok;
};

struct ChunkMap {
  const int32_t* cu;
  int T, Ttot, N, Lc;
};

__device__ __forceinline__ int chunk_first(const ChunkMap& m, int n) {
  return min(max(m.cu[n], 0), m.Ttot) / m.Lc + n;
}

__device__ __forceinline__ void chunk_seq(const ChunkMap& m, int n, int& bos, int& eos) {
  if (m.cu) {
    bos = min(max(m.cu[n], 0), m.Ttot);
    eos = min(max(m.cu[n + 1], bos), m.Ttot);
  } else {
    bos = n * m.T;
    eos = bos + m.T;
  }
}

__device__ __forceinline__ int chunk_count(int len, int Lc) {
  return max(1, (int)(((long)len + Lc - 1) / Lc));
}

__device__ __forceinline__ Chunk chunk_of(const ChunkMap& m, int slot) {
  Chunk c;
  int first, eos;
  if (m.cu) {
    int lo = 0, hi = m.N - 1;  // the last sequence whose first slot is at most this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (chunk_first(m, mid) <= slot) lo = mid; else hi = mid - 1;
    }
    c.n = lo;
    first = chunk_first(m, lo);
  } else {
    const int k = chunk_count(m.T, m.Lc);
    c.n = slot / k;
    first = c.n * k;
  }
  chunk_seq(m, c.n, c.bos, eos);
  c.count = chunk_count(eos - c.bos, m.Lc);
  c.i = slot - first;
  c.ok = c.i >= 0 && c.i < c.count;
  c.t0 = c.bos + (c.ok ? c.i * m.Lc : 0);
  c.len = max(0, min(m.Lc, eos - c.t0));
  return c;
}

}  // namespace gdn
