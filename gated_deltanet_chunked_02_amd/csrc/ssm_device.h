// Device-side pieces shared by the selective scan's kernels and the norms.
#pragma once

#include "gdn_device.h"
#include "ssm.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|), with log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3.
// 2 atanh(s) / s is a polynomial of degree 4 in s^2, interpolated at the Chebyshev points of
// [0, 1/9]: off by 8e-9 of its value, an eighth of a rounding.  (A log of 1 + e would lose e's low
// bits: steps of 0.001 are the usual ones here.)
__device__ __forceinline__ float softplus_f32(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float q = s * s;
  float p = 0.28157779574394226f;
  p = fmaf(p, q, 0.27965158224105835f);
  p = fmaf(p, q, 0.4002459645271301f);
  p = fmaf(p, q, 0.6666632294654846f);
  p = fmaf(p, q, 2.f);
  return fmaf(s, p, fmaxf(v, 0.f));  // a NaN comes through s
}

// softplus(v) where `mask` has all bits set, v where it has none: no branch.
__device__ __forceinline__ float step_f32(float v, uint32_t mask) {
  return __uint_as_float((__float_as_uint(softplus_f32(v)) & mask) |
                         (__float_as_uint(v) & ~mask));
}

// One lane's column of a token-major tensor from some token on: a buffer resource whose base is
// that token's row, the lane's column as the vector offset and the row as a scalar one (so an
// access costs no vector address arithmetic).  A lane whose column is kNoColumn reads zeros and
// its stores are dropped by the resource's bounds.  The rows reached must lie within 2 GiB of the
// base, which the plans see to.
constexpr uint32_t kNoColumn = 0x7FFFFFFF;
template <typename E>
struct Column {
  __amdgpu_buffer_rsrc_t rs;
  uint32_t col;  // bytes
  int row;       // bytes from one token's row to the next
  // rows: how many the chunk has; width: elements of a row that belong to the tensor
  __device__ __forceinline__ void open(const void* base, long first, long stride, int rows,
                                       int width, int c, bool live) {
    E* p = const_cast<E*>(static_cast<const E*>(base)) + first * stride;
    const long bytes = ((rows - 1) * stride + width) * (long)sizeof(E);
    rs = __builtin_amdgcn_make_buffer_rsrc(p, 0, rows > 0 ? (int)bytes : 0, 0x00020000);
    col = live ? (uint32_t)(c * (int)sizeof(E)) : kNoColumn;
    row = (int)(stride * (long)sizeof(E));
  }
  // The value's bits, to be widened later: nothing waits for the load here.
  __device__ __forceinline__ uint32_t load(int r) const {
    if constexpr (sizeof(E) == 2)
      return (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, col, r * row, 0);
    else
      return __builtin_amdgcn_raw_buffer_load_b32(rs, col, r * row, 0);
  }
  static __device__ __forceinline__ float wide(uint32_t bits) {
    return __uint_as_float(sizeof(E) == 2 ? bits << 16 : bits);
  }
  __device__ __forceinline__ void store(int r, float v) const {
    if constexpr (sizeof(E) == 2)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (E)v), rs, col,
                                            r * row, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rs, col, r * row, 0);
  }
};

// A wave-uniform row of fp32 values read through the scalar cache: the address space tells the
// compiler that nothing in the kernel writes it.
typedef const float __attribute__((address_space(4))) * scalar_row;
__device__ __forceinline__ scalar_row as_scalar(const float* p) {
  return (scalar_row)(uintptr_t)p;
}

// Column c's sum over `rows` rows of partial sums `stride` apart, in a fixed order: the workgroup's
// 16 waves take every 16th row each, four loads ahead, and are added in order.  The first wave has
// the sum; every wave calls it, lane by lane for its 64 columns.
constexpr int kColumnThreads = 1024;
__device__ __forceinline__ float column_sum(const float* p, long stride, long rows, int c, int C) {
  __shared__ float s[kColumnThreads / 64][64];
  constexpr int WAVES = kColumnThreads / 64;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < C) {
    long i = wave_id();
    for (; i + 3 * WAVES < rows; i += 4 * WAVES) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += p[(i + j * WAVES) * stride + c];
    }
    for (; i < rows; i += WAVES) v[0] += p[i * stride + c];
  }
  s[wave_id()][lane_id()] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  float r = 0.f;
  if (threadIdx.x < 64) {
#pragma unroll
    for (int k = 0; k < WAVES; ++k) r += s[k][lane_id()];
  }
  return r;
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
  return (int)((uint32_t)min(max(m.cu[n], 0), m.Ttot) / (uint32_t)m.Lc) + n;
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
  // len and Lc are at most 2^30, so the sum fits 32 bits
  return max(1, (int)(((uint32_t)len + (uint32_t)Lc - 1u) / (uint32_t)Lc));
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
