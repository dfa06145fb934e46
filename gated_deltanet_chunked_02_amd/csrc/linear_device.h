// Device-side pieces of the linear attention kernels: matrix products of 16-byte operand
// fragments, state tiles that serve as operands, rows of a head staged through registers, and the
// decays of a chunk.
//
// State tiles.  A state of R x N values is held by columns: wave w has 16 (or more) columns, all R
// rows, as 16 x 16 accumulator tiles in pairs; row r of tile t of pair P is row
// 32 P + 8 (r / 4) + 4 t + r % 4 of the state.  In a lane of group g = lane / 16 a pair then holds the
// eight consecutive rows 32 P + 8 g .. + 7, which is what one matrix-core operand takes along k: a
// state goes into a product over its rows without leaving the registers, against 16-byte reads of
// the other operand.
#pragma once

#include "gdn_operands.h"
#include "linear.h"
#include "ssm_device.h"

namespace gdn {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Products of 16-byte fragments: 32 k of bf16 in one instruction, 16 k of fp32 in four.  Lane
// group g holds k = k0 + EPL g .. + EPL - 1 of row (or column) lane % 16.
template <typename E> struct Mx;
template <> struct Mx<bf16> {
  static constexpr int KF = 32, EPL = 8, TERMS = 3;
  typedef bf16x8 frag;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mx<float> {
  static constexpr int KF = 16, EPL = 4, TERMS = 1;
  typedef f32x4 frag;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// Row (or column) r = lane % 16 of a k-contiguous LDS matrix.
template <typename E>
__device__ __forceinline__ typename Mx<E>::frag mx_ld(const E* m, int ld, int row0, int k0) {
  const int l = lane_id();
  return *reinterpret_cast<const typename Mx<E>::frag*>(m + (row0 + (l & 15)) * ld + k0 +
                                                       Mx<E>::EPL * (l >> 4));
}

// The same fragment of a matrix stored [k][n]: column n0 + lane % 16, or with PERM the row of a
// state tile (tile t of pair P, n0 = 32 P + 4 t).
template <typename E, bool PERM>
__device__ __forceinline__ typename Mx<E>::frag mx_tr(const E* m, int ld, int k0, int n0) {
  const int l = lane_id(), c = l & 15, g = l >> 4;
  if constexpr (sizeof(E) == 2) {
    const E* p = m + (k0 + 8 * g + (c >> 2)) * ld + n0 + (PERM ? 8 : 4) * (c & 3);
    const bf16x4 a = read_tr4(p), b = read_tr4(p + 4 * ld);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const E* p = m + (k0 + 4 * g) * ld + n0 + (PERM ? 8 * (c >> 2) + (c & 3) : c);
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = p[i * ld];
    return r;
  }
}

// Column offset (n0 of mx_tr with PERM) of state tile t.
__device__ __forceinline__ int tile_col(int t) { return 32 * (t >> 1) + 4 * (t & 1); }
// A lane's first row of state tile t; it holds four.
__device__ __forceinline__ int tile_row(int t) { return tile_col(t) + 8 * (lane_id() >> 4); }

// x as TERMS operands whose sum is x to fp32's last bits: three bf16 terms carry 24 bits, so a
// state or a weighted row in a product with bf16 data loses nothing that fp32 would keep.
template <typename E, int TERMS = Mx<E>::TERMS>
__device__ __forceinline__ void split(const float* x, typename Mx<E>::frag* out) {
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float r = x[e];
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        const bf16 b = (bf16)r;
        out[t][e] = b;
        r -= (float)b;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[0][e] = x[e];
  }
}

// Operand fragments of a state over its NT row tiles: NT / 2 of bf16, NT of fp32, TERMS each.
template <typename E, int NT, int TERMS>
struct StateOperand {
  static constexpr int STEPS = sizeof(E) == 2 ? NT / 2 : NT;
  typename Mx<E>::frag f[STEPS][TERMS];
  __device__ __forceinline__ void from(const f32x4* tiles) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      float x[8];
      if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = tiles[2 * s][i], x[4 + i] = tiles[2 * s + 1][i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = tiles[s][i];
      }
      split<E, TERMS>(x, f[s]);
    }
  }
  // acc[state column, row of m] += sum over the state's rows r of state[r][.] m[.][r]
  __device__ __forceinline__ f32x4 times(const E* m, int ld, int row0, f32x4 acc) const {
    const int l = lane_id();
    const E* p = m + (row0 + (l & 15)) * ld + 8 * (l >> 4);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const auto b = *reinterpret_cast<const typename Mx<E>::frag*>(
          p + (sizeof(E) == 2 ? 32 * s : tile_col(s)));
#pragma unroll
      for (int t = TERMS - 1; t >= 0; --t) acc = Mx<E>::mma(f[s][t], b, acc);
    }
    return acc;
  }
};

// A chunk's rows of one head, C x D values (D a tile size; the head's own `width` may be less), on
// their way from memory to LDS through registers.  A buffer resource ends behind the chunk's last
// row, so rows past it and columns past the head read as zeros.
template <typename E, int D, int C, int NTH>
struct Rows {
  static constexpr int V = 16 / (int)sizeof(E), VPR = D / V, N = C * VPR / NTH;
  static_assert(C * VPR % NTH == 0 && NTH % VPR == 0, "block shape");
  uint32_t off;  // bytes of this thread's first vector
  int step;      // bytes to the next one
  int at;        // elements into LDS rows
  u32x4 reg[N];
  __device__ __forceinline__ void open(int64_t stride, int width, int ld) {
    const int row = threadIdx.x / VPR, col = threadIdx.x % VPR;
    off = col * V < width ? (uint32_t)(row * (int)stride * (int)sizeof(E) + col * 16) : kNoColumn;
    step = col * V < width ? NTH / VPR * (int)stride * (int)sizeof(E) : 0;
    at = row * ld + col * V;
  }
  // base: the chunk's first row of this head; len: its rows; all uniform
  __device__ __forceinline__ void load(const E* base, int64_t stride, int width, int len) {
    const int bytes = len > 0 ? (int)(((len - 1) * stride + width) * (int64_t)sizeof(E)) : 0;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(base), 0, bytes, 0x00020000);
#pragma unroll
    for (int j = 0; j < N; ++j)
      reg[j] = __builtin_amdgcn_raw_buffer_load_b128(rs, off + (uint32_t)(j * step), 0, 0);
  }
  __device__ __forceinline__ void store(E* lds, int ld) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
      *reinterpret_cast<u32x4*>(lds + at + j * (NTH / VPR) * ld) = reg[j];
  }
};

// Four consecutive columns of a row, rounded once, through a buffer resource that drops rows past
// the chunk's end.
template <typename E>
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t rs, uint32_t off, f32x4 x) {
  if constexpr (sizeof(E) == 2)
    __builtin_amdgcn_raw_buffer_store_b64(
        __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4)), rs, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), rs, off, 0, 0);
}

template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(E* base, int64_t stride, int width,
                                                          int len) {
  const int bytes = len > 0 ? (int)(((len - 1) * stride + width) * (int64_t)sizeof(E)) : 0;
  return __builtin_amdgcn_make_buffer_rsrc(base, 0, bytes, 0x00020000);
}

__device__ __forceinline__ float exp2_f32(float x) { return __builtin_amdgcn_exp2f(x); }

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_d(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive prefix sum across a wave (the order of wave_incl_scan).
__device__ __forceinline__ double wave_incl_scan(double x) {
  x += dpp_d<0x111>(x);
  x += dpp_d<0x112>(x);
  x += dpp_d<0x114>(x);
  x += dpp_d<0x118>(x);
  x += dpp_d<0x142, 0xA>(x);
  x += dpp_d<0x143, 0xC>(x);
  return x;
}

__device__ __forceinline__ double last_lane(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63),
                 hi = __builtin_amdgcn_readlane((int)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the four lane groups that share lane % 16.
__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor(x, 16);
  x += __shfl_xor(x, 32);
  return x;
}

// A chunk's decays.  G_t, the sum of log2 decays up to token t, is held in fp64: the decay between
// two tokens is a difference of two of them, which in fp32 would lose its last bits behind tokens of
// strong decay.  A log2 decay below -1000 (an infinity, or a mask's lowest value: a state forgotten)
// is taken as that, which is as good as none left, and keeps the differences finite.
template <int C>
struct Decays {
  double G[C];
  float into[C];  // 2^G_t: from the chunk's start
  float left[C];  // 2^(G_end - G_t): to its end; into[C - 1] is the whole chunk's
  // one wave's work; x: the log-decay of the lane's token (lane < C), 0 past the chunk's end
  __device__ __forceinline__ double make(float x) {
    const int t = lane_id();
    double g2 = (double)x * 1.4426950408889634;
    g2 = g2 < -1000.0 ? -1000.0 : g2;
    const double s = wave_incl_scan(t < C ? g2 : 0.0);
    const double end = last_lane(s);
    if (t < C) {
      G[t] = s;
      into[t] = exp2_f32((float)s);
      left[t] = exp2_f32((float)(end - s));
    }
    return end;
  }
};

// The log-decay of token t of a chunk that starts at token t0 (0 past its end).
__device__ __forceinline__ float load_decay(const LinearProblem& p, long t0, int t, int len, int h) {
  return t < len ? p.g[p.head_decay ? h : (t0 + t) * p.H + h] : 0.f;
}

// Workgroup b's unit of work: the `group` units in a row that read the same q and k rows run on one
// XCD one after another (workgroups go to the 8 XCDs in turn), the groups on the XCDs in turn.
__device__ __forceinline__ int unit_of(int b, int blocks, int group) {
  const int full = blocks / (8 * group) * (8 * group);
  if (b >= full) return b;
  const int xcd = b & 7, slot = b >> 3;
  return ((slot / group) * 8 + xcd) * group + slot % group;
}

// For unit_of: the value heads (and slabs) of a q/k head, unless that leaves too few groups for the
// XCDs.
inline int group_of(const LinearProblem& p, int slabs, int blocks) {
  int group = p.H / p.Hg * slabs;
  while (group > 1 && blocks / group < 32) group = (group + 1) / 2;
  return group;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A segment slot's chunk (see ssm_device.h), its values known to be the same in every lane.
__device__ __forceinline__ Chunk uniform_chunk(const LinearProblem& p, int slot) {
  const ChunkMap m = {p.cu, p.T, p.Ttot, p.N, p.Lc};
  Chunk c = chunk_of(m, slot);
  c.n = uniform(c.n);
  c.i = uniform(c.i);
  c.count = uniform(c.count);
  c.bos = uniform(c.bos);
  c.t0 = uniform(c.t0);
  c.len = uniform(c.len);
  c.ok = uniform(c.ok) != 0;
  return c;
}

}  // namespace gdn
