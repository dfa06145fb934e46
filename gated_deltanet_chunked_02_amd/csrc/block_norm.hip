// Norms before and after a block with its gate and residual scale, and their gradient.  For a row of
// the residual stream x, a block's output h and its gate,
//
//   n = h rstd1 w1,  rstd1 = (E[h^2] + eps)^-1/2  (n = h without a post-norm)
//   z = n act(gate),   x' = x + alpha z,  alpha = residual_scale scale
//   y = x' rstd2 w2,   rstd2 = (E[x'^2] + eps)^-1/2
//
// and with dxo, dy the gradients of x' and y, hat = x' rstd2, dhat = dy w2, xh = h rstd1,
//
//   dR = dxo + rstd2 (dhat - hat E[dhat hat]),   dx = dR,   dw2 = sum dy hat,
//   dscale = residual_scale sum dR z,   dgate = alpha dR n act'(gate),   dn = alpha dR act(gate)
//   dw1 = sum dn xh,   dh = rstd1 (dn w1 - xh E[dn w1 xh])
//
// The bytes bound both: x, h, gate in and x', y out; five tensors in and three out.  A row is held in
// registers, eight values a thread and as many waves as it takes (rows of up to 512 values: one wave a
// row, four rows a workgroup), so every tensor is read once; y comes from x' before it is rounded.  A
// thread keeps to the same channels over the rows of its workgroup: parameters are loaded once and
// their gradients gather in registers, one partial row a workgroup, added in a fixed order by a second
// launch.  The next row's loads are in flight while a row is worked on.  The backward's second mean
// follows from two more sums of the first reduction (E[dn w1 xh] is linear in E[dhat hat]), so it has
// one exchange between waves, not two.
//
// Rows of more than 8192 values go through memory again instead (k_block_norm_wide*), the second and
// third reading from the caches, their parameters' gradients through a workgroup's own partial row.
//
// Measured: 16384 rows of 4096 channels, gated, bf16 130 us (5.1 TB/s), beside an fp32 stream 171 and, with
// the gradient, 447 (5.3 TB/s).  Replayed from a graph, whose start is about 14 us of each: 8192 rows of
// 8192 136 and 250 (no registers for the next row's loads); 4096 rows of 16384 205 and 513 (728 and 1221
// with a value a thread at a time); 16384 rows of 1024 33 and 77.
#include "block_norm.h"
#include "ssm_device.h"

namespace gdn {

namespace {

constexpr int kEach = 8;               // values a thread holds
constexpr int kMostRow = 1024 * kEach;  // values of a row held in registers
// Threads of the wide kernels: values loaded one at a time take registers for their offsets as well.
constexpr int wide_threads(int VEC) { return VEC == 8 ? 1024 : 512; }

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A thread's eight values of a row of C, in runs of VEC consecutive ones, `width` threads times VEC
// apart, as loads and stores of up to 16 bytes through a buffer resource of the row, which reads zeros
// behind its end and drops stores there.
template <typename E, int VEC>
struct Slice {
  static constexpr int kWords = kEach * (int)sizeof(E) / 4, kRun = VEC * (int)sizeof(E);
  typedef uint32_t words __attribute__((ext_vector_type(kWords)));
  union {
    uint32_t u[kWords];
    uint16_t s[kWords * 2];
  };
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t open(const E* row, int C) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(row), 0, C * (int)sizeof(E), 0x00020000);
  }
  __device__ __forceinline__ void load(const E* row, int t, int width, int C) {
    const __amdgpu_buffer_rsrc_t rs = open(row, C);
#pragma unroll
    for (int j = 0; j < kEach / VEC; ++j) {
      const int off = (j * width + t) * kRun;
      if constexpr (kRun >= 16) {
#pragma unroll
        for (int k = 0; k < kRun / 16; ++k) {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, off + 16 * k, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) u[(j * kRun + 16 * k) / 4 + i] = v[i];
        }
      } else if constexpr (kRun == 8) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0);
        u[2 * j] = v[0];
        u[2 * j + 1] = v[1];
      } else if constexpr (kRun == 4) {
        u[j] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
      } else {
        s[j] = __builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0);
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(E) == 4) return __uint_as_float(u[i]);
    return __uint_as_float(i % 2 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
  }
  static __device__ __forceinline__ void store(E* row, int t, int width, int C, const float* v) {
    const __amdgpu_buffer_rsrc_t rs = open(row, C);
#pragma unroll
    for (int j = 0; j < kEach / VEC; ++j) {
      const int off = (j * width + t) * kRun;
      typedef E run __attribute__((ext_vector_type(VEC > 1 ? VEC : 2)));
      run o;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = (E)v[j * VEC + i];
      if constexpr (kRun == 32) {
        const auto w = __builtin_bit_cast(words, o);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, rs, off, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[4], w[5], w[6], w[7]}, rs, off + 16, 0, 0);
      } else if constexpr (kRun == 16) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), rs, off, 0, 0);
      } else if constexpr (kRun == 8) {
        typedef uint32_t two __attribute__((ext_vector_type(2)));
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(two, o), rs, off, 0, 0);
      } else if constexpr (kRun == 4 && VEC == 2) {
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, o), rs, off, 0, 0);
      } else if constexpr (kRun == 4) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[j]), rs, off, 0, 0);
      } else {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (E)o[0]), rs, off, 0, 0);
      }
    }
  }
};

// A parameter's values of a thread's channels (ones when absent).
template <int VEC>
__device__ __forceinline__ void params(const float* p, int t, int width, int C, float* v) {
  Slice<float, VEC> s;
  if (p) s.load(p, t, width, C);
#pragma unroll
  for (int i = 0; i < kEach; ++i) v[i] = p ? s[i] : 1.f;
}

__device__ __forceinline__ float wave_sum(float x) {
  x += __shfl_xor(x, 32);
  x += __shfl_xor(x, 16);
  x += dpp_f<0x128>(x);
  x += dpp_f<0x124>(x);
  x += dpp_f<0x122>(x);
  x += dpp_f<0x121>(x);
  return x;
}

// Sums of N values over a row's waves.  A workgroup of one row exchanges them through LDS, in turn
// through two buffers: a wave writes a buffer again only after an exchange through the other.
template <int N>
struct RowSum {
  float (*lds)[2][N][16];
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&x)[N], int waves) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = wave_sum(x[i]);
    if (waves == 1) return;
    if (lane_id() == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) (*lds)[turn][i][wave_id()] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
      for (int w = 0; w < waves; ++w) s += (*lds)[turn][i][w];
      x[i] = s;
    }
    turn ^= 1;
  }
};

__device__ __forceinline__ float gate_act(float g, bool silu) {
  return silu ? g * sigmoid_f32(g) : g;
}
__device__ __forceinline__ float gate_slope(float g, bool silu) {
  const float s = sigmoid_f32(g);
  return silu ? s * (1.f + g * (1.f - s)) : 1.f;
}

// How rows go to waves: `waves` a row; rows of one wave four a workgroup.
struct RowWork {
  int waves, first, step, t;
  __device__ __forceinline__ RowWork(int C) {
    waves = (C + 64 * kEach - 1) / (64 * kEach);
    if (waves == 1) {
      first = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(wave_id());
      step = gridDim.x * 4;
      t = lane_id();
    } else {
      first = blockIdx.x;
      step = gridDim.x;
      t = threadIdx.x;
    }
  }
};

// PARTS: 0 no block output (x' = x), 1 without a gate, 2 with one.
template <typename E, typename R, int VEC, int PARTS, int MOST>
__global__ __launch_bounds__(MOST) void k_block_norm(BlockNormProblem p) {
  __shared__ float lds[2][1][16];
  constexpr bool AHEAD = MOST <= 512;  // registers for the next row's loads
  const RowWork w(p.C);
  const int C = p.C, t = w.t, width = 64 * w.waves;
  RowSum<1> sum{&lds};
  float wa[kEach], w2[kEach];
  params<VEC>(p.w2, t, width, C, w2);
  if constexpr (PARTS > 0) {
    float s[kEach];
    params<VEC>(p.w1, t, width, C, wa);
    params<VEC>(p.scale, t, width, C, s);
#pragma unroll
    for (int i = 0; i < kEach; ++i) wa[i] *= s[i] * p.residual_scale;
  }
  const float inv = 1.f / (float)C;
  Slice<R, VEC> xs;
  Slice<E, VEC> hs, gs;
  auto fetch = [&](int row) {
    xs.load(static_cast<const R*>(p.x) + (long)row * C, t, width, C);
    if constexpr (PARTS > 0) hs.load(static_cast<const E*>(p.h) + row * p.sh, t, width, C);
    if constexpr (PARTS > 1) gs.load(static_cast<const E*>(p.gate) + row * p.sg, t, width, C);
  };
  if (AHEAD && w.first < p.rows) fetch(w.first);
  for (int row = w.first; row < p.rows; row += w.step) {
    if (!AHEAD) fetch(row);
    float x[kEach];
    float square[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = xs[i];
    if constexpr (PARTS > 0) {
      float z[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        z[i] = hs[i];
        square[0] = fmaf(z[i], z[i], square[0]);
        z[i] *= PARTS > 1 ? gate_act(gs[i], p.silu) * wa[i] : wa[i];
      }
      if (AHEAD && row + w.step < p.rows) fetch(row + w.step);
      float rstd = 1.f;
      if (p.post) {
        sum(square, w.waves);
        rstd = rsqrtf(square[0] * inv + p.eps);
        if (p.rstd1 && t == 0) p.rstd1[row] = rstd;
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) x[i] = fmaf(z[i], rstd, x[i]);
      Slice<R, VEC>::store(static_cast<R*>(p.xo) + (long)row * C, t, width, C, x);
    } else if (row + w.step < p.rows) {
      fetch(row + w.step);
    }
    if (p.y) {
      square[0] = 0.f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) square[0] = fmaf(x[i], x[i], square[0]);
      sum(square, w.waves);
      const float rstd = rsqrtf(square[0] * inv + p.eps);
      if (p.rstd2 && t == 0) p.rstd2[row] = rstd;
#pragma unroll
      for (int i = 0; i < kEach; ++i) x[i] *= rstd * w2[i];
      Slice<E, VEC>::store(static_cast<E*>(p.y) + (long)row * C, t, width, C, x);
    }
  }
}

template <typename E, typename R, int VEC, int PARTS, int MOST>
__global__ __launch_bounds__(MOST) void k_block_norm_bwd(BlockNormProblem p) {
  __shared__ float lds[2][3][16];
  constexpr bool AHEAD = MOST <= 512;  // registers for the next row's loads
  const RowWork w(p.C);
  const int C = p.C, t = w.t, width = 64 * w.waves;
  RowSum<3> sum{&lds};
  float w1[kEach], al[kEach], w2[kEach], d1[kEach], ds[kEach], d2[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) d1[i] = ds[i] = d2[i] = 0.f;
  auto place = [&]() {  // t; without registers to spare, offsets are made at each use
    int own = t;
    if (!AHEAD) opaque(own);
    return own;
  };
  auto weights = [&]() {  // of the block's half; read at each use, from the caches
    const int own = place();
    if constexpr (PARTS > 0) {
      params<VEC>(p.w1, own, width, C, w1);
      params<VEC>(p.scale, own, width, C, al);
#pragma unroll
      for (int i = 0; i < kEach; ++i) al[i] *= p.residual_scale;
    }
  };
  if (AHEAD) {
    params<VEC>(p.w2, t, width, C, w2);
    weights();
  }
  const float inv = 1.f / (float)C;
  Slice<R, VEC> xs, dxs;
  Slice<E, VEC> hs, gs, dys;
  float rstd1 = 1.f, rstd2 = 0.f;
#pragma unroll
  for (int i = 0; i < Slice<R, VEC>::kWords; ++i) dxs.u[i] = 0;
#pragma unroll
  for (int i = 0; i < Slice<E, VEC>::kWords; ++i) dys.u[i] = 0;
  auto fetch = [&](int row) {
    const int own = place();
    xs.load(static_cast<const R*>(p.x) + (long)row * C, own, width, C);
    if constexpr (PARTS > 0) {
      hs.load(static_cast<const E*>(p.h) + row * p.sh, own, width, C);
      if (p.post) rstd1 = p.rstd1[row];
    }
    if constexpr (PARTS > 1) gs.load(static_cast<const E*>(p.gate) + row * p.sg, own, width, C);
    if (p.dxo) dxs.load(static_cast<const R*>(p.dxo) + (long)row * C, own, width, C);
    if (p.dy) {
      dys.load(static_cast<const E*>(p.dy) + (long)row * C, own, width, C);
      rstd2 = p.rstd2[row];
    }
  };
  if (AHEAD && w.first < p.rows) fetch(w.first);
  for (int row = w.first; row < p.rows; row += w.step) {
    if (!AHEAD) {
      fetch(row);
      params<VEC>(p.w2, place(), width, C, w2);
      weights();
    }
    float hat[kEach], dR[kEach];
    float s[3] = {0.f, 0.f, 0.f};
    const float r1 = rstd1, r2 = rstd2;
    const Slice<E, VEC> h = hs, g = gs;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      float f = 0.f;  // alpha act(gate) w1 xh
      if constexpr (PARTS > 0) {
        f = h[i] * r1 * w1[i] * al[i];
        if constexpr (PARTS > 1) f *= gate_act(g[i], p.silu);
      }
      hat[i] = (f + xs[i]) * r2;
      const float dy = dys[i], dhat = dy * w2[i];
      d2[i] = fmaf(dy, hat[i], d2[i]);
      dR[i] = fmaf(r2, dhat, dxs[i]);
      s[0] = fmaf(dhat, hat[i], s[0]);
      s[1] = fmaf(f, dR[i], s[1]);
      s[2] = fmaf(f, hat[i], s[2]);
    }
    if (AHEAD && row + w.step < p.rows) fetch(row + w.step);
    sum(s, w.waves);
    const float m = r2 * s[0] * inv;           // E[dhat hat] rstd2
    const float m1 = (s[1] - m * s[2]) * inv;  // E[dn w1 xh]
#pragma unroll
    for (int i = 0; i < kEach; ++i) dR[i] = fmaf(-hat[i], m, dR[i]);
    Slice<R, VEC>::store(static_cast<R*>(p.dx) + (long)row * C, place(), width, C, dR);
    if constexpr (PARTS > 0) {
      if (!AHEAD) weights();
      float dg[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float xh = h[i] * r1, n = xh * w1[i], dz = al[i] * dR[i];
        float a = 1.f;
        if constexpr (PARTS > 1) {
          a = gate_act(g[i], p.silu);
          dg[i] = dz * n * gate_slope(g[i], p.silu);
        }
        const float dn = dz * a;
        ds[i] = fmaf(dR[i], n * a, ds[i]);
        d1[i] = fmaf(dn, xh, d1[i]);
        dR[i] = p.post ? r1 * fmaf(dn, w1[i], -xh * m1) : dn;
      }
      Slice<E, VEC>::store(static_cast<E*>(p.dh) + (long)row * C, place(), width, C, dR);
      if constexpr (PARTS > 1)
        Slice<E, VEC>::store(static_cast<E*>(p.dgate) + (long)row * C, place(), width, C, dg);
    }
  }
  float* part = p.part + (long)(w.waves == 1 ? w.first : (int)blockIdx.x) * 3 * C;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int c = ((i / VEC) * width + t) * VEC + i % VEC;
    if (c < C) {
      if (p.dw1) part[c] = d1[i];
      if (p.dscale) part[C + c] = ds[i] * p.residual_scale;
      if (p.dw2) part[2 * C + c] = d2[i];
    }
  }
}

// One row a workgroup at a time, in blocks of eight values a thread, read again for each
// step.
template <typename E, typename R, int VEC>
__global__ __launch_bounds__(wide_threads(VEC)) void k_block_norm_wide(BlockNormProblem p) {
  __shared__ float lds[2][1][16];
  constexpr int WIDE = wide_threads(VEC), BLOCK = WIDE * kEach;
  RowSum<1> sum{&lds};
  const int C = p.C, t = threadIdx.x;
  const float inv = 1.f / (float)C;
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const R* x = static_cast<const R*>(p.x) + (long)row * C;
    const E* h = static_cast<const E*>(p.h) + row * p.sh;
    const E* g = static_cast<const E*>(p.gate) + row * p.sg;
    float s[1] = {0.f}, rstd1 = 1.f;
    if (p.h && p.post) {
      for (int b = 0; b < C; b += BLOCK) {
        Slice<E, VEC> hs;
        hs.load(h + b, t, WIDE, C - b);
#pragma unroll
        for (int i = 0; i < kEach; ++i) s[0] = fmaf(hs[i], hs[i], s[0]);
      }
      sum(s, WIDE / 64);
      rstd1 = rsqrtf(s[0] * inv + p.eps);
      if (p.rstd1 && t == 0) p.rstd1[row] = rstd1;
    }
    auto values = [&](int b, float (&v)[kEach]) {
      Slice<R, VEC> xs;
      xs.load(x + b, t, WIDE, C - b);
      if (!p.h) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] = xs[i];
        return;
      }
      Slice<E, VEC> hs, gs;
      hs.load(h + b, t, WIDE, C - b);
      if (p.gate) gs.load(g + b, t, WIDE, C - b);
      float w[kEach], al[kEach];
      params<VEC>(p.w1 ? p.w1 + b : nullptr, t, WIDE, C - b, w);
      params<VEC>(p.scale ? p.scale + b : nullptr, t, WIDE, C - b, al);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float a = (p.gate ? gate_act(gs[i], p.silu) : 1.f) * w[i] * al[i] * p.residual_scale;
        v[i] = fmaf(hs[i] * rstd1, a, xs[i]);
      }
    };
    float v[kEach], rstd2 = 0.f;
    if (p.y) {
      s[0] = 0.f;
      for (int b = 0; b < C; b += BLOCK) {
        values(b, v);
#pragma unroll
        for (int i = 0; i < kEach; ++i) s[0] = fmaf(v[i], v[i], s[0]);
      }
      sum(s, WIDE / 64);
      rstd2 = rsqrtf(s[0] * inv + p.eps);
      if (p.rstd2 && t == 0) p.rstd2[row] = rstd2;
    }
    // x' last: it may be x's buffer
    for (int b = 0; b < C; b += BLOCK) {
      values(b, v);
      if (p.h)
        Slice<R, VEC>::store(static_cast<R*>(p.xo) + (long)row * C + b, t, WIDE, C - b, v);
      if (p.y) {
        float w[kEach];
        params<VEC>(p.w2 ? p.w2 + b : nullptr, t, WIDE, C - b, w);
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] *= rstd2 * w[i];
        Slice<E, VEC>::store(static_cast<E*>(p.y) + (long)row * C + b, t, WIDE, C - b, v);
      }
    }
  }
}

struct No { static constexpr bool value = false; };
struct Yes { static constexpr bool value = true; };

// The parameters' gradients gather in the workgroup's partial row.
template <typename E, typename R, int VEC>
__global__ __launch_bounds__(wide_threads(VEC)) void k_block_norm_wide_bwd(BlockNormProblem p) {
  __shared__ float lds[2][3][16];
  constexpr int WIDE = wide_threads(VEC), BLOCK = WIDE * kEach;
  RowSum<3> sum{&lds};
  const int C = p.C;
  const float inv = 1.f / (float)C;
  float* part = p.part + (long)blockIdx.x * 3 * C;
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const long at = (long)row * C;
    const float r1 = p.h && p.post ? p.rstd1[row] : 1.f, r2 = p.dy ? p.rstd2[row] : 0.f;
    float s[3] = {0.f, 0.f, 0.f}, m = 0.f, m1 = 0.f;
    auto walk = [&](auto second) {  // three sums of the row, then what follows from them
      constexpr bool SECOND = decltype(second)::value;
      auto place = [] {  // offsets are made at each use
        int t = threadIdx.x;
        opaque(t);
        return t;
      };
      for (int b = 0; b < C; b += BLOCK) {
        Slice<R, VEC> xs, dxs;
        Slice<E, VEC> hs, gs, dys;
        float w1[kEach], al[kEach], w2[kEach];
        xs.load(static_cast<const R*>(p.x) + at + b, place(), WIDE, C - b);
        if (p.dxo) dxs.load(static_cast<const R*>(p.dxo) + at + b, place(), WIDE, C - b);
        if (p.dy) dys.load(static_cast<const E*>(p.dy) + at + b, place(), WIDE, C - b);
        if (p.h) hs.load(static_cast<const E*>(p.h) + row * p.sh + b, place(), WIDE, C - b);
        if (p.gate) gs.load(static_cast<const E*>(p.gate) + row * p.sg + b, place(), WIDE, C - b);
        params<VEC>(p.w1 ? p.w1 + b : nullptr, place(), WIDE, C - b, w1);
        params<VEC>(p.scale ? p.scale + b : nullptr, place(), WIDE, C - b, al);
        params<VEC>(p.w2 ? p.w2 + b : nullptr, place(), WIDE, C - b, w2);
        float dR[kEach], dh[kEach], dg[kEach], d1[kEach], ds[kEach], d2[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const float alpha = al[i] * p.residual_scale;
          const float a = p.gate ? gate_act(gs[i], p.silu) : 1.f;
          const float xh = p.h ? hs[i] * r1 : 0.f, n = xh * w1[i];
          const float hat = fmaf(n * a, alpha, xs[i]) * r2;
          const float dy = p.dy ? dys[i] : 0.f;
          dR[i] = fmaf(r2, dy * w2[i], p.dxo ? dxs[i] : 0.f);
          if constexpr (!SECOND) {
            const float f = alpha * a * n;
            s[0] = fmaf(dy * w2[i], hat, s[0]);
            s[1] = fmaf(f, dR[i], s[1]);
            s[2] = fmaf(f, hat, s[2]);
          } else {
            dR[i] = fmaf(-hat, m, dR[i]);
            const float dz = alpha * dR[i], dn = dz * a;
            d1[i] = dn * xh;
            ds[i] = dR[i] * p.residual_scale * (n * a);
            d2[i] = dy * hat;
            dg[i] = p.gate ? dz * n * gate_slope(gs[i], p.silu) : 0.f;
            dh[i] = p.post ? r1 * fmaf(dn, w1[i], -xh * m1) : dn;
          }
        }
        if constexpr (SECOND) {
          auto gather = [&](float* to, float (&v)[kEach]) {
            const int t = place();
            if (row != (int)blockIdx.x) {
              Slice<float, VEC> before;
              before.load(to + b, t, WIDE, C - b);
#pragma unroll
              for (int i = 0; i < kEach; ++i) v[i] += before[i];
            }
            Slice<float, VEC>::store(to + b, t, WIDE, C - b, v);
            sched_fence();
          };
          if (p.dw1) gather(part, d1);
          if (p.dscale) gather(part + C, ds);
          if (p.dw2) gather(part + 2 * C, d2);
          Slice<R, VEC>::store(static_cast<R*>(p.dx) + at + b, place(), WIDE, C - b, dR);
          if (p.h) Slice<E, VEC>::store(static_cast<E*>(p.dh) + at + b, place(), WIDE, C - b, dh);
          if (p.gate)
            Slice<E, VEC>::store(static_cast<E*>(p.dgate) + at + b, place(), WIDE, C - b, dg);
        }
      }
    };
    walk(No());
    sum(s, WIDE / 64);
    m = r2 * s[0] * inv;
    m1 = (s[1] - m * s[2]) * inv;
    walk(Yes());
  }
}

__global__ __launch_bounds__(kColumnThreads) void k_block_norm_params(BlockNormProblem p, int parts) {
  float* to = blockIdx.y == 0 ? p.dw1 : blockIdx.y == 1 ? p.dscale : p.dw2;
  if (!to) return;
  const int c = blockIdx.x * 64 + lane_id();
  const float s = column_sum(p.part + (long)blockIdx.y * p.C, 3L * p.C, parts, c, p.C);
  if (threadIdx.x < 64 && c < p.C) to[c] = s;
}

int waves_of(int C) { return (C + 64 * kEach - 1) / (64 * kEach); }

// Workgroups: no more than run at once (32 waves a CU forward, 12 backward, by their registers), each
// of one row a wave at least, in the backward, whose partial row of sums costs as much as a row, four.
int blocks_of(const BlockNormProblem& p, bool backward) {
  if (p.C > kMostRow) {
    const int most = backward ? 256 : 512, want = backward ? (p.rows + 3) / 4 : p.rows;
    return want < most ? want : most;
  }
  const int waves = waves_of(p.C), each = waves == 1 ? 4 : 1, size = waves * each;
  const int most = 256 * (backward ? (size < 12 ? 12 / size : 1) : 32 / size);
  const long rows = each * (backward ? 4 : 1), want = (p.rows + rows - 1) / rows;
  return (int)(want < most ? want : most);
}

// The longest vector that every row starts on.
int vector_of(const BlockNormProblem& p) {
  const int e = p.f32 ? 4 : 2, r = p.residual_f32 ? 4 : 2;
  for (int v : {8, 2}) {
    const auto ok = [v](const void* q, int size) {
      const int bytes = v * size < 16 ? v * size : 16;
      return reinterpret_cast<uintptr_t>(q) % bytes == 0;
    };
    if (p.C % v == 0 && p.sh % v == 0 && p.sg % v == 0 && ok(p.x, r) && ok(p.xo, r) &&
        ok(p.dxo, r) && ok(p.dx, r) && ok(p.h, e) && ok(p.gate, e) && ok(p.y, e) && ok(p.dy, e) &&
        ok(p.dh, e) && ok(p.dgate, e))
      return v;
  }
  return 1;
}

template <typename E, typename R, int VEC, int PARTS>
void run(const BlockNormProblem& p, bool backward, hipStream_t st) {
  const int blocks = blocks_of(p, backward), waves = waves_of(p.C);
  if (waves == 1) {
    if (backward)
      k_block_norm_bwd<E, R, VEC, PARTS, 512><<<blocks, 256, 0, st>>>(p);
    else
      k_block_norm<E, R, VEC, PARTS, 512><<<blocks, 256, 0, st>>>(p);
  } else if (waves <= 8) {
    if (backward)
      k_block_norm_bwd<E, R, VEC, PARTS, 512><<<blocks, 64 * waves, 0, st>>>(p);
    else
      k_block_norm<E, R, VEC, PARTS, 512><<<blocks, 64 * waves, 0, st>>>(p);
  } else if (backward) {
    k_block_norm_bwd<E, R, VEC, PARTS, 1024><<<blocks, 64 * waves, 0, st>>>(p);
  } else {
    k_block_norm<E, R, VEC, PARTS, 1024><<<blocks, 64 * waves, 0, st>>>(p);
  }
}

template <typename E, typename R, int VEC>
void run_parts(const BlockNormProblem& p, bool backward, hipStream_t st) {
  if (!p.h)
    run<E, R, VEC, 0>(p, backward, st);
  else if (!p.gate)
    run<E, R, VEC, 1>(p, backward, st);
  else
    run<E, R, VEC, 2>(p, backward, st);
}

template <typename E, typename R, int VEC>
void run_wide(const BlockNormProblem& p, bool backward, hipStream_t st) {
  const int blocks = blocks_of(p, backward);
  if (!backward)
    k_block_norm_wide<E, R, VEC><<<blocks, wide_threads(VEC), 0, st>>>(p);
  else
    k_block_norm_wide_bwd<E, R, VEC><<<blocks, wide_threads(VEC), 0, st>>>(p);
}

template <typename E, typename R>
void run_types(const BlockNormProblem& p, bool backward, hipStream_t st) {
  if (p.C > kMostRow) {
    if (vector_of(p) == 8)
      run_wide<E, R, 8>(p, backward, st);
    else
      run_wide<E, R, 1>(p, backward, st);
    return;
  }
  switch (vector_of(p)) {
    case 8: run_parts<E, R, 8>(p, backward, st); break;
    case 2: run_parts<E, R, 2>(p, backward, st); break;
    default: run_parts<E, R, 1>(p, backward, st);
  }
}

hipError_t launch(const BlockNormProblem& p, bool backward, hipStream_t st) {
  if (p.f32)
    run_types<float, float>(p, backward, st);
  else if (p.residual_f32)
    run_types<bf16, float>(p, backward, st);
  else
    run_types<bf16, bf16>(p, backward, st);
  return hipGetLastError();
}

}  // namespace

int block_norm_parts(const BlockNormProblem& p) {
  if (p.rows == 0) return 0;
  return blocks_of(p, true) * (p.C <= kMostRow && waves_of(p.C) == 1 ? 4 : 1);
}

hipError_t launch_block_norm_fwd(const BlockNormProblem& p, hipStream_t st) {
  return p.rows == 0 ? hipSuccess : launch(p, false, st);
}

hipError_t launch_block_norm_bwd(const BlockNormProblem& p, hipStream_t st) {
  if (p.rows > 0) {
    const hipError_t e = launch(p, true, st);
    if (e != hipSuccess) return e;
  }
  if (p.dw1 || p.dscale || p.dw2)
    k_block_norm_params<<<dim3((p.C + 63) / 64, 3), kColumnThreads, 0, st>>>(p,
                                                                            block_norm_parts(p));
  return hipGetLastError();
}

}  // namespace gdn
