// The selective scan over prompts.  For a sequence, a channel c (of group g = c / (C / G)) and
// its S states, with step_t = softplus(dt_t + bias) (or dt_t + bias),
//
//   h_t[s] = exp(step_t A[s]) h_{t-1}[s] + step_t x_t B_t[g, s]
//   y_t    = (sum_s C_t[g, s] h_t[s] + D x_t) silu(z_t)
//
// Every product is elementwise in (channel, state), so nothing here is a matrix product: the
// work is one v_exp_f32 and four fp32 operations per (token, channel, state), about 24 cycles
// of a SIMD for 64 of them, against 8 bytes per (token, channel): with S = 16 the vector units
// bound it, not memory.  The layout is made for them:
//   * a lane is a channel, so B_t and C_t are the same for the whole wave and come through the
//     scalar cache into scalar registers, which the vector operations read for free; loads and
//     stores of x, dt, z and y are contiguous over the lanes;
//   * the S states of 64 channels are split over the waves of a workgroup (ns states a lane),
//     which share each token's step and step * x through LDS (one softplus per token and
//     channel) and sum y there; few states a lane keep the registers low and many waves live;
//   * when the (sequence, channel block) pairs are too few to fill the GPU, sequences are split
//     into chunks: a first pass finds each chunk's own end state from a zero start and its sum
//     of steps, a small kernel composes the chunks' start states in order (the decay of a
//     chunk is exp(A * sum of steps)), and the output pass starts from them.
#include "ssm_device.h"

namespace gdn {

namespace {

constexpr int TT = kScanTile;

struct ScanArgs {
  const void* x;
  const void* dt;
  const void* z;
  const float* bc;
  const float* A;
  const float* D;
  const float* bias;
  const float* h0;
  float* hst;
  float* dsum;
  void* y;
  float* ht;
  long sx, sdt, sz;
  ChunkMap map;
  int C, G, S, per, nblk, Sp;
  int softplus, split;
};

// B and C of every token and group as padded fp32 rows, so that the scan reads them through the
// scalar cache whatever their type, alignment, strides and number.
template <typename E>
__global__ __launch_bounds__(256) void k_scan_pack(const E* Bm, const E* Cm, long sb, long sc,
                                                   float* bc, int Ttot, int G, int S, int Sp) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  const int row = 2 * Sp;
  if (i >= (long)Ttot * G * row) return;
  const int k = (int)(i % row);
  const long tg = i / row;
  const int g = (int)(tg % G);
  const long t = tg / G;
  const int s = k < Sp ? k : k - Sp;
  float v = 0.f;
  if (s < S) v = (float)(k < Sp ? Bm[t * sb + (long)g * S + s] : Cm[t * sc + (long)g * S + s]);
  bc[i] = v;
}

// What a lane works on: its channel (clamped, so that every lane has one) and whether it is the
// lane that owns it.
struct Lane {
  int g, c;
  bool live;
};
__device__ __forceinline__ Lane lane_channel(int per, int nblk) {
  Lane l;
  l.g = blockIdx.y / nblk;
  const int cl = (blockIdx.y - l.g * nblk) * kScanLanes + lane_id();
  l.live = cl < per;
  l.c = l.g * per + min(cl, per - 1);
  return l;
}

// One chunk's outputs from its start state; the last chunk writes the final state.
template <int NS, int NW, typename E>
__global__ __launch_bounds__(64 * NW) void k_scan_out(ScanArgs a) {
  constexpr int TPW = TT / NW;  // tokens of a tile that a wave prepares and finishes
  __shared__ float2 sd[TT][kScanLanes];  // (step, step * x)
  __shared__ float yp[NW][TT][kScanLanes];
  const int slot = blockIdx.x;
  const Chunk ch = chunk_of(a.map, slot);
  if (!ch.ok) return;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const Lane l = lane_channel(a.per, a.nblk);
  const E* x = static_cast<const E*>(a.x) + l.c;
  const E* dt = static_cast<const E*>(a.dt) + l.c;
  const E* z = static_cast<const E*>(a.z) + l.c;
  E* y = static_cast<E*>(a.y) + l.c;
  const float bias = a.bias ? a.bias[l.c] : 0.f;
  const float Dc = a.D ? a.D[l.c] : 0.f;
  const int s0 = w * NS;

  float A2[NS], h[NS];
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int s = s0 + k;
    A2[k] = s < a.S ? a.A[(long)l.c * a.S + s] * kLog2e : 0.f;
    h[k] = 0.f;
    if (s < a.S) {
      if (a.split)
        h[k] = a.hst[((long)slot * a.S + s) * a.C + l.c];
      else if (a.h0)
        h[k] = a.h0[((long)ch.n * a.C + l.c) * a.S + s];
    }
  }

  E rx[TPW], rd[TPW], rz[TPW];
  auto fetch = [&](int tile) {  // this wave's tokens of a tile (past the chunk: its last one)
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const long r = ch.t0 + min(tile * TT + w * TPW + i, ch.len - 1);
      rx[i] = x[r * a.sx];
      rd[i] = dt[r * a.sdt];
      if (a.z) rz[i] = z[r * a.sz];
    }
  };
  const int tiles = (ch.len + TT - 1) / TT;
  if (tiles > 0) fetch(0);
  for (int tile = 0; tile < tiles; ++tile) {
    float xv[TPW], zv[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      xv[i] = (float)rx[i];
      zv[i] = a.z ? (float)rz[i] : 0.f;
      float v = (float)rd[i] + bias;
      if (a.softplus) v = softplus_f32(v);
      sd[w * TPW + i][lane] = make_float2(v, v * xv[i]);
    }
    if (tile + 1 < tiles) fetch(tile + 1);
    __syncthreads();
    const int m = min(TT, ch.len - tile * TT);
    const float* row = a.bc + ((long)(ch.t0 + tile * TT) * a.G + l.g) * (2 * a.Sp) + s0;
    const long step = (long)a.G * (2 * a.Sp);
    auto token = [&](int t) {
      const scalar_row b = as_scalar(row + t * step);
      const scalar_row c = as_scalar(row + t * step + a.Sp);
      const float2 v = sd[t][lane];
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        h[k] = fmaf(__builtin_amdgcn_exp2f(v.x * A2[k]), h[k], v.y * b[k]);
        s = fmaf(c[k], h[k], s);
      }
      yp[w][t][lane] = s;
    };
    if (m == TT) {
#pragma unroll
      for (int t = 0; t < TT; ++t) token(t);
    } else {
      for (int t = 0; t < m; ++t) token(t);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int t = w * TPW + i;
      if (t < m) {
        float s = Dc * xv[i];
#pragma unroll
        for (int k = 0; k < NW; ++k) s += yp[k][t][lane];
        if (a.z) s *= zv[i] * sigmoid_f32(zv[i]);
        if (l.live) y[(long)(ch.t0 + tile * TT + t) * a.C] = (E)s;
      }
    }
  }
  if (a.ht && ch.i == ch.count - 1 && l.live) {
#pragma unroll
    for (int k = 0; k < NS; ++k)
      if (s0 + k < a.S) a.ht[((long)ch.n * a.C + l.c) * a.S + s0 + k] = h[k];
  }
}

// One chunk's own end state (from a zero start) and its sum of steps; a sequence's last chunk
// has no successor and is skipped.
template <int NS, int NW, typename E>
__global__ __launch_bounds__(64 * NW) void k_scan_state(ScanArgs a) {
  constexpr int TPW = TT / NW;
  __shared__ float2 sd[2][TT][kScanLanes];
  const int slot = blockIdx.x;
  const Chunk ch = chunk_of(a.map, slot);
  if (!ch.ok || ch.i == ch.count - 1) return;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const Lane l = lane_channel(a.per, a.nblk);
  const E* x = static_cast<const E*>(a.x) + l.c;
  const E* dt = static_cast<const E*>(a.dt) + l.c;
  const float bias = a.bias ? a.bias[l.c] : 0.f;
  const int s0 = w * NS;
  float A2[NS], h[NS], sum = 0.f;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    A2[k] = s0 + k < a.S ? a.A[(long)l.c * a.S + s0 + k] * kLog2e : 0.f;
    h[k] = 0.f;
  }
  E rx[TPW], rd[TPW];
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const long r = ch.t0 + min(tile * TT + w * TPW + i, ch.len - 1);
      rx[i] = x[r * a.sx];
      rd[i] = dt[r * a.sdt];
    }
  };
  const int tiles = (ch.len + TT - 1) / TT;
  if (tiles > 0) fetch(0);
  for (int tile = 0; tile < tiles; ++tile) {
    float2(*buf)[kScanLanes] = sd[tile & 1];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      float v = (float)rd[i] + bias;
      if (a.softplus) v = softplus_f32(v);
      buf[w * TPW + i][lane] = make_float2(v, v * (float)rx[i]);
    }
    if (tile + 1 < tiles) fetch(tile + 1);
    __syncthreads();
    const int m = min(TT, ch.len - tile * TT);
    const float* row = a.bc + ((long)(ch.t0 + tile * TT) * a.G + l.g) * (2 * a.Sp) + s0;
    const long step = (long)a.G * (2 * a.Sp);
    auto token = [&](int t) {
      const scalar_row b = as_scalar(row + t * step);
      const float2 v = buf[t][lane];
      sum += v.x;
#pragma unroll
      for (int k = 0; k < NS; ++k)
        h[k] = fmaf(__builtin_amdgcn_exp2f(v.x * A2[k]), h[k], v.y * b[k]);
    };
    if (m == TT) {
#pragma unroll
      for (int t = 0; t < TT; ++t) token(t);
    } else {
      for (int t = 0; t < m; ++t) token(t);
    }
  }
  if (!l.live) return;
#pragma unroll
  for (int k = 0; k < NS; ++k)
    if (s0 + k < a.S) a.hst[((long)slot * a.S + s0 + k) * a.C + l.c] = h[k];
  if (w == 0) a.dsum[(long)slot * a.C + l.c] = sum;
}

// Start states in place of the chunks' own end states: one thread per (sequence, state,
// channel) goes over the sequence's chunks, eight of them loaded ahead.
__global__ __launch_bounds__(256) void k_scan_combine(ScanArgs a) {
  const int c = blockIdx.y * 256 + threadIdx.x;
  const int n = blockIdx.x / a.S, s = blockIdx.x - n * a.S;
  if (c >= a.C) return;
  int bos, eos;
  chunk_seq(a.map, n, bos, eos);
  const int count = chunk_count(eos - bos, a.map.Lc);
  const long first = a.map.cu ? chunk_first(a.map, n) : n * chunk_count(a.map.T, a.map.Lc);
  const float A2 = a.A[(long)c * a.S + s] * kLog2e;
  float h = a.h0 ? a.h0[((long)n * a.C + c) * a.S + s] : 0.f;
  float* hst = a.hst + (first * a.S + s) * a.C + c;
  const float* ds = a.dsum + first * a.C + c;
  const long hstep = (long)a.S * a.C;
  for (int i0 = 0; i0 < count; i0 += 8) {
    float e[8], d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool has = i0 + j < count - 1;  // the last chunk has no end state here
      e[j] = has ? hst[(i0 + j) * hstep] : 0.f;
      d[j] = has ? ds[(long)(i0 + j) * a.C] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i0 + j < count) hst[(i0 + j) * hstep] = h;
      h = fmaf(__builtin_amdgcn_exp2f(d[j] * A2), h, e[j]);
    }
  }
}

template <int NS, int NW, typename E>
hipError_t launch_cfg(const ScanProblem& p, const ScanArgs& a, hipStream_t st) {
  const dim3 grid(p.slots, p.G * p.nblk);
  if (a.split) {
    k_scan_state<NS, NW, E><<<grid, 64 * NW, 0, st>>>(a);
    k_scan_combine<<<dim3(p.N * p.S, (p.C + 255) / 256), 256, 0, st>>>(a);
  }
  k_scan_out<NS, NW, E><<<grid, 64 * NW, 0, st>>>(a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_e(const ScanProblem& p, const ScanArgs& a, hipStream_t st) {
  if (p.ns == 4) {
    if (p.nw == 1) return launch_cfg<4, 1, E>(p, a, st);
    if (p.nw == 2) return launch_cfg<4, 2, E>(p, a, st);
    return launch_cfg<4, 4, E>(p, a, st);
  }
  if (p.ns == 8) return launch_cfg<8, 4, E>(p, a, st);
  if (p.nw == 4) return launch_cfg<16, 4, E>(p, a, st);
  if (p.nw == 8) return launch_cfg<16, 8, E>(p, a, st);
  return launch_cfg<16, 16, E>(p, a, st);
}

}  // namespace

hipError_t launch_scan_pack(const ScanProblem& p, hipStream_t st) {
  const long n = (long)p.Ttot * p.G * 2 * p.Sp;
  if (n == 0) return hipSuccess;
  const unsigned grid = (unsigned)((n + 255) / 256);
  if (p.f32)
    k_scan_pack<float><<<grid, 256, 0, st>>>((const float*)p.Bm, (const float*)p.Cm, p.sb, p.sc,
                                             p.bc, p.Ttot, p.G, p.S, p.Sp);
  else
    k_scan_pack<bf16><<<grid, 256, 0, st>>>((const bf16*)p.Bm, (const bf16*)p.Cm, p.sb, p.sc,
                                            p.bc, p.Ttot, p.G, p.S, p.Sp);
  return hipGetLastError();
}

hipError_t launch_scan_fwd(const ScanProblem& p, hipStream_t st) {
  const hipError_t e = launch_scan_pack(p, st);
  if (e != hipSuccess) return e;
  ScanArgs a;
  a.x = p.x;
  a.dt = p.dt;
  a.z = p.z;
  a.bc = p.bc;
  a.A = p.A;
  a.D = p.D;
  a.bias = p.bias;
  a.h0 = p.h0;
  a.hst = p.hst;
  a.dsum = p.dsum;
  a.y = p.y;
  a.ht = p.ht;
  a.sx = p.sx;
  a.sdt = p.sdt;
  a.sz = p.sz;
  a.map = ChunkMap{p.cu, p.T, p.Ttot, p.N, p.Lc};
  a.C = p.C;
  a.G = p.G;
  a.S = p.S;
  a.per = p.per;
  a.nblk = p.nblk;
  a.Sp = p.Sp;
  a.softplus = p.softplus;
  a.split = p.Lc != kScanNoSplit;
  return p.f32 ? launch_e<float>(p, a, st) : launch_e<bf16>(p, a, st);
}

}  // namespace gdn
