// Group norm of channels-last data with an activation or a gate, and its gradient.  For a sample
// n, its positions p and a group g of cpg = C / G channels, over M = P cpg values,
//
//   mean = sum x / M,  rstd = (sum (x - mean)^2 / M + eps)^-1/2,  xhat = (x - mean) rstd
//   u = xhat w + b,    y = act(u),  or  y = u act(gate)  with a gate
//
// and with du the gradient of u and dhat = du w,
//
//   dx = rstd (dhat - sum dhat / M - xhat sum (dhat xhat) / M),
//   dw = sum du xhat,  db = sum du  (over samples and positions).
//
// The bytes bound all of it.  Three shapes of it:
//   * rows (P = 1: a token's heads).  A group is cpg consecutive values, which LPS lanes hold in
//     registers: one pass, the variance about the mean itself.  A thread keeps to the same
//     channels over the rows of its workgroup, so weights are loaded once and the parameters'
//     gradients gather in registers.
//   * maps (P > 1).  A group's channels are a short piece of every position's row, so a
//     workgroup takes whole rows: a thread keeps to VEC channels and goes over positions with a
//     running mean and sum of squares about it for each (joined exactly, never as a difference
//     of large sums); a small kernel joins the pieces of each (sample, group), many pieces after
//     another has folded them; a last pass applies them.
//   * a workgroup for each (sample, group), for maps so small that three launches would cost
//     more than reading them in short pieces.
// Statistics and sums are fp32; every output is rounded once; sums have a fixed order.
//
// 16384 gated rows of 4096 channels in 32 groups, bf16 (403 MB) take 74 us, 5.4 TB/s, an addition
// of the same tensors 70; their gradient (671 MB) 133 to 143 us; in fp32 170 us (805 MB) and 267
// (1342 MB).  8 maps of 4096 positions and 512 channels take 30 us forward and 46 us backward, in
// which every pass of 33 to 100 MB has about 5 us of start and end.
#include "norm.h"
#include "ssm_device.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// VEC consecutive values: as one load or store of up to 16 bytes (two for 8 fp32), and widened.
template <typename E, int VEC>
struct Row {
  static constexpr int kBytes = VEC * (int)sizeof(E);
  struct alignas(kBytes < 16 ? kBytes : 16) raw {
    E e[VEC];
  };
  static __device__ __forceinline__ raw load_raw(const E* p) {
    return *reinterpret_cast<const raw*>(p);
  }
  static __device__ __forceinline__ void wide(const raw& r, float* v) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (float)r.e[i];
  }
  static __device__ __forceinline__ void load(const E* p, float* v) { wide(load_raw(p), v); }
  static __device__ __forceinline__ void store(E* p, const float* v) {
    raw r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.e[i] = (E)v[i];
    // past the caches where a store is 16 bytes: a map's second pass finds more of x there, and a
    // large output would not stay (16384 gated rows of 4096 channels 84 to 79 us).  The 32 bytes of 8
    // fp32 values are ordinary stores: past the caches 16384 ungated rows of 4096 take 95 us for 110,
    // but the gradient of gated ones 280 for 267, and 8 maps of 4096 x 512 47 forward for 44
    if constexpr (kBytes == 16)
      __builtin_nontemporal_store(__builtin_bit_cast(f32x4, r), reinterpret_cast<f32x4*>(p));
    else
      *reinterpret_cast<raw*>(p) = r;
  }
};

__device__ __forceinline__ float act_f32(float v, bool silu) {
  return silu ? v * sigmoid_f32(v) : v;
}
__device__ __forceinline__ float act_slope(float v, bool silu) {
  if (!silu) return 1.f;
  const float s = sigmoid_f32(v);
  return s * fmaf(v, 1.f - s, 1.f);
}
// y from u and the gate's value; the gradient of u (and of the gate) from dy.
__device__ __forceinline__ float norm_out(float u, float gate, bool gated, bool silu) {
  return gated ? u * act_f32(gate, silu) : act_f32(u, silu);
}
__device__ __forceinline__ float norm_du(float u, float gate, float dy, bool gated, bool silu) {
  return dy * (gated ? act_f32(gate, silu) : act_slope(u, silu));
}

// VEC per-channel parameters from channel c on (wide: 16-byte aligned there), or `other` of each.
template <int VEC>
__device__ __forceinline__ void load_params(const float* p, int c, bool wide, float other,
                                            float* v) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = other;
  } else if (wide && VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i + 3 < VEC; i += 4) {
      const f32x4 r = *reinterpret_cast<const f32x4*>(p + c + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = r[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = p[c + i];
  }
}

// The statistics (stride values a group) of channels c .. c + VEC - 1 of a sample: read again only
// where a new group begins.
template <int VEC>
__device__ __forceinline__ void load_stats(const float* p, int stride, int c, int cpg, float* v) {
  int g = c / cpg, at = c - g * cpg;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if (i == 0 || at == 0)
      v[i] = p[g * stride];
    else
      v[i] = v[i ? i - 1 : 0];
    if (++at == cpg) {
      at = 0;
      ++g;
    }
  }
}

// Sum over the lps lanes (a power of two, or the whole workgroup) that share a segment.
__device__ __forceinline__ float seg_sum(float v, int lps, float* lds) {
  const int in = min(lps, 64);
  for (int o = in >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if (lps > 64) {
    __syncthreads();
    if (lane_id() == 0) lds[wave_id()] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
  return v;
}

// --- rows -------------------------------------------------------------------------------------

struct RowPlan {
  int lps;   // lanes a segment: a power of two to 64, or 256
  int gp;    // groups a workgroup (a power of two)
  int gblk;  // workgroups a row
  int wgs;   // workgroups that share out the rows
};

template <typename E, int VEC, int K>
__global__ __launch_bounds__(kThreads) void k_norm_rows(NormProblem p, RowPlan q) {
  __shared__ float lds[4];
  const int seg = (int)threadIdx.x / q.lps, l = (int)threadIdx.x % q.lps;
  const int g = blockIdx.y * q.gp + seg % q.gp;
  const int rw = kThreads / q.lps / q.gp;  // rows side by side
  const int nv = p.cpg / VEC;
  const E* x = static_cast<const E*>(p.x);
  const E* gate = static_cast<const E*>(p.gate);
  E* y = static_cast<E*>(p.y);
  const bool ok = g < p.G;
  float w[K][VEC], b[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = l + q.lps * k;
    if (ok && v < nv) {
      load_params<VEC>(p.weight, g * p.cpg + v * VEC, p.wide, 1.f, w[k]);
      load_params<VEC>(p.bias, g * p.cpg + v * VEC, p.wide, 0.f, b[k]);
    }
  }
  const float inv = 1.f / (float)p.cpg;
  typedef Row<E, VEC> R;
  typename R::raw rx[K], rg[K];
  const int step = gridDim.x * rw;  // rows taken at once by all workgroups, one after another
  auto fetch = [&](int r) {
    const long at = (long)r * p.C + (long)g * p.cpg;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int iv = l + q.lps * k;
      if (ok && r < p.N && iv < nv) {
        rx[k] = R::load_raw(x + at + iv * VEC);
        if (gate) rg[k] = R::load_raw(gate + at + iv * VEC);
      }
    }
  };
  const int first = blockIdx.x * rw + seg / q.gp;
  fetch(first);
  for (int r0 = blockIdx.x * rw; r0 < p.N; r0 += step) {
    const int r = r0 + seg / q.gp;
    const bool live = ok && r < p.N;
    const long at = (long)r * p.C + (long)g * p.cpg;
    float v[K][VEC], gt[K][VEC], s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int iv = l + q.lps * k;
      if (live && iv < nv) {
        R::wide(rx[k], v[k]);
        if (gate) R::wide(rg[k], gt[k]);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[k][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += v[k][i];
    }
    fetch(r + step);
    const float mean = seg_sum(s, q.lps, lds) * inv;
    float m2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = l + q.lps * k < nv;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[k][i] -= mean;
        if (in) m2 = fmaf(v[k][i], v[k][i], m2);
      }
    }
    const float rstd = rsqrtf(seg_sum(m2, q.lps, lds) * inv + p.eps);
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int iv = l + q.lps * k;
      if (iv >= nv) continue;
      float out[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        out[i] = norm_out(fmaf(v[k][i] * rstd, w[k][i], b[k][i]), gate ? gt[k][i] : 0.f,
                          gate != nullptr, p.silu);
      Row<E, VEC>::store(y + at + iv * VEC, out);
    }
    if (l == 0) {
      if (p.mean) p.mean[(long)r * p.G + g] = mean;
      if (p.rstd) p.rstd[(long)r * p.G + g] = rstd;
    }
  }
}

template <typename E, int VEC, int K>
__global__ __launch_bounds__(kThreads) void k_norm_rows_bwd(NormProblem p, RowPlan q) {
  __shared__ float lds[4];
  const int seg = (int)threadIdx.x / q.lps, l = (int)threadIdx.x % q.lps;
  const int g = blockIdx.y * q.gp + seg % q.gp;
  const int rw = kThreads / q.lps / q.gp;
  const int nv = p.cpg / VEC;
  const E* x = static_cast<const E*>(p.x);
  const E* gate = static_cast<const E*>(p.gate);
  const E* dy = static_cast<const E*>(p.dy);
  const bool ok = g < p.G;
  const bool gated = gate != nullptr;
  // the parameters stay in registers where they leave enough of them
  constexpr bool KEEP = K * VEC <= 16;
  float dw[K][VEC], db[K][VEC], wk[KEEP ? K : 1][VEC], bk[KEEP ? K : 1][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[k][i] = db[k][i] = 0.f;
    const int v = l + q.lps * k;
    if (KEEP && ok && v < nv) {
      load_params<VEC>(p.weight, g * p.cpg + v * VEC, p.wide, 1.f, wk[KEEP ? k : 0]);
      load_params<VEC>(p.bias, g * p.cpg + v * VEC, p.wide, 0.f, bk[KEEP ? k : 0]);
    }
  }
  const float inv = 1.f / (float)p.cpg;
  for (int r0 = blockIdx.x * rw; r0 < p.N; r0 += gridDim.x * rw) {
    const int r = r0 + seg / q.gp;
    const bool live = ok && r < p.N;
    const long at = (long)r * p.C + (long)g * p.cpg;
    const float mean = live ? p.mean[(long)r * p.G + g] : 0.f;
    const float rstd = live ? p.rstd[(long)r * p.G + g] : 0.f;
    float hat[K][VEC], dh[K][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int iv = l + q.lps * k;
      if (live && iv < nv) {
        float xv[VEC], dv[VEC], gt[VEC], dg[VEC];
        Row<E, VEC>::load(x + at + iv * VEC, xv);
        Row<E, VEC>::load(dy + at + iv * VEC, dv);
        if (gated) Row<E, VEC>::load(gate + at + iv * VEC, gt);
        if constexpr (!KEEP) {
          load_params<VEC>(p.weight, g * p.cpg + iv * VEC, p.wide, 1.f, wk[0]);
          load_params<VEC>(p.bias, g * p.cpg + iv * VEC, p.wide, 0.f, bk[0]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float w = wk[KEEP ? k : 0][i];
          hat[k][i] = (xv[i] - mean) * rstd;
          const float u = fmaf(hat[k][i], w, bk[KEEP ? k : 0][i]);
          const float gv = gated ? gt[i] : 0.f;
          const float du = norm_du(u, gv, dv[i], gated, p.silu);
          if (gated) dg[i] = dv[i] * u * act_slope(gv, p.silu);
          dw[k][i] = fmaf(du, hat[k][i], dw[k][i]);
          db[k][i] += du;
          dh[k][i] = du * w;
          s1 += dh[k][i];
          s2 = fmaf(dh[k][i], hat[k][i], s2);
        }
        if (gated) Row<E, VEC>::store(static_cast<E*>(p.dgate) + at + iv * VEC, dg);
      }
    }
    s1 = seg_sum(s1, q.lps, lds) * inv;
    s2 = seg_sum(s2, q.lps, lds) * inv;
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int iv = l + q.lps * k;
      if (iv >= nv) continue;
      float out[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) out[i] = rstd * (dh[k][i] - s1 - hat[k][i] * s2);
      Row<E, VEC>::store(static_cast<E*>(p.dx) + at + iv * VEC, out);
    }
  }
  if (!ok) return;
  // one row of partial sums for each of the rows taken side by side
  float* part = p.ws + ((long)blockIdx.x * rw + seg / q.gp) * 2 * p.C + (long)g * p.cpg;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int iv = l + q.lps * k;
    if (iv >= nv) continue;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      part[iv * VEC + i] = dw[k][i];
      part[p.C + iv * VEC + i] = db[k][i];
    }
  }
}

// --- maps -------------------------------------------------------------------------------------

// A sample's positions go to its `slabs` workgroups in turn, ty at a time, so that the workgroups
// running at once read neighbouring rows (pieces far apart fall on the same memory channels).
struct MapPlan {
  int tx, ty;  // threads over channel vectors and over positions (tx ty = 256)
  int cblk;    // workgroups a row
  int slabs;   // workgroups that share a sample's positions
};

struct Stat {
  float n, mean, m2;
};
// The statistics of two sets together.
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  const float n = a.n + b.n;
  if (n == 0.f) return a;
  const float d = b.mean - a.mean, r = b.n / n;
  return Stat{n, fmaf(d, r, a.mean), a.m2 + b.m2 + d * d * a.n * r};
}

// Mean and sum of squares about it of every channel of a (sample, slab): ws [n][slab][2][C].
template <typename E, int VEC>
__global__ __launch_bounds__(kThreads) void k_norm_stats(NormProblem p, MapPlan q) {
  __shared__ float lds[kThreads][2 * VEC + 1];
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx;
  const int n = blockIdx.x / q.slabs, slab = blockIdx.x - n * q.slabs;
  const int c0 = (blockIdx.y * q.tx + tx) * VEC;
  const int p0 = slab * q.ty + ty, step = q.slabs * q.ty;
  const bool ok = c0 < p.C;
  const E* x = static_cast<const E*>(p.x) + (long)n * p.P * p.C + c0;
  float mean[VEC], m2[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) mean[i] = m2[i] = 0.f;
  float cnt = 0.f;
  if (ok) {
#pragma unroll 4
    for (int pos = p0; pos < p.P; pos += step) {
      float v[VEC];
      Row<E, VEC>::load(x + (long)pos * p.C, v);
      cnt += 1.f;
      const float r = __builtin_amdgcn_rcpf(cnt);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = v[i] - mean[i];
        mean[i] = fmaf(d, r, mean[i]);
        m2[i] = fmaf(d, v[i] - mean[i], m2[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    lds[threadIdx.x][i] = mean[i];
    lds[threadIdx.x][VEC + i] = m2[i];
  }
  lds[threadIdx.x][2 * VEC] = cnt;
  __syncthreads();
  if (ty == 0 && ok) {
    float* ws = p.ws + (long)blockIdx.x * 2 * p.C + c0;
    for (int i = 0; i < VEC; ++i) {
      Stat s{cnt, mean[i], m2[i]};
      for (int k = 1; k < q.ty; ++k) {
        const float* o = lds[tx + k * q.tx];
        s = join(s, Stat{o[2 * VEC], o[i], o[VEC + i]});
      }
      ws[i] = s.mean;
      ws[p.C + i] = s.m2;
    }
  }
}

// A workgroup sum, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  return seg_sum(v, kThreads, lds);
}

// Positions that a sample's slab takes.
__device__ __forceinline__ float slab_count(const NormProblem& p, const MapPlan& q, int slab) {
  const int all = q.slabs * q.ty, rest = p.P % all - slab * q.ty;
  return (float)(p.P / all * q.ty + min(max(rest, 0), q.ty));
}

// Every channel's statistics over a sample's slabs, in place of the first slab's: a workgroup takes
// 64 channels, its 16 waves every 16th slab each, and nothing else touches those columns.
__global__ __launch_bounds__(kColumnThreads) void k_norm_fold(NormProblem p, MapPlan q) {
  constexpr int WAVES = kColumnThreads / 64;
  __shared__ Stat lds[WAVES][64];
  const int cols = (p.C + 63) / 64;
  const int n = blockIdx.x / cols, c = (blockIdx.x - n * cols) * 64 + lane_id();
  float* ws = p.ws + (long)n * q.slabs * 2 * p.C + c;
  Stat s{0.f, 0.f, 0.f};
  if (c < p.C)
    for (int slab = wave_id(); slab < q.slabs; slab += WAVES) {
      const float* o = ws + (long)slab * 2 * p.C;
      s = join(s, Stat{slab_count(p, q, slab), o[0], o[p.C]});
    }
  lds[wave_id()][lane_id()] = s;
  __syncthreads();
  if (threadIdx.x >= 64 || c >= p.C) return;
  for (int k = 1; k < WAVES; ++k) s = join(s, lds[k][lane_id()]);
  ws[0] = s.mean;
  ws[p.C] = s.m2;
}

// mean and rstd of each (sample, group) from the channels' pieces, one for each of the slabs or one
// in all (folded): to p.mean and p.rstd.
__global__ __launch_bounds__(kThreads) void k_norm_join(NormProblem p, MapPlan q, bool folded,
                                                        float* mean, float* rstd) {
  __shared__ float lds[4];
  const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
  const float* ws = p.ws + (long)n * q.slabs * 2 * p.C + (long)g * p.cpg;
  const int items = (folded ? 1 : q.slabs) * p.cpg;
  auto count = [&](int slab) { return folded ? (float)p.P : slab_count(p, q, slab); };
  float s = 0.f;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int slab = i / p.cpg, c = i - slab * p.cpg;
    s = fmaf(count(slab), ws[(long)slab * 2 * p.C + c], s);
  }
  const float inv = 1.f / ((float)p.P * (float)p.cpg);
  const float mu = block_sum(s, lds) * inv;
  float m2 = 0.f;
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int slab = i / p.cpg, c = i - slab * p.cpg;
    const float* o = ws + (long)slab * 2 * p.C + c;
    const float d = o[0] - mu;
    m2 += fmaf(count(slab) * d, d, o[p.C]);
  }
  m2 = block_sum(m2, lds);
  if (threadIdx.x == 0) {
    mean[blockIdx.x] = mu;
    rstd[blockIdx.x] = rsqrtf(m2 * inv + p.eps);
  }
}

template <typename E, int VEC>
__global__ __launch_bounds__(kThreads) void k_norm_apply(NormProblem p, MapPlan q,
                                                         const float* mean, const float* rstd) {
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx;
  const int n = blockIdx.x / q.slabs, slab = blockIdx.x - n * q.slabs;
  const int c0 = (blockIdx.y * q.tx + tx) * VEC;
  if (c0 >= p.C) return;
  const int p0 = slab * q.ty + ty, step = q.slabs * q.ty;
  const long at = (long)n * p.P * p.C + c0;
  const E* x = static_cast<const E*>(p.x) + at;
  const E* gate = static_cast<const E*>(p.gate) + at;
  E* y = static_cast<E*>(p.y) + at;
  const bool gated = p.gate != nullptr;
  float mu[VEC], sc[VEC], b[VEC], w[VEC];
  load_stats<VEC>(mean + (long)n * p.G, 1, c0, p.cpg, mu);
  load_stats<VEC>(rstd + (long)n * p.G, 1, c0, p.cpg, sc);
  load_params<VEC>(p.weight, c0, p.wide, 1.f, w);
  load_params<VEC>(p.bias, c0, p.wide, 0.f, b);
#pragma unroll
  for (int i = 0; i < VEC; ++i) sc[i] *= w[i];
#pragma unroll 4
  for (int pos = p0; pos < p.P; pos += step) {
    float v[VEC], gt[VEC];
    Row<E, VEC>::load(x + (long)pos * p.C, v);
    if (gated) Row<E, VEC>::load(gate + (long)pos * p.C, gt);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      v[i] = norm_out(fmaf(v[i] - mu[i], sc[i], b[i]), gated ? gt[i] : 0.f, gated, p.silu);
    Row<E, VEC>::store(y + (long)pos * p.C, v);
  }
}

// Sums of du and du xhat of every channel of a (sample, slab): ws [n][slab][2][C].
template <typename E, int VEC>
__global__ __launch_bounds__(kThreads) void k_norm_bwd_sums(NormProblem p, MapPlan q) {
  __shared__ float lds[kThreads][2 * VEC + 1];
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx;
  const int n = blockIdx.x / q.slabs, slab = blockIdx.x - n * q.slabs;
  const int c0 = (blockIdx.y * q.tx + tx) * VEC;
  const int p0 = slab * q.ty + ty, step = q.slabs * q.ty;
  const bool ok = c0 < p.C;
  const long at = (long)n * p.P * p.C + c0;
  const E* x = static_cast<const E*>(p.x) + at;
  const E* dy = static_cast<const E*>(p.dy) + at;
  const E* gate = static_cast<const E*>(p.gate) + at;
  const bool gated = p.gate != nullptr;
  float a[VEC], ah[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) a[i] = ah[i] = 0.f;
  if (ok) {
    float mu[VEC], rs[VEC], w[VEC], b[VEC];
    load_stats<VEC>(p.mean + (long)n * p.G, 1, c0, p.cpg, mu);
    load_stats<VEC>(p.rstd + (long)n * p.G, 1, c0, p.cpg, rs);
    load_params<VEC>(p.weight, c0, p.wide, 1.f, w);
    load_params<VEC>(p.bias, c0, p.wide, 0.f, b);
#pragma unroll 2
    for (int pos = p0; pos < p.P; pos += step) {
      float v[VEC], d[VEC], gt[VEC];
      Row<E, VEC>::load(x + (long)pos * p.C, v);
      Row<E, VEC>::load(dy + (long)pos * p.C, d);
      if (gated) Row<E, VEC>::load(gate + (long)pos * p.C, gt);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float hat = (v[i] - mu[i]) * rs[i];
        const float du = norm_du(fmaf(hat, w[i], b[i]), gated ? gt[i] : 0.f, d[i], gated, p.silu);
        a[i] += du;
        ah[i] = fmaf(du, hat, ah[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    lds[threadIdx.x][i] = ah[i];
    lds[threadIdx.x][VEC + i] = a[i];
  }
  __syncthreads();
  if (ty == 0 && ok) {
    float* ws = p.ws + (long)blockIdx.x * 2 * p.C + c0;
    for (int i = 0; i < VEC; ++i) {
      float s = ah[i], t = a[i];
      for (int k = 1; k < q.ty; ++k) {
        s += lds[tx + k * q.tx][i];
        t += lds[tx + k * q.tx][VEC + i];
      }
      ws[i] = s;
      ws[p.C + i] = t;
    }
  }
}

// The sums over a sample's slabs in place of the first slab's, as k_norm_fold: 64 columns of a plane
// to a workgroup.
__global__ __launch_bounds__(kColumnThreads) void k_norm_bwd_fold(NormProblem p, MapPlan q) {
  const int cols = (p.C + 63) / 64;
  const int row = blockIdx.x / cols, c = (blockIdx.x - row * cols) * 64 + lane_id();
  float* ws = p.ws + ((long)(row >> 1) * q.slabs * 2 + (row & 1)) * p.C;
  const float r = column_sum(ws, 2L * p.C, q.slabs, c, p.C);
  if (threadIdx.x < 64 && c < p.C) ws[c] = r;
}

// The first N G workgroups: sum dhat / M and sum (dhat xhat) / M of each (sample, group), to sums
// [N, G, 2]; the others: dw and db from the same partial sums, 64 channels each.  folded: one piece
// a sample, else one for each of its slabs.
__global__ __launch_bounds__(kColumnThreads) void k_norm_bwd_join(NormProblem p, MapPlan q,
                                                                  bool folded, float* sums) {
  const int joins = p.N * p.G;
  if ((int)blockIdx.x >= joins) {
    const int cols = (p.C + 63) / 64;
    const int row = (blockIdx.x - joins) / cols;
    float* to = row == 0 ? p.dweight : p.dbias;
    if (!to) return;
    const int c = (blockIdx.x - joins - row * cols) * 64 + lane_id();
    const long pieces = folded ? q.slabs : 1;
    const float r = column_sum(p.ws + (long)row * p.C, 2L * p.C * pieces,
                               (long)p.N * q.slabs / pieces, c, p.C);
    if (threadIdx.x < 64 && c < p.C) to[c] = r;
    return;
  }
  __shared__ float lds[2][kColumnThreads / 64];
  const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
  const float* ws = p.ws + (long)n * q.slabs * 2 * p.C + (long)g * p.cpg;
  const int items = (folded ? 1 : q.slabs) * p.cpg;
  float s1 = 0.f, s2 = 0.f;
  for (int i = threadIdx.x; i < items; i += kColumnThreads) {
    const int slab = i / p.cpg, c = i - slab * p.cpg;
    const float* o = ws + (long)slab * 2 * p.C + c;
    const float w = p.weight ? p.weight[g * p.cpg + c] : 1.f;
    s2 = fmaf(w, o[0], s2);
    s1 = fmaf(w, o[p.C], s1);
  }
  for (int o = 32; o > 0; o >>= 1) {
    s1 += __shfl_xor(s1, o);
    s2 += __shfl_xor(s2, o);
  }
  if (lane_id() == 0) {
    lds[0][wave_id()] = s1;
    lds[1][wave_id()] = s2;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float s = 0.f;
    for (int k = 0; k < kColumnThreads / 64; ++k) s += lds[threadIdx.x][k];
    sums[2 * blockIdx.x + threadIdx.x] = s / ((float)p.P * (float)p.cpg);
  }
}

template <typename E, int VEC>
__global__ __launch_bounds__(kThreads) void k_norm_bwd_apply(NormProblem p, MapPlan q,
                                                             const float* sums) {
  const int tx = threadIdx.x % q.tx, ty = threadIdx.x / q.tx;
  const int n = blockIdx.x / q.slabs, slab = blockIdx.x - n * q.slabs;
  const int c0 = (blockIdx.y * q.tx + tx) * VEC;
  if (c0 >= p.C) return;
  const int p0 = slab * q.ty + ty, step = q.slabs * q.ty;
  const long at = (long)n * p.P * p.C + c0;
  const E* x = static_cast<const E*>(p.x) + at;
  const E* dy = static_cast<const E*>(p.dy) + at;
  const E* gate = static_cast<const E*>(p.gate) + at;
  E* dx = static_cast<E*>(p.dx) + at;
  E* dgate = static_cast<E*>(p.dgate) + at;
  const bool gated = p.gate != nullptr;
  float mu[VEC], rs[VEC], w[VEC], b[VEC], s1[VEC], s2[VEC];
  load_stats<VEC>(p.mean + (long)n * p.G, 1, c0, p.cpg, mu);
  load_stats<VEC>(p.rstd + (long)n * p.G, 1, c0, p.cpg, rs);
  load_stats<VEC>(sums + 2L * n * p.G, 2, c0, p.cpg, s1);
  load_stats<VEC>(sums + 2L * n * p.G + 1, 2, c0, p.cpg, s2);
  load_params<VEC>(p.weight, c0, p.wide, 1.f, w);
  load_params<VEC>(p.bias, c0, p.wide, 0.f, b);
#pragma unroll 2
  for (int pos = p0; pos < p.P; pos += step) {
    float v[VEC], d[VEC], gt[VEC];
    Row<E, VEC>::load(x + (long)pos * p.C, v);
    Row<E, VEC>::load(dy + (long)pos * p.C, d);
    if (gated) Row<E, VEC>::load(gate + (long)pos * p.C, gt);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float hat = (v[i] - mu[i]) * rs[i];
      const float u = fmaf(hat, w[i], b[i]);
      const float gv = gated ? gt[i] : 0.f;
      const float du = norm_du(u, gv, d[i], gated, p.silu);
      if (gated) gt[i] = d[i] * u * act_slope(gv, p.silu);
      v[i] = rs[i] * (du * w[i] - s1[i] - hat * s2[i]);
    }
    Row<E, VEC>::store(dx + (long)pos * p.C, v);
    if (gated) Row<E, VEC>::store(dgate + (long)pos * p.C, gt);
  }
}

// dw and db from rows [rows][2][C] of partial sums.
__global__ __launch_bounds__(kColumnThreads) void k_norm_params(const float* ws, float* dw,
                                                                float* db, long rows, int C) {
  float* to = blockIdx.y == 0 ? dw : db;
  if (!to) return;
  const int c = blockIdx.x * 64 + lane_id();
  const float r = column_sum(ws + (long)blockIdx.y * C, 2L * C, rows, c, C);
  if (threadIdx.x < 64 && c < C) to[c] = r;
}

// --- one workgroup for each (sample, group) ----------------------------------------------------

template <typename E>
__global__ __launch_bounds__(kThreads) void k_norm_group(NormProblem p) {
  __shared__ float lds[4];
  const int n = blockIdx.x / p.G, g = blockIdx.x - n * p.G;
  const long at = (long)n * p.P * p.C + (long)g * p.cpg;
  const E* x = static_cast<const E*>(p.x) + at;
  const E* gate = static_cast<const E*>(p.gate) + at;
  E* y = static_cast<E*>(p.y) + at;
  const long items = (long)p.P * p.cpg;
  auto place = [&](long i) {
    const long pos = i / p.cpg;
    return pos * p.C + (i - pos * p.cpg);
  };
  float s = 0.f;
  for (long i = threadIdx.x; i < items; i += kThreads) s += (float)x[place(i)];
  const float inv = 1.f / ((float)p.P * (float)p.cpg);
  const float mean = block_sum(s, lds) * inv;
  float m2 = 0.f;
  for (long i = threadIdx.x; i < items; i += kThreads) {
    const float d = (float)x[place(i)] - mean;
    m2 = fmaf(d, d, m2);
  }
  const float rstd = rsqrtf(block_sum(m2, lds) * inv + p.eps);
  for (long i = threadIdx.x; i < items; i += kThreads) {
    const long o = place(i);
    const int c = g * p.cpg + (int)(i % p.cpg);
    const float u = fmaf(((float)x[o] - mean) * rstd, p.weight ? p.weight[c] : 1.f,
                         p.bias ? p.bias[c] : 0.f);
    y[o] = (E)norm_out(u, p.gate ? (float)gate[o] : 0.f, p.gate != nullptr, p.silu);
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[blockIdx.x] = mean;
    if (p.rstd) p.rstd[blockIdx.x] = rstd;
  }
}

// The mean and deviation of no values.
__global__ __launch_bounds__(kThreads) void k_norm_no_stats(float* mean, float* rstd, int n) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  if (mean) mean[i] = __builtin_nanf("");
  if (rstd) rstd[i] = __builtin_nanf("");
}

// --- plans ------------------------------------------------------------------------------------

bool all_aligned(const NormProblem& p, size_t bytes) {
  for (const void* q : {p.x, p.gate, (const void*)p.y, p.dy, (const void*)p.dx,
                        (const void*)p.dgate})
    if (reinterpret_cast<uintptr_t>(q) % bytes) return false;
  return true;
}

// The widest vector that divides `width` channels and that every pointer is aligned to.
int vector_of(const NormProblem& p, int width) {
  const size_t e = p.f32 ? 4 : 2;
  for (int v : {8, 4, 2})
    if (width % v == 0 && all_aligned(p, e * v < 16 ? e * v : 16)) return v;
  return 1;
}

int pow2_at_least(int n) {
  int v = 1;
  while (v < n) v *= 2;
  return v;
}

constexpr int kRowVecs = 4;       // vectors of a segment a lane holds, at most
constexpr int kWantGroups = 2048;  // workgroups of a map's pass
// workgroups that share out rows: four a CU, which all run at once (16384 gated rows of 4096 channels,
// in one run: 81 us; 107 with 512, 93 with 2048, 83 with 8192; 74 since y is stored past the caches)
constexpr int kRowGroups = 1024;

// Rows: P = 1 and a group that fits the lanes' registers.
bool row_plan(const NormProblem& p, int vec, RowPlan* q, int* k) {
  if (p.P != 1) return false;
  const int nv = p.cpg / vec;
  if (nv > kRowVecs * kThreads) return false;
  q->lps = nv > kRowVecs * 64 ? kThreads : pow2_at_least(nv);
  if (q->lps > 64 && q->lps < kThreads) q->lps = 64;
  *k = pow2_at_least((nv + q->lps - 1) / q->lps);
  const int segs = kThreads / q->lps;
  const int g = pow2_at_least(p.G);
  q->gp = g < segs ? g : segs;
  q->gblk = (p.G + q->gp - 1) / q->gp;
  const int rw = segs / q->gp;
  long wgs = (p.N + rw - 1L) / rw;
  const long most = (kRowGroups + q->gblk - 1) / q->gblk;
  q->wgs = (int)(wgs < most ? wgs : most);
  return true;
}

MapPlan map_plan(const NormProblem& p, int vec) {
  MapPlan q;
  const int nv = (p.C + vec - 1) / vec;
  q.tx = pow2_at_least(nv);
  if (q.tx > kThreads) q.tx = kThreads;
  q.ty = kThreads / q.tx;
  q.cblk = (nv + q.tx - 1) / q.tx;
  // enough workgroups to fill the GPU, but at least 16 positions a thread
  const long most = (p.P + 16L * q.ty - 1) / (16L * q.ty);
  const long want = (kWantGroups + (long)p.N * q.cblk - 1) / ((long)p.N * q.cblk);
  q.slabs = (int)(want < most ? want : most);
  return q;
}

// A (sample, group)'s pieces, slabs times channels, are joined by one workgroup, which many of them
// (few samples, wide groups) keep busy long after the passes; more than these are first folded over
// the slabs by a launch of its own.  8 maps of 4096 x 512, folded and not: forward 2048 pieces 31.1
// and 32.0 us, 4096 30.7 and 38.8, 32768 32.0 and 120; backward 8192 pieces 44.6 and 45.6, 16384 44.3
// and 49.1.  A map of 16384 x 4096 in one group takes 121 us forward and 145 backward, 11.6 and 1.82
// ms with its 4 million pieces joined at once.
constexpr int kFoldItems = 2048, kBwdFoldItems = 8192;
bool fold_slabs(const NormProblem& p, const MapPlan& q, int most) {
  return q.slabs > 1 && (long)q.slabs * p.cpg > most;
}

// Maps so small that one launch with short reads is quicker than three: at most this many values
// a (sample, group), or a row too wide for the lanes' registers.  bf16, one launch and three: 64
// groups of 630 values 4.7 and 20.7 us, 64 of 2560 10.5 and 21.1, 256 of 4096 (one channel each)
// 21.6 and 73; 256 of 8192 26.9 and 21.4.  Of many groups the three passes are already quicker near
// the bound, which does not look at their number: 8192 of 1024 32.9 and 30.9, 1024 of 4096 39.5 and
// 32.7, 2048 of 4096 35.6 and 23.1; 524288 of 64 take 498 and 553.
constexpr long kGroupItems = 4096;
bool group_shape(const NormProblem& p) { return p.P == 1 || (long)p.P * p.cpg <= kGroupItems; }

template <typename E, int VEC>
hipError_t fwd_vec(const NormProblem& p, hipStream_t st) {
  RowPlan r;
  int k;
  if (row_plan(p, VEC, &r, &k)) {
    const dim3 grid(r.wgs, r.gblk);
    if (k == 1) k_norm_rows<E, VEC, 1><<<grid, kThreads, 0, st>>>(p, r);
    else if (k == 2) k_norm_rows<E, VEC, 2><<<grid, kThreads, 0, st>>>(p, r);
    else k_norm_rows<E, VEC, 4><<<grid, kThreads, 0, st>>>(p, r);
    return hipGetLastError();
  }
  if (group_shape(p)) {
    k_norm_group<E><<<p.N * p.G, kThreads, 0, st>>>(p);
    return hipGetLastError();
  }
  const MapPlan q = map_plan(p, VEC);
  const dim3 grid(p.N * q.slabs, q.cblk);
  float* stats = p.ws + (long)p.N * q.slabs * 2 * p.C;
  float* mean = p.mean ? p.mean : stats;
  float* rstd = p.rstd ? p.rstd : stats + (long)p.N * p.G;
  k_norm_stats<E, VEC><<<grid, kThreads, 0, st>>>(p, q);
  const bool fold = fold_slabs(p, q, kFoldItems);
  if (fold) k_norm_fold<<<p.N * ((p.C + 63) / 64), kColumnThreads, 0, st>>>(p, q);
  k_norm_join<<<p.N * p.G, kThreads, 0, st>>>(p, q, fold, mean, rstd);
  k_norm_apply<E, VEC><<<grid, kThreads, 0, st>>>(p, q, mean, rstd);
  return hipGetLastError();
}

template <typename E, int VEC>
hipError_t bwd_vec(const NormProblem& p, hipStream_t st) {
  RowPlan r;
  int k;
  if (row_plan(p, VEC, &r, &k)) {
    const dim3 grid(r.wgs, r.gblk);
    if (k == 1) k_norm_rows_bwd<E, VEC, 1><<<grid, kThreads, 0, st>>>(p, r);
    else if (k == 2) k_norm_rows_bwd<E, VEC, 2><<<grid, kThreads, 0, st>>>(p, r);
    else k_norm_rows_bwd<E, VEC, 4><<<grid, kThreads, 0, st>>>(p, r);
    if (p.dweight || p.dbias)
      k_norm_params<<<dim3((p.C + 63) / 64, 2), kColumnThreads, 0, st>>>(
          p.ws, p.dweight, p.dbias, (long)grid.x * (kThreads / r.lps / r.gp), p.C);
    return hipGetLastError();
  }
  const MapPlan q = map_plan(p, VEC);
  const dim3 grid(p.N * q.slabs, q.cblk);
  float* sums = p.ws + (long)p.N * q.slabs * 2 * p.C;
  k_norm_bwd_sums<E, VEC><<<grid, kThreads, 0, st>>>(p, q);
  const bool fold = fold_slabs(p, q, kBwdFoldItems);
  if (fold) k_norm_bwd_fold<<<p.N * 2 * ((p.C + 63) / 64), kColumnThreads, 0, st>>>(p, q);
  k_norm_bwd_join<<<p.N * p.G + (p.C + 63) / 64 * 2, kColumnThreads, 0, st>>>(p, q, fold, sums);
  k_norm_bwd_apply<E, VEC><<<grid, kThreads, 0, st>>>(p, q, sums);
  return hipGetLastError();
}

template <bool BWD, typename E>
hipError_t launch_e(const NormProblem& given, hipStream_t st) {
  NormProblem p = given;
  p.wide = (reinterpret_cast<uintptr_t>(p.weight) | reinterpret_cast<uintptr_t>(p.bias)) % 16 == 0;
  // in a row a segment's vectors must not cross into the next group
  const int vec = vector_of(p, p.P == 1 ? p.cpg : p.C);
  if constexpr (BWD) {
    if (vec == 8) return bwd_vec<E, 8>(p, st);
    if (vec == 4) return bwd_vec<E, 4>(p, st);
    if (vec == 2) return bwd_vec<E, 2>(p, st);
    return bwd_vec<E, 1>(p, st);
  } else {
    if (vec == 8) return fwd_vec<E, 8>(p, st);
    if (vec == 4) return fwd_vec<E, 4>(p, st);
    if (vec == 2) return fwd_vec<E, 2>(p, st);
    return fwd_vec<E, 1>(p, st);
  }
}

}  // namespace

// The query cannot see the pointers' alignment, so it takes the largest need over the vectors.
size_t norm_workspace(const NormProblem& p, bool backward) {
  long most = 0;
  for (int vec : {8, 4, 2, 1}) {
    if ((p.P == 1 ? p.cpg : p.C) % vec) continue;
    RowPlan r;
    int k;
    long need = 0;
    if (row_plan(p, vec, &r, &k)) {
      if (backward) need = (long)r.wgs * (kThreads / r.lps / r.gp) * 2 * p.C;
    } else if (backward || !group_shape(p)) {
      need = (long)p.N * map_plan(p, vec).slabs * 2 * p.C + 2L * p.N * p.G;
    }
    if (need > most) most = need;
  }
  return (size_t)most * 4;
}

hipError_t launch_norm_fwd(const NormProblem& p, hipStream_t st) {
  return p.f32 ? launch_e<false, float>(p, st) : launch_e<false, bf16>(p, st);
}

hipError_t launch_norm_no_stats(const NormProblem& p, hipStream_t st) {
  if (!p.mean && !p.rstd) return hipSuccess;
  const int n = p.N * p.G;  // at most 2^21 where the positions are not 1
  k_norm_no_stats<<<(n + kThreads - 1) / kThreads, kThreads, 0, st>>>(p.mean, p.rstd, n);
  return hipGetLastError();
}

hipError_t launch_norm_no_params(const NormProblem& p, hipStream_t st) {
  if (!p.dweight && !p.dbias) return hipSuccess;
  k_norm_params<<<dim3((p.C + 63) / 64, 2), kColumnThreads, 0, st>>>(nullptr, p.dweight, p.dbias, 0,
                                                               p.C);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormProblem& p, hipStream_t st) {
  return p.f32 ? launch_e<true, float>(p, st) : launch_e<true, bf16>(p, st);
}

}  // namespace gdn
