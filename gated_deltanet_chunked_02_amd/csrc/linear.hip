// Linear attention with a decay for each head, prompts.  For a value head with q/k head hk,
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t
//
// evaluated in chunks of C tokens (64 in bf16, 32 in fp32).  With G_t the sum of log-decays from the
// chunk's start and S the state there,
//
//   o_i = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
//
// Every factor is the decay between two tokens, at most 1 for g <= 0, and nothing is divided.
//
// k_linear_fwd: a workgroup has one head of one segment of a sequence and up to 128 of its value
// columns, 16 a wave, whose state stays in registers (as tiles that are operands themselves,
// linear_device.h) from the segment's first chunk to its last.  q, k and v go through LDS, the next
// chunk's in registers meanwhile; the C x C scores are shared out over the waves and come back as
// bf16.  Two tensors are rounded to bf16 on the way to o, the scores and the state that meets q, one
// rounding on each of the two paths; the state itself and what is added to it are held to fp32's last
// bits (v times its decay enters as three bf16 terms).
//
// Few or long sequences are cut into segments: k_linear_state makes each segment's own end state
// (k and v alone), k_linear_compose turns those into start states in order, and k_linear_fwd runs
// the segments side by side.
#include "linear_device.h"

namespace gdn {

namespace {

template <typename E, int DK, int DV, int OCC>
__global__ __launch_bounds__(DV * 4, OCC) void k_linear_fwd(LinearProblem p) {
  constexpr int C = sizeof(E) == 2 ? kLinearChunk : kLinearChunkF32;
  constexpr int NTH = DV * 4, NW = DV / 16, KT = DK / 16, TT = C / 16, PAD = 16 / (int)sizeof(E);
  constexpr int LK = DK + PAD, LV = DV + PAD, LP = C + PAD, KF = Mx<E>::KF, KS = C / KF;
  constexpr int TERMS = Mx<E>::TERMS;
  typedef typename Mx<E>::frag frag;
  __shared__ __align__(16) E Qs[C * LK];
  __shared__ __align__(16) E Ks[C * LK];
  __shared__ __align__(16) E Vs[C * LV];
  __shared__ __align__(16) E Ps[C * LP];
  __shared__ __align__(16) Decays<C> dec[2];

  const int slabs = (p.Dv + DV - 1) / DV;
  const int unit = unit_of(blockIdx.x, gridDim.x, p.group);
  const int slab = unit % slabs, sh = unit / slabs, slot = sh / p.H, h = sh - slot * p.H;
  const Chunk c = uniform_chunk(p, slot);
  if (!c.ok) return;
  const int l = lane_id(), wave = uniform(wave_id()), lc = l & 15, lg = l >> 4;
  const int hk = h / (p.H / p.Hg), v0 = slab * DV, width = min(DV, p.Dv - v0);
  const int col = v0 + 16 * wave + lc;  // this lane's state column
  const long cell = (long)p.Dk * p.Dv;

  f32x4 S[KT];
  const float* from = p.Lc != kScanNoSplit ? p.states + ((long)slot * p.H + h) * cell
                      : p.h0               ? p.h0 + ((long)c.n * p.H + h) * cell
                                           : nullptr;
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      S[t][i] = from && tile_row(t) + i < p.Dk && col < p.Dv
                    ? from[(long)(tile_row(t) + i) * p.Dv + col] : 0.f;

  const E* qp = static_cast<const E*>(p.q) + c.t0 * p.sq + (long)hk * p.Dk;
  const E* kp = static_cast<const E*>(p.k) + c.t0 * p.sk + (long)hk * p.Dk;
  const E* vp = static_cast<const E*>(p.v) + c.t0 * p.sv + (long)h * p.Dv + v0;
  const int64_t so = (int64_t)p.H * p.Dv;
  E* op = static_cast<E*>(p.o) + c.t0 * so + (long)h * p.Dv + v0;
  const uint32_t oat = 16 * wave + 4 * lg < width
                           ? (uint32_t)((lc * so + 16 * wave + 4 * lg) * sizeof(E)) : kNoColumn;
  const uint32_t ostep = 16 * wave + 4 * lg < width ? (uint32_t)(16 * so * sizeof(E)) : 0;

  Rows<E, DK, C, NTH> q, k;
  Rows<E, DV, C, NTH> v;
  q.open(p.sq, p.Dk, LK);
  k.open(p.sk, p.Dk, LK);
  v.open(p.sv, width, LV);
  const int chunks = (c.len + C - 1) / C;
  float gnext = 0.f;
  auto fetch = [&](int m) {
    const int len = min(C, c.len - m * C);
    q.load(qp + (long)m * C * p.sq, p.sq, p.Dk, len);
    k.load(kp + (long)m * C * p.sk, p.sk, p.Dk, len);
    v.load(vp + (long)m * C * p.sv, p.sv, width, len);
  };
  if (chunks > 0) {
    fetch(0);
    if (wave == NW - 1) {
      dec[0].make(load_decay(p, c.t0, l, min(C, c.len), h));
      if (chunks > 1) gnext = load_decay(p, c.t0 + C, l, min(C, c.len - C), h);
    }
    // scores above the diagonal's tiles are never written, and read where a product's k covers two
    for (int i = threadIdx.x; i < C * LP; i += NTH) Ps[i] = (E)0.f;
  }

  for (int m = 0; m < chunks; ++m) {
    const int len = min(C, c.len - m * C);
    const Decays<C>& d = dec[m & 1];
    q.store(Qs, LK);
    k.store(Ks, LK);
    v.store(Vs, LV);
    __syncthreads();
    if (m + 1 < chunks) fetch(m + 1);

    // scores: the lower tiles, rows j of tile tj against columns i of tile ti
    for (int x = wave; x < TT * (TT + 1) / 2; x += NW) {
      const int ti = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, tj = x - ti * (ti + 1) / 2;
      if (16 * ti >= len) break;
      f32x4 a = zero4();
#pragma unroll
      for (int s = 0; s < DK / KF; ++s)
        a = Mx<E>::mma(mx_ld<E>(Ks, LK, 16 * tj, KF * s), mx_ld<E>(Qs, LK, 16 * ti, KF * s), a);
      const int i = 16 * ti + lc, j = 16 * tj + 4 * lg;
      const double Gi = d.G[i];
      E* to = Ps + i * LP + j;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x2 = a[e] * exp2_f32((float)(Gi - d.G[j + e]));
        a[e] = j + e <= i ? x2 : 0.f;
      }
      if constexpr (sizeof(E) == 2)
        *reinterpret_cast<bf16x4*>(to) = __builtin_convertvector(a, bf16x4);
      else
        *reinterpret_cast<f32x4*>(to) = a;
    }
    if (wave == NW - 1 && m + 1 < chunks) {
      dec[(m + 1) & 1].make(gnext);
      if (m + 2 < chunks)
        gnext = load_decay(p, c.t0 + (m + 2) * C, l, min(C, c.len - (m + 2) * C), h);
    }
    // the state's share
    f32x4 acc[TT];
    {
      StateOperand<E, KT, 1> f;
      f.from(S);
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (16 * t < len) {
          acc[t] = f.times(Qs, LK, 16 * t, zero4());
          acc[t] *= d.into[16 * t + lc];
        }
    }
    __syncthreads();

    frag vf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) vf[s] = mx_tr<E, false>(Vs, LV, KF * s, 16 * wave);
    const __amdgpu_buffer_rsrc_t ors = rows_of(op + (long)m * C * so, so, width, len);
#pragma unroll
    for (int t = 0; t < TT; ++t)
      if (16 * t < len) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
          if (KF * s < 16 * (t + 1))
            acc[t] = Mx<E>::mma(vf[s], mx_ld<E>(Ps, LP, 16 * t, KF * s), acc[t]);
        store4<E>(ors, oat + t * ostep, acc[t] * p.scale);
      }

    // the state: v times its decay as TERMS operands
    const float keep = d.into[C - 1];
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] *= keep;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8];
#pragma unroll
      for (int e = 0; e < Mx<E>::EPL; ++e)
        x[e] = (float)vf[s][e] * d.left[KF * s + Mx<E>::EPL * lg + e];
      frag f[TERMS];
      split<E>(x, f);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const frag a = mx_tr<E, true>(Ks, LK, KF * s, tile_col(t));
#pragma unroll
        for (int e = TERMS - 1; e >= 0; --e) S[t] = Mx<E>::mma(a, f[e], S[t]);
      }
    }
    __syncthreads();
  }

  if (p.ht && c.i == c.count - 1 && col < p.Dv) {
    float* to = p.ht + ((long)c.n * p.H + h) * cell + col;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (tile_row(t) + i < p.Dk) to[(long)(tile_row(t) + i) * p.Dv] = S[t][i];
  }
}

// Start states from the segments' own end states, in place: a thread has four values of a state
// and walks its sequence's segments.
__global__ __launch_bounds__(256) void k_linear_compose(LinearProblem p) {
  const long cell = (long)p.Dk * p.Dv;
  const int blocks = (int)((cell / 4 + 255) / 256);
  const int nh = blockIdx.x / blocks, n = nh / p.H, h = nh - n * p.H;
  const long at = ((long)(blockIdx.x - nh * blocks) * 256 + threadIdx.x) * 4;
  if (at >= cell) return;
  const ChunkMap m = {p.cu, p.T, p.Ttot, p.N, p.Lc};
  int bos, eos;
  chunk_seq(m, n, bos, eos);
  const int count = chunk_count(eos - bos, p.Lc);
  const int first = p.cu ? chunk_first(m, n) : n * count;
  f32x4 s = zero4();
  if (p.h0) s = *reinterpret_cast<const f32x4*>(p.h0 + ((long)n * p.H + h) * cell + at);
  for (int i = 0; i < count; ++i) {
    const long sh = (long)(first + i) * p.H + h;
    f32x4* x = reinterpret_cast<f32x4*>(p.states + sh * cell + at);
    if (i + 1 < count) {
      const f32x4 own = *x;
      *x = s;
      s = s * exp2_f32(p.sums[sh]) + own;
    } else {
      *x = s;
    }
  }
}

// Sums of outer products x_t y_t^T over a segment, without its outputs: forward (x = k, y = v, decays
// to the chunk's end), or in REV backward (x = q, y = dout, decays from the chunk's start, the last
// chunk first: the gradients of states).  Wave w holds columns of x (rows of the state) as tiles over
// y.  STORE: from the segment's start state on, every chunk's start state is written out in the
// tiles' order; otherwise the segment's own sum alone, from zero, and its decay.
template <typename E, int DK, int DV, bool REV, bool STORE>
__global__ __launch_bounds__(DK < 128 ? DK * 4 : 512, 2) void k_linear_state(LinearProblem p,
                                                                          LinearPass a) {
  constexpr int C = sizeof(E) == 2 ? kLinearChunk : kLinearChunkF32;
  constexpr int NW = DK < 128 ? DK / 16 : 8, NTH = 64 * NW, TK = DK / 16 / NW, VT = DV / 16;
  constexpr int PAD = 16 / (int)sizeof(E), LX = DK + PAD, LY = DV + PAD;
  constexpr int KF = Mx<E>::KF, KS = C / KF, TERMS = Mx<E>::TERMS;
  typedef typename Mx<E>::frag frag;
  __shared__ __align__(16) E Xs[C * LX];
  __shared__ __align__(16) E Ys[C * LY];
  __shared__ __align__(16) Decays<C> dec[2];

  const int slabs = (p.Dv + DV - 1) / DV;
  const int unit = unit_of(blockIdx.x, gridDim.x, p.group);
  const int slab = unit % slabs, sh = unit / slabs, slot = sh / p.H, h = sh - slot * p.H;
  const Chunk c = uniform_chunk(p, slot);
  // nothing comes after the last segment (before the first)
  if (!c.ok || (!STORE && c.i == (REV ? 0 : c.count - 1))) return;
  const int l = lane_id(), wave = uniform(wave_id()), lc = l & 15, lg = l >> 4;
  const int hk = h / (p.H / p.Hg), v0 = slab * DV, width = min(DV, p.Dv - v0);
  const long cell = (long)p.Dk * p.Dv, at = ((long)slot * p.H + h) * cell;

  f32x4 S[TK][VT];
  const float* from = !STORE                 ? nullptr
                      : p.Lc != kScanNoSplit ? p.states + at
                      : p.h0                 ? p.h0 + ((long)c.n * p.H + h) * cell
                                             : nullptr;
#pragma unroll
  for (int j = 0; j < TK; ++j)
#pragma unroll
    for (int t = 0; t < VT; ++t) {
      const int row = 16 * (wave * TK + j) + lc, y = tile_row(t);
      S[j][t] = from && row < p.Dk && y < width
                    ? *reinterpret_cast<const f32x4*>(from + (long)row * p.Dv + v0 + y) : zero4();
    }

  const E* xp = static_cast<const E*>(a.x) + c.t0 * a.sx + (long)hk * p.Dk;
  const E* yp = static_cast<const E*>(a.y) + c.t0 * a.sy + (long)h * p.Dv + v0;
  Rows<E, DK, C, NTH> x;
  Rows<E, DV, C, NTH> y;
  x.open(a.sx, p.Dk, LX);
  y.open(a.sy, width, LY);
  const int chunks = (c.len + C - 1) / C;
  auto chunk_at = [&](int m) { return REV ? chunks - 1 - m : m; };
  auto fetch = [&](int m) {
    const int len = min(C, c.len - m * C);
    x.load(xp + (long)m * C * a.sx, a.sx, p.Dk, len);
    y.load(yp + (long)m * C * a.sy, a.sy, width, len);
  };
  auto decay_of = [&](int m) {
    return load_decay(p, c.t0 + m * C, l, min(C, c.len - m * C), h);
  };
  double sum = 0.0;
  float gnext = 0.f;
  if (chunks > 0) {
    fetch(chunk_at(0));
    if (wave == NW - 1) {
      sum = dec[0].make(decay_of(chunk_at(0)));
      if (chunks > 1) gnext = decay_of(chunk_at(1));
    }
  }
  float* out = nullptr;
  if constexpr (STORE) {
    const ChunkMap map = {p.cu, p.T, p.Ttot, p.N, C};
    const int first = uniform(p.cu ? chunk_first(map, c.n) : c.n * chunk_count(p.T, C));
    out = a.chunks + ((long)(first + (c.t0 - c.bos) / C) * p.H + h) * (DK * DV);
  }

  for (int m = 0; m < chunks; ++m) {
    const Decays<C>& d = dec[m & 1];
    if constexpr (STORE) {
      float* to = out + (long)m * p.H * (DK * DV) + 4 * l;
#pragma unroll
      for (int j = 0; j < TK; ++j)
#pragma unroll
        for (int t = 0; t < VT; ++t)
          *reinterpret_cast<f32x4*>(to + ((wave * TK + j) * VT + t) * 256) = S[j][t];
    }
    x.store(Xs, LX);
    y.store(Ys, LY);
    __syncthreads();
    if (m + 1 < chunks) {
      fetch(chunk_at(m + 1));
      if (wave == NW - 1) {
        sum += dec[(m + 1) & 1].make(gnext);
        if (m + 2 < chunks) gnext = decay_of(chunk_at(m + 2));
      }
    }
    const float keep = d.into[C - 1];
#pragma unroll
    for (int j = 0; j < TK; ++j)
#pragma unroll
      for (int t = 0; t < VT; ++t) S[j][t] *= keep;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      frag f[TK][TERMS];
#pragma unroll
      for (int j = 0; j < TK; ++j) {
        const frag b = mx_tr<E, false>(Xs, LX, KF * s, 16 * (wave * TK + j));
        float w[8];
#pragma unroll
        for (int e = 0; e < Mx<E>::EPL; ++e) {
          const int i = KF * s + Mx<E>::EPL * lg + e;
          w[e] = (float)b[e] * (REV ? p.scale * d.into[i] : d.left[i]);
        }
        split<E>(w, f[j]);
      }
#pragma unroll
      for (int t = 0; t < VT; ++t) {
        const frag r = mx_tr<E, true>(Ys, LY, KF * s, tile_col(t));
#pragma unroll
        for (int j = 0; j < TK; ++j)
#pragma unroll
          for (int e = TERMS - 1; e >= 0; --e) S[j][t] = Mx<E>::mma(r, f[j][e], S[j][t]);
      }
    }
    __syncthreads();
  }
  if constexpr (!STORE) {
#pragma unroll
    for (int j = 0; j < TK; ++j)
#pragma unroll
      for (int t = 0; t < VT; ++t) {
        const int row = 16 * (wave * TK + j) + lc, y0 = tile_row(t);
        if (row < p.Dk && y0 < width)
          *reinterpret_cast<f32x4*>(a.own + at + (long)row * p.Dv + v0 + y0) = S[j][t];
      }
    if (slab == 0 && threadIdx.x == NTH - 1) p.sums[(long)slot * p.H + h] = (float)sum;
  }
}

template <typename E, int DK, int DV, int OCC>
hipError_t launch_fwd(const LinearProblem& p, hipStream_t st) {
  const int slabs = (p.Dv + DV - 1) / DV;
  const int blocks = p.slots * p.H * slabs;
  LinearProblem q = p;
  q.group = group_of(p, slabs, blocks);
  k_linear_fwd<E, DK, DV, OCC><<<blocks, DV * 4, 0, st>>>(q);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_fwd_e(const LinearProblem& p, hipStream_t st) {
  if (p.Dv <= 64) {
    if (p.Dk <= 64) return launch_fwd<E, 64, 64, 2>(p, st);
    if (p.Dk <= 128) return launch_fwd<E, 128, 64, 2>(p, st);
    return launch_fwd<E, 256, 64, 1>(p, st);
  }
  if (p.Dk <= 64) return launch_fwd<E, 64, 128, 2>(p, st);
  if (p.Dk <= 128) return launch_fwd<E, 128, 128, 4>(p, st);
  return launch_fwd<E, 256, 128, 2>(p, st);
}

template <typename E, int DK, int DV>
hipError_t launch_state(const LinearProblem& p, const LinearPass& a, hipStream_t st) {
  const int slabs = (p.Dv + DV - 1) / DV;
  const int blocks = p.slots * p.H * slabs;
  LinearProblem q = p;
  q.group = group_of(p, slabs, blocks);
  constexpr int NTH = DK < 128 ? DK * 4 : 512;
  if (a.reverse)
    k_linear_state<E, DK, DV, true, false><<<blocks, NTH, 0, st>>>(q, a);
  else if (!a.chunks)
    k_linear_state<E, DK, DV, false, false><<<blocks, NTH, 0, st>>>(q, a);
  else if constexpr (DK <= 128)
    k_linear_state<E, DK, DV, false, true><<<blocks, NTH, 0, st>>>(q, a);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

template <typename E>
hipError_t launch_state_e(const LinearProblem& p, const LinearPass& a, hipStream_t st) {
  if (p.Dv <= 64) {
    if (p.Dk <= 64) return launch_state<E, 64, 64>(p, a, st);
    if (p.Dk <= 128) return launch_state<E, 128, 64>(p, a, st);
    return launch_state<E, 256, 64>(p, a, st);
  }
  if (p.Dk <= 64) return launch_state<E, 64, 128>(p, a, st);
  if (p.Dk <= 128) return launch_state<E, 128, 128>(p, a, st);
  return launch_state<E, 256, 128>(p, a, st);
}

}  // namespace

hipError_t launch_linear_state(const LinearProblem& p, const LinearPass& a, hipStream_t st) {
  return p.f32 ? launch_state_e<float>(p, a, st) : launch_state_e<bf16>(p, a, st);
}

hipError_t launch_linear_compose(const LinearProblem& p, hipStream_t st) {
  const long blocks = ((long)p.Dk * p.Dv / 4 + 255) / 256 * p.N * p.H;
  k_linear_compose<<<(unsigned)blocks, 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_linear_fwd(const LinearProblem& p, hipStream_t st) {
  if (p.Lc != kScanNoSplit) {
    LinearPass a = {};
    a.x = p.k;
    a.y = p.v;
    a.sx = p.sk;
    a.sy = p.sv;
    a.own = p.states;
    hipError_t e = launch_linear_state(p, a, st);
    if (e == hipSuccess) e = launch_linear_compose(p, st);
    if (e != hipSuccess) return e;
  }
  return p.f32 ? launch_fwd_e<float>(p, st) : launch_fwd_e<bf16>(p, st);
}

}  // namespace gdn
