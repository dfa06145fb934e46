// The gradient of linear attention with a decay for each head (linear.hip).  With dS the gradient of
// the state at a chunk's end, S the state at its start, G_t the sum of log-decays from its start,
// D_ij = e^{G_i - G_j} for j <= i and 0 above the diagonal,
//
//   M = scale (dO V^T) * D,  P = scale (Q K^T) * D
//   dQ = scale e^{G} dO S^T + M K          dK = e^{G_C - G} V dS^T + M^T Q
//   dV = e^{G_C - G} K dS + P^T dO         dS <- e^{G_C} dS + scale (e^{G} Q)^T dO
//
// A log-decay is in the product of every two tokens that lie on either side of it, of every earlier
// token with the chunk's and of the chunk's with every later one, and of what passes through:
//
//   dg_t = sum_{s >= t} (a_s + r_s) + sum_{s < t} b_s + e^{G_C} <dS, S>
//   a_s = q_s . (scale e^{G_s} S dO_s),  b_s = k_s . (e^{G_C - G_s} dS v_s)
//   r = rowsum(E) - colsum(E),  E = M * (Q K^T) below the diagonal
//
// Nothing here is a difference of sums that run over the sequence.  Within a chunk r does cancel, for
// the pairs that lie on one side of t: both its sums are taken in fp64 of the same fp32 values, so what
// is left is dg's own size however strong the decay at t.
//
// Two passes over the tokens: k_linear_state writes the state at every chunk's start (fp32, in the
// order of its tiles), then k_linear_bwd walks each segment's chunks from the last to the first with
// dS in registers and makes everything else.  dS is held by key rows: a wave has 16 of them and all
// value columns, so products over the value columns take it from registers; the one over key rows
// (dV) takes a copy rounded to bf16 from LDS.  Rounded to bf16 are M, P and that copy, once each; the
// products that make a, b and dS use three bf16 terms for what is not bf16 already.
#include "linear_device.h"

namespace gdn {

namespace {

// Sum over the 16 lanes of a row, in all of them: rotations within the row.
__device__ __forceinline__ double row_sum(double x) {
  x += dpp_d<0x128>(x);
  x += dpp_d<0x124>(x);
  x += dpp_d<0x122>(x);
  x += dpp_d<0x121>(x);
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
  x += dpp_f<0x128>(x);
  x += dpp_f<0x124>(x);
  x += dpp_f<0x122>(x);
  x += dpp_f<0x121>(x);
  return x;
}

template <typename E, int DK, int DV>
__global__ __launch_bounds__(DK * 4, 2) void k_linear_bwd(LinearProblem p, LinearBwd b) {
  constexpr int C = sizeof(E) == 2 ? kLinearChunk : kLinearChunkF32;
  constexpr int NW = DK / 16, NTH = 64 * NW, VT = DV / 16, TT = C / 16;
  constexpr int PAD = 16 / (int)sizeof(E), LK = DK + PAD, LV = DV + PAD, LP = C + PAD;
  constexpr int KF = Mx<E>::KF, KS = C / KF, TERMS = Mx<E>::TERMS, EPL = Mx<E>::EPL;
  typedef typename Mx<E>::frag frag;
  __shared__ __align__(16) E Qs[C * LK];
  __shared__ __align__(16) E Ks[C * LK];
  __shared__ __align__(16) E Vs[C * LV];
  __shared__ __align__(16) E Os[C * LV];   // dO
  __shared__ __align__(16) E Ds[DK * LV];  // dS, rounded
  __shared__ __align__(16) E Ps[C * LP];
  __shared__ __align__(16) E Ms[C * LP];
  __shared__ __align__(16) Decays<C> dec[2];
  __shared__ double rows[TT][C];  // E summed over a tile's columns, by tile column
  __shared__ double cols[TT][C];  // and over its rows, by tile row
  __shared__ float as[NW][C], bs[NW][C], cs[NW];

  const int unit = unit_of(blockIdx.x, gridDim.x, p.group);
  const int slot = unit / p.H, h = unit - slot * p.H;
  const int l = lane_id(), wave = uniform(wave_id()), lc = l & 15, lg = l >> 4;
  const Chunk c = uniform_chunk(p, slot);
  if (!c.ok) {
    if (b.dg && p.head_decay && threadIdx.x == 0) b.dgp[unit] = 0.f;
    return;
  }
  const int hk = h / (p.H / p.Hg);
  const long cell = (long)p.Dk * p.Dv;
  const int row = 16 * wave + lc;  // this lane's key row of the state

  f32x4 dS[VT];
  const float* from = p.Lc != kScanNoSplit ? b.grads + (long)unit * cell
                      : b.dht              ? b.dht + ((long)c.n * p.H + h) * cell
                                           : nullptr;
#pragma unroll
  for (int t = 0; t < VT; ++t)
    dS[t] = from && row < p.Dk && tile_row(t) < p.Dv
                ? *reinterpret_cast<const f32x4*>(from + (long)row * p.Dv + tile_row(t)) : zero4();

  const int64_t so = (int64_t)p.H * p.Dv;
  const E* qp = static_cast<const E*>(p.q) + c.t0 * p.sq + (long)hk * p.Dk;
  const E* kp = static_cast<const E*>(p.k) + c.t0 * p.sk + (long)hk * p.Dk;
  const E* vp = static_cast<const E*>(p.v) + c.t0 * p.sv + (long)h * p.Dv;
  const E* op = static_cast<const E*>(b.dout) + c.t0 * so + (long)h * p.Dv;
  E* dvp = static_cast<E*>(b.dv) + c.t0 * so + (long)h * p.Dv;
  // shared q/k heads: every value head's share in fp32, added by k_linear_shares
  const bool shares = p.H != p.Hg;
  const int64_t sg = (int64_t)p.H * p.Dk;  // p.H = p.Hg rows, or shares of p.H heads
  const long gat = c.t0 * sg + (long)h * p.Dk;
  const bool mine = 16 * wave + 4 * lg < p.Dk;

  Rows<E, DK, C, NTH> q, k;
  Rows<E, DV, C, NTH> v, o;
  q.open(p.sq, p.Dk, LK);
  k.open(p.sk, p.Dk, LK);
  v.open(p.sv, p.Dv, LV);
  o.open(so, p.Dv, LV);
  const int chunks = (c.len + C - 1) / C;
  auto fetch = [&](int m) {
    const int len = min(C, c.len - m * C);
    q.load(qp + (long)m * C * p.sq, p.sq, p.Dk, len);
    k.load(kp + (long)m * C * p.sk, p.sk, p.Dk, len);
    v.load(vp + (long)m * C * p.sv, p.sv, p.Dv, len);
    o.load(op + (long)m * C * so, so, p.Dv, len);
  };
  auto decay_of = [&](int m) {
    return load_decay(p, c.t0 + m * C, l, min(C, c.len - m * C), h);
  };
  float gnext = 0.f;
  if (chunks > 0) {
    fetch(chunks - 1);
    if (wave == NW - 1) {
      dec[(chunks - 1) & 1].make(decay_of(chunks - 1));
      if (chunks > 1) gnext = decay_of(chunks - 2);
    }
    // scores above the diagonal's tiles, and of the last chunk's rows past its end, stay zero
    for (int i = threadIdx.x; i < C * LP; i += NTH) Ps[i] = (E)0.f, Ms[i] = (E)0.f;
  }
  const ChunkMap map = {p.cu, p.T, p.Ttot, p.N, C};
  const int first = uniform(p.cu ? chunk_first(map, c.n) : c.n * chunk_count(p.T, C));
  const float* states = b.chunks + ((long)(first + (c.t0 - c.bos) / C) * p.H + h) * (DK * DV) +
                        wave * (DV * 16) + 4 * l;
  double gsum = 0.0;

  for (int m = chunks - 1; m >= 0; --m) {
    const int len = min(C, c.len - m * C);
    const Decays<C>& d = dec[m & 1];
    q.store(Qs, LK);
    k.store(Ks, LK);
    v.store(Vs, LV);
    o.store(Os, LV);
#pragma unroll
    for (int t = 0; t < VT; t += 2) {
      E* to = Ds + row * LV + tile_row(t);
      if constexpr (sizeof(E) == 2) {
        const bf16x4 x = __builtin_convertvector(dS[t], bf16x4),
                     y = __builtin_convertvector(dS[t + 1], bf16x4);
        *reinterpret_cast<bf16x8*>(to) = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
        *reinterpret_cast<f32x4*>(to) = dS[t];
        *reinterpret_cast<f32x4*>(to + 4) = dS[t + 1];
      }
    }
    __syncthreads();
    if (m > 0) fetch(m - 1);
    f32x4 S[VT];
#pragma unroll
    for (int t = 0; t < VT; ++t)
      S[t] = *reinterpret_cast<const f32x4*>(states + (long)m * p.H * (DK * DV) + t * 256);

    for (int x = wave; x < TT * (TT + 1) / 2; x += NW) {
      const int ti = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, tj = x - ti * (ti + 1) / 2;
      if (16 * ti >= len) break;
      f32x4 qk = zero4(), ov = zero4();
#pragma unroll
      for (int s = 0; s < DK / KF; ++s)
        qk = Mx<E>::mma(mx_ld<E>(Ks, LK, 16 * tj, KF * s), mx_ld<E>(Qs, LK, 16 * ti, KF * s), qk);
#pragma unroll
      for (int s = 0; s < DV / KF; ++s)
        ov = Mx<E>::mma(mx_ld<E>(Vs, LV, 16 * tj, KF * s), mx_ld<E>(Os, LV, 16 * ti, KF * s), ov);
      const int i = 16 * ti + lc, j = 16 * tj + 4 * lg;
      const double Gi = d.G[i];
      f32x4 pp, mm, ee;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = p.scale * exp2_f32((float)(Gi - d.G[j + e]));
        pp[e] = j + e <= i ? qk[e] * w : 0.f;
        mm[e] = j + e <= i ? ov[e] * w : 0.f;
        ee[e] = j + e < i ? mm[e] * qk[e] : 0.f;
      }
      E *tp = Ps + i * LP + j, *tm = Ms + i * LP + j;
      if constexpr (sizeof(E) == 2) {
        *reinterpret_cast<bf16x4*>(tp) = __builtin_convertvector(pp, bf16x4);
        *reinterpret_cast<bf16x4*>(tm) = __builtin_convertvector(mm, bf16x4);
      } else {
        *reinterpret_cast<f32x4*>(tp) = pp;
        *reinterpret_cast<f32x4*>(tm) = mm;
      }
      if (b.dg) {
        double r = ((double)ee[0] + ee[1]) + ((double)ee[2] + ee[3]);
        r += __shfl_xor(r, 16);
        r += __shfl_xor(r, 32);
        if (lg == 0) rows[tj][i] = r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double s = row_sum((double)ee[e]);
          if (lc == 0) cols[ti][j + e] = s;
        }
      }
    }
    if (wave == NW - 1 && m > 0) {
      dec[(m - 1) & 1].make(gnext);
      if (m > 1) gnext = decay_of(m - 2);
    }
    __syncthreads();

    const float keep = d.into[C - 1];
    if (b.dg) {
      float x = 0.f;
#pragma unroll
      for (int t = 0; t < VT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x = fmaf(S[t][e], dS[t][e], x);
      x = row_sum(x);
      x = group_sum(x);
      if (l == 0) cs[wave] = x;
    }
    const int n = (len + 15) / 16;
    const long at = gat + (long)m * C * sg;
    auto put = [&](int which, void* to, int t, f32x4 x) {
      if (shares) {
        const auto rs = rows_of(b.part + (which ? (long)p.Ttot * sg : 0) + at, sg, p.Dk, len);
        store4<float>(rs, mine ? (uint32_t)((16 * t + lc) * sg + 16 * wave + 4 * lg) * 4 : kNoColumn,
                      x);
      } else {
        const auto rs = rows_of(static_cast<E*>(to) + at, sg, p.Dk, len);
        store4<E>(rs, mine ? (uint32_t)((16 * t + lc) * sg + 16 * wave + 4 * lg) * (int)sizeof(E)
                           : kNoColumn, x);
      }
    };
    // dQ
    {
      StateOperand<E, VT, TERMS> f;
      f.from(S);
      frag kf[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) kf[s] = mx_tr<E, false>(Ks, LK, KF * s, 16 * wave);
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < n) {
          f32x4 x = f.times(Os, LV, 16 * t, zero4());
          x *= p.scale * d.into[16 * t + lc];
          if (b.dg) {
            float r = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              r = fmaf(x[e], (float)Qs[(16 * t + lc) * LK + 16 * wave + 4 * lg + e], r);
            r = group_sum(r);
            if (lg == 0) as[wave][16 * t + lc] = r;
          }
#pragma unroll
          for (int s = 0; s < KS; ++s)
            if (KF * s < 16 * (t + 1))
              x = Mx<E>::mma(kf[s], mx_ld<E>(Ms, LP, 16 * t, KF * s), x);
          put(0, b.dq, t, x);
        }
    }
    // dK, and dS for the chunk before
    {
      StateOperand<E, VT, TERMS> f;
      f.from(dS);
      frag qf[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) qf[s] = mx_tr<E, false>(Qs, LK, KF * s, 16 * wave);
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < n) {
          f32x4 x = f.times(Vs, LV, 16 * t, zero4());
          x *= d.left[16 * t + lc];
          if (b.dg) {
            float r = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              r = fmaf(x[e], (float)Ks[(16 * t + lc) * LK + 16 * wave + 4 * lg + e], r);
            r = group_sum(r);
            if (lg == 0) bs[wave][16 * t + lc] = r;
          }
#pragma unroll
          for (int s = 0; s < KS; ++s)
            if (KF * (s + 1) > 16 * t)
              x = Mx<E>::mma(qf[s], mx_tr<E, false>(Ms, LP, KF * s, 16 * t), x);
          put(1, b.dk, t, x);
        }
#pragma unroll
      for (int t = 0; t < VT; ++t) dS[t] *= keep;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float w[8];
#pragma unroll
        for (int e = 0; e < EPL; ++e)
          w[e] = (float)qf[s][e] * (p.scale * d.into[KF * s + EPL * lg + e]);
        frag x[TERMS];
        split<E>(w, x);
#pragma unroll
        for (int t = 0; t < VT; ++t) {
          const frag r = mx_tr<E, true>(Os, LV, KF * s, tile_col(t));
#pragma unroll
          for (int e = TERMS - 1; e >= 0; --e) dS[t] = Mx<E>::mma(r, x[e], dS[t]);
        }
      }
    }
    // dV
    for (int vt = wave; vt < VT; vt += NW) {
      frag of[KS], sf[DK / KF];
#pragma unroll
      for (int s = 0; s < KS; ++s) of[s] = mx_tr<E, false>(Os, LV, KF * s, 16 * vt);
#pragma unroll
      for (int s = 0; s < DK / KF; ++s) sf[s] = mx_tr<E, false>(Ds, LV, KF * s, 16 * vt);
      const auto rs = rows_of(dvp + (long)m * C * so, so, p.Dv, len);
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < n) {
          f32x4 x = zero4();
#pragma unroll
          for (int s = 0; s < DK / KF; ++s)
            x = Mx<E>::mma(sf[s], mx_ld<E>(Ks, LK, 16 * t, KF * s), x);
          x *= d.left[16 * t + lc];
#pragma unroll
          for (int s = 0; s < KS; ++s)
            if (KF * (s + 1) > 16 * t)
              x = Mx<E>::mma(of[s], mx_tr<E, false>(Ps, LP, KF * s, 16 * t), x);
          store4<E>(rs, 16 * vt + 4 * lg < p.Dv
                            ? (uint32_t)((16 * t + lc) * so + 16 * vt + 4 * lg) * (int)sizeof(E)
                            : kNoColumn, x);
        }
    }
    __syncthreads();
    // the others go on to the next chunk, which writes none of these before its second barrier
    if (b.dg && wave == 0) {
      double up = 0.0, down = 0.0, through = 0.0;
      if (l < len) {
        for (int t = 0; t <= l / 16; ++t) up += rows[t][l];
        for (int t = l / 16; t < n; ++t) up -= cols[t][l];
        for (int w = 0; w < NW; ++w) up += as[w][l], down += bs[w][l];
      }
      for (int w = 0; w < NW; ++w) through += cs[w];
      const double from0 = wave_incl_scan(up), before = wave_incl_scan(down) - down;
      double x = (last_lane(from0) - from0 + up) + before + keep * through;
      // nothing passes a decay that is 0 in fp32
      if (l < len && d.G[l] - (l > 0 ? d.G[l - 1] : 0.0) < -150.0) x = 0.0;
      if (l < len) {
        if (p.head_decay)
          gsum += x;
        else
          b.dg[(long)(c.t0 + m * C + l) * p.H + h] = (float)x;
      }
    }
  }

  if (b.dg && p.head_decay && wave == 0) {
    const double x = wave_incl_scan(gsum);
    if (l == 63) b.dgp[unit] = (float)x;
  }
  if (b.dh0 && c.i == 0 && row < p.Dk) {
    float* to = b.dh0 + ((long)c.n * p.H + h) * cell + (long)row * p.Dv;
#pragma unroll
    for (int t = 0; t < VT; ++t)
      if (tile_row(t) < p.Dv) *reinterpret_cast<f32x4*>(to + tile_row(t)) = dS[t];
  }
}

// The gradients of the states at the segments' ends from the segments' own shares, in place, last to
// first (k_linear_compose the other way round).
__global__ __launch_bounds__(256) void k_linear_compose_bwd(LinearProblem p, LinearBwd b) {
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
  if (b.dht) s = *reinterpret_cast<const f32x4*>(b.dht + ((long)n * p.H + h) * cell + at);
  for (int i = count - 1; i >= 0; --i) {
    const long sh = (long)(first + i) * p.H + h;
    f32x4* x = reinterpret_cast<f32x4*>(b.grads + sh * cell + at);
    if (i > 0) {
      const f32x4 own = *x;
      *x = s;
      s = s * exp2_f32(p.sums[sh]) + own;
    } else {
      *x = s;
    }
  }
}

// dq and dk of a q/k head: the sum of its value heads' shares, in order, four values a thread.
template <typename E>
__global__ __launch_bounds__(256) void k_linear_shares(LinearProblem p, LinearBwd b) {
  const long vecs = (long)p.Hg * p.Dk / 4, total = p.cu ? min(max(p.cu[p.N], 0), p.Ttot) : p.Ttot;
  const long at = (long)blockIdx.x * 256 + threadIdx.x;
  if (at >= total * vecs) return;
  const long t = at / vecs;
  const int x = (int)(at - t * vecs) * 4, hk = x / p.Dk, col = x - hk * p.Dk, rep = p.H / p.Hg;
  const float* from = b.part + (blockIdx.y ? (long)p.Ttot * p.H * p.Dk : 0) +
                      (t * p.H + (long)hk * rep) * p.Dk + col;
  f32x4 s = zero4();
  for (int r = 0; r < rep; ++r) s += *reinterpret_cast<const f32x4*>(from + (long)r * p.Dk);
  E* to = static_cast<E*>(blockIdx.y ? b.dk : b.dq) + at * 4;
  if constexpr (sizeof(E) == 2)
    *reinterpret_cast<bf16x4*>(to) = __builtin_convertvector(s, bf16x4);
  else
    *reinterpret_cast<f32x4*>(to) = s;
}

__global__ __launch_bounds__(kColumnThreads) void k_linear_heads(const float* part, float* dg,
                                                                 int slots, int H) {
  const int c = blockIdx.x * 64 + lane_id();
  const float s = column_sum(part, H, slots, c, H);
  if (threadIdx.x < 64 && c < H) dg[c] = s;
}

template <typename E, int DK, int DV>
hipError_t launch_grads(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  const int blocks = p.slots * p.H;
  LinearProblem q = p;
  q.group = group_of(p, 1, blocks);
  k_linear_bwd<E, DK, DV><<<blocks, DK * 4, 0, st>>>(q, b);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_grads_e(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  if (p.Dv <= 64)
    return p.Dk <= 64 ? launch_grads<E, 64, 64>(p, b, st) : launch_grads<E, 128, 64>(p, b, st);
  return p.Dk <= 64 ? launch_grads<E, 64, 128>(p, b, st) : launch_grads<E, 128, 128>(p, b, st);
}

template <typename E>
hipError_t launch_shares(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  const long vecs = (long)p.Ttot * p.Hg * p.Dk / 4;
  k_linear_shares<E><<<dim3((unsigned)((vecs + 255) / 256), 2), 256, 0, st>>>(p, b);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_bwd(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (p.slots > 0) {
    LinearPass a = {};
    a.x = p.k;
    a.y = p.v;
    a.sx = p.sk;
    a.sy = p.sv;
    if (p.Lc != kScanNoSplit) {
      a.own = p.states;
      e = launch_linear_state(p, a, st);
      if (e == hipSuccess) e = launch_linear_compose(p, st);
      LinearPass r = {};
      r.x = p.q;
      r.y = b.dout;
      r.sx = p.sq;
      r.sy = (int64_t)p.H * p.Dv;
      r.reverse = true;
      r.own = b.grads;
      if (e == hipSuccess) e = launch_linear_state(p, r, st);
      if (e != hipSuccess) return e;
      const long blocks = ((long)p.Dk * p.Dv / 4 + 255) / 256 * p.N * p.H;
      k_linear_compose_bwd<<<(unsigned)blocks, 256, 0, st>>>(p, b);
      e = hipGetLastError();
    }
    a.own = nullptr;
    a.chunks = b.chunks;
    if (e == hipSuccess && p.Ttot > 0) e = launch_linear_state(p, a, st);
    if (e == hipSuccess)
      e = p.f32 ? launch_grads_e<float>(p, b, st) : launch_grads_e<bf16>(p, b, st);
    if (e == hipSuccess && p.H != p.Hg && p.Ttot > 0)
      e = p.f32 ? launch_shares<float>(p, b, st) : launch_shares<bf16>(p, b, st);
    if (e != hipSuccess) return e;
  }
  if (b.dg && p.head_decay) {
    k_linear_heads<<<(p.H + 63) / 64, kColumnThreads, 0, st>>>(b.dgp, b.dg, p.slots, p.H);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace gdn
