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
// Two passes over the tokens.  Forwards, dQ is the recurrence itself over other tensors
// (k_linear_fwd with GRAD, which also leaves a); backwards, k_linear_bwd makes the rest with dS in
// registers.  Neither has both states, so what passes through a chunk comes from <dS, S> at its end,
//
//   e^{G_C} <dS, S_start> = <dS, S_end> - sum b,    <dS, S>_start = <dS, S>_end + sum a - sum b,
//
// carried in fp64 from chunk to chunk and taken afresh at the anchors (every 8 chunks at most), where the forward
// pass leaves its state: a difference of sums over 512 tokens at most, each term good to fp32's last
// bits, so dg keeps fp32's accuracy.  A head's own decay sums all of a sequence's dg, and with it one error
// many times over: there anchors are twice as many, and what the carried value is off by at each is
// taken off the sum, as having grown evenly since the last (dg of 64 heads, 824 tokens, fp32: relative
// error 1.1e-6 without that, 4.5e-7 with it at every 8 chunks).  Within a chunk r cancels for the pairs on
// one side of t: both its sums are taken in fp64 of the same fp32 values, so what is left has dg's own
// size.
//
// dS is held by key rows: a wave has 16 of them and all value columns, so the product over the value
// columns (dK) takes it from registers as three bf16 terms (its b is a term of dg); the one over key rows
// (dV) takes it from LDS as two, like M and P: 16 bits or more of each value, so that every output is fp32
// sums rounded once (with one term, dv of a carried gradient came out 1.25 times as far off, and the
// gradient took 4 % less).
//
// Measured (8 x 2048 tokens, 32 heads of 128 x 128, bf16): dQ's pass 223 us and this one 326, a workgroup a
// CU (158 KB of LDS), vector units busy 47 %, matrix units 23 %, LDS 30 %, the waves waiting 29 % of their
// cycles (43 % and a twelfth longer with every operand read where it is used).
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

template <bool FIRST, typename A, typename B> struct Pick { typedef A type; };
template <typename A, typename B> struct Pick<false, A, B> { typedef B type; };

// One workgroup walks a segment's chunks from the last to the first; a wave has 16 key rows of dS.
template <typename E, int DK, int DV, bool SHARES>
__global__ __launch_bounds__(DK * 4, 2) void k_linear_bwd(LinearProblem p, LinearBwd b) {
  constexpr int C = sizeof(E) == 2 ? kLinearChunk : kLinearChunkF32;
  constexpr int NW = DK / 16, NTH = 64 * NW, VT = DV / 16, TT = C / 16;
  constexpr int KF = Mx<E>::KF, KS = C / KF, TERMS = Mx<E>::TERMS, EPL = Mx<E>::EPL;
  constexpr int STEPS = sizeof(E) == 2 ? VT / 2 : VT;
  typedef typename Mx<E>::frag frag;
  typedef Tile<E, DK> TK;
  typedef Tile<E, DV> TV;
  typedef Tile<E, C> TP;
  __shared__ __align__(256) E Qs[C * TK::LD];
  __shared__ __align__(256) E Ks[C * TK::LD];
  __shared__ __align__(256) E Vs[C * TV::LD];
  __shared__ __align__(256) E Os[C * TV::LD];   // dO
  // dS as two bf16 terms (or as itself): the second one's first C rows take the place of V, which a
  // chunk's last products do not read
  constexpr bool TWO = sizeof(E) == 2;
  __shared__ __align__(256) E Ds[DK * TV::LD];
  __shared__ __align__(256) E Dl[TWO && DK > C ? (DK - C) * TV::LD : 1];
  __shared__ Scores<E, C> Ps, Ms;
  __shared__ __align__(16) Decays<C> dec[2];
  __shared__ double rows[TT][C];  // E summed over a tile's columns, by tile column
  __shared__ double cols[TT][C];  // and over its rows, by tile row
  __shared__ double bs[NW][C];
  // <dS, S> by waves, two anchors may follow each other: where rows has nothing, in front of its last
  // tile column's diagonal
  static_assert(2 * NW <= 16 && TT > 1, "cs fits into a tile's width");
  double* const cs = rows[TT - 1];

  const int unit = unit_of(blockIdx.x, gridDim.x, p.group);
  const int slot = unit / p.H, h = unit - slot * p.H;
  const int l = lane_id(), wave = uniform(wave_id());
  const Chunk c = uniform_chunk(p, slot);
  if (!c.ok) {
    if (p.head_decay && threadIdx.x == 0) b.dgp[unit] = 0.0;
    return;
  }
  const int hk = h / (p.H / p.Hg);
  const long cell = (long)p.Dk * p.Dv;

  const bool made = p.Lc != kScanNoSplit && (c.i + 1 < c.count || !b.direct);
  const float* from = made    ? b.grads + (long)unit * cell
                      : b.dht ? b.dht + ((long)c.n * p.H + h) * cell
                              : nullptr;
  // a state's rows through a buffer: this lane's, four columns at a time
  const __amdgpu_buffer_rsrc_t frs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(from), 0, from ? (int)cell * 4 : 0, 0x00020000);
  f32x4 dS[VT];
#pragma unroll
  for (int t = 0; t < VT; ++t)
    dS[t] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
        frs, tile_row(t, l) < p.Dv
                 ? (uint32_t)((16 * wave + (l & 15)) * p.Dv + tile_row(t, l)) * 4 : kNoColumn, 0, 0));

  const int64_t so = (int64_t)p.H * p.Dv;
  const E* qp = static_cast<const E*>(p.q) + c.t0 * p.sq + (long)hk * p.Dk;
  const E* kp = static_cast<const E*>(p.k) + c.t0 * p.sk + (long)hk * p.Dk;
  const E* vp = static_cast<const E*>(p.v) + c.t0 * p.sv + (long)h * p.Dv;
  const E* op = static_cast<const E*>(b.dout) + c.t0 * so + (long)h * p.Dv;
  E* dvp = static_cast<E*>(b.dv) + c.t0 * so + (long)h * p.Dv;
  // dk, or with shared q/k heads every value head's share of it in fp32 (added up by
  // k_linear_shares): rows of H heads either way
  typedef typename Pick<SHARES, float, E>::type G;
  const int64_t sg = (int64_t)p.H * p.Dk;
  G* gp = (SHARES ? reinterpret_cast<G*>(b.part) + (long)p.Ttot * sg : static_cast<G*>(b.dk)) +
          c.t0 * sg + (long)h * p.Dk;

  Rows<E, DK, C, NTH> q, k;
  Rows<E, DV, C, NTH> v, o;
  const int chunks = (c.len + C - 1) / C;
  auto fetch = [&](int m, int tid) {  // nothing before the first chunk
    const int len = m < 0 ? 0 : min(C, c.len - m * C);
    q.load(qp + (long)m * C * p.sq, p.sq, p.Dk, len, tid);
    k.load(kp + (long)m * C * p.sk, p.sk, p.Dk, len, tid);
    v.load(vp + (long)m * C * p.sv, p.sv, p.Dv, len, tid);
    o.load(op + (long)m * C * so, so, p.Dv, len, tid);
  };
  auto decay_of = [&](int m) {
    return load_decay(p, c.t0 + (long)m * C, m < 0 ? 0 : min(C, c.len - m * C), h);
  };
  f32x4 S[VT];  // at the next anchor, this wave's part
  const int anchors = first_anchor(p, c, b.every, C);
  auto fetch_state = [&](int m, int l) {
    const float* at = b.anchors + ((long)(anchors + m / b.every) * p.H + h) * (DK * DV) +
                      wave * (DV * 16) + 4 * l;
#pragma unroll
    for (int t = 0; t < VT; ++t) S[t] = *reinterpret_cast<const f32x4*>(at + t * 256);
  };
  float gnext = 0.f;
  if (chunks > 0) {
    fetch(chunks - 1, threadIdx.x);
    fetch_state(chunks - 1, l);
    const float g = decay_of(chunks - 1);
    gnext = decay_of(chunks - 2);
    if (wave == NW - 1) dec[(chunks - 1) & 1].make(g);
    // scores above the diagonal's tiles stay zero
    Ps.clear(threadIdx.x, NTH);
    Ms.clear(threadIdx.x, NTH);
  }
  loads_done();
  double sums = 0.0;  // of dg at the lane's place in its chunk (head_decay, wave 0)
  double pass = 0.0;  // <dS, S> at the chunk's end (wave 0)
  // What the carried value turns out to be off by at the next anchor had grown over the tokens since the
  // last: half of it for each of them (head_decay, wave 0)
  double off = 0.0;
  int since = 0;
  // what bf16 leaves of this wave's rows of dS, into a tile's rows
  auto rest = [&](E* m, int row, int l) {
#pragma unroll
    for (int t = 0; t < VT; ++t)
      put4<E, DV>(m, row, tile_row(t, l),
                  dS[t] - __builtin_convertvector(__builtin_convertvector(dS[t], bf16x4), f32x4));
  };

  for (int m = chunks - 1; m >= 0; --m) {
    const int len = min(C, c.len - m * C);
    const Decays<C>& d = dec[m & 1];
    int lo = l, tid = threadIdx.x;
    opaque(lo);
    opaque(tid);
    const int lc = lo & 15, lg = lo >> 4;
    const bool anchor = (m + 1) % b.every == 0 || m == chunks - 1;
    if (anchor) {
      double x = 0.0;
#pragma unroll
      for (int t = 0; t < VT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x = fma((double)S[t][e], (double)dS[t][e], x);
      x = group_sum(row_sum(x));
      if (lo == 0) cs[(m & 1) * NW + wave] = x;
    }
    q.store(Qs, tid);
    k.store(Ks, tid);
    v.store(Vs, tid);
    o.store(Os, tid);
#pragma unroll
    for (int t = 0; t < VT; ++t) put4<E, DV>(Ds, 16 * wave + lc, tile_row(t, lo), dS[t]);
    if constexpr (TWO && DK > C) {
      if (wave >= C / 16) rest(Dl, 16 * wave - C + lc, lo);
    }
    __syncthreads();
    // a of this chunk, for its last step
    const __amdgpu_buffer_rsrc_t ars = __builtin_amdgcn_make_buffer_rsrc(
        b.a + (c.t0 + (long)m * C) * p.H + h, 0, ((len - 1) * p.H + 1) * 8, 0x00020000);
    const double a = __builtin_bit_cast(double, __builtin_amdgcn_raw_buffer_load_b64(
        ars, lo < len ? (uint32_t)(lo * p.H * 8) : kNoColumn, 0, 0));
    fetch(m - 1, tid);
    if (m > 0 && m % b.every == 0) fetch_state(m - 1, lo);

    lower_tiles<TT, NW, true>(wave, [&](auto count, int first) {
      constexpr int N = decltype(count)::value;
      int ti[N], tj[N];
      f32x4 qk[N], ov[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int x = first + n * NW;
        ti[n] = tile_i(x);
        tj[n] = x - ti[n] * (ti[n] + 1) / 2;
        qk[n] = ov[n] = zero4();
      }
#pragma unroll
      for (int s = 0; s < DK / KF; ++s)
#pragma unroll
        for (int n = 0; n < N; ++n)
          qk[n] = Mx<E>::mma(TK::ld(Ks, 16 * tj[n], KF * s, lo), TK::ld(Qs, 16 * ti[n], KF * s, lo),
                             qk[n]);
#pragma unroll
      for (int s = 0; s < DV / KF; ++s)
#pragma unroll
        for (int n = 0; n < N; ++n)
          ov[n] = Mx<E>::mma(TV::ld(Vs, 16 * tj[n], KF * s, lo), TV::ld(Os, 16 * ti[n], KF * s, lo),
                             ov[n]);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int i = 16 * ti[n] + lc, j = 16 * tj[n] + 4 * lg;
        const f32x4 w = decays(d, i, j) * p.scale;
        f32x4 pp, mm, ee;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pp[e] = j + e <= i ? qk[n][e] * w[e] : 0.f;
          mm[e] = j + e <= i ? ov[n][e] * w[e] : 0.f;
          ee[e] = j + e < i ? mm[e] * qk[n][e] : 0.f;
        }
        Ps.put(i, j, pp);
        Ms.put(i, j, mm);
        double r = ((double)ee[0] + ee[1]) + ((double)ee[2] + ee[3]);
        r = group_sum(r);
        if (lg == 0) rows[tj[n]][i] = r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double s = row_sum((double)ee[e]);
          if (lc == 0) cols[ti[n]][j + e] = s;
        }
      }
    });
    const float g = gnext;
    gnext = decay_of(m - 2);
    if (wave == NW - 1) dec[(m - 1) & 1].make(g);
    // dK from dS and V.  Here and below the next step's operands are read before a step's products, and
    // kept from sinking to their use, where each would be waited for.
    f32x4 acc[TT];
    frag y[2][TT];
    auto v_rows = [&](int s) {
#pragma unroll
      for (int t = 0; t < TT; ++t) y[s & 1][t] = TV::ld_state(Vs, 16 * t, s, lo);
    };
    v_rows(0);
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = zero4();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s + 1 < STEPS) v_rows(s + 1);
      sched_fence();
      frag f[TERMS];
      float x[8];
#pragma unroll
      for (int e = 0; e < EPL; ++e) x[e] = sizeof(E) == 2 ? dS[2 * s + e / 4][e % 4] : dS[s][e % 4];
      split<E>(x, f);
#pragma unroll
      for (int e = TERMS - 1; e >= 0; --e)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = Mx<E>::mma(f[e], y[s & 1][t], acc[t]);
    }
    sched_fence();
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      acc[t] *= d.left[16 * t + lc];
      const double r = group_sum((double)dot4<E, DK>(Ks, 16 * t + lc, 16 * wave + 4 * lg, acc[t]));
      if (lg == 0) bs[wave][16 * t + lc] = r;
    }
    __syncthreads();

    if constexpr (TWO) {
      if (wave < C / 16) rest(Vs, 16 * wave + lc, lo);
    }
    const float keep = d.into[C - 1];
    frag own[KS];  // Q transposed: this wave's 16 columns
#pragma unroll
    for (int s = 0; s < KS; ++s) own[s] = TK::tr(Qs, KF * s, 16 * wave, lo);
    frag z[2][KS][Ms.TERMS];  // rows 16 t .. of M or P transposed
    auto columns = [&](const Scores<E, C>& m, int t) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < Ms.TERMS; ++e)
          if (KF * (s + 1) > 16 * t) z[t & 1][s][e] = TP::tr(m.m[e], KF * s, 16 * t, lo);
    };
    auto product = [&](const frag (&x)[KS], int t) {
#pragma unroll
      for (int e = Ms.TERMS - 1; e >= 0; --e)
#pragma unroll
        for (int s = 0; s < KS; ++s)
          if (KF * (s + 1) > 16 * t) acc[t] = Mx<E>::mma(x[s], z[t & 1][s][e], acc[t]);
    };
    {
      const __amdgpu_buffer_rsrc_t rs = rows_of(gp + (long)m * C * sg, sg, p.Dk, len);
      const int col = 16 * wave + 4 * lg;
      columns(Ms, 0);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t + 1 < TT) columns(Ms, t + 1);
        sched_fence();
        product(own, t);
        store4<G>(rs, col < p.Dk ? (row_at(16 * t + lc, sg) + col) * (int)sizeof(G) : kNoColumn,
                  acc[t]);
      }
    }
    // dV
    if constexpr (TWO) __syncthreads();
    const __amdgpu_buffer_rsrc_t rs = rows_of(dvp + (long)m * C * so, so, p.Dv, len);
#pragma unroll
    for (int w = 0; w < (VT + NW - 1) / NW; ++w) {
      const int vt = wave + w * NW;
      if (VT % NW != 0 && vt >= VT) break;
      frag sf[2][1 + TWO];
      auto k_rows = [&](int s) {
        sf[s & 1][0] = TV::tr(Ds, KF * s, 16 * vt, lo);
        if constexpr (TWO)
          sf[s & 1][TWO] = KF * s < C ? TV::tr(Vs, KF * s, 16 * vt, lo)
                                      : TV::tr(Dl, KF * s - C, 16 * vt, lo);
#pragma unroll
        for (int t = 0; t < TT; ++t) y[s & 1][t] = TK::ld(Ks, 16 * t, KF * s, lo);
      };
      k_rows(0);
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = zero4();
#pragma unroll
      for (int s = 0; s < DK / KF; ++s) {
        if (s + 1 < DK / KF) k_rows(s + 1);
        sched_fence();
#pragma unroll
        for (int e = TWO; e >= 0; --e)
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[t] = Mx<E>::mma(sf[s & 1][e], y[s & 1][t], acc[t]);
      }
      frag of[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) of[s] = TV::tr(Os, KF * s, 16 * vt, lo);
      columns(Ps, 0);
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] *= d.left[16 * t + lc];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (t + 1 < TT) columns(Ps, t + 1);
        sched_fence();
        product(of, t);
        const int col = 16 * vt + 4 * lg;
        store4<E>(rs, col < p.Dv ? (row_at(16 * t + lc, so) + col) * (int)sizeof(E) : kNoColumn,
                  acc[t]);
      }
    }
    // dS for the chunk before, four tiles at a time
    constexpr int GROUP = 4, GROUPS = KS * VT / GROUP;
    frag r[2][GROUP];
    auto o_rows = [&](int n) {
#pragma unroll
      for (int t = 0; t < GROUP; ++t)
        r[n & 1][t] = TV::tr_state(Os, KF * (n * GROUP / VT), n * GROUP % VT + t, lo);
    };
    o_rows(0);
#pragma unroll
    for (int t = 0; t < VT; ++t) dS[t] *= keep;
    frag f[TERMS];
#pragma unroll
    for (int n = 0; n < GROUPS; ++n) {
      const int s = n * GROUP / VT, first = n * GROUP % VT;
      if (n + 1 < GROUPS) o_rows(n + 1);
      sched_fence();
      if (first == 0) {
        float w[8];
#pragma unroll
        for (int e = 0; e < EPL; ++e)
          w[e] = (float)own[s][e] * (p.scale * d.into[KF * s + EPL * lg + e]);
        split<E>(w, f);
      }
#pragma unroll
      for (int e = TERMS - 1; e >= 0; --e)
#pragma unroll
        for (int t = 0; t < GROUP; ++t) dS[first + t] = Mx<E>::mma(r[n & 1][t], f[e], dS[first + t]);
    }
    __syncthreads();
    // the others go on to the next chunk, whose first barrier comes before its first write of any of these (but cs's other half)
    if (wave == 0) {
      double up = a, down = 0.0, in = 0.0;
      const int t = min(lo, C - 1);
      for (int x = 0; x < TT; ++x) {
        if (x <= t / 16) in += rows[x][t];
        if (x >= t / 16) in -= cols[x][t];
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) down += bs[w][t];
      if (anchor) {
        double x = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) x += cs[(m & 1) * NW + w];
        off += (x - pass) * since;
        pass = x;
        since = 0;
      }
      // nothing passes a decay that is 0 in fp32, nor of what the carried value is off by (a head's own
      // decay: every token's)
      if (!(d.G[0] < -150.0)) since += len;
      up = lo < len ? up : 0.0;
      down = lo < len ? down : 0.0;
      in = lo < len ? in : 0.0;
      const double suffix = wave_incl_scan(up + in), prefix = wave_incl_scan(down);
      const double all = last_lane(prefix);
      double x = (last_lane(suffix) - suffix + up + in) + (prefix - down) + (pass - all);
      pass += last_lane(wave_incl_scan(up)) - all;
      if (d.G[t] - (t > 0 ? d.G[t - 1] : 0.0) < -150.0) x = 0.0;
      if (lo < len) {
        if (p.head_decay)
          sums += x;
        else if (b.dg)
          b.dg[(c.t0 + (long)m * C + lo) * p.H + h] = (float)x;
      }
    }
  }

  if (p.head_decay) {
    // the start's <dS, S> too
    const float* at = c.i > 0 ? p.states + (long)unit * cell
                      : p.h0  ? p.h0 + ((long)c.n * p.H + h) * cell
                              : nullptr;
    const __amdgpu_buffer_rsrc_t srs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(at), 0, at ? (int)cell * 4 : 0, 0x00020000);
    double x = 0.0;
#pragma unroll
    for (int t = 0; t < VT; ++t) {
      const f32x4 s0 = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
          srs, tile_row(t, l) < p.Dv
                   ? (uint32_t)((16 * wave + (l & 15)) * p.Dv + tile_row(t, l)) * 4 : kNoColumn, 0,
          0));
#pragma unroll
      for (int e = 0; e < 4; ++e) x = fma((double)s0[e], (double)dS[t][e], x);
    }
    x = group_sum(row_sum(x));
    if (l == 0) cs[NW + wave] = x;  // chunk 0 may be an anchor and has the other half
    __syncthreads();
    if (wave == 0) {
      x = 0.0;
#pragma unroll
      for (int w = 0; w < NW; ++w) x += cs[NW + w];
      if (since > 0) off += (x - pass) * since;
      x = wave_incl_scan(l < C ? sums : 0.0) + 0.5 * off;
      if (l == 63) b.dgp[unit] = x;
    }
  }
  if (b.dh0 && c.i == 0) {
    const __amdgpu_buffer_rsrc_t trs = __builtin_amdgcn_make_buffer_rsrc(
        b.dh0 + ((long)c.n * p.H + h) * cell, 0, (int)cell * 4, 0x00020000);
    int lo = l;
    opaque(lo);  // addresses are made here, not kept from the loads
#pragma unroll
    for (int t = 0; t < VT; ++t)
      __builtin_amdgcn_raw_buffer_store_b128(
          __builtin_bit_cast(u32x4, dS[t]), trs,
          tile_row(t, lo) < p.Dv ? (uint32_t)((16 * wave + (lo & 15)) * p.Dv + tile_row(t, lo)) * 4
                                 : kNoColumn, 0, 0);
  }
}

// What is left after the passes, each grid row a part: dq (0) and dk (1) of a q/k head, the sum of its
// value heads' shares in order, four values a thread; dg of a head (2), the sum over its segments.
template <typename E>
__global__ __launch_bounds__(kColumnThreads) void k_linear_sums(LinearProblem p, LinearBwd b, int first) {
  const int part = first + blockIdx.y;
  if (part == 2) {
    __shared__ double sums[kColumnThreads / 64][64];
    if ((int)blockIdx.x >= (p.H + 63) / 64) return;
    const int c = blockIdx.x * 64 + lane_id();
    double s = 0.0;
    if (c < p.H)
      for (int r = wave_id(); r < p.slots; r += kColumnThreads / 64) s += b.dgp[(long)r * p.H + c];
    sums[wave_id()][lane_id()] = s;
    __syncthreads();
    if (threadIdx.x >= 64 || c >= p.H) return;
    for (int w = 1; w < kColumnThreads / 64; ++w) s += sums[w][lane_id()];
    b.dg[c] = (float)s;
    return;
  }
  const long vecs = (long)p.Hg * p.Dk / 4, total = p.cu ? min(max(p.cu[p.N], 0), p.Ttot) : p.Ttot;
  const long at = (long)blockIdx.x * kColumnThreads + threadIdx.x;
  if (at >= total * vecs) return;
  const long t = at / vecs;
  const int x = (int)(at - t * vecs) * 4, hk = x / p.Dk, col = x - hk * p.Dk, rep = p.H / p.Hg;
  const float* from = b.part + (part ? (long)p.Ttot * p.H * p.Dk : 0) +
                      (t * p.H + (long)hk * rep) * p.Dk + col;
  f32x4 s = zero4();
  for (int r = 0; r < rep; ++r) s += *reinterpret_cast<const f32x4*>(from + (long)r * p.Dk);
  E* to = static_cast<E*>(part ? b.dk : b.dq) + at * 4;
  if constexpr (sizeof(E) == 2)
    *reinterpret_cast<bf16x4*>(to) = __builtin_convertvector(s, bf16x4);
  else
    *reinterpret_cast<f32x4*>(to) = s;
}

template <typename E, int DK, int DV>
hipError_t launch_grads(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  const int blocks = p.slots * p.H;
  LinearProblem q = p;
  q.group = group_of(p, 1, blocks);
  if (p.H != p.Hg)
    k_linear_bwd<E, DK, DV, true><<<blocks, DK * 4, 0, st>>>(q, b);
  else
    k_linear_bwd<E, DK, DV, false><<<blocks, DK * 4, 0, st>>>(q, b);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_grads_e(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  if (p.Dv <= 64)
    return p.Dk <= 64 ? launch_grads<E, 64, 64>(p, b, st) : launch_grads<E, 128, 64>(p, b, st);
  return p.Dk <= 64 ? launch_grads<E, 64, 128>(p, b, st) : launch_grads<E, 128, 128>(p, b, st);
}

template <typename E>
hipError_t launch_sums(const LinearProblem& p, const LinearBwd& b, bool shares, bool heads,
                       hipStream_t st) {
  const long vecs = shares ? (long)p.Ttot * p.Hg * p.Dk / 4 : 0, cols = heads ? (p.H + 63) / 64 : 0;
  const long blocks = (vecs + kColumnThreads - 1) / kColumnThreads;
  k_linear_sums<E><<<dim3((unsigned)(blocks > cols ? blocks : cols), 2 * shares + heads),
                     kColumnThreads, 0, st>>>(p, b, shares ? 0 : 2);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_bwd(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (p.slots > 0) {
    if (p.Lc != kScanNoSplit) e = launch_linear_states(p, &b, st);
    if (e == hipSuccess && p.Ttot > 0) e = launch_linear_dq(p, b, st);
    if (e == hipSuccess)
      e = p.f32 ? launch_grads_e<float>(p, b, st) : launch_grads_e<bf16>(p, b, st);
    if (e != hipSuccess) return e;
  }
  // without a sequence there is no gradient to write but the heads' zeros
  const bool shares = p.H != p.Hg && p.Ttot > 0 && p.slots > 0, heads = b.dg && p.head_decay;
  if (shares || heads)
    e = p.f32 ? launch_sums<float>(p, b, shares, heads, st)
              : launch_sums<bf16>(p, b, shares, heads, st);
  return e;
}

}  // namespace gdn
