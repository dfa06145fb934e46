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
// chunk's in registers meanwhile; the C x C scores are shared out over the waves and come back as two
// bf16 terms, and so does the state meet q (16 bits or more of each value; with one term, o of a carried
// state came out 1.25 times as far from the definition as fp32 sums rounded once, and 8 x 2048 tokens took
// 168 us where they take 182); the state itself and what is added to it are held to fp32's last bits (v
// times its decay enters as three bf16 terms).
//
// Few or long sequences are cut into segments: k_linear_state makes each segment's own end state
// (k and v alone), k_linear_compose turns those into start states in order, and k_linear_fwd runs
// the segments side by side.  A few segments make their start states themselves.
//
// Measured (bf16, heads of 128 x 128): 8 x 2048 tokens of 32 heads 167 to 182 us, whose loads
// and stores alone take 113 with this order of accesses (4.7 TB/s), the matrix units busy 27 % and the
// vector units 41 %; 16384 tokens of 32 heads 64 + 12 + 141 us.  Four waves of 32 columns instead of
// eight of 16 took 8 % longer; a single barrier a chunk, with two or three buffers of everything, no less; 64
// narrow heads (4 x 4096 tokens, 64 columns) are one wave a SIMD, 227 us.
#include "linear_device.h"

namespace gdn {

namespace {

// GRAD: the same pass over other tensors makes dq.  With S^T as the state, whose rows run over the value
// columns, dq_t = scale S_t dout_t is the recurrence with dout for q, v for k and k for v.  There the
// state meets dout as three bf16 terms, not two, because the sums q . dq that leave the chunk (a) are terms of
// dg, an fp32 result; and the state is written out at every r.every-th chunk's end, and the segment's, for the
// other half of the gradient.
template <typename E, int DK, int DV, int NW, int OCC, bool GRAD, typename G>
__global__ __launch_bounds__(NW * 64, OCC) void k_linear_fwd(LinearProblem p, LinearRun r) {
  constexpr int C = sizeof(E) == 2 ? kLinearChunk : kLinearChunkF32;
  constexpr int NTH = NW * 64, CW = DV / 16 / NW, KT = DK / 16, TT = C / 16;
  constexpr int KF = Mx<E>::KF, KS = C / KF, TERMS = Mx<E>::TERMS, EPL = Mx<E>::EPL;
  constexpr int STEPS = sizeof(E) == 2 ? KT / 2 : KT, STERMS = GRAD || TERMS < 2 ? TERMS : 2;
  // Products are taken a step at a time where waves are short of registers; four waves of a CU's 16 are
  // not, and have the more to gain from reads ahead (4 x 4096 tokens, 64 heads of 64 columns: 6 % less)
  auto fence = [] { if constexpr (NW * OCC >= 16) sched_fence(); };
  typedef typename Mx<E>::frag frag;
  typedef Tile<E, DK> TK;
  typedef Tile<E, DV> TV;
  typedef Tile<E, C> TP;
  __shared__ __align__(256) E Qs[C * TK::LD];
  __shared__ __align__(256) E Ks[C * TK::LD];
  __shared__ __align__(256) E Vs[C * TV::LD];
  __shared__ __align__(256) E Xs[GRAD ? C * TV::LD : 1];
  __shared__ Scores<E, C> Ps;
  __shared__ __align__(16) Decays<C> dec[2];
  __shared__ double as[GRAD ? NW : 1][GRAD ? C : 1];

  const int slabs = (r.Dv + DV - 1) / DV;
  const int unit = unit_of(blockIdx.x, gridDim.x, p.group);
  const int slab = unit % slabs, sh = unit / slabs, slot = sh / p.H, h = sh - slot * p.H;
  const Chunk c = uniform_chunk(p, slot);
  if (!c.ok) return;
  const int l = lane_id(), wave = uniform(wave_id());
  const int v0 = slab * DV, width = min(DV, r.Dv - v0);
  const int col0 = 16 * CW * wave;  // this wave's columns of the slab
  const long cell = (long)p.Dk * p.Dv;

  // The state in memory is [Dk, Dv]: this one's rows (GRAD: its columns) are the first axis.  Rows past
  // the head lie past the buffer, or are sent there.
  f32x4 S[CW][KT];
  // every way to a start state adds to what is there: one that loads into S itself took 3 % longer over a
  // packed batch of 12454 tokens
  auto state = [&](const float* from, float keep) {
    const __amdgpu_buffer_rsrc_t frs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(from), 0, from ? (int)cell * 4 : 0, 0x00020000);
#pragma unroll
    for (int w = 0; w < CW; ++w) {
      const int col = col0 + 16 * w + (l & 15);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        f32x4 x;
        if constexpr (GRAD) {
          x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
              frs, col < width && tile_row(t, l) < r.Dk
                       ? (uint32_t)(col * r.Dk + tile_row(t, l)) * 4 : kNoColumn, 0, 0));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                frs, col < width ? (uint32_t)((tile_row(t, l) + i) * r.Dv + v0 + col) * 4
                                 : kNoColumn, 0, 0));
        }
        S[w][t] = S[w][t] * keep + x;
      }
    }
  };
#pragma unroll
  for (int w = 0; w < CW; ++w)
#pragma unroll
    for (int t = 0; t < KT; ++t) S[w][t] = zero4();
  const bool made = p.Lc != kScanNoSplit && !p.join && (c.i > 0 || !p.direct);
  state(made   ? p.states + ((long)slot * p.H + h) * cell
        : p.h0 ? p.h0 + ((long)c.n * p.H + h) * cell
               : nullptr, 1.f);
  if constexpr (!GRAD) {
    if (p.join)
      for (int s = slot - c.i; s < slot; ++s) {
        const long at = (long)s * p.H + h;
        state(p.states + at * cell, exp2_f32(p.sums[at]));
      }
  }

  const E* qp = static_cast<const E*>(r.q) + c.t0 * r.sq + (long)(h / r.qrep) * r.Dk;
  const E* kp = static_cast<const E*>(r.k) + c.t0 * r.sk + (long)(h / r.qrep) * r.Dk;
  const E* vp = static_cast<const E*>(r.v) + c.t0 * r.sv + (long)(h / r.vrep) * r.Dv + v0;
  const E* xp = static_cast<const E*>(r.x) + c.t0 * r.sx + (long)(h / r.vrep) * r.Dv + v0;
  const int64_t so = (int64_t)p.H * r.Dv;
  G* op = static_cast<G*>(r.out) + c.t0 * so + (long)h * r.Dv + v0;

  Rows<E, DK, C, NTH> q, k;
  Rows<E, DV, C, NTH> v, x;
  const int chunks = (c.len + C - 1) / C, anchors = GRAD ? first_anchor(p, c, r.every, C) : 0;
  float gnext = 0.f;
  auto fetch = [&](int m, int tid) {
    const int len = max(0, min(C, c.len - m * C));  // none past the last chunk
    q.load(qp + (long)m * C * r.sq, r.sq, r.Dk, len, tid);
    k.load(kp + (long)m * C * r.sk, r.sk, r.Dk, len, tid);
    v.load(vp + (long)m * C * r.sv, r.sv, width, len, tid);
    if constexpr (GRAD) x.load(xp + (long)m * C * r.sx, r.sx, width, len, tid);
  };
  auto decay_of = [&](int m) {
    return load_decay(p, c.t0 + (long)m * C, max(0, min(C, c.len - m * C)), h);
  };
  if (chunks > 0) {
    fetch(0, threadIdx.x);
    const float g = decay_of(0);
    gnext = decay_of(1);
    if (wave == NW - 1) dec[0].make(g);
    // scores above the diagonal's tiles are never written, and read where a product's k covers two
    Ps.clear(threadIdx.x, NTH);
  }
  loads_done();

  for (int m = 0; m < chunks; ++m) {
    const int len = min(C, c.len - m * C);
    const Decays<C>& d = dec[m & 1];
    int lo = l, tid = threadIdx.x;
    opaque(lo);
    opaque(tid);
    const int lc = lo & 15, lg = lo >> 4;
    q.store(Qs, tid);
    k.store(Ks, tid);
    v.store(Vs, tid);
    if constexpr (GRAD) x.store(Xs, tid);
    __syncthreads();
    // loads and stores of a chunk are the same in every wave and chunk, so that a wait for a load does
    // not have to wait for later stores
    fetch(m + 1, tid);

    // scores: the lower tiles, rows j of tile tj against columns i of tile ti
    lower_tiles<TT, NW, !GRAD>(wave, [&](auto count, int first) {
      constexpr int N = decltype(count)::value;
      int ti[N], tj[N];
      f32x4 a[N];
      int lx = lo;
      if constexpr (GRAD) opaque(lx);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int x = first + n * NW;
        ti[n] = tile_i(x);
        tj[n] = x - ti[n] * (ti[n] + 1) / 2;
        a[n] = zero4();
      }
#pragma unroll
      for (int s = 0; s < DK / KF; ++s)
#pragma unroll
        for (int n = 0; n < N; ++n)
          a[n] = Mx<E>::mma(TK::ld(Ks, 16 * tj[n], KF * s, lx), TK::ld(Qs, 16 * ti[n], KF * s, lx),
                            a[n]);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int i = 16 * ti[n] + (lx & 15), j = 16 * tj[n] + 4 * (lx >> 4);
        const f32x4 w = decays(d, i, j);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[n][e] = j + e <= i ? a[n][e] * w[e] * p.scale : 0.f;
        Ps.put(i, j, a[n]);
      }
    });
    const float g = gnext;
    gnext = decay_of(m + 2);
    if (wave == NW - 1) dec[(m + 1) & 1].make(g);
    // the state's share, a step's operands at a time
    f32x4 acc[CW][TT];
#pragma unroll
    for (int w = 0; w < CW; ++w)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[w][t] = zero4();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      fence();
      frag f[CW][STERMS];
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        float y[8];
#pragma unroll
        for (int e = 0; e < EPL; ++e)
          y[e] = sizeof(E) == 2 ? S[w][2 * s + e / 4][e % 4] : S[w][s][e % 4];
        split<E, STERMS>(y, f[w]);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const frag b = TK::ld_state(Qs, 16 * t, s, lo);
#pragma unroll
        for (int e = STERMS - 1; e >= 0; --e)
#pragma unroll
          for (int w = 0; w < CW; ++w) acc[w][t] = Mx<E>::mma(f[w][e], b, acc[w][t]);
      }
    }
    fence();
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float in = p.scale * d.into[16 * t + lc];
      double sum = 0.0;
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        acc[w][t] *= in;
        if constexpr (GRAD) sum += dot4<E, DV>(Xs, 16 * t + lc, col0 + 16 * w + 4 * lg, acc[w][t]);
      }
      if constexpr (GRAD) {
        sum = group_sum(sum);
        if (lg == 0) as[wave][16 * t + lc] = sum;
      }
    }
    __syncthreads();

    if constexpr (GRAD) {  // a_t, from every wave's columns in order
      double sum = 0.0;
      const int t = lo & (C - 1);
#pragma unroll
      for (int w = 0; w < NW; ++w) sum += as[w][t];
      const __amdgpu_buffer_rsrc_t ars = __builtin_amdgcn_make_buffer_rsrc(
          r.a + (c.t0 + (long)m * C) * p.H + h, 0, ((len - 1) * p.H + 1) * 8, 0x00020000);
      __builtin_amdgcn_raw_buffer_store_b64(
          __builtin_bit_cast(u32x2, sum), ars,
          wave == 0 && lo < len ? (uint32_t)(t * p.H * 8) : kNoColumn, 0, 0);
    }
    frag vf[CW][KS];
#pragma unroll
    for (int w = 0; w < CW; ++w)
#pragma unroll
      for (int s = 0; s < KS; ++s) vf[w][s] = TV::tr(Vs, KF * s, col0 + 16 * w, lo);
    const __amdgpu_buffer_rsrc_t ors = rows_of(op + (long)m * C * so, so, width, len);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
        if (KF * s < 16 * (t + 1)) {
#pragma unroll
          for (int e = Ps.TERMS - 1; e >= 0; --e) {
            const frag b = TP::ld(Ps.m[e], 16 * t, KF * s, lo);
#pragma unroll
            for (int w = 0; w < CW; ++w) acc[w][t] = Mx<E>::mma(vf[w][s], b, acc[w][t]);
          }
        }
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const int col = col0 + 16 * w + 4 * lg;
        store4<G>(ors, col < width ? (row_at(16 * t + lc, so) + col) * (int)sizeof(G)
                                   : kNoColumn, acc[w][t]);
      }
    }

    fence();
    // the state: v times its decay as TERMS operands
    const float keep = d.into[C - 1];
#pragma unroll
    for (int w = 0; w < CW; ++w)
#pragma unroll
      for (int t = 0; t < KT; ++t) S[w][t] *= keep;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      fence();
      frag f[CW][TERMS];
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        float x[8];
#pragma unroll
        for (int e = 0; e < EPL; ++e) x[e] = (float)vf[w][s][e] * d.left[KF * s + EPL * lg + e];
        split<E>(x, f[w]);
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        if (t % 4 == 0) fence();
        const frag a = TK::tr_state(Ks, KF * s, t, lo);
#pragma unroll
        for (int e = TERMS - 1; e >= 0; --e)
#pragma unroll
          for (int w = 0; w < CW; ++w) S[w][t] = Mx<E>::mma(a, f[w][e], S[w][t]);
      }
    }
    if constexpr (GRAD) {
      if ((m + 1) % r.every == 0 || m + 1 == chunks) {
        float* to = r.anchors + ((long)(anchors + m / r.every) * p.H + h) * (DK * DV) + 4 * lo;
#pragma unroll
        for (int w = 0; w < CW; ++w)
#pragma unroll
          for (int t = 0; t < KT; ++t)
            *reinterpret_cast<f32x4*>(to + ((wave * CW + w) * KT + t) * 256) = S[w][t];
      }
    }
    __syncthreads();
  }

  if (!GRAD && p.ht && c.i == c.count - 1) {
    const __amdgpu_buffer_rsrc_t trs = __builtin_amdgcn_make_buffer_rsrc(
        p.ht + ((long)c.n * p.H + h) * cell, 0, (int)cell * 4, 0x00020000);
    int lo = l;
    opaque(lo);  // the addresses are made here, not kept from the loads
#pragma unroll
    for (int w = 0; w < CW; ++w) {
      const int col = col0 + 16 * w + (lo & 15);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_buffer_store_b32(
              __float_as_uint(S[w][t][i]), trs,
              col < width ? (uint32_t)((tile_row(t, lo) + i) * r.Dv + v0 + col) * 4 : kNoColumn, 0,
              0);
    }
  }
}

// Start states from the segments' own end states, in place: a thread has four values of a state and
// walks its sequence's segments, four loads ahead of the one it is at.  The grid's second row makes the
// gradients at the segments' ends from their own shares, last to first.  Where the passes after this
// one take the first segment's start (the last one's end) from the caller's buffer, it is not copied.
struct LinearEnds {
  const float* from;  // dht or null
  float* grads;
  bool direct;
};
__global__ __launch_bounds__(256) void k_linear_compose(LinearProblem p, LinearEnds b) {
  constexpr int AHEAD = 4;
  const long cell = (long)p.Dk * p.Dv;
  const int blocks = (int)((cell / 4 + 255) / 256);
  const int nh = blockIdx.x / blocks, n = nh / p.H, h = nh - n * p.H;
  const long at = ((long)(blockIdx.x - nh * blocks) * 256 + threadIdx.x) * 4;
  if (at >= cell) return;
  const bool back = blockIdx.y != 0, direct = back ? b.direct : p.direct;
  const ChunkMap m = {p.cu, p.T, p.Ttot, p.N, p.Lc};
  int bos, eos;
  chunk_seq(m, n, bos, eos);
  const int count = chunk_count(eos - bos, p.Lc);
  if (count == 1 && direct) return;
  const int first = p.cu ? chunk_first(m, n) : n * count;
  const float* from = back ? b.from : p.h0;
  float* states = back ? b.grads : p.states;
  f32x4 s = zero4();
  if (from) s = *reinterpret_cast<const f32x4*>(from + ((long)n * p.H + h) * cell + at);
  // the i-th segment on the way
  auto slot = [&](int i) { return ((long)first + (back ? count - 1 - i : i)) * p.H + h; };
  for (int i = 0; i < count; i += AHEAD) {
    f32x4 own[AHEAD];
    float keep[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (i + j + 1 < count) {
        own[j] = *reinterpret_cast<const f32x4*>(states + slot(i + j) * cell + at);
        keep[j] = p.sums[slot(i + j)];
      }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (i + j < count) {
        if (i + j > 0 || !direct) *reinterpret_cast<f32x4*>(states + slot(i + j) * cell + at) = s;
        if (i + j + 1 < count) s = s * exp2_f32(keep[j]) + own[j];
      }
  }
}

// Sums of outer products x_t y_t^T over a segment, without its outputs, and the segment's decay: the end
// state from zero (x = k, y = v, decays to the segment's end), or in REV the gradient at its start
// (x = q, y = dout, decays from there).  Wave w holds columns of x (rows of the state) as tiles over y.
// Both take the last chunk first, so that the passes after this one, which begin with the first, find
// those rows in the last-level cache; the end state then needs no scaling from chunk to chunk, as a
// chunk's rows bring the decay of all that follow.
template <typename E, int DK, int DV, int NW, bool REV>
__device__ __forceinline__ void linear_state(const LinearProblem& p, const LinearPass& a) {
  constexpr int C = sizeof(E) == 2 ? kLinearChunk : kLinearChunkF32;
  constexpr int NTH = 64 * NW, TK = DK / 16 / NW, VT = DV / 16;
  constexpr int KF = Mx<E>::KF, KS = C / KF, TERMS = Mx<E>::TERMS;
  typedef typename Mx<E>::frag frag;
  typedef Tile<E, DK> TX;
  typedef Tile<E, DV> TY;
  __shared__ __align__(256) E Xs[C * TX::LD];
  __shared__ __align__(256) E Ys[C * TY::LD];
  __shared__ __align__(16) Decays<C> dec[2];

  const int slabs = (p.Dv + DV - 1) / DV;
  const int unit = unit_of(blockIdx.x, gridDim.x, p.group);
  const int slab = unit % slabs, sh = unit / slabs, slot = sh / p.H, h = sh - slot * p.H;
  const Chunk c = uniform_chunk(p, slot);
  // nothing comes after the last segment (before the first)
  if (!c.ok || c.i == (REV ? 0 : c.count - 1)) return;
  const int l = lane_id(), wave = uniform(wave_id()), lc = l & 15, lg = l >> 4;
  const int hk = h / (p.H / p.Hg), v0 = slab * DV, width = min(DV, p.Dv - v0);
  const long cell = (long)p.Dk * p.Dv, at = ((long)slot * p.H + h) * cell;

  f32x4 S[TK][VT];
#pragma unroll
  for (int j = 0; j < TK; ++j)
#pragma unroll
    for (int t = 0; t < VT; ++t) S[j][t] = zero4();

  const E* xp = static_cast<const E*>(a.x) + c.t0 * a.sx + (long)hk * p.Dk;
  const E* yp = static_cast<const E*>(a.y) + c.t0 * a.sy + (long)h * p.Dv + v0;
  Rows<E, DK, C, NTH> x;
  Rows<E, DV, C, NTH> y;
  const int chunks = (c.len + C - 1) / C;
  auto chunk_at = [&](int m) { return chunks - 1 - m; };
  auto fetch = [&](int m, int tid) {  // nothing past the last chunk
    const int len = max(0, m < 0 ? 0 : min(C, c.len - m * C));
    x.load(xp + (long)m * C * a.sx, a.sx, p.Dk, len, tid);
    y.load(yp + (long)m * C * a.sy, a.sy, width, len, tid);
  };
  auto decay_of = [&](int m) {
    return load_decay(p, c.t0 + (long)m * C, max(0, m < 0 ? 0 : min(C, c.len - m * C)), h);
  };
  double sum = 0.0;
  float gnext = 0.f, after = 1.f;  // the decay of the chunks after this one
  if (chunks > 0) {
    fetch(chunk_at(0), threadIdx.x);
    const float g = decay_of(chunk_at(0));
    gnext = decay_of(chunk_at(1));
    if (wave == NW - 1) sum = dec[0].make(g);
  }
  loads_done();
  for (int m = 0; m < chunks; ++m) {
    const Decays<C>& d = dec[m & 1];
    int lo = l, tid = threadIdx.x;
    opaque(lo);
    opaque(tid);
    const int lc = lo & 15, lg = lo >> 4;
    x.store(Xs, tid);
    y.store(Ys, tid);
    __syncthreads();
    fetch(chunk_at(m + 1), tid);
    const float g = gnext;
    gnext = decay_of(chunk_at(m + 2));
    if (wave == NW - 1) sum += dec[(m + 1) & 1].make(g);
    const float keep = d.into[C - 1];
    if constexpr (REV) {
#pragma unroll
      for (int j = 0; j < TK; ++j)
#pragma unroll
        for (int t = 0; t < VT; ++t) S[j][t] *= keep;
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      frag f[TK][TERMS];
#pragma unroll
      for (int j = 0; j < TK; ++j) {
        const frag b = TX::tr(Xs, KF * s, 16 * (wave * TK + j), lo);
        float w[8];
#pragma unroll
        for (int e = 0; e < Mx<E>::EPL; ++e) {
          const int i = KF * s + Mx<E>::EPL * lg + e;
          w[e] = (float)b[e] * (REV ? p.scale * d.into[i] : after * d.left[i]);
        }
        split<E>(w, f[j]);
      }
#pragma unroll
      for (int t = 0; t < VT; ++t) {
        const frag r = TY::tr_state(Ys, KF * s, t, lo);
#pragma unroll
        for (int j = 0; j < TK; ++j)
#pragma unroll
          for (int e = TERMS - 1; e >= 0; --e) S[j][t] = Mx<E>::mma(r, f[j][e], S[j][t]);
      }
    }
    after *= keep;
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < TK; ++j)
#pragma unroll
    for (int t = 0; t < VT; ++t) {
      const int row = 16 * (wave * TK + j) + lc, y0 = tile_row(t, l);
      if (row < p.Dk && y0 < width)
        *reinterpret_cast<f32x4*>(a.own + at + (long)row * p.Dv + v0 + y0) = S[j][t];
    }
  // each segment's decay once: the way back leaves the last one's, which the way there leaves out
  if (slab == 0 && threadIdx.x == NTH - 1 && (!REV || c.i == c.count - 1))
    p.sums[(long)slot * p.H + h] = (float)sum;
}

// Both directions in one launch: the grid's second row goes back.
template <typename E, int DK, int DV, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_linear_state(LinearProblem p, LinearPass a,
                                                             LinearPass back) {
  if (blockIdx.y == 0)
    linear_state<E, DK, DV, NW, false>(p, a);
  else
    linear_state<E, DK, DV, NW, true>(p, back);
}

template <typename E, int DK, int DV, int NW, int OCC>
hipError_t launch_fwd(const LinearProblem& p, const LinearRun& r, hipStream_t st) {
  const int slabs = (r.Dv + DV - 1) / DV;
  const int blocks = p.slots * p.H * slabs;
  LinearProblem q = p;
  q.group = group_of(p, slabs, blocks);
  k_linear_fwd<E, DK, DV, NW, OCC, false, E><<<blocks, NW * 64, 0, st>>>(q, r);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_fwd_e(const LinearProblem& p, const LinearRun& r, hipStream_t st) {
  if (p.Dv <= 64) {
    if (p.Dk <= 64) return launch_fwd<E, 64, 64, 4, 2>(p, r, st);
    if (p.Dk <= 128) return launch_fwd<E, 128, 64, 4, 2>(p, r, st);
    return launch_fwd<E, 256, 64, 4, 1>(p, r, st);
  }
  if (p.Dk <= 64) return launch_fwd<E, 64, 128, 4, 2>(p, r, st);
  if (p.Dk <= 128) return launch_fwd<E, 128, 128, 8, 4>(p, r, st);
  return launch_fwd<E, 256, 128, 8, 2>(p, r, st);
}

template <typename E, int DK, int DV>
hipError_t launch_dq(const LinearProblem& p, const LinearRun& r, hipStream_t st) {
  const int blocks = p.slots * p.H;
  LinearProblem q = p;
  q.group = group_of(p, 1, blocks);
  // Four waves a SIMD where registers allow: two workgroups a CU in fp32 (75 KB of LDS each).  In bf16 (88 KB)
  // one fits whatever the registers, and a budget for two waves takes no less (534 us the gradient, and 536).
  constexpr int NW = DV / 16, OCC = DK == 128 && DV == 128 ? 4 : 2;
  if (p.H != p.Hg)
    k_linear_fwd<E, DK, DV, NW, OCC, true, float><<<blocks, NW * 64, 0, st>>>(q, r);
  else
    k_linear_fwd<E, DK, DV, NW, OCC, true, E><<<blocks, NW * 64, 0, st>>>(q, r);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_dq_e(const LinearProblem& p, const LinearRun& r, hipStream_t st) {
  if (r.Dv <= 64) return r.Dk <= 64 ? launch_dq<E, 64, 64>(p, r, st) : launch_dq<E, 128, 64>(p, r, st);
  return r.Dk <= 64 ? launch_dq<E, 64, 128>(p, r, st) : launch_dq<E, 128, 128>(p, r, st);
}

template <typename E, int DK, int DV>
hipError_t launch_state(const LinearProblem& p, const LinearPass& a, const LinearPass* back,
                        hipStream_t st) {
  const int slabs = (p.Dv + DV - 1) / DV;
  const int blocks = p.slots * p.H * slabs;
  LinearProblem q = p;
  q.group = group_of(p, slabs, blocks);
  constexpr int NW = DK <= 64 ? 4 : 8;
  k_linear_state<E, DK, DV, NW>
      <<<dim3(blocks, back ? 2 : 1), NW * 64, 0, st>>>(q, a, back ? *back : LinearPass{});
  return hipGetLastError();
}

template <typename E>
hipError_t launch_state_e(const LinearProblem& p, const LinearPass& a, const LinearPass* back,
                          hipStream_t st) {
  if (p.Dv <= 64) {
    if (p.Dk <= 64) return launch_state<E, 64, 64>(p, a, back, st);
    if (p.Dk <= 128) return launch_state<E, 128, 64>(p, a, back, st);
    return launch_state<E, 256, 64>(p, a, back, st);
  }
  if (p.Dk <= 64) return launch_state<E, 64, 128>(p, a, back, st);
  if (p.Dk <= 128) return launch_state<E, 128, 128>(p, a, back, st);
  return launch_state<E, 256, 128>(p, a, back, st);
}

}  // namespace

hipError_t launch_linear_states(const LinearProblem& p, const LinearBwd* b, hipStream_t st) {
  LinearPass a = {}, back = {};
  a.x = p.k;
  a.y = p.v;
  a.sx = p.sk;
  a.sy = p.sv;
  a.own = p.states;
  LinearEnds ends = {};
  if (b) {
    back.x = p.q;
    back.y = b->dout;
    back.sx = p.sq;
    back.sy = (int64_t)p.H * p.Dv;
    back.own = b->grads;
    ends.from = b->dht;
    ends.grads = b->grads;
    ends.direct = b->direct;
  }
  const hipError_t e = p.f32 ? launch_state_e<float>(p, a, b ? &back : nullptr, st)
                             : launch_state_e<bf16>(p, a, b ? &back : nullptr, st);
  if (e != hipSuccess || p.join) return e;
  const long blocks = ((long)p.Dk * p.Dv / 4 + 255) / 256 * p.N * p.H;
  k_linear_compose<<<dim3((unsigned)blocks, b ? 2 : 1), 256, 0, st>>>(p, ends);
  return hipGetLastError();
}

hipError_t launch_linear_fwd(const LinearProblem& p, hipStream_t st) {
  if (p.Lc != kScanNoSplit) {
    const hipError_t e = launch_linear_states(p, nullptr, st);
    if (e != hipSuccess) return e;
  }
  LinearRun r = {};
  r.q = p.q;
  r.k = p.k;
  r.v = p.v;
  r.sq = p.sq;
  r.sk = p.sk;
  r.sv = p.sv;
  r.Dk = p.Dk;
  r.Dv = p.Dv;
  r.qrep = p.H / p.Hg;
  r.vrep = 1;
  r.out = p.o;
  return p.f32 ? launch_fwd_e<float>(p, r, st) : launch_fwd_e<bf16>(p, r, st);
}

hipError_t launch_linear_dq(const LinearProblem& p, const LinearBwd& b, hipStream_t st) {
  LinearRun r = {};
  r.q = b.dout;
  r.k = p.v;
  r.v = p.k;
  r.x = p.q;
  r.sq = (int64_t)p.H * p.Dv;
  r.sk = p.sv;
  r.sv = p.sk;
  r.sx = p.sq;
  r.Dk = p.Dv;
  r.Dv = p.Dk;
  r.qrep = 1;
  r.vrep = p.H / p.Hg;
  r.out = p.H != p.Hg ? static_cast<void*>(b.part) : b.dq;
  r.a = b.a;
  r.anchors = b.anchors;
  r.every = b.every;
  return p.f32 ? launch_dq_e<float>(p, r, st) : launch_dq_e<bf16>(p, r, st);
}

}  // namespace gdn
