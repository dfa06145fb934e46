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
//     of steps, the chunks' start states are composed in order (the decay of a chunk is
//     exp(A * sum of steps)), and the output pass starts from them.
//
// Measured with 4096 channels, 16 states, bf16, gated (bytes alone at a copy's 5.1 TB/s in
// brackets): 8 x 2048 tokens 268 us (71), the vector units busy in 90 % of the cycles (127 M vector
// instructions, 80 of 121 a token and channel in the recurrence itself); 12454 packed tokens in
// eight sequences 246 us (80); one sequence of 8192 tokens, in 8 chunks, 246 us (52).
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
  int nb;  // channel blocks in all (G nblk)
  int softplus, split;
};

// Chunks' start states: none (whole sequences), composed by k_scan_combine, or by each workgroup of
// the output pass from the chunks before its own.  The last saves a launch and is quicker with 2
// states a lane for up to 8 chunks a sequence (12454 packed tokens in eight sequences 254 to 246 us,
// 300 tokens of 4096 channels 26.9 to 24.2 us); 13 chunks of 1000 channels take 20.6 us so and 19.0
// composed, and 64 states in 16 chunks 85 and 72 us.  It reads h0 in every chunk's workgroup while the
// last chunk's writes ht, so a call with one buffer for both is composed instead (the same bits).
constexpr int kComposed = 1, kOwn = 2;
constexpr int kOwnChunks = 8;

// B and C of every token and group as padded fp32 rows [G][Sp / ns][Ttot][2][ns], so that the
// scan reads them through the scalar cache whatever their type, alignment, strides and number: a
// wave's ns states of consecutive tokens are one contiguous piece.
template <typename E>
__global__ __launch_bounds__(256) void k_scan_pack(const E* Bm, const E* Cm, long sb, long sc,
                                                   float* bc, int Ttot, int G, int S, int Sp,
                                                   int ns) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  const int row = 2 * Sp;  // a thread reads row element k of token t, group g
  if (i >= (long)Ttot * G * row) return;
  const int k = (int)(i % row);
  const long tg = i / row;
  const int g = (int)(tg % G);
  const long t = tg / G;
  const int s = k < Sp ? k : k - Sp;
  float v = 0.f;
  if (s < S) v = (float)(k < Sp ? Bm[t * sb + (long)g * S + s] : Cm[t * sc + (long)g * S + s]);
  const long block = (long)g * (Sp / ns) + s / ns;
  bc[((block * Ttot + t) * 2 + (k >= Sp)) * ns + s % ns] = v;
}

// What the 16 / NS tokens of a step need: their B and C rows (32 values, two 64-byte scalar loads)
// and their (step, step x) from LDS.
template <int NS>
struct Step {
  static constexpr int TOKENS = 16 / NS;
  float bc[32];
  float2 v[TOKENS];
  __device__ __forceinline__ void load(const float* rows, const float2 (*sd)[kScanLanes],
                                       int lane) {
    const scalar_row r = as_scalar(rows);
#pragma unroll
    for (int i = 0; i < 32; ++i) bc[i] = r[i];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) v[i] = sd[i][lane];
  }
};

// What a lane works on: its channel (clamped, so that every lane has one) and whether it is the
// lane that owns it.
struct Lane {
  int g, c;
  bool live;
};
__device__ __forceinline__ Lane lane_channel(int block, int per, int nblk) {
  Lane l;
  l.g = block / nblk;
  const int cl = (block - l.g * nblk) * kScanLanes + lane_id();
  l.live = cl < per;
  l.c = l.g * per + min(cl, per - 1);
  return l;
}

// One chunk's outputs from its start state (OUT; the last chunk writes the final state), or its
// own end state from a zero start and its sum of steps (a sequence's last chunk has no successor
// and is skipped).
//
// A tile goes through three stages: its owners load x, dt, z and put (step, step x) into LDS; all
// waves take its tokens through their states and put their share of sum_s C h into LDS; its owners
// add the shares up and store y.  Between two barriers a wave does the first stage of the next
// tile, the second of this one and the third of the last, all independent, so there is one
// barrier a tile; loads are issued a tile before they are needed.
template <int NS, int NW, bool OUT, bool GATED, typename E>
__global__ __launch_bounds__(64 * NW) void k_scan(ScanArgs a) {
  constexpr int TPW = TT / NW;  // tokens of a tile that a wave prepares and finishes
  __shared__ float2 sd[2][TT][kScanLanes];
  __shared__ float yp[OUT ? 2 : 1][OUT ? NW : 1][OUT ? TT : 1][kScanLanes];
  const int slot = blockIdx.x / a.nb;
  const Chunk ch = chunk_of(a.map, slot);
  if (!ch.ok || (!OUT && ch.i == ch.count - 1)) return;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const Lane l = lane_channel(blockIdx.x - slot * a.nb, a.per, a.nblk);
  Column<E> x, dt, z, y;
  x.open(a.x, ch.t0, a.sx, ch.len, a.C, l.c, true);
  dt.open(a.dt, ch.t0, a.sdt, ch.len, a.C, l.c, true);
  if (GATED) z.open(a.z, ch.t0, a.sz, ch.len, a.C, l.c, true);
  if (OUT) y.open(a.y, ch.t0, a.C, ch.len, a.C, l.c, l.live);
  const float bias = a.bias ? a.bias[l.c] : 0.f;
  const float Dc = a.D ? a.D[l.c] : 0.f;
  const uint32_t mask = a.softplus ? 0xFFFFFFFFu : 0u;
  const int s0 = w * NS;
  const float* rows = a.bc + (((long)l.g * NW + w) * a.map.Ttot + ch.t0) * 2 * NS;
  const int tiles = (ch.len + TT - 1) / TT;

  uint32_t rx[TPW], rd[TPW], rz[TPW];
  auto fetch = [&](int tile) {  // past the chunk: its last token
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int r = min(tile * TT + w * TPW + i, ch.len - 1);
      rx[i] = x.load(r);
      rd[i] = dt.load(r);
      if (GATED) rz[i] = z.load(r);
    }
  };
  if (tiles > 0) fetch(0);

  float A2[NS], h[NS], sum = 0.f;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int s = s0 + k;
    A2[k] = s < a.S ? a.A[(long)l.c * a.S + s] * kLog2e : 0.f;
    h[k] = 0.f;
    if (OUT && s < a.S) {
      if (a.split == kComposed)
        h[k] = a.hst[((long)slot * a.S + s) * a.C + l.c];
      else if (a.h0)
        h[k] = a.h0[((long)ch.n * a.C + l.c) * a.S + s];
    }
  }
  if (OUT && NS == 2 && a.split == kOwn) {  // over the chunks before this one
    const float* ds = a.dsum + (long)(slot - ch.i) * a.C + l.c;
    const float* hst = a.hst + ((long)(slot - ch.i) * a.S + s0) * a.C + l.c;
#pragma unroll 4
    for (int j = 0; j < ch.i; ++j) {
      const float d = ds[(long)j * a.C];
#pragma unroll
      for (int k = 0; k < NS; ++k)
        if (s0 + k < a.S)
          h[k] = fmaf(__builtin_amdgcn_exp2f(d * A2[k]), h[k],
                      hst[((long)j * a.S + k) * a.C]);
    }
  }

  // of the newest prepared tile and of the one before
  float xv[TPW] = {}, zv[TPW] = {}, xl[TPW] = {}, zl[TPW] = {};
  auto prepare = [&](int tile) {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      xv[i] = Column<E>::wide(rx[i]);
      if (GATED) zv[i] = Column<E>::wide(rz[i]);
      const float v = step_f32(Column<E>::wide(rd[i]) + bias, mask);
      sd[tile & 1][w * TPW + i][lane] = make_float2(v, v * xv[i]);
    }
    fetch(tile + 1);
  };
  auto token = [&](int p, int t, const float2& v, const float* b, const float* c) {
    float s = 0.f;
    if (!OUT) sum += v.x;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      h[k] = fmaf(__builtin_amdgcn_exp2f(v.x * A2[k]), h[k], v.y * b[k]);
      if (OUT) s = k ? fmaf(c[k], h[k], s) : c[k] * h[k];
    }
    if (OUT) yp[p][w][t][lane] = s;
  };
  float share[TPW][NW];  // of y, of this wave's tokens, from every wave
  auto gather = [&](int p) {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
#pragma unroll
      for (int k = 0; k < NW; ++k) share[i][k] = yp[p][k][w * TPW + i][lane];
    }
  };
  auto finish = [&](int tile, const float* xs, const float* zs) {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int t = w * TPW + i;
      float s = Dc * xs[i];
#pragma unroll
      for (int k = 0; k < NW; ++k) s += share[i][k];
      if (GATED) s *= zs[i] * sigmoid_f32(zs[i]);
      if (tile >= 0 && tile * TT + t < ch.len) y.store(tile * TT + t, s);
    }
  };

  // Scalar loads and LDS reads share one counter, and scalar loads return in no order: waiting for
  // one read is waiting for all of them.  So a step's reads of both kinds are issued together, a
  // step ahead (the first step's and the shares' right after the barrier, ahead of the next tile's
  // preparation), and waited for once.
  //
  // Waves in different stages take turns better with priorities than by age, which lets the older
  // workgroup of a CU run away from the younger: the next tile's preparation goes first and a wave's
  // claim falls as its tile is done (8 x 2048 tokens of 4096 channels 324 to 268 us).
  const int full = ch.len / TT;
  if (tiles > 0) prepare(0);
  for (int tile = 0; tile < full; ++tile) {
    const int p = tile & 1;
    const float* row = rows + (long)tile * TT * 2 * NS;
    constexpr int N = Step<NS>::TOKENS;
    Step<NS> buf[2];
    __syncthreads();
    buf[0].load(row, sd[p], lane);
    if (OUT) gather(p ^ 1);  // of no tile, and not used, before the first one
    __builtin_amdgcn_sched_barrier(0);
    float px[TPW], pz[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      px[i] = xl[i];
      xl[i] = xv[i];
      if (GATED) {
        pz[i] = zl[i];
        zl[i] = zv[i];
      }
    }
    __builtin_amdgcn_s_setprio(3);
    prepare(tile + 1);  // past the last tile: never used
    if (OUT) finish(tile - 1, px, pz);
#pragma unroll
    for (int step = 0; step < TT / N; ++step) {
      if (step + 1 < TT / N)
        buf[(step + 1) & 1].load(row + (step + 1) * 32, sd[p] + (step + 1) * N, lane);
      __builtin_amdgcn_sched_barrier(0);
      if (2 * step < TT / N) __builtin_amdgcn_s_setprio(2); else __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const Step<NS>& q = buf[step & 1];
        token(p, step * N + i, q.v[i], q.bc + i * 2 * NS, q.bc + i * 2 * NS + NS);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  }
  if (full < tiles) {  // the chunk's last tokens
    const int p = full & 1;
    __syncthreads();
    if (OUT) {
      gather(p ^ 1);
      finish(full - 1, xl, zl);
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        xl[i] = xv[i];
        if (GATED) zl[i] = zv[i];
      }
    }
    for (int t = 0; t < ch.len - full * TT; ++t) {
      float b[2 * NS];
      const scalar_row r = as_scalar(rows + (long)(full * TT + t) * 2 * NS);
#pragma unroll
      for (int i = 0; i < 2 * NS; ++i) b[i] = r[i];
      token(p, t, sd[p][t][lane], b, b + NS);
    }
  }
  if (OUT && tiles > 0) {
    __syncthreads();
    gather((tiles - 1) & 1);
    finish(tiles - 1, xl, zl);
  }
  if (!l.live || (OUT && (!a.ht || ch.i != ch.count - 1))) return;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int s = s0 + k;
    if (s < a.S) {
      if (OUT)
        a.ht[((long)ch.n * a.C + l.c) * a.S + s] = h[k];
      else
        a.hst[((long)slot * a.S + s) * a.C + l.c] = h[k];
    }
  }
  if (!OUT && w == 0) a.dsum[(long)slot * a.C + l.c] = sum;
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
  // workgroups in a row (and so on XCDs in turn) are a chunk's channel blocks: chunks of unlike
  // lengths then load the XCDs alike
  const unsigned grid = (unsigned)p.slots * a.nb;
  if (a.split) {
    k_scan<NS, NW, false, false, E><<<grid, 64 * NW, 0, st>>>(a);
    if (a.split == kComposed)
      k_scan_combine<<<dim3(p.N * p.S, (p.C + 255) / 256), 256, 0, st>>>(a);
  }
  if (a.z)
    k_scan<NS, NW, true, true, E><<<grid, 64 * NW, 0, st>>>(a);
  else
    k_scan<NS, NW, true, false, E><<<grid, 64 * NW, 0, st>>>(a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_e(const ScanProblem& p, const ScanArgs& a, hipStream_t st) {
  switch (p.ns * 100 + p.nw) {
    case 202: return launch_cfg<2, 2, E>(p, a, st);
    case 204: return launch_cfg<2, 4, E>(p, a, st);
    case 208: return launch_cfg<2, 8, E>(p, a, st);
    case 408: return launch_cfg<4, 8, E>(p, a, st);
    case 808: return launch_cfg<8, 8, E>(p, a, st);
    case 816: return launch_cfg<8, 16, E>(p, a, st);
    default: return launch_cfg<16, 16, E>(p, a, st);
  }
}

}  // namespace

hipError_t launch_scan_pack(const ScanProblem& p, hipStream_t st) {
  const long n = (long)p.Ttot * p.G * 2 * p.Sp;
  if (n == 0) return hipSuccess;
  const unsigned grid = (unsigned)((n + 255) / 256);
  if (p.f32)
    k_scan_pack<float><<<grid, 256, 0, st>>>((const float*)p.Bm, (const float*)p.Cm, p.sb, p.sc,
                                             p.bc, p.Ttot, p.G, p.S, p.Sp, p.ns);
  else
    k_scan_pack<bf16><<<grid, 256, 0, st>>>((const bf16*)p.Bm, (const bf16*)p.Cm, p.sb, p.sc,
                                            p.bc, p.Ttot, p.G, p.S, p.Sp, p.ns);
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
  a.nb = p.G * p.nblk;
  a.Sp = p.Sp;
  a.softplus = p.softplus;
  const long chunks = ((p.cu ? p.Ttot : p.T) + p.Lc - 1L) / p.Lc;
  const bool in_place = p.h0 && p.h0 == p.ht;
  a.split = p.Lc == kScanNoSplit                              ? 0
            : p.ns == 2 && chunks <= kOwnChunks && !in_place ? kOwn
                                                              : kComposed;
  return p.f32 ? launch_e<float>(p, a, st) : launch_e<bf16>(p, a, st);
}

}  // namespace gdn
