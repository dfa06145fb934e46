// The gradient of the selective scan.  With e_t = dy_t silu(z_t), a_t = exp(step_t A) and g_t the
// gradient of h_t,
//
//   g_t = e_t C_t + a_{t+1} g_{t+1}   (a g after the last token: dht),   q_t = g_t a_t h_{t-1}
//   dA      = sum_t step_t q_t                  dstep_t = sum_s (A q_t + x_t B_t g_t)
//   dx_t    = step_t sum_s B_t g_t + D e_t      dz_t    = dy_t (sum_s C_t h_t + D x_t) silu'(z_t)
//   dB_t[s] = sum_c step_t x_t g_t[c, s]        dC_t[s] = sum_c e_t h_t[c, s]
//
// The mapping is the forward's: a lane is a channel, B and C come through the scalar cache, the
// states of 64 channels are split over the waves of a workgroup.  Nothing of the forward is kept:
// every sequence is split into chunks of up to kBwdChunk tokens, and
//   * k_scan_bwd_state finds, for every chunk from zero boundaries, its end state and the gradient
//     a g that it hands to the chunk before it (both in one pass over its tokens: the gradient's
//     factors are the running products of a), and its sum of steps;
//   * k_scan_bwd_combine composes the chunks' start states forwards and their end gradients
//     backwards;
//   * k_scan_bwd goes over a chunk's tiles once to find the states at their starts, then over the
//     tiles from the last to the first: the tile's states and decays again, kept in registers,
//     then its tokens backwards;
//   * sums over channels (dB, dC) and over time (dA, dD, dt_bias) leave partial sums per channel
//     block and per chunk, which a small kernel adds in a fixed order (no atomics).
// The sums over the 64 lanes of a wave are the awkward part: dB and dC need one for each (token,
// state).  A transposing butterfly merges two registers into one at every step (lanes keep the
// half of the pair that their lane bit names), so 64 sums cost 63 merges, and end one to a lane.
//
// Measured on 8 x 2048 tokens of 4096 channels, 16 states, bf16, gated: 1.55 ms a call among others.
// Profiled, each kernel by itself, 1.59 ms: packing B and C 5 us, the chunks' states 336 us (the
// vector units busy throughout), their composition 59 us (the states' bytes), the gradients 1.15 ms
// (79 % busy: 202 registers leave two waves a SIMD; a cap at 168 for three spills), the partial sums
// 40 us.
#include <type_traits>

#include "ssm_device.h"

namespace gdn {

namespace {

constexpr int BT = 8;                  // tokens of a tile
constexpr int KT = kBwdChunk / BT;     // tiles of a chunk, at most
constexpr int NS = 4;                  // states a lane

struct BwdArgs {
  const void* x;
  const void* dt;
  const void* z;
  const void* dy;
  const float* bc;
  const float* A;
  const float* D;
  const float* bias;
  const float* h0;
  const float* dht;
  float* hst;   // [slots, S, C] end states, then start states
  float* gst;   // [slots, S, C] gradients handed back, then end gradients
  float* dsum;  // [slots, C]
  float* bcp;   // [nblk, Ttot, G, 2, Sp] partial dB, dC
  float* dAp;   // [slots, S, C] partial dA
  float* dvp;   // [slots, 2, C] partial dD, d(dt_bias)
  void* dx;
  void* ddt;
  void* dz;
  float* dh0;
  long sx, sdt, sz;
  ChunkMap map;
  int C, G, S, per, nblk, Sp;
  int nb;  // channel blocks in all (G nblk)
  int softplus, split;
};

struct Lane {
  int g, blk, c;
  bool live;
};
__device__ __forceinline__ Lane lane_channel(int block, int per, int nblk) {
  Lane l;
  l.g = block / nblk;
  l.blk = block - l.g * nblk;
  const int cl = l.blk * kScanLanes + lane_id();
  l.live = cl < per;
  l.c = l.g * per + min(cl, per - 1);
  return l;
}

// The transposing butterfly's merges: lanes that differ in one lane bit add up, and of the pair's
// two registers the lanes without the bit keep p0's sums, those with it p1's.
//
// Bits 3 and 2, four merges at a time: a 16-lane row's 4-lane banks are where the bits change, so a
// DPP addition of p0 for all lanes and one of p1 that writes only the banks with the bit make a
// merge in two instructions (a selection before an addition takes three).  Bit 2 adds the mirrored
// lane of its eight, which pairs the same halves.  A DPP operand must not have been written by the
// two instructions before: hence the s_nop.  The lane swaps of the merges after bit 2 have the same
// rule, and the compiler does not see what these instructions write: hence TAIL.
#define GDN_MERGE4(CTRL, BANKS, TAIL)                                                  \
  asm("s_nop 1\n\t"                                                                    \
      "v_add_f32_dpp %0, %4, %4 " CTRL " row_mask:0xf bank_mask:0xf\n\t"               \
      "v_add_f32_dpp %1, %5, %5 " CTRL " row_mask:0xf bank_mask:0xf\n\t"               \
      "v_add_f32_dpp %2, %6, %6 " CTRL " row_mask:0xf bank_mask:0xf\n\t"               \
      "v_add_f32_dpp %3, %7, %7 " CTRL " row_mask:0xf bank_mask:0xf\n\t"               \
      "v_add_f32_dpp %0, %8, %8 " CTRL " row_mask:0xf bank_mask:" BANKS "\n\t"         \
      "v_add_f32_dpp %1, %9, %9 " CTRL " row_mask:0xf bank_mask:" BANKS "\n\t"         \
      "v_add_f32_dpp %2, %10, %10 " CTRL " row_mask:0xf bank_mask:" BANKS "\n\t"       \
      "v_add_f32_dpp %3, %11, %11 " CTRL " row_mask:0xf bank_mask:" BANKS TAIL         \
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])                             \
      : "v"(p0[0]), "v"(p0[1]), "v"(p0[2]), "v"(p0[3]), "v"(p1[0]), "v"(p1[1]),        \
        "v"(p1[2]), "v"(p1[3]))
__device__ __forceinline__ void merge4_bit3(const float* p0, const float* p1, float* r) {
  GDN_MERGE4("row_ror:8", "0xc", "");
}
__device__ __forceinline__ void merge4_bit2(const float* p0, const float* p1, float* r) {
  GDN_MERGE4("row_half_mirror", "0xa", "\n\ts_nop 1");
}
#undef GDN_MERGE4

// One merge over lane bit 5, 4, 1 or 0.
template <int BIT>
__device__ __forceinline__ float merge(float p0, float p1) {
  if constexpr (BIT == 5) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(p0), __float_as_uint(p1),
                                                    false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else if constexpr (BIT == 4) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(p0), __float_as_uint(p1),
                                                    false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    constexpr int ctrl = BIT == 1 ? 0x4E : 0xB1;
    const bool hi = (lane_id() & (1 << BIT)) != 0;
    const float keep = hi ? p1 : p0, give = hi ? p0 : p1;
    return keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), ctrl, 0xf,
                                                             0xf, true));
  }
}

// A lane's columns of the inputs from a chunk's first token on.
template <typename E, bool GATED>
struct Inputs {
  Column<E> x, dt, z, dy;
  float bias;
  uint32_t mask;
  int last;  // the chunk's last token
  __device__ __forceinline__ void open(const BwdArgs& a, const Chunk& ch, const Lane& l) {
    x.open(a.x, ch.t0, a.sx, ch.len, a.C, l.c, true);
    dt.open(a.dt, ch.t0, a.sdt, ch.len, a.C, l.c, true);
    if (GATED) z.open(a.z, ch.t0, a.sz, ch.len, a.C, l.c, true);
    dy.open(a.dy, ch.t0, a.C, ch.len, a.C, l.c, true);
    bias = a.bias ? a.bias[l.c] : 0.f;
    mask = a.softplus ? 0xFFFFFFFFu : 0u;
    last = ch.len - 1;
  }
};

// A token's inputs as loaded (bits, to be widened when they are needed).
template <typename E, bool GATED>
struct Raw {
  uint32_t x, dt, z, dy;
  __device__ __forceinline__ void load(const Inputs<E, GATED>& in, int r) {
    r = min(r, in.last);  // past the chunk: its last token
    x = in.x.load(r);
    dt = in.dt.load(r);
    if (GATED) z = in.z.load(r);
    dy = in.dy.load(r);
  }
  // e = dy silu(z)
  __device__ __forceinline__ float e() const {
    const float d = Column<E>::wide(dy);
    if (!GATED) return d;
    const float v = Column<E>::wide(z);
    return d * (v * sigmoid_f32(v));
  }
};

// The B and C rows of four tokens, through the scalar cache.
struct Rows4 {
  float v[4 * 2 * NS];
  __device__ __forceinline__ void load(const float* rows, int t) {
    const scalar_row r = as_scalar(rows + t * 2 * NS);
#pragma unroll
    for (int i = 0; i < 4 * 2 * NS; ++i) v[i] = r[i];
  }
  __device__ __forceinline__ float b(int i, int k) const { return v[i * 2 * NS + k]; }
  __device__ __forceinline__ float c(int i, int k) const { return v[i * 2 * NS + NS + k]; }
};

template <int NW, bool GATED, typename E>
__global__ __launch_bounds__(64 * NW) void k_scan_bwd_state(BwdArgs a) {
  constexpr int TPW = BT / NW;
  __shared__ float sv[2][3][BT][kScanLanes];  // step, step x, e
  const int slot = blockIdx.x / a.nb;
  const Chunk ch = chunk_of(a.map, slot);
  if (!ch.ok) return;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const Lane l = lane_channel(blockIdx.x - slot * a.nb, a.per, a.nblk);
  Inputs<E, GATED> in;
  in.open(a, ch, l);
  const int tiles = (ch.len + BT - 1) / BT;
  for (int sb = 0; sb < a.Sp; sb += NS * NW) {
    const int s0 = sb + w * NS;
    const float* rows =
        a.bc + (((long)l.g * (a.Sp / NS) + s0 / NS) * a.map.Ttot + ch.t0) * 2 * NS;
    Raw<E, GATED> raw[TPW];
    auto fetch = [&](int tile) {
#pragma unroll
      for (int i = 0; i < TPW; ++i) raw[i].load(in, tile * BT + w * TPW + i);
    };
    if (tiles > 0) fetch(0);
    float A2[NS], h[NS], P[NS], g[NS], sum = 0.f;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      A2[k] = s0 + k < a.S ? a.A[(long)l.c * a.S + s0 + k] * kLog2e : 0.f;
      h[k] = g[k] = 0.f;
      P[k] = 1.f;
    }
    for (int tile = 0; tile < tiles; ++tile) {
      float(*buf)[BT][kScanLanes] = sv[tile & 1];
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const float v = step_f32(Column<E>::wide(raw[i].dt) + in.bias, in.mask);
        buf[0][w * TPW + i][lane] = v;
        buf[1][w * TPW + i][lane] = v * Column<E>::wide(raw[i].x);
        buf[2][w * TPW + i][lane] = raw[i].e();
      }
      fetch(tile + 1);
      __syncthreads();
      const int m = min(BT, ch.len - tile * BT);
      const float* row = rows + (long)tile * BT * 2 * NS;
      auto token = [&](int t, auto b, auto c) {
        const float v = buf[0][t][lane], dx = buf[1][t][lane], e = buf[2][t][lane];
        sum += v;
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const float d = __builtin_amdgcn_exp2f(v * A2[k]);
          h[k] = fmaf(d, h[k], dx * b(k));
          P[k] *= d;
          g[k] = fmaf(P[k], e * c(k), g[k]);
        }
      };
      if (m == BT) {
        Rows4 r0, r1;
        r0.load(row, 0);
        r1.load(row, 4);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < BT; ++t)
          token(t, [&](int k) { return t < 4 ? r0.b(t & 3, k) : r1.b(t & 3, k); },
                [&](int k) { return t < 4 ? r0.c(t & 3, k) : r1.c(t & 3, k); });
      } else {
        for (int t = 0; t < m; ++t) {
          const scalar_row r = as_scalar(row + t * 2 * NS);
          token(t, [&](int k) { return r[k]; }, [&](int k) { return r[NS + k]; });
        }
      }
    }
    if (l.live) {
#pragma unroll
      for (int k = 0; k < NS; ++k)
        if (s0 + k < a.S) {
          a.hst[((long)slot * a.S + s0 + k) * a.C + l.c] = h[k];
          a.gst[((long)slot * a.S + s0 + k) * a.C + l.c] = g[k];
        }
      if (sb == 0 && w == 0) a.dsum[(long)slot * a.C + l.c] = sum;
    }
    __syncthreads();  // the next states' first tile reuses the buffers
  }
}

// One thread per (sequence, state, channel): blockIdx.z 0 composes the start states forwards, 1
// the end gradients backwards, eight chunks loaded ahead.
__global__ __launch_bounds__(256) void k_scan_bwd_combine(BwdArgs a) {
  const int c = blockIdx.y * 256 + threadIdx.x;
  const int n = blockIdx.x / a.S, s = blockIdx.x - n * a.S;
  if (c >= a.C) return;
  int bos, eos;
  chunk_seq(a.map, n, bos, eos);
  const int count = chunk_count(eos - bos, a.map.Lc);
  const long first = a.map.cu ? chunk_first(a.map, n) : (long)n * chunk_count(a.map.T, a.map.Lc);
  const float A2 = a.A[(long)c * a.S + s] * kLog2e;
  const bool back = blockIdx.z == 1;
  const float* from = back ? a.dht : a.h0;
  float v = from ? from[((long)n * a.C + c) * a.S + s] : 0.f;
  float* st = (back ? a.gst : a.hst) + (first * a.S + s) * a.C + c;
  const float* ds = a.dsum + first * a.C + c;
  const long stride = (long)a.S * a.C;
  for (int i0 = 0; i0 < count; i0 += 8) {
    float e[8], d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = back ? count - 1 - (i0 + j) : i0 + j;
      const bool has = i0 + j < count;
      e[j] = has ? st[i * stride] : 0.f;
      d[j] = has ? ds[(long)i * a.C] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = back ? count - 1 - (i0 + j) : i0 + j;
      if (i0 + j < count) st[i * stride] = v;
      v = fmaf(__builtin_amdgcn_exp2f(d[j] * A2), v, e[j]);
    }
  }
}

// One chunk's gradients.  MULTI: more states than the waves hold at once; the sums over states
// are then carried over the state blocks in LDS.
template <int NW, bool MULTI, bool GATED, typename E>
__global__ __launch_bounds__(64 * NW) void k_scan_bwd(BwdArgs a) {
  constexpr int TPW = BT / NW;
  constexpr int PLANES = GATED ? 3 : 2;
  __shared__ float sv[2][3][BT][kScanLanes];          // step, step x, e
  __shared__ float part[PLANES][NW][BT][kScanLanes];  // sum_s B g, sum_s A q, sum_s C h of a tile
  __shared__ float acc[MULTI ? PLANES : 1][MULTI ? kBwdChunk : 1][kScanLanes];
  const int slot = blockIdx.x / a.nb;
  const Chunk ch = chunk_of(a.map, slot);
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const Lane l = lane_channel(blockIdx.x - slot * a.nb, a.per, a.nblk);
  float* dv = a.dvp + (long)slot * 2 * a.C + l.c;
  if (!ch.ok) {  // an unused slot adds nothing
    if (l.live) {
      for (int s = w; s < a.S; s += NW) a.dAp[((long)slot * a.S + s) * a.C + l.c] = 0.f;
      if (w == 0) dv[0] = dv[a.C] = 0.f;
    }
    return;
  }
  Inputs<E, GATED> in;
  in.open(a, ch, l);
  const float Dc = a.D ? a.D[l.c] : 0.f;
  const int tiles = (ch.len + BT - 1) / BT;
  // a lane without a channel adds zeros to the sums over lanes: zero boundaries and inputs
  const float alive = l.live ? 1.f : 0.f;
  float sumD = 0.f, sumb = 0.f;

  for (int sb = 0; sb < a.Sp; sb += NS * NW) {
    const int s0 = sb + w * NS;
    const bool last_sb = !MULTI || sb + NS * NW >= a.Sp;
    const float* rows =
        a.bc + (((long)l.g * (a.Sp / NS) + s0 / NS) * a.map.Ttot + ch.t0) * 2 * NS;
    float A2[NS], h[NS], carry[NS], dA[NS], ck[KT][NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const int s = s0 + k;
      A2[k] = s < a.S ? a.A[(long)l.c * a.S + s] * kLog2e : 0.f;
      h[k] = carry[k] = dA[k] = 0.f;
      if (s < a.S && l.live) {
        const long at = ((long)slot * a.S + s) * a.C + l.c;
        const long out = ((long)ch.n * a.C + l.c) * a.S + s;
        h[k] = a.split ? a.hst[at] : a.h0 ? a.h0[out] : 0.f;
        carry[k] = a.split ? a.gst[at] : a.dht ? a.dht[out] : 0.f;
      }
    }

    // the states at the tiles' starts
#pragma unroll
    for (int j = 0; j < KT; ++j) {
#pragma unroll
      for (int k = 0; k < NS; ++k) ck[j][k] = h[k];
    }
    {
      uint32_t rx[TPW], rd[TPW];
      auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
          const int r = min(tile * BT + w * TPW + i, in.last);
          rx[i] = in.x.load(r);
          rd[i] = in.dt.load(r);
        }
      };
      if (tiles > 1) fetch(0);
      for (int tile = 0; tile + 1 < tiles; ++tile) {
        float(*buf)[BT][kScanLanes] = sv[tile & 1];
        const float* row = rows + tile * BT * 2 * NS;
        Rows4 r0, r1;
        r0.load(row, 0);
        r1.load(row, 4);
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
          const float v = step_f32(Column<E>::wide(rd[i]) + in.bias, in.mask);
          buf[0][w * TPW + i][lane] = v;
          buf[1][w * TPW + i][lane] = v * Column<E>::wide(rx[i]) * alive;
        }
        fetch(tile + 1);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < BT; ++t) {
          const float v = buf[0][t][lane], dx = buf[1][t][lane];
#pragma unroll
          for (int k = 0; k < NS; ++k)
            h[k] = fmaf(__builtin_amdgcn_exp2f(v * A2[k]), h[k],
                        dx * (t < 4 ? r0.b(t & 3, k) : r1.b(t & 3, k)));
        }
#pragma unroll
        for (int j = 1; j < KT; ++j)
          if (j == tile + 1) {
            asm volatile("");  // a branch for the whole wave, not a selection for every value
#pragma unroll
            for (int k = 0; k < NS; ++k) ck[j][k] = h[k];
          }
      }
      __syncthreads();
    }

    Raw<E, GATED> raw[TPW];
    auto fetch = [&](int tile) {
#pragma unroll
      for (int i = 0; i < TPW; ++i) raw[i].load(in, tile * BT + w * TPW + i);
    };
    if (tiles > 0) fetch(tiles - 1);
    for (int tile = tiles - 1; tile >= 0; --tile) {
      const int m = min(BT, ch.len - tile * BT);
      const float* row = rows + tile * BT * 2 * NS;
      // a wave's claim on the vector units falls as its tile is done (see k_scan): 1880 to 1850 us
      // the 8 x 2048-token step
      __builtin_amdgcn_s_setprio(3);
      Rows4 r0, r1;  // asked for before the tile's preparation, which hides their latency
      r0.load(row, 0);
      if (m > 4) r1.load(row, 4);
      Raw<E, GATED> own[TPW];
      float sig[TPW];  // sigmoid(z)
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        own[i] = raw[i];
        const float v = step_f32(Column<E>::wide(own[i].dt) + in.bias, in.mask);
        const float d = Column<E>::wide(own[i].dy);
        if (GATED) sig[i] = sigmoid_f32(Column<E>::wide(own[i].z));
        const float e = GATED ? d * (Column<E>::wide(own[i].z) * sig[i]) : d;
        sv[0][0][w * TPW + i][lane] = v;
        sv[0][1][w * TPW + i][lane] = v * Column<E>::wide(own[i].x) * alive;
        sv[0][2][w * TPW + i][lane] = e * alive;
      }
      if (tile > 0) fetch(tile - 1);
      __syncthreads();

      float start[NS];
#pragma unroll
      for (int k = 0; k < NS; ++k) start[k] = ck[0][k];
#pragma unroll
      for (int j = 1; j < KT; ++j)
        if (j == tile) {
          asm volatile("");
#pragma unroll
          for (int k = 0; k < NS; ++k) start[k] = ck[j][k];
        }
      // the tile's states and decays again, then its tokens backwards, two at a time; FULL: all its
      // tokens are the chunk's.  A token's products for dB and dC (4 states each) merge over the
      // lanes as they come: lane bit 3 takes dB or dC, bit 2 the state's upper bit, bit 4 its
      // lower one, bits 5 1 0 the token's bits 0 1 2
      float all = 0.f;
      auto body = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        float hs[BT][NS], as[BT][NS];
#pragma unroll
        for (int t = 0; t < BT; ++t) {
          if (FULL || t < m) {
            const float v = sv[0][0][t][lane], dx = sv[0][1][t][lane];
#pragma unroll
            for (int k = 0; k < NS; ++k) {
              as[t][k] = __builtin_amdgcn_exp2f(v * A2[k]);
              hs[t][k] = fmaf(as[t][k], t ? hs[t ? t - 1 : 0][k] : start[k],
                              dx * (t < 4 ? r0.b(t & 3, k) : r1.b(t & 3, k)));
            }
          }
        }
        __builtin_amdgcn_s_setprio(1);
        float m1[2], m0[2];
        m1[0] = m1[1] = m0[0] = m0[1] = 0.f;
#pragma unroll
        for (int t1 = BT - 1; t1 >= 0; t1 -= 2) {
          float x2[2][4];  // of the pair's tokens, merged over lane bit 3
#pragma unroll
          for (int t = t1; t > t1 - 2; --t) {
            float* to = x2[t & 1];
            if (FULL || t < m) {
              const float v = sv[0][0][t][lane], dx = sv[0][1][t][lane], e = sv[0][2][t][lane];
              float u = 0.f, q1 = 0.f, yy = 0.f, pb[NS], pc[NS];
#pragma unroll
              for (int k = 0; k < NS; ++k) {
                const float b = t < 4 ? r0.b(t & 3, k) : r1.b(t & 3, k);
                const float c = t < 4 ? r0.c(t & 3, k) : r1.c(t & 3, k);
                const float g = fmaf(e, c, carry[k]);
                carry[k] = as[t][k] * g;
                const float q = carry[k] * (t ? hs[t ? t - 1 : 0][k] : start[k]);
                dA[k] = fmaf(v, q, dA[k]);
                q1 = k ? fmaf(q, A2[k], q1) : q * A2[k];
                u = k ? fmaf(g, b, u) : g * b;
                if (GATED) yy = k ? fmaf(hs[t][k], c, yy) : hs[t][k] * c;
                pb[k] = g * dx;
                pc[k] = e * hs[t][k];
              }
              part[0][w][t][lane] = u;
              part[1][w][t][lane] = q1;
              if (GATED) part[PLANES - 1][w][t][lane] = yy;
              merge4_bit3(pb, pc, to);
            } else {
              to[0] = to[1] = to[2] = to[3] = 0.f;
            }
          }
          // states 0, 1 of the even and the odd token against their states 2, 3
          const float lo[4] = {x2[0][0], x2[0][1], x2[1][0], x2[1][1]};
          const float hi[4] = {x2[0][2], x2[0][3], x2[1][2], x2[1][3]};
          float y4[4];
          merge4_bit2(lo, hi, y4);
          const int j = (t1 >> 1) & 3;  // the pair
          m1[j & 1] = merge<5>(merge<4>(y4[0], y4[1]), merge<4>(y4[2], y4[3]));
          if ((j & 1) == 0) {
            m0[j >> 1] = merge<1>(m1[0], m1[1]);
            if (j == 0) all = merge<0>(m0[0], m0[1]);
          }
        }
      };
      __builtin_amdgcn_s_setprio(2);
      if (m == BT)
        body(std::true_type());
      else
        body(std::false_type());
      __builtin_amdgcn_s_setprio(3);
      {
        const int t = ((lane >> 5) & 1) | (lane & 2) | ((lane & 1) << 2);
        const int k = ((lane >> 1) & 2) | ((lane >> 4) & 1), kind = (lane >> 3) & 1;
        if (t < m)
          a.bcp[(((long)l.blk * a.map.Ttot + ch.t0 + tile * BT + t) * a.G + l.g) * (2 * a.Sp) +
                kind * a.Sp + s0 + k] = all;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const int t = w * TPW + i;
        if (t < m) {
          float u = 0.f, q1 = 0.f, yy = 0.f;
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            u += part[0][k][t][lane];
            q1 += part[1][k][t][lane];
            if (GATED) yy += part[PLANES - 1][k][t][lane];
          }
          if constexpr (MULTI) {
            float* p = &acc[0][tile * BT + t][lane];
            constexpr int plane = kBwdChunk * kScanLanes;
            if (sb > 0) {
              u += p[0];
              q1 += p[plane];
              if (GATED) yy += p[(PLANES - 1) * plane];
            }
            if (!last_sb) {
              p[0] = u;
              p[plane] = q1;
              if (GATED) p[(PLANES - 1) * plane] = yy;
            }
          }
          if (last_sb) {
            const long r = (long)(ch.t0 + tile * BT + t) * a.C;
            const float xv = Column<E>::wide(own[i].x);
            // only this wave writes these, with its next tile
            const float step = sv[0][0][t][lane], e = sv[0][2][t][lane];
            // A q was summed with A log2(e); the slope of softplus is the sigmoid
            float gd = fmaf(q1, 0.6931471805599453f, xv * u);
            if (in.mask) gd *= sigmoid_f32(Column<E>::wide(own[i].dt) + in.bias);
            sumD = fmaf(xv, e, sumD);
            sumb += gd;
            if (l.live) {
              static_cast<E*>(a.dx)[r + l.c] = (E)fmaf(step, u, Dc * e);
              static_cast<E*>(a.ddt)[r + l.c] = (E)gd;
              if (GATED)
                static_cast<E*>(a.dz)[r + l.c] =
                    (E)(Column<E>::wide(own[i].dy) * fmaf(Dc, xv, yy) *
                        (sig[i] * fmaf(Column<E>::wide(own[i].z), 1.f - sig[i], 1.f)));
            }
          }
        }
      }
    }
    if (l.live) {
#pragma unroll
      for (int k = 0; k < NS; ++k)
        if (s0 + k < a.S) {
          a.dAp[((long)slot * a.S + s0 + k) * a.C + l.c] = dA[k];
          if (a.dh0 && ch.i == 0) a.dh0[((long)ch.n * a.C + l.c) * a.S + s0 + k] = carry[k];
        }
    }
    __syncthreads();  // the tiles' buffers are free again
  }
  // the owners' sums over their tokens, through the partial sums' buffer
  part[0][w][0][lane] = sumD;
  part[1][w][0][lane] = sumb;
  __syncthreads();
  if (w == 0 && l.live) {
    float s = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      s += part[0][k][0][lane];
      b += part[1][k][0][lane];
    }
    dv[0] = s;
    dv[a.C] = b;
  }
}

// The partial sums added up.  The first `sums` workgroups take the chunk slots' rows
// [slots][rows][C]: 64 channels each of a row of dA (transposed to [C, S]), dD or d(dt_bias); the
// others take dB and dC, a value a thread, over the channel blocks in order.
template <typename E>
__global__ __launch_bounds__(kColumnThreads) void k_scan_bwd_sums(
    const float* dAp, const float* dvp, const float* bcp, float* dA, float* dD, float* dbias, E* dB,
    E* dC, int slots, int C, int Ttot, int G, int S, int Sp, int nblk, int sums) {
  if ((int)blockIdx.x < sums) {
    const int cols = (C + 63) / 64;
    const int s = blockIdx.x / cols;  // S rows of dA, then dD, d(dt_bias)
    const bool vec = s >= S;
    float* to = !vec ? dA : s == S ? dD : dbias;
    if (!to) return;
    const int c = (blockIdx.x - s * cols) * 64 + lane_id();
    const float r = vec ? column_sum(dvp + (long)(s - S) * C, 2L * C, slots, c, C)
                        : column_sum(dAp + (long)s * C, (long)S * C, slots, c, C);
    if (threadIdx.x < 64 && c < C) to[vec ? c : (long)c * S + s] = r;
    return;
  }
  const long i = (long)(blockIdx.x - sums) * kColumnThreads + threadIdx.x;
  const int row = 2 * Sp;
  const long plane = (long)Ttot * G * row;
  if (i >= plane) return;
  const int k = (int)(i % row);
  const int s = k < Sp ? k : k - Sp;
  if (s >= S) return;
  float v = 0.f;
#pragma unroll 4
  for (int b = 0; b < nblk; ++b) v += bcp[b * plane + i];
  (k < Sp ? dB : dC)[(i / row) * S + s] = (E)v;
}

template <int NW, bool MULTI, typename E>
hipError_t launch_cfg(const ScanProblem& p, const ScanBwd& b, const BwdArgs& a, hipStream_t st) {
  // workgroups in a row (and so on XCDs in turn) are a chunk's channel blocks: chunks of unlike
  // lengths then load the XCDs alike
  const unsigned grid = (unsigned)p.slots * a.nb;
  const int sums = (p.C + 63) / 64 * (p.S + 2);
  auto add_up = [&](long values) {
    k_scan_bwd_sums<E><<<(unsigned)(sums + (values + kColumnThreads - 1) / kColumnThreads),
                         kColumnThreads, 0, st>>>(b.dAp, b.dvp, b.bcp, b.dA, b.dD, b.dbias,
                                                  (E*)b.dB, (E*)b.dC, p.slots, p.C, p.Ttot, p.G,
                                                  p.S, p.Sp, p.nblk, sums);
    return hipGetLastError();
  };
  if (p.slots == 0) return add_up(0);  // no sequences: the parameters' gradients are zero
  if (a.split) {
    if (a.z)
      k_scan_bwd_state<NW, true, E><<<grid, 64 * NW, 0, st>>>(a);
    else
      k_scan_bwd_state<NW, false, E><<<grid, 64 * NW, 0, st>>>(a);
    k_scan_bwd_combine<<<dim3(p.N * p.S, (p.C + 255) / 256, 2), 256, 0, st>>>(a);
  }
  if (a.z)
    k_scan_bwd<NW, MULTI, true, E><<<grid, 64 * NW, 0, st>>>(a);
  else
    k_scan_bwd<NW, MULTI, false, E><<<grid, 64 * NW, 0, st>>>(a);
  return add_up((long)p.Ttot * p.G * 2 * p.Sp);
}

template <typename E>
hipError_t launch_e(const ScanProblem& p, const ScanBwd& b, const BwdArgs& a, hipStream_t st) {
  if (p.nw == 1) return launch_cfg<1, false, E>(p, b, a, st);
  if (p.nw == 2) return launch_cfg<2, false, E>(p, b, a, st);
  if (p.nw == 4) return launch_cfg<4, false, E>(p, b, a, st);
  if (p.S <= 32) return launch_cfg<8, false, E>(p, b, a, st);
  return launch_cfg<8, true, E>(p, b, a, st);
}

}  // namespace

hipError_t launch_scan_bwd(const ScanProblem& p, const ScanBwd& b, hipStream_t st) {
  if (p.slots > 0) {
    const hipError_t e = launch_scan_pack(p, st);
    if (e != hipSuccess) return e;
  }
  BwdArgs a;
  a.x = p.x;
  a.dt = p.dt;
  a.z = p.z;
  a.dy = b.dy;
  a.bc = p.bc;
  a.A = p.A;
  a.D = p.D;
  a.bias = p.bias;
  a.h0 = p.h0;
  a.dht = b.dht;
  a.hst = p.hst;
  a.gst = b.gst;
  a.dsum = p.dsum;
  a.bcp = b.bcp;
  a.dAp = b.dAp;
  a.dvp = b.dvp;
  a.dx = b.dx;
  a.ddt = b.ddt;
  a.dz = b.dz;
  a.dh0 = b.dh0;
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
  a.split = p.slots > p.N;  // otherwise every sequence is one chunk
  return p.f32 ? launch_e<float>(p, b, a, st) : launch_e<bf16>(p, b, a, st);
}

}  // namespace gdn
