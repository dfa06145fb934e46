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
// every sequence is split into chunks of kBwdChunk tokens, and
//   * k_scan_bwd_state finds, for every chunk from zero boundaries, its end state and the gradient
//     a g that it hands to the chunk before it (both in one pass over its tokens: the gradient's
//     factors are the running products of a), and its sum of steps;
//   * k_scan_bwd_combine composes the chunks' start states forwards and their end gradients
//     backwards;
//   * k_scan_bwd goes over a chunk's tiles once to find the states at their starts, then over the
//     tiles from the last to the first: the tile's states and decays again, kept in registers,
//     then its tokens backwards;
//   * sums over channels (dB, dC) and over time (dA, dD, dt_bias) leave partial sums per channel
//     block and per chunk, which two small kernels add in a fixed order (no atomics).
// The sums over the 64 lanes of a wave are the awkward part: dB and dC need one for each (token,
// state).  A transposing butterfly merges two registers into one at every step (lanes keep the
// half of the pair that their lane bit names), so 64 sums cost 63 merges, and end one to a lane.
#include "ssm_device.h"

namespace gdn {

namespace {

constexpr int BT = 8;                  // tokens of a tile
constexpr int KT = kBwdChunk / BT;     // tiles of a chunk
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
  int softplus, split;
};

struct Lane {
  int g, blk, c;
  bool live;
};
__device__ __forceinline__ Lane lane_channel(int per, int nblk) {
  Lane l;
  l.g = blockIdx.y / nblk;
  l.blk = blockIdx.y - l.g * nblk;
  const int cl = l.blk * kScanLanes + lane_id();
  l.live = cl < per;
  l.c = l.g * per + min(cl, per - 1);
  return l;
}

// Adds the lanes that differ in lane bit BIT: lanes without the bit keep p0's sums, lanes with it
// p1's (for BIT 4 the partner is the mirrored lane of its eight, which pairs the same halves).
template <int BIT>
__device__ __forceinline__ float merge(float p0, float p1) {
  if constexpr (BIT == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(p0), __float_as_uint(p1),
                                                    false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else if constexpr (BIT == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(p0), __float_as_uint(p1),
                                                    false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    constexpr int ctrl = BIT == 8 ? 0x128 : BIT == 4 ? 0x141 : BIT == 2 ? 0x4E : 0xB1;
    const bool hi = (lane_id() & BIT) != 0;
    const float keep = hi ? p1 : p0, give = hi ? p0 : p1;
    return keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), ctrl, 0xf,
                                                             0xf, true));
  }
}

// What a token's owner wave makes of its inputs.
struct Token {
  float x, step, slope, dy, z, e;
};
template <typename E>
__device__ __forceinline__ Token make_token(E x, E dt, E dy, E z, float bias, bool softplus,
                                            bool gate) {
  Token k;
  k.x = (float)x;
  const float raw = (float)dt + bias;
  k.step = softplus ? softplus_f32(raw) : raw;
  k.slope = softplus ? sigmoid_f32(raw) : 1.f;
  k.dy = (float)dy;
  k.z = gate ? (float)z : 0.f;
  k.e = gate ? k.dy * (k.z * sigmoid_f32(k.z)) : k.dy;
  return k;
}

template <int NW, typename E>
__global__ __launch_bounds__(64 * NW) void k_scan_bwd_state(BwdArgs a) {
  constexpr int TPW = BT / NW;
  __shared__ float4 sv[2][BT][kScanLanes];  // (step, step x, e, -)
  const int slot = blockIdx.x;
  const Chunk ch = chunk_of(a.map, slot);
  if (!ch.ok) return;
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const Lane l = lane_channel(a.per, a.nblk);
  const E* x = static_cast<const E*>(a.x) + l.c;
  const E* dt = static_cast<const E*>(a.dt) + l.c;
  const E* z = static_cast<const E*>(a.z) + l.c;
  const E* dy = static_cast<const E*>(a.dy) + l.c;
  const float bias = a.bias ? a.bias[l.c] : 0.f;
  const int tiles = (ch.len + BT - 1) / BT;
  for (int sb = 0; sb < a.Sp; sb += NS * NW) {
    const int s0 = sb + w * NS;
    float A2[NS], h[NS], P[NS], g[NS], sum = 0.f;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      A2[k] = s0 + k < a.S ? a.A[(long)l.c * a.S + s0 + k] * kLog2e : 0.f;
      h[k] = g[k] = 0.f;
      P[k] = 1.f;
    }
    E rx[TPW], rd[TPW], rz[TPW], ry[TPW];
    auto fetch = [&](int tile) {
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const long r = ch.t0 + min(tile * BT + w * TPW + i, ch.len - 1);
        rx[i] = x[r * a.sx];
        rd[i] = dt[r * a.sdt];
        ry[i] = dy[r * a.C];
        if (a.z) rz[i] = z[r * a.sz];
      }
    };
    if (tiles > 0) fetch(0);
    for (int tile = 0; tile < tiles; ++tile) {
      float4(*buf)[kScanLanes] = sv[tile & 1];
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const Token k = make_token<E>(rx[i], rd[i], ry[i], rz[i], bias, a.softplus, a.z);
        buf[w * TPW + i][lane] = make_float4(k.step, k.step * k.x, k.e, 0.f);
      }
      if (tile + 1 < tiles) fetch(tile + 1);
      __syncthreads();
      const int m = min(BT, ch.len - tile * BT);
      const float* row = a.bc + ((long)(ch.t0 + tile * BT) * a.G + l.g) * (2 * a.Sp) + s0;
      const long step = (long)a.G * (2 * a.Sp);
      auto token = [&](int t) {
        const scalar_row b = as_scalar(row + t * step);
        const scalar_row c = as_scalar(row + t * step + a.Sp);
        const float4 v = buf[t][lane];
        sum += v.x;
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const float d = __builtin_amdgcn_exp2f(v.x * A2[k]);
          h[k] = fmaf(d, h[k], v.y * b[k]);
          P[k] *= d;
          g[k] = fmaf(P[k], v.z * c[k], g[k]);
        }
      };
      if (m == BT) {
#pragma unroll
        for (int t = 0; t < BT; ++t) token(t);
      } else {
        for (int t = 0; t < m; ++t) token(t);
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
template <int NW, bool MULTI, typename E>
__global__ __launch_bounds__(64 * NW) void k_scan_bwd(BwdArgs a) {
  constexpr int TPW = BT / NW;
  __shared__ float4 sv[2][BT][kScanLanes];
  __shared__ float part[3][NW][BT][kScanLanes];  // sum_s B g, sum_s A q, sum_s C h of a tile
  __shared__ float acc[MULTI ? 3 : 1][MULTI ? kBwdChunk : 1][kScanLanes];
  const int slot = blockIdx.x;
  const Chunk ch = chunk_of(a.map, slot);
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(wave_id());
  const Lane l = lane_channel(a.per, a.nblk);
  float* dv = a.dvp + (long)slot * 2 * a.C + l.c;
  if (!ch.ok) {  // an unused slot adds nothing
    if (l.live) {
      for (int s = w; s < a.S; s += NW) a.dAp[((long)slot * a.S + s) * a.C + l.c] = 0.f;
      if (w == 0) dv[0] = dv[a.C] = 0.f;
    }
    return;
  }
  const E* x = static_cast<const E*>(a.x) + l.c;
  const E* dt = static_cast<const E*>(a.dt) + l.c;
  const E* z = static_cast<const E*>(a.z) + l.c;
  const E* dy = static_cast<const E*>(a.dy) + l.c;
  E* dx = static_cast<E*>(a.dx) + l.c;
  E* ddt = static_cast<E*>(a.ddt) + l.c;
  E* dz = static_cast<E*>(a.dz) + l.c;
  const float bias = a.bias ? a.bias[l.c] : 0.f;
  const float Dc = a.D ? a.D[l.c] : 0.f;
  const int tiles = (ch.len + BT - 1) / BT;
  const long step = (long)a.G * (2 * a.Sp);
  float sumD = 0.f, sumb = 0.f;

  for (int sb = 0; sb < a.Sp; sb += NS * NW) {
    const int s0 = sb + w * NS;
    const bool last_sb = !MULTI || sb + NS * NW >= a.Sp;
    const float* rows = a.bc + ((long)ch.t0 * a.G + l.g) * (2 * a.Sp) + s0;
    float A2[NS], h[NS], carry[NS], dA[NS], ck[KT][NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const int s = s0 + k;
      A2[k] = s < a.S ? a.A[(long)l.c * a.S + s] * kLog2e : 0.f;
      h[k] = carry[k] = dA[k] = 0.f;
      // a lane without a channel adds zeros to the sums over lanes: zero boundaries and inputs
      if (s < a.S && l.live) {
        const long in = ((long)slot * a.S + s) * a.C + l.c;
        const long out = ((long)ch.n * a.C + l.c) * a.S + s;
        h[k] = a.split ? a.hst[in] : a.h0 ? a.h0[out] : 0.f;
        carry[k] = a.split ? a.gst[in] : a.dht ? a.dht[out] : 0.f;
      }
    }

    // the states at the tiles' starts
    {
      E rx[TPW], rd[TPW];
      auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
          const long r = ch.t0 + min(tile * BT + w * TPW + i, ch.len - 1);
          rx[i] = x[r * a.sx];
          rd[i] = dt[r * a.sdt];
        }
      };
      if (tiles > 1) fetch(0);
#pragma unroll
      for (int k = 0; k < NS; ++k) ck[0][k] = h[k];
      for (int tile = 0; tile + 1 < tiles; ++tile) {
        float4(*buf)[kScanLanes] = sv[tile & 1];
#pragma unroll
        for (int i = 0; i < TPW; ++i) {
          float v = (float)rd[i] + bias;
          if (a.softplus) v = softplus_f32(v);
          buf[w * TPW + i][lane] = make_float4(v, l.live ? v * (float)rx[i] : 0.f, 0.f, 0.f);
        }
        if (tile + 2 < tiles) fetch(tile + 1);
        __syncthreads();
        const float* row = rows + (long)tile * BT * step;
#pragma unroll
        for (int t = 0; t < BT; ++t) {
          const scalar_row b = as_scalar(row + t * step);
          const float4 v = buf[t][lane];
#pragma unroll
          for (int k = 0; k < NS; ++k)
            h[k] = fmaf(__builtin_amdgcn_exp2f(v.x * A2[k]), h[k], v.y * b[k]);
        }
#pragma unroll
        for (int j = 1; j < KT; ++j)
          if (j == tile + 1) {
#pragma unroll
            for (int k = 0; k < NS; ++k) ck[j][k] = h[k];
          }
      }
      __syncthreads();
    }

    E rx[TPW], rd[TPW], rz[TPW], ry[TPW];
    auto fetch = [&](int tile) {
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const long r = ch.t0 + min(tile * BT + w * TPW + i, ch.len - 1);
        rx[i] = x[r * a.sx];
        rd[i] = dt[r * a.sdt];
        ry[i] = dy[r * a.C];
        if (a.z) rz[i] = z[r * a.sz];
      }
    };
    if (tiles > 0) fetch(tiles - 1);
    for (int tile = tiles - 1; tile >= 0; --tile) {
      Token own[TPW];
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        own[i] = make_token<E>(rx[i], rd[i], ry[i], rz[i], bias, a.softplus, a.z);
        sv[0][w * TPW + i][lane] =
            l.live ? make_float4(own[i].step, own[i].step * own[i].x, own[i].e, 0.f)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (tile > 0) fetch(tile - 1);
      __syncthreads();
      const int m = min(BT, ch.len - tile * BT);
      const float* row = rows + (long)tile * BT * step;

      float start[NS], hs[BT][NS], as[BT][NS];
#pragma unroll
      for (int j = 0; j < KT; ++j)
        if (j == tile) {
#pragma unroll
          for (int k = 0; k < NS; ++k) start[k] = ck[j][k];
        }
#pragma unroll
      for (int t = 0; t < BT; ++t) {
        if (t < m) {
          const scalar_row b = as_scalar(row + t * step);
          const float4 v = sv[0][t][lane];
#pragma unroll
          for (int k = 0; k < NS; ++k) {
            as[t][k] = __builtin_amdgcn_exp2f(v.x * A2[k]);
            hs[t][k] = fmaf(as[t][k], t ? hs[t ? t - 1 : 0][k] : start[k], v.y * b[k]);
          }
        }
      }
      // tokens backwards; their 8 products a token (4 states of dB, 4 of dC) merge over the
      // lanes as they come: lane bits 5 4 3 take the product's index, bits 2 1 0 the token's
      // bits 0 1 2
      float m2[2], m1[2], m0[2], all = 0.f;
      m2[0] = m2[1] = m1[0] = m1[1] = m0[0] = m0[1] = 0.f;
#pragma unroll
      for (int t = BT - 1; t >= 0; --t) {
        float token_sum = 0.f;
        if (t < m) {
          const scalar_row b = as_scalar(row + t * step);
          const scalar_row c = as_scalar(row + t * step + a.Sp);
          const float4 v = sv[0][t][lane];
          float u = 0.f, q1 = 0.f, yy = 0.f, pb[NS], pc[NS];
#pragma unroll
          for (int k = 0; k < NS; ++k) {
            const float g = fmaf(v.z, c[k], carry[k]);
            const float ah = as[t][k] * (t ? hs[t ? t - 1 : 0][k] : start[k]);
            const float q = g * ah;
            dA[k] = fmaf(v.x, q, dA[k]);
            q1 = fmaf(q, A2[k], q1);
            u = fmaf(g, b[k], u);
            yy = fmaf(hs[t][k], c[k], yy);
            pb[k] = g * v.y;
            pc[k] = v.z * hs[t][k];
            carry[k] = as[t][k] * g;
          }
          part[0][w][t][lane] = u;
          part[1][w][t][lane] = q1;
          part[2][w][t][lane] = yy;
          const float r0 = merge<32>(pb[0], pc[0]), r1 = merge<32>(pb[1], pc[1]);
          const float r2 = merge<32>(pb[2], pc[2]), r3 = merge<32>(pb[3], pc[3]);
          token_sum = merge<8>(merge<16>(r0, r2), merge<16>(r1, r3));
        }
        m2[t & 1] = token_sum;
        if ((t & 1) == 0) {
          m1[(t >> 1) & 1] = merge<4>(m2[0], m2[1]);
          if ((t & 2) == 0) {
            m0[(t >> 2) & 1] = merge<2>(m1[0], m1[1]);
            if (t == 0) all = merge<1>(m0[0], m0[1]);
          }
        }
      }
      {
        const int t = ((lane >> 2) & 1) | (lane & 2) | ((lane & 1) << 2);
        const int k = (lane >> 3) & 3, kind = lane >> 5;
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
            yy += part[2][k][t][lane];
          }
          if constexpr (MULTI) {
            float* p = &acc[0][tile * BT + t][lane];
            constexpr int plane = kBwdChunk * kScanLanes;
            if (sb > 0) {
              u += p[0];
              q1 += p[plane];
              yy += p[2 * plane];
            }
            if (!last_sb) {
              p[0] = u;
              p[plane] = q1;
              p[2 * plane] = yy;
            }
          }
          if (last_sb) {
            const Token& o = own[i];
            const long r = (long)(ch.t0 + tile * BT + t) * a.C;
            // A q was summed with A log2(e)
            const float gd = fmaf(q1, 0.6931471805599453f, o.x * u) * o.slope;
            sumD = fmaf(o.x, o.e, sumD);
            sumb += gd;
            if (l.live) {
              dx[r] = (E)fmaf(o.step, u, Dc * o.e);
              ddt[r] = (E)gd;
              if (a.z) {
                const float sg = sigmoid_f32(o.z);
                dz[r] = (E)(o.dy * fmaf(Dc, o.x, yy) * (sg * fmaf(o.z, 1.f - sg, 1.f)));
              }
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

// dB and dC: the channel blocks' partial sums, in order.
template <typename E>
__global__ __launch_bounds__(256) void k_scan_bwd_bc(const float* bcp, E* dB, E* dC, int Ttot,
                                                     int G, int S, int Sp, int nblk) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  const int row = 2 * Sp;
  const long plane = (long)Ttot * G * row;
  if (i >= plane) return;
  const int k = (int)(i % row);
  const int s = k < Sp ? k : k - Sp;
  if (s >= S) return;
  float v = 0.f;
  for (int b = 0; b < nblk; ++b) v += bcp[b * plane + i];
  (k < Sp ? dB : dC)[(i / row) * S + s] = (E)v;
}

// Sums over the chunk slots of rows [slots][rows][C]: dA (transposed to [C, S]) or dD and
// d(dt_bias).
__global__ __launch_bounds__(256) void k_scan_bwd_params(const float* dAp, const float* dvp,
                                                         float* dA, float* dD, float* dbias,
                                                         int slots, int C, int S) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  const int s = blockIdx.y;  // S rows of dA, then dD, d(dt_bias)
  if (c >= C) return;
  const bool vec = s >= S;
  float* to = !vec ? dA + (long)c * S + s : s == S ? dD : dbias;
  if (!to) return;
  const float* p = vec ? dvp + (long)(s - S) * C + c : dAp + (long)s * C + c;
  const long stride = (long)(vec ? 2 : S) * C;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  int i = 0;
  for (; i + 4 <= slots; i += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += p[(long)(i + j) * stride];
  }
  for (; i < slots; ++i) v[0] += p[(long)i * stride];
  const float r = (v[0] + v[1]) + (v[2] + v[3]);
  if (vec) to[c] = r; else *to = r;
}

template <int NW, bool MULTI, typename E>
hipError_t launch_cfg(const ScanProblem& p, const ScanBwd& b, const BwdArgs& a, hipStream_t st) {
  const dim3 grid(p.slots, p.G * p.nblk);
  if (p.slots == 0) {  // no sequences: the parameters' gradients are zero
    k_scan_bwd_params<<<dim3((p.C + 255) / 256, p.S + 2), 256, 0, st>>>(
        b.dAp, b.dvp, b.dA, b.dD, b.dbias, 0, p.C, p.S);
    return hipGetLastError();
  }
  if (a.split) {
    k_scan_bwd_state<NW, E><<<grid, 64 * NW, 0, st>>>(a);
    k_scan_bwd_combine<<<dim3(p.N * p.S, (p.C + 255) / 256, 2), 256, 0, st>>>(a);
  }
  k_scan_bwd<NW, MULTI, E><<<grid, 64 * NW, 0, st>>>(a);
  const long n = (long)p.Ttot * p.G * 2 * p.Sp;
  if (n > 0)
    k_scan_bwd_bc<E><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(
        b.bcp, (E*)b.dB, (E*)b.dC, p.Ttot, p.G, p.S, p.Sp, p.nblk);
  k_scan_bwd_params<<<dim3((p.C + 255) / 256, p.S + 2), 256, 0, st>>>(
      b.dAp, b.dvp, b.dA, b.dD, b.dbias, p.slots, p.C, p.S);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_e(const ScanProblem& p, const ScanBwd& b, const BwdArgs& a, hipStream_t st) {
  if (p.nw == 1) return launch_cfg<1, false, E>(p, b, a, st);
  if (p.nw == 2) return launch_cfg<2, false, E>(p, b, a, st);
  if (p.S <= 16) return launch_cfg<4, false, E>(p, b, a, st);
  return launch_cfg<4, true, E>(p, b, a, st);
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
  a.Sp = p.Sp;
  a.softplus = p.softplus;
  a.split = p.slots > p.N;  // otherwise every sequence is one chunk
  return p.f32 ? launch_e<float>(p, b, a, st) : launch_e<bf16>(p, b, a, st);
}

}  // namespace gdn
