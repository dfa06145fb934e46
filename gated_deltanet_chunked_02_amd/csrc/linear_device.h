// Device-side pieces of the linear attention kernels: matrix products of 16-byte operand
// fragments, state tiles that serve as operands, rows of a head staged through registers, and the
// decays of a chunk.
//
// State tiles.  A state of R x N values is held by columns: wave w has 16 (or more) columns, all R
// rows, as 16 x 16 accumulator tiles in pairs; row r of tile t of pair P is row
// 32 P + 8 (r / 4) + 4 t + r % 4 of the state.  In a lane of group g = lane / 16 a pair then holds the
// eight consecutive rows 32 P + 8 g .. + 7, which is what one matrix-core operand takes along k: a
// state goes into a product over its rows without leaving the registers, against 16-byte reads of
// the other operand.
#pragma once

#include "gdn_operands.h"
#include "linear.h"
#include "ssm_device.h"

namespace gdn {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Products of 16-byte fragments: 32 k of bf16 in one instruction, 16 k of fp32 in four.  Lane
// group g holds k = k0 + EPL g .. + EPL - 1 of row (or column) lane % 16.
template <typename E> struct Mx;
template <> struct Mx<bf16> {
  static constexpr int KF = 32, EPL = 8, TERMS = 3;
  typedef bf16x8 frag;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mx<float> {
  static constexpr int KF = 16, EPL = 4, TERMS = 1;
  typedef f32x4 frag;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

// A tile of rows in LDS, D values each.  In bf16 a row has no padding and its 16-byte pieces are
// exchanged by the row (piece j lies at j ^ turn(row)).  LDS gives 256 bytes a cycle where the lanes it
// serves in one have banks of their own: for a row fragment, rows 0-3 and 12-15 of one piece with rows
// 4-11 of its neighbour (or the other way round), hence turns that agree in rows r and r + 4 but differ
// otherwise; for a transposing read of two pieces, 4 rows each of two lane groups (4 and 2 cycles a
// read, with none lost).  A transposing read of halves of four pieces (tr_state) and a write of halves
// take twice their least, whatever the order.  fp32 rows, read transposed one value at a time, are padded
// by 16 bytes.
// l: the lane, or the lane made opaque in a loop, so that addresses are made where they are used and
// not kept in registers throughout.
template <typename E, int D>
struct Tile {
  static constexpr int LD = sizeof(E) == 2 ? D : D + 4;
  static __device__ __forceinline__ int turn(int row) {
    if constexpr (sizeof(E) == 4) return 0;
    if constexpr (D == 64) return (row >> 3 & 1) * 4 + (row >> 1 & 1) * 2 + (row & 1);
    return (row >> 3 & 1) * 9 + (row & 3) * 2;
  }
  // Element offset of piece j (16 bytes) of a row.
  static __device__ __forceinline__ int piece(int row, int j) {
    return row * LD + (j ^ turn(row)) * (16 / (int)sizeof(E));
  }
  // Rows row0 + lane % 16, k from k0 on (row0 a multiple of 16, k0 of KF).
  static __device__ __forceinline__ typename Mx<E>::frag ld(const E* m, int row0, int k0, int l) {
    const int c = l & 15, g = l >> 4;
    return *reinterpret_cast<const typename Mx<E>::frag*>(
        m + row0 * LD + c * LD + ((k0 / Mx<E>::EPL) ^ (g ^ turn(c))) * Mx<E>::EPL);
  }
  // The same rows of a product over a state's rows, step s of it: the tiles 2 s and 2 s + 1 in bf16, tile
  // s in fp32.
  static __device__ __forceinline__ typename Mx<E>::frag ld_state(const E* m, int row0, int s,
                                                                        int l) {
    if constexpr (sizeof(E) == 2) return ld(m, row0, 32 * s, l);
    return *reinterpret_cast<const typename Mx<E>::frag*>(
        m + (row0 + (l & 15)) * LD + 32 * (s >> 1) + 4 * (s & 1) + 8 * (l >> 4));
  }
  // Transposed: rows k0 .. of the tile run along k, and lane % 16 counts columns from n0 on.
  static __device__ __forceinline__ typename Mx<E>::frag tr(const E* m, int k0, int n0, int l) {
    const int c = l & 15, g = l >> 4;
    if constexpr (sizeof(E) == 2) {
      const int row = 8 * g + (c >> 2);
      const int j = (n0 / 8) ^ ((c >> 1 & 1) ^ turn(row));
      return pair(m + k0 * LD + row * LD + 4 * (c & 1), j);
    } else {
      return column(m + (k0 + 4 * g) * LD + n0 + c);
    }
  }
  // Transposed, the columns that state tile t has as rows.
  static __device__ __forceinline__ typename Mx<E>::frag tr_state(const E* m, int k0, int t, int l) {
    const int c = l & 15, g = l >> 4;
    if constexpr (sizeof(E) == 2) {
      const int row = 8 * g + (c >> 2);
      const int j = (4 * (t >> 1)) ^ ((c & 3) ^ turn(row));
      return pair(m + k0 * LD + row * LD + 4 * (t & 1), j);
    } else {
      return column(m + (k0 + 4 * g) * LD + 32 * (t >> 1) + 4 * (t & 1) + 8 * (c >> 2) + (c & 3));
    }
  }

 private:
  // turn(row + 4) = turn(row) for the rows of the first half
  static __device__ __forceinline__ bf16x8 pair(const E* row, int j) {
    const bf16x4 a = read_tr4(row + j * 8), b = read_tr4(row + 4 * LD + j * 8);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  static __device__ __forceinline__ f32x4 column(const E* p) {
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = p[i * LD];
    return r;
  }
};

// Column offset of state tile t.
__device__ __forceinline__ int tile_col(int t) { return 32 * (t >> 1) + 4 * (t & 1); }
// A lane's first row of state tile t; it holds four.
__device__ __forceinline__ int tile_row(int t, int l) { return tile_col(t) + 8 * (l >> 4); }

// x as TERMS operands whose sum is x to fp32's last bits: three bf16 terms carry 24 bits, so a
// state or a weighted row in a product with bf16 data loses nothing that fp32 would keep.
template <typename E, int TERMS = Mx<E>::TERMS>
__device__ __forceinline__ void split(const float* x, typename Mx<E>::frag* out) {
  if constexpr (sizeof(E) == 2) {
    // two values at a time: one conversion makes both, and each is half of its 32 bits
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      f32x2 r = {x[e], x[e + 1]};
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        const bf16x2_t b = __builtin_convertvector(r, bf16x2_t);
        out[t][e] = b[0];
        out[t][e + 1] = b[1];
        const uint32_t u = __builtin_bit_cast(uint32_t, b);
        r[0] -= __uint_as_float(u << 16);
        r[1] -= __uint_as_float(u & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[0][e] = x[e];
  }
}

// A chunk's rows of one head; nothing where there are none.
template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const E* base, int64_t stride, int width,
                                                          int len) {
  // rows are at least as far apart as wide: no rows, no bytes
  const int bytes = max(((len - 1) * (int)stride + width) * (int)sizeof(E), 0);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(base), 0, bytes, 0x00020000);
}

// x . four consecutive columns of a tile's row
template <typename E, int D>
__device__ __forceinline__ float dot4(const E* m, int row, int col, f32x4 x) {
  typedef E four __attribute__((ext_vector_type(4)));
  constexpr int V = 16 / (int)sizeof(E);
  const four y = *reinterpret_cast<const four*>(m + Tile<E, D>::piece(row, col / V) + col % V);
  float r = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) r = fmaf(x[e], (float)y[e], r);
  return r;
}

// A chunk's rows of one head, C x D values (D a tile size; the head's own `width` may be less), on
// their way from memory to LDS through registers.  A buffer resource ends behind the chunk's last
// row, so rows past it and columns past the head read as zeros.
template <typename E, int D, int C, int NTH>
struct Rows {
  typedef Tile<E, D> T;
  static constexpr int V = 16 / (int)sizeof(E), VPR = D / V, RS = NTH / VPR;
  // vectors a thread; a small tile leaves the last threads without
  static constexpr int N = C * VPR < NTH ? 1 : C * VPR / NTH;
  static_assert((C * VPR % NTH == 0 || C * VPR < NTH) && NTH % VPR == 0, "block shape");
  u32x4 reg[N];
  // base: the chunk's first row of this head; len: its rows; all uniform.  t: the thread, or its number
  // made opaque in a loop.
  __device__ __forceinline__ void load(const E* base, int64_t stride, int width, int len, int t) {
    const __amdgpu_buffer_rsrc_t rs = rows_of(base, stride, width, len);
    const int row = t / VPR, col = t % VPR, bytes = (int)stride * (int)sizeof(E);
    // steps of less than 2^31 bytes leave kNoColumn past every buffer
    const uint32_t off = col * V < width && row < C ? (uint32_t)(row * bytes + col * 16) : kNoColumn;
#pragma unroll
    for (int j = 0; j < N; ++j)
      reg[j] = __builtin_amdgcn_raw_buffer_load_b128(
          rs, off + (uint32_t)j * (uint32_t)(RS * bytes), 0, 0);
  }
  __device__ __forceinline__ void store(E* lds, int t) const {
    const int row = t / VPR, col = t % VPR;
    if (C * VPR < NTH && row >= C) return;
#pragma unroll
    for (int j = 0; j < N; ++j)
      *reinterpret_cast<u32x4*>(lds + T::piece(row + j * RS, col)) = reg[j];
  }
};

// Element offset of a row of a chunk: fewer than 64 rows, less than 2^23 elements apart, in one 24-bit
// multiplication.
__device__ __forceinline__ uint32_t row_at(int row, int64_t stride) {
  return __umul24((uint32_t)row, (uint32_t)stride);
}

// Four consecutive columns of a row, rounded once, through a buffer resource that drops rows past
// the chunk's end.
template <typename E>
__device__ __forceinline__ void store4(__amdgpu_buffer_rsrc_t rs, uint32_t off, f32x4 x) {
  if constexpr (sizeof(E) == 2)
    __builtin_amdgcn_raw_buffer_store_b64(
        __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4)), rs, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), rs, off, 0, 0);
}

// The same into an LDS tile of D columns.
template <typename E, int D>
__device__ __forceinline__ void put4(E* m, int row, int col, f32x4 x) {
  constexpr int V = 16 / (int)sizeof(E);
  E* to = m + Tile<E, D>::piece(row, col / V) + col % V;
  if constexpr (sizeof(E) == 2)
    *reinterpret_cast<bf16x4*>(to) = __builtin_convertvector(x, bf16x4);
  else
    *reinterpret_cast<f32x4*>(to) = x;
}

// Scores in LDS: C x C values as two bf16 terms (16 bits or more of each), or as themselves in fp32.  One
// term would be a rounding that all of a token's columns share, which shows in a short sequence's o.
template <typename E, int C>
struct Scores {
  typedef Tile<E, C> T;
  static constexpr int TERMS = sizeof(E) == 2 ? 2 : 1;
  __align__(256) E m[TERMS][C * T::LD];
  __device__ __forceinline__ void clear(int t, int threads) {
    for (int i = t; i < TERMS * C * T::LD; i += threads) m[0][i] = (E)0.f;
  }
  __device__ __forceinline__ void put(int row, int col, f32x4 x) {
    put4<E, C>(m[0], row, col, x);
    if constexpr (TERMS == 2) {
      const bf16x4 b = __builtin_convertvector(x, bf16x4);
      put4<E, C>(m[TERMS - 1], row, col, x - __builtin_convertvector(b, f32x4));
    }
  }
};

__device__ __forceinline__ float exp2_f32(float x) { return __builtin_amdgcn_exp2f(x); }

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_d(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive prefix sum across a wave (the order of wave_incl_scan).
__device__ __forceinline__ double wave_incl_scan(double x) {
  x += dpp_d<0x111>(x);
  x += dpp_d<0x112>(x);
  x += dpp_d<0x114>(x);
  x += dpp_d<0x118>(x);
  x += dpp_d<0x142, 0xA>(x);
  x += dpp_d<0x143, 0xC>(x);
  return x;
}

__device__ __forceinline__ double last_lane(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63),
                 hi = __builtin_amdgcn_readlane((int)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum over the four lane groups that share lane % 16, in all of them, without LDS: the two instructions
// exchange rows 1, 3 of one operand with 0, 2 of the other, and rows 2, 3 with 0, 1.
__device__ __forceinline__ float group_sum(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ double group_sum(double x) {
  auto join = [](uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  uint64_t u = __builtin_bit_cast(uint64_t, x);
  auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  x = join(lo[0], hi[0]) + join(lo[1], hi[1]);
  u = __builtin_bit_cast(uint64_t, x);
  lo = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
  hi = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  return join(lo[0], hi[0]) + join(lo[1], hi[1]);
}

// A chunk's decays.  G_t, the sum of log2 decays up to token t, is held in fp64: the decay between
// two tokens is a difference of two of them, which in fp32 would lose its last bits behind tokens of
// strong decay.  A log2 decay below -1000 (an infinity, or a mask's lowest value: a state forgotten)
// is taken as that, which is as good as none left, and keeps the differences finite.
template <int C>
struct Decays {
  double G[C];
  float into[C];  // 2^G_t: from the chunk's start
  float left[C];  // 2^(G_end - G_t): to its end; into[C - 1] is the whole chunk's
  // one wave's work; x: the log-decay of the lane's token (lane < C), 0 past the chunk's end
  __device__ __forceinline__ double make(float x) {
    const int t = lane_id();
    double g2 = (double)x * 1.4426950408889634;
    g2 = g2 < -1000.0 ? -1000.0 : g2;
    const double s = wave_incl_scan(t < C ? g2 : 0.0);
    const double end = last_lane(s);
    if (t < C) {
      G[t] = s;
      into[t] = exp2_f32((float)s);
      left[t] = exp2_f32((float)(end - s));
    }
    return end;
  }
};

// The decays from tokens j .. j + 3 of a chunk to token i, whatever they are for tokens behind i: all
// four at once, because a compiler that makes each where it is wanted waits for LDS each time.
template <int C>
__device__ __forceinline__ f32x4 decays(const Decays<C>& d, int i, int j) {
  typedef double two __attribute__((ext_vector_type(2)));
  const double Gi = d.G[i];
  const two a = *reinterpret_cast<const two*>(d.G + j), b = *reinterpret_cast<const two*>(d.G + j + 2);
  f32x4 r = {exp2_f32((float)(Gi - a[0])), exp2_f32((float)(Gi - a[1])),
             exp2_f32((float)(Gi - b[0])), exp2_f32((float)(Gi - b[1]))};
  opaque(r);
  return r;
}

// The log-decay of the lane's token of a chunk that starts at token t0 (0 past its end): always one
// load, so that the number of loads in flight is known.
__device__ __forceinline__ float load_decay(const LinearProblem& p, long t0, int len, int h) {
  const int t = lane_id(), step = p.head_decay ? 0 : p.H;
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(p.g) + (p.head_decay ? 0 : t0 * p.H) + h, 0,
      len > 0 ? ((len - 1) * step + 1) * 4 : 0, 0x00020000);
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
      rs, t < len ? (uint32_t)(t * step * 4) : kNoColumn, 0, 0));
}

// Workgroup b's unit of work: the `group` units in a row that read the same q and k rows run on one
// XCD one after another (workgroups go to the 8 XCDs in turn), the groups on the XCDs in turn.
__device__ __forceinline__ int unit_of(int b, int blocks, int group) {
  const int full = blocks / (8 * group) * (8 * group);
  if (b >= full) return b;
  const int xcd = b & 7, slot = b >> 3;
  return ((slot / group) * 8 + xcd) * group + slot % group;
}

// For unit_of: the value heads (and slabs) of a q/k head, unless that leaves too few groups for the
// XCDs.
inline int group_of(const LinearProblem& p, int slabs, int blocks) {
  int group = p.H / p.Hg * slabs;
  while (group > 1 && blocks / group < 32) group = (group + 1) / 2;
  return group;
}

// Waits for every load.  Before a loop that keeps loads in flight: its waits then count the loop's own
// loads and stores, and need not suit a first round that came without stores as well, which would have
// each later round wait for the stores of the one before.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0F70); }

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The slot of the state kept at the end of a segment's chunk m is this + m / every (slots of the form of
// ssm.h, every * C tokens long; a segment is no longer than that or a multiple of it).
__device__ __forceinline__ int first_anchor(const LinearProblem& p, const Chunk& c, int every, int C) {
  const ChunkMap map = {p.cu, p.T, p.Ttot, p.N, every * C};
  const int first = p.cu ? chunk_first(map, c.n) : c.n * chunk_count(p.T, every * C);
  return uniform(first + (c.t0 - c.bos) / (every * C));
}

// A wave's share of the TT (TT + 1) / 2 lower tiles of a chunk's scores, every NW-th: handed to `f` at
// once (f(Count<N>, the first's number)), so that their products overlap, or one after the other where
// registers are short.
template <int N> struct Count { static constexpr int value = N; };
template <int TT, int NW, bool TOGETHER, typename F>
__device__ __forceinline__ void lower_tiles(int wave, F f) {
  constexpr int TILES = TT * (TT + 1) / 2, MOST = (TILES + NW - 1) / NW;
  if constexpr (!TOGETHER) {
    for (int x = wave; x < TILES; x += NW) f(Count<1>(), x);
  } else if (wave + (MOST - 1) * NW < TILES) {
    f(Count<MOST>(), wave);
  } else if constexpr (MOST > 1) {
    f(Count<MOST - 1>(), wave);
  }
}
__device__ __forceinline__ int tile_i(int x) { return x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3; }

// A segment slot's chunk (see ssm_device.h), its values known to be the same in every lane.
__device__ __forceinline__ Chunk uniform_chunk(const LinearProblem& p, int slot) {
  const ChunkMap m = {p.cu, p.T, p.Ttot, p.N, p.Lc};
  Chunk c = chunk_of(m, slot);
  c.n = uniform(c.n);
  c.i = uniform(c.i);
  c.count = uniform(c.count);
  c.bos = uniform(c.bos);
  c.t0 = uniform(c.t0);
  c.len = uniform(c.len);
  c.ok = uniform(c.ok) != 0;
  return c;
}

}  // namespace gdn
