// The gradient of the causal depthwise convolution.  With x~ a sequence's inputs behind the W - 1
// before it, u[t] = bias + sum_i w[i] x~[t + i] and y = act(u),
//
//   du[t]    = dy[t] act'(u[t])
//   dx~[e]   = sum_i w[i] du[e - i]  (over the tokens the sequence has), plus the gradient of the
//              final state where x~[e] is one of its last W - 1 entries
//   dw[i]    = sum_t du[t] x~[t + i],   dbias = sum_t du[t]
//
// One thread per 4 channels and a block of tokens, walked in order with the last W - 1 inputs
// and du in registers: x and dy are read once (but for the W - 1 tokens after a block, whose du
// its last outputs need), dx is written once.  Each block leaves its share of dw and dbias as a
// partial sum; a second kernel adds them in order.  4 x 8192 tokens of 12288 channels, W = 4, SiLU,
// bf16 (2.4 GB) take 509 us (4.7 TB/s, 92 % of a copy's rate) and 9 us for the sums.
#include "gdn_device.h"
#include "norm.h"
#include "ssm_device.h"
#include "vec4.h"

namespace gdn {

namespace {

constexpr int kVec = 4;    // channels a thread: 8 would take 183 registers (2 waves a SIMD)
constexpr int kGroup = 4;  // tokens whose loads are issued together
constexpr int kThreads = 256;

struct Span {
  int bos, eos;
};

__device__ __forceinline__ Span conv_span(const ConvBwdProblem& p, int n) {
  Span s;
  if (p.cu) {
    s.bos = min(max(p.cu[n], 0), p.Ttot);
    s.eos = min(max(p.cu[n + 1], s.bos), p.Ttot);
  } else {
    s.bos = n * p.T;
    s.eos = s.bos + p.T;
  }
  return s;
}

// The last sequence that starts at or before token t.
__device__ __forceinline__ int conv_seq(const ConvBwdProblem& p, int t) {
  if (!p.cu) return t / p.T;
  int lo = 0, hi = p.N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (min(max(p.cu[mid], 0), p.Ttot) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// x~ at the inputs' token t of sequence n (tokens before bos are the initial state's).
template <int W, typename E>
__device__ __forceinline__ void load_input(const ConvBwdProblem& p, int n, int bos, int t, int c0,
                                           float* v) {
  if (t >= bos) {
    Vec4<E>::load(static_cast<const E*>(p.x) + (long)t * p.C + c0, v);
  } else if (p.init) {
    Vec4<E>::load(static_cast<const E*>(p.init) +
                      ((long)n * (W - 1) + (W - 1) + (t - bos)) * p.C + c0, v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = 0.f;
  }
}

// du at token t of a sequence, from the window x~[t - (W - 1)] .. x~[t].
template <int W>
__device__ __forceinline__ void make_du(const float (*w)[kVec], const float* b,
                                        const float (*win)[kVec], const float* dy, bool silu,
                                        float* du) {
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    if (!silu) {
      du[v] = dy[v];
      continue;
    }
    float u = b[v];
#pragma unroll
    for (int i = 0; i < W; ++i) u = fmaf(w[i][v], win[i][v], u);
    const float s = sigmoid_f32(u);
    du[v] = dy[v] * (s * fmaf(u, 1.f - s, 1.f));
  }
}

template <int W, typename E>
__global__ __launch_bounds__(kThreads) void k_conv1d_bwd(ConvBwdProblem p) {
  const int c0 = (blockIdx.y * kThreads + threadIdx.x) * kVec;
  if (c0 >= p.C) return;
  const int t0 = blockIdx.x * p.tokens;
  const int t1 = min(t0 + p.tokens, p.Ttot);
  float w[W][kVec], b[kVec], dw[W][kVec], db[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    b[v] = p.bias ? p.bias[c0 + v] : 0.f;
    db[v] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      w[i][v] = p.weight[(long)(c0 + v) * W + i];
      dw[i][v] = 0.f;
    }
  }
  int n = conv_seq(p, t0);
  Span sp = conv_span(p, n);
  int t = t0;
  while (t < t1) {
    while (t >= sp.eos) {  // the next sequence that holds t
      if (++n >= p.N) break;
      sp = conv_span(p, n);
    }
    if (n >= p.N) break;  // tokens that no sequence has
    t = max(t, sp.bos);
    const int end = min(t1, sp.eos);            // this block's tokens of the sequence
    const int last = min(end + W - 1, sp.eos);  // and the ones whose du they need
    float win[W][kVec];  // x~[t - (W - 1)] .. x~[t]
    float du[W][kVec];   // du[t - (W - 1)] .. du[t]; zero before the first one needed
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i < W - 1) load_input<W, E>(p, n, sp.bos, t - (W - 1) + i, c0, win[i + 1]);
#pragma unroll
      for (int v = 0; v < kVec; ++v) du[i][v] = 0.f;
    }
    // the initial window sits one place late: a step moves it before it takes a token in
    const E* xs = static_cast<const E*>(p.x) + c0;
    const E* dys = static_cast<const E*>(p.dy) + c0;
    E* dxs = static_cast<E*>(p.dx) + c0;
    auto shift = [&]() {
#pragma unroll
      for (int i = 0; i + 1 < W; ++i) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          win[i][v] = win[i + 1][v];
          du[i][v] = du[i + 1][v];
        }
      }
    };
    auto take = [&](const typename Vec4<E>::raw& rx, const typename Vec4<E>::raw& rd, bool own) {
      float dy[kVec];
      Vec4<E>::wide(rx, win[W - 1]);
      Vec4<E>::wide(rd, dy);
      make_du<W>(w, b, win, dy, p.silu, du[W - 1]);
      if (own) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          db[v] += du[W - 1][v];
#pragma unroll
          for (int i = 0; i < W; ++i) dw[i][v] = fmaf(du[W - 1][v], win[i][v], dw[i][v]);
        }
      }
    };
    auto emit = [&](int o, bool tail) {  // dx[o] = sum_i w[i] du[o + W - 1 - i]
      float out[kVec];
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        out[v] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) out[v] = fmaf(w[i][v], du[W - 1 - i][v], out[v]);
      }
      const int j = o - (sp.eos - (W - 1));  // its place among the final state's entries
      if (tail && p.dfinal && j >= 0) {
        float f[kVec];
        Vec4<E>::load(static_cast<const E*>(p.dfinal) + ((long)n * (W - 1) + j) * p.C + c0, f);
#pragma unroll
        for (int v = 0; v < kVec; ++v) out[v] += f[v];
      }
      Vec4<E>::store(dxs + (long)o * p.C, out);
    };
    int tt = t;
    for (; tt < min(t + W - 1, end); ++tt) {  // the first tokens end no output of this block
      shift();
      take(Vec4<E>::load_raw(xs + (long)tt * p.C), Vec4<E>::load_raw(dys + (long)tt * p.C), true);
    }
    // whole groups, the next group's loads issued before this one computes
    const int groups = (end - tt) / kGroup;
    typename Vec4<E>::raw rx[kGroup], rd[kGroup];
    auto fetch = [&](int at) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        rx[i] = Vec4<E>::load_raw(xs + (long)(at + i) * p.C);
        rd[i] = Vec4<E>::load_raw(dys + (long)(at + i) * p.C);
      }
    };
    if (groups > 0) fetch(tt);
    for (int gi = 0; gi < groups; ++gi, tt += kGroup) {
      typename Vec4<E>::raw cx[kGroup], cd[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        cx[i] = rx[i];
        cd[i] = rd[i];
      }
      if (gi + 1 < groups) fetch(tt + kGroup);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        shift();
        take(cx[i], cd[i], true);
        emit(tt + i - (W - 1), false);  // before the sequence's last W - 1 tokens
      }
    }
    for (; tt < end + W - 1; ++tt) {
      shift();
      if (tt < last) {
        take(Vec4<E>::load_raw(xs + (long)tt * p.C), Vec4<E>::load_raw(dys + (long)tt * p.C),
             tt < end);
      } else {
#pragma unroll
        for (int v = 0; v < kVec; ++v) du[W - 1][v] = 0.f;
      }
      if (tt - (W - 1) >= t && tt - (W - 1) < end) emit(tt - (W - 1), true);
    }
    t = end;
  }
  float* part = p.part + (long)blockIdx.x * (W + 1) * p.C + c0;
#pragma unroll
  for (int i = 0; i < W; ++i) Vec4<float>::store(part + (long)i * p.C, dw[i]);
  Vec4<float>::store(part + (long)W * p.C, db);
}

// The gradient of the W - 1 inputs before each sequence: e < W - 1 of x~.
template <int W, typename E>
__global__ __launch_bounds__(kThreads) void k_conv1d_dinit(ConvBwdProblem p) {
  const long gid = (long)blockIdx.x * kThreads + threadIdx.x;
  const int groups = p.C / kVec;
  if (gid >= (long)p.N * groups) return;
  const int n = (int)(gid / groups);
  const int c0 = (int)(gid - (long)n * groups) * kVec;
  const Span sp = conv_span(p, n);
  const int len = sp.eos - sp.bos;
  float w[W][kVec], b[kVec], acc[W - 1][kVec], win[W][kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    b[v] = p.bias ? p.bias[c0 + v] : 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) w[i][v] = p.weight[(long)(c0 + v) * W + i];
#pragma unroll
    for (int e = 0; e < W - 1; ++e) acc[e][v] = 0.f;
  }
  // entry e is also the final state's entry e - len of a sequence shorter than W - 1
#pragma unroll
  for (int e = 0; e < W - 1; ++e)
    if (p.dfinal && e >= len)
      Vec4<E>::load(static_cast<const E*>(p.dfinal) + ((long)n * (W - 1) + e - len) * p.C + c0,
                    acc[e]);
#pragma unroll
  for (int i = 0; i + 1 < W; ++i)
    load_input<W, E>(p, n, sp.bos, sp.bos - (W - 1) + i, c0, win[i + 1]);
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
    if (t < len) {
      float dy[kVec], du[kVec];
#pragma unroll
      for (int i = 0; i + 1 < W; ++i)
#pragma unroll
        for (int v = 0; v < kVec; ++v) win[i][v] = win[i + 1][v];
      Vec4<E>::load(static_cast<const E*>(p.x) + (long)(sp.bos + t) * p.C + c0, win[W - 1]);
      Vec4<E>::load(static_cast<const E*>(p.dy) + (long)(sp.bos + t) * p.C + c0, dy);
      make_du<W>(w, b, win, dy, p.silu, du);
#pragma unroll
      for (int e = 0; e < W - 1; ++e)  // tap i = e - t
        if (e >= t) {
#pragma unroll
          for (int v = 0; v < kVec; ++v) acc[e][v] = fmaf(w[e >= t ? e - t : 0][v], du[v], acc[e][v]);
        }
    }
  }
#pragma unroll
  for (int e = 0; e < W - 1; ++e)
    Vec4<E>::store(static_cast<E*>(p.dinit) + ((long)n * (W - 1) + e) * p.C + c0, acc[e]);
}

// dw and dbias from the blocks' partial sums [blocks][W + 1][C].
__global__ __launch_bounds__(kColumnThreads) void k_conv1d_sum(const float* part, float* dweight,
                                                               float* dbias, int blocks, int C,
                                                               int W) {
  const int row = blockIdx.y;
  float* to = row < W ? dweight : dbias;
  if (!to) return;
  const int c = blockIdx.x * 64 + lane_id();
  const float r = column_sum(part + (long)row * C, (long)(W + 1) * C, blocks, c, C);
  if (threadIdx.x < 64 && c < C) to[row < W ? (long)c * W + row : c] = r;
}

template <int W, typename E>
hipError_t launch_w(const ConvBwdProblem& p, hipStream_t st) {
  if (p.blocks > 0)
    k_conv1d_bwd<W, E><<<dim3(p.blocks, (p.C / kVec + kThreads - 1) / kThreads), kThreads, 0,
                         st>>>(p);
  if (p.dinit && p.N > 0) {
    const long n = (long)p.N * (p.C / kVec);
    k_conv1d_dinit<W, E><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  }
  if (p.dweight || p.dbias)
    k_conv1d_sum<<<dim3((p.C + 63) / 64, W + 1), kColumnThreads, 0, st>>>(p.part, p.dweight, p.dbias,
                                                               p.blocks, p.C, W);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_e(const ConvBwdProblem& p, hipStream_t st) {
  if (p.W == 2) return launch_w<2, E>(p, st);
  if (p.W == 3) return launch_w<3, E>(p, st);
  return launch_w<4, E>(p, st);
}

}  // namespace

hipError_t launch_conv1d_bwd(const ConvBwdProblem& p, hipStream_t st) {
  return p.f32 ? launch_e<float>(p, st) : launch_e<bf16>(p, st);
}

}  // namespace gdn
