// The gradient of the causal depthwise convolution.  With x~ a sequence's inputs behind the W - 1
// before it, u[t] = bias + sum_i w[i] x~[t + i] and y = act(u),
//
//   du[t]    = dy[t] act'(u[t])
//   dx~[e]   = sum_i w[i] du[e - i]  (over the tokens the sequence has), plus the gradient of the
//              final state where x~[e] is one of its last W - 1 entries
//   dw[i]    = sum_t du[t] x~[t + i],   dbias = sum_t du[t]
//
// One thread per 8 channels and a block of tokens, walked in order with the last W - 1 inputs
// and du in registers: x and dy are read once (but for the W - 1 tokens after a block, whose du
// its last outputs need), dx is written once.  Each block leaves its share of dw and dbias as a
// partial sum; a second kernel adds them in order.
#include "gdn_device.h"
#include "norm.h"
#include "ssm_device.h"
#include "vec8.h"

namespace gdn {

namespace {

constexpr int kVec = 8;
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
    Vec8<E>::load(static_cast<const E*>(p.x) + (long)t * p.C + c0, v);
  } else if (p.init) {
    Vec8<E>::load(static_cast<const E*>(p.init) +
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
    // the initial window sits one place late: the first step moves it
    for (int tt = t; tt < end + W - 1; ++tt) {
#pragma unroll
      for (int i = 0; i + 1 < W; ++i) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          win[i][v] = win[i + 1][v];
          du[i][v] = du[i + 1][v];
        }
      }
      if (tt < last) {
        float dy[kVec];
        Vec8<E>::load(static_cast<const E*>(p.x) + (long)tt * p.C + c0, win[W - 1]);
        Vec8<E>::load(static_cast<const E*>(p.dy) + (long)tt * p.C + c0, dy);
        make_du<W>(w, b, win, dy, p.silu, du[W - 1]);
        if (tt < end) {
#pragma unroll
          for (int v = 0; v < kVec; ++v) {
            db[v] += du[W - 1][v];
#pragma unroll
            for (int i = 0; i < W; ++i) dw[i][v] = fmaf(du[W - 1][v], win[i][v], dw[i][v]);
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < kVec; ++v) du[W - 1][v] = 0.f;
      }
      const int o = tt - (W - 1);  // dx[o] = sum_i w[i] du[o + W - 1 - i]
      if (o >= t && o < end) {
        float out[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          out[v] = 0.f;
#pragma unroll
          for (int i = 0; i < W; ++i) out[v] = fmaf(w[i][v], du[W - 1 - i][v], out[v]);
        }
        const int j = o - (sp.eos - (W - 1));  // its place among the final state's entries
        if (p.dfinal && j >= 0) {
          float f[kVec];
          Vec8<E>::load(static_cast<const E*>(p.dfinal) + ((long)n * (W - 1) + j) * p.C + c0, f);
#pragma unroll
          for (int v = 0; v < kVec; ++v) out[v] += f[v];
        }
        Vec8<E>::store(static_cast<E*>(p.dx) + (long)o * p.C + c0, out);
      }
    }
    t = end;
  }
  float* part = p.part + (long)blockIdx.x * (W + 1) * p.C + c0;
#pragma unroll
  for (int i = 0; i < W; ++i) Vec8<float>::store(part + (long)i * p.C, dw[i]);
  Vec8<float>::store(part + (long)W * p.C, db);
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
      Vec8<E>::load(static_cast<const E*>(p.dfinal) + ((long)n * (W - 1) + e - len) * p.C + c0,
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
      Vec8<E>::load(static_cast<const E*>(p.x) + (long)(sp.bos + t) * p.C + c0, win[W - 1]);
      Vec8<E>::load(static_cast<const E*>(p.dy) + (long)(sp.bos + t) * p.C + c0, dy);
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
    Vec8<E>::store(static_cast<E*>(p.dinit) + ((long)n * (W - 1) + e) * p.C + c0, acc[e]);
}

// dw and dbias from the blocks' partial sums: a workgroup takes 64 channels of one row, its four
// waves every fourth block.
__global__ __launch_bounds__(256) void k_conv1d_sum(const float* part, float* dweight,
                                                    float* dbias, int blocks, int C, int W) {
  __shared__ float s[4][64];
  const int lane = lane_id(), w = wave_id();
  const int c = blockIdx.x * 64 + lane, row = blockIdx.y;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < C) {
    const float* q = part + (long)row * C + c;
    const long step = (long)(W + 1) * C;
    int i = w;
    for (; i + 12 < blocks; i += 16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += q[(long)(i + 4 * j) * step];
    }
    for (; i < blocks; i += 4) v[0] += q[(long)i * step];
  }
  s[w][lane] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (w == 0 && c < C) {
    const float r = (s[0][lane] + s[1][lane]) + (s[2][lane] + s[3][lane]);
    if (row < W) {
      if (dweight) dweight[(long)c * W + row] = r;
    } else if (dbias) {
      dbias[c] = r;
    }
  }
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
    k_conv1d_sum<<<dim3((p.C + 63) / 64, W + 1), 256, 0, st>>>(p.part, p.dweight, p.dbias,
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
