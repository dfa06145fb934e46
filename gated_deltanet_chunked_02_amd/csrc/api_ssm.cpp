// C ABI of the selective state-space layer's calls (the scan, the convolution's backward, the
// group norm; declared in include/gdn.h): host-side validation,
// workspace layout and dispatch to the launchers.  No allocation, no synchronisation.
#include <stdint.h>
#include <string.h>

#include "gdn.h"
#include "norm.h"
#include "ssm.h"

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Row strides: 0 is a row after another; a given one is at least a row.
bool stride_ok(int64_t given, int64_t row, int64_t* out) {
  *out = given == 0 ? row : given;
  return given == 0 || (given >= row && given <= (int64_t)1 << 40);
}

constexpr int kLongestTile = 64;  // tokens that a chunk length is a multiple of, at most

// Descriptor checks shared by the entry points; fills the shape part of the problem, for a
// packed batch (cu_seqlens given) or a dense one.
gdn_status check_scan(const gdn_scan_desc* d, bool packed, gdn::ScanProblem* p) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->B < 1 || d->T < 0 || d->N < 0 || d->channels < 1 || d->groups < 1 || d->dstate < 1)
    return GDN_ERR_INVALID_ARG;
  if (d->channels % d->groups != 0) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (d->dt_softplus != 0 && d->dt_softplus != 1) return GDN_ERR_INVALID_ARG;
  if (packed ? d->B != 1 : (d->N != 0 && d->N != d->B)) return GDN_ERR_INVALID_ARG;
  memset(p, 0, sizeof(*p));
  const int64_t bcw = (int64_t)d->groups * d->dstate;
  if (!stride_ok(d->x_stride, d->channels, &p->sx) ||
      !stride_ok(d->dt_stride, d->channels, &p->sdt) ||
      !stride_ok(d->z_stride, d->channels, &p->sz) || !stride_ok(d->b_stride, bcw, &p->sb) ||
      !stride_ok(d->c_stride, bcw, &p->sc))
    return GDN_ERR_INVALID_ARG;
  if (d->dstate > 256) return GDN_ERR_UNSUPPORTED;
  const long long Ttot = (long long)d->B * d->T;
  p->N = packed ? d->N : d->B;
  if (Ttot > (1LL << 30) || p->N > (1 << 16) || d->channels > (1 << 20))
    return GDN_ERR_UNSUPPORTED;
  p->T = d->T;
  p->Ttot = (int)Ttot;
  p->C = d->channels;
  p->G = d->groups;
  p->S = d->dstate;
  p->per = p->C / p->G;
  p->nblk = (p->per + gdn::kScanLanes - 1) / gdn::kScanLanes;
  p->f32 = d->dtype == GDN_F32;
  p->softplus = d->dt_softplus != 0;
  return GDN_OK;
}

// Prompts reach a chunk's rows from its first token by 31-bit offsets (the single-token form has a
// 64-bit offset for each row): fills the tokens whose rows lie within 2 GiB of the first one's, for
// every tensor.  Sequences longer than that are split, into chunks of no fewer than 4 * 64 tokens.
gdn_status check_reach(bool packed, gdn::ScanProblem* p) {
  const int longest = packed ? p->Ttot : p->T;
  int64_t row = p->C;
  for (int64_t v : {p->sx, p->sdt, p->sz})
    if (v > row) row = v;
  int64_t reach = (((int64_t)1 << 31) - 1) / (row * (p->f32 ? 4 : 2)) - 1;
  if (reach < 1) reach = 1;  // a token's own row, whatever comes after it
  if (reach < longest && reach < 4 * kLongestTile) return GDN_ERR_UNSUPPORTED;
  if (reach > (1 << 30)) reach = 1 << 30;
  p->reach = (int)(reach < longest ? reach / kLongestTile * kLongestTile : reach);
  return GDN_OK;
}

// How the forward runs: states a lane and waves a workgroup (ns nw >= dstate), and the chunk
// length.  Few states a lane give many waves: with 16 states, 2 a lane take 268 us for 8 x 2048
// tokens of 4096 channels and 18.3 us for 129 tokens of 1000, 4 a lane 281 and 24.1 us.
//   * where the (sequence, 64-channel block) pairs are more than a third of the workgroups that run
//     at once, whole sequences are quicker than chunks, which cost a second pass: 3 x 2048 tokens of
//     4096 channels take 191 us whole and 243 us in two chunks each, 4 x 2048 of 2560 channels as
//     long whole and 171 us in three each.  A packed batch is split at twice its mean length, so that
//     one long sequence does not run alone;
//   * below that the sequences are split into as many chunks as run at once, which LDS bounds
//     (k_scan: 16 KB and 8 KB a wave of a CU's 160 KB): 1 x 8192 tokens of 4096 channels take 247 us
//     in 8 chunks, 257 us in 32, 325 us in 10 (a second round), and about 700 us whole;
//   * a chunk has at least 32 tokens, which pay for the two more launches: 400 tokens of 1000 channels
//     take 18.9 us in chunks of 32, 21.7 us of 16, 22.8 us of 64 and 38.5 us of 128.  Splitting saves
//     7 us of 25 on 200 tokens; on 129 it saves 1 us, less than a host needs for the launches.
constexpr int kUnits = 256;  // CUs
constexpr int kMinChunk = 32;
constexpr int kMinSplit = 192;

void plan_fwd(gdn::ScanProblem* p, bool packed) {
  const long long blocks = (long long)p->G * p->nblk;
  p->ns = p->S <= 16 ? 2 : p->S <= 32 ? 4 : p->S <= 128 ? 8 : 16;
  p->nw = p->ns == 2 ? 2 : p->ns == 16 ? 16 : 8;
  while (p->nw * p->ns < p->S) p->nw *= 2;
  p->Sp = p->ns * p->nw;
  p->Lc = gdn::kScanNoSplit;
  if (p->N > 0 && p->Ttot > 0) {
    const long long longest = packed ? p->Ttot : p->T;
    long long L = longest;
    const long long fill = kUnits * (160 / (16 + 8 * p->nw)) / blocks;
    if (fill >= 3 * p->N) {
      const long long each = packed ? fill : fill / p->N;
      L = (longest + each - 1) / each;
    } else if (packed) {
      L = 2LL * ((p->Ttot + p->N - 1) / p->N);
    }
    L = (L + gdn::kScanTile - 1) / gdn::kScanTile * gdn::kScanTile;
    if (L < kMinChunk) L = kMinChunk;
    // a chunk's rows are reached with 31-bit offsets
    if (L > p->reach) L = p->reach;
    if ((2 * L <= longest && longest >= kMinSplit) || longest > p->reach) p->Lc = (int)L;
  }
  p->slots = packed ? p->Ttot / p->Lc + p->N
                    : p->N * (int)(p->T > p->Lc ? ((long long)p->T + p->Lc - 1) / p->Lc : 1);
}

// A launch has fewer than 2^32 threads; so have the passes over B and C rows, over the chunks'
// channel blocks and over the states, and the gradient's sums (launch_scan_bwd), in workgroups of
// 1024 threads.
bool grids_ok(const gdn::ScanProblem& p, bool backward) {
  const long long most = 1LL << 32, rows = (long long)p.Ttot * p.G * 2 * p.Sp;
  const long long sums = backward ? (p.C + 63LL) / 64 * (p.S + 2) + (rows + 1023) / 1024 : 0;
  return rows < most - 256 && (long long)p.slots * p.G * p.nblk * 64 * p.nw < most &&
         (long long)p.N * p.S * 256 < most && sums * 1024 < most;
}

struct ScanLayout {
  size_t bc, hst, dsum, total;
};

ScanLayout scan_layout(const gdn::ScanProblem& p) {
  ScanLayout L;
  size_t o = 0;
  L.bc = o;
  o += align_up((size_t)p.Ttot * p.G * 2 * p.Sp * 4);
  L.hst = o;
  const bool split = p.Lc != gdn::kScanNoSplit;
  if (split) o += align_up((size_t)p.slots * p.S * p.C * 4);
  L.dsum = o;
  if (split) o += align_up((size_t)p.slots * p.C * 4);
  L.total = o;
  return L;
}

// The backward's plan: chunks of kBwdChunk tokens and blocks of up to 32 states (eight waves of 4:
// with blocks of 16 the sums carried from block to block leave LDS for one workgroup of four
// waves a CU, and 4 x 2048 tokens of 4096 channels and 64 states took 4950 us).  A packed batch has
// more slots than sequences unless it has fewer tokens than a chunk, so it is composed even when no
// sequence is long.
// Chunks are halved, down to 16 tokens, while they give fewer waves than SIMDs: forward and
// backward of 257 tokens of 2 x 768 channels take 53.8 us (64-token chunks: 71), of 1000 tokens of
// 1024 channels 74 us in chunks of 32 (64: 81, 16: 83), of 1000 tokens of 2048 channels 101 us in
// chunks of 64 (32: 108).
constexpr int kBwdMin = 16;
constexpr int kBwdFill = 1024;

void plan_bwd(gdn::ScanProblem* p, bool packed) {
  p->ns = 4;
  p->nw = p->S <= 4 ? 1 : p->S <= 8 ? 2 : p->S <= 16 ? 4 : 8;
  const int block = p->ns * p->nw;
  p->Sp = (p->S + block - 1) / block * block;
  p->Lc = gdn::kBwdChunk;
  while (p->Lc > kBwdMin && (long long)(p->Ttot / p->Lc) * p->G * p->nblk * p->nw < kBwdFill)
    p->Lc /= 2;
  p->slots = p->N == 0 ? 0
             : packed  ? p->Ttot / p->Lc + p->N
                       : p->N * (p->T > p->Lc ? (p->T + p->Lc - 1) / p->Lc : 1);
}

struct BwdLayout {
  size_t bc, hst, gst, dsum, bcp, dAp, dvp, total;
};

BwdLayout bwd_layout(const gdn::ScanProblem& p) {
  BwdLayout L;
  size_t o = 0;
  const size_t rows = align_up((size_t)p.Ttot * p.G * 2 * p.Sp * 4);
  const size_t states = align_up((size_t)p.slots * p.S * p.C * 4);
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.bc = take(rows);
  L.hst = take(states);
  L.gst = take(states);
  L.dsum = take((size_t)p.slots * p.C * 4);
  L.bcp = take((size_t)p.nblk * p.Ttot * p.G * 2 * p.Sp * 4);
  L.dAp = take(states);
  L.dvp = take((size_t)p.slots * 2 * p.C * 4);
  L.total = o;
  return L;
}

// Token blocks of the convolution's backward: the longest power of two up to 256 tokens that
// still gives 1024 workgroups (a block costs W - 1 tokens more of reading and a row of partial
// sums), at least 8.
void plan_conv_bwd(gdn::ConvBwdProblem* p) {
  const long long slabs = (p->C / 4 + 255) / 256;
  p->tokens = 256;
  while (p->tokens > 8 && (p->Ttot + p->tokens - 1LL) / p->tokens * slabs < 1024)
    p->tokens >>= 1;
  p->blocks = (p->Ttot + p->tokens - 1) / p->tokens;
}

gdn_status check_conv_bwd(const gdn_conv_desc* d, bool packed, gdn::ConvBwdProblem* p) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->B < 1 || d->T < 0 || d->N < 0 || d->channels < 1) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (d->activation != GDN_ACT_NONE && d->activation != GDN_ACT_SILU) return GDN_ERR_INVALID_ARG;
  if (packed ? d->B != 1 : (d->N != 0 && d->N != d->B)) return GDN_ERR_INVALID_ARG;
  if (d->width < 2 || d->width > 4 || d->channels % 8 != 0) return GDN_ERR_UNSUPPORTED;
  const long long Ttot = (long long)d->B * d->T;
  if (Ttot > (1LL << 30) || (long long)d->channels * 8 > (1LL << 30) || d->N > (1 << 24))
    return GDN_ERR_UNSUPPORTED;
  // the grid's y axis counts blocks of 1024 channels, in 16 bits
  if ((d->channels + 1023LL) / 1024 > 65535) return GDN_ERR_UNSUPPORTED;
  memset(p, 0, sizeof(*p));
  p->T = d->T;
  p->Ttot = (int)Ttot;
  p->N = packed ? d->N : d->B;
  p->C = d->channels;
  p->W = d->width;
  p->f32 = d->dtype == GDN_F32;
  p->silu = d->activation == GDN_ACT_SILU;
  plan_conv_bwd(p);
  if ((long long)p->N * (p->C / 4) >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_norm(const gdn_norm_desc* d, gdn::NormProblem* p) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->samples < 0 || d->positions < 0 || d->channels < 1 || d->groups < 1 ||
      d->channels % d->groups != 0 || !(d->eps >= 0.f))
    return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (d->activation != GDN_ACT_NONE && d->activation != GDN_ACT_SILU) return GDN_ERR_INVALID_ARG;
  // the kernels step over positions in 32 bits, by less than 2^20 at a time
  if (d->positions > (1 << 30)) return GDN_ERR_UNSUPPORTED;
  // a workgroup of 1024 threads for each (sample, group), except for rows whose groups fit the
  // lanes' registers at any alignment
  const bool rows = d->positions == 1 && d->channels / d->groups <= 1024;
  if ((rows ? d->samples > (1 << 30) : (long long)d->samples * d->groups > (1 << 21)) ||
      d->channels > (1 << 20))
    return GDN_ERR_UNSUPPORTED;
  memset(p, 0, sizeof(*p));
  p->N = d->samples;
  p->P = d->positions;
  p->C = d->channels;
  p->G = d->groups;
  p->cpg = p->C / p->G;
  p->f32 = d->dtype == GDN_F32;
  p->silu = d->activation == GDN_ACT_SILU;
  p->eps = d->eps;
  return GDN_OK;
}

gdn_status norm_space(const gdn_norm_desc* d, bool backward, gdn::NormProblem* p) {
  const size_t need = gdn::norm_workspace(*p, backward);
  if (need > 0 && (!d->workspace || d->workspace_bytes < need || !aligned(d->workspace, kAlign)))
    return GDN_ERR_WORKSPACE;
  p->ws = static_cast<float*>(d->workspace);
  return GDN_OK;
}

bool looks_packed(const gdn_scan_desc* d) { return d && d->N != 0 && d->N != d->B; }

}  // namespace

extern "C" {

size_t gdn_selective_scan_workspace_size(const gdn_scan_desc* d, gdn_status* status) {
  gdn::ScanProblem p;
  const bool packed = looks_packed(d);
  gdn_status s = check_scan(d, packed, &p);
  if (s == GDN_OK) s = check_reach(packed, &p);
  if (status) *status = s;
  if (s != GDN_OK) return 0;
  plan_fwd(&p, packed);
  if (!grids_ok(p, false)) {
    if (status) *status = GDN_ERR_UNSUPPORTED;
    return 0;
  }
  size_t need = scan_layout(p).total;
  if (!packed && d->B == 1) {  // one sequence may also come as a packed batch of one
    gdn::ScanProblem q = p;
    q.N = 1;
    plan_fwd(&q, true);
    const size_t alt = scan_layout(q).total;
    if (alt > need) need = alt;
  }
  return need;
}

gdn_status gdn_selective_scan_fwd(const gdn_scan_desc* d, const void* x, const void* dt,
                                  const float* A, const void* Bm, const void* Cm,
                                  const float* D, const void* z, const float* dt_bias,
                                  const float* h0, const int32_t* cu_seqlens, void* y, float* ht,
                                  hipStream_t stream) {
  gdn::ScanProblem p;
  gdn_status s = check_scan(d, cu_seqlens != nullptr, &p);
  if (s == GDN_OK) s = check_reach(cu_seqlens != nullptr, &p);
  if (s != GDN_OK) return s;
  if (!A || (p.Ttot > 0 && (!x || !dt || !Bm || !Cm || !y))) return GDN_ERR_INVALID_ARG;
  const size_t e = p.f32 ? 4 : 2;
  if (!aligned(x, e) || !aligned(dt, e) || !aligned(z, e) || !aligned(Bm, e) ||
      !aligned(Cm, e) || !aligned(y, e) || !aligned(A, 4) || !aligned(D, 4) ||
      !aligned(dt_bias, 4) || !aligned(h0, 4) || !aligned(ht, 4) || !aligned(cu_seqlens, 4))
    return GDN_ERR_INVALID_ARG;
  if (p.N == 0) return GDN_OK;
  plan_fwd(&p, cu_seqlens != nullptr);
  if (!grids_ok(p, false)) return GDN_ERR_UNSUPPORTED;
  const ScanLayout L = scan_layout(p);
  if (L.total > 0 && (!d->workspace || d->workspace_bytes < L.total ||
                      !aligned(d->workspace, kAlign)))
    return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(d->workspace);
  p.bc = reinterpret_cast<float*>(ws + L.bc);
  p.hst = reinterpret_cast<float*>(ws + L.hst);
  p.dsum = reinterpret_cast<float*>(ws + L.dsum);
  p.x = x;
  p.dt = dt;
  p.z = z;
  p.Bm = Bm;
  p.Cm = Cm;
  p.A = A;
  p.D = D;
  p.bias = dt_bias;
  p.h0 = h0;
  p.cu = cu_seqlens;
  p.y = y;
  p.ht = ht;
  return gdn::launch_scan_fwd(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_selective_scan_bwd_workspace_size(const gdn_scan_desc* d, gdn_status* status) {
  gdn::ScanProblem p;
  const bool packed = looks_packed(d);
  gdn_status s = check_scan(d, packed, &p);
  if (s == GDN_OK) s = check_reach(packed, &p);
  if (status) *status = s;
  if (s != GDN_OK) return 0;
  // one dense sequence may also come as a packed batch of one, which never has fewer slots
  const bool one = !packed && d->B == 1;
  if (one) p.N = 1;
  plan_bwd(&p, packed || one);
  if (!grids_ok(p, true)) {
    if (status) *status = GDN_ERR_UNSUPPORTED;
    return 0;
  }
  return bwd_layout(p).total;
}

gdn_status gdn_selective_scan_bwd(const gdn_scan_desc* d, const void* x, const void* dt,
                                  const float* A, const void* Bm, const void* Cm,
                                  const float* D, const void* z, const float* dt_bias,
                                  const float* h0, const int32_t* cu_seqlens, const void* dy,
                                  const float* dht, void* dx, void* ddt, float* dA, void* dB,
                                  void* dC, float* dD, void* dz, float* ddt_bias, float* dh0,
                                  hipStream_t stream) {
  gdn::ScanProblem p;
  gdn_status s = check_scan(d, cu_seqlens != nullptr, &p);
  if (s == GDN_OK) s = check_reach(cu_seqlens != nullptr, &p);
  if (s != GDN_OK) return s;
  if (!A || !dA) return GDN_ERR_INVALID_ARG;
  if (p.Ttot > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || !dB || !dC || (z && !dz)))
    return GDN_ERR_INVALID_ARG;
  const size_t e = p.f32 ? 4 : 2;
  for (const void* q : {x, dt, Bm, Cm, z, dy, (const void*)dx, (const void*)ddt, (const void*)dB,
                        (const void*)dC, (const void*)dz})
    if (!aligned(q, e)) return GDN_ERR_INVALID_ARG;
  for (const void* q : {(const void*)A, (const void*)D, (const void*)dt_bias, (const void*)h0,
                        (const void*)cu_seqlens, (const void*)dht, (const void*)dA,
                        (const void*)dD, (const void*)ddt_bias, (const void*)dh0})
    if (!aligned(q, 4)) return GDN_ERR_INVALID_ARG;
  plan_bwd(&p, cu_seqlens != nullptr);
  if (!grids_ok(p, true)) return GDN_ERR_UNSUPPORTED;
  const BwdLayout L = bwd_layout(p);
  if (L.total > 0 && (!d->workspace || d->workspace_bytes < L.total ||
                      !aligned(d->workspace, kAlign)))
    return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(d->workspace);
  auto at = [ws](size_t o) { return reinterpret_cast<float*>(ws + o); };
  p.bc = at(L.bc);
  p.hst = at(L.hst);
  p.dsum = at(L.dsum);
  p.x = x;
  p.dt = dt;
  p.z = z;
  p.Bm = Bm;
  p.Cm = Cm;
  p.A = A;
  p.D = D;
  p.bias = dt_bias;
  p.h0 = h0;
  p.cu = cu_seqlens;
  gdn::ScanBwd b;
  b.dy = dy;
  b.dht = dht;
  b.gst = at(L.gst);
  b.bcp = at(L.bcp);
  b.dAp = at(L.dAp);
  b.dvp = at(L.dvp);
  b.dx = dx;
  b.ddt = ddt;
  b.dz = dz;
  b.dB = dB;
  b.dC = dC;
  b.dA = dA;
  b.dD = dD;
  b.dbias = ddt_bias;
  b.dh0 = dh0;
  return gdn::launch_scan_bwd(p, b, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

gdn_status gdn_selective_state_update(const gdn_scan_desc* d, float* state, const void* x,
                                      const void* dt, const float* A, const void* Bm,
                                      const void* Cm, const float* D, const void* z,
                                      const float* dt_bias, const int32_t* cache_indices,
                                      const int32_t* out_indices, void* y, hipStream_t stream) {
  gdn::ScanProblem p;
  const gdn_status s = check_scan(d, false, &p);
  if (s != GDN_OK) return s;
  if (d->T != 1 || d->state_lines < 1) return GDN_ERR_INVALID_ARG;
  if (!state || !x || !dt || !A || !Bm || !Cm || !y) return GDN_ERR_INVALID_ARG;
  const size_t e = p.f32 ? 4 : 2;
  if (!aligned(state, 4) || !aligned(x, e) || !aligned(dt, e) || !aligned(z, e) ||
      !aligned(Bm, e) || !aligned(Cm, e) || !aligned(y, e) || !aligned(A, 4) ||
      !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(cache_indices, 4) ||
      !aligned(out_indices, 4))
    return GDN_ERR_INVALID_ARG;
  // one workgroup for each 16 channels of a sequence, at most
  if ((long long)d->B * ((p.C + 15) / 16) >= (1LL << 24)) return GDN_ERR_UNSUPPORTED;
  gdn::ScanStepProblem q;
  q.B = d->B;
  q.C = p.C;
  q.G = p.G;
  q.S = p.S;
  q.per = p.per;
  q.lines = d->state_lines;
  q.f32 = p.f32;
  q.softplus = p.softplus;
  q.vec4 = p.S % 4 == 0 && aligned(state, 16) && aligned(A, 16);
  q.wide = q.vec4 && p.sb % 4 == 0 && p.sc % 4 == 0 && aligned(Bm, 4 * e) && aligned(Cm, 4 * e);
  q.state = state;
  q.x = x;
  q.dt = dt;
  q.z = z;
  q.Bm = Bm;
  q.Cm = Cm;
  q.A = A;
  q.D = D;
  q.bias = dt_bias;
  q.read = cache_indices;
  q.write = out_indices;
  q.sx = p.sx;
  q.sdt = p.sdt;
  q.sz = p.sz;
  q.sb = p.sb;
  q.sc = p.sc;
  q.y = y;
  return gdn::launch_scan_step(q, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_causal_conv1d_bwd_workspace_size(const gdn_conv_desc* d, gdn_status* status) {
  gdn::ConvBwdProblem p;
  const gdn_status s = check_conv_bwd(d, d && d->N != 0 && d->N != d->B, &p);
  if (status) *status = s;
  return s == GDN_OK ? align_up((size_t)p.blocks * (p.W + 1) * p.C * 4) : 0;
}

gdn_status gdn_causal_conv1d_bwd(const gdn_conv_desc* d, const void* x, const float* weight,
                                 const float* bias, const void* initial,
                                 const int32_t* cu_seqlens, const void* dy, const void* dfinal,
                                 void* dx, float* dweight, float* dbias, void* dinitial,
                                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
  gdn::ConvBwdProblem p;
  const gdn_status s = check_conv_bwd(d, cu_seqlens != nullptr, &p);
  if (s != GDN_OK) return s;
  if (!weight || (p.Ttot > 0 && (!x || !dy || !dx))) return GDN_ERR_INVALID_ARG;
  for (const void* q : {x, initial, dy, dfinal, (const void*)dx, (const void*)dinitial})
    if (!aligned(q, 16)) return GDN_ERR_INVALID_ARG;
  for (const void* q : {(const void*)weight, (const void*)bias, (const void*)cu_seqlens,
                        (const void*)dweight, (const void*)dbias})
    if (!aligned(q, 4)) return GDN_ERR_INVALID_ARG;
  if (p.N == 0) {
    p.blocks = 0;  // no sequence has a token: the parameters' gradients are zero
    dinitial = nullptr;
  }
  const size_t need = align_up((size_t)p.blocks * (p.W + 1) * p.C * 4);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, kAlign)))
    return GDN_ERR_WORKSPACE;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.init = initial;
  p.cu = cu_seqlens;
  p.dy = dy;
  p.dfinal = dfinal;
  p.dx = dx;
  p.dweight = dweight;
  p.dbias = dbias;
  p.dinit = dinitial;
  p.part = static_cast<float*>(workspace);
  return gdn::launch_conv1d_bwd(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_group_norm_workspace_size(const gdn_norm_desc* d, int32_t backward,
                                     gdn_status* status) {
  gdn::NormProblem p;
  const gdn_status s = check_norm(d, &p);
  if (status) *status = s;
  if (s != GDN_OK || p.N == 0 || p.P == 0) return 0;
  return gdn::norm_workspace(p, backward != 0);
}

gdn_status gdn_group_norm_fwd(const gdn_norm_desc* d, const void* x, const float* weight,
                              const float* bias, const void* gate, void* y, float* mean,
                              float* rstd, hipStream_t stream) {
  gdn::NormProblem p;
  gdn_status s = check_norm(d, &p);
  if (s != GDN_OK) return s;
  if (p.N == 0) return GDN_OK;
  if (p.P > 0 && (!x || !y)) return GDN_ERR_INVALID_ARG;
  const size_t e = p.f32 ? 4 : 2;
  if (!aligned(x, e) || !aligned(gate, e) || !aligned(y, e) || !aligned(weight, 4) ||
      !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return GDN_ERR_INVALID_ARG;
  if (p.P == 0) {
    p.mean = mean;
    p.rstd = rstd;
    return gdn::launch_norm_no_stats(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  }
  s = norm_space(d, false, &p);
  if (s != GDN_OK) return s;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.gate = gate;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  return gdn::launch_norm_fwd(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

gdn_status gdn_group_norm_bwd(const gdn_norm_desc* d, const void* x, const float* weight,
                              const float* bias, const void* gate, const float* mean,
                              const float* rstd, const void* dy, void* dx, float* dweight,
                              float* dbias, void* dgate, hipStream_t stream) {
  gdn::NormProblem p;
  gdn_status s = check_norm(d, &p);
  if (s != GDN_OK) return s;
  const bool empty = p.N == 0 || p.P == 0;
  if (!empty && (!x || !mean || !rstd || !dy || !dx || (gate && !dgate)))
    return GDN_ERR_INVALID_ARG;
  const size_t e = p.f32 ? 4 : 2;
  for (const void* q : {x, gate, dy, (const void*)dx, (const void*)dgate})
    if (!aligned(q, e)) return GDN_ERR_INVALID_ARG;
  for (const void* q : {(const void*)weight, (const void*)bias, (const void*)mean,
                        (const void*)rstd, (const void*)dweight, (const void*)dbias})
    if (!aligned(q, 4)) return GDN_ERR_INVALID_ARG;
  p.dweight = dweight;
  p.dbias = dbias;
  if (empty)
    return gdn::launch_norm_no_params(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
  s = norm_space(d, true, &p);
  if (s != GDN_OK) return s;
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.gate = gate;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.dy = dy;
  p.dx = dx;
  p.dgate = dgate;
  return gdn::launch_norm_bwd(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
