// C ABI of the linear attention calls (declared in include/gdn.h): host-side validation, workspace
// layout and dispatch to the launchers.  No allocation, no synchronisation.
#include <stdint.h>
#include <string.h>

#include "gdn.h"
#include "linear.h"
#include "ssm.h"

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows are read 16 bytes at a time and reached from a chunk's first one by 31-bit byte offsets, so
// they are less than 2^23 elements apart (64 rows of 4 bytes).
constexpr int64_t kFar = (int64_t)1 << 23;

gdn_status check_row(int64_t given, int64_t row, int e, int64_t* out) {
  *out = given == 0 ? row : given;
  if (*out < row || (*out * e) % 16 != 0) return GDN_ERR_INVALID_ARG;
  return *out < kFar ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// Descriptor checks shared by the entry points; fills the shape part of the problem.
gdn_status check_linear(const gdn_linear_desc* d, bool packed, gdn::LinearProblem* p) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->B < 1 || d->T < 0 || d->N < 0 || d->H < 1 || d->Hg < 1 || d->H % d->Hg != 0 ||
      d->Dk < 1 || d->Dv < 1)
    return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (d->head_decay != 0 && d->head_decay != 1) return GDN_ERR_INVALID_ARG;
  if (packed ? d->B != 1 : (d->N != 0 && d->N != d->B)) return GDN_ERR_INVALID_ARG;
  if (d->Dk % 8 != 0 || d->Dv % 8 != 0 || d->Dk > 256 || d->Dv > 256) return GDN_ERR_UNSUPPORTED;
  memset(p, 0, sizeof(*p));
  const long long Ttot = (long long)d->B * d->T;
  p->N = packed ? d->N : d->B;
  if (Ttot > (1LL << 30) || p->N > (1 << 16) || (int64_t)d->H * d->Dk >= kFar ||
      (int64_t)d->H * d->Dv >= kFar)
    return GDN_ERR_UNSUPPORTED;
  const int e = d->dtype == GDN_F32 ? 4 : 2;
  const int64_t kw = (int64_t)d->Hg * d->Dk, vw = (int64_t)d->H * d->Dv;
  gdn_status s = check_row(d->q_stride, kw, e, &p->sq);
  if (s == GDN_OK) s = check_row(d->k_stride, kw, e, &p->sk);
  if (s == GDN_OK) s = check_row(d->v_stride, vw, e, &p->sv);
  if (s != GDN_OK) return s;
  p->T = d->T;
  p->Ttot = (int)Ttot;
  p->H = d->H;
  p->Hg = d->Hg;
  p->Dk = d->Dk;
  p->Dv = d->Dv;
  p->f32 = d->dtype == GDN_F32;
  p->head_decay = d->head_decay != 0;
  p->scale = d->scale;
  return GDN_OK;
}

// Segment length.  Short of heads (times the value slabs), sequences are cut into as many segments as make
// `fill` workgroups, two chunks long at least (16384 tokens of 32 heads: 16 segments, where 8 took a fifth
// more); but not those of fewer than six chunks, whose few steps take less than two more launches.
//
// Segments cost a pass over their states, so that a dense batch is cut where `least` of them fit and is run
// whole elsewhere.  Forward, 2048 tokens in bf16, whole and cut: 128 (sequence, head) pairs 147 and 119 us,
// 160 (three segments) 147 and 138, 180 (two) 147 and 179, 224 157 and 193, 256 165 and 208; 1024 tokens in
// fp32: 128 pairs 191 and 154, 192 193 and 263.  Gradient: 96 (two) 454 and 296, 128 479 and 321.
//
// A packed batch's lengths are on the device.  Whole, it takes as long as its longest sequence; cut, about
// as long whatever they are.  So it is always cut, with `fill` up to `most` pairs and at twice its mean length
// beyond, where that is as good.  Forward, 12454 tokens in 8 sequences, whole, by `fill` and by the mean: lengths
// to 2048, 256 pairs 147, 187 and 224 us, 288 161, 223 and 223, 320 169, 255 and 229; one of 8192,
// 256 pairs 523, 196 and 319, 288 538, 214 and 323, 320 548, 243 and 327.  Gradient: the same lengths, 288 pairs
// 485, 498 and 497, 320 648, 664 and 663; with one of 8192 1797, 642 and 972, 1821, 753 and 1033 (at 512 pairs
// both give the same length).
struct Cut {
  int fill, least, most;  // most: no more than twice fill, so that two sequences' heads are within it
};
constexpr Cut kFwdCut = {512, 3, 288}, kBwdCut = {256, 2, 512};

int slots_of(const gdn::LinearProblem& p, bool packed) {
  return p.N == 0 ? 0
         : packed ? p.Ttot / p.Lc + p.N
                  : p.N * (int)(p.T > p.Lc ? ((long long)p.T + p.Lc - 1) / p.Lc : 1);
}

void plan(gdn::LinearProblem* p, bool packed, int slabs, const Cut& cut) {
  p->Lc = gdn::kScanNoSplit;
  const int C = gdn::linear_chunk(p->f32);
  const long long longest = packed ? p->Ttot : p->T;
  if (p->N > 0 && longest >= 6 * C) {
    const long long units = (long long)p->H * slabs;
    const bool unlike = packed && p->N > 1;  // a packed batch of one has one length
    long long L = longest;
    if (unlike && units * p->N > cut.most) {
      L = 2LL * ((p->Ttot + p->N - 1) / p->N);
    } else {
      const long long each = unlike ? cut.fill / units : cut.fill / (units * p->N);
      if (unlike || each >= cut.least) L = (longest + each - 1) / each;
    }
    if (L < 2 * C) L = 2 * C;
    L = (L + gdn::kLinearChunk - 1) / gdn::kLinearChunk * gdn::kLinearChunk;
    if (L < longest) p->Lc = (int)L;
  }
  p->slots = slots_of(*p, packed);
}

int slabs_of(const gdn::LinearProblem& p) { return (p.Dv + gdn::kLinearSlab - 1) / gdn::kLinearSlab; }

// A few segments make their start states themselves, each from all before it, and no launch composes them.
// Every one of those is a read that the next waits for, and all of them together grow with the square of the
// segments.  So no more than this many values of a head's states at the segments' ends (128 x 128: 512
// tokens of 32 heads, four segments, 28 us and not 33; 1024 and 2048, eight segments, 35 and not 37, and
// 56 either way), and no more segments than 16 (64 x 64: 2048 tokens of 32 heads, 16 segments, 29 us and not
// 31; 4096 of 16, 32 segments, 35 and 34 composed; 32 x 32, 16384 tokens of a head, 128 segments, 67 and 42).
constexpr long long kMostJoined = 8 * 128 * 128, kMostSegments = 16;

bool joins(const gdn::LinearProblem& p, bool packed) {
  if (p.Lc == gdn::kScanNoSplit) return false;
  const long long most = packed ? p.Ttot / p.Lc + 1 : ((long long)p.T + p.Lc - 1) / p.Lc;
  return most <= kMostSegments && most * p.Dk * p.Dv <= kMostJoined;
}

void plan_fwd(gdn::LinearProblem* p, bool packed) { plan(p, packed, slabs_of(*p), kFwdCut); }
void plan_bwd(gdn::LinearProblem* p, bool packed) {
  plan(p, packed, 1, kBwdCut);
  // a segment holds whole spans between the states kept for the gradient, or is one
  const int span = gdn::linear_anchor(*p) * gdn::linear_chunk(p->f32);
  if (p->Lc != gdn::kScanNoSplit && p->Lc > span) {
    p->Lc = (p->Lc + span - 1) / span * span;
    if (p->Lc >= (packed ? p->Ttot : p->T)) p->Lc = gdn::kScanNoSplit;
    p->slots = slots_of(*p, packed);
  }
}

// A launch has fewer than 2^32 threads: segments' heads and slabs in workgroups of up to 512, there and
// back; the composition's four values a thread, likewise; the shared heads' sums, four values of dq and
// of dk a thread and another row of the grid.
bool grids_ok(const gdn::LinearProblem& p) {
  const long long most = 1LL << 32, cell = ((long long)p.Dk * p.Dv / 4 + 255) / 256 * 256;
  return (long long)p.slots * p.H * slabs_of(p) * 512 * 2 < most &&
         (long long)p.N * p.H * cell * 2 < most &&
         ((long long)p.Ttot * p.Hg * p.Dk / 4 + p.H * 16LL + 1024) * 3 < most;
}

struct FwdLayout {
  size_t states, sums, total;
};

FwdLayout fwd_layout(const gdn::LinearProblem& p) {
  FwdLayout L = {};
  if (p.Lc == gdn::kScanNoSplit) return L;
  const size_t heads = (size_t)p.slots * p.H;
  L.sums = align_up(heads * p.Dk * p.Dv * 4);
  L.total = L.sums + align_up(heads * 4);
  return L;
}

struct BwdLayout {
  size_t states, sums, grads, anchors, a, part, dgp, total;
  int every;
};

BwdLayout bwd_layout(const gdn::LinearProblem& p, bool packed) {
  BwdLayout L = {};
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  const size_t heads = (size_t)p.slots * p.H;
  // the states kept for the gradient: at some chunks' ends, or a shorter segment's
  const int C = gdn::linear_chunk(p.f32);
  L.every = p.Lc < gdn::linear_anchor(p) * C ? p.Lc / C : gdn::linear_anchor(p);
  const size_t span = (size_t)L.every * C;
  const size_t anchors = p.Ttot == 0 ? 0
                         : packed    ? (size_t)p.Ttot / span + p.N
                                     : (size_t)p.N * (((size_t)p.T + span - 1) / span);
  const bool split = p.Lc != gdn::kScanNoSplit;
  L.states = take(split ? heads * p.Dk * p.Dv * 4 : 0);
  L.sums = take(split ? heads * 4 : 0);
  L.grads = take(split ? heads * p.Dk * p.Dv * 4 : 0);
  L.anchors = take(anchors * p.H * gdn::linear_tile(p.Dk) * gdn::linear_tile(p.Dv) * 4);
  L.a = take((size_t)p.Ttot * p.H * 8);
  L.part = take(p.H != p.Hg ? (size_t)p.Ttot * p.H * p.Dk * 8 : 0);
  L.dgp = take(p.head_decay ? heads * 8 : 0);
  L.total = o;
  return L;
}

bool looks_packed(const gdn_linear_desc* d) { return d && d->N != 0 && d->N != d->B; }

gdn_status check_bwd(const gdn_linear_desc* d, bool packed, gdn::LinearProblem* p) {
  gdn_status s = check_linear(d, packed, p);
  if (s != GDN_OK) return s;
  if (d->Dk > 128 || d->Dv > 128) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

bool space_ok(const gdn_linear_desc* d, size_t need) {
  return need == 0 || (d->workspace && d->workspace_bytes >= need && aligned(d->workspace, kAlign));
}

}  // namespace

extern "C" {

size_t gdn_linear_attn_workspace_size(const gdn_linear_desc* d, gdn_status* status) {
  gdn::LinearProblem p;
  const bool packed = looks_packed(d);
  gdn_status s = check_linear(d, packed, &p);
  size_t need = 0;
  if (s == GDN_OK) {
    plan_fwd(&p, packed);
    if (!grids_ok(p)) s = GDN_ERR_UNSUPPORTED;
    need = fwd_layout(p).total;
    if (!packed && d->B == 1) {  // one sequence may also come as a packed batch of one
      plan_fwd(&p, true);
      const size_t alt = fwd_layout(p).total;
      if (alt > need) need = alt;
    }
  }
  if (status) *status = s;
  return s == GDN_OK ? need : 0;
}

gdn_status gdn_linear_attn_fwd(const gdn_linear_desc* d, const void* q, const void* k,
                               const void* v, const float* g, const float* h0,
                               const int32_t* cu_seqlens, void* o, float* ht,
                               hipStream_t stream) {
  gdn::LinearProblem p;
  const gdn_status s = check_linear(d, cu_seqlens != nullptr, &p);
  if (s != GDN_OK) return s;
  if (p.Ttot > 0 && (!q || !k || !v || !g || !o)) return GDN_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, (const void*)o, (const void*)h0, (const void*)ht})
    if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  if (!aligned(g, 4) || !aligned(cu_seqlens, 4)) return GDN_ERR_INVALID_ARG;
  if (p.N == 0) return GDN_OK;
  plan_fwd(&p, cu_seqlens != nullptr);
  if (!grids_ok(p)) return GDN_ERR_UNSUPPORTED;
  const FwdLayout L = fwd_layout(p);
  if (!space_ok(d, L.total)) return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(d->workspace);
  p.states = reinterpret_cast<float*>(ws + L.states);
  p.sums = reinterpret_cast<float*>(ws + L.sums);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.h0 = h0;
  p.cu = cu_seqlens;
  p.o = o;
  p.ht = ht;
  p.direct = !h0 || h0 != ht;
  p.join = p.direct && joins(p, cu_seqlens != nullptr);
  return gdn::launch_linear_fwd(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_linear_attn_bwd_workspace_size(const gdn_linear_desc* d, gdn_status* status) {
  gdn::LinearProblem p;
  const bool packed = looks_packed(d);
  gdn_status s = check_bwd(d, packed, &p);
  size_t need = 0;
  if (s == GDN_OK) {
    plan_bwd(&p, packed);
    if (!grids_ok(p)) s = GDN_ERR_UNSUPPORTED;
    need = bwd_layout(p, packed).total;
    if (!packed && d->B == 1) {
      plan_bwd(&p, true);
      const size_t alt = bwd_layout(p, true).total;
      if (alt > need) need = alt;
    }
  }
  if (status) *status = s;
  return s == GDN_OK ? need : 0;
}

gdn_status gdn_linear_attn_bwd(const gdn_linear_desc* d, const void* q, const void* k,
                               const void* v, const float* g, const float* h0,
                               const int32_t* cu_seqlens, const void* dout, const float* dht,
                               void* dq, void* dk, void* dv, float* dg, float* dh0,
                               hipStream_t stream) {
  const bool packed = cu_seqlens != nullptr;
  gdn::LinearProblem p;
  const gdn_status s = check_bwd(d, packed, &p);
  if (s != GDN_OK) return s;
  if (p.Ttot > 0 && (!q || !k || !v || !g || !dout || !dq || !dk || !dv)) return GDN_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, dout, (const void*)h0, (const void*)dht, (const void*)dq,
                        (const void*)dk, (const void*)dv, (const void*)dh0})
    if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  for (const void* x : {(const void*)g, (const void*)cu_seqlens, (const void*)dg})
    if (!aligned(x, 4)) return GDN_ERR_INVALID_ARG;
  plan_bwd(&p, packed);
  if (!grids_ok(p)) return GDN_ERR_UNSUPPORTED;
  const BwdLayout L = bwd_layout(p, packed);
  if (!space_ok(d, L.total)) return GDN_ERR_WORKSPACE;
  char* ws = static_cast<char*>(d->workspace);
  auto at = [ws](size_t o) { return reinterpret_cast<float*>(ws + o); };
  p.states = at(L.states);
  p.sums = at(L.sums);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.h0 = h0;
  p.cu = cu_seqlens;
  p.direct = true;  // this call writes no final states
  gdn::LinearBwd b;
  b.dout = dout;
  b.dht = dht;
  b.dq = dq;
  b.dk = dk;
  b.dv = dv;
  b.dg = dg;
  b.dh0 = dh0;
  b.direct = !dht || dht != dh0;
  b.grads = at(L.grads);
  b.anchors = at(L.anchors);
  b.a = reinterpret_cast<double*>(ws + L.a);
  b.every = L.every;
  b.part = at(L.part);
  b.dgp = reinterpret_cast<double*>(ws + L.dgp);
  return gdn::launch_linear_bwd(p, b, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

gdn_status gdn_linear_state_update(const gdn_linear_desc* d, float* state, const void* q,
                                   const void* k, const void* v, const float* g,
                                   const int32_t* cache_indices, const int32_t* out_indices,
                                   void* o, hipStream_t stream) {
  gdn::LinearProblem p;
  const gdn_status s = check_linear(d, false, &p);
  if (s != GDN_OK) return s;
  if (d->T != 1 || d->state_lines < 1) return GDN_ERR_INVALID_ARG;
  if (!state || !q || !k || !v || !g || !o) return GDN_ERR_INVALID_ARG;
  for (const void* x : {(const void*)state, q, k, v, (const void*)o})
    if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  if (!aligned(g, 4) || !aligned(cache_indices, 4) || !aligned(out_indices, 4))
    return GDN_ERR_INVALID_ARG;
  // a workgroup of 256 threads for each 32 columns of a head
  if ((long long)d->B * p.H * ((p.Dv + 31) / 32) >= (1LL << 24)) return GDN_ERR_UNSUPPORTED;
  gdn::LinearStepProblem x;
  x.B = d->B;
  x.H = p.H;
  x.Hg = p.Hg;
  x.Dk = p.Dk;
  x.Dv = p.Dv;
  x.lines = d->state_lines;
  x.f32 = p.f32;
  x.head_decay = p.head_decay;
  x.scale = p.scale;
  x.sq = p.sq;
  x.sk = p.sk;
  x.sv = p.sv;
  x.state = state;
  x.q = q;
  x.k = k;
  x.v = v;
  x.g = g;
  x.read = cache_indices;
  x.write = out_indices;
  x.o = o;
  return gdn::launch_linear_step(x, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
