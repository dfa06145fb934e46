// C ABI of the block norm (declared in include/gdn.h): host-side validation, workspace and dispatch.
// No allocation, no synchronisation.
#include <stdint.h>
#include <string.h>

#include "block_norm.h"
#include "gdn.h"

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

gdn_status check_block(const gdn_block_norm_desc* d, gdn::BlockNormProblem* p) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->rows < 0 || d->channels < 1 || !(d->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if ((d->dtype != GDN_F32 && d->dtype != GDN_BF16) ||
      (d->residual_dtype != GDN_F32 && d->residual_dtype != GDN_BF16))
    return GDN_ERR_INVALID_ARG;
  if ((d->post_norm != 0 && d->post_norm != 1) ||
      (d->activation != GDN_ACT_NONE && d->activation != GDN_ACT_SILU))
    return GDN_ERR_INVALID_ARG;
  memset(p, 0, sizeof(*p));
  p->sh = d->h_stride == 0 ? d->channels : d->h_stride;
  p->sg = d->gate_stride == 0 ? d->channels : d->gate_stride;
  if (p->sh < d->channels || p->sg < d->channels) return GDN_ERR_INVALID_ARG;
  // a bf16 stream of fp32 additions would lose what they add
  if (d->dtype == GDN_F32 && d->residual_dtype == GDN_BF16) return GDN_ERR_UNSUPPORTED;
  // rows are stepped over in 32 bits, by at most 2^14 at a time
  if (d->rows > (1 << 30) || d->channels > (1 << 20) || p->sh > ((int64_t)1 << 32) ||
      p->sg > ((int64_t)1 << 32))
    return GDN_ERR_UNSUPPORTED;
  p->rows = d->rows;
  p->C = d->channels;
  p->f32 = d->dtype == GDN_F32;
  p->residual_f32 = d->residual_dtype == GDN_F32;
  p->post = d->post_norm != 0;
  p->silu = d->activation == GDN_ACT_SILU;
  p->eps = d->eps;
  p->residual_scale = d->residual_scale;
  return GDN_OK;
}

// What belongs to the block's output is given with it alone.
bool parts_ok(const gdn::BlockNormProblem& p, const void* h, const void* gate, const float* w1,
              const float* scale) {
  return (h || (!gate && !w1 && !scale && !p.post)) && (p.post || !w1);
}

}  // namespace

extern "C" {

gdn_status gdn_block_norm_fwd(const gdn_block_norm_desc* d, const void* x, const void* h,
                              const void* gate, const float* post_weight, const float* scale,
                              const float* weight, void* x_out, void* y, float* post_rstd,
                              float* rstd, hipStream_t stream) {
  gdn::BlockNormProblem p;
  const gdn_status s = check_block(d, &p);
  if (s != GDN_OK) return s;
  if (p.rows == 0) return GDN_OK;
  if (!x || (!h && !y) || (h && !x_out) || !parts_ok(p, h, gate, post_weight, scale))
    return GDN_ERR_INVALID_ARG;
  const size_t e = p.f32 ? 4 : 2, r = p.residual_f32 ? 4 : 2;
  if (!aligned(x, r) || !aligned(x_out, r) || !aligned(h, e) || !aligned(gate, e) || !aligned(y, e))
    return GDN_ERR_INVALID_ARG;
  for (const float* q : {post_weight, scale, weight, (const float*)post_rstd, (const float*)rstd})
    if (!aligned(q, 4)) return GDN_ERR_INVALID_ARG;
  p.x = x;
  p.h = h;
  p.gate = gate;
  p.w1 = post_weight;
  p.scale = scale;
  p.w2 = weight;
  p.xo = h ? x_out : nullptr;
  p.y = y;
  p.rstd1 = post_rstd;
  p.rstd2 = rstd;
  return gdn::launch_block_norm_fwd(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_block_norm_bwd_workspace_size(const gdn_block_norm_desc* d, gdn_status* status) {
  gdn::BlockNormProblem p;
  const gdn_status s = check_block(d, &p);
  if (status) *status = s;
  if (s != GDN_OK) return 0;
  return ((size_t)gdn::block_norm_parts(p) * 3 * p.C * 4 + kAlign - 1) / kAlign * kAlign;
}

gdn_status gdn_block_norm_bwd(const gdn_block_norm_desc* d, const void* x, const void* h,
                              const void* gate, const float* post_weight, const float* scale,
                              const float* weight, const float* post_rstd, const float* rstd,
                              const void* dx_out, const void* dy, void* dx, void* dh, void* dgate,
                              float* dpost_weight, float* dscale, float* dweight,
                              hipStream_t stream) {
  gdn::BlockNormProblem p;
  const gdn_status s = check_block(d, &p);
  if (s != GDN_OK) return s;
  if (p.rows > 0 && (!x || !dx || (!dx_out && !dy) || (dy && !rstd) || (h && !dh) ||
                     (h && p.post && !post_rstd) || (gate && !dgate)))
    return GDN_ERR_INVALID_ARG;
  if (p.rows > 0 && !parts_ok(p, h, gate, post_weight, scale)) return GDN_ERR_INVALID_ARG;
  const size_t e = p.f32 ? 4 : 2, r = p.residual_f32 ? 4 : 2;
  for (const void* q : {x, dx_out, (const void*)dx})
    if (!aligned(q, r)) return GDN_ERR_INVALID_ARG;
  for (const void* q : {h, gate, dy, (const void*)dh, (const void*)dgate})
    if (!aligned(q, e)) return GDN_ERR_INVALID_ARG;
  for (const float* q : {post_weight, scale, weight, post_rstd, rstd, (const float*)dpost_weight,
                         (const float*)dscale, (const float*)dweight})
    if (!aligned(q, 4)) return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_block_norm_bwd_workspace_size(d, nullptr);
  if (need > 0 && (!d->workspace || d->workspace_bytes < need || !aligned(d->workspace, kAlign)))
    return GDN_ERR_WORKSPACE;
  p.x = x;
  p.h = h;
  p.gate = gate;
  p.w1 = post_weight;
  p.scale = scale;
  p.w2 = weight;
  p.rstd1 = const_cast<float*>(post_rstd);
  p.rstd2 = const_cast<float*>(rstd);
  p.dxo = dx_out;
  p.dy = dy;
  p.dx = dx;
  p.dh = dh;
  p.dgate = dgate;
  p.dw1 = dpost_weight;
  p.dscale = dscale;
  p.dw2 = dweight;
  p.part = static_cast<float*>(d->workspace);
  return gdn::launch_block_norm_bwd(p, stream) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
