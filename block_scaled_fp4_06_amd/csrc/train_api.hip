// train_api.hip -- the C ABI of the operators around the linear layers (declared in
// include/nvfp4.h): residual norm, gated scan, AdamW.
//
// Every argument check happens here, before any HIP call, so a bad call returns its
// status synchronously and can be exercised on a machine without a GPU.
#include <math.h>
#include <string.h>

#include "nvfp4.h"
#include "train_launch.hpp"

namespace {

// Largest element offset of a strided tensor: far beyond any memory, and small enough that
// the kernels' 64-bit byte addresses never wrap.
constexpr int64_t kMaxSpan = (int64_t)1 << 60;
// Largest element count of one tensor.
constexpr int64_t kMaxElems = (int64_t)1 << 40;

bool is_dtype(int32_t d) { return d == NVFP4_DT_BF16 || d == NVFP4_DT_FP32; }
size_t size_of(int32_t d) { return d == NVFP4_DT_FP32 ? 4 : 2; }
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// a * b <= max for a, b >= 0, without forming a product that could overflow.
bool product_ok(int64_t a, int64_t b, int64_t max) { return a >= 0 && b >= 0 && (b == 0 || a <= max / b); }

// n steps of a stride >= 0 stay within kMaxSpan.
bool stride_ok(int64_t n, int64_t stride) {
  return stride >= 0 && (n <= 1 || stride <= kMaxSpan / (n - 1));
}

// rows x cols with row stride ld >= cols; one row has no stride to check.
bool rows_ok(int64_t rows, int64_t cols, int64_t ld) {
  return rows <= 1 || (ld >= cols && stride_ok(rows, ld));
}

nvfp4_status from_hip(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

// ---------------------------------------------------------------- residual norm
nvfp4_status check_norm_params(const nvfp4_norm_params *p) {
  if (!p) return NVFP4_ERR_NULL;
  if (p->rows < 0 || p->cols < 0 || p->cols > NVFP4_NORM_MAX_COLS ||
      !product_ok(p->rows, p->cols, kMaxElems) || p->rows > 0x7FFFFFFF)
    return NVFP4_ERR_SHAPE;
  if (p->gate_rows < 1 || p->rows % p->gate_rows || (p->rows > 0 && p->gate_rows > p->rows))
    return NVFP4_ERR_SHAPE;
  if (!is_dtype(p->x_dtype) || !is_dtype(p->z_dtype) || !is_dtype(p->weight_dtype) ||
      !is_dtype(p->gate_dtype))
    return NVFP4_ERR_UNSUPPORTED;
  if (p->x_dtype == NVFP4_DT_BF16 && p->z_dtype == NVFP4_DT_FP32) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

// ---------------------------------------------------------------- gated scan
bool scan_sizes_ok(int64_t batch, int64_t time, int64_t chan) {
  return batch >= 0 && time >= 0 && chan >= 0 && time <= 0x7FFFFFFF && chan <= 0x7FFFFFFF &&
         product_ok(batch, chan, kMaxElems) && product_ok(batch * chan, time, kMaxElems);
}

bool scan_strides_ok(const nvfp4_scan_args &a, int64_t sb, int64_t st) {
  return stride_ok(a.batch, sb) && stride_ok(a.time, st) && (a.time <= 1 || st >= a.chan);
}

// An output: besides, no two of its steps share memory.
bool scan_rows_apart(const nvfp4_scan_args &a, int64_t sb, int64_t st) {
  if (a.batch == 0 || a.time == 0) return true;
  const int64_t b = a.batch > 1 ? sb : 0, t = a.time > 1 ? st : 0;
  const int64_t near = b < t ? b : t, far = b < t ? t : b, n_near = b < t ? a.batch : a.time,
                n_far = b < t ? a.time : a.batch;
  return (n_near <= 1 || near >= a.chan) && (n_far <= 1 || far >= (n_near - 1) * near + a.chan);
}

// Whether dg and du share memory: where the ranges of addresses meet, only the same strides
// can keep them apart (the halves of one projection's gradient).
bool scan_grads_apart(const nvfp4_scan_args &a, const nvfp4_scan_grads &d, size_t size) {
  if (a.batch == 0 || a.time == 0) return true;
  const int64_t nb = a.batch - 1, nt = a.time - 1;
  const int64_t gb = nb ? d.dg_batch : 0, gt = nt ? d.dg_time : 0, ub = nb ? d.du_batch : 0, ut = nt ? d.du_time : 0;
  const uint64_t pg = (uint64_t)(uintptr_t)d.dg / size, pu = (uint64_t)(uintptr_t)d.du / size;
  const uint64_t eg = (uint64_t)(nb * gb + nt * gt + a.chan), eu = (uint64_t)(nb * ub + nt * ut + a.chan);
  if (pg <= pu ? pu - pg >= eg : pg - pu >= eu) return true;
  if (gb != ub || gt != ut) return false;
  // rows that lie apart: only the steps next to the distance can meet
  const bool batch_far = gb >= gt;
  const int64_t far = batch_far ? gb : gt, near = batch_far ? gt : gb, n_far = batch_far ? nb : nt,
                n_near = batch_far ? nt : nb;
  const int64_t dist = (int64_t)(pu - pg), i0 = far ? -dist / far : 0;
  for (int64_t i = i0 - 2; i <= i0 + 2; ++i) {
    if (i < -n_far || i > n_far) continue;
    const int64_t v = dist + i * far, j0 = near ? -v / near : 0;
    for (int64_t j = j0 - 2; j <= j0 + 2; ++j) {
      if (j < -n_near || j > n_near) continue;
      const int64_t w = v + j * near;
      if (w > -a.chan && w < a.chan) return false;
    }
  }
  return true;
}

nvfp4_status check_scan(const nvfp4_scan_args *a) {
  if (!a) return NVFP4_ERR_NULL;
  if (!scan_sizes_ok(a->batch, a->time, a->chan) || !scan_strides_ok(*a, a->g_batch, a->g_time) ||
      !scan_strides_ok(*a, a->u_batch, a->u_time) || !scan_strides_ok(*a, a->y_batch, a->y_time))
    return NVFP4_ERR_SHAPE;
  if (!is_dtype(a->dtype) || a->reserved) return NVFP4_ERR_UNSUPPORTED;
  if (a->batch && a->chan && a->time && (!a->g || !a->u || !a->y)) return NVFP4_ERR_NULL;
  const size_t e = size_of(a->dtype);
  if (!aligned(a->g, e) || !aligned(a->u, e) || !aligned(a->y, e) || !aligned(a->floor, 4) ||
      !aligned(a->h0, 4) || !aligned(a->h_last, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

nvfp4_status check_workspace(const void *ws, size_t bytes, size_t need) {
  if (need == 0) return NVFP4_OK;
  if (!ws || bytes < need) return NVFP4_ERR_WORKSPACE;
  return aligned(ws, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_residual_norm_forward(const nvfp4_norm_params *p,
                                         const nvfp4_norm_forward_args *a,
                                         nvfp4_stream_t stream) {
  const nvfp4_status st = check_norm_params(p);
  if (st != NVFP4_OK) return st;
  if (!a) return NVFP4_ERR_NULL;
  const bool branch = a->z != nullptr, next = a->next_weight != nullptr;
  if (!rows_ok(p->rows, p->cols, a->ld_x) || (branch && !rows_ok(p->rows, p->cols, a->ld_z)) ||
      (branch && !rows_ok(p->rows, p->cols, a->ld_x_out)) ||
      (next && !rows_ok(p->rows, p->cols, a->ld_h)) ||
      (a->gate && !rows_ok(p->gate_rows, p->cols, a->ld_gate)))
    return NVFP4_ERR_SHAPE;
  if (p->rows == 0 || p->cols == 0) return NVFP4_OK;  // nothing to write
  if (!a->x || (!branch && !next)) return NVFP4_ERR_NULL;
  if (branch ? (!a->post_weight || !a->x_out || !a->rstd_post)
             : (a->post_weight || a->gate || a->x_out || a->rstd_post))
    return NVFP4_ERR_NULL;
  if (next ? (!a->h || !a->rstd) : (a->h || a->rstd)) return NVFP4_ERR_NULL;
  if (a->x_out == a->x && p->rows > 1 && a->ld_x_out != a->ld_x) return NVFP4_ERR_UNSUPPORTED;
  const size_t ex = size_of(p->x_dtype), ez = size_of(p->z_dtype), ew = size_of(p->weight_dtype);
  if (!aligned(a->x, ex) || !aligned(a->x_out, ex) || !aligned(a->z, ez) || !aligned(a->h, ez) ||
      !aligned(a->post_weight, ew) || !aligned(a->next_weight, ew) ||
      !aligned(a->gate, size_of(p->gate_dtype)) || !aligned(a->rstd, 4) ||
      !aligned(a->rstd_post, 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4::NormForward n = {*p, *a};
  return from_hip(nvfp4::launch_norm_forward(n, reinterpret_cast<hipStream_t>(stream)));
}

size_t nvfp4_residual_norm_workspace_bytes(const nvfp4_norm_params *p) {
  if (check_norm_params(p) != NVFP4_OK || p->rows == 0 || p->cols == 0) return 0;
  return nvfp4::norm_workspace_bytes(*p);
}

nvfp4_status nvfp4_residual_norm_backward(const nvfp4_norm_params *p,
                                          const nvfp4_norm_backward_args *a, void *workspace,
                                          size_t workspace_bytes, nvfp4_stream_t stream) {
  const nvfp4_status st = check_norm_params(p);
  if (st != NVFP4_OK) return st;
  if (!a) return NVFP4_ERR_NULL;
  const int64_t r = p->rows, c = p->cols;
  const bool branch = a->z != nullptr, next = a->next_weight != nullptr;
  if (!rows_ok(r, c, a->ld_x_out) || !rows_ok(r, c, a->ld_dx) ||
      (a->dx_out && !rows_ok(r, c, a->ld_dx_out)) ||
      (branch && (!rows_ok(r, c, a->ld_z) || !rows_ok(r, c, a->ld_dz))) ||
      (next && !rows_ok(r, c, a->ld_dh)) ||
      (a->gate && !rows_ok(p->gate_rows, c, a->ld_gate)) ||
      (a->dgate && !rows_ok(p->gate_rows, c, a->ld_dgate)))
    return NVFP4_ERR_SHAPE;
  if (c == 0) return NVFP4_OK;
  if (r > 0) {
    if (!a->x_out || !a->dx || (!branch && !next)) return NVFP4_ERR_NULL;
    if (branch ? (!a->post_weight || !a->rstd_post || !a->dz)
               : (a->post_weight || a->gate || a->rstd_post || a->dz))
      return NVFP4_ERR_NULL;
    if (next ? (!a->rstd || !a->dh) : (a->rstd || a->dh)) return NVFP4_ERR_NULL;
    if ((a->dpost_weight && !branch) || (a->dnext_weight && !next) || (a->dgate && !a->gate))
      return NVFP4_ERR_NULL;
    if ((a->dx == a->dx_out && r > 1 && a->ld_dx != a->ld_dx_out) ||
        (branch && a->dz == a->dh && r > 1 && a->ld_dz != a->ld_dh))
      return NVFP4_ERR_UNSUPPORTED;
  }
  const size_t ex = size_of(p->x_dtype), ez = size_of(p->z_dtype), ew = size_of(p->weight_dtype),
               eg = size_of(p->gate_dtype);
  if (!aligned(a->x_out, ex) || !aligned(a->dx_out, ex) || !aligned(a->dx, ex) ||
      !aligned(a->z, ez) || !aligned(a->dh, ez) || !aligned(a->dz, ez) ||
      !aligned(a->post_weight, ew) || !aligned(a->next_weight, ew) ||
      !aligned(a->dpost_weight, ew) || !aligned(a->dnext_weight, ew) || !aligned(a->gate, eg) ||
      !aligned(a->dgate, eg) || !aligned(a->rstd, 4) || !aligned(a->rstd_post, 4))
    return NVFP4_ERR_ALIGN;
  const size_t need = r > 0 ? nvfp4::norm_workspace_bytes(*p) : 0;
  const nvfp4_status ws = check_workspace(workspace, workspace_bytes, need);
  if (ws != NVFP4_OK) return ws;
  const nvfp4::NormBackward n = {*p, *a, workspace};
  return from_hip(nvfp4::launch_norm_backward(n, reinterpret_cast<hipStream_t>(stream)));
}

size_t nvfp4_gated_scan_workspace_bytes(int64_t batch, int64_t time, int64_t chan,
                                        int32_t backward) {
  if (!scan_sizes_ok(batch, time, chan) || !batch || !time || !chan) return 0;
  return nvfp4::scan_workspace_bytes(batch, time, chan, backward != 0);
}

nvfp4_status nvfp4_gated_scan_forward(const nvfp4_scan_args *a, void *workspace,
                                      size_t workspace_bytes, nvfp4_stream_t stream) {
  const nvfp4_status st = check_scan(a);
  if (st != NVFP4_OK) return st;
  if (a->batch == 0 || a->chan == 0) return NVFP4_OK;
  const nvfp4_status ws =
      check_workspace(workspace, workspace_bytes,
                      nvfp4_gated_scan_workspace_bytes(a->batch, a->time, a->chan, 0));
  if (ws != NVFP4_OK) return ws;
  if (!scan_rows_apart(*a, a->y_batch, a->y_time)) return NVFP4_ERR_SHAPE;
  nvfp4::ScanLaunch s;
  memset(&s, 0, sizeof s);
  s.a = *a;
  s.ws = workspace;
  return from_hip(nvfp4::launch_scan_forward(s, reinterpret_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_gated_scan_backward(const nvfp4_scan_args *a, const nvfp4_scan_grads *d,
                                       void *workspace, size_t workspace_bytes,
                                       nvfp4_stream_t stream) {
  const nvfp4_status st = check_scan(a);
  if (st != NVFP4_OK) return st;
  if (!d) return NVFP4_ERR_NULL;
  if (!scan_strides_ok(*a, d->dy_batch, d->dy_time) || !scan_strides_ok(*a, d->dg_batch, d->dg_time) ||
      !scan_strides_ok(*a, d->du_batch, d->du_time))
    return NVFP4_ERR_SHAPE;
  if (d->dfloor && !a->floor) return NVFP4_ERR_NULL;
  if (a->chan == 0) return NVFP4_OK;
  if (a->batch && a->time && (!d->dy || !d->dg || !d->du)) return NVFP4_ERR_NULL;
  const size_t e = size_of(a->dtype);
  if (!aligned(d->dy, e) || !aligned(d->dg, e) || !aligned(d->du, e) || !aligned(d->dh_last, 4) ||
      !aligned(d->dh0, 4) || !aligned(d->dfloor, 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4_status ws =
      check_workspace(workspace, workspace_bytes,
                      nvfp4_gated_scan_workspace_bytes(a->batch, a->time, a->chan, 1));
  if (ws != NVFP4_OK) return ws;
  if (!scan_rows_apart(*a, d->dg_batch, d->dg_time) || !scan_rows_apart(*a, d->du_batch, d->du_time))
    return NVFP4_ERR_SHAPE;
  if (!scan_grads_apart(*a, *d, e)) return NVFP4_ERR_UNSUPPORTED;
  nvfp4::ScanLaunch s;
  memset(&s, 0, sizeof s);
  s.a = *a;
  s.d = *d;
  s.ws = workspace;
  return from_hip(nvfp4::launch_scan_backward(s, reinterpret_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------------- AdamW
size_t nvfp4_adamw_table_bytes(int64_t count) {
  if (count < 0 || count > ((int64_t)1 << 24)) return 0;
  return sizeof(nvfp4::AdamHeader) + (size_t)count * sizeof(nvfp4::AdamRow);
}

nvfp4_status nvfp4_adamw_table(const nvfp4_adamw_tensor *tensors, int64_t count,
                               int32_t state_bits, void *table, size_t table_bytes) {
  const size_t need = nvfp4_adamw_table_bytes(count);
  if (need == 0) return NVFP4_ERR_SHAPE;
  if (state_bits != 32 && state_bits != 8) return NVFP4_ERR_UNSUPPORTED;
  if ((count > 0 && !tensors) || !table) return NVFP4_ERR_NULL;
  if (table_bytes < need) return NVFP4_ERR_WORKSPACE;
  if (!aligned(table, 16)) return NVFP4_ERR_ALIGN;
  auto *h = static_cast<nvfp4::AdamHeader *>(table);
  auto *rows = reinterpret_cast<nvfp4::AdamRow *>(h + 1);
  h->magic = 0;   // an interrupted table is not one
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    const nvfp4_adamw_tensor &t = tensors[i];
    if (t.n < 0 || t.n > kMaxElems) return NVFP4_ERR_SHAPE;
    if (!is_dtype(t.param_dtype) || !is_dtype(t.grad_dtype) || !isfinite(t.weight_decay) ||
        (t.master && t.param_dtype != NVFP4_DT_BF16))
      return NVFP4_ERR_UNSUPPORTED;
    if (t.n > 0 && (!t.param || !t.exp_avg || !t.exp_avg_sq ||
                    (state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale))))
      return NVFP4_ERR_NULL;
    if (!aligned(t.param, size_of(t.param_dtype)) || !aligned(t.master, 4) ||
        !aligned(t.exp_avg, 16) || !aligned(t.exp_avg_sq, 16) || !aligned(t.exp_avg_scale, 4) ||
        !aligned(t.exp_avg_sq_scale, 4))
      return NVFP4_ERR_ALIGN;
    rows[i].t = t;
    rows[i].first_chunk = chunks;
    chunks += (t.n + nvfp4::kAdamChunk - 1) / nvfp4::kAdamChunk;
    if (chunks > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  }
  h->count = count;
  h->chunks = chunks;
  h->state_bits = state_bits;
  h->reserved = 0;
  h->magic = nvfp4::kAdamMagic;
  return NVFP4_OK;
}

nvfp4_status nvfp4_adamw_step(const void *table, const void *table_device,
                              const void *const *grads, const nvfp4_adamw_params *p,
                              nvfp4_stream_t stream) {
  if (!table || !p) return NVFP4_ERR_NULL;
  if (!aligned(table, 16) || !aligned(table_device, 16) || !aligned(p->grad_scale, 4))
    return NVFP4_ERR_ALIGN;
  const auto *h = static_cast<const nvfp4::AdamHeader *>(table);
  if (h->magic != nvfp4::kAdamMagic || p->reserved ||
      (p->stochastic_param != 0 && p->stochastic_param != 1))
    return NVFP4_ERR_UNSUPPORTED;
  if (p->step < 1 || p->step > 0xFFFFFFFFll) return NVFP4_ERR_SHAPE;
  // (a NaN fails these)
  if (!(p->beta1 >= 0.0 && p->beta1 < 1.0) || !(p->beta2 >= 0.0 && p->beta2 < 1.0) ||
      !(p->eps >= 0.0 && p->eps < 1e30) || !isfinite(p->lr) ||
      (h->state_bits == 8 && p->beta1 > NVFP4_ADAMW_MAX_BETA1_8))
    return NVFP4_ERR_UNSUPPORTED;
  if (h->chunks == 0) return NVFP4_OK;
  if (!table_device || !grads) return NVFP4_ERR_NULL;
  const auto *rows = reinterpret_cast<const nvfp4::AdamRow *>(h + 1);
  for (int64_t i = 0; i < h->count; ++i)
    if (!aligned(grads[i], size_of(rows[i].t.grad_dtype))) return NVFP4_ERR_ALIGN;
  nvfp4::AdamLaunch l;
  l.host = h;
  l.device = table_device;
  l.grads = grads;
  l.s.beta1 = (float)p->beta1;
  l.s.omb1 = (float)(1.0 - p->beta1);
  l.s.beta2 = (float)p->beta2;
  l.s.omb2 = (float)(1.0 - p->beta2);
  l.s.rate = (float)(p->lr / (1.0 - pow(p->beta1, (double)p->step)));
  l.s.root = (float)(1.0 / sqrt(1.0 - pow(p->beta2, (double)p->step)));
  l.s.eps = (float)p->eps;
  l.s.lr = p->lr;
  l.s.step = (uint32_t)p->step;
  l.s.k0 = (uint32_t)p->seed;
  l.s.k1 = (uint32_t)(p->seed >> 32);
  l.s.stochastic_param = p->stochastic_param;
  l.s.grad_scale = p->grad_scale;
  return from_hip(nvfp4::launch_adamw(l, reinterpret_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_adamw_moments(const uint8_t *exp_avg, const float *exp_avg_scale,
                                 const uint8_t *exp_avg_sq, const float *exp_avg_sq_scale,
                                 int64_t n, void *m_out, void *v_out, int32_t out_dtype,
                                 nvfp4_stream_t stream) {
  if (n < 0 || n > kMaxElems) return NVFP4_ERR_SHAPE;
  if (!is_dtype(out_dtype)) return NVFP4_ERR_UNSUPPORTED;
  if (n == 0) return NVFP4_OK;
  if (!exp_avg || !exp_avg_scale || !exp_avg_sq || !exp_avg_sq_scale || !m_out || !v_out)
    return NVFP4_ERR_NULL;
  if (!aligned(exp_avg, 16) || !aligned(exp_avg_sq, 16) || !aligned(m_out, 16) ||
      !aligned(v_out, 16) || !aligned(exp_avg_scale, 4) || !aligned(exp_avg_sq_scale, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4::AdamMoments l;
  l.m = exp_avg;
  l.v = exp_avg_sq;
  l.ms = exp_avg_scale;
  l.vs = exp_avg_sq_scale;
  l.n = n;
  l.m_out = m_out;
  l.v_out = v_out;
  l.out_f32 = out_dtype == NVFP4_DT_FP32;
  return from_hip(nvfp4::launch_adamw_moments(l, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
