// atlas_ops.cu -- C-ABI entry points of the layer operators: argument checks, strides and
// the choice between wide (16-byte) and element-wise accesses.  Every computation happens
// in norm.cu, layernorm_*.cu, conv_*.cu, scan_*.cu and glr_*.cu.
#include "atlas_ops.h"

#include <algorithm>
#include <initializer_list>

#include "ops.h"

using namespace atlas;

namespace {

bool float_type(int t) { return t == ATLAS_F32 || t == ATLAS_BF16 || t == ATLAS_F16; }
int size_of(int t) { return t == ATLAS_F32 ? 4 : t == ATLAS_E4M3 ? 1 : 2; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
cudaStream_t stream_of(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// ------------------------------------------------------------------ norm

int check_norm(const atlas_norm_cfg* c) {
  if (!c || c->rows < 0 || c->d < 1 || c->group < 0) return ATLAS_ERR_INVALID;
  if (!float_type(c->dtype) || !float_type(c->r_dtype) || !float_type(c->w_dtype))
    return ATLAS_ERR_INVALID;
  if (!float_type(c->out_dtype) && c->out_dtype != ATLAS_E4M3) return ATLAS_ERR_INVALID;
  if (!(c->eps >= 0.f && c->eps < 3e38f)) return ATLAS_ERR_INVALID;
  if (c->x_stride < 0 || c->r_stride < 0 || c->y_stride < 0) return ATLAS_ERR_INVALID;
  // rows that are written do not overlap
  if ((c->r_stride && c->r_stride < c->d) || (c->y_stride && c->y_stride < c->d))
    return ATLAS_ERR_INVALID;
  if (c->d > ATLAS_NORM_MAX_D) return ATLAS_ERR_UNSUPPORTED;
  return ATLAS_OK;
}

int check_layernorm(const atlas_norm_cfg* c) {
  const int rc = check_norm(c);
  if (rc != ATLAS_OK) return rc;
  return c->eps > 0.f ? ATLAS_OK : ATLAS_ERR_INVALID;
}

void norm_args(const atlas_norm_cfg* c, NormArgs& a) {
  a.rows = c->rows;
  a.d = c->d;
  a.dt = c->dtype;
  a.rt = c->r_dtype;
  a.wt = c->w_dtype;
  a.ot = c->out_dtype;
  a.group = c->group >= c->d ? 0 : c->group;
  a.eps = c->eps;
  a.sx = c->x_stride ? c->x_stride : c->d;
  a.sr = c->r_stride ? c->r_stride : c->d;
  a.sy = c->y_stride ? c->y_stride : c->d;
}
NormArgs norm_args(const atlas_norm_cfg* c) {
  NormArgs a = {};
  norm_args(c, a);
  return a;
}
LayerNormArgs layernorm_args(const atlas_norm_cfg* c) {
  LayerNormArgs a = {};
  norm_args(c, a);
  return a;
}

// -------------------------------------------------------------- sequences

int check_seq(int B, int L, const int* slot, int n_slots) {
  if (B < 0 || L < 0) return ATLAS_ERR_INVALID;
  if (slot && n_slots < 1) return ATLAS_ERR_INVALID;
  return ATLAS_OK;
}

// Strides 0, 0 ask for the contiguous layout of `width` elements a token.
void strides(long& sb, long& st, long width, int L) {
  if (sb == 0 && st == 0) {
    st = width;
    sb = width * L;
  }
}

struct Dim {
  long n, stride;
};
// Whether the elements of a tensor that is written lie apart: blocks of `width` neighbours, along dimensions
// nested in any order, each with a stride of at least what those inside it span.
bool apart(std::initializer_list<Dim> dims, long width) {
  Dim d[3];
  int k = 0;
  for (const Dim& v : dims) {
    if (v.n == 0) return true;  // none
    if (v.n > 1) d[k++] = v;
  }
  std::sort(d, d + k, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  long span = width;
  for (int i = 0; i < k; ++i) {
    if (d[i].stride < span) return false;
    span += (d[i].n - 1) * d[i].stride;
  }
  return true;
}
bool apart(long sb, long st, long width, int B, int L, bool packed) {
  return apart({{packed ? 1 : B, sb}, {L, st}}, width);
}

// ------------------------------------------------------------------ conv

int check_conv(const atlas_conv_cfg* c) {
  if (!c) return ATLAS_ERR_INVALID;
  const int rc = check_seq(c->B, c->L, c->slot, c->n_slots);
  if (rc != ATLAS_OK) return rc;
  if (c->C < 1 || c->W < 1 || c->head_dim < 0) return ATLAS_ERR_INVALID;
  if (c->act != ATLAS_ACT_NONE && c->act != ATLAS_ACT_SILU) return ATLAS_ERR_INVALID;
  if (!float_type(c->dtype) || !float_type(c->w_dtype)) return ATLAS_ERR_INVALID;
  if (c->head_dim && c->C % c->head_dim) return ATLAS_ERR_INVALID;
  if (c->x_batch_stride < 0 || c->x_token_stride < 0 || c->y_batch_stride < 0 ||
      c->y_token_stride < 0 || c->y_head_stride < 0)
    return ATLAS_ERR_INVALID;
  if (c->W > ATLAS_CONV_MAX_W) return ATLAS_ERR_UNSUPPORTED;
  return ATLAS_OK;
}

ConvArgs conv_args(const atlas_conv_cfg* c) {
  ConvArgs a = {};
  a.s = SeqArgs{c->seq_start, c->slot, c->carry, c->status_dev, c->B, c->L, c->n_slots};
  a.C = c->C;
  a.W = c->W;
  a.act = c->act;
  a.dt = c->dtype;
  a.wt = c->w_dtype;
  a.hd = c->head_dim;
  a.xb = c->x_batch_stride;
  a.xt = c->x_token_stride;
  strides(a.xb, a.xt, c->C, c->L);
  a.yb = c->y_batch_stride;
  a.yt = c->y_token_stride;
  a.yh = c->y_head_stride;
  if (!a.hd) {
    strides(a.yb, a.yt, c->C, c->L);
  } else if (a.yb == 0 && a.yt == 0 && a.yh == 0) {
    a.yt = a.hd;
    a.yh = (long)a.hd * c->L;
    a.yb = (long)c->C * c->L;
  }
  return a;
}

bool conv_y_apart(const ConvArgs& a) {
  if (!a.hd) return apart(a.yb, a.yt, a.C, a.s.B, a.s.L, a.s.start);
  return apart({{a.s.start ? 1 : a.s.B, a.yb}, {a.s.L, a.yt}, {a.C / a.hd, a.yh}}, a.hd);
}

// Whether rows, heads and states keep `bytes` (a power of two) aligned.
bool conv_wide(const ConvArgs& a, const void* x, const void* y, const void* s0, const void* s1, int bytes) {
  const int v = bytes / size_of(a.dt), n = bytes;
  return aligned(x, n) && aligned(y, n) && aligned(s0, n) && aligned(s1, n) && a.C % v == 0 &&
         a.xb % v == 0 && a.xt % v == 0 && a.yb % v == 0 && a.yt % v == 0 && a.yh % v == 0 &&
         (!a.hd || a.hd % v == 0);
}

// ------------------------------------------------------------------ scan

int check_scan(const atlas_scan_cfg* c) {
  if (!c) return ATLAS_ERR_INVALID;
  const int rc = check_seq(c->B, c->L, c->slot, c->n_slots);
  if (rc != ATLAS_OK) return rc;
  if (c->D < 1 || c->N < 1 || c->G < 1 || c->D % c->G) return ATLAS_ERR_INVALID;
  if (!float_type(c->dtype)) return ATLAS_ERR_INVALID;
  const long s[] = {c->x_batch_stride, c->x_token_stride, c->dt_batch_stride, c->dt_token_stride,
                    c->z_batch_stride, c->z_token_stride, c->y_batch_stride, c->y_token_stride,
                    c->b_batch_stride, c->b_token_stride, c->c_batch_stride, c->c_token_stride};
  for (long v : s)
    if (v < 0) return ATLAS_ERR_INVALID;
  if (c->N > ATLAS_SCAN_MAX_N || c->B > 65535) return ATLAS_ERR_UNSUPPORTED;
  return ATLAS_OK;
}

ScanArgs scan_args(const atlas_scan_cfg* c) {
  ScanArgs a = {};
  a.s = SeqArgs{c->seq_start, c->slot, c->carry, c->status_dev, c->B, c->L, c->n_slots};
  a.D = c->D;
  a.N = c->N;
  a.G = c->G;
  a.type = c->dtype;
  a.softplus = c->softplus != 0;
  a.xb = c->x_batch_stride, a.xt = c->x_token_stride;
  a.tb = c->dt_batch_stride, a.tt = c->dt_token_stride;
  a.zb = c->z_batch_stride, a.zt = c->z_token_stride;
  a.yb = c->y_batch_stride, a.yt = c->y_token_stride;
  a.bb = c->b_batch_stride, a.bt = c->b_token_stride;
  a.cb = c->c_batch_stride, a.ct = c->c_token_stride;
  strides(a.xb, a.xt, c->D, c->L);
  strides(a.tb, a.tt, c->D, c->L);
  strides(a.zb, a.zt, c->D, c->L);
  strides(a.yb, a.yt, c->D, c->L);
  strides(a.bb, a.bt, (long)c->G * c->N, c->L);
  strides(a.cb, a.ct, (long)c->G * c->N, c->L);
  return a;
}

bool scan_wide(const ScanArgs& a) {
  const int v = 16 / size_of(a.type);
  const long s[] = {a.xb, a.xt, a.tb, a.tt, a.zb, a.zt, a.yb, a.yt, a.D / a.G};
  for (long x : s)
    if (x % v) return false;
  const void* p[] = {a.x, a.dt, a.z, a.y, a.dy, a.dx, a.ddt, a.dz};
  for (const void* q : p)
    if (!aligned(q, 16)) return false;
  return true;
}

bool scan_wide_n(const ScanArgs& a) {
  const int v = 16 / size_of(a.type);
  return a.N % v == 0 && a.bb % v == 0 && a.bt % v == 0 && a.cb % v == 0 && a.ct % v == 0 &&
         aligned(a.Bm, 16) && aligned(a.Cm, 16);
}

// ------------------------------------------------------------------ glr

int check_glr(const atlas_glr_cfg* c) {
  if (!c) return ATLAS_ERR_INVALID;
  const int rc = check_seq(c->B, c->L, c->slot, c->n_slots);
  if (rc != ATLAS_OK) return rc;
  if (c->D < 1 || !float_type(c->dtype) || !(c->c > 0.f && c->c < 3e38f)) return ATLAS_ERR_INVALID;
  const long s[] = {c->x_batch_stride, c->x_token_stride, c->r_batch_stride, c->r_token_stride,
                    c->i_batch_stride, c->i_token_stride, c->z_batch_stride, c->z_token_stride,
                    c->y_batch_stride, c->y_token_stride};
  for (long v : s)
    if (v < 0) return ATLAS_ERR_INVALID;
  if (c->D > 0x7FFFFF00) return ATLAS_ERR_UNSUPPORTED;
  return ATLAS_OK;
}

GlrArgs glr_args(const atlas_glr_cfg* c) {
  GlrArgs a = {};
  a.s = SeqArgs{c->seq_start, c->slot, c->carry, c->status_dev, c->B, c->L, c->n_slots};
  a.D = c->D;
  a.type = c->dtype;
  a.c = c->c;
  a.xb = c->x_batch_stride, a.xt = c->x_token_stride;
  a.rbs = c->r_batch_stride, a.rt = c->r_token_stride;
  a.ibs = c->i_batch_stride, a.it = c->i_token_stride;
  a.zb = c->z_batch_stride, a.zt = c->z_token_stride;
  a.yb = c->y_batch_stride, a.yt = c->y_token_stride;
  strides(a.xb, a.xt, c->D, c->L);
  strides(a.rbs, a.rt, c->D, c->L);
  strides(a.ibs, a.it, c->D, c->L);
  strides(a.zb, a.zt, c->D, c->L);
  strides(a.yb, a.yt, c->D, c->L);
  return a;
}
int check_glr(const atlas_glr_cfg* c, GlrArgs& a) {
  const int rc = check_glr(c);
  if (rc != ATLAS_OK) return rc;
  a = glr_args(c);
  return glr_covered(a) ? ATLAS_OK : ATLAS_ERR_UNSUPPORTED;
}

// How many elements of a row, 4, 2 or 1, are one access in every tensor.
int glr_wide(const GlrArgs& a) {
  const long s[] = {a.xb, a.xt, a.rbs, a.rt, a.ibs, a.it, a.zb, a.zt, a.yb, a.yt, a.D};
  const void* p[] = {a.x, a.r, a.i, a.z, a.y, a.dy, a.dx, a.dr, a.di, a.dz};
  int n = 4;
  for (long v : s)
    while (v % n) n /= 2;
  for (const void* q : p)
    while (!aligned(q, n * size_of(a.type))) n /= 2;
  return n;
}

}  // namespace

extern "C" {

int atlas_norm_forward(const void* x, const void* residual, const void* weight,
                       const atlas_norm_cfg* cfg, void* y, void* residual_out, float* scale,
                       void* stream) {
  const int rc = check_norm(cfg);
  if (rc != ATLAS_OK) return rc;
  if (cfg->rows == 0) return ATLAS_OK;
  if (!x || !y || (cfg->out_dtype == ATLAS_E4M3) != (scale != nullptr)) return ATLAS_ERR_INVALID;
  NormArgs a = norm_args(cfg);
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.y = y;
  a.r_out = residual_out;
  a.scale = scale;
  if (!aligned(x, size_of(a.dt)) || !aligned(residual, size_of(a.rt)) ||
      !aligned(weight, size_of(a.wt)) || !aligned(y, size_of(a.ot)) ||
      !aligned(residual_out, size_of(a.rt)) || !aligned(scale, 4))
    return ATLAS_ERR_INVALID;
  a.wide = a.d % 8 == 0 && a.sx % 8 == 0 && a.sr % 8 == 0 && a.sy % 8 == 0 && aligned(x, 16) &&
           aligned(residual, 16) && aligned(weight, 16) && aligned(y, 16) && aligned(residual_out, 16);
  return norm_forward_launch(a, stream_of(stream));
}

size_t atlas_norm_backward_workspace_bytes(const atlas_norm_cfg* cfg) {
  if (check_norm(cfg) != ATLAS_OK) return (size_t)-1;
  return norm_backward_workspace(norm_args(cfg));
}

int atlas_norm_backward(const void* h, const void* weight, const void* dy, const void* dh,
                        const atlas_norm_cfg* cfg, void* dx, float* dw, void* stream) {
  const int rc = check_norm(cfg);
  if (rc != ATLAS_OK) return rc;
  if (dw && !weight) return ATLAS_ERR_INVALID;
  if (cfg->rows > 0 && (!h || !dy || !dx)) return ATLAS_ERR_INVALID;
  NormArgs a = norm_args(cfg);
  if (!aligned(h, size_of(a.rt)) || !aligned(weight, size_of(a.wt)) || !aligned(dy, size_of(a.dt)) ||
      !aligned(dh, size_of(a.rt)) || !aligned(dx, size_of(a.rt)) || !aligned(dw, 4))
    return ATLAS_ERR_INVALID;
  const size_t need = norm_backward_workspace(a);
  if (dw && need && (!cfg->workspace || cfg->workspace_bytes < need || !aligned(cfg->workspace, 16)))
    return ATLAS_ERR_WORKSPACE;
  if (cfg->rows == 0 && !dw) return ATLAS_OK;
  a.x = h;
  a.r = dh;
  a.w = weight;
  a.dy = dy;
  a.y = dx;
  a.dw = dw;
  a.part = reinterpret_cast<float*>(cfg->workspace);
  a.wide = a.d % 8 == 0 && a.sr % 8 == 0 && a.sy % 8 == 0 && aligned(h, 16) && aligned(weight, 16) &&
           aligned(dy, 16) && aligned(dh, 16) && aligned(dx, 16);
  return norm_backward_launch(a, stream_of(stream));
}

int atlas_layernorm_forward(const void* x, const void* residual, const void* weight, const void* bias,
                            const atlas_norm_cfg* cfg, void* y, void* residual_out, float* scale,
                            void* stream) {
  const int rc = check_layernorm(cfg);
  if (rc != ATLAS_OK) return rc;
  if (cfg->rows == 0) return ATLAS_OK;
  if (!x || !y || (cfg->out_dtype == ATLAS_E4M3) != (scale != nullptr)) return ATLAS_ERR_INVALID;
  LayerNormArgs a = layernorm_args(cfg);
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.r_out = residual_out;
  a.scale = scale;
  if (!aligned(x, size_of(a.dt)) || !aligned(residual, size_of(a.rt)) ||
      !aligned(weight, size_of(a.wt)) || !aligned(bias, size_of(a.wt)) || !aligned(y, size_of(a.ot)) ||
      !aligned(residual_out, size_of(a.rt)) || !aligned(scale, 4))
    return ATLAS_ERR_INVALID;
  a.wide = a.d % 8 == 0 && a.sx % 8 == 0 && a.sr % 8 == 0 && a.sy % 8 == 0 && aligned(x, 16) &&
           aligned(residual, 16) && aligned(weight, 16) && aligned(bias, 16) && aligned(y, 16) &&
           aligned(residual_out, 16);
  return layernorm_forward_launch(a, stream_of(stream));
}

size_t atlas_layernorm_backward_workspace_bytes(const atlas_norm_cfg* cfg) {
  if (check_layernorm(cfg) != ATLAS_OK) return (size_t)-1;
  return layernorm_backward_workspace(layernorm_args(cfg));
}

int atlas_layernorm_backward(const void* h, const void* weight, const void* dy, const void* dh,
                             const atlas_norm_cfg* cfg, void* dx, float* dw, float* dbias, void* stream) {
  const int rc = check_layernorm(cfg);
  if (rc != ATLAS_OK) return rc;
  if (dw && !weight) return ATLAS_ERR_INVALID;
  if (cfg->rows > 0 && (!h || !dy || !dx)) return ATLAS_ERR_INVALID;
  LayerNormArgs a = layernorm_args(cfg);
  if (!aligned(h, size_of(a.rt)) || !aligned(weight, size_of(a.wt)) || !aligned(dy, size_of(a.dt)) ||
      !aligned(dh, size_of(a.rt)) || !aligned(dx, size_of(a.rt)) || !aligned(dw, 4) || !aligned(dbias, 4))
    return ATLAS_ERR_INVALID;
  const size_t need = layernorm_backward_workspace(a);
  if ((dw || dbias) && need && (!cfg->workspace || cfg->workspace_bytes < need || !aligned(cfg->workspace, 16)))
    return ATLAS_ERR_WORKSPACE;
  if (cfg->rows == 0 && !dw && !dbias) return ATLAS_OK;
  a.x = h;
  a.r = dh;
  a.w = weight;
  a.dy = dy;
  a.y = dx;
  a.dw = dw;
  a.db = dbias;
  a.part = reinterpret_cast<float*>(cfg->workspace);
  a.wide = a.d % 8 == 0 && a.sr % 8 == 0 && a.sy % 8 == 0 && aligned(h, 16) && aligned(weight, 16) &&
           aligned(dy, 16) && aligned(dh, 16) && aligned(dx, 16);
  return layernorm_backward_launch(a, stream_of(stream));
}

int atlas_conv_forward(const void* x, const void* weight, const void* bias,
                       const atlas_conv_cfg* cfg, void* y, const void* state_in, void* state_out,
                       void* stream) {
  const int rc = check_conv(cfg);
  if (rc != ATLAS_OK) return rc;
  if (cfg->B == 0) return ATLAS_OK;
  ConvArgs a = conv_args(cfg);
  const int e = size_of(a.dt), we = size_of(a.wt);
  if (!weight || (cfg->L > 0 && (!x || !y))) return ATLAS_ERR_INVALID;
  if (!aligned(x, e) || !aligned(y, e) || !aligned(state_in, e) || !aligned(state_out, e) ||
      !aligned(weight, we) || !aligned(bias, we))
    return ATLAS_ERR_INVALID;
  if (!conv_y_apart(a)) return ATLAS_ERR_INVALID;
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.y = y;
  a.st_in = state_in;
  a.st_out = state_out;
  a.wide = conv_wide(a, x, y, state_in, state_out, 4 * e);  // four elements a lane
  return conv_forward_launch(a, stream_of(stream));
}

size_t atlas_conv_backward_workspace_bytes(const atlas_conv_cfg* cfg) {
  if (check_conv(cfg) != ATLAS_OK || cfg->slot) return (size_t)-1;
  return conv_backward_workspace(conv_args(cfg));
}

int atlas_conv_backward(const void* x, const void* weight, const void* bias,
                        const atlas_conv_cfg* cfg, const void* state_in, const void* dy,
                        float* dstate, void* dx, float* dw, float* dbias, void* stream) {
  const int rc = check_conv(cfg);
  if (rc != ATLAS_OK) return rc;
  if (cfg->slot) return ATLAS_ERR_UNSUPPORTED;
  ConvArgs a = conv_args(cfg);
  const int e = size_of(a.dt), we = size_of(a.wt);
  if (!weight || !dw || (cfg->L > 0 && cfg->B > 0 && (!x || !dy || !dx))) return ATLAS_ERR_INVALID;
  if (!aligned(x, e) || !aligned(dy, e) || !aligned(dx, e) || !aligned(state_in, e) ||
      !aligned(dstate, 4) || !aligned(dw, 4) || !aligned(dbias, 4) || !aligned(weight, we) ||
      !aligned(bias, we))
    return ATLAS_ERR_INVALID;
  if (!apart(a.xb, a.xt, a.C, a.s.B, a.s.L, a.s.start)) return ATLAS_ERR_INVALID;
  const size_t need = conv_backward_workspace(a);
  if (need && (!cfg->workspace || cfg->workspace_bytes < need || !aligned(cfg->workspace, 16)))
    return ATLAS_ERR_WORKSPACE;
  a.x = x;
  a.w = weight;
  a.bias = bias;
  a.st_in = state_in;
  a.dy = dy;
  a.dstate = dstate;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.ws = cfg->workspace;
  a.wide = conv_wide(a, x, dy, state_in, dx, 16);  // 16-byte copies
  return conv_backward_launch(a, stream_of(stream));
}

size_t atlas_scan_workspace_bytes(const atlas_scan_cfg* cfg) {
  if (check_scan(cfg) != ATLAS_OK) return (size_t)-1;
  return scan_workspace(scan_args(cfg));
}

int atlas_scan_forward(const void* x, const void* dt, const float* A, const void* B, const void* C,
                       const float* Dskip, const void* z, const float* dt_bias,
                       const atlas_scan_cfg* cfg, void* y, const float* h_in, float* h_out,
                       void* stream) {
  const int rc = check_scan(cfg);
  if (rc != ATLAS_OK) return rc;
  if (cfg->B == 0) return ATLAS_OK;
  ScanArgs a = scan_args(cfg);
  const int e = size_of(a.type);
  if (!A || (cfg->L > 0 && (!x || !dt || !B || !C || !y))) return ATLAS_ERR_INVALID;
  if (!aligned(x, e) || !aligned(dt, e) || !aligned(B, e) || !aligned(C, e) || !aligned(z, e) ||
      !aligned(y, e) || !aligned(A, 4) || !aligned(Dskip, 4) || !aligned(dt_bias, 4) ||
      !aligned(h_in, 4) || !aligned(h_out, 4))
    return ATLAS_ERR_INVALID;
  if (!apart(a.yb, a.yt, a.D, a.s.B, a.s.L, a.s.start)) return ATLAS_ERR_INVALID;
  const size_t need = scan_workspace(a);
  if (need && (!cfg->workspace || cfg->workspace_bytes < need || !aligned(cfg->workspace, 16)))
    return ATLAS_ERR_WORKSPACE;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.Bm = B;
  a.Cm = C;
  a.Dk = Dskip;
  a.z = z;
  a.bias = dt_bias;
  a.y = y;
  a.h_in = h_in;
  a.h_out = h_out;
  a.ws = cfg->workspace;
  a.wide = scan_wide(a);
  a.wide_n = scan_wide_n(a);
  return scan_forward_launch(a, stream_of(stream));
}

size_t atlas_scan_backward_workspace_bytes(const atlas_scan_cfg* cfg) {
  if (check_scan(cfg) != ATLAS_OK || cfg->slot) return (size_t)-1;
  return scan_backward_workspace(scan_args(cfg));
}

int atlas_scan_backward(const void* x, const void* dt, const float* A, const void* B,
                        const void* C, const float* Dskip, const void* z, const float* dt_bias,
                        const atlas_scan_cfg* cfg, const float* h_in, const void* dy, float* dh,
                        void* dx, void* ddt, float* dA, void* dB, void* dC, float* dD, void* dz,
                        float* ddt_bias, void* stream) {
  const int rc = check_scan(cfg);
  if (rc != ATLAS_OK) return rc;
  if (cfg->slot) return ATLAS_ERR_UNSUPPORTED;
  ScanArgs a = scan_args(cfg);
  const int e = size_of(a.type);
  if (!A || !dA || (dD != nullptr) != (Dskip != nullptr) || (dz != nullptr) != (z != nullptr) ||
      (ddt_bias != nullptr) != (dt_bias != nullptr))
    return ATLAS_ERR_INVALID;
  if (cfg->L > 0 && cfg->B > 0 && (!x || !dt || !B || !C || !dy || !dx || !ddt || !dB || !dC))
    return ATLAS_ERR_INVALID;
  const void* elems[] = {x, dt, B, C, z, dy, dx, ddt, dB, dC, dz};
  for (const void* p : elems)
    if (!aligned(p, e)) return ATLAS_ERR_INVALID;
  const void* words[] = {A, Dskip, dt_bias, h_in, dh, dA, dD, ddt_bias};
  for (const void* p : words)
    if (!aligned(p, 4)) return ATLAS_ERR_INVALID;
  const int nB = a.s.B, L = a.s.L;
  const long gn = (long)a.G * a.N;
  if (!apart(a.xb, a.xt, a.D, nB, L, a.s.start) || !apart(a.tb, a.tt, a.D, nB, L, a.s.start) ||
      (z && !apart(a.zb, a.zt, a.D, nB, L, a.s.start)) ||
      !apart(a.bb, a.bt, gn, nB, L, a.s.start) || !apart(a.cb, a.ct, gn, nB, L, a.s.start))
    return ATLAS_ERR_INVALID;
  const size_t need = scan_backward_workspace(a);
  if (need && (!cfg->workspace || cfg->workspace_bytes < need || !aligned(cfg->workspace, 16)))
    return ATLAS_ERR_WORKSPACE;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.Bm = B;
  a.Cm = C;
  a.Dk = Dskip;
  a.z = z;
  a.bias = dt_bias;
  a.h_in = h_in;
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.ddt = ddt;
  a.dA = dA;
  a.dB = dB;
  a.dC = dC;
  a.dD = dD;
  a.dz = dz;
  a.dbias = ddt_bias;
  a.ws = cfg->workspace;
  a.wide = scan_wide(a);
  a.wide_n = scan_wide_n(a);
  return scan_backward_launch(a, stream_of(stream));
}

size_t atlas_glr_workspace_bytes(const atlas_glr_cfg* cfg) {
  GlrArgs a;
  return check_glr(cfg, a) == ATLAS_OK ? glr_workspace(a) : (size_t)-1;
}

size_t atlas_glr_kept_bytes(const atlas_glr_cfg* cfg) {
  GlrArgs a;
  return check_glr(cfg, a) == ATLAS_OK ? glr_kept(a) : (size_t)-1;
}

int atlas_glr_forward(const void* x, const void* r, const void* i, const void* z, const float* lambda,
                      const float* r_bias, const float* i_bias, const atlas_glr_cfg* cfg, void* y,
                      const float* h_in, float* h_out, void* kept, void* stream) {
  GlrArgs a;
  const int rc = check_glr(cfg, a);
  if (rc != ATLAS_OK) return rc;
  if (cfg->B == 0) return ATLAS_OK;
  const int e = size_of(a.type);
  if (!lambda || (cfg->L > 0 && (!x || !r || !y || (i_bias && !i)))) return ATLAS_ERR_INVALID;
  const void* elems[] = {x, r, i, z, y};
  for (const void* p : elems)
    if (!aligned(p, e)) return ATLAS_ERR_INVALID;
  const void* words[] = {lambda, r_bias, i_bias, h_in, h_out, kept};
  for (const void* p : words)
    if (!aligned(p, 4)) return ATLAS_ERR_INVALID;
  if (!apart(a.yb, a.yt, a.D, a.s.B, a.s.L, a.s.start)) return ATLAS_ERR_INVALID;
  const size_t need = glr_workspace(a);
  if (need && (!cfg->workspace || cfg->workspace_bytes < need || !aligned(cfg->workspace, 16)))
    return ATLAS_ERR_WORKSPACE;
  a.x = x;
  a.r = r;
  a.i = i;
  a.z = z;
  a.lam = lambda;
  a.rb = r_bias;
  a.ib = i_bias;
  a.y = y;
  a.h_in = h_in;
  a.h_out = h_out;
  a.kept = reinterpret_cast<float*>(kept);
  a.ws = cfg->workspace;
  a.wide = glr_wide(a);
  return glr_forward_launch(a, stream_of(stream));
}

size_t atlas_glr_backward_workspace_bytes(const atlas_glr_cfg* cfg) {
  GlrArgs a;
  return check_glr(cfg, a) == ATLAS_OK && !cfg->slot ? glr_backward_workspace(a) : (size_t)-1;
}

int atlas_glr_backward(const void* x, const void* r, const void* i, const void* z, const float* lambda,
                       const float* r_bias, const float* i_bias, const atlas_glr_cfg* cfg,
                       const float* h_in, const void* kept, const void* dy, float* dh, void* dx, void* dr,
                       void* di, void* dz, float* dlambda, float* dr_bias, float* di_bias, void* stream) {
  GlrArgs a;
  const int rc = check_glr(cfg, a);
  if (rc != ATLAS_OK) return rc;
  if (cfg->slot) return ATLAS_ERR_UNSUPPORTED;
  const int e = size_of(a.type);
  if (!lambda || !dlambda || (dr_bias != nullptr) != (r_bias != nullptr) ||
      (di_bias != nullptr) != (i_bias != nullptr))
    return ATLAS_ERR_INVALID;
  if (cfg->L > 0 && cfg->B > 0 &&  // (tensors without elements may have no address)
      (!x || !r || !dy || !dx || !dr || (i_bias && !i) || (di != nullptr) != (i != nullptr) ||
       (dz != nullptr) != (z != nullptr)))
    return ATLAS_ERR_INVALID;
  const void* elems[] = {x, r, i, z, dy, dx, dr, di, dz};
  for (const void* p : elems)
    if (!aligned(p, e)) return ATLAS_ERR_INVALID;
  const void* words[] = {lambda, r_bias, i_bias, h_in, kept, dh, dlambda, dr_bias, di_bias};
  for (const void* p : words)
    if (!aligned(p, 4)) return ATLAS_ERR_INVALID;
  const int nB = a.s.B, L = a.s.L;
  if (!apart(a.xb, a.xt, a.D, nB, L, a.s.start) || !apart(a.rbs, a.rt, a.D, nB, L, a.s.start) ||
      (i && !apart(a.ibs, a.it, a.D, nB, L, a.s.start)) || (z && !apart(a.zb, a.zt, a.D, nB, L, a.s.start)))
    return ATLAS_ERR_INVALID;
  const size_t need = glr_backward_workspace(a);
  if (need && (!cfg->workspace || cfg->workspace_bytes < need || !aligned(cfg->workspace, 16)))
    return ATLAS_ERR_WORKSPACE;
  a.x = x;
  a.r = r;
  a.i = i;
  a.z = z;
  a.lam = lambda;
  a.rb = r_bias;
  a.ib = i_bias;
  a.h_in = h_in;
  a.kept = const_cast<float*>(reinterpret_cast<const float*>(kept));
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.dr = dr;
  a.di = di;
  a.dz = dz;
  a.dlam = dlambda;
  a.drb = dr_bias;
  a.dib = di_bias;
  a.ws = cfg->workspace;
  a.wide = glr_wide(a);
  return glr_backward_launch(a, stream_of(stream));
}

}  // extern "C"
