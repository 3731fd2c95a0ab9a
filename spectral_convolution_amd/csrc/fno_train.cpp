// fno_train.cpp - the C ABI of the training operators around a block: the
// 8-bit activation checkpoints, the channel mix that keeps them with its
// backward, and the norms with gate and residual scale. Arguments are checked
// on the host; the kernels are in checkpoint.hip, mix_train.hip and norm.hip.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "call_check.hpp"
#include "checkpoint.hpp"

using namespace fno;

namespace {

uint8_t *at(void *p, size_t off) { return static_cast<uint8_t *>(p) + off; }

// ---- checkpoints

fno_status_t checkpoint_shape(long rows, long n, fno_dtype_t dtype) {
  if (rows < 1 || n < 1 || !valid_dtype(dtype)) return FNO_ERR_INVALID_ARG;
  if (n > kMaxRow || !values_in_range(rows, n, 1)) return FNO_ERR_UNSUPPORTED;
  return FNO_OK;
}

fno_status_t run_checkpoint(const void *x, void *y, const void *saved, bool pack, long rows, long n,
                            fno_dtype_t dtype, void *stream) {
  if (!saved || !(pack ? x : y)) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = checkpoint_shape(rows, n, dtype);
  if (st != FNO_OK) return st;
  const CkLayout l = ck_layout(rows, n);
  const size_t bytes = (size_t)rows * n * esize(dtype);
  Spans s;
  if (pack) {
    s.in(x, bytes, 16);
    s.out(saved, l.bytes, 256);
  } else {
    s.in(saved, l.bytes, 256);
    s.out(y, bytes, 16);
  }
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  uint8_t *base = static_cast<uint8_t *>(const_cast<void *>(saved));
  const CkArgs a{x, y, base, reinterpret_cast<int8_t *>(base + l.exps), rows, n, l.nb};
  return status_of(launch_checkpoint(a, pack, (int)dtype, (hipStream_t)stream));
}

// ---- norms

fno_status_t norm_shape(const fno_norm_params_t *p, int batch, int channels, long pixels, fno_dtype_t dtype) {
  if (!p || (p->kind != FNO_NORM_RMS && p->kind != FNO_NORM_LAYER) || !std::isnormal(p->eps) || p->eps < 0.f)
    return FNO_ERR_INVALID_ARG;
  if (batch < 1 || channels < 1 || pixels < 1 || !valid_dtype(dtype)) return FNO_ERR_INVALID_ARG;
  if (channels > (pixels == 1 ? kNormMaxToken : kNormMaxField)) return FNO_ERR_UNSUPPORTED;
  if ((pixels > 1 && batch > 65535) || pixels > kNormMaxPixels || !values_in_range(batch, channels, pixels))
    return FNO_ERR_UNSUPPORTED;
  return FNO_OK;
}

NormArgs norm_args(const fno_norm_params_t *p, int batch, int channels, long pixels, Spans &s, fno_dtype_t dtype) {
  NormArgs a{};
  a.w_post = p->w_post, a.b_post = p->b_post, a.gate = p->gate, a.scale = p->scale, a.w_pre = p->w_pre,
  a.b_pre = p->b_pre;
  a.kind = p->kind, a.eps = p->eps, a.B = batch, a.C = channels, a.P = pixels;
  const size_t es = esize(dtype), nc = channels * es;
  for (const void *q : {a.w_post, a.b_post, a.scale, a.w_pre, a.b_pre}) s.in(q, nc, es);
  s.in(a.gate, batch * nc, es);
  return a;
}

// the two checkpoints of a norm: x's, then v's
size_t norm_saved(int batch, int channels, long pixels, CkLayout &l) {
  l = pixels == 1 ? ck_layout(batch, channels) : ck_layout((long)batch * channels, pixels);
  return 2 * l.bytes;
}

void norm_attach(NormArgs &a, const void *saved, const CkLayout &l) {
  void *m = const_cast<void *>(saved);
  a.xq = at(m, 0), a.xe = reinterpret_cast<int8_t *>(at(m, l.exps));
  a.vq = at(m, l.bytes), a.ve = reinterpret_cast<int8_t *>(at(m, l.bytes + l.exps));
}

fno_status_t norm_forward(const fno_norm_params_t *p, const void *x, const void *v, void *y, void *u, void *saved,
                          bool save, int batch, int channels, long pixels, fno_dtype_t dtype, void *stream) {
  if (!x || !v || !y || (save && !saved)) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = norm_shape(p, batch, channels, pixels, dtype);
  if (st != FNO_OK) return st;
  Spans s;
  NormArgs a = norm_args(p, batch, channels, pixels, s, dtype);
  const size_t n = (size_t)batch * channels * pixels * esize(dtype);
  s.in(x, n, 16);
  s.in(v, n, 16);
  s.out(y, n, 16);
  s.out(u, n, 16);
  a.x = x, a.v = v, a.y = y, a.u = u;
  if (save) {
    CkLayout l;
    s.out(saved, norm_saved(batch, channels, pixels, l), 256);
    norm_attach(a, saved, l);
  }
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  return status_of(launch_norm_fwd(a, (int)dtype, (hipStream_t)stream));
}

fno_status_t norm_backward(const fno_norm_params_t *p, const void *x, const void *v, const void *saved, bool from_saved,
                           const void *gy, const void *gu, void *gx, void *gv, const fno_norm_grads_t *grads,
                           void *workspace, int batch, int channels, long pixels, fno_dtype_t dtype, void *stream) {
  if (!gy || (from_saved ? !saved : (!x || !v))) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = norm_shape(p, batch, channels, pixels, dtype);
  if (st != FNO_OK) return st;
  const fno_norm_grads_t none{}, g = grads ? *grads : none;
  const bool any = g.w_post || g.b_post || g.gate || g.scale || g.w_pre || g.b_pre;
  if (!gx && !gv && !any) return FNO_ERR_INVALID_ARG;
  if (any && !workspace) return FNO_ERR_INVALID_ARG;
  // a gradient of a parameter that is not there, or of u's norm without gu
  if ((g.w_post && !p->w_post) || (g.b_post && !p->b_post) || (g.gate && !p->gate) || (g.scale && !p->scale) ||
      (g.w_pre && !p->w_pre) || (g.b_pre && !p->b_pre))
    return FNO_ERR_INVALID_ARG;
  if (!gu && (g.w_pre || g.b_pre)) return FNO_ERR_INVALID_ARG;
  Spans s;
  NormArgs a = norm_args(p, batch, channels, pixels, s, dtype);
  const size_t es = esize(dtype), nc = channels * es, n = (size_t)batch * channels * pixels * es;
  if (from_saved) {
    CkLayout l;
    s.in(saved, norm_saved(batch, channels, pixels, l), 256);
    norm_attach(a, saved, l);
  } else {
    s.in(x, n, 16);
    s.in(v, n, 16);
    a.x = x, a.v = v;
  }
  s.in(gy, n, 16);
  s.in(gu, n, 16);
  s.out(gx, n, 16);
  s.out(gv, n, 16);
  for (void *q : {g.w_post, g.b_post, g.scale, g.w_pre, g.b_pre}) s.out(q, nc, es);
  s.out(g.gate, batch * nc, es);
  if (any) s.out(workspace, norm_workspace_bytes(batch, channels, pixels, (int)dtype), 16);
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  a.gy = gy, a.gu = gu, a.gx = gx, a.gv = gv;
  a.g_w_post = g.w_post, a.g_b_post = g.b_post, a.g_gate = g.gate, a.g_scale = g.scale, a.g_w_pre = g.w_pre,
  a.g_b_pre = g.b_pre;
  a.part = any ? static_cast<float *>(workspace) : nullptr;
  return status_of(launch_norm_bwd(a, (int)dtype, (hipStream_t)stream));
}

// ---- channel mix

fno_status_t mix_shape(int batch, int c_in, int c_out, long pixels, int act, int has_add, fno_dtype_t dtype) {
  if (batch < 1 || c_in < 1 || c_out < 1 || pixels < 1 || (act != 0 && act != 1) || (has_add != 0 && has_add != 1) ||
      !valid_dtype(dtype))
    return FNO_ERR_INVALID_ARG;
  if (c_in > kMixTrainMax || c_out > kMixTrainMax || pixels > kMixTrainPixels ||
      (pixels + 63) / 64 > kMixTrainTiles / batch)
    return FNO_ERR_UNSUPPORTED;
  return FNO_OK;
}

// the kept inputs: the checkpoint of x, then (GELU with add) that of add
struct MixSaved {
  CkLayout x, add;
  bool both;
  size_t bytes;
};
MixSaved mix_saved(int batch, int c_in, int c_out, long pixels, int act, int has_add) {
  MixSaved m;
  m.x = ck_layout((long)batch * c_in, pixels);
  m.add = ck_layout((long)batch * c_out, pixels);
  m.both = act == 1 && has_add;
  m.bytes = m.x.bytes + (m.both ? m.add.bytes : 0);
  return m;
}

void mix_attach(MixTrainArgs &a, const void *saved, const MixSaved &m) {
  void *s = const_cast<void *>(saved);
  a.xq = at(s, 0), a.xe = reinterpret_cast<int8_t *>(at(s, m.x.exps));
  if (m.both) a.aq = at(s, m.x.bytes), a.ae = reinterpret_cast<int8_t *>(at(s, m.x.bytes + m.add.exps));
}

}  // namespace

extern "C" {

fno_status_t fno_channel_mix_saved_bytes(int batch, int c_in, int c_out, long pixels, int act, int has_add,
                                         size_t *bytes) {
  if (!bytes) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = mix_shape(batch, c_in, c_out, pixels, act, has_add, FNO_F32);
  if (st == FNO_OK) *bytes = mix_saved(batch, c_in, c_out, pixels, act, has_add).bytes;
  return st;
}

fno_status_t fno_channel_mix_workspace_bytes(int batch, int c_in, int c_out, long pixels, fno_dtype_t dtype,
                                             size_t *bytes) {
  if (!bytes) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = mix_shape(batch, c_in, c_out, pixels, 0, 0, dtype);
  if (st == FNO_OK) *bytes = mix_train_workspace_bytes(batch, c_in, c_out, pixels, (int)dtype);
  return st;
}

fno_status_t fno_channel_mix_save(const void *x, const void *A, const void *bias, const void *add, void *y, void *saved,
                                  int batch, int c_in, int c_out, long pixels, int act, fno_dtype_t dtype,
                                  void *stream) {
  if (!x || !A || !y || !saved) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = mix_shape(batch, c_in, c_out, pixels, act, add != nullptr, dtype);
  if (st != FNO_OK) return st;
  const size_t es = esize(dtype), nx = (size_t)batch * c_in * pixels * es, ny = (size_t)batch * c_out * pixels * es;
  const MixSaved m = mix_saved(batch, c_in, c_out, pixels, act, add != nullptr);
  Spans s;
  s.in(x, nx, 16);
  s.in(A, (size_t)c_out * c_in * es, es);
  s.in(bias, c_out * es, es);
  s.in(add, ny, 16);
  s.out(y, ny, 16);
  s.out(saved, m.bytes, 256);
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  MixTrainArgs a{};
  a.x = x, a.add = add, a.A = A, a.bias = bias, a.y = y;
  a.B = batch, a.I = c_in, a.O = c_out, a.P = pixels, a.act = act;
  mix_attach(a, saved, m);
  return status_of(launch_mix_save(a, (int)dtype, (hipStream_t)stream));
}

fno_status_t fno_channel_mix_backward_saved(const void *saved, const void *A, const void *bias, const void *gy, void *gx,
                                            void *gA, void *gbias, void *gadd, void *workspace, int batch, int c_in,
                                            int c_out, long pixels, int act, int has_add, fno_dtype_t dtype,
                                            void *stream) {
  if (!saved || !A || !gy || (!gx && !gA && !gbias && !gadd)) return FNO_ERR_INVALID_ARG;
  if (((gA || gbias) && !workspace) || (gadd && !has_add)) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = mix_shape(batch, c_in, c_out, pixels, act, has_add, dtype);
  if (st != FNO_OK) return st;
  const size_t es = esize(dtype), nx = (size_t)batch * c_in * pixels * es, ny = (size_t)batch * c_out * pixels * es;
  const MixSaved m = mix_saved(batch, c_in, c_out, pixels, act, has_add);
  Spans s;
  s.in(saved, m.bytes, 256);
  s.in(A, (size_t)c_out * c_in * es, es);
  s.in(bias, c_out * es, es);
  s.in(gy, ny, 16);
  s.out(gx, nx, 16);
  s.out(gA, (size_t)c_out * c_in * es, es);
  s.out(gbias, c_out * es, es);
  s.out(gadd, ny, 16);
  const bool sums = gA || gbias;
  if (sums) s.out(workspace, mix_train_workspace_bytes(batch, c_in, c_out, pixels, (int)dtype), 16);
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  MixTrainArgs a{};
  a.A = A, a.bias = bias, a.gy = gy, a.gx = gx, a.gadd = gadd, a.gA = gA, a.gbias = gbias;
  a.part = sums ? static_cast<float *>(workspace) : nullptr;
  a.B = batch, a.I = c_in, a.O = c_out, a.P = pixels, a.act = act;
  mix_attach(a, saved, m);
  return status_of(launch_mix_bwd(a, (int)dtype, (hipStream_t)stream));
}

fno_status_t fno_checkpoint_bytes(long rows, long n, size_t *bytes) {
  if (!bytes) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = checkpoint_shape(rows, n, FNO_F32);
  if (st == FNO_OK) *bytes = ck_layout(rows, n).bytes;
  return st;
}

fno_status_t fno_checkpoint_pack(const void *x, void *saved, long rows, long n, fno_dtype_t dtype, void *stream) {
  return run_checkpoint(x, nullptr, saved, true, rows, n, dtype, stream);
}

fno_status_t fno_checkpoint_unpack(const void *saved, void *y, long rows, long n, fno_dtype_t dtype, void *stream) {
  return run_checkpoint(nullptr, y, saved, false, rows, n, dtype, stream);
}

fno_status_t fno_norm_residual_saved_bytes(int batch, int channels, long pixels, size_t *bytes) {
  if (!bytes) return FNO_ERR_INVALID_ARG;
  const fno_norm_params_t p{FNO_NORM_RMS, 1e-5f, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  const fno_status_t st = norm_shape(&p, batch, channels, pixels, FNO_F32);
  CkLayout l;
  if (st == FNO_OK) *bytes = norm_saved(batch, channels, pixels, l);
  return st;
}

fno_status_t fno_norm_residual_workspace_bytes(int batch, int channels, long pixels, fno_dtype_t dtype,
                                               size_t *bytes) {
  if (!bytes) return FNO_ERR_INVALID_ARG;
  const fno_norm_params_t p{FNO_NORM_RMS, 1e-5f, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  const fno_status_t st = norm_shape(&p, batch, channels, pixels, dtype);
  if (st == FNO_OK) *bytes = norm_workspace_bytes(batch, channels, pixels, (int)dtype);
  return st;
}

fno_status_t fno_norm_residual(const fno_norm_params_t *params, const void *x, const void *v, void *y, void *u,
                               int batch, int channels, long pixels, fno_dtype_t dtype, void *stream) {
  return norm_forward(params, x, v, y, u, nullptr, false, batch, channels, pixels, dtype, stream);
}

fno_status_t fno_norm_residual_save(const fno_norm_params_t *params, const void *x, const void *v, void *y, void *u,
                                    void *saved, int batch, int channels, long pixels, fno_dtype_t dtype,
                                    void *stream) {
  return norm_forward(params, x, v, y, u, saved, true, batch, channels, pixels, dtype, stream);
}

fno_status_t fno_norm_residual_backward(const fno_norm_params_t *params, const void *x, const void *v, const void *gy,
                                        const void *gu, void *gx, void *gv, const fno_norm_grads_t *grads,
                                        void *workspace, int batch, int channels, long pixels, fno_dtype_t dtype,
                                        void *stream) {
  return norm_backward(params, x, v, nullptr, false, gy, gu, gx, gv, grads, workspace, batch, channels, pixels, dtype,
                       stream);
}

fno_status_t fno_norm_residual_backward_saved(const fno_norm_params_t *params, const void *saved, const void *gy,
                                              const void *gu, void *gx, void *gv, const fno_norm_grads_t *grads,
                                              void *workspace, int batch, int channels, long pixels,
                                              fno_dtype_t dtype, void *stream) {
  return norm_backward(params, nullptr, nullptr, saved, true, gy, gu, gx, gv, grads, workspace, batch, channels,
                       pixels, dtype, stream);
}

}  // extern "C"
