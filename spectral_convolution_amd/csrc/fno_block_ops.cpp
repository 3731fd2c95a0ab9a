// fno_block_ops.cpp - the C ABI of the operators of a regularised block (group norm with
// an activation and dropout, dropout into a residual stream) and of its 4-bit serving form
// (microscaled floats, the channel mix of two operands kept in them). Arguments are
// checked on the host; the kernels are in gnorm.hip, drop.hip, mx4.hip and mx4_mix.hip.

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "block_ops.hpp"
#include "call_check.hpp"

using namespace fno;

namespace {

// ---- dropout

// d's host form in `out` (NULL: no dropout); false: not a valid one
bool drop_of(const fno_dropout_t *d, Drop &out) {
  out = Drop{0, 1.f, kDropElement, 0, 0, nullptr};
  if (!d) return true;
  if (!(d->p >= 0.f && d->p <= 1.f)) return false;  // NaN is neither
  if (d->unit < FNO_DROP_ELEMENT || d->unit > FNO_DROP_SAMPLE || !aligned(d->step, 8)) return false;
  const uint32_t t = (uint32_t)std::rint((double)d->p * 65536.0);
  out = Drop{t, t < 65536 ? (float)(65536.0 / (65536 - t)) : 0.f, d->unit, d->seed, d->offset, d->step};
  return true;
}

fno_status_t field_shape(int batch, int channels, long pixels, int channels_last, long max_pixels, fno_dtype_t dtype) {
  if (batch < 1 || channels < 1 || pixels < 1 || (channels_last != 0 && channels_last != 1) || !valid_dtype(dtype))
    return FNO_ERR_INVALID_ARG;
  if (pixels > max_pixels || !values_in_range(batch, channels, pixels)) return FNO_ERR_UNSUPPORTED;
  return FNO_OK;
}

// ---- group norm

// the shape and its limits
fno_status_t gn_shape(int batch, int channels, long pixels, int groups, int channels_last, fno_dtype_t dtype, GnArgs &a) {
  if (groups < 1 || channels < 1 || channels % groups != 0) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = field_shape(batch, channels, pixels, channels_last, kGnMaxPixels, dtype);
  if (st != FNO_OK) return st;
  if (channels > kGnMaxChannels || (long)batch * groups > INT_MAX) return FNO_ERR_UNSUPPORTED;
  a.B = batch, a.C = channels, a.P = pixels, a.G = groups, a.Cg = channels / groups, a.last = channels_last;
  return FNO_OK;
}

fno_status_t gn_params(const fno_group_norm_params_t *p, const fno_dropout_t *drop, int batch, int channels, long pixels,
                       fno_dtype_t dtype, GnArgs &a, Spans &s) {
  if (!p || !std::isnormal(p->eps) || p->eps < 0.f || p->act < 0 || p->act > 2 || !drop_of(drop, a.drop))
    return FNO_ERR_INVALID_ARG;
  const fno_status_t st = gn_shape(batch, channels, pixels, p->groups, p->channels_last, dtype, a);
  if (st != FNO_OK) return st;
  a.w = p->weight, a.b = p->bias, a.act = p->act, a.eps = p->eps;
  const size_t es = esize(dtype);
  s.in(a.w, channels * es, es);
  s.in(a.b, channels * es, es);
  s.in(a.drop.step, 8, 8);
  return FNO_OK;
}

}  // namespace

extern "C" {

fno_status_t fno_dropout_residual(const fno_dropout_t *drop, const void *x, const void *v, void *y, int batch,
                                  int channels, long pixels, int channels_last, fno_dtype_t dtype, void *stream) {
  DropArgs a{};
  if (!drop || !v || !y || !drop_of(drop, a.drop)) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = field_shape(batch, channels, pixels, channels_last, kMaxRow, dtype);
  if (st != FNO_OK) return st;
  const size_t n = (size_t)batch * channels * pixels * esize(dtype);
  Spans s;
  s.in(x, n, 16);
  s.in(v, n, 16);
  s.in(drop->step, 8, 8);
  s.out(y, n, 16);
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  a.x = x, a.v = v, a.y = y, a.B = batch, a.C = channels, a.P = pixels, a.last = channels_last;
  return status_of(launch_drop(a, (int)dtype, (hipStream_t)stream));
}

fno_status_t fno_group_norm_workspace_bytes(int batch, int channels, long pixels, int groups, int channels_last,
                                            fno_dtype_t dtype, size_t *bytes) {
  if (!bytes) return FNO_ERR_INVALID_ARG;
  GnArgs a{};
  const fno_status_t st = gn_shape(batch, channels, pixels, groups, channels_last, dtype, a);
  if (st == FNO_OK) *bytes = gnorm_workspace_bytes(a, (int)dtype);
  return st;
}

fno_status_t fno_group_norm(const fno_group_norm_params_t *params, const fno_dropout_t *drop, const void *x, void *y,
                            float *stats, void *workspace, int batch, int channels, long pixels, fno_dtype_t dtype,
                            void *stream) {
  if (!x || !y || !workspace) return FNO_ERR_INVALID_ARG;
  GnArgs a{};
  Spans s;
  const fno_status_t st = gn_params(params, drop, batch, channels, pixels, dtype, a, s);
  if (st != FNO_OK) return st;
  const size_t n = (size_t)batch * channels * pixels * esize(dtype);
  s.in(x, n, 16);
  s.out(y, n, 16);
  s.out(stats, (size_t)batch * a.G * sizeof(float2), 8);
  s.out(workspace, gnorm_workspace_bytes(a, (int)dtype), 16);
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  a.x = x, a.y = y, a.stats = reinterpret_cast<float2 *>(stats);
  return status_of(launch_gnorm(a, true, workspace, (int)dtype, (hipStream_t)stream));
}

fno_status_t fno_group_norm_backward(const fno_group_norm_params_t *params, const fno_dropout_t *drop, const void *x,
                                     const float *stats, const void *gy, void *gx, void *gw, void *gb, void *workspace,
                                     int batch, int channels, long pixels, fno_dtype_t dtype, void *stream) {
  if (!x || !stats || !gy || !workspace || (!gx && !gw && !gb)) return FNO_ERR_INVALID_ARG;
  GnArgs a{};
  Spans s;
  const fno_status_t st = gn_params(params, drop, batch, channels, pixels, dtype, a, s);
  if (st != FNO_OK) return st;
  if ((gw && !a.w) || (gb && !a.b)) return FNO_ERR_INVALID_ARG;  // a gradient of a parameter that is not there
  const size_t es = esize(dtype), n = (size_t)batch * channels * pixels * es;
  s.in(x, n, 16);
  s.in(gy, n, 16);
  s.in(stats, (size_t)batch * a.G * sizeof(float2), 8);
  s.out(gx, n, 16);
  s.out(gw, channels * es, es);
  s.out(gb, channels * es, es);
  s.out(workspace, gnorm_workspace_bytes(a, (int)dtype), 16);
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  a.x = x, a.gy = gy, a.gx = gx, a.gw = gw, a.gb = gb;
  a.stats = reinterpret_cast<float2 *>(const_cast<float *>(stats));
  return status_of(launch_gnorm(a, false, workspace, (int)dtype, (hipStream_t)stream));
}

}  // extern "C"
