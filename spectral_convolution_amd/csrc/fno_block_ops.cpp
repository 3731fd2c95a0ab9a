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
#include "mx4.hpp"

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

// ---- 4-bit floats

fno_status_t mx4_shape(int batch, int channels, long pixels, fno_dtype_t dtype) {
  if (batch < 1 || channels < 1 || pixels < 1 || !valid_dtype(dtype)) return FNO_ERR_INVALID_ARG;
  if (channels > kMx4MaxChannels || pixels > kMx4MaxRows / batch || !values_in_range(batch, channels, pixels))
    return FNO_ERR_UNSUPPORTED;
  return FNO_OK;
}

fno_status_t run_mx4(const void *x, void *y, const void *packed, bool pack, int batch, int channels, long pixels,
                     fno_dtype_t dtype, void *stream) {
  if (!packed || !(pack ? x : y)) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = mx4_shape(batch, channels, pixels, dtype);
  if (st != FNO_OK) return st;
  const Mx4Layout l = mx4_layout(batch * pixels, channels);
  const size_t bytes = (size_t)batch * channels * pixels * esize(dtype);
  Spans s;
  if (pack) {
    s.in(x, bytes, 16);
    s.out(packed, l.bytes, 256);
  } else {
    s.in(packed, l.bytes, 256);
    s.out(y, bytes, 16);
  }
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  uint8_t *base = static_cast<uint8_t *>(const_cast<void *>(packed));
  const Mx4Args a{x, y, base, base + l.exps, batch, channels, pixels, l.nb, 1};
  return status_of(launch_mx4(a, pack, (int)dtype, (hipStream_t)stream));
}

}  // namespace

extern "C" {

fno_status_t fno_mx4_bytes(int batch, int channels, long pixels, size_t *bytes) {
  if (!bytes) return FNO_ERR_INVALID_ARG;
  const fno_status_t st = mx4_shape(batch, channels, pixels, FNO_F32);
  if (st == FNO_OK) *bytes = mx4_layout(batch * pixels, channels).bytes;
  return st;
}

fno_status_t fno_mx4_pack(const void *x, void *packed, int batch, int channels, long pixels, fno_dtype_t dtype,
                          void *stream) {
  return run_mx4(x, nullptr, packed, true, batch, channels, pixels, dtype, stream);
}

fno_status_t fno_mx4_unpack(const void *packed, void *y, int batch, int channels, long pixels, fno_dtype_t dtype,
                            void *stream) {
  return run_mx4(nullptr, y, packed, false, batch, channels, pixels, dtype, stream);
}

fno_status_t fno_channel_mix_mx4(const void *xq, const void *Aq, const void *bias, const void *add, void *y, int batch,
                                 int c_in, int c_out, long pixels, int act, fno_dtype_t dtype, void *stream) {
  if (!xq || !Aq || !y || (act != 0 && act != 1)) return FNO_ERR_INVALID_ARG;
  for (int c : {c_in, c_out}) {
    const fno_status_t st = mx4_shape(batch, c, pixels, dtype);
    if (st != FNO_OK) return st;
  }
  const Mx4Layout lx = mx4_layout(batch * pixels, c_in), la = mx4_layout(c_out, c_in);
  const size_t es = esize(dtype), n = (size_t)batch * c_out * pixels * es;
  Spans s;
  s.in(xq, lx.bytes, 256);
  s.in(Aq, la.bytes, 256);
  s.in(bias, c_out * es, es);
  s.in(add, n, 16);
  s.out(y, n, 16);
  if (!s.ok()) return FNO_ERR_INVALID_ARG;
  const uint8_t *x = static_cast<const uint8_t *>(xq), *A = static_cast<const uint8_t *>(Aq);
  const Mx4MixArgs a{x, x + lx.exps, A, A + la.exps, bias, add, y, batch, c_in, c_out, pixels, lx.nb, act};
  return status_of(launch_mx4_mix(a, (int)dtype, (hipStream_t)stream));
}

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
