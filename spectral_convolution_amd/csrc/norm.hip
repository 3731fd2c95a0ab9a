// norm.hip - the norms before and after a block, fused with its gate and
// residual scale, forward and backward.
//
// For every sample b and pixel p, over the channels c (C of them):
//   N(v)[c] = (v[c] - m) r w_post[c] + b_post[c]
//   y[c]    = x[c] + scale[c] gate[b][c] N(v)[c]
//   u[c]    = (y[c] - m') r' w_pre[c] + b_pre[c]
// with m the mean over c (layer norm; 0 for the root-mean-square norm), r =
// 1 / sqrt(mean((v - m)^2) + eps), and m', r' the same of y. v is a block's
// branch output, y the residual stream and u the next block's input.
//
// Backward, at gy = dL/dy and gu = dL/du: with a unit-scale norm h^ = (h - m) r
// and g = dL/dh^, dL/dh = r (g - h^ mean(g h^) - [layer] mean(g)). So
//   gx = gy + [that of y at g = gu w_pre],
//   gv = [that of v at g = gx scale gate w_post],
// and with the per-(b, c) sums over pixels
//   T = sum gx v^,  G = sum gx,  U = sum gu y^,  V = sum gu:
//   g_gate = scale (w_post T + b_post G),  g_scale = sum_b gate (w_post T + b_post G),
//   g_w_post = scale sum_b gate T,  g_b_post = scale sum_b gate G,
//   g_w_pre = sum_b U,  g_b_pre = sum_b V.
//
// Statistics, sums and everything between load and store are fp32; the
// variance is the mean of squared deviations from the mean already known, so
// a large mean costs no digits. Means are divided, not multiplied by 1 / C: with
// equal channels h - m is then 0, where an m one rounding off times r = eps^-1/2
// would not be. y's statistics are those of the unrounded y.
//
// Fields ([B][C][P], P > 1; fno_norm_fwd / fno_norm_bwd): a tile is all
// channels of 128 bytes of each row (64 pixels in 16 bits, 32 in fp32), one
// checkpoint block or two. A wave holds 8 CPT channels of it in registers: lane l
// owns 16 bytes of pixels (l % 8) of the channels l / 8 + 8 k, so every
// access covers 8 whole 128-byte lines, each input is read once and each
// output written once. The sums over channels are folded across the wave with
// row and half swaps that halve the values held with each step (14 operations for 8
// pixels instead of the 24 of a butterfly) and, where the channels need more
// than one wave, joined through LDS. Bound by memory.
//
// Token layout (P = 1; fno_norm_tok_fwd / _bwd): channels are contiguous, a
// row is held by one wave up to 1024 channels (bf16: 512 with one access
// per lane) and by a workgroup above.
//
// The backward's sums over pixels or rows stay in registers over a
// workgroup's run and go to the workspace once; fno_norm_params adds them in
// a fixed order, so results do not change from run to run.

#include <algorithm>

#include "checkpoint.hpp"

namespace fno {

namespace {
constexpr int kRms = 0;
constexpr int kLayer = 1;

__device__ __forceinline__ float param(const void *p, int dtype, size_t i, float none) {
  if (!p) return none;
  if (dtype == DT_F32) return reinterpret_cast<const float *>(p)[i];
  if (dtype == DT_F16) return (float)reinterpret_cast<const _Float16 *>(p)[i];
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16);
}

template <int DT>
__device__ __forceinline__ void put(void *p, size_t i, float v) {
  if (!p) return;
  if constexpr (DT == DT_F32) reinterpret_cast<float *>(p)[i] = v;
  else if constexpr (DT == DT_F16) reinterpret_cast<_Float16 *>(p)[i] = (_Float16)v;
  else reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)f32_to_bf16(v);
}

__device__ __forceinline__ float rsq(float v) { return __builtin_amdgcn_rsqf(v); }

__device__ __forceinline__ void swap32(float a, float b, float &x, float &y) {
  const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  x = __uint_as_float(t[0]);
  y = __uint_as_float(t[1]);
}
__device__ __forceinline__ void swap16(float a, float b, float &x, float &y) {
  const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  x = __uint_as_float(t[0]);
  y = __uint_as_float(t[1]);
}
template <int CTRL>
__device__ __forceinline__ float fdpp(float v) {
  return __uint_as_float(ck_dpp<CTRL>(__float_as_uint(v)));
}

// sum over the 8 lanes that share l / 8
__device__ __forceinline__ float sum8(float v) {
  v += fdpp<kDppXor1>(v);
  v += fdpp<kDppXor2>(v);
  return v + fdpp<kDppHalfMirror>(v);
}

// sum over the wave, in every lane
__device__ __forceinline__ float sum64(float v) {
  float x, y;
  v = sum8(v);
  v += fdpp<kDppRor8>(v);
  swap16(v, v, x, y);
  v = x + y;
  swap32(v, v, x, y);
  return x + y;
}

// Sums of s[0 .. V-1] over the lanes with equal l % 8; lane l keeps the totals
// of the V / 4 values i + (V / 4) (l / 16 % 2) + (V / 2) (l / 32).
template <int V>
__device__ __forceinline__ void fold(const float (&s)[V], float (&o)[V / 4]) {
  float h[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    float x, y;
    swap32(s[i], s[i + V / 2], x, y);
    h[i] = x + y;
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    float x, y;
    swap16(h[i], h[i + V / 4], x, y);
    o[i] = x + y;
    o[i] += fdpp<kDppRor8>(o[i]);
  }
}

// the inverse distribution: every lane gets all V values
template <int V>
__device__ __forceinline__ void unfold(const float (&o)[V / 4], float (&s)[V]) {
  float h[V / 2];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) swap16(o[i], o[i], h[i], h[i + V / 4]);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) swap32(h[i], h[i], s[i], s[i + V / 2]);
}

// Joins NQ folded sums over the WPT waves of a tile through LDS. Two buffers in
// turn: a wave that writes one again has passed the barrier of the other.
template <int NQ, int V, int WPT>
struct Join {
  static __device__ __forceinline__ void run(float (&o)[NQ][V / 4], float *red, int &turn, int wave, int lane) {
    if constexpr (WPT > 1) {
      constexpr int ROW = 2 * V * 8;  // two quantities of the 8 V pixels
      const int waves = blockDim.x >> 6;
      float *buf = red + (size_t)(turn & 1) * waves * ROW;
      ++turn;
      const int slot = (lane & 7) * V + (V / 4) * ((lane >> 4) & 1) + (V / 2) * (lane >> 5);
      if ((lane & 8) == 0) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int i = 0; i < V / 4; ++i) buf[wave * ROW + q * 8 * V + slot + i] = o[q][i];
      }
      __syncthreads();
      const int w0 = wave / WPT * WPT;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          float t = 0.f;
#pragma unroll
          for (int w = 0; w < WPT; ++w) t += buf[(w0 + w) * ROW + q * 8 * V + slot + i];
          o[q][i] = t;
        }
    }
  }
};

template <int WPT>
constexpr int norm_threads() { return WPT > 4 ? 64 * WPT : 256; }

}  // namespace

// One row piece of a field: 16 bytes of channel c at pixel p, from the field
// or from its checkpoint; zeros past the channels or the row's end.
template <int DT>
__device__ __forceinline__ ck_u32x4 norm_load(const void *f, size_t row, long p, long P, bool whole, bool ok) {
  ck_u32x4 r;
  if (whole) {
    r = ck_load<DT>(f, row * P + p, 8);
    if (!ok) r = ck_u32x4{0u, 0u, 0u, 0u};
  } else {
    r = ck_load<DT>(f, row * P + p, ok ? P - p : 0);
  }
  return r;
}

template <int DT>
__device__ __forceinline__ ck_u32x4 norm_decode(const uint8_t *q, const int8_t *e, size_t row, long p, long nb, bool ok) {
  if (!ok || p >= nb * kCkBlock) return ck_u32x4{0u, 0u, 0u, 0u};
  const uint8_t *s = q + row * nb * kCkBlock + p;
  uint2 c;
  if constexpr (DT == DT_F32) c = make_uint2(*reinterpret_cast<const uint32_t *>(s), 0u);
  else c = *reinterpret_cast<const uint2 *>(s);
  return ck_decode<DT>(c, e[row * nb + p / kCkBlock]);
}

template <int DT>
__device__ __forceinline__ void norm_encode(const ck_u32x4 &r, uint8_t *q, int8_t *e, size_t row, long p, long nb, bool ok) {
  constexpr int L = kCkBlock / ck_vec<DT>();  // lanes of a block
  const int ex = ck_exponent<DT>(ck_groupmax<L>(ck_maxkey<DT>(r)));
  const uint2 c = ck_codes<DT>(r, ex);
  if (!ok || p >= nb * kCkBlock) return;
  uint8_t *d = q + row * nb * kCkBlock + p;
  if constexpr (DT == DT_F32) *reinterpret_cast<uint32_t *>(d) = c.x;
  else *reinterpret_cast<uint2 *>(d) = c;
  if (p % kCkBlock == 0) e[row * nb + p / kCkBlock] = (int8_t)ex;
}

// {scale gate w_post, scale gate b_post, w_pre, b_pre} of the channels of sample b
template <int DT>
__device__ __forceinline__ void norm_table(const NormArgs &a, int b, int n, float4 *tab) {
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.C) {
      const float sg = param(a.scale, DT, c, 1.f) * param(a.gate, DT, (size_t)b * a.C + c, 1.f);
      t = make_float4(sg * param(a.w_post, DT, c, 1.f), sg * param(a.b_post, DT, c, 0.f), param(a.w_pre, DT, c, 1.f),
                      param(a.b_pre, DT, c, 0.f));
    }
    tab[c] = t;
  }
}

template <int DT, int CPT, int WPT, int KIND>
__global__ __launch_bounds__(norm_threads<WPT>()) void fno_norm_fwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), PX = 8 * V, WAVES = norm_threads<WPT>() / 64, TPG = WAVES / WPT, NC = 8 * CPT * WPT;
  __shared__ float4 tab[NC];
  __shared__ float red[WPT > 1 ? 2 * WAVES * 2 * PX : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.y;
  norm_table<DT>(a, b, NC, tab);
  __syncthreads();
  const int pl = lane & 7, c0 = (wave % WPT) * 8 * CPT + (lane >> 3);
  const long P = a.P, nt = (P + PX - 1) / PX, per = (nt + gridDim.x - 1) / gridDim.x;
  const long t0 = blockIdx.x * per, t1 = min(nt, t0 + per), nb = (P + kCkBlock - 1) / kCkBlock;
  const float invC = 1.f / (float)a.C;
  int turn = 0;
  for (long tt = t0; tt < t1; tt += TPG) {
    const long t = tt + wave / WPT;
    const bool active = t < t1;
    if (WPT == 1 && !active) break;
    const long p = t * PX + pl * V;
    const bool whole = active && (t + 1) * PX <= P;
    ck_u32x4 vr[CPT], xr[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const int c = c0 + 8 * k;
      const size_t row = (size_t)b * a.C + (c < a.C ? c : 0);
      vr[k] = norm_load<DT>(a.v, row, p, P, whole, active && c < a.C);
      xr[k] = norm_load<DT>(a.x, row, p, P, whole, active && c < a.C);
    }
    if (a.vq) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const int c = c0 + 8 * k;
        const size_t row = (size_t)b * a.C + c;
        norm_encode<DT>(vr[k], a.vq, a.ve, row, p, nb, active && c < a.C);
        norm_encode<DT>(xr[k], a.xq, a.xe, row, p, nb, active && c < a.C);
      }
    }
    float s[1][V], o[1][V / 4], m[V], r[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = 0.f;
    if constexpr (KIND == kLayer) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0][e] = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) s[0][e] += ck_get<DT>(vr[k], e);
      }
      fold<V>(s[0], o[0]);
      Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) o[0][i] /= (float)a.C;
      unfold<V>(o[0], m);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s[0][e] = 0.f;
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        float d = ck_get<DT>(vr[k], e) - m[e];
        if (KIND == kLayer && c0 + 8 * k >= a.C) d = 0.f;
        s[0][e] = fmaf(d, d, s[0][e]);
      }
    }
    fold<V>(s[0], o[0]);
    Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) o[0][i] = rsq(fmaf(o[0][i], invC, a.eps));
    unfold<V>(o[0], r);
    float y[CPT][V];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const int c = c0 + 8 * k;
      const float4 w = tab[c];
#pragma unroll
      for (int e = 0; e < V; ++e)
        y[k][e] = ck_get<DT>(xr[k], e) + fmaf((ck_get<DT>(vr[k], e) - m[e]) * r[e], w.x, w.y);
      if (active && c < a.C) ck_store<DT>(a.y, ((size_t)b * a.C + c) * P + p, whole ? 8 : P - p, ck_raw<DT>(y[k]));
    }
    if (a.u) {
      if constexpr (KIND == kLayer) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[0][e] = 0.f;
#pragma unroll
          for (int k = 0; k < CPT; ++k) s[0][e] += y[k][e];
        }
        fold<V>(s[0], o[0]);
        Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) o[0][i] /= (float)a.C;
        unfold<V>(o[0], m);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0][e] = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          float d = y[k][e] - m[e];
          if (KIND == kLayer && c0 + 8 * k >= a.C) d = 0.f;
          s[0][e] = fmaf(d, d, s[0][e]);
        }
      }
      fold<V>(s[0], o[0]);
      Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) o[0][i] = rsq(fmaf(o[0][i], invC, a.eps));
      unfold<V>(o[0], r);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const int c = c0 + 8 * k;
        const float4 w = tab[c];
        float u[V];
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = fmaf((y[k][e] - m[e]) * r[e], w.z, w.w);
        if (active && c < a.C) ck_store<DT>(a.u, ((size_t)b * a.C + c) * P + p, whole ? 8 : P - p, ck_raw<DT>(u));
      }
    }
  }
}

// Backward of a field. The wave's registers hold v, gy and gu as stored and y
// (then gx) in fp32; v^ is formed again from v where it is needed.
template <int DT, int CPT, int WPT, int KIND>
__global__ __launch_bounds__(norm_threads<WPT>()) __attribute__((amdgpu_waves_per_eu(2))) void fno_norm_bwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), PX = 8 * V, WAVES = norm_threads<WPT>() / 64, TPG = WAVES / WPT, NC = 8 * CPT * WPT;
  __shared__ float4 tab[NC];
  __shared__ float4 sums[TPG > 1 ? TPG * NC : NC];
  __shared__ float red[WPT > 1 ? 2 * WAVES * 2 * PX : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.y;
  norm_table<DT>(a, b, NC, tab);
  __syncthreads();
  const int pl = lane & 7, c0 = (wave % WPT) * 8 * CPT + (lane >> 3);
  const long P = a.P, nt = (P + PX - 1) / PX, per = (nt + gridDim.x - 1) / gridDim.x;
  const long t0 = blockIdx.x * per, t1 = min(nt, t0 + per), nb = (P + kCkBlock - 1) / kCkBlock;
  const float invC = 1.f / (float)a.C;
  int turn = 0;
  float accT[CPT], accG[CPT], accU[CPT], accV[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) accT[k] = accG[k] = accU[k] = accV[k] = 0.f;
  for (long tt = t0; tt < t1; tt += TPG) {
    const long t = tt + wave / WPT;
    const bool active = t < t1;
    if (WPT == 1 && !active) break;
    const long p = t * PX + pl * V;
    const bool whole = active && (t + 1) * PX <= P;
    ck_u32x4 vr[CPT], xr[CPT], gyr[CPT], gur[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const int c = c0 + 8 * k;
      const bool ok = active && c < a.C;
      const size_t row = (size_t)b * a.C + (c < a.C ? c : 0);
      if (a.vq) {
        vr[k] = norm_decode<DT>(a.vq, a.ve, row, p, nb, ok);
        xr[k] = norm_decode<DT>(a.xq, a.xe, row, p, nb, ok);
      } else {
        vr[k] = norm_load<DT>(a.v, row, p, P, whole, ok);
        xr[k] = norm_load<DT>(a.x, row, p, P, whole, ok);
      }
      gyr[k] = norm_load<DT>(a.gy, row, p, P, whole, ok);
      gur[k] = ck_u32x4{0u, 0u, 0u, 0u};
      if (a.gu) gur[k] = norm_load<DT>(a.gu, row, p, P, whole, ok);
    }
    float s[1][V], o[1][V / 4], m[V], r[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = 0.f;
    if constexpr (KIND == kLayer) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0][e] = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) s[0][e] += ck_get<DT>(vr[k], e);
      }
      fold<V>(s[0], o[0]);
      Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) o[0][i] /= (float)a.C;
      unfold<V>(o[0], m);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      s[0][e] = 0.f;
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        float d = ck_get<DT>(vr[k], e) - m[e];
        if (KIND == kLayer && c0 + 8 * k >= a.C) d = 0.f;
        s[0][e] = fmaf(d, d, s[0][e]);
      }
    }
    fold<V>(s[0], o[0]);
    Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) o[0][i] = rsq(fmaf(o[0][i], invC, a.eps));
    unfold<V>(o[0], r);
    float y[CPT][V];
    if (a.gu) {
      float my[V], ry[V];
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float4 w = tab[c0 + 8 * k];
#pragma unroll
        for (int e = 0; e < V; ++e)
          y[k][e] = ck_get<DT>(xr[k], e) + fmaf((ck_get<DT>(vr[k], e) - m[e]) * r[e], w.x, w.y);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) my[e] = 0.f;
      if constexpr (KIND == kLayer) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          s[0][e] = 0.f;
#pragma unroll
          for (int k = 0; k < CPT; ++k) s[0][e] += y[k][e];
        }
        fold<V>(s[0], o[0]);
        Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) o[0][i] /= (float)a.C;
        unfold<V>(o[0], my);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0][e] = 0.f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          float d = y[k][e] - my[e];
          if (KIND == kLayer && c0 + 8 * k >= a.C) d = 0.f;
          s[0][e] = fmaf(d, d, s[0][e]);
        }
      }
      fold<V>(s[0], o[0]);
      Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) o[0][i] = rsq(fmaf(o[0][i], invC, a.eps));
      unfold<V>(o[0], ry);
      float q[2][V], oq[2][V / 4];
#pragma unroll
      for (int e = 0; e < V; ++e) q[0][e] = q[1][e] = 0.f;
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float wp = tab[c0 + 8 * k].z;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float gu = ck_get<DT>(gur[k], e), yh = (y[k][e] - my[e]) * ry[e];
          y[k][e] = yh;
          accU[k] = fmaf(gu, yh, accU[k]);
          accV[k] += gu;
          q[0][e] = fmaf(gu * wp, yh, q[0][e]);
          if (KIND == kLayer) q[1][e] = fmaf(gu, wp, q[1][e]);
        }
      }
      fold<V>(q[0], oq[0]);
      if (KIND == kLayer) fold<V>(q[1], oq[1]);
      else
#pragma unroll
        for (int i = 0; i < V / 4; ++i) oq[1][i] = 0.f;
      Join<2, V, WPT>::run(oq, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        oq[0][i] *= invC;
        oq[1][i] *= invC;
      }
      unfold<V>(oq[0], q[0]);
      if (KIND == kLayer) unfold<V>(oq[1], q[1]);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float wp = tab[c0 + 8 * k].z;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float g = fmaf(-y[k][e], q[0][e], ck_get<DT>(gur[k], e) * wp);
          if (KIND == kLayer) g -= q[1][e];
          y[k][e] = fmaf(ry[e], g, ck_get<DT>(gyr[k], e));
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) y[k][e] = ck_get<DT>(gyr[k], e);
    }
    // y holds gx
    float q[2][V], oq[2][V / 4];
#pragma unroll
    for (int e = 0; e < V; ++e) q[0][e] = q[1][e] = 0.f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const int c = c0 + 8 * k;
      const float w = tab[c].x;
      if (a.gx && active && c < a.C)
        ck_store<DT>(a.gx, ((size_t)b * a.C + c) * P + p, whole ? 8 : P - p, ck_raw<DT>(y[k]));
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float vh = (ck_get<DT>(vr[k], e) - m[e]) * r[e], g = y[k][e];
        accT[k] = fmaf(g, vh, accT[k]);
        accG[k] += g;
        q[0][e] = fmaf(g * w, vh, q[0][e]);
        if (KIND == kLayer) q[1][e] = fmaf(g, w, q[1][e]);
      }
    }
    fold<V>(q[0], oq[0]);
    if (KIND == kLayer) fold<V>(q[1], oq[1]);
    else
#pragma unroll
      for (int i = 0; i < V / 4; ++i) oq[1][i] = 0.f;
    Join<2, V, WPT>::run(oq, red, turn, wave, lane);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      oq[0][i] *= invC;
      oq[1][i] *= invC;
    }
    unfold<V>(oq[0], q[0]);
    if (KIND == kLayer) unfold<V>(oq[1], q[1]);
    if (a.gv) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const int c = c0 + 8 * k;
        const float w = tab[c].x;
        float gv[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float vh = (ck_get<DT>(vr[k], e) - m[e]) * r[e];
          float g = fmaf(-vh, q[0][e], y[k][e] * w);
          if (KIND == kLayer) g -= q[1][e];
          gv[e] = r[e] * g;
        }
        if (active && c < a.C) ck_store<DT>(a.gv, ((size_t)b * a.C + c) * P + p, whole ? 8 : P - p, ck_raw<DT>(gv));
      }
    }
  }
  if (!a.part) return;
  // the run's sums: over a channel's 8 lanes, then over the workgroup's tiles
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const float4 t = make_float4(sum8(accT[k]), sum8(accG[k]), sum8(accU[k]), sum8(accV[k]));
    if (pl == 0) sums[(wave / WPT) * NC + c0 + 8 * k] = t;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * NC; i += blockDim.x) {
    const int c = i >> 2, q = i & 3;
    if (c >= a.C) continue;
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < TPG; ++g) t += reinterpret_cast<const float *>(sums + g * NC + c)[q];
    a.part[(((size_t)q * a.C + c) * a.B + b) * gridDim.x + blockIdx.x] = t;
  }
}

// Parameter gradients of a field from the runs' sums part[4][C][B][S]: one
// workgroup per channel, a wave per sample in turn.
template <int DT>
__global__ __launch_bounds__(256) void fno_norm_params(NormArgs a, int S) {
  __shared__ float red[4][5];
  const int c = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float w = param(a.w_post, DT, c, 1.f), bp = param(a.b_post, DT, c, 0.f), sc = param(a.scale, DT, c, 1.f);
  const size_t kstep = (size_t)a.C * a.B * S;
  float t[5] = {0.f, 0.f, 0.f, 0.f, 0.f};  // sums over b of gate T, gate G, U, V and gate (w_post T + b_post G)
  for (int b = wave; b < a.B; b += 4) {
    const float *src = a.part + ((size_t)c * a.B + b) * S;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = lane; i < S; i += 64)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += src[q * kstep + i];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = sum64(v[q]);
    const float g = param(a.gate, DT, (size_t)b * a.C + c, 1.f), n = fmaf(w, v[0], bp * v[1]);
    if (lane == 0) put<DT>(a.g_gate, (size_t)b * a.C + c, sc * n);
    t[0] = fmaf(g, v[0], t[0]);
    t[1] = fmaf(g, v[1], t[1]);
    t[2] += v[2];
    t[3] += v[3];
    t[4] = fmaf(g, n, t[4]);
  }
  if (lane == 0)
#pragma unroll
    for (int q = 0; q < 5; ++q) red[wave][q] = t[q];
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int q = 0; q < 5; ++q) t[q] = (red[0][q] + red[1][q]) + (red[2][q] + red[3][q]);
  put<DT>(a.g_w_post, c, sc * t[0]);
  put<DT>(a.g_b_post, c, sc * t[1]);
  put<DT>(a.g_w_pre, c, t[2]);
  put<DT>(a.g_b_pre, c, t[3]);
  put<DT>(a.g_scale, c, t[4]);
}

// ------------------------------------------------------------ token layout

namespace {

template <int NT>
constexpr int tok_threads() { return NT > 256 ? NT : 256; }

// sums of NQ values over a row's NT threads
template <int NT, int NQ>
__device__ __forceinline__ void row_sum(float (&s)[NQ], float *red, int &turn) {
#pragma unroll
  for (int q = 0; q < NQ; ++q) s[q] = sum64(s[q]);
  if constexpr (NT > 64) {
    constexpr int W = NT / 64;
    float *buf = red + (turn & 1) * 2 * W;
    ++turn;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int q = 0; q < NQ; ++q) buf[q * W + wave] = s[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      s[q] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s[q] += buf[q * W + w];
    }
  }
}

// the elements' squared distance from m; elements past n do not count
template <int V>
__device__ __forceinline__ float dev2(const float *h, float m, long n) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float d = e < n ? h[e] - m : 0.f;
    s = fmaf(d, d, s);
  }
  return s;
}

// parameter values of 16 bytes' worth of channels, `none` where there is no parameter
template <int DT>
__device__ __forceinline__ void tok_param(const void *p, size_t i, long n, float none, float *v) {
  constexpr int V = ck_vec<DT>();
  if (p) {
    const ck_u32x4 r = ck_load<DT>(p, i, n);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = ck_get<DT>(r, e);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = none;
  }
}

}  // namespace

// NT threads hold a row, CH 16-byte pieces each
template <int DT, int NT, int CH, int KIND>
__global__ __launch_bounds__(tok_threads<NT>()) void fno_norm_tok_fwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), RPG = tok_threads<NT>() / NT;
  __shared__ float red[NT > 64 ? 4 * (NT / 64) : 1];
  const int t = threadIdx.x % NT, C = a.C;
  const float invC = 1.f / (float)C;
  const long nb = (C + kCkBlock - 1) / kCkBlock;
  int turn = 0;
  for (long b = (long)blockIdx.x * RPG + threadIdx.x / NT; b < a.B; b += (long)gridDim.x * RPG) {
    ck_u32x4 vr[CH], xr[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const long c = (long)(j * NT + t) * V;
      vr[j] = ck_load<DT>(a.v, (size_t)b * C + c, C - c);
      xr[j] = ck_load<DT>(a.x, (size_t)b * C + c, C - c);
    }
    if (a.vq) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const long c = (long)(j * NT + t) * V;
        norm_encode<DT>(vr[j], a.vq, a.ve, b, c, nb, true);
        norm_encode<DT>(xr[j], a.xq, a.xe, b, c, nb, true);
      }
    }
    float h[CH][V], s[1], m = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) h[j][e] = ck_get<DT>(vr[j], e);
    if constexpr (KIND == kLayer) {
      s[0] = 0.f;
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += h[j][e];
      row_sum<NT, 1>(s, red, turn);
      m = s[0] / (float)C;
    }
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) s[0] += dev2<V>(h[j], m, C - (long)(j * NT + t) * V);
    row_sum<NT, 1>(s, red, turn);
    const float r = rsq(fmaf(s[0], invC, a.eps));
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const long c = (long)(j * NT + t) * V, n = C - c;
      float g[V], sc[V], w[V], bp[V];
      tok_param<DT>(a.gate, (size_t)b * C + c, n, 1.f, g);
      tok_param<DT>(a.scale, c, n, 1.f, sc);
      tok_param<DT>(a.w_post, c, n, 1.f, w);
      tok_param<DT>(a.b_post, c, n, 0.f, bp);
#pragma unroll
      for (int e = 0; e < V; ++e)
        h[j][e] = ck_get<DT>(xr[j], e) + sc[e] * g[e] * fmaf((h[j][e] - m) * r, w[e], bp[e]);
      ck_store<DT>(a.y, (size_t)b * C + c, n, ck_raw<DT>(h[j]));
    }
    if (!a.u) continue;
    m = 0.f;
    if constexpr (KIND == kLayer) {
      s[0] = 0.f;
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += e < C - (long)(j * NT + t) * V ? h[j][e] : 0.f;
      row_sum<NT, 1>(s, red, turn);
      m = s[0] / (float)C;
    }
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) s[0] += dev2<V>(h[j], m, C - (long)(j * NT + t) * V);
    row_sum<NT, 1>(s, red, turn);
    const float ry = rsq(fmaf(s[0], invC, a.eps));
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const long c = (long)(j * NT + t) * V, n = C - c;
      float w[V], bp[V];
      tok_param<DT>(a.w_pre, c, n, 1.f, w);
      tok_param<DT>(a.b_pre, c, n, 0.f, bp);
#pragma unroll
      for (int e = 0; e < V; ++e) h[j][e] = fmaf((h[j][e] - m) * ry, w[e], bp[e]);
      ck_store<DT>(a.u, (size_t)b * C + c, n, ck_raw<DT>(h[j]));
    }
  }
}

// Backward of tokens; the column sums of a workgroup's rows (gate T, gate G, U, V)
// stay in registers and go to part[workgroup][4][C].
template <int DT, int NT, int CH, int KIND>
__global__ __launch_bounds__(tok_threads<NT>()) void fno_norm_tok_bwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), RPG = tok_threads<NT>() / NT;
  __shared__ float red[NT > 64 ? 4 * (NT / 64) : 1];
  __shared__ float sums[RPG > 1 ? RPG * NT * V : 1];
  const int t = threadIdx.x % NT, C = a.C;
  const float invC = 1.f / (float)C;
  const long nb = (C + kCkBlock - 1) / kCkBlock;
  int turn = 0;
  float acc[4][CH][V];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[q][j][e] = 0.f;
  for (long b = (long)blockIdx.x * RPG + threadIdx.x / NT; b < a.B; b += (long)gridDim.x * RPG) {
    ck_u32x4 vr[CH], xr[CH], gyr[CH], gur[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const long c = (long)(j * NT + t) * V, n = C - c;
      if (a.vq) {
        vr[j] = norm_decode<DT>(a.vq, a.ve, b, c, nb, true);
        xr[j] = norm_decode<DT>(a.xq, a.xe, b, c, nb, true);
      } else {
        vr[j] = ck_load<DT>(a.v, (size_t)b * C + c, n);
        xr[j] = ck_load<DT>(a.x, (size_t)b * C + c, n);
      }
      gyr[j] = ck_load<DT>(a.gy, (size_t)b * C + c, n);
      gur[j] = ck_u32x4{0u, 0u, 0u, 0u};
      if (a.gu) gur[j] = ck_load<DT>(a.gu, (size_t)b * C + c, n);
    }
    float vh[CH][V], y[CH][V], s[1], m = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) vh[j][e] = ck_get<DT>(vr[j], e);
    if constexpr (KIND == kLayer) {
      s[0] = 0.f;
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += vh[j][e];
      row_sum<NT, 1>(s, red, turn);
      m = s[0] / (float)C;
    }
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) s[0] += dev2<V>(vh[j], m, C - (long)(j * NT + t) * V);
    row_sum<NT, 1>(s, red, turn);
    const float r = rsq(fmaf(s[0], invC, a.eps));
    float q[2];
    if (a.gu) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const long c = (long)(j * NT + t) * V, n = C - c;
        float g[V], sc[V], w[V], bp[V];
        tok_param<DT>(a.gate, (size_t)b * C + c, n, 1.f, g);
        tok_param<DT>(a.scale, c, n, 1.f, sc);
        tok_param<DT>(a.w_post, c, n, 1.f, w);
        tok_param<DT>(a.b_post, c, n, 0.f, bp);
#pragma unroll
        for (int e = 0; e < V; ++e)
          y[j][e] = ck_get<DT>(xr[j], e) + sc[e] * g[e] * fmaf((vh[j][e] - m) * r, w[e], bp[e]);
      }
      float my = 0.f;
      if constexpr (KIND == kLayer) {
        s[0] = 0.f;
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) s[0] += e < C - (long)(j * NT + t) * V ? y[j][e] : 0.f;
        row_sum<NT, 1>(s, red, turn);
        my = s[0] / (float)C;
      }
      s[0] = 0.f;
#pragma unroll
      for (int j = 0; j < CH; ++j) s[0] += dev2<V>(y[j], my, C - (long)(j * NT + t) * V);
      row_sum<NT, 1>(s, red, turn);
      const float ry = rsq(fmaf(s[0], invC, a.eps));
      q[0] = q[1] = 0.f;
      float gp[CH][V];
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const long c = (long)(j * NT + t) * V, n = C - c;
        tok_param<DT>(a.w_pre, c, n, 1.f, gp[j]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float gu = ck_get<DT>(gur[j], e);
          y[j][e] = (y[j][e] - my) * ry;
          acc[2][j][e] = fmaf(gu, y[j][e], acc[2][j][e]);
          acc[3][j][e] += gu;
          gp[j][e] *= gu;
          q[0] = fmaf(gp[j][e], y[j][e], q[0]);
          if (KIND == kLayer) q[1] += gp[j][e];
        }
      }
      row_sum<NT, 2>(q, red, turn);
      q[0] *= invC;
      q[1] *= invC;
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float g = fmaf(-y[j][e], q[0], gp[j][e]);
          if (KIND == kLayer) g -= q[1];
          y[j][e] = fmaf(ry, g, ck_get<DT>(gyr[j], e));
        }
    } else {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) y[j][e] = ck_get<DT>(gyr[j], e);
    }
    // y holds gx, h below the gradient of v^
    float h[CH][V];
    q[0] = q[1] = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const long c = (long)(j * NT + t) * V, n = C - c;
      if (a.gx) ck_store<DT>(a.gx, (size_t)b * C + c, n, ck_raw<DT>(y[j]));
      float g[V], sc[V], w[V], bp[V], gg[V];
      tok_param<DT>(a.gate, (size_t)b * C + c, n, 1.f, g);
      tok_param<DT>(a.scale, c, n, 1.f, sc);
      tok_param<DT>(a.w_post, c, n, 1.f, w);
      tok_param<DT>(a.b_post, c, n, 0.f, bp);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float vv = e < n ? (vh[j][e] - m) * r : 0.f, gx = e < n ? y[j][e] : 0.f;
        vh[j][e] = vv;
        gg[e] = gx * sc[e] * fmaf(vv, w[e], bp[e]);
        acc[0][j][e] = fmaf(gx * g[e], vv, acc[0][j][e]);
        acc[1][j][e] = fmaf(gx, g[e], acc[1][j][e]);
        h[j][e] = gx * sc[e] * g[e] * w[e];
        q[0] = fmaf(h[j][e], vv, q[0]);
        if (KIND == kLayer) q[1] += h[j][e];
      }
      if (a.g_gate) ck_store<DT>(a.g_gate, (size_t)b * C + c, n, ck_raw<DT>(gg));
    }
    row_sum<NT, 2>(q, red, turn);
    if (!a.gv) continue;
    q[0] *= invC;
    q[1] *= invC;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const long c = (long)(j * NT + t) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float g = fmaf(-vh[j][e], q[0], h[j][e]);
        if (KIND == kLayer) g -= q[1];
        h[j][e] = r * g;
      }
      ck_store<DT>(a.gv, (size_t)b * C + c, C - c, ck_raw<DT>(h[j]));
    }
  }
  if (!a.part) return;
  float *out = a.part + (size_t)blockIdx.x * 4 * C;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const long c = (long)(j * NT + t) * V;
      if constexpr (RPG > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) sums[((threadIdx.x / NT) * NT + t) * V + e] = acc[q][j][e];
        __syncthreads();
        for (int i = threadIdx.x; i < NT * V; i += tok_threads<NT>()) {
          const long cc = (long)j * NT * V + i;
          if (cc >= C) continue;
          float v = 0.f;
#pragma unroll
          for (int g = 0; g < RPG; ++g) v += sums[g * NT * V + i];
          out[(size_t)q * C + cc] = v;
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c + e < C) out[(size_t)q * C + c + e] = acc[q][j][e];
      }
    }
}

// Parameter gradients of tokens from part[S][4][C]: 32 channels a workgroup,
// 32 slices of the runs.
template <int DT>
__global__ __launch_bounds__(1024) void fno_norm_tok_params(NormArgs a, int S) {
  __shared__ float red[4][32][33];
  const int l = threadIdx.x & 31, sl = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < a.C)
    for (int i = sl; i < S; i += 32)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += a.part[((size_t)i * 4 + q) * a.C + c];
#pragma unroll
  for (int q = 0; q < 4; ++q) red[q][sl][l] = v[q];
  __syncthreads();
  if (threadIdx.x >= 32 || c >= a.C) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = 0.f;
    for (int i = 0; i < 32; ++i) v[q] += red[q][i][l];
  }
  const float w = param(a.w_post, DT, c, 1.f), bp = param(a.b_post, DT, c, 0.f), sc = param(a.scale, DT, c, 1.f);
  put<DT>(a.g_w_post, c, sc * v[0]);
  put<DT>(a.g_b_post, c, sc * v[1]);
  put<DT>(a.g_w_pre, c, v[2]);
  put<DT>(a.g_b_pre, c, v[3]);
  put<DT>(a.g_scale, c, fmaf(w, v[0], bp * v[1]));
}

// ------------------------------------------------------------------ launch

namespace {

template <int DT, int KIND>
const void *field_kernel(bool fwd, int C) {
#define FNO_PICK(CPT, WPT) \
  (fwd ? (const void *)fno_norm_fwd<DT, CPT, WPT, KIND> : (const void *)fno_norm_bwd<DT, CPT, WPT, KIND>)
  if (C <= 8) return FNO_PICK(1, 1);
  if (C <= 16) return FNO_PICK(2, 1);
  if (C <= 32) return FNO_PICK(4, 1);
  if (C <= 64) return FNO_PICK(8, 1);
  if (C <= 128) return FNO_PICK(8, 2);
  if (C <= 256) return FNO_PICK(8, 4);
  return FNO_PICK(8, 8);
#undef FNO_PICK
}

template <int DT, int KIND>
const void *tok_kernel(bool fwd, int C, int &threads, int &rpg) {
#define FNO_PICK(NT, CH)                                       \
  (threads = tok_threads<NT>(), rpg = tok_threads<NT>() / NT,  \
   fwd ? (const void *)fno_norm_tok_fwd<DT, NT, CH, KIND> : (const void *)fno_norm_tok_bwd<DT, NT, CH, KIND>)
  if constexpr (DT == DT_F32) {
    if (C <= 256) return FNO_PICK(64, 1);
    if (C <= 512) return FNO_PICK(64, 2);
    if (C <= 1024) return FNO_PICK(64, 4);
    if (C <= 2048) return FNO_PICK(256, 2);
    if (C <= 4096) return FNO_PICK(256, 4);
    return FNO_PICK(512, 4);
  } else {
    if (C <= 512) return FNO_PICK(64, 1);
    if (C <= 1024) return FNO_PICK(64, 2);
    if (C <= 2048) return FNO_PICK(256, 1);
    if (C <= 4096) return FNO_PICK(256, 2);
    return FNO_PICK(512, 2);
  }
#undef FNO_PICK
}

template <int DT>
const void *any_kernel(bool tok, int kind, bool fwd, int C, int &threads, int &rpg) {
  if (tok) return kind == kLayer ? tok_kernel<DT, kLayer>(fwd, C, threads, rpg) : tok_kernel<DT, kRms>(fwd, C, threads, rpg);
  threads = C > 256 ? 512 : 256;
  rpg = C <= 64 ? 4 : C <= 128 ? 2 : 1;  // tiles a workgroup handles at once
  return kind == kLayer ? field_kernel<DT, kLayer>(fwd, C) : field_kernel<DT, kRms>(fwd, C);
}

const void *pick(const NormArgs &a, bool fwd, int dtype, int &threads, int &rpg) {
  const bool tok = a.P == 1;
  if (dtype == DT_F32) return any_kernel<DT_F32>(tok, a.kind, fwd, a.C, threads, rpg);
  if (dtype == DT_F16) return any_kernel<DT_F16>(tok, a.kind, fwd, a.C, threads, rpg);
  return any_kernel<DT_BF16>(tok, a.kind, fwd, a.C, threads, rpg);
}

// Runs per sample (fields) or in all (tokens). Backward: about 1024 in all,
// two rounds of the workgroups the chip holds at two waves per SIMD.
constexpr long kNormRuns = 1024;
long norm_runs(const NormArgs &a, int dtype, int rpg, long most) {
  if (a.P == 1) return std::min((a.B + (long)rpg - 1) / rpg, most);
  const long px = dtype == DT_F32 ? 32 : 64, nt = (a.P + px - 1) / px;
  return std::min((nt + rpg - 1) / rpg, std::max(1L, (most + a.B - 1) / a.B));
}

}  // namespace

size_t norm_workspace_bytes(int B, int C, long P, int dtype) {
  NormArgs a{};
  a.B = B, a.C = C, a.P = P;
  int threads, rpg;
  (void)pick(a, false, dtype, threads, rpg);
  const long S = norm_runs(a, dtype, rpg, kNormRuns);
  return (size_t)4 * C * S * (P == 1 ? 1 : B) * 4;
}

hipError_t launch_norm_fwd(const NormArgs &a, int dtype, hipStream_t s) {
  FNO_BOUNDS(check_norm(a, true, 0, dtype);)
  int threads, rpg;
  const void *k = pick(a, true, dtype, threads, rpg);
  const long S = norm_runs(a, dtype, rpg, 4 * kNormRuns);
  const dim3 grid((unsigned)S, a.P == 1 ? 1u : (unsigned)a.B);
  NormArgs arg = a;
  void *args[] = {(void *)&arg};
  return hipLaunchKernel(k, grid, dim3((unsigned)threads), args, 0, s);
}

hipError_t launch_norm_bwd(const NormArgs &a, int dtype, hipStream_t s) {
  int threads, rpg;
  const void *k = pick(a, false, dtype, threads, rpg);
  int S = (int)norm_runs(a, dtype, rpg, kNormRuns);
  FNO_BOUNDS(check_norm(a, false, S, dtype);)
  const bool tok = a.P == 1;
  const dim3 grid((unsigned)S, tok ? 1u : (unsigned)a.B);
  NormArgs arg = a;
  void *args[] = {(void *)&arg};
  hipError_t e = hipLaunchKernel(k, grid, dim3((unsigned)threads), args, 0, s);
  if (e != hipSuccess || !a.part) return e;
  void *pargs[] = {(void *)&arg, (void *)&S};
#define FNO_PICK(DT) (tok ? (const void *)fno_norm_tok_params<DT> : (const void *)fno_norm_params<DT>)
  const void *pk = dtype == DT_F32 ? FNO_PICK(DT_F32) : dtype == DT_F16 ? FNO_PICK(DT_F16) : FNO_PICK(DT_BF16);
#undef FNO_PICK
  return hipLaunchKernel(pk, dim3((unsigned)(tok ? (a.C + 31) / 32 : a.C)), dim3(tok ? 1024u : 256u), pargs, 0, s);
}

}  // namespace fno
