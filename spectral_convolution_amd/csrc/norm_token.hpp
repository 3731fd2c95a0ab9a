// norm_token.hpp - forward and backward of the norms around a block on tokens
// (norm.hip has the mathematics and the design).
#pragma once

#include "norm_common.hpp"

namespace fno {

// the tokens' form of decode and encode: 16 bytes' worth of channels from c on
template <int DT>
__device__ __forceinline__ ck_u32x4 norm_decode(const uint8_t *q, const int8_t *e, size_t row, long p, long nb) {
  if (p >= nb * kCkBlock) return ck_u32x4{0u, 0u, 0u, 0u};
  const uint8_t *s = q + row * nb * kCkBlock + p;
  uint2 c;
  if constexpr (DT == DT_F32) c = make_uint2(*reinterpret_cast<const uint32_t *>(s), 0u);
  else c = *reinterpret_cast<const uint2 *>(s);
  return ck_decode<DT>(c, e[row * nb + p / kCkBlock]);
}

template <int DT>
__device__ __forceinline__ void norm_encode(const ck_u32x4 &r, uint8_t *q, int8_t *e, size_t row, long p, long nb) {
  constexpr int L = kCkBlock / ck_vec<DT>();
  const int ex = ck_exponent<DT>(ck_groupmax<L>(ck_maxkey<DT>(r)));
  const uint2 c = ck_codes<DT>(r, ex);
  if (p >= nb * kCkBlock) return;
  uint8_t *d = q + row * nb * kCkBlock + p;
  if constexpr (DT == DT_F32) *reinterpret_cast<uint32_t *>(d) = c.x;
  else *reinterpret_cast<uint2 *>(d) = c;
  if (p % kCkBlock == 0) e[row * nb + p / kCkBlock] = (int8_t)ex;
}

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
        norm_encode<DT>(vr[j], a.vq, a.ve, b, c, nb);
        norm_encode<DT>(xr[j], a.xq, a.xe, b, c, nb);
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
        vr[j] = norm_decode<DT>(a.vq, a.ve, b, c, nb);
        xr[j] = norm_decode<DT>(a.xq, a.xe, b, c, nb);
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

}  // namespace fno
