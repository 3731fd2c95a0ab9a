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
constexpr int tok_threads() { return NT > 64 ? NT : 256; }

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

// 16 bytes of a row of C channels for channel c on. A lane that would pass the
// row's end reads its last 16 bytes; tok_fix moves them into place once all of a
// row's loads are on their way (element by element, each load waited for, that lane
// took longer than the rest of the row: 76 us instead of 21 at 16000 x 100, bf16).
// Rows shorter than 16 bytes are read by the element.
template <int DT>
__device__ __forceinline__ ck_u32x4 tok_load(const void *p, size_t row, int c, int C) {
  constexpr int V = ck_vec<DT>(), ES = DT == DT_F32 ? 4 : 2;
  if (C < V) return ck_load<DT>(p, row, c == 0 ? C : 0);
  return *reinterpret_cast<const ck_u32x4_any *>(static_cast<const char *>(p) + (row + min(c, C - V)) * ES);
}

// the same of a parameter, `none` for each channel where there is no parameter
template <int DT>
__device__ __forceinline__ ck_u32x4 tok_param(const void *p, size_t row, int c, int C, float none) {
  constexpr int V = ck_vec<DT>();
  if (p) return tok_load<DT>(p, row, c, C);
  float v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = C >= V || e < C ? none : 0.f;
  return ck_raw<DT>(v);
}

// what tok_load and tok_param gave for channel c on, in place, zeros past the row's end
template <int DT>
__device__ __forceinline__ ck_u32x4 tok_fix1(const ck_u32x4 &r, int c, int C) {
  constexpr int V = ck_vec<DT>(), ES = DT == DT_F32 ? 4 : 2;
  if (C % V == 0 || C < V) return c < C ? r : ck_u32x4{0u, 0u, 0u, 0u};
  return ck_shift(r, min(max(c - (C - V), 0), V) * ES);
}
template <int DT, int NT, int CH>
__device__ __forceinline__ void tok_fix(ck_u32x4 (&r)[CH], int t, int C) {
  constexpr int V = ck_vec<DT>();
  if (C == NT * CH * V) return;
#pragma unroll
  for (int j = 0; j < CH; ++j) r[j] = tok_fix1<DT>(r[j], (j * NT + t) * V, C);
}

// NT threads hold a row, CH 16-byte pieces each. Parameters are loaded where they
// are used: held from the start they cost more in waves than their latency does (8192
// x 1024 bf16, the forward as it was then: 29.4 us instead of 26.3).
template <int DT, int NT, int CH, int KIND>
__global__ __launch_bounds__(tok_threads<NT>()) void fno_norm_tok_fwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), RPG = tok_threads<NT>() / NT;
  __shared__ float red[NT > 64 ? 4 * (NT / 64) : 1];
  const int t = threadIdx.x % NT, C = a.C;
  const float invC = 1.f / (float)C;
  const long nb = (C + kCkBlock - 1) / kCkBlock;
  int turn = 0;
  auto get = [&](const void *p, int j, float none) {
    const int c = (j * NT + t) * V;
    const ck_u32x4 r = tok_param<DT>(p, 0, c, C, none);
    return C == NT * CH * V ? r : tok_fix1<DT>(r, c, C);
  };
  for (long b = (long)blockIdx.x * RPG + threadIdx.x / NT; b < a.B; b += (long)gridDim.x * RPG) {
    ck_u32x4 vr[CH], xr[CH], gr[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * NT + t) * V;
      vr[j] = tok_load<DT>(a.v, (size_t)b * C, c, C);
      xr[j] = tok_load<DT>(a.x, (size_t)b * C, c, C);
      gr[j] = tok_param<DT>(a.gate, (size_t)b * C, c, C, 1.f);
    }
    tok_fix<DT, NT, CH>(vr, t, C);
    tok_fix<DT, NT, CH>(xr, t, C);
    tok_fix<DT, NT, CH>(gr, t, C);
    if (a.vq) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const long c = (long)(j * NT + t) * V;
        norm_encode<DT>(vr[j], a.vq, a.ve, b, c, nb);
        norm_encode<DT>(xr[j], a.xq, a.xe, b, c, nb);
      }
    }
    // mean (layer norm) and inverse deviation of h(j, e)
    auto stats = [&](auto &&h, float &m, float &r) {
      float s[1] = {0.f};
      m = 0.f;
      if constexpr (KIND == kLayer) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) s[0] += h(j, e);
        row_sum<NT, 1>(s, red, turn);
        m = s[0] / (float)C;
        s[0] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = h(j, e) - m;
          s[0] += KIND == kRms || (j * NT + t) * V + e < C ? d * d : 0.f;
        }
      row_sum<NT, 1>(s, red, turn);
      r = rsq(fmaf(s[0], invC, a.eps));
    };
    float y[CH][V], m, r;
    stats([&](int j, int e) { return ck_get<DT>(vr[j], e); }, m, r);
    // with one piece u's parameters are loaded ahead of y's store, which they would wait for
    constexpr bool EARLY = CH == 1;
    ck_u32x4 wu, bu;
    if (EARLY && a.u) {
      wu = get(a.w_pre, 0, 1.f);
      bu = get(a.b_pre, 0, 0.f);
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const ck_u32x4 sc = get(a.scale, j, 1.f), w = get(a.w_post, j, 1.f), bp = get(a.b_post, j, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e)
        y[j][e] = fmaf(ck_get<DT>(sc, e) * ck_get<DT>(gr[j], e),
                       fmaf((ck_get<DT>(vr[j], e) - m) * r, ck_get<DT>(w, e), ck_get<DT>(bp, e)), ck_get<DT>(xr[j], e));
      const int c = (j * NT + t) * V;
      ck_store_row<DT>(a.y, (size_t)b * C + c, C - c, ck_raw<DT>(y[j]));
    }
    if (!a.u) continue;
    stats([&](int j, int e) { return y[j][e]; }, m, r);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const ck_u32x4 w = EARLY ? wu : get(a.w_pre, j, 1.f), bp = EARLY ? bu : get(a.b_pre, j, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e) y[j][e] = fmaf((y[j][e] - m) * r, ck_get<DT>(w, e), ck_get<DT>(bp, e));
      const int c = (j * NT + t) * V;
      ck_store_row<DT>(a.u, (size_t)b * C + c, C - c, ck_raw<DT>(y[j]));
    }
  }
}

// Backward of tokens, in the passes of a field's (norm_field.hpp). A row's
// fields and gate stay as stored and are converted again in each pass; scale,
// w_post, b_post and w_pre wait in LDS, a thread's own 16 bytes each; the column
// sums of a workgroup's rows (gate T, gate G, U, V) stay in registers and go
// to part[workgroup][4][C]. Stores come last in a row, so that no load waits
// for one.
template <int DT, int NT, int CH, int KIND>
__global__ __launch_bounds__(tok_threads<NT>()) __attribute__((amdgpu_waves_per_eu(2))) void fno_norm_tok_bwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), RPG = tok_threads<NT>() / NT;
  extern __shared__ ck_u32x4 prm[];  // [4][CH][NT]
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
  if (threadIdx.x < NT) {
    ck_u32x4 p[4][CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * NT + t) * V;
      p[0][j] = tok_param<DT>(a.scale, 0, c, C, 1.f);
      p[1][j] = tok_param<DT>(a.w_post, 0, c, C, 1.f);
      p[2][j] = tok_param<DT>(a.b_post, 0, c, C, 0.f);
      p[3][j] = tok_param<DT>(a.w_pre, 0, c, C, 1.f);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      tok_fix<DT, NT, CH>(p[q], t, C);
#pragma unroll
      for (int j = 0; j < CH; ++j) prm[(q * CH + j) * NT + t] = p[q][j];
    }
  }
  __syncthreads();
  for (long b = (long)blockIdx.x * RPG + threadIdx.x / NT; b < a.B; b += (long)gridDim.x * RPG) {
    ck_u32x4 vr[CH], xr[CH], gyr[CH], gur[CH], gr[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * NT + t) * V;
      if (a.vq) {
        vr[j] = norm_decode<DT>(a.vq, a.ve, b, c, nb);
        xr[j] = norm_decode<DT>(a.xq, a.xe, b, c, nb);
      } else {
        vr[j] = tok_load<DT>(a.v, (size_t)b * C, c, C);
        xr[j] = tok_load<DT>(a.x, (size_t)b * C, c, C);
      }
      gr[j] = tok_param<DT>(a.gate, (size_t)b * C, c, C, 1.f);
      gur[j] = ck_u32x4{0u, 0u, 0u, 0u};
      if (a.gu) gur[j] = tok_load<DT>(a.gu, (size_t)b * C, c, C);
      gyr[j] = tok_load<DT>(a.gy, (size_t)b * C, c, C);
    }
    if (!a.vq) {
      tok_fix<DT, NT, CH>(vr, t, C);
      tok_fix<DT, NT, CH>(xr, t, C);
    }
    tok_fix<DT, NT, CH>(gr, t, C);
    tok_fix<DT, NT, CH>(gur, t, C);
    tok_fix<DT, NT, CH>(gyr, t, C);
    auto at = [&](int q, int j) { return prm[(q * CH + j) * NT + t]; };
    auto in = [&](int j, int e) { return (j * NT + t) * V + e < C; };
    float s[1] = {0.f}, m = 0.f;
    if constexpr (KIND == kLayer) {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += ck_get<DT>(vr[j], e);
      row_sum<NT, 1>(s, red, turn);
      m = s[0] / (float)C;
      s[0] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = ck_get<DT>(vr[j], e) - m;
        s[0] += KIND == kRms || in(j, e) ? d * d : 0.f;
      }
    row_sum<NT, 1>(s, red, turn);
    const float r = rsq(fmaf(s[0], invC, a.eps));
    float y[CH][V], q[2];  // y, then gx
    fresh<DT>(vr);
    if (a.gu) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const ck_u32x4 sc = at(0, j), w = at(1, j), bp = at(2, j);
#pragma unroll
        for (int e = 0; e < V; ++e)
          y[j][e] = fmaf(ck_get<DT>(sc, e) * ck_get<DT>(gr[j], e),
                         fmaf((ck_get<DT>(vr[j], e) - m) * r, ck_get<DT>(w, e), ck_get<DT>(bp, e)), ck_get<DT>(xr[j], e));
        channel_done();
      }
      float my = 0.f;
      q[0] = q[1] = 0.f;
      if constexpr (KIND == kLayer) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          const ck_u32x4 w = at(3, j);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            q[0] += y[j][e];
            q[1] = fmaf(ck_get<DT>(gur[j], e), ck_get<DT>(w, e), q[1]);
          }
        }
        row_sum<NT, 2>(q, red, turn);
        my = q[0] / (float)C;
      }
      const float mg = q[1] * invC;  // mean of g = gu w_pre
      q[0] = q[1] = 0.f;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const ck_u32x4 w = at(3, j);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = KIND == kRms || in(j, e) ? y[j][e] - my : 0.f;
          y[j][e] = d;
          q[0] = fmaf(d, d, q[0]);
          q[1] = fmaf(ck_get<DT>(gur[j], e) * ck_get<DT>(w, e), d, q[1]);
        }
      }
      row_sum<NT, 2>(q, red, turn);
      const float ry = rsq(fmaf(q[0], invC, a.eps)), gy = q[1] * invC * ry;  // gy = mean(g y^)
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const ck_u32x4 w = at(3, j);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float gu = ck_get<DT>(gur[j], e), yh = y[j][e] * ry;
          acc[2][j][e] = fmaf(gu, yh, acc[2][j][e]);
          acc[3][j][e] += gu;
          float g = fmaf(-yh, gy, gu * ck_get<DT>(w, e));
          if (KIND == kLayer) g -= mg;
          y[j][e] = fmaf(ry, g, ck_get<DT>(gyr[j], e));
        }
        channel_done();
      }
    } else {
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) y[j][e] = ck_get<DT>(gyr[j], e);
    }
    fresh<DT>(vr);
    q[0] = q[1] = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const ck_u32x4 sc = at(0, j), w = at(1, j);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float vh = (ck_get<DT>(vr[j], e) - m) * r, gx = y[j][e], g = ck_get<DT>(gr[j], e), wv = ck_get<DT>(w, e);
        acc[0][j][e] = fmaf(gx * g, vh, acc[0][j][e]);
        acc[1][j][e] = fmaf(gx, g, acc[1][j][e]);
        const float h = gx * (ck_get<DT>(sc, e) * g * wv);
        q[0] = fmaf(h, vh, q[0]);
        if (KIND == kLayer) q[1] += h;
      }
      channel_done();
    }
    row_sum<NT, 2>(q, red, turn);
    const float hv = q[0] * invC, mh = q[1] * invC;
    fresh<DT>(vr);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * NT + t) * V;
      const size_t to = (size_t)b * C + c;
      if (a.gx) ck_store_row<DT>(a.gx, to, C - c, ck_raw<DT>(y[j]));
      const ck_u32x4 sc = at(0, j), w = at(1, j), bp = at(2, j);
      float gg[V], gv[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float vh = (ck_get<DT>(vr[j], e) - m) * r, s = ck_get<DT>(sc, e), wv = ck_get<DT>(w, e);
        gg[e] = y[j][e] * s * fmaf(vh, wv, ck_get<DT>(bp, e));
        // h rounded as in its mean above: over one channel the two are then equal and gv is 0
        float g = fmaf(-vh, hv, y[j][e] * (s * ck_get<DT>(gr[j], e) * wv));
        if (KIND == kLayer) g -= mh;
        gv[e] = r * g;
      }
      if (a.g_gate) ck_store_row<DT>(a.g_gate, to, C - c, ck_raw<DT>(gg));
      if (a.gv) ck_store_row<DT>(a.gv, to, C - c, ck_raw<DT>(gv));
      channel_done();
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

template <int DT, int KIND, bool FWD, int NT, int CH>
NormPick tok_pick() {
  if constexpr (FWD) return {(const void *)fno_norm_tok_fwd<DT, NT, CH, KIND>, tok_threads<NT>(), tok_threads<NT>() / NT, 0, NT, CH};
  else return {(const void *)fno_norm_tok_bwd<DT, NT, CH, KIND>, tok_threads<NT>(), tok_threads<NT>() / NT, (size_t)64 * CH * NT, NT, CH};
}

template <int DT, int KIND>
NormPick tok_kernel(bool fwd, int C) {
  // Forward: one piece a thread, so that many waves have loads in flight (8192 x 1024
  // bf16 in a kernel trace: 23.3 us with one, 27.8 with two). Backward: two where that needs no more
  // threads than 512, as each workgroup leaves sums to add (1024 x 8192 fp16: 71 us
  // with 512 threads, 105 with 1024); four, in fp32 above 4096 channels, spill 350 bytes a lane
  // (1024 x 8192 fp32: 116 us, 2.3 TB/s).
  if constexpr (DT == DT_F32) {
    if (C <= 256) return fwd ? tok_pick<DT, KIND, true, 64, 1>() : tok_pick<DT, KIND, false, 64, 1>();
    if (C <= 512) return fwd ? tok_pick<DT, KIND, true, 128, 1>() : tok_pick<DT, KIND, false, 128, 1>();
    if (C <= 1024) return fwd ? tok_pick<DT, KIND, true, 256, 1>() : tok_pick<DT, KIND, false, 256, 1>();
    if (C <= 2048) return fwd ? tok_pick<DT, KIND, true, 512, 1>() : tok_pick<DT, KIND, false, 256, 2>();
    if (C <= 4096) return fwd ? tok_pick<DT, KIND, true, 1024, 1>() : tok_pick<DT, KIND, false, 512, 2>();
    return fwd ? tok_pick<DT, KIND, true, 512, 4>() : tok_pick<DT, KIND, false, 512, 4>();
  } else {
    if (C <= 512) return fwd ? tok_pick<DT, KIND, true, 64, 1>() : tok_pick<DT, KIND, false, 64, 1>();
    if (C <= 1024) return fwd ? tok_pick<DT, KIND, true, 128, 1>() : tok_pick<DT, KIND, false, 64, 2>();
    if (C <= 2048) return fwd ? tok_pick<DT, KIND, true, 256, 1>() : tok_pick<DT, KIND, false, 256, 1>();
    if (C <= 4096) return fwd ? tok_pick<DT, KIND, true, 512, 1>() : tok_pick<DT, KIND, false, 512, 1>();
    return fwd ? tok_pick<DT, KIND, true, 1024, 1>() : tok_pick<DT, KIND, false, 512, 2>();
  }
}

}  // namespace fno
