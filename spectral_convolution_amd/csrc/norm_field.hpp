// norm_field.hpp - forward and backward of the norms around a block on fields
// (norm.hip has the mathematics and the design).
#pragma once

#include <algorithm>

#include "norm_common.hpp"

namespace fno {

// {scale gate w_post, scale gate b_post, w_pre, b_pre} of the channels of sample b
template <int DT>
__device__ __forceinline__ void norm_table(const NormArgs &a, int b, int n, float4 *tab) {
  const void *any = a.gy ? a.gy : a.x;  // a field: at least a sample's channels long
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    const int i = min(c, a.C - 1);
    const uint32_t sc = param_bits<DT>(a.scale, any, i), g = param_bits<DT>(a.gate, any, (size_t)b * a.C + i),
                   w = param_bits<DT>(a.w_post, any, i), bp = param_bits<DT>(a.b_post, any, i),
                   wu = param_bits<DT>(a.w_pre, any, i), bu = param_bits<DT>(a.b_pre, any, i);
    const float sg = param_value<DT>(a.scale, sc, 1.f) * param_value<DT>(a.gate, g, 1.f);
    const float4 t = make_float4(sg * param_value<DT>(a.w_post, w, 1.f), sg * param_value<DT>(a.b_post, bp, 0.f),
                                 param_value<DT>(a.w_pre, wu, 1.f), param_value<DT>(a.b_pre, bu, 0.f));
    tab[c] = c < a.C ? t : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// The pieces of a tile that a wave holds: its k-th group of 8 channels is group
// k WPT + (wave in tile), so only the last one can reach past the channels. Lane l
// has the 16 bytes of channel l / 8 of each group and of pixels V (l % 8) .. of the tile: a
// uniform base (sample, group, tile) plus one 32-bit offset that no loop
// changes, so an access takes no address registers of its own (P <= 2^27
// keeps 7 rows inside 32 bits).
template <int DT, int CPT, int WPT>
struct FieldTile {
  static constexpr int V = ck_vec<DT>(), PX = 8 * V, ES = DT == DT_F32 ? 4 : 2;
  long P, nb;  // row length and its blocks
  int sample, channels;
  int first;      // the wave's first group
  int last;       // its last group, or the field's where it has none
  int cl, clast;  // channel within a group, within the last one (clamped to the field's)
  int pl;
  bool ok;        // the lane's channel of the last group exists
  uint32_t off, off_last, code, code_last, exp, exp_last;

  __device__ __forceinline__ FieldTile(const NormArgs &a, int b, int lane, int w) {
    P = a.P;
    nb = (P + kCkBlock - 1) / kCkBlock;
    sample = b;
    channels = a.C;
    first = w;
    const int g = (CPT - 1) * WPT + w;
    last = min(g, (a.C - 1) / 8);
    cl = lane >> 3;
    pl = lane & 7;
    clast = min(cl, a.C - 1 - 8 * last);
    ok = 8 * g + cl < a.C;
    off = (uint32_t)cl * (uint32_t)P * ES + 16u * pl;
    off_last = (uint32_t)clast * (uint32_t)P * ES + 16u * pl;
    code = (uint32_t)cl * (uint32_t)nb * kCkBlock + (uint32_t)V * pl;
    code_last = (uint32_t)clast * (uint32_t)nb * kCkBlock + (uint32_t)V * pl;
    exp = (uint32_t)cl * (uint32_t)nb + (uint32_t)V * pl / kCkBlock;
    exp_last = (uint32_t)clast * (uint32_t)nb + (uint32_t)V * pl / kCkBlock;
  }
  // The tile being worked on: uniform byte offsets of the wave's first and last
  // groups in a field, its codes and its exponents. The lane offsets (and
  // the row length) pass through an opaque move, or the compiler adds them to
  // every base ahead of the loop and keeps the sums (40 register pairs in the
  // backward, spilled).
  size_t f0, f1, c0, c1, e0, e1;
  __device__ __forceinline__ void at(int t) {
    asm volatile("" : "+v"(off), "+v"(off_last), "+v"(code), "+v"(code_last), "+v"(exp), "+v"(exp_last));
    uint32_t p = (uint32_t)P;
    asm volatile("" : "+v"(p));
    P = __builtin_amdgcn_readfirstlane(p);
    nb = (P + kCkBlock - 1) / kCkBlock;
    const size_t r = (size_t)sample * channels;
    const size_t first_row = r + 8 * first, last_row = r + 8 * last;
    f0 = (first_row * P + (long)t * PX) * ES;
    f1 = (last_row * P + (long)t * PX) * ES;
    c0 = first_row * nb * kCkBlock + (long)t * PX;
    c1 = last_row * nb * kCkBlock + (long)t * PX;
    e0 = first_row * nb + (long)t * (PX / kCkBlock);
    e1 = last_row * nb + (long)t * (PX / kCkBlock);
  }
  __device__ __forceinline__ size_t field_at(int k) const { return k < CPT - 1 ? f0 + (size_t)k * 8 * WPT * P * ES : f1; }
  __device__ __forceinline__ size_t code_at(int k) const { return k < CPT - 1 ? c0 + (size_t)k * 8 * WPT * nb * kCkBlock : c1; }
  __device__ __forceinline__ size_t exp_at(int k) const { return k < CPT - 1 ? e0 + (size_t)k * 8 * WPT * nb : e1; }
  // whether the lane's channel of group k exists, and its place in the channel table
  __device__ __forceinline__ bool has(int k) const { return k < CPT - 1 || ok; }
  __device__ __forceinline__ int channel(int k) const { return 8 * (k * WPT + first) + cl; }

  __device__ __forceinline__ ck_u32x4 only(int k, const ck_u32x4 &r) const {
    return k < CPT - 1 || ok ? r : ck_u32x4{0u, 0u, 0u, 0u};
  }
  // a tile that lies within the row
  __device__ __forceinline__ ck_u32x4 load(const void *f, int t, int k) const {
    const char *s = static_cast<const char *>(f) + field_at(k);
    return only(k, __builtin_nontemporal_load(reinterpret_cast<const ck_u32x4_any *>(s + (k < CPT - 1 ? off : off_last))));
  }
  // The row's last tile, zeros past its end: a lane that would pass it reads the
  // row's last 16 bytes instead (`back` elements before its own) and shifts
  // them into place. Rows shorter than 16 bytes are read by the element.
  struct End {
    uint32_t off, off_last;  // lane offsets from 16 bytes before the tile
    int back;                // in bytes, 16 and more: nothing of the piece is in the row
    long n;
  };
  __device__ __forceinline__ End end(int t) const {
    End x;
    x.n = P - ((long)t * PX + pl * V);
    const int b = (int)max(0L, V - x.n) * ES;
    x.off = off + 16 - b;
    x.off_last = off_last + 16 - b;
    x.back = min(b, 16);
    return x;
  }
  __device__ __forceinline__ ck_u32x4 load_end(const void *f, const End &x, int k) const {
    const char *s = static_cast<const char *>(f) + field_at(k);
    if (P < V) return only(k, ck_load<DT>(s + (k < CPT - 1 ? off : off_last), 0, x.n));
    const ck_u32x4 r = *reinterpret_cast<const ck_u32x4_any *>(s - 16 + (k < CPT - 1 ? x.off : x.off_last));
    return only(k, ck_shift(r, x.back));
  }
  __device__ __forceinline__ void store(void *f, int t, int k, bool whole, const ck_u32x4 &r) const {
    if (!has(k)) return;
    if (whole) {
      char *d = static_cast<char *>(f) + field_at(k);
      __builtin_nontemporal_store((ck_u32x4_any)r, reinterpret_cast<ck_u32x4_any *>(d + (k < CPT - 1 ? off : off_last)));
    } else {
      ck_store_row<DT>(static_cast<char *>(f) + field_at(k) + (k < CPT - 1 ? off : off_last), 0, P - ((long)t * PX + pl * V), r);
    }
  }
  // whether the lane's piece begins inside the row's blocks
  __device__ __forceinline__ bool coded(int t) const { return (long)t * PX + pl * V < nb * kCkBlock; }
  __device__ __forceinline__ ck_u32x4 decode(const uint8_t *q, const int8_t *e, int t, int k) const {
    const uint8_t *s = q + code_at(k);
    uint2 c = make_uint2(0u, 0u);
    int x = 0;
    if (coded(t)) {
      if constexpr (DT == DT_F32) c.x = *reinterpret_cast<const uint32_t *>(s + (k < CPT - 1 ? code : code_last));
      else c = *reinterpret_cast<const uint2 *>(s + (k < CPT - 1 ? code : code_last));
      x = (e + exp_at(k))[k < CPT - 1 ? exp : exp_last];
    }
    return only(k, ck_decode<DT>(c, x));
  }
  __device__ __forceinline__ void encode(const ck_u32x4 &r, uint8_t *q, int8_t *e, int t, int k) const {
    constexpr int L = kCkBlock / V;  // lanes of a block
    const int ex = ck_exponent<DT>(ck_groupmax<L>(ck_maxkey<DT>(r)));
    const uint2 c = ck_codes<DT>(r, ex);
    if (!has(k) || !coded(t)) return;
    uint8_t *d = q + code_at(k);
    if constexpr (DT == DT_F32) *reinterpret_cast<uint32_t *>(d + code) = c.x;
    else *reinterpret_cast<uint2 *>(d + code) = c;
    if (pl % L == 0) (e + exp_at(k))[exp] = (int8_t)ex;
  }
};

template <int DT, int CPT, int WPT, int KIND>
__global__ __launch_bounds__(norm_threads<WPT>()) void fno_norm_fwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), PX = 8 * V, WAVES = norm_threads<WPT>() / 64, TPG = WAVES / WPT, NC = 8 * CPT * WPT;
  __shared__ float4 tab[NC];
  __shared__ float red[WPT > 1 ? 2 * WAVES * 2 * PX : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), b = blockIdx.y;
  norm_table<DT>(a, b, NC, tab);
  __syncthreads();
  const int t0 = blockIdx.x * a.per, t1 = min((int)((a.P + PX - 1) / PX), t0 + a.per);
  FieldTile<DT, CPT, WPT> tile(a, b, lane, wave % WPT);
  const float invC = 1.f / (float)a.C;
  int turn = 0;
  for (int t = t0 + wave / WPT; t < t1; t += TPG) {
    const bool whole = (t + 1L) * PX <= a.P;
    tile.at(t);
    ck_u32x4 vr[CPT], xr[CPT];
    if (whole) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        vr[k] = tile.load(a.v, t, k);
        xr[k] = tile.load(a.x, t, k);
      }
    } else {
      const auto end = tile.end(t);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        vr[k] = tile.load_end(a.v, end, k);
        xr[k] = tile.load_end(a.x, end, k);
        channel_done();
      }
    }
    if (a.vq) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        tile.encode(vr[k], a.vq, a.ve, t, k);
        tile.encode(xr[k], a.xq, a.xe, t, k);
      }
    }
    fresh<DT>(vr);
    float s[1][V], o[1][V / 4], m[V], r[V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = 0.f;
    if constexpr (KIND == kLayer) {
      channel_sum<V, CPT, false>(s[0], [&](int k, int e) { return ck_get<DT>(vr[k], e); });
      fold<V>(s[0], o[0]);
      Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) o[0][i] /= (float)a.C;
      unfold<V>(o[0], m);
      fresh<DT>(vr);
    }
    channel_sum<V, CPT, true>(s[0], [&](int k, int e) {
      const float d = ck_get<DT>(vr[k], e) - m[e];
      return KIND == kLayer && !tile.has(k) ? 0.f : d;
    });
    fold<V>(s[0], o[0]);
    Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) o[0][i] = rsq(fmaf(o[0][i], invC, a.eps));
    unfold<V>(o[0], r);
    fresh<DT>(vr);
    float y[CPT][V];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const float4 w = tab[tile.channel(k)];
#pragma unroll
      for (int e = 0; e < V; ++e)
        y[k][e] = ck_get<DT>(xr[k], e) + fmaf((ck_get<DT>(vr[k], e) - m[e]) * r[e], w.x, w.y);
      tile.store(a.y, t, k, whole, ck_raw<DT>(y[k]));
    }
    if (a.u) {
      if constexpr (KIND == kLayer) {
        channel_sum<V, CPT, false>(s[0], [&](int k, int e) { return y[k][e]; });
        fold<V>(s[0], o[0]);
        Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) o[0][i] /= (float)a.C;
        unfold<V>(o[0], m);
      }
      channel_sum<V, CPT, true>(s[0], [&](int k, int e) {
        const float d = y[k][e] - m[e];
        return KIND == kLayer && !tile.has(k) ? 0.f : d;
      });
      fold<V>(s[0], o[0]);
      Join<1, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) o[0][i] = rsq(fmaf(o[0][i], invC, a.eps));
      unfold<V>(o[0], r);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
          const float4 w = tab[tile.channel(k)];
        float u[V];
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = fmaf((y[k][e] - m[e]) * r[e], w.z, w.w);
        tile.store(a.u, t, k, whole, ck_raw<DT>(u));
      }
    }
  }
}

// Backward of a field, in passes over the wave's registers, each ending in a
// sum over the channels:
//   v's mean (layer norm) and deviation;
//   y's mean and that of g = gu w_pre (layer norm);  y's deviation and g . (y - m');
//   gx, its sums over pixels and h . v^, h = gx scale gate w_post (and h's mean);
//   gv.
// x, v, gy and gu stay as stored and y is formed from them again in each
// pass: kept in fp32 it would spill, and a spilled value read back after a
// store waits for that store (measured 46 us a tile instead of 12). The layer norm of 16-bit
// fields with eight groups a wave (57 to 64 channels and their multiples) still spills 44 to 76 bytes
// a lane: 20 x 64 x 256^2 fp16 217 us, 186 with 56 channels (1.10 and 1.08 of their bytes' time).
template <int DT, int CPT, int WPT, int KIND>
__global__ __launch_bounds__(norm_threads<WPT>()) __attribute__((amdgpu_waves_per_eu(2))) void fno_norm_bwd(NormArgs a) {
  constexpr int V = ck_vec<DT>(), PX = 8 * V, WAVES = norm_threads<WPT>() / 64, TPG = WAVES / WPT, NC = 8 * CPT * WPT;
  constexpr int NQ = KIND == kLayer ? 2 : 1;
  __shared__ float4 tab[NC];
  constexpr bool HELD = CPT <= 2;  // the run's sums: in registers, or in LDS where those are needed
  __shared__ float4 accs[CPT * WAVES * (HELD ? 8 : 64)];
  __shared__ float red[WPT > 1 ? 2 * WAVES * 2 * PX : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), b = blockIdx.y;
  norm_table<DT>(a, b, NC, tab);
  __syncthreads();
  const int t0 = blockIdx.x * a.per, t1 = min((int)((a.P + PX - 1) / PX), t0 + a.per);
  FieldTile<DT, CPT, WPT> tile(a, b, lane, wave % WPT);
  const float invC = 1.f / (float)a.C;
  int turn = 0;
  // this thread's sums {T, G, U, V} of its k-th channel. Private, so read, added to
  // and written back: LDS atomics took a third of the kernel's time.
  float4 held[HELD ? CPT : 1];
  auto sums = [&](int k) -> float4 & {
    if constexpr (HELD) return held[k];
    else return accs[k * (64 * WAVES) + threadIdx.x];
  };
#pragma unroll
  for (int k = 0; k < CPT; ++k) sums(k) = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t = t0 + wave / WPT; t < t1; t += TPG) {
    const bool whole = (t + 1L) * PX <= a.P;
    tile.at(t);
    ck_u32x4 vr[CPT], xr[CPT], gyr[CPT], gur[CPT];
    if (a.vq) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        vr[k] = tile.decode(a.vq, a.ve, t, k);
        xr[k] = tile.decode(a.xq, a.xe, t, k);
      }
    } else if (whole) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        vr[k] = tile.load(a.v, t, k);
        xr[k] = tile.load(a.x, t, k);
      }
    } else {
      const auto end = tile.end(t);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        vr[k] = tile.load_end(a.v, end, k);
        xr[k] = tile.load_end(a.x, end, k);
        channel_done();
      }
    }
    const void *gu = a.gu ? a.gu : a.gy;  // without gu its values are not used
    if (whole) {
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        gur[k] = tile.load(gu, t, k);
        gyr[k] = tile.load(a.gy, t, k);
      }
    } else {
      const auto end = tile.end(t);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        gur[k] = tile.load_end(gu, end, k);
        gyr[k] = tile.load_end(a.gy, end, k);
        channel_done();
      }
    }
    float m[V], r[V], my[V], ry[V], q[2][V];
    // joins NQ sums over the channels: each lane then holds `out` of its pixels
    auto all = [&](auto &s, auto &&f) {
      constexpr int N = sizeof(s) / sizeof(s[0]);
      float o[N][V / 4];
#pragma unroll
      for (int i = 0; i < N; ++i) fold<V>(s[i], o[i]);
      Join<N, V, WPT>::run(o, red, turn, wave, lane);
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int j = 0; j < V / 4; ++j) o[i][j] = f(i, o[i][j]);
        unfold<V>(o[i], s[i]);
      }
    };
    auto mean = [&](int, float s) { return s / (float)a.C; };
    auto scale = [&](int, float s) { return s * invC; };
    auto zero = [&](auto &s) {
#pragma unroll
      for (int i = 0; i < (int)(sizeof(s) / sizeof(s[0])); ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[i][e] = 0.f;
    };
    float s1[1][V], s2[NQ][V];
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = my[e] = 0.f;
    fresh<DT>(vr);
    if constexpr (KIND == kLayer) {
      channel_sum<V, CPT, false>(s1[0], [&](int k, int e) { return ck_get<DT>(vr[k], e); });
      all(s1, mean);
#pragma unroll
      for (int e = 0; e < V; ++e) m[e] = s1[0][e];
      fresh<DT>(vr);
    }
    channel_sum<V, CPT, true>(s1[0], [&](int k, int e) {
      const float d = ck_get<DT>(vr[k], e) - m[e];
      return KIND == kLayer && !tile.has(k) ? 0.f : d;
    });
    all(s1, [&](int, float s) { return rsq(fmaf(s, invC, a.eps)); });
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = s1[0][e];
    auto y = [&](int k, int e, const float4 &w) {
      return ck_get<DT>(xr[k], e) + fmaf((ck_get<DT>(vr[k], e) - m[e]) * r[e], w.x, w.y);
    };
    if (a.gu) {
      if constexpr (KIND == kLayer) {
        zero(s2);
        fresh<DT>(vr);
        fresh<DT>(xr);
        fresh<DT>(gur);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          const float4 w = tab[tile.channel(k)];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            s2[0][e] += y(k, e, w);
            s2[NQ - 1][e] = fmaf(ck_get<DT>(gur[k], e), w.z, s2[NQ - 1][e]);
          }
          channel_done();
        }
        all(s2, mean);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          my[e] = s2[0][e];
          q[1][e] = s2[NQ - 1][e];
        }
      }
      float s[2][V];
      zero(s);
      fresh<DT>(vr);
      fresh<DT>(xr);
      fresh<DT>(gur);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float4 w = tab[tile.channel(k)];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float d = y(k, e, w) - my[e];
          if (KIND == kLayer && !tile.has(k)) d = 0.f;
          s[0][e] = fmaf(d, d, s[0][e]);
          s[1][e] = fmaf(ck_get<DT>(gur[k], e) * w.z, d, s[1][e]);
        }
        channel_done();
      }
      all(s, [&](int i, float v) { return i == 0 ? rsq(fmaf(v, invC, a.eps)) : v * invC; });
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ry[e] = s[0][e];
        q[0][e] = s[1][e] * s[0][e];  // mean(g y^)
      }
    }
    float gx[CPT][V];
    zero(s2);
    fresh<DT>(vr);
    fresh<DT>(xr);
    fresh<DT>(gur);
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      const float4 w = tab[tile.channel(k)];
      float4 sum = sums(k);
      float sT = 0.f, sG = 0.f;
      if (a.gu) {
        float sU = 0.f, sV = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float gu = ck_get<DT>(gur[k], e), yh = (y(k, e, w) - my[e]) * ry[e];
          sU = fmaf(gu, yh, sU);
          sV += gu;
          float g = fmaf(-yh, q[0][e], gu * w.z);
          if (KIND == kLayer) g -= q[1][e];
          gx[k][e] = fmaf(ry[e], g, ck_get<DT>(gyr[k], e));
        }
        sum.z += sU;
        sum.w += sV;
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) gx[k][e] = ck_get<DT>(gyr[k], e);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float vh = (ck_get<DT>(vr[k], e) - m[e]) * r[e], g = gx[k][e];
        sT = fmaf(g, vh, sT);
        sG += g;
        s2[0][e] = fmaf(g * w.x, vh, s2[0][e]);
        if (KIND == kLayer) s2[NQ - 1][e] = fmaf(g, w.x, s2[NQ - 1][e]);
      }
      sum.x += sT;
      sum.y += sG;
      sums(k) = sum;
      if (a.gx) tile.store(a.gx, t, k, whole, ck_raw<DT>(gx[k]));
      channel_done();
    }
    all(s2, scale);
    if (a.gv) {
      fresh<DT>(vr);
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        const float w = tab[tile.channel(k)].x;
        float gv[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float vh = (ck_get<DT>(vr[k], e) - m[e]) * r[e];
          float g = fmaf(-vh, s2[0][e], gx[k][e] * w);
          if (KIND == kLayer) g -= s2[NQ - 1][e];
          gv[e] = r[e] * g;
        }
        tile.store(a.gv, t, k, whole, ck_raw<DT>(gv));
        channel_done();
      }
    }
  }
  if (!a.part) return;
  // the run's sums: over a channel's 8 lanes, then over the workgroup's tiles
  float4 tot[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const float4 sum = sums(k);
    tot[k] = make_float4(sum8(sum.x), sum8(sum.y), sum8(sum.z), sum8(sum.w));
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    if ((lane & 7) == 0) accs[(wave / WPT) * NC + tile.channel(k)] = tot[k];
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * NC; i += blockDim.x) {
    const int c = i >> 2, q = i & 3;
    if (c >= a.C) continue;
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < TPG; ++g) t += reinterpret_cast<const float *>(accs + g * NC + c)[q];
    a.part[(((size_t)q * a.C + c) * a.B + b) * gridDim.x + blockIdx.x] = t;
  }
}

// The variant for C channels: groups of 8 spread over `waves` waves, exactly
// ceil(groups / waves) of them each, so that no group but a wave's last is ever
// empty.
template <int DT, int KIND, int WPT, bool FWD>
const void *field_pick(int cpt) {
#define FNO_PICK(CPT) (FWD ? (const void *)fno_norm_fwd<DT, CPT, WPT, KIND> : (const void *)fno_norm_bwd<DT, CPT, WPT, KIND>)
  if constexpr (WPT == 1 || WPT == 4) {
    if (cpt == 1) return FNO_PICK(1);
    if (cpt == 2) return FNO_PICK(2);
    if (cpt == 3) return FNO_PICK(3);
    if (cpt == 4) return FNO_PICK(4);
  }
  if (cpt <= 5) return FNO_PICK(5);
  if (cpt == 6) return FNO_PICK(6);
  if (cpt == 7) return FNO_PICK(7);
  return FNO_PICK(8);
#undef FNO_PICK
}

// Waves that share a tile: as few as hold its channels, 64 each. In the
// backward that leaves two waves a SIMD instead of three from 40 channels on,
// yet two waves that share a tile wait for each other four times a tile (64
// channels, fp16: 193 us with one wave, 226 with two). With fewer than 512
// tiles a call is as long as one wave's work, so four share it.
inline int field_waves(int C, long tiles) {
  if (C > 8 && C <= 128 && tiles < 512) return 4;
  return C <= 64 ? 1 : C <= 128 ? 2 : C <= 256 ? 4 : 8;
}

template <int DT, int KIND, bool FWD>
NormPick field_kernel(int C, int w) {
  const int cpt = ((C + 7) / 8 + w - 1) / w;
  const void *k = w == 1   ? field_pick<DT, KIND, 1, FWD>(cpt)
                  : w == 2 ? field_pick<DT, KIND, 2, FWD>(cpt)
                  : w == 4 ? field_pick<DT, KIND, 4, FWD>(cpt)
                           : field_pick<DT, KIND, 8, FWD>(cpt);
  return {k, w == 1 ? 256 : 64 * w, w == 1 ? 4 : 1, 0, w, w == 1 || w == 4 ? cpt : std::max(cpt, 5)};
}

template <int DT, int KIND>
NormPick field_kernel(bool fwd, int C, int w) {
  return fwd ? field_kernel<DT, KIND, true>(C, w) : field_kernel<DT, KIND, false>(C, w);
}

}  // namespace fno
