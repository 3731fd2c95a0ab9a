// gnorm_kernels.hpp - the kernels of group norm with an activation and dropout, and their launches
// (gnorm.hip has the mathematics and the design).
#pragma once

#include <algorithm>

#include "gnorm.hpp"

namespace fno {

// ------------------------------------------------------------ small groups

// T threads hold a group, NC chunks of 16 bytes each.
template <int DT, bool LAST, bool BWD, int T, int NC>
__global__ __launch_bounds__(T > kThreads ? T : kThreads) void fno_gnorm_small(GnArgs a) {
  constexpr int V = ck_vec<DT>(), TEAMS = T > kThreads ? 1 : kThreads / T;
  __shared__ float red[2][16];
  const int t = threadIdx.x % T;
  const uint32_t len = LAST ? (uint32_t)a.Cg : (uint32_t)a.P, rows = LAST ? (uint32_t)a.P : (uint32_t)a.Cg;
  const uint32_t cpr = (len + V - 1) / V, chunks = rows * cpr;  // at most T NC
  const bool whole = len % V == 0;
  const float n = (float)len * (float)rows;
  const DropKey key = drop_key(a.drop);
  const long groups = (long)a.B * a.G;
  for (long u = blockIdx.x; u * TEAMS < groups; u += gridDim.x) {
    const long id = u * TEAMS + threadIdx.x / T;
    const bool there = id < groups;
    const uint32_t gid = (uint32_t)(there ? id : groups - 1);
    const uint32_t b = gid / (uint32_t)a.G, g = gid - b * (uint32_t)a.G, c0 = g * a.Cg;
    // value 0 of the group, and the distance of its rows
    const size_t first = LAST ? (size_t)b * a.P * a.C + c0 : ((size_t)b * a.C + c0) * a.P;
    const size_t pitch = LAST ? a.C : a.P;
    ck_u32x4 rx[NC], rg[BWD ? NC : 1];
    uint32_t row[NC], k[NC];
    int nv[NC];  // values of the chunk, 0 where there is none
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t q = t + i * T, qc = min(q, chunks - 1);
      row[i] = qc / cpr;
      k[i] = (qc - row[i] * cpr) * V;
      nv[i] = q < chunks ? (int)min(len - k[i], (uint32_t)V) : 0;
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < NC; ++i) rx[i] = ck_load<DT>(a.x, first + row[i] * pitch + k[i], V);
      if constexpr (BWD)
#pragma unroll
        for (int i = 0; i < NC; ++i) rg[i] = ck_load<DT>(a.gy, first + row[i] * pitch + k[i], V);
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        rx[i] = ck_load<DT>(a.x, first + row[i] * pitch + k[i], nv[i]);
        if constexpr (BWD) rg[i] = ck_load<DT>(a.gy, first + row[i] * pitch + k[i], nv[i]);
      }
    }
    float mean, r;
    if constexpr (!BWD) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s += e < nv[i] ? ck_get<DT>(rx[i], e) : 0.f;
      mean = team_sum<T>(s, red[0]) / n;
      s = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = ck_get<DT>(rx[i], e) - mean;
          s = e < nv[i] ? fmaf(d, d, s) : s;
        }
      r = rsq(team_sum<T>(s, red[1]) / n + a.eps);
      if (a.stats && there && t == 0) a.stats[gid] = make_float2(mean, r);
    } else {
      const float2 st = a.stats[gid];
      mean = st.x, r = st.y;
    }
    auto params = [&](int i, float *w, float *bb) {
      if constexpr (LAST) {
        param_piece<DT>(a.w, c0 + k[i], nv[i] ? (long)len - k[i] : 0, 1.f, w);
        param_piece<DT>(a.b, c0 + k[i], nv[i] ? (long)len - k[i] : 0, 0.f, bb);
      } else {
        const float w1 = param(a.w, DT, c0 + row[i], 1.f), b1 = param(a.b, DT, c0 + row[i], 0.f);
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = w1, bb[e] = b1;
      }
    };
    auto keep = [&](int i) {
      const size_t at = first + row[i] * pitch + k[i];
      return chunk_keep<V, LAST>(a, key, at, b, (int)(LAST ? c0 + k[i] : c0 + row[i]));
    };
    const float scale = a.drop.scale;
    if constexpr (!BWD) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (i * T >= (int)chunks) break;
        float w[V], bb[V], o[V];
        params(i, w, bb);
        const uint32_t m = keep(i);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float z = fmaf((ck_get<DT>(rx[i], e) - mean) * r, w[e], bb[e]);
          o[e] = m >> e & 1 ? act_of(z, a.act) * scale : 0.f;
        }
        if (there && nv[i]) ck_store<DT>(a.y, first + row[i] * pitch + k[i], nv[i], ck_raw<DT>(o));
      }
    } else {
      float g1[NC][V], h[NC][V], s1 = 0.f, s2 = 0.f;  // w gz and x^
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float w[V], bb[V];
        params(i, w, bb);
        const uint32_t m = keep(i);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          h[i][e] = (ck_get<DT>(rx[i], e) - mean) * r;
          const float z = fmaf(h[i][e], w[e], bb[e]);
          const float gz = ck_get<DT>(rg[i], e) * scale * act_slope(z, a.act);
          g1[i][e] = (m >> e & 1) && e < nv[i] ? gz * w[e] : 0.f;
          s1 += g1[i][e];
          s2 = e < nv[i] ? fmaf(g1[i][e], h[i][e], s2) : s2;
        }
      }
      s1 = team_sum<T>(s1, red[0]) / n;
      s2 = team_sum<T>(s2, red[1]) / n;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = r * (g1[i][e] - s1 - h[i][e] * s2);
        if (there && nv[i]) ck_store<DT>(a.gx, first + row[i] * pitch + k[i], nv[i], ck_raw<DT>(o));
      }
    }
  }
}

// ------------------------------------------- channels first: a row a channel

// What a lane does with the values of its chunks of a row, in order.
template <int DT, bool BWD, bool OUT>
struct Row {
  static constexpr int V = ck_vec<DT>();
  const GnArgs &a;
  const DropKey &key;
  long b;
  int c;
  size_t base;
  float mean, r, w, bias, m1, m2;
  float s1 = 0.f, s2 = 0.f, shift = 0.f, cnt = 0.f;

  __device__ __forceinline__ Row(const GnArgs &args, const DropKey &k, long row) : a(args), key(k) {
    b = row / a.C;
    c = (int)(row - b * a.C);
    base = (size_t)row * a.P;
    if constexpr (BWD || OUT) {
      const size_t g = (size_t)b * a.G + c / a.Cg;
      const float2 st = a.stats[g];
      mean = st.x, r = st.y;
      w = param(a.w, DT, c, 1.f);
      bias = param(a.b, DT, c, 0.f);
      if constexpr (BWD && OUT) {
        const float2 m = a.gsum[g];
        m1 = m.x, m2 = m.y;
      }
    }
  }

  // chunk at value p of the row, n of its values there
  __device__ __forceinline__ void chunk(const ck_u32x4 &x, const ck_u32x4 &gy, uint32_t p, int n) {
    if constexpr (!BWD && !OUT) {
      if (cnt == 0.f) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) s += e < n ? ck_get<DT>(x, e) : 0.f;
        shift = s / (float)n;
      }
      cnt += (float)n;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = e < n ? ck_get<DT>(x, e) - shift : 0.f;
        s1 += d;
        s2 = fmaf(d, d, s2);
      }
      return;
    }
    const uint32_t m = chunk_keep<V, false>(a, key, base + p, b, c);
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float h = (ck_get<DT>(x, e) - mean) * r, z = fmaf(h, w, bias);
      const bool kept = m >> e & 1;
      if constexpr (!BWD) {
        o[e] = kept ? act_of(z, a.act) * a.drop.scale : 0.f;
      } else {
        const float gz = kept && e < n ? ck_get<DT>(gy, e) * a.drop.scale * act_slope(z, a.act) : 0.f;
        if constexpr (OUT) {
          o[e] = r * (w * gz - m1 - h * m2);
        } else {
          s1 += gz;
          s2 = e < n ? fmaf(gz, h, s2) : s2;
        }
      }
    }
    if constexpr (OUT) ck_store<DT>(BWD ? a.gx : a.y, base + p, n, ck_raw<DT>(o));
  }
};

// T lanes a row, S pieces a row. OUT: the second pass; else the sums of the pieces.
template <int DT, bool BWD, bool OUT, int T>
__global__ __launch_bounds__(kThreads) void fno_gnorm_rows(GnArgs a) {
  constexpr int V = ck_vec<DT>(), R = kThreads / T, AHEAD = 4;
  __shared__ float red[4][3];
  const int t = threadIdx.x % T;
  const DropKey key = drop_key(a.drop);
  const long rows = (long)a.B * a.C, units = (rows + R - 1) / R * a.S;
  const uint32_t cpr = (uint32_t)((a.P + V - 1) / V), full = (uint32_t)(a.P / V);
  const ck_u32x4 none{0u, 0u, 0u, 0u};
  for (long u = blockIdx.x; u < units; u += gridDim.x) {
    const long rg = u / a.S;
    const int s = (int)(u - rg * a.S);
    const long rid = rg * R + threadIdx.x / T, row = min(rid, rows - 1);
    Row<DT, BWD, OUT> st(a, key, row);
    const uint32_t end = (uint32_t)min((long)cpr, (s + 1L) * a.per);
    uint32_t k = (uint32_t)(s * a.per) + t;
    if (!OUT || rid < rows) {
      for (; k + (AHEAD - 1) * T < min(end, full); k += AHEAD * T) {
        ck_u32x4 x[AHEAD], g[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = ck_load<DT>(a.x, st.base + (size_t)(k + i * T) * V, V);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          g[i] = BWD ? ck_load<DT>(a.gy, st.base + (size_t)(k + i * T) * V, V) : none;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) st.chunk(x[i], g[i], (k + i * T) * V, V);
      }
      for (; k < end; k += T) {
        const uint32_t p = k * V;
        const int n = (int)min((uint32_t)a.P - p, (uint32_t)V);
        const ck_u32x4 x = ck_load<DT>(a.x, st.base + p, n), g = BWD ? ck_load<DT>(a.gy, st.base + p, n) : none;
        st.chunk(x, g, p, n);
      }
    }
    if constexpr (!OUT) {
      float n = st.cnt, v0 = st.s1, v1 = st.s2;
      constexpr int W = T < 64 ? T : 64;
      if constexpr (!BWD) {
        const float d = n > 0.f ? v0 / n : 0.f;
        v1 = fmaxf(v1 - v0 * d, 0.f) + (v1 - v1);  // not below 0, NaN where it is NaN
        v0 = st.shift + d;
#pragma unroll
        for (int o = 1; o < W; o <<= 1) {
          const float nb = __shfl_xor(n, o, 64), mb = __shfl_xor(v0, o, 64), qb = __shfl_xor(v1, o, 64);
          join_moments(n, v0, v1, nb, mb, qb);
        }
      } else {
        v0 = lane_sum<W>(v0);
        v1 = lane_sum<W>(v1);
      }
      if constexpr (T > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[wave][0] = n, red[wave][1] = v0, red[wave][2] = v1;
        __syncthreads();
        if (threadIdx.x == 0)
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            if constexpr (BWD) v0 += red[i][1], v1 += red[i][2];
            else join_moments(n, v0, v1, red[i][0], red[i][1], red[i][2]);
          }
      }
      if (t == 0 && rid < rows) a.part[rid * a.S + s] = make_float2(v0, v1);
    }
  }
}

// --------------------------------------- channels last: a row a pixel's channels

// A lane has a chunk of V channels and every PL-th of a unit's rows; 256 chunks of channels
// a workgroup (blockIdx.y). A unit is `per` rows: a piece of a sample, or with
// RUNS rows of any samples (the parameters' sums of small groups).
template <int DT, bool BWD, bool OUT, bool RUNS>
__global__ __launch_bounds__(kThreads) void fno_gnorm_cols(GnArgs a) {
  constexpr int V = ck_vec<DT>(), AHEAD = 2;
  __shared__ float2 red[OUT ? 1 : kThreads * V];
  __shared__ float cnt[OUT || BWD ? 1 : kThreads];
  const int cpr = (a.C + V - 1) / V, kb = blockIdx.y * kThreads, kn = min(kThreads, cpr - kb), PL = kThreads / kn;
  const int kl = threadIdx.x % kn, pl = threadIdx.x / kn, c0 = (kb + kl) * V;
  const bool lane = pl < PL;
  const int n = min(V, a.C - c0);
  const DropKey key = drop_key(a.drop);
  const ck_u32x4 none{0u, 0u, 0u, 0u};
  const long units = RUNS ? a.S : (long)a.B * a.S, all = (long)a.B * a.P;
  float w[V], bias[V];
  int grp[V];
  if constexpr (BWD || OUT) {
    param_piece<DT>(a.w, c0, n, 1.f, w);
    param_piece<DT>(a.b, c0, n, 0.f, bias);
#pragma unroll
    for (int e = 0; e < V; ++e) grp[e] = min(c0 + e, a.C - 1) / a.Cg;
  }
  for (long u = blockIdx.x; u < units; u += gridDim.x) {
    long b = RUNS ? 0 : u / a.S, r0, r1;  // rows of the whole field
    if constexpr (RUNS) {
      r0 = u * a.per, r1 = min(all, r0 + a.per);
    } else {
      const long p0 = (u - b * a.S) * a.per;
      r0 = b * a.P + p0, r1 = b * a.P + min(a.P, p0 + a.per);
    }
    float mean[V], r[V], m1[V], m2[V], s1[V], s2[V], shift[V], count = 0.f;
    auto stats = [&](long sample) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (e > 0 && grp[e] == grp[e - 1]) {
          mean[e] = mean[e - 1], r[e] = r[e - 1];
          if constexpr (BWD && OUT) m1[e] = m1[e - 1], m2[e] = m2[e - 1];
          continue;
        }
        const float2 st = a.stats[sample * a.G + grp[e]];
        mean[e] = st.x, r[e] = st.y;
        if constexpr (BWD && OUT) {
          const float2 m = a.gsum[sample * a.G + grp[e]];
          m1[e] = m.x, m2[e] = m.y;
        }
      }
    };
#pragma unroll
    for (int e = 0; e < V; ++e) s1[e] = s2[e] = shift[e] = 0.f;
    auto chunk = [&](const ck_u32x4 &x, const ck_u32x4 &gy, long row) {
      if constexpr (!BWD && !OUT) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float v = ck_get<DT>(x, e);
          if (count == 0.f) shift[e] = v;
          const float d = v - shift[e];
          s1[e] += d;
          s2[e] = fmaf(d, d, s2[e]);
        }
        count += 1.f;
        return;
      }
      const size_t at = (size_t)row * a.C + c0;
      const uint32_t m = chunk_keep<V, true>(a, key, at, b, c0);
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float h = (ck_get<DT>(x, e) - mean[e]) * r[e], z = fmaf(h, w[e], bias[e]);
        const bool kept = m >> e & 1;
        if constexpr (!BWD) {
          o[e] = kept ? act_of(z, a.act) * a.drop.scale : 0.f;
        } else {
          const float gz = kept ? ck_get<DT>(gy, e) * a.drop.scale * act_slope(z, a.act) : 0.f;
          if constexpr (OUT) {
            o[e] = r[e] * (w[e] * gz - m1[e] - h * m2[e]);
          } else {
            s1[e] += gz;
            s2[e] = fmaf(gz, h, s2[e]);
          }
        }
      }
      if constexpr (OUT) ck_store<DT>(BWD ? a.gx : a.y, at, n, ck_raw<DT>(o));
    };
    if (lane) {
      if constexpr ((BWD || OUT) && !RUNS) stats(b);
      long seen = -1;
      long row = r0 + pl;
      if (n == V) {
        for (; row + (AHEAD - 1) * PL < r1; row += AHEAD * PL) {
          ck_u32x4 x[AHEAD], g[AHEAD];
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) x[i] = ck_load<DT>(a.x, (size_t)(row + i * PL) * a.C + c0, V);
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) g[i] = BWD ? ck_load<DT>(a.gy, (size_t)(row + i * PL) * a.C + c0, V) : none;
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            if constexpr (RUNS) {
              b = (row + i * PL) / a.P;
              if (b != seen) stats(b);
              seen = b;
            }
            chunk(x[i], g[i], row + i * PL);
          }
        }
      }
      for (; row < r1; row += PL) {
        const ck_u32x4 x = ck_load<DT>(a.x, (size_t)row * a.C + c0, n);
        const ck_u32x4 g = BWD ? ck_load<DT>(a.gy, (size_t)row * a.C + c0, n) : none;
        if constexpr (RUNS) {
          b = row / a.P;
          if (b != seen) stats(b);
          seen = b;
        }
        chunk(x, g, row);
      }
    }
    if constexpr (!OUT) {
      __syncthreads();  // the last unit's sums have been read
      if (lane) {
        if constexpr (!BWD) cnt[threadIdx.x] = count;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float v0 = s1[e], v1 = s2[e];
          if constexpr (!BWD) {
            const float d = count > 0.f ? v0 / count : 0.f;
            v1 = fmaxf(v1 - v0 * d, 0.f) + (v1 - v1);
            v0 = shift[e] + d;
          }
          red[(pl * V + e) * kn + kl] = make_float2(v0, v1);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < kn * V; i += kThreads) {  // channel kb V + i
        const int e = i % V, l = i / V;
        if (kb * V + i >= a.C) continue;
        float2 v = red[e * kn + l];
        float nn = BWD ? 0.f : cnt[l];
        for (int q = 1; q < PL; ++q) {
          const float2 o = red[(q * V + e) * kn + l];
          if constexpr (BWD) v.x += o.x, v.y += o.y;
          else join_moments(nn, v.x, v.y, cnt[q * kn + l], o.x, o.y);
        }
        a.part[u * a.C + kb * V + i] = v;
      }
    }
  }
}

// ------------------------------------------------------------------- joins

// A wave a group: its statistics (forward), or M1 and M2 (backward), from the pieces' sums.
template <int DT, bool BWD>
__global__ __launch_bounds__(64) void fno_gnorm_join(GnArgs a) {
  const int lane = threadIdx.x;
  const long piece = a.last ? a.per : a.per * ck_vec<DT>(), groups = (long)a.B * a.G;
  for (long id = blockIdx.x; id < groups; id += gridDim.x) {
    const long b = id / a.G;
    const int c0 = (int)(id - b * a.G) * a.Cg;
    float n = 0.f, v0 = 0.f, v1 = 0.f;
    for (long i = lane; i < (long)a.Cg * a.S; i += 64) {
      // neighbours in memory one after the other
      const int c = c0 + (int)(a.last ? i % a.Cg : i / a.S);
      const long s = a.last ? i / a.Cg : i % a.S;
      const float2 p = a.part[b * a.sb + c * a.sc + s * a.ss];
      if constexpr (BWD) {
        const float w = param(a.w, DT, c, 1.f);
        v0 = fmaf(w, p.x, v0);
        v1 = fmaf(w, p.y, v1);
      } else {
        join_moments(n, v0, v1, (float)(min(a.P, (s + 1) * piece) - s * piece), p.x, p.y);
      }
    }
    if constexpr (BWD) {
      v0 = lane_sum<64>(v0);
      v1 = lane_sum<64>(v1);
      const float size = (float)a.Cg * (float)a.P;
      if (lane == 0) a.gsum[id] = make_float2(v0 / size, v1 / size);
    } else {
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float nb = __shfl_xor(n, o, 64), mb = __shfl_xor(v0, o, 64), qb = __shfl_xor(v1, o, 64);
        join_moments(n, v0, v1, nb, mb, qb);
      }
      if (lane == 0) a.stats[id] = make_float2(v0, rsq(v1 / n + a.eps));
    }
  }
}

// gw and gb from `samples` x S pieces' sums: 32 channels a workgroup, 32 slices of the sums.
template <int DT>
__global__ __launch_bounds__(1024) void fno_gnorm_params(GnArgs a, int samples) {
  __shared__ float2 red[32][33];
  const int l = threadIdx.x & 31, sl = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
  float2 v = make_float2(0.f, 0.f);
  if (c < a.C)
    for (long i = sl; i < (long)samples * a.S; i += 32) {
      const long b = i / a.S;
      const float2 p = a.part[b * a.sb + c * a.sc + (i - b * a.S) * a.ss];
      v.x += p.x, v.y += p.y;
    }
  red[sl][l] = v;
  __syncthreads();
  if (sl != 0 || c >= a.C) return;
  v = red[0][l];
  for (int i = 1; i < 32; ++i) v.x += red[i][l].x, v.y += red[i][l].y;
  put<DT>(a.gb, c, v.x);
  put<DT>(a.gw, c, v.y);
}

// ------------------------------------------------------------------ launch

inline void gn_attach(GnArgs &a, const GnPlan &p, void *workspace, bool runs) {
  a.part = static_cast<float2 *>(workspace);
  a.gsum = a.part + p.parts;
  a.last = p.last;
  if (!p.last) {
    a.S = p.S, a.per = p.per;
    a.sb = (long)a.C * p.S, a.sc = p.S, a.ss = 1;
  } else {
    a.S = runs ? p.runs : p.S, a.per = runs ? p.per_run : p.per;
    a.sb = runs ? 0 : (long)a.C * p.S, a.sc = 1, a.ss = a.C;
  }
}

inline hipError_t gn_run(const void *k, long gx, long gy, int threads, void **args, hipStream_t s) {
  return hipLaunchKernel(k, dim3((unsigned)std::min(gx, kMaxGrid), (unsigned)gy), dim3((unsigned)threads), args, 0, s);
}

template <int DT, bool LAST, bool BWD>
hipError_t gn_small(const GnArgs &a, int team, hipStream_t s) {
  GnArgs arg = a;
  void *args[] = {(void *)&arg};
  const void *k = team == 16 ? (const void *)fno_gnorm_small<DT, LAST, BWD, 16, 4>
                  : team == 64 ? (const void *)fno_gnorm_small<DT, LAST, BWD, 64, 4>
                  : team == 256 ? (const void *)fno_gnorm_small<DT, LAST, BWD, 256, 4>
                                : (const void *)fno_gnorm_small<DT, LAST, BWD, 1024, BWD ? 2 : 4>;
  const int threads = team > kThreads ? team : kThreads;
  FNO_BOUNDS(check_gnorm_small(a, LAST, BWD, team, BWD && team == 1024 ? 2 : 4, DT);)
  return gn_run(k, up((long)a.B * a.G, threads / team), 1, threads, args, s);
}

template <int DT, bool BWD, bool OUT>
hipError_t gn_rows(const GnArgs &a, int T, hipStream_t s) {
  GnArgs arg = a;
  void *args[] = {(void *)&arg};
  const void *k = T == 8 ? (const void *)fno_gnorm_rows<DT, BWD, OUT, 8>
                  : T == 64 ? (const void *)fno_gnorm_rows<DT, BWD, OUT, 64>
                            : (const void *)fno_gnorm_rows<DT, BWD, OUT, 256>;
  FNO_BOUNDS(check_gnorm_rows(a, BWD, OUT, T, DT);)
  return gn_run(k, up((long)a.B * a.C, kThreads / T) * a.S, 1, kThreads, args, s);
}

template <int DT, bool BWD, bool OUT, bool RUNS>
hipError_t gn_cols(const GnArgs &a, hipStream_t s) {
  GnArgs arg = a;
  void *args[] = {(void *)&arg};
  FNO_BOUNDS(check_gnorm_cols(a, BWD, OUT, RUNS, DT);)
  return gn_run((const void *)fno_gnorm_cols<DT, BWD, OUT, RUNS>, RUNS ? a.S : (long)a.B * a.S,
             up(up(a.C, ck_vec<DT>()), kThreads), kThreads, args, s);
}

template <int DT, bool BWD>
hipError_t gn_join(const GnArgs &a, hipStream_t s) {
  GnArgs arg = a;
  void *args[] = {(void *)&arg};
  FNO_BOUNDS(check_gnorm_join(a, BWD, DT);)
  return gn_run((const void *)fno_gnorm_join<DT, BWD>, (long)a.B * a.G, 1, 64, args, s);
}

template <int DT>
hipError_t gn_params(const GnArgs &a, int samples, hipStream_t s) {
  GnArgs arg = a;
  void *args[] = {(void *)&arg, (void *)&samples};
  FNO_BOUNDS(check_gnorm_params(a, samples, DT);)
  return gn_run((const void *)fno_gnorm_params<DT>, up(a.C, 32), 1, 1024, args, s);
}

template <int DT>
hipError_t gn_forward(GnArgs a, void *workspace, hipStream_t s) {
  const GnPlan p = gn_plan(a, DT);
  a.last = p.last;
  if (p.team) return p.last ? gn_small<DT, true, false>(a, p.team, s) : gn_small<DT, false, false>(a, p.team, s);
  gn_attach(a, p, workspace, false);
  if (!a.stats) a.stats = a.gsum;  // kept for nobody
  hipError_t e = p.last ? gn_cols<DT, false, false, false>(a, s) : gn_rows<DT, false, false>(a, p.T, s);
  if (e == hipSuccess) e = gn_join<DT, false>(a, s);
  if (e == hipSuccess) e = p.last ? gn_cols<DT, false, true, false>(a, s) : gn_rows<DT, false, true>(a, p.T, s);
  return e;
}

template <int DT>
hipError_t gn_backward(GnArgs a, void *workspace, hipStream_t s) {
  const GnPlan p = gn_plan(a, DT);
  const bool sums = a.gw || a.gb;
  a.last = p.last;
  hipError_t e = hipSuccess;
  if (p.bteam && a.gx) e = p.last ? gn_small<DT, true, true>(a, p.bteam, s) : gn_small<DT, false, true>(a, p.bteam, s);
  if (e != hipSuccess || (p.bteam && !sums)) return e;
  const bool runs = p.bteam && p.last;
  gn_attach(a, p, workspace, runs);
  if (!p.last) e = gn_rows<DT, true, false>(a, p.T, s);
  else e = runs ? gn_cols<DT, true, false, true>(a, s) : gn_cols<DT, true, false, false>(a, s);
  if (e == hipSuccess && sums) e = gn_params<DT>(a, runs ? 1 : a.B, s);
  if (p.bteam || !a.gx) return e;
  if (e == hipSuccess) e = gn_join<DT, true>(a, s);
  if (e == hipSuccess) e = p.last ? gn_cols<DT, true, true, false>(a, s) : gn_rows<DT, true, true>(a, p.T, s);
  return e;
}

}  // namespace fno
