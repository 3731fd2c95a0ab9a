// gnorm_kernels.hpp - the kernels of group norm with an activation and dropout, and their launches
// (gnorm.hip has the mathematics and the design).
#pragma once

#include <algorithm>

#include "gnorm.hpp"

namespace fno {

// ------------------------------------------------------------ small groups

// T threads hold a group, NC chunks of 16 bytes each (8192 x 1024 bf16 in 16 groups of 8 chunks, a step: 112 us by
// teams of 16 with four chunks, 54 by teams of 8 with two and half the runs of the parameters). Bound by vector issue
// on tokens, by latency on few groups.
template <int DT, bool LAST, bool BWD, int T, int NC>
__global__ __launch_bounds__(T > kThreads ? T : kThreads) void fno_gnorm_small(GnArgs a) {
  constexpr int V = ck_vec<DT>(), TEAMS = T > kThreads ? 1 : kThreads / T;
  __shared__ float red[2][16];
  const int t = threadIdx.x % T;
  const uint32_t len = LAST ? (uint32_t)a.Cg : (uint32_t)a.P, rows = LAST ? (uint32_t)a.P : (uint32_t)a.Cg;
  const uint32_t cpr = (len + V - 1) / V, chunks = rows * cpr;  // at most T NC
  const uint32_t by_cpr = (0x80000000u + cpr - 1) / cpr;  // q / cpr is the high half of 2 q by_cpr: q cpr < 2^31
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
    const uint32_t pitch = LAST ? (uint32_t)a.C : (uint32_t)a.P;  // a group's values span fewer than 2^28
    ck_u32x4 rx[NC], rg[BWD ? NC : 1];
    // Where chunk i of a thread lies; each phase works it out again, since the registers go to the values (kept through the
    // phases: 8192 x 4096 fp16 in 32 groups, a step, 164 us).
    struct Place {
      uint32_t row, k;
      int n;  // values of the chunk, 0 where there is none
      size_t at;
    };
    uint32_t mine = t;
    auto place = [&](int i) __attribute__((always_inline)) {
      const uint32_t q = mine + i * T, qc = min(q, chunks - 1);
      Place p;
      p.row = __umulhi(2 * qc, by_cpr);
      p.k = (qc - p.row * cpr) * V;
      p.n = q < chunks ? (int)min(len - p.k, (uint32_t)V) : 0;
      p.at = first + p.row * pitch + p.k;
      return p;
    };
    auto again = [&]() __attribute__((always_inline)) { asm volatile("" : "+v"(mine)); };
    if (whole) {
#pragma unroll
      for (int i = 0; i < NC; ++i) rx[i] = ck_load<DT>(a.x, place(i).at, V);
      if constexpr (BWD)
#pragma unroll
        for (int i = 0; i < NC; ++i) rg[i] = ck_load<DT>(a.gy, place(i).at, V);
    } else if (len >= V) {  // a row's last chunk as the 16 bytes that end with the row: no load waits for another
      // by the chunk's own length, also where it is loaded for a slot that has none: the field may end with it
      auto back = [&](const Place &p) __attribute__((always_inline)) { return V - min(len - p.k, (uint32_t)V); };
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const Place p = place(i);
        rx[i] = ck_load<DT>(a.x, p.at - back(p), V);
        if constexpr (BWD) rg[i] = ck_load<DT>(a.gy, p.at - back(p), V);
      }
      again();
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int gone = (int)back(place(i)) * (16 / V);
        rx[i] = ck_shift(rx[i], gone);
        if constexpr (BWD) rg[i] = ck_shift(rg[i], gone);
      }
    } else {  // rows shorter than a chunk: 16 bytes all the same, of which the first values count
      const size_t last = (size_t)a.B * a.C * a.P;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const Place p = place(i);
        const int n = p.at + V <= last ? V : p.n;
        rx[i] = ck_load<DT>(a.x, p.at, n);
        if constexpr (BWD) rg[i] = ck_load<DT>(a.gy, p.at, n);
      }
    }
    float mean, r;
    if constexpr (!BWD) {
      // f(sums, value) over a thread's values, the sums chosen by chunk where chunks are whole
      auto sum = [&](float2 &s, auto f) __attribute__((always_inline)) {
        again();
        if (whole) {
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            float2 c = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < V; ++e) f(c, ck_get<DT>(rx[i], e));
            const bool in = mine + i * T < chunks;
            s.x += in ? c.x : 0.f, s.y += in ? c.y : 0.f;
            channel_done();
          }
        } else {
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int nv = place(i).n;
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float2 c = s;
              f(c, ck_get<DT>(rx[i], e));
              s.x = e < nv ? c.x : s.x, s.y = e < nv ? c.y : s.y;
            }
            channel_done();
          }
        }
      };
      // The sum's rounding moves the mean, by steps of the level; the deviations from it, which are exact where they are
      // small, move it back, and their squares are about it. (The second sum costs a forward 2 to 5 %: 256 x 64 x 1024 fp16
      // 19.8 us without, 20.7 with it; a constant group at 1000 then has y = act(b) and not b plus a hundredth.)
      float2 level = make_float2(0.f, 0.f), dev = make_float2(0.f, 0.f);
      sum(level, [](float2 &s, float v) __attribute__((always_inline)) { s.x += v; });
      mean = team_sum<T>(level.x, red[0]) / n;
      fresh<DT>(rx);
      sum(dev, [&](float2 &s, float v) __attribute__((always_inline)) {
        const float d = v - mean;
        s.x += d;
        s.y = fmaf(d, d, s.y);
      });
      dev = team_sums<T>(dev, red);
      const float off = dev.x / n, off2 = off * off, var = dev.y / n;
      mean += off;
      // less the correction's square, not below 0; what overflowed stays infinite, a NaN stays one
      r = rsq((off2 < var ? var - off2 : var < __builtin_inff() ? 0.f : var) + a.eps);
      fresh<DT>(rx);
      if (a.stats && there && t == 0) a.stats[gid] = make_float2(mean, r);
    } else {
      const float2 st = a.stats[gid];
      mean = st.x, r = st.y;
    }
    const float scale = a.drop.scale;
    // a chunk's w and b, and with DROP its kept bits
    auto chunk = [&](auto drop, const Place &p, float *w, float *bb) __attribute__((always_inline)) {
      if constexpr (LAST) {
        param_piece<DT>(a.w, c0 + p.k, p.n ? (long)len - p.k : 0, 1.f, w);
        param_piece<DT>(a.b, c0 + p.k, p.n ? (long)len - p.k : 0, 0.f, bb);
      } else {
        const float w1 = param(a.w, DT, c0 + p.row, 1.f), b1 = param(a.b, DT, c0 + p.row, 0.f);
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = w1, bb[e] = b1;
      }
      return decltype(drop)::value ? chunk_keep<V, LAST>(a, key, p.at, b, (int)(LAST ? c0 + p.k : c0 + p.row)) : 0xffu;
    };
    if constexpr (!BWD) {
      again();
      with_act(a, [&](auto act, auto drop) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (i * T >= (int)chunks) break;
          const Place p = place(i);
          float w[V], bb[V], o[V];
          const uint32_t m = chunk(drop, p, w, bb);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float z = fmaf((ck_get<DT>(rx[i], e) - mean) * r, w[e], bb[e]);
            o[e] = drop_masked(m, e, act_of<ACT>(z) * scale);
          }
          if (there && p.n) store_chunk<DT>(a.y, p.at, p.n, ck_raw<DT>(o));
          channel_done();
        }
      });
    } else {
      // Twice over the values in registers: the second time with the sums of the first. w gz waits in registers of its own
      // where a team's workgroup leaves room for it; else it is computed again from the values, whose 16-bit forms take
      // half the room.
      constexpr bool KEEP = T <= 256;
      float s1 = 0.f, s2 = 0.f, kept[KEEP ? NC : 1][V];
      auto each = [&](auto out) __attribute__((always_inline)) {
        constexpr bool OUT = decltype(out)::value;
        again();
        with_act(a, [&](auto act, auto drop) __attribute__((always_inline)) {
          constexpr int ACT = decltype(act)::value;
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            if (i * T >= (int)chunks) break;
            const Place p = place(i);
            float w[V], bb[V], o[V];
            const uint32_t m = chunk(drop, p, w, bb);
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float h = (ck_get<DT>(rx[i], e) - mean) * r, z = fmaf(h, w[e], bb[e]);
              const float gz = ck_get<DT>(rg[i], e) * scale * act_slope<ACT>(z);
              const float g = drop_masked(m, e, e < p.n ? gz * w[e] : 0.f);
              if constexpr (OUT) {
                o[e] = r * (g - s1 - h * s2);
              } else {
                if constexpr (KEEP) kept[i][e] = g;
                s1 += g;
                s2 = e < p.n ? fmaf(g, h, s2) : s2;
              }
            }
            if constexpr (OUT)
              if (there && p.n) store_chunk<DT>(a.gx, p.at, p.n, ck_raw<DT>(o));
            channel_done();
          }
        });
      };
      each(std::false_type{});
      s1 = team_sum<T>(s1, red[0]) / n;
      s2 = team_sum<T>(s2, red[1]) / n;
      fresh<DT>(rx);
      if constexpr (KEEP) {
        again();
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (i * T >= (int)chunks) break;
          const Place p = place(i);
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = r * (kept[i][e] - s1 - (ck_get<DT>(rx[i], e) - mean) * r * s2);
          if (there && p.n) store_chunk<DT>(a.gx, p.at, p.n, ck_raw<DT>(o));
          channel_done();
        }
      } else {
        fresh<DT>(rg);
        each(std::true_type{});
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
  float mean, r, rw, bias, c1, c2;  // z = (x - mean) rw + bias; gx = rw gz + c1 + (x - mean) c2
  float s1 = 0.f, s2 = 0.f, shift = 0.f, cnt = 0.f;

  __device__ __forceinline__ Row(const GnArgs &args, const DropKey &k, long row) : a(args), key(k) {
    b = row / a.C;
    c = (int)(row - b * a.C);
    base = (size_t)row * a.P;
  }
  __device__ __forceinline__ size_t group() const { return (size_t)b * a.G + c / a.Cg; }
  // st: the group's statistics; m: its M1 and M2
  __device__ __forceinline__ void use(const float2 &st, const float2 &m) {
    mean = st.x, r = st.y;
    rw = r * param(a.w, DT, c, 1.f);
    bias = param(a.b, DT, c, 0.f);
    c1 = -r * m.x, c2 = -r * r * m.y;
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
    with_act(a, [&](auto act, auto drop) __attribute__((always_inline)) {
      constexpr int ACT = decltype(act)::value;
      constexpr bool DROP = decltype(drop)::value;
      const uint32_t m = DROP ? chunk_keep<V, false>(a, key, base + p, b, c) : 0;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = ck_get<DT>(x, e) - mean, z = fmaf(d, rw, bias);
        if constexpr (!BWD) {
          o[e] = act_of<ACT>(z);
          if constexpr (DROP) o[e] = drop_masked(m, e, o[e] * a.drop.scale);
        } else {
          float gz = ck_get<DT>(gy, e) * act_slope<ACT>(z);
          if constexpr (DROP) gz = drop_masked(m, e, gz * a.drop.scale);
          if constexpr (OUT) {
            o[e] = fmaf(rw, gz, fmaf(d, c2, c1));
          } else {
            gz = e < n ? gz : 0.f;
            s1 += gz;
            s2 = e < n ? fmaf(gz, d, s2) : s2;
          }
        }
      }
      if constexpr (OUT) store_chunk<DT>(BWD ? a.gx : a.y, base + p, n, ck_raw<DT>(o));
    });
  }
};

// A float2 each of T threads' (n, v0, v1) joined: moments, or with BWD sums. T threads a team; red: three floats a wave.
template <bool BWD, int T>
__device__ __forceinline__ void team_join(float &n, float &v0, float &v1, float (*red)[3]) {
  constexpr int W = T < 64 ? T : 64;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    const float nb = BWD ? 0.f : __shfl_xor(n, o, 64), mb = __shfl_xor(v0, o, 64), qb = __shfl_xor(v1, o, 64);
    if constexpr (BWD) v0 += mb, v1 += qb;
    else join_moments(n, v0, v1, nb, mb, qb);
  }
  if constexpr (T > 64) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[wave][0] = n, red[wave][1] = v0, red[wave][2] = v1;
    __syncthreads();
    n = red[0][0], v0 = red[0][1], v1 = red[0][2];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) {
      if constexpr (BWD) v0 += red[i][1], v1 += red[i][2];
      else join_moments(n, v0, v1, red[i][0], red[i][1], red[i][2]);
    }
  }
}

// gw and gb of channels 8 block .. + 7 from the sums of the samples' pieces: 32 threads a channel
template <int DT>
__device__ __forceinline__ void params_block(const GnArgs &a, int block) {
  __shared__ float2 slice[32][9];
  const int l = threadIdx.x & 7, sl = threadIdx.x >> 3, c = block * 8 + l;
  float2 v = make_float2(0.f, 0.f);
  const uint32_t all = (uint32_t)a.B * (uint32_t)a.S;
  if (c < a.C)
#pragma unroll 4
    for (uint32_t i = sl; i < all; i += 32) {
      const uint32_t b = i / (uint32_t)a.S;
      const float2 p = a.part[(long)b * a.sb + c * a.sc + (long)(i - b * a.S) * a.ss];
      v.x += p.x, v.y += p.y;
    }
  slice[sl][l] = v;
  __syncthreads();
  if (sl > 0 || c >= a.C) return;
  for (int i = 1; i < 32; ++i) v.x += slice[i][l].x, v.y += slice[i][l].y;
  put<DT>(a.gb, c, v.x);
  put<DT>(a.gw, c, v.y);
}

// T lanes a row, S pieces a row. OUT: the second pass; else the sums of the pieces. FOLD: the second pass joins
// its group's pieces itself (a launch less), and workgroups behind the rows' (from a.main on) join the parameters'.
template <int DT, bool BWD, bool OUT, bool FOLD, int T>
__global__ __launch_bounds__(kThreads) void fno_gnorm_rows(GnArgs a) {
  constexpr int V = ck_vec<DT>(), R = kThreads / T, AHEAD = 4;
  __shared__ float red[4][3];
  if constexpr (BWD && FOLD)
    if ((int)blockIdx.x >= a.main) {
      params_block<DT>(a, (int)blockIdx.x - a.main);
      return;
    }
  const int t = threadIdx.x % T;
  const DropKey key = drop_key(a.drop);
  const long rows = (long)a.B * a.C, units = (rows + R - 1) / R * a.S;
  const uint32_t cpr = (uint32_t)((a.P + V - 1) / V), full = (uint32_t)(a.P / V);
  const ck_u32x4 none{0u, 0u, 0u, 0u};
  auto load = [&](const void *p, size_t i) { return ck_load<DT>(p, i, V); };
  for (long u = blockIdx.x; u < units; u += FOLD ? a.main : (int)gridDim.x) {
    const long rg = u / a.S;
    const int s = (int)(u - rg * a.S);
    const long rid = rg * R + threadIdx.x / T, row = min(rid, rows - 1);
    Row<DT, BWD, OUT> st(a, key, row);
    if constexpr (FOLD) {
      const int g = st.c / a.Cg, c0 = g * a.Cg;
      const float2 *part = a.part + ((size_t)st.b * a.C + c0) * a.S;  // the group's Cg rows of S
      float n = 0.f, v0 = 0.f, v1 = 0.f;
      for (int i = t; i < a.Cg * a.S; i += T) {
        const int ch = i / a.S;
        const float2 p = part[i];
        if constexpr (BWD) {
          const float w = param(a.w, DT, c0 + ch, 1.f);
          v0 = fmaf(w, p.x, v0), v1 = fmaf(w, p.y, v1);
        } else {
          const long at = (long)(i - ch * a.S) * a.per * V;
          join_moments(n, v0, v1, (float)(min(a.P, at + a.per * V) - at), p.x, p.y);
        }
      }
      team_join<BWD, T>(n, v0, v1, red);
      const float size = (float)a.Cg * (float)a.P;  // n has been rounded at every join
      if constexpr (BWD) {
        st.use(a.stats[st.group()], make_float2(v0 / size, v1 / size));
      } else {
        const float2 m = make_float2(v0, rsq(v1 / size + a.eps));
        if (a.stats && t == 0 && s == 0 && st.c == c0 && rid < rows) a.stats[st.group()] = m;
        st.use(m, make_float2(0.f, 0.f));
      }
    } else if constexpr (BWD || OUT) {
      const size_t g = st.group();
      st.use(a.stats[g], BWD && OUT ? a.gsum[g] : make_float2(0.f, 0.f));
    }
    const uint32_t end = (uint32_t)min((long)cpr, (s + 1L) * a.per);
    uint32_t k = (uint32_t)(s * a.per) + t;
    if (!OUT || rid < rows) {
      for (; k + (AHEAD - 1) * T < min(end, full); k += AHEAD * T) {
        ck_u32x4 x[AHEAD], g[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = load(a.x, st.base + (size_t)(k + i * T) * V);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) g[i] = BWD ? load(a.gy, st.base + (size_t)(k + i * T) * V) : none;
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
      if constexpr (!BWD) {
        const float d = n > 0.f ? v0 / n : 0.f;
        v1 = fmaxf(v1 - v0 * d, 0.f) + (v1 - v1);  // not below 0, NaN where it is NaN
        v0 = st.shift + d;
      } else {
        v1 *= st.r;
      }
      team_join<BWD, T>(n, v0, v1, red);
      if (t == 0 && rid < rows) a.part[rid * a.S + s] = make_float2(v0, v1);
    }
  }
}

// --------------------------------------- channels last: a row a pixel's channels

// A lane has a chunk of V channels and every PL-th of a unit's rows; 256 chunks of channels
// a workgroup (blockIdx.y). A unit is `per` rows: a piece of a sample, or with
// RUNS rows of any samples (the parameters' sums of small groups). A lane sums kStretch rows at a time and joins
// what they come to: where values' squares share their last digits every addition to a long sum rounds the same way
// (2000 squares of fp16 values: 13 half steps off on average).
constexpr int kStretch = 256;
template <int DT, bool BWD, bool OUT, bool RUNS>
__global__ __launch_bounds__(kThreads) void fno_gnorm_cols(GnArgs a) {
  constexpr int V = ck_vec<DT>(), AHEAD = BWD || OUT ? 2 : 4;
  __shared__ float2 red[OUT ? 1 : kThreads * V];
  __shared__ float cnt[OUT || BWD ? 1 : kThreads];
  const int cpr = (a.C + V - 1) / V, kb = blockIdx.y * kThreads, kn = min(kThreads, cpr - kb), PL = kThreads / kn;
  const int kl = threadIdx.x % kn, pl = threadIdx.x / kn, c0 = (kb + kl) * V;
  const bool lane = pl < PL;
  const int n = min(V, a.C - c0);
  const DropKey key = drop_key(a.drop);
  const ck_u32x4 none{0u, 0u, 0u, 0u};
  const long units = RUNS ? a.S : (long)a.B * a.S, all = (long)a.B * a.P;
  auto load = [&](const void *p, size_t i) { return ck_load<DT>(p, i, V); };
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
    // z = (x - mean) rw + bias; gx = rw gz + c1 + (x - mean) c2
    float mean[V], r[V], rw[V], c1[V], c2[V], s1[V], s2[V], shift[V], count = 0.f;
    float joined = 0.f;  // values in the stretches that red and cnt hold already
    auto stats = [&](long sample) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (e > 0 && grp[e] == grp[e - 1]) {
          mean[e] = mean[e - 1], r[e] = r[e - 1];
          if constexpr (BWD && OUT) c1[e] = c1[e - 1], c2[e] = c2[e - 1];
        } else {
          const float2 st = a.stats[sample * a.G + grp[e]];
          mean[e] = st.x, r[e] = st.y;
          if constexpr (BWD && OUT) {
            const float2 m = a.gsum[sample * a.G + grp[e]];
            c1[e] = -r[e] * m.x, c2[e] = -r[e] * r[e] * m.y;
          }
        }
        rw[e] = r[e] * w[e];
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
      with_act(a, [&](auto act, auto drop) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
        constexpr bool DROP = decltype(drop)::value;
        const uint32_t m = DROP ? chunk_keep<V, true>(a, key, at, b, c0) : 0;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = ck_get<DT>(x, e) - mean[e], z = fmaf(d, rw[e], bias[e]);
          if constexpr (!BWD) {
            o[e] = act_of<ACT>(z);
            if constexpr (DROP) o[e] = drop_masked(m, e, o[e] * a.drop.scale);
          } else {
            float gz = ck_get<DT>(gy, e) * act_slope<ACT>(z);
            if constexpr (DROP) gz = drop_masked(m, e, gz * a.drop.scale);
            if constexpr (OUT) {
              o[e] = fmaf(rw[e], gz, fmaf(d, c2[e], c1[e]));
            } else {
              s1[e] += gz;
              s2[e] = fmaf(gz, RUNS ? d * r[e] : d, s2[e]);  // a run's samples have an r each
            }
          }
        }
        if constexpr (OUT) store_chunk<DT>(BWD ? a.gx : a.y, at, n, ck_raw<DT>(o));
      });
    };
    // the sums of a stretch into the lane's own places, to those of the stretches before it
    auto flush = [&](bool more) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float2 &v = red[(pl * V + e) * kn + kl];
        float v0 = s1[e], v1 = s2[e];
        if constexpr (BWD) {
          if constexpr (!RUNS) v1 *= r[e];
          if (more) v0 += v.x, v1 += v.y;
        } else {
          const float d = count > 0.f ? v0 / count : 0.f;
          v1 = fmaxf(v1 - v0 * d, 0.f) + (v1 - v1);  // not below 0, NaN where it is NaN
          v0 = shift[e] + d;
          if (more) {
            float na = joined, m = v.x, q = v.y;
            join_moments(na, m, q, count, v0, v1);
            v0 = m, v1 = q;
          }
        }
        v = make_float2(v0, v1);
        s1[e] = s2[e] = 0.f;
      }
      joined += count, count = 0.f;
    };
    if constexpr (!OUT) __syncthreads();  // the last unit's sums have been read
    if (lane) {
      if constexpr ((BWD || OUT) && !RUNS) stats(b);
      long seen = -1;
      long row = r0 + pl;
      // 16 bytes also where fewer of their values count, up to the rows at whose end the field ends
      const long within = n == V ? r1 : all * a.C < V + c0 ? 0 : min(r1, (all * a.C - V - c0) / a.C + 1);
      for (long from = r0; from < r1; from += (long)kStretch * PL) {
        const long to = OUT ? r1 : min(r1, from + (long)kStretch * PL), safe = min(to, within);
        for (; row + (AHEAD - 1) * PL < safe; row += AHEAD * PL) {
          ck_u32x4 x[AHEAD], g[AHEAD];
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) x[i] = load(a.x, (size_t)(row + i * PL) * a.C + c0);
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) g[i] = BWD ? load(a.gy, (size_t)(row + i * PL) * a.C + c0) : none;
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            if constexpr (RUNS) {
              b = a.P == 1 ? row + i * PL : (row + i * PL) / a.P;
              if (b != seen) stats(b);
              seen = b;
            }
            chunk(x[i], g[i], row + i * PL);
          }
        }
        for (; row < to; row += PL) {
          const ck_u32x4 x = ck_load<DT>(a.x, (size_t)row * a.C + c0, n);
          const ck_u32x4 g = BWD ? ck_load<DT>(a.gy, (size_t)row * a.C + c0, n) : none;
          if constexpr (RUNS) {
            b = a.P == 1 ? row : row / a.P;
            if (b != seen) stats(b);
            seen = b;
          }
          chunk(x, g, row);
        }
        if constexpr (OUT) break;
        flush(from > r0);
      }
    }
    if constexpr (!OUT) {
      if constexpr (!BWD)
        if (lane) cnt[threadIdx.x] = joined;
      __syncthreads();
      int left = PL;  // lanes' sums of a channel: halved until one thread's turn through them is short
      while (left > 16) {
        const int h = (left + 1) / 2;
        if (pl + h < left) {
          const float nb = BWD ? 0.f : cnt[(pl + h) * kn + kl];
          float na = BWD ? 0.f : cnt[threadIdx.x];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float2 &v = red[(pl * V + e) * kn + kl];
            const float2 o = red[((pl + h) * V + e) * kn + kl];
            if constexpr (BWD) {
              v.x += o.x, v.y += o.y;
            } else {
              float n1 = na;
              join_moments(n1, v.x, v.y, nb, o.x, o.y);
            }
          }
          if constexpr (!BWD) cnt[threadIdx.x] = na + nb;
        }
        left = h;
        __syncthreads();
      }
      for (int i = threadIdx.x; i < kn * V; i += kThreads) {  // channel kb V + i
        const int e = i % V, l = i / V;
        if (kb * V + i >= a.C) continue;
        float2 v = red[e * kn + l];
        float nn = BWD ? 0.f : cnt[l];
        for (int q = 1; q < left; ++q) {
          const float2 o = red[(q * V + e) * kn + l];
          if constexpr (BWD) v.x += o.x, v.y += o.y;
          else join_moments(nn, v.x, v.y, cnt[q * kn + l], o.x, o.y);
        }
        if (!RUNS && a.whole) red[e * kn + l] = v;  // nobody else reads this place
        if (BWD || !a.whole) a.part[u * a.C + kb * V + i] = v;
      }
      if constexpr (!RUNS)
        if (a.whole) {  // the channels' sums joined to the groups', a small group's by fewer lanes (16 x 128^2 x 128 bf16
                        // in 32 groups: 25 us by a wave each, 16 by 8 lanes)
          __syncthreads();
          auto join = [&](auto width) __attribute__((always_inline)) {
            constexpr int W = decltype(width)::value;
            const int me = threadIdx.x % W;
            for (int g = threadIdx.x / W; g < a.G; g += kThreads / W) {
              float nn = 0.f, v0 = 0.f, v1 = 0.f;
              for (int i = me; i < a.Cg; i += W) {
                const int c = g * a.Cg + i;
                const float2 o = red[c % V * kn + c / V];
                if constexpr (BWD) {
                  const float wc = param(a.w, DT, c, 1.f);
                  v0 = fmaf(wc, o.x, v0), v1 = fmaf(wc, o.y, v1);
                } else {
                  join_moments(nn, v0, v1, (float)(r1 - r0), o.x, o.y);
                }
              }
              team_join<BWD, W>(nn, v0, v1, nullptr);
              if (me == 0) a.gpart[u * a.G + g] = make_float2(v0, v1);
            }
          };
          if (a.Cg <= 16) join(std::integral_constant<int, 8>{});
          else join(std::integral_constant<int, 64>{});
        }
    }
  }
}

// ------------------------------------------------------------------- joins

constexpr int kJoin = 1024;

// The sums of pieces joined. The first `groups` workgroups: a group's statistics (forward), or its M1 and M2
// (backward), a wave a group or, WIDE, all waves; the others: gw and gb of 8 channels each, 128 slices of the
// sums of `samples` samples (or runs).
template <int DT, bool BWD, bool WIDE>
__global__ __launch_bounds__(kJoin) void fno_gnorm_join(GnArgs a, int groups, int samples) {
  __shared__ float red[16][3];
  __shared__ float2 slice[128][9];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (BWD && (int)blockIdx.x >= groups) {
    const int l = threadIdx.x & 7, sl = threadIdx.x >> 3, c = ((int)blockIdx.x - groups) * 8 + l;
    float2 v = make_float2(0.f, 0.f);
    const uint32_t all = (uint32_t)samples * (uint32_t)a.S;
    if (c < a.C)
#pragma unroll 4
      for (uint32_t i = sl; i < all; i += 128) {
        const uint32_t b = i / (uint32_t)a.S;
        const float2 p = a.part[(long)b * a.sb + c * a.sc + (long)(i - b * a.S) * a.ss];
        v.x += p.x, v.y += p.y;
      }
    slice[sl][l] = v;
    __syncthreads();
    if (sl < 16) {  // two waves
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        const float2 p = slice[sl + 16 * i][l];
        v.x += p.x, v.y += p.y;
      }
      // eight slices a wave, 8 lanes each
#pragma unroll
      for (int o = 8; o < 64; o <<= 1) v.x += __shfl_xor(v.x, o, 64), v.y += __shfl_xor(v.y, o, 64);
      if (lane < 8) red[wave * 8 + l][0] = v.x, red[wave * 8 + l][1] = v.y;
    }
    __syncthreads();
    if (threadIdx.x < 8 && c < a.C) {
      put<DT>(a.gb, c, red[l][0] + red[8 + l][0]);
      put<DT>(a.gw, c, red[l][1] + red[8 + l][1]);
    }
    return;
  }
  const long piece = a.last ? a.per : a.per * ck_vec<DT>(), all = (long)a.B * a.G;
  const int step = WIDE ? kJoin : 64, me = WIDE ? threadIdx.x : lane;
  // a.whole: the pieces' sums are the groups' already
  const uint32_t n_part = (uint32_t)(a.whole ? 1 : a.Cg) * (uint32_t)a.S, inner = a.last && !a.whole ? (uint32_t)a.Cg : (uint32_t)a.S;
  for (long id = WIDE ? blockIdx.x : blockIdx.x * 16L + wave; id < all; id += WIDE ? groups : groups * 16L) {
    const long b = id / a.G;
    const int c0 = (int)(id - b * a.G) * a.Cg;
    float n = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll 4
    for (uint32_t i = me; i < n_part; i += step) {  // neighbours in memory one after the other
      const uint32_t outer = i / inner, in = i - outer * inner;
      const int c = c0 + (int)(a.last ? in : outer);
      const long s = a.last && !a.whole ? outer : in;
      const float2 p = a.whole ? a.gpart[(b * a.S + s) * a.G + id - b * a.G] : a.part[b * a.sb + c * a.sc + s * a.ss];
      if constexpr (BWD) {
        const float w = a.whole ? 1.f : param(a.w, DT, c, 1.f);
        v0 = fmaf(w, p.x, v0);
        v1 = fmaf(w, p.y, v1);
      } else {
        const long rows = min(a.P, (s + 1) * piece) - s * piece;
        join_moments(n, v0, v1, (float)(a.whole ? rows * a.Cg : rows), p.x, p.y);
      }
    }
    if constexpr (BWD) {
      v0 = lane_sum<64>(v0);
      v1 = lane_sum<64>(v1);
    } else {
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float nb = __shfl_xor(n, o, 64), mb = __shfl_xor(v0, o, 64), qb = __shfl_xor(v1, o, 64);
        join_moments(n, v0, v1, nb, mb, qb);
      }
    }
    if constexpr (WIDE) {
      __syncthreads();  // the last group's are read
      if (lane == 0) red[wave][0] = n, red[wave][1] = v0, red[wave][2] = v1;
      __syncthreads();
      if (threadIdx.x == 0)
        for (int i = 1; i < 16; ++i) {
          if constexpr (BWD) v0 += red[i][1], v1 += red[i][2];
          else join_moments(n, v0, v1, red[i][0], red[i][1], red[i][2]);
        }
    }
    if (me == 0) {
      const float size = (float)a.Cg * (float)a.P;
      if constexpr (BWD) a.gsum[id] = make_float2(v0 / size, v1 / size);
      else a.stats[id] = make_float2(v0, rsq(v1 / size + a.eps));  // n has been rounded at every join
    }
  }
}

// ------------------------------------------------------------------ launch

inline void gn_attach(GnArgs &a, const GnPlan &p, void *workspace, bool runs) {
  a.part = static_cast<float2 *>(workspace);
  a.gpart = a.part + p.parts;
  a.gsum = a.gpart + p.gparts;
  a.whole = p.gparts != 0 && !runs;
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
  return hipLaunchKernel(k, dim3((unsigned)std::min({gx, kMaxGrid, kMaxLaunch / threads}), (unsigned)gy), dim3((unsigned)threads), args, 0, s);
}

template <int DT, bool LAST, bool BWD>
hipError_t gn_small(const GnArgs &a, int team, hipStream_t s) {
  GnArgs arg = a;
  void *args[] = {(void *)&arg};
  const void *k = team == 8 ? (const void *)fno_gnorm_small<DT, LAST, BWD, 8, 2>
                  : team == 16 ? (const void *)fno_gnorm_small<DT, LAST, BWD, 16, 4>
                  : team == 64 ? (const void *)fno_gnorm_small<DT, LAST, BWD, 64, 4>
                  : team == 256 ? (const void *)fno_gnorm_small<DT, LAST, BWD, 256, 4>
                                : (const void *)fno_gnorm_small<DT, LAST, BWD, 1024, 4>;
  if constexpr (!BWD)
    if (team > 1024) k = (const void *)fno_gnorm_small<DT, LAST, BWD, 1024, 8>;
  const int threads = std::max(kThreads, std::min(team, 1024));
  FNO_BOUNDS(check_gnorm_small(a, LAST, BWD, std::min(team, 1024), team > 1024 ? 8 : team == 8 ? 2 : 4, DT);)
  return gn_run(k, up((long)a.B * a.G, std::max(1, threads / team)), 1, threads, args, s);
}

// fold: as in the kernel; params: its backward joins the parameters' sums too
template <int DT, bool BWD, bool OUT, bool FOLD>
hipError_t gn_rows(const GnArgs &a, int T, bool params, hipStream_t s) {
  GnArgs arg = a;
  // no gx: the parameters' sums alone, in the order that they have beside it
  arg.main = BWD && OUT && !a.gx ? 0 : (int)std::min(up((long)a.B * a.C, kThreads / T) * a.S, kMaxGrid);
  void *args[] = {(void *)&arg};
  const void *k = T == 64 ? (const void *)fno_gnorm_rows<DT, BWD, OUT, FOLD, 64> : (const void *)fno_gnorm_rows<DT, BWD, OUT, FOLD, 256>;
  if constexpr (!FOLD)
    if (T == 8) k = (const void *)fno_gnorm_rows<DT, BWD, OUT, FOLD, 8>;
  FNO_BOUNDS(check_gnorm_rows(arg, BWD, OUT, FOLD, params, T, DT);)
  return hipLaunchKernel(k, dim3((unsigned)(arg.main + (params ? up(a.C, 8) : 0))), dim3(kThreads), args, 0, s);
}

template <int DT, bool BWD, bool OUT, bool RUNS>
hipError_t gn_cols(const GnArgs &a, hipStream_t s) {
  GnArgs arg = a;
  void *args[] = {(void *)&arg};
  FNO_BOUNDS(check_gnorm_cols(a, BWD, OUT, RUNS, DT);)
  return gn_run((const void *)fno_gnorm_cols<DT, BWD, OUT, RUNS>, RUNS ? a.S : (long)a.B * a.S,
             up(up(a.C, ck_vec<DT>()), kThreads), kThreads, args, s);
}

// samples 0: no parameters' gradients; group: the groups' sums are wanted
template <int DT, bool BWD>
hipError_t gn_join(const GnArgs &a, bool group, int samples, hipStream_t s) {
  GnArgs arg = a;
  const bool wide = (long)(a.whole ? 1 : a.Cg) * a.S > 256;
  const long all = (long)a.B * a.G;
  int groups = group ? (int)std::min(wide ? all : up(all, 16), kMaxGrid / 4) : 0;
  void *args[] = {(void *)&arg, (void *)&groups, (void *)&samples};
  FNO_BOUNDS(check_gnorm_join(a, BWD, group, samples, DT);)
  const void *k = wide ? (const void *)fno_gnorm_join<DT, BWD, true> : (const void *)fno_gnorm_join<DT, BWD, false>;
  return gn_run(k, groups + (samples ? up(a.C, 8) : 0), 1, kJoin, args, s);
}

// channels first: a group's pieces are few enough for each of its second pass's teams to join them
// (of short rows, T = 8, a group that a team does not hold whole has too many)
inline bool gn_fold(const GnArgs &a, const GnPlan &p) { return !p.last && p.T > 8 && (long)a.Cg * a.S <= 4 * p.T; }

template <int DT>
hipError_t gn_forward(GnArgs a, void *workspace, hipStream_t s) {
  const GnPlan p = gn_plan(a, DT);
  a.last = p.last;
  if (p.team) return p.last ? gn_small<DT, true, false>(a, p.team, s) : gn_small<DT, false, false>(a, p.team, s);
  gn_attach(a, p, workspace, false);
  hipError_t e = p.last ? gn_cols<DT, false, false, false>(a, s) : gn_rows<DT, false, false, false>(a, p.T, false, s);
  if (e != hipSuccess) return e;
  if (gn_fold(a, p)) return gn_rows<DT, false, true, true>(a, p.T, false, s);
  if (!a.stats) a.stats = a.gsum;  // kept for nobody
  e = gn_join<DT, false>(a, true, 0, s);
  if (e != hipSuccess) return e;
  return p.last ? gn_cols<DT, false, true, false>(a, s) : gn_rows<DT, false, true, false>(a, p.T, false, s);
}

template <int DT>
hipError_t gn_backward(GnArgs a, void *workspace, hipStream_t s) {
  const GnPlan p = gn_plan(a, DT);
  const bool sums = a.gw || a.gb;
  a.last = p.last;
  hipError_t e = hipSuccess;
  if (p.bteam && a.gx) e = p.last ? gn_small<DT, true, true>(a, p.bteam, s) : gn_small<DT, false, true>(a, p.bteam, s);
  if (e != hipSuccess || (p.bteam && !sums)) return e;
  const bool runs = p.bteam && p.last, out = !p.bteam && a.gx;
  gn_attach(a, p, workspace, runs);
  if (!p.last) e = gn_rows<DT, true, false, false>(a, p.T, false, s);
  else e = runs ? gn_cols<DT, true, false, true>(a, s) : gn_cols<DT, true, false, false>(a, s);
  if (e != hipSuccess) return e;
  if (!p.bteam && gn_fold(a, p)) return gn_rows<DT, true, true, true>(a, p.T, sums, s);
  e = gn_join<DT, true>(a, out, !sums ? 0 : runs ? 1 : a.B, s);
  if (e != hipSuccess || !out) return e;
  return p.last ? gn_cols<DT, true, true, false>(a, s) : gn_rows<DT, true, true, false>(a, p.T, false, s);
}

}  // namespace fno
