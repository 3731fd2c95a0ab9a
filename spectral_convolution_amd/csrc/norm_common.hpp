// norm_common.hpp - sums over channels shared by the norm kernels (norm.hip).
#pragma once

#include "checkpoint.hpp"

namespace fno {

// a call's kernel, its threads, the tiles (rows) a workgroup has at a time, the LDS it is
// launched with, and how a tile (row) is split: waves and groups of 8 channels a wave (threads
// and 16-byte pieces a thread)
struct NormPick {
  const void *kernel;
  int threads, rpg;
  size_t lds;
  int wide, deep;
};

constexpr int kRms = 0;
constexpr int kLayer = 1;

__device__ __forceinline__ float param(const void *p, int dtype, size_t i, float none) {
  if (!p) return none;
  if (dtype == DT_F32) return reinterpret_cast<const float *>(p)[i];
  if (dtype == DT_F16) return (float)reinterpret_cast<const _Float16 *>(p)[i];
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16);
}

// The storage bits of p[i], of any[i] where there is no p: several of these follow
// each other without a wait, which a branch around each load would bring (param()).
template <int DT>
__device__ __forceinline__ uint32_t param_bits(const void *p, const void *any, size_t i) {
  const void *q = p ? p : any;
  if constexpr (DT == DT_F32) return reinterpret_cast<const uint32_t *>(q)[i];
  else return reinterpret_cast<const uint16_t *>(q)[i];
}
template <int DT>
__device__ __forceinline__ float param_value(const void *p, uint32_t bits, float none) {
  float v;
  if constexpr (DT == DT_F32) v = __uint_as_float(bits);
  else if constexpr (DT == DT_F16) v = (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  else v = __uint_as_float(bits << 16);
  return p ? v : none;
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

// The scheduler may not mix the channels of a phase: converting all of them
// ahead of their use doubles the registers held.
__device__ __forceinline__ void channel_done() { __builtin_amdgcn_sched_barrier(0x4 | 0x10 | 0x80); }

// s[e] = sum over a lane's channels k of h(k, e), or of its square
template <int V, int CPT, bool SQUARE, typename F>
__device__ __forceinline__ void channel_sum(float (&s)[V], F h) {
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = 0.f;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = h(k, e);
      s[e] = SQUARE ? fmaf(d, d, s[e]) : s[e] + d;
    }
    channel_done();
  }
}

// Joins NQ folded sums over the WPT waves of a tile through LDS. Two buffers in
// turn: a wave that writes one again has passed the barrier of the other.
template <int NQ, int V, int WPT>
struct Join {
  static __device__ __forceinline__ void run(float (&o)[NQ][V / 4], float *red, int &turn, int wave, int lane) {
    if constexpr (WPT > 1) {
      constexpr int ROW = 2 * V * 8;  // two quantities of the 8 V pixels
      float *buf = red + (turn & 1) * WPT * ROW;
      ++turn;
      const int slot = (lane & 7) * V + (V / 4) * ((lane >> 4) & 1) + (V / 2) * (lane >> 5);
      if ((lane & 8) == 0) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int i = 0; i < V / 4; ++i) buf[wave * ROW + q * 8 * V + slot + i] = o[q][i];
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          float t = 0.f;
#pragma unroll
          for (int w = 0; w < WPT; ++w) t += buf[w * ROW + q * 8 * V + slot + i];
          o[q][i] = t;
        }
    }
  }
};

// threads of a field's workgroup: four waves with tiles of their own, or the
// waves that share a tile
template <int WPT>
constexpr int norm_threads() { return WPT == 1 ? 256 : 64 * WPT; }

// Keeps the compiler from carrying the fp32 forms of a stored piece from one
// phase of a kernel to the next (twice the registers, spilled): each phase
// converts again.
template <int DT, int N>
__device__ __forceinline__ void fresh(ck_u32x4 (&r)[N]) {
  if constexpr (DT != DT_F32)
#pragma unroll
    for (int k = 0; k < N; ++k) asm volatile("" : "+v"(r[k]));
}

}  // namespace fno
