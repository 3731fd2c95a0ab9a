// mix_train.hpp - pieces shared by the kernels of the training channel mix
// (mix_train.hip).
#pragma once

#include "checkpoint.hpp"
#include "gelu.hpp"

namespace fno {

// 16 consecutive elements of a row
template <int DT>
struct Px16 {
  static constexpr int N = DT == DT_F32 ? 4 : 2, V = ck_vec<DT>();
  ck_u32x4 r[N];
  __device__ __forceinline__ void load(const void *p, size_t i, long n) {
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = ck_load<DT>(p, i + k * V, n - k * V);
  }
  __device__ __forceinline__ float get(int e) const { return ck_get<DT>(r[e / V], e % V); }
  __device__ __forceinline__ uint32_t key() const {
    uint32_t m = ck_maxkey<DT>(r[0]);
#pragma unroll
    for (int k = 1; k < N; ++k) m = max(m, ck_maxkey<DT>(r[k]));
    return m;
  }
  __device__ __forceinline__ ck_u32x4 codes(int e) const {
    ck_u32x4 q;
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = ck_codes<DT>(r[k], e).x;
    } else {
      const uint2 a = ck_codes<DT>(r[0], e), b = ck_codes<DT>(r[1], e);
      q = ck_u32x4{a.x, a.y, b.x, b.y};
    }
    return q;
  }
};

template <int DT>
__device__ __forceinline__ void store16(void *p, size_t i, long n, const float (&v)[16]) {
  constexpr int V = ck_vec<DT>();
#pragma unroll
  for (int k = 0; k < 16 / V; ++k) ck_store<DT>(p, i + k * V, n - k * V, ck_raw<DT>(v + k * V));
}

template <int DT>
__device__ __forceinline__ float mt_load1(const void *p, size_t i) {
  if constexpr (DT == DT_F32) return reinterpret_cast<const float *>(p)[i];
  else if constexpr (DT == DT_F16) return (float)reinterpret_cast<const _Float16 *>(p)[i];
  else return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16);
}

// bias of channel o, 0 where there is none; loaded without a branch
template <int DT>
__device__ __forceinline__ float mt_bias(const MixTrainArgs &a, int o) {
  const float v = mt_load1<DT>(a.bias ? a.bias : a.A, a.bias ? min(o, a.O - 1) : 0);
  return a.bias && o < a.O ? v : 0.f;
}

// 16 codes of a row's piece at pixel p (zeros past the row's blocks) and their exponent
struct Code16 {
  ck_u32x4 q;
  int e;
  __device__ __forceinline__ void load(const uint8_t *codes, const int8_t *exps, size_t row, long p, long nb, bool ok) {
    q = ck_u32x4{0u, 0u, 0u, 0u};
    e = 0;
    if (ok && p < nb * kCkBlock) {
      q = *reinterpret_cast<const ck_u32x4 *>(codes + row * nb * kCkBlock + p);
      e = exps[row * nb + p / kCkBlock];
    }
  }
  __device__ __forceinline__ float get(int k, float step) const { return ck_value(q[k >> 2], k & 3, step); }
};

template <int DT>
__device__ __forceinline__ float mt_gelu(float z) { return DT == DT_F32 ? gelu_train(z) : gelu_half(z); }
template <int DT>
__device__ __forceinline__ float mt_slope(float z) { return DT == DT_F32 ? gelu_slope(z) : gelu_slope_half(z); }

// The workgroup's sums of gA (ga[it]: rows 16 ow + 4 (lane / 16) + j, columns
// 16 it + lane % 16, ow = wave % OT) and gbias (gb, a lane's share of row
// 16 ow + lane % 16) to the workspace, the WP pixel parts added through LDS
// (WP OT 16 (IT 16 + 1) floats, where WP > 1).
template <int OT, int IT, int WP, int THREADS>
__device__ __forceinline__ void mt_finish(const MixTrainArgs &a, const v4f (&ga)[IT], float gb, float *lds, int wave,
                                          int lane) {
  constexpr int RO = OT * 16, RI = IT * 16 + 1;  // rows; a row of gA and its gbias
  const int g = lane >> 4, n = lane & 15, ow = wave % OT, part = wave / OT;
  float *out = a.part + (size_t)blockIdx.x * ((size_t)a.O * a.I + a.O);
  gb += __shfl_xor(gb, 16);
  gb += __shfl_xor(gb, 32);
  __syncthreads();
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = 16 * ow + 4 * g + j, i = 16 * it + n;
      if constexpr (WP > 1) lds[(part * RO + o) * RI + i] = ga[it][j];
      else if (o < a.O && i < a.I) out[(size_t)o * a.I + i] = ga[it][j];
    }
  if (g == 0) {
    if constexpr (WP > 1) lds[(part * RO + 16 * ow + n) * RI + IT * 16] = gb;
    else if (16 * ow + n < a.O) out[(size_t)a.O * a.I + 16 * ow + n] = gb;
  }
  if constexpr (WP > 1) {
    __syncthreads();
    for (int u = threadIdx.x; u < RO * RI; u += THREADS) {
      const int o = u / RI, i = u - o * RI;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WP; ++w) v += lds[(w * RO + o) * RI + i];
      if (o < a.O && i < a.I) out[(size_t)o * a.I + i] = v;
      if (o < a.O && i == IT * 16) out[(size_t)a.O * a.I + o] = v;
    }
  }
}

// a call's kernels; of each its tile's pixels, LDS and threads, and how many of the
// backward's workgroups the chip holds at once
struct MtPick {
  const void *fwd, *bwd;
  int pt_fwd, pt_bwd;
  size_t lds_fwd, lds_bwd;
  int threads_fwd, threads_bwd;
  int resident;
};
MtPick mix_train_f16(int O, int I);
MtPick mix_train_bf16(int O, int I);

}  // namespace fno
