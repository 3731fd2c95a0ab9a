// mix_train.hpp - pieces shared by the kernels of the training channel mix
// (mix_train.hip).
#pragma once

#include "checkpoint.hpp"
#include "gelu.hpp"

namespace fno {

// fp32 rows. The four lanes of one l % 16 hold 64 pixels of a row, lane g = l / 16
// the four pieces (16 bytes) from 4 g on. Exchanged among them (a 4 x 4 transposition, its
// own inverse), r[k] of lane g is piece 4 k + g: an access then takes 64 consecutive bytes of
// a row, and the outputs can be written past the caches (with a lane's own
// pieces it takes 16 bytes of every 64; 16 x 32 x 32 channels, 128^2: 81 us a step
// instead of 69). 16-bit rows, 16 bytes of every 32, gained nothing by it.
__device__ __forceinline__ void mt_exchange(ck_u32x4 (&r)[4]) {
  auto swap = [](ck_u32x4 &a, ck_u32x4 &b, bool halves) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const auto t = halves ? __builtin_amdgcn_permlane32_swap(a[d], b[d], false, false)
                            : __builtin_amdgcn_permlane16_swap(a[d], b[d], false, false);
      a[d] = t[0];
      b[d] = t[1];
    }
  };
  swap(r[0], r[2], true);
  swap(r[1], r[3], true);
  swap(r[0], r[1], false);
  swap(r[2], r[3], false);
}

// 16 consecutive elements of a row
template <int DT>
struct Px16 {
  static constexpr int N = DT == DT_F32 ? 4 : 2, V = ck_vec<DT>();
  ck_u32x4 r[N];
  __device__ __forceinline__ void load(const void *p, size_t i, long n) {
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = ck_load<DT>(p, i + k * V, n - k * V);
  }
  // a lane's part of the 64 pixels from p[i] on; its own pieces after mt_exchange(r)
  __device__ __forceinline__ void load64(const void *p, size_t i, int lane) {
    static_assert(DT == DT_F32, "the exchange is that of fp32 rows");
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] = ck_load<DT>(p, i + 16 * k + 4 * (lane >> 4), V);
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

// 64 pixels of a row from p[i] on, v a lane's 16 of them
__device__ __forceinline__ void store64(void *p, size_t i, int lane, const float (&v)[16]) {
  ck_u32x4 r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = ck_raw<DT_F32>(v + 4 * k);
  mt_exchange(r);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float *d = static_cast<float *>(p) + i + 16 * k + 4 * (lane >> 4);
    __builtin_nontemporal_store((ck_u32x4_any)r[k], reinterpret_cast<ck_u32x4_any *>(d));
  }
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
