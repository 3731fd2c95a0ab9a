// gnorm.hpp - group norm with an activation and dropout: what its kernels share (gnorm.hip
// has the mathematics and the design).
#pragma once

#include "checkpoint.hpp"
#include "drop.hpp"
#include "gelu.hpp"
#include "norm_common.hpp"

namespace fno {

constexpr int kThreads = 256;
constexpr long kMaxGrid = 1L << 22;      // workgroups of a launch: the kernels loop past it
constexpr long kMaxLaunch = 1L << 31;    // threads of it: the runtime takes fewer than 2^32

inline int gn_vec(int dtype) { return dtype == DT_F32 ? 4 : 8; }
inline long up(long a, long b) { return (a + b - 1) / b; }

// How a shape runs. team 0: the groups are too large for a workgroup's registers.
struct GnPlan {
  bool last;       // rows are a pixel's channels (one pixel: either order)
  int team, bteam; // threads that hold a group, forward and backward; 2048: 1024 with twice the chunks each
  int T;           // lanes of a row (channels first)
  int S, runs;     // pieces of a row or sample; channels last, small groups: runs of the parameters' sums
  long per, per_run;
  size_t parts, gparts;  // sums in the workspace: of channels' pieces or runs, of groups' pieces
};

GnPlan gn_plan(const GnArgs &a, int dtype);

enum : int { kActNone = 0, kActGelu = 1, kActSilu = 2 };

// z / (1 + exp(-z)) and its derivative s (1 + z (1 - s)), s = 1 / (1 + exp(-z)); |z| is cut off
// where it multiplies a vanished term, so infinities have their limits
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == kActGelu) return gelu_train(z);
  if constexpr (ACT == kActSilu) return fmaxf(z, -126.f) * sigmoid(z);
  return z;
}
// GELU's derivative is gelu_slope() with a step fewer: with q the upper tail at |z| and bell the density,
// g = |z| bell - q is even in z, and the derivative 1 + g above 0, -g below.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActGelu) {
    const float a = fabsf(z);
    const float x = fmaf(fminf(a, 100.f), 0.39894228040143268f, -normal_tail(a, 1.f));
    return 0.5f + copysignf(fmaf(normal_bell(z), x, 0.5f), z);
  }
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(z);
    return s * fmaf(__builtin_amdgcn_fmed3f(z, -126.f, 126.f), 1.f - s, 1.f);
  }
  return 1.f;
}
// f(activation, dropout or not) as integral constants: a branch a chunk, not one a value. The kernels are as near to
// the vector units' rate as to memory's (20 x 64 x 256^2 fp16, GELU, backward sums: 100 us with branches and
// selects at every value).
template <typename F>
__device__ __forceinline__ void with_act(const GnArgs &a, F f) {
  auto act = [&](auto drop) __attribute__((always_inline)) {
    if (a.act == kActGelu) f(std::integral_constant<int, kActGelu>{}, drop);
    else if (a.act == kActSilu) f(std::integral_constant<int, kActSilu>{}, drop);
    else f(std::integral_constant<int, kActNone>{}, drop);
  };
  if (a.drop.thr) act(std::true_type{});
  else act(std::false_type{});
}

// (mean, sum of squared deviations) of na and nb values joined (Chan, Golub, LeVeque: Updating
// formulae and a pairwise algorithm for computing sample variances, 1979)
__device__ __forceinline__ void join_moments(float &n, float &mean, float &m2, float nb, float meanb, float m2b) {
  const float t = n + nb;
  if (nb == 0.f) return;
  const float f = nb * __builtin_amdgcn_rcpf(t), d = meanb - mean;  // off by a step or two of the mean's change
  mean = n == 0.f ? meanb : fmaf(d, f, mean);
  m2 = n == 0.f ? m2b : m2 + m2b + d * d * n * f;
  n = t;
}

// A whole chunk goes past the caches, which keep what is still to be read
template <int DT>
__device__ __forceinline__ void store_chunk(void *p, size_t i, int n, const ck_u32x4 &r) {
  using E = typename std::conditional<DT == DT_F32, float, uint16_t>::type;
  if (n == ck_vec<DT>()) __builtin_nontemporal_store((ck_u32x4_any)r, reinterpret_cast<ck_u32x4_any *>(reinterpret_cast<E *>(p) + i));
  else ck_store_row<DT>(p, i, n, r);
}

template <int W>
__device__ __forceinline__ float lane_sum(float v) {  // over aligned groups of W lanes
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// sum over the T threads of a group, in every one of them; red: a float a wave
template <int T>
__device__ __forceinline__ float team_sum(float v, float *red) {
  if constexpr (T <= 64) {
    return lane_sum<T>(v);
  } else {
    v = lane_sum<64>(v);
    const int wave = threadIdx.x >> 6;
    __syncthreads();  // whoever still reads the last sum
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += red[i];
    return v;
  }
}

// the same of two at once
template <int T>
__device__ __forceinline__ float2 team_sums(float2 v, float (*red)[16]) {
  v = make_float2(lane_sum<(T < 64 ? T : 64)>(v.x), lane_sum<(T < 64 ? T : 64)>(v.y));
  if constexpr (T > 64) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[0][wave] = v.x, red[1][wave] = v.y;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v.x += red[0][i], v.y += red[1][i];
  }
  return v;
}

// V consecutive parameters p[i] .. as fp32, `none` where there is no p or i + e >= n
template <int DT>
__device__ __forceinline__ void param_piece(const void *p, size_t i, long n, float none, float *o) {
  constexpr int V = ck_vec<DT>();
  ck_u32x4 r{0u, 0u, 0u, 0u};
  if (p) r = ck_load<DT>(p, i, n);
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = p ? ck_get<DT>(r, e) : none;
}

// kept bits of a chunk: its first value is value `i` of the field in memory order, of channel c and sample b
template <int V, bool LAST>
__device__ __forceinline__ uint32_t chunk_keep(const GnArgs &a, const DropKey &key, uint64_t i, long b, int c) {
  if (a.drop.unit == kDropElement) return drop_units(key, a.drop.thr, i, V);
  if (a.drop.unit == kDropSample) return drop_one(key, a.drop.thr, (uint64_t)b);
  const uint64_t u = (uint64_t)b * a.C + c;
  return LAST ? drop_units(key, a.drop.thr, u, V) : drop_one(key, a.drop.thr, u);
}

}  // namespace fno
