// mx4_mix.hip - the channel mix of two operands in 4-bit floats (mx4.hpp),
//   y[b][o][p] = act(sum_i A[o][i] x[b][i][p] + bias[o] + add[b][o][p]),
// on the scaled matrix instructions v_mfma_scale_f32_16x16x128_f8f6f4, which take the blocks' powers of two with
// the codes: lane l has row l % 16 and block l / 16 of four, 16 bytes of codes and one scale byte of either operand.
// Products of codes are exact, sums are fp32 (a product of 128 off by up to 4e-8 of its terms' sizes, measured).
//
// The rows that are neighbours in y are the instruction's first operand (pixels of a field, output
// channels of tokens): a lane then has four neighbouring results.

#include <algorithm>

#include "gelu.hpp"
#include "mx4.hpp"

namespace fno {

namespace {

constexpr int kThreads = 256;
constexpr long kMaxGrid = 1L << 22;

typedef int v8i __attribute__((ext_vector_type(8)));

// first operand f, second operand s: y[b][s][f] with strides ybatch, ys, 1
struct Gemm {
  const uint8_t *fq, *fe, *sq, *se;
  const void *bias, *add;
  void *y;
  long nf, ns, nb, batches;
  long ybatch, ys;
  int act;
  int bias_f;  // bias belongs to f (tokens), else to s
};

__device__ __forceinline__ v4f mx4_product(const ck_u32x4 &a, uint32_t sa, const ck_u32x4 &b, uint32_t sb, const v4f &c) {
  const v8i x{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0}, y{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

template <int DT>
__device__ __forceinline__ float value_at(const void *p, size_t i) {
  if constexpr (DT == DT_F32) return reinterpret_cast<const float *>(p)[i];
  else if constexpr (DT == DT_F16) return (float)reinterpret_cast<const _Float16 *>(p)[i];
  else return bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
}

// four neighbouring results z at y[at] .., n of them there
template <int DT>
__device__ __forceinline__ void mx4_finish(const Gemm &g, const v4f &acc, const float *bias, size_t at, int n) {
  typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
  float o[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) o[r] = acc[r] + bias[r];
  if (n >= 4) {
    if (g.add) {
      if constexpr (DT == DT_F32) {
        const ck_u32x4 v = *reinterpret_cast<const ck_u32x4_any *>(reinterpret_cast<const float *>(g.add) + at);
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] += __uint_as_float(v[r]);
      } else {
        const u32x2_any v = *reinterpret_cast<const u32x2_any *>(reinterpret_cast<const uint16_t *>(g.add) + at);
        const ck_u32x4 w{v[0], v[1], 0u, 0u};
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] += ck_get<DT>(w, r);
      }
    }
    if (g.act)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = gelu_train(o[r]);
    if constexpr (DT == DT_F32) {
      *reinterpret_cast<ck_u32x4_any *>(reinterpret_cast<float *>(g.y) + at) = ck_raw<DT>(o);
    } else {
      *reinterpret_cast<u32x2_any *>(reinterpret_cast<uint16_t *>(g.y) + at) =
          u32x2_any{ck_pair<DT>(o[0], o[1]), ck_pair<DT>(o[2], o[3])};
    }
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < n) {
        if (g.add) o[r] += value_at<DT>(g.add, at + r);
        if (g.act) o[r] = gelu_train(o[r]);
        if constexpr (DT == DT_F32) reinterpret_cast<float *>(g.y)[at + r] = o[r];
        else if constexpr (DT == DT_F16) reinterpret_cast<_Float16 *>(g.y)[at + r] = (_Float16)o[r];
        else reinterpret_cast<uint16_t *>(g.y)[at + r] = (uint16_t)f32_to_bf16(o[r]);
      }
  }
}

template <int DT>
__device__ __forceinline__ float bias_at(const Gemm &g, long i, long n) {
  return g.bias ? value_at<DT>(g.bias, (size_t)min(i, n - 1)) : 0.f;
}

}  // namespace

// A wave has 64 f x 64 s, four waves side by side along f; operands straight from memory to registers, the
// next step's loaded before this one's products.
template <int DT>
__global__ __launch_bounds__(kThreads) void fno_mx4_mix(Gemm g) {
  constexpr int F = 4, S = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quad = lane >> 4;
  const long ft = (g.nf + 255) / 256, st = (g.ns + 63) / 64, tiles = ft * st * g.batches, steps = (g.nb + 3) / 4;
  for (long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const long si = t % st, fb = t / st, b = fb / ft, f0 = (fb - b * ft) * 256 + wave * 64, s0 = si * 64;
    if (f0 >= g.nf) continue;
    size_t fr[F], sr[S];
#pragma unroll
    for (int i = 0; i < F; ++i) fr[i] = (size_t)(b * g.nf + min(f0 + 16 * i + l16, g.nf - 1)) * g.nb;
#pragma unroll
    for (int j = 0; j < S; ++j) sr[j] = (size_t)min(s0 + 16 * j + l16, g.ns - 1) * g.nb;
    v4f acc[F][S];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    ck_u32x4 fc[F], sc[S];
    uint32_t fx[F], sx[S];
    auto load = [&](long k) {
      const long kb = 4 * k + quad, kc = min(kb, g.nb - 1);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        fc[i] = *reinterpret_cast<const ck_u32x4 *>(g.fq + (fr[i] + kc) * 16);
        fx[i] = g.fe[fr[i] + kc];
      }
#pragma unroll
      for (int j = 0; j < S; ++j) {
        sc[j] = *reinterpret_cast<const ck_u32x4 *>(g.sq + (sr[j] + kc) * 16);
        sx[j] = g.se[sr[j] + kc];
      }
      if (kb >= g.nb) {  // no such block: codes of 0, a scale that makes 0 of them
#pragma unroll
        for (int i = 0; i < F; ++i) fc[i] = ck_u32x4{0u, 0u, 0u, 0u}, fx[i] = 127;
#pragma unroll
        for (int j = 0; j < S; ++j) sc[j] = ck_u32x4{0u, 0u, 0u, 0u}, sx[j] = 127;
      }
    };
    load(0);
    for (long k = 0; k < steps; ++k) {
      ck_u32x4 fn[F], sn[S];
      uint32_t fxn[F], sxn[S];
#pragma unroll
      for (int i = 0; i < F; ++i) fn[i] = fc[i], fxn[i] = fx[i];
#pragma unroll
      for (int j = 0; j < S; ++j) sn[j] = sc[j], sxn[j] = sx[j];
      if (k + 1 < steps) load(k + 1);
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j) acc[i][j] = mx4_product(fn[i], fxn[i], sn[j], sxn[j], acc[i][j]);
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const long s = s0 + 16 * j + l16;
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const long f = f0 + 16 * i + 4 * quad;
        if (s >= g.ns || f >= g.nf) continue;
        float bias[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) bias[r] = g.bias_f ? bias_at<DT>(g, f + r, g.nf) : bias_at<DT>(g, s, g.ns);
        mx4_finish<DT>(g, acc[i][j], bias, (size_t)(b * g.ybatch + s * g.ys + f), (int)min(4L, g.nf - f));
      }
    }
  }
}

hipError_t launch_mx4_mix(const Mx4MixArgs &a, int dtype, hipStream_t s) {
  Gemm g{};
  g.bias = a.bias, g.add = a.add, g.y = a.y, g.nb = a.nb, g.act = a.act;
  if (a.P == 1) {
    g.fq = a.aq, g.fe = a.ae, g.sq = a.xq, g.se = a.xe;
    g.nf = a.O, g.ns = a.B, g.batches = 1, g.ybatch = 0, g.ys = a.O, g.bias_f = 1;
  } else {
    g.fq = a.xq, g.fe = a.xe, g.sq = a.aq, g.se = a.ae;
    g.nf = a.P, g.ns = a.O, g.batches = a.B, g.ybatch = a.O * a.P, g.ys = a.P, g.bias_f = 0;
  }
  FNO_BOUNDS(check_mx4_mix(a, dtype);)
  const long tiles = (g.nf + 255) / 256 * ((g.ns + 63) / 64) * g.batches;
  void *args[] = {(void *)&g};
  const void *k = dtype == DT_F32 ? (const void *)fno_mx4_mix<DT_F32>
                  : dtype == DT_F16 ? (const void *)fno_mx4_mix<DT_F16> : (const void *)fno_mx4_mix<DT_BF16>;
  return hipLaunchKernel(k, dim3((unsigned)std::min(tiles, kMaxGrid)), dim3(kThreads), args, 0, s);
}

}  // namespace fno
