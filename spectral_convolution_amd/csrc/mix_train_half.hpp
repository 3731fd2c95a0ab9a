// mix_train_half.hpp - the training channel mix on fp16 / bf16 fields
// (mix_train.hip has the operator and the shape of a tile). The three products
// run on v_mfma_f32_16x16x32_{f16,bf16}: values read back from 8 bits are
// exact in either type, weights and the forward's x are used as stored, and
// gz = gy act'(z), an fp32 value, enters its two products as 16-bit pieces: gx and gA
// are small where the gz of several channels or pixels cancel, and one rounding of gz would
// show there. bf16: three pieces of 8 bits, which are all 24 (two left gx off by
// 2^-17 of its terms; the backward of 32 x 64 x 64 channels, 256^2, takes 309 us with three,
// 293 with two). They lie one after the other as further channels of the summed index.
// fp16: two pieces, 22 bits. It has too little range for that as it stands: gz / 2 is
// taken (|act'| < 1.13 would pass the type's largest) and the remainder of its rounding times
// 2^11, whose products have accumulators of their own, so a gz far below the smallest
// normal number keeps its digits (without it, gy around 2^-12 left gA off by 2^-13).
//
// LDS holds [channel][pixel] halves. A product that sums over channels reads
// its pixel-major operand with transposing reads (ds_read_b64_tr_b16: 16
// lanes take 4 channels x 16 pixels and each gets 4 channels of its pixel); the
// product that sums over pixels reads rows as they lie. Rows are 8 bytes longer than
// the tile: the 32 lanes that read at a time (16 rows, 8 bytes of each of 4
// chunks) then touch all 64 banks once.
#pragma once

#include "mix_train.hpp"

namespace fno {

typedef short mt_s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 mt_h8 __attribute__((ext_vector_type(8)));
typedef __bf16 mt_b8 __attribute__((ext_vector_type(8)));

// WAVES in a workgroup. Backward: four, or eight for eight tiles of c_out, so that
// a wave has one of them; its registers (a row of gA, a tile's inputs ahead)
// fit three waves a SIMD up to 16 tiles of gA, where few waves do not stage many
// rows of x (five variants spill: 16 to 44 bytes a lane, bf16 with one tile of c_out and eight of
// c_in 424: 16 x 128 x 16 channels, 128^2, 101 us where fp16 takes 55). Forward: eight
// from four tiles of c_out on, tiles of 128 pixels: with 64, a row's piece of the codes
// is half a line, and evicted as such.
template <int OT>
constexpr int mh_waves(bool fwd) { return OT == 8 || (fwd && OT == 4) ? 8 : 4; }

// pieces of gz, and the accumulators of a product with them
template <int DT>
constexpr int mh_pieces() { return DT == DT_F16 ? 2 : 3; }
template <int DT>
constexpr int mh_sums() { return DT == DT_F16 ? 2 : 1; }

template <int DT, int OT, int IT, bool FWD>
struct MhGeom {
  static constexpr int WAVES = mh_waves<OT>(FWD), THREADS = 64 * WAVES;
  static constexpr int PER_EU = OT * IT <= 16 && IT <= 2 * OT ? 3 : 2;
  static constexpr int WO = OT, WP = WAVES / WO;                       // waves over c_out, over pixels
  static constexpr int WI = IT < WAVES ? IT : WAVES, ITW = IT / WI;    // gx: waves over c_in; tiles of a wave
  static constexpr int KI = (IT + 1) / 2, KO = (OT + 1) / 2;              // 32-channel steps
  static constexpr int PT = 64 * WP, PITCH = PT + 4;                      // pixels of a tile; halves of an LDS row
  // gz in LDS: pieces, the rows of one and the 32-row steps of all (fp16's pieces share no step)
  static constexpr int NP = mh_pieces<DT>(), ROWS = DT == DT_F16 ? KO * 32 : OT * 16, KS = (NP * ROWS + 31) / 32;
  static constexpr int XS = KI * 32 * PITCH * 2, GS = KS * 32 * PITCH * 2;
  static constexpr int UNITS = IT * 16 * (PT / 16), NU = (UNITS + THREADS - 1) / THREADS;
  static constexpr int SUMS = WP > 1 ? WP * OT * 16 * (IT * 16 + 1) * 4 : 0;
  static constexpr int LDS_FWD = 2 * XS, LDS_BWD = XS + GS > SUMS ? XS + GS : SUMS;
};

template <int DT>
__device__ __forceinline__ v4f mh_mma(ck_u32x4 a, ck_u32x4 b, v4f c) {
  if constexpr (DT == DT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(mt_h8, a), __builtin_bit_cast(mt_h8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mt_b8, a), __builtin_bit_cast(mt_b8, b), c, 0, 0, 0);
}

// First of the four channels that slots 8 g + 4 h .. + 3 of a 32-channel step stand for
// (g: lane / 16). Groups read in the same cycle are 16 rows apart.
__device__ __forceinline__ int mh_slot(int g, int h) { return 16 * (g & 1) + 8 * (g >> 1) + 4 * h; }

// Operand with rows = pixels and the 32 channels of step k as the summed index: row r
// of pixel tile pt is pixel 16 (r / 4) + 4 pt + r % 4 of the 64 from pb on.
template <int PITCH>
__device__ __forceinline__ ck_u32x4 mh_pixels(const uint16_t *s, int k, int pb, int pt, int lane) {
  const int g = lane >> 4, l = lane & 15;
  ck_u32x4 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint16_t *p = s + (32 * k + mh_slot(g, h) + (l >> 2)) * PITCH + pb + 16 * (l & 3) + 4 * pt;
    const mt_s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) mt_s16x4 *)p);
    const uint2 u = __builtin_bit_cast(uint2, v);
    r[2 * h] = u.x;
    r[2 * h + 1] = u.y;
  }
  return r;
}

// 16 bytes at an 8-byte boundary of LDS
__device__ __forceinline__ ck_u32x4 mh_read16(const uint16_t *p) {
  const uint2 a = reinterpret_cast<const uint2 *>(p)[0], b = reinterpret_cast<const uint2 *>(p)[1];
  return ck_u32x4{a.x, a.y, b.x, b.y};
}
__device__ __forceinline__ void mh_write16(uint16_t *p, const ck_u32x4 &v) {
  reinterpret_cast<uint2 *>(p)[0] = make_uint2(v[0], v[1]);
  reinterpret_cast<uint2 *>(p)[1] = make_uint2(v[2], v[3]);
}

// Weights as an operand: lane's column is `col`, the summed index the 32 of step k (DUP:
// 16, twice); at(col, s) addresses A. The addresses are clamped and the values selected: with a
// branch around each load, each is waited for before the next (5 us of a small call).
template <bool DUP = false, typename F>
__device__ __forceinline__ ck_u32x4 mh_weights(const uint16_t *A, int col, int ncol, int ns, int k, int lane, F at) {
  uint32_t h[8];
  const int c = min(col, ncol - 1), last = DUP ? 15 : ~0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int s = 32 * k + ((mh_slot(lane >> 4, q >> 2) + (q & 3)) & last);
    h[q] = A[at(c, min(s, ns - 1))];
  }
  ck_u32x4 r;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int s = 32 * k + ((mh_slot(lane >> 4, q >> 1) + 2 * (q & 1)) & last);
    r[q] = (col < ncol && s < ns ? h[2 * q] : 0u) | (col < ncol && s + 1 < ns ? h[2 * q + 1] << 16 : 0u);
  }
  return r;
}

// four codes -> two dwords of storage halves (exact)
template <int DT>
__device__ __forceinline__ uint2 mh_decode4(uint32_t q, float step) {
  if constexpr (DT == DT_F16) {
    // bytes 128 + code as the low bits of 1024 + .. halves, less 1152, times 2^e
    const uint32_t b = q ^ 0x80808080u;
    const _Float16 s = (_Float16)step;
    const half2_t off = {(_Float16)-1152.f, (_Float16)-1152.f}, ss = {s, s};
    half2_t lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u));
    half2_t hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u));
    lo = (lo + off) * ss;
    hi = (hi + off) * ss;
    return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
  } else {
    const uint32_t a = __float_as_uint(ck_value(q, 0, step)), b = __float_as_uint(ck_value(q, 1, step));
    const uint32_t c = __float_as_uint(ck_value(q, 2, step)), d = __float_as_uint(ck_value(q, 3, step));
    return make_uint2(__builtin_amdgcn_perm(b, a, 0x07060302u), __builtin_amdgcn_perm(d, c, 0x07060302u));
  }
}

// Two values in pieces; mh_join puts the products' sums together
template <int DT>
__device__ __forceinline__ void mh_split(float a, float b, int e, uint32_t (&w)[mh_pieces<DT>()][8]) {
  if constexpr (DT == DT_F16) {
    half2_t h;
    h.x = (_Float16)(0.5f * a);
    h.y = (_Float16)(0.5f * b);
    w[0][e] = __builtin_bit_cast(uint32_t, h);
    w[1][e] = ck_pair<DT>(fmaf((float)h.x, -2048.f, 1024.f * a), fmaf((float)h.y, -2048.f, 1024.f * b));
  } else {
#pragma unroll
    for (int q = 0; q < 3; ++q) {  // each the upper 8 bits of what is left, the last all of it
      const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
      w[q][e] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
      a -= __uint_as_float(ua & 0xffff0000u);
      b -= __uint_as_float(ub & 0xffff0000u);
    }
  }
}

template <int DT>
__device__ __forceinline__ float mh_join(float hi, float lo) { return DT == DT_F16 ? fmaf(lo, 0x1p-10f, hi + hi) : hi; }

// zero the LDS rows past T tiles of 16 (half of the last of K 32-row steps): never written again
template <int T, int K, int PITCH, int THREADS>
__device__ __forceinline__ void mh_clear(uint16_t *s) {
  if constexpr (16 * T < 32 * K)
    for (int v = threadIdx.x; v < (32 * K - 16 * T) * PITCH; v += THREADS) s[16 * T * PITCH + v] = 0;
}

template <int DT, int OT, int IT>
__global__ __launch_bounds__((MhGeom<DT, OT, IT, true>::THREADS)) void fno_mix_save_half(MixTrainArgs a) {
  using G = MhGeom<DT, OT, IT, true>;
  extern __shared__ float4 lds4[];
  uint16_t *xs0 = reinterpret_cast<uint16_t *>(lds4);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, n = lane & 15;
  const int ow = wave % G::WO, pb = 64 * (wave / G::WO);
  const long P = a.P, nb = (P + kCkBlock - 1) / kCkBlock;
  const uint16_t *A = reinterpret_cast<const uint16_t *>(a.A);
  ck_u32x4 wf[G::KI];
  float bias;
  {
    const int o = 16 * (ow) + n;
    bias = mt_bias<DT>(a, o);
#pragma unroll
    for (int k = 0; k < G::KI; ++k)
      wf[k] = mh_weights(A, o, a.O, a.I, k, lane, [&](int c, int s) { return c * a.I + s; });
  }
  mh_clear<IT, G::KI, G::PITCH, G::THREADS>(xs0);
  mh_clear<IT, G::KI, G::PITCH, G::THREADS>(xs0 + G::XS / 2);
  const int t0 = blockIdx.x * a.per, t1 = min(a.tiles, t0 + a.per);
  // the next tile's x and add, in flight over a whole tile's work
  Px16<DT> xv[G::NU], nadd;
#pragma unroll
    for (int q = 0; q < 2; ++q) nadd.r[q] = ck_u32x4{0u, 0u, 0u, 0u};
  auto fetch = [&](int t) {
    const int b = t / a.tpb;
    const long p0 = (long)(t - b * a.tpb) * G::PT;
#pragma unroll
    for (int k = 0; k < G::NU; ++k) {
      const int u = tid + k * G::THREADS, i = u / (G::PT / 16), pu = 16 * (u % (G::PT / 16));
      const bool ok = (G::UNITS % G::THREADS == 0 || u < G::UNITS) && i < a.I;
      const size_t row = (size_t)b * a.I + (ok ? i : 0);
      if (p0 + G::PT <= P) {
        xv[k].load(a.x, row * P + p0 + pu, 16);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (!ok) xv[k].r[q] = ck_u32x4{0u, 0u, 0u, 0u};
      } else {
        xv[k].load(a.x, row * P + p0 + pu, ok ? P - p0 - pu : 0);
      }
    }
    if (a.add)
      {
        const int o = 16 * (ow) + n;
        const long p = p0 + pb + 16 * g;
        const size_t row = (size_t)b * a.O + min(o, a.O - 1);
        nadd.load(a.add, row * P + p, p0 + G::PT <= P ? 16 : o < a.O ? P - p : 0);
      }
  };
  if (t0 < t1) fetch(t0);
  for (int t = t0; t < t1; ++t) {
    const int b = t / a.tpb;
    const long p0 = (long)(t - b * a.tpb) * G::PT;
    const bool whole = p0 + G::PT <= P;
    uint16_t *xs = xs0 + (t & 1) * (G::XS / 2);  // the other buffer may still be read by a slower wave
#pragma unroll
    for (int k = 0; k < G::NU; ++k) {
      const int u = tid + k * G::THREADS, i = u / (G::PT / 16), pu = 16 * (u % (G::PT / 16));
      if (G::UNITS % G::THREADS != 0 && u >= G::UNITS) break;  // whole pairs of lanes
      const long p = p0 + pu;
      uint32_t key = xv[k].key();
      key = max(key, ck_dpp<kDppXor1>(key));
      const int e = ck_exponent<DT>(key);
      if (i < a.I && p < nb * kCkBlock) {
        const size_t row = (size_t)b * a.I + i;
        *reinterpret_cast<ck_u32x4 *>(a.xq + row * nb * kCkBlock + p) = xv[k].codes(e);
        if ((tid & 1) == 0) a.xe[row * nb + p / kCkBlock] = (int8_t)e;
      }
      uint16_t *d = xs + i * G::PITCH + pu;
      mh_write16(d, xv[k].r[0]);
      mh_write16(d + 8, xv[k].r[1]);
    }
    const long p = p0 + pb + 16 * g;
    Px16<DT> ad;
    ad = nadd;
    __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
    v4f z[4];
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) z[pt] = v4f{bias, bias, bias, bias};
#pragma unroll
    for (int k = 0; k < G::KI; ++k)
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) {
        const ck_u32x4 xa = mh_pixels<G::PITCH>(xs, k, pb, pt, lane);
        z[pt] = mh_mma<DT>(xa, wf[k], z[pt]);
      }
    {
      const int o = 16 * (ow) + n;
      const bool ok = o < a.O;
      const size_t row = (size_t)b * a.O + o;
      if (a.aq) {
        uint32_t key = ad.key();
        const auto s = __builtin_amdgcn_permlane16_swap(key, key, false, false);  // the block's other 16 pixels
        const int e = ck_exponent<DT>(max(s[0], s[1]));
        if (ok && p < nb * kCkBlock) {
          *reinterpret_cast<ck_u32x4 *>(a.aq + row * nb * kCkBlock + p) = ad.codes(e);
          if ((g & 1) == 0) a.ae[row * nb + p / kCkBlock] = (int8_t)e;
        }
      }
      float y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float v = z[e >> 2][e & 3] + ad.get(e);
        y[e] = a.act ? gelu_train(v) : v;
      }
      if (ok) store16<DT>(a.y, row * P + p, whole ? 16 : P - p, y);
    }
  }
}

template <int DT, int OT, int IT>
__global__ __launch_bounds__((MhGeom<DT, OT, IT, false>::THREADS))
    __attribute__((amdgpu_waves_per_eu(MhGeom<DT, OT, IT, false>::PER_EU))) void fno_mix_bwd_half(MixTrainArgs a) {
  using G = MhGeom<DT, OT, IT, false>;
  extern __shared__ float4 lds4[];
  uint16_t *xs = reinterpret_cast<uint16_t *>(lds4), *gs = xs + G::XS / 2;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, n = lane & 15;
  const int ow = wave % G::WO, pb = 64 * (wave / G::WO), iw = wave % G::WI;
  const long P = a.P, nb = (P + kCkBlock - 1) / kCkBlock;
  const uint16_t *A = reinterpret_cast<const uint16_t *>(a.A);
  ck_u32x4 wf[G::KI], wt[G::ITW][G::KO];
  float bias, gb;
  constexpr int NP = G::NP, NS = mh_sums<DT>();
  v4f ga[NS][IT];
  {
    const int o = 16 * (ow) + n;
    gb = 0.f;
    bias = mt_bias<DT>(a, o);
#pragma unroll
    for (int k = 0; k < G::KI; ++k)
      wf[k] = mh_weights(A, o, a.O, a.I, k, lane, [&](int c, int s) { return c * a.I + s; });
#pragma unroll
    for (int it = 0; it < IT; ++it) ga[0][it] = ga[NS - 1][it] = v4f{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int m = 0; m < G::ITW; ++m)
#pragma unroll
    for (int k = 0; k < G::KO; ++k)
      wt[m][k] = mh_weights<DT == DT_BF16 && OT == 1>(A, 16 * (iw + G::WI * m) + n, a.I, a.O, k, lane, [&](int c, int s) { return s * a.I + c; });
  mh_clear<IT, G::KI, G::PITCH, G::THREADS>(xs);
  if constexpr (DT == DT_F16) {
#pragma unroll
    for (int q = 0; q < NP; ++q) mh_clear<OT, G::KO, G::PITCH, G::THREADS>(gs + q * G::ROWS * G::PITCH);
  } else {
    mh_clear<NP * OT, G::KS, G::PITCH, G::THREADS>(gs);
  }
  const int t0 = blockIdx.x * a.per, t1 = min(a.tiles, t0 + a.per);
  // the next tile's codes of x and add and its gy, in flight over a whole tile's work
  Code16 xc[G::NU], nac;
  Px16<DT> ngy;
  auto fetch = [&](int t) {
    const int b = t / a.tpb;
    const long p0 = (long)(t - b * a.tpb) * G::PT;
#pragma unroll
    for (int k = 0; k < G::NU; ++k) {
      const int u = tid + k * G::THREADS, i = u / (G::PT / 16), pu = 16 * (u % (G::PT / 16));
      xc[k].load(a.xq, a.xe, (size_t)b * a.I + i, p0 + pu, nb, (G::UNITS % G::THREADS == 0 || u < G::UNITS) && i < a.I);
    }
    const long p = p0 + pb + 16 * g;
    {
      const int o = 16 * (ow) + n;
      const size_t row = (size_t)b * a.O + min(o, a.O - 1);
      if (p0 + G::PT <= P) {
        ngy.load(a.gy, row * P + p, 16);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (o >= a.O) ngy.r[q] = ck_u32x4{0u, 0u, 0u, 0u};
      } else {
        ngy.load(a.gy, row * P + p, o < a.O ? P - p : 0);
      }
      nac.load(a.aq, a.ae, row, p, nb, a.aq && o < a.O);
    }
  };
  if (t0 < t1) fetch(t0);
  for (int t = t0; t < t1; ++t) {
    const int b = t / a.tpb;
    const long p0 = (long)(t - b * a.tpb) * G::PT;
    const bool whole = p0 + G::PT <= P;
    const long p = p0 + pb + 16 * g;
    Px16<DT> gy;
    Code16 ac;
    {
      gy = ngy;
      ac = nac;
    }
#pragma unroll
    for (int k = 0; k < G::NU; ++k) {
      const int u = tid + k * G::THREADS, i = u / (G::PT / 16), pu = 16 * (u % (G::PT / 16));
      if (G::UNITS % G::THREADS != 0 && u >= G::UNITS) break;
      const float s = ck_step(xc[k].e);
      uint2 *d = reinterpret_cast<uint2 *>(xs + i * G::PITCH + pu);
#pragma unroll
      for (int q = 0; q < 4; ++q) d[q] = mh_decode4<DT>(xc[k].q[q], s);
    }
    __syncthreads();
    if (t + 1 < t1) fetch(t + 1);
    v4f z[4];
    if (a.act) {
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) z[pt] = v4f{bias, bias, bias, bias};
#pragma unroll
      for (int k = 0; k < G::KI; ++k)
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) {
          const ck_u32x4 xa = mh_pixels<G::PITCH>(xs, k, pb, pt, lane);
          z[pt] = mh_mma<DT>(xa, wf[k], z[pt]);
        }
    }
    {
      const int o = 16 * (ow) + n;
      float gz[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) gz[e] = gy.get(e);
      if (a.act) {
        const float s = ck_step(ac.e);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          gz[e] *= gelu_slope(fmaf((float)(int8_t)(ac.q[e >> 2] >> (8 * (e & 3))), s, z[e >> 2][e & 3]));
      }
      if (a.gadd && o < a.O) store16<DT>(a.gadd, ((size_t)b * a.O + o) * P + p, whole ? 16 : P - p, gz);
      uint32_t w[NP][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mh_split<DT>(gz[2 * e], gz[2 * e + 1], e, w);
      const int at = (16 * (ow) + n) * G::PITCH + pb + 16 * g;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < NP; ++c)
          reinterpret_cast<uint2 *>(gs + c * G::ROWS * G::PITCH + at)[q] = make_uint2(w[c][2 * q], w[c][2 * q + 1]);
      if (a.part) {
#pragma unroll
        for (int e = 0; e < 16; ++e) gb += gz[e];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ck_u32x4 h[NP];
#pragma unroll
          for (int c = 0; c < NP; ++c) h[c] = ck_u32x4{w[c][4 * k], w[c][4 * k + 1], w[c][4 * k + 2], w[c][4 * k + 3]};
#pragma unroll
          for (int it = 0; it < IT; ++it) {
            const ck_u32x4 xv = mh_read16(xs + (16 * it + n) * G::PITCH + pb + 16 * g + 8 * k);
#pragma unroll
            for (int c = 0; c < NP; ++c) ga[c % NS][it] = mh_mma<DT>(h[c], xv, ga[c % NS][it]);
          }
        }
      }
    }
    __syncthreads();
    if (a.gx) {
#pragma unroll
      for (int m = 0; m < G::ITW; ++m) {
        const int i = 16 * (iw + G::WI * m) + n;
        for (int sb = 64 * (wave / G::WI); sb < G::PT; sb += 64 * (G::WAVES / G::WI)) {
          v4f acc[NS][4];
#pragma unroll
          for (int q = 0; q < NS; ++q)
#pragma unroll
            for (int pt = 0; pt < 4; ++pt) acc[q][pt] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < G::KO; ++k)
#pragma unroll
            for (int pt = 0; pt < 4; ++pt)
#pragma unroll
              for (int c = 0; c < G::KS / G::KO; ++c)  // the channels once more: the next piece of their gz
                acc[c % NS][pt] = mh_mma<DT>(mh_pixels<G::PITCH>(gs + c * G::KO * 32 * G::PITCH, k, sb, pt, lane), wt[m][k],
                                             acc[c % NS][pt]);
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = mh_join<DT>(acc[0][e >> 2][e & 3], acc[NS - 1][e >> 2][e & 3]);
          const long q = p0 + sb + 16 * g;
          if (i < a.I) store16<DT>(a.gx, ((size_t)b * a.I + i) * P + q, whole ? 16 : P - q, v);
        }
      }
    }
    // the next tile's channels overwrite xs, last read before the barrier above;
    // its gz overwrite gs only after the next barrier
  }
  if (!a.part) return;
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
      for (int j = 0; j < 4; ++j) ga[0][it][j] = mh_join<DT>(ga[0][it][j], ga[NS - 1][it][j]);
  mt_finish<OT, IT, G::WP, G::THREADS>(a, ga[0], gb, reinterpret_cast<float *>(lds4), wave, lane);
}

template <int DT, int OT, int IT>
MtPick mh_pick3() {
  using F = MhGeom<DT, OT, IT, true>;
  using G = MhGeom<DT, OT, IT, false>;
  constexpr int by_lds = 160 * 1024 / G::LDS_BWD, by_regs = 4 * G::PER_EU / G::WAVES;
  return {(const void *)fno_mix_save_half<DT, OT, IT>,
          (const void *)fno_mix_bwd_half<DT, OT, IT>,
          F::PT,
          G::PT,
          (size_t)F::LDS_FWD,
          (size_t)G::LDS_BWD,
          F::THREADS,
          G::THREADS,
          256 * (by_lds < by_regs ? by_lds : by_regs)};
}
template <int DT, int OT>
MtPick mh_pick2(int I) {
  return I <= 16 ? mh_pick3<DT, OT, 1>() : I <= 32 ? mh_pick3<DT, OT, 2>() : I <= 64 ? mh_pick3<DT, OT, 4>()
                                                                                     : mh_pick3<DT, OT, 8>();
}
template <int DT>
MtPick mh_pick(int O, int I) {
  return O <= 16 ? mh_pick2<DT, 1>(I) : O <= 32 ? mh_pick2<DT, 2>(I) : O <= 64 ? mh_pick2<DT, 4>(I) : mh_pick2<DT, 8>(I);
}

}  // namespace fno
