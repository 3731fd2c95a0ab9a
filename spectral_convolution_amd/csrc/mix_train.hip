// mix_train.hip - the channel mix of a training step: a forward that keeps its
// inputs in 8 bits, and the backward from them.
//
//   forward   z = A x + bias + add,  y = act(z);  x (and add where act needs z
//             again) kept as checkpoints (checkpoint.hpp)
//   backward  z from the kept values, gz = gy act'(z),
//             gx = A^T gz,  gA = sum over pixels of gz x^T,  gbias = sum gz,  gadd = gz
// for every sample and pixel, [batch][channels][pixels], act none or GELU.
//
// A workgroup takes tiles of 64 WP pixels and all channels (c_out in OT, c_in in
// IT tiles of 16): the OT waves of a 64-pixel part have one tile of the output
// channels each, WP parts go side by side to make four waves (eight where OT is). The
// channels' values are staged in LDS, [channel][pixel], once; every product
// runs on matrix cores with fp32 accumulation:
//   z   D[pixel][o], from x (A operand) and A^T (B operand, in registers)
//   gA  D[o][i], from gz straight out of the registers (a lane's 16 pixels of
//       one o are 16 steps of the sum) and x from LDS
//   gx  D[pixel][i], from gz (through LDS: the waves exchange their channels)
//       and A (B operand, in registers)
// The rows of a product tile are assigned to pixels so that a lane ends up with
// 16 consecutive pixels of one channel: every access to the fields and codes is
// 16 bytes or more of a row, with no staging of outputs.
// gA and gbias stay in registers over a workgroup's run of tiles, go to the
// workspace once and are added in a fixed order by fno_mix_params.
//
// Measured (MI355X; forward + backward, a pass among others): 32 x 64 x 64 channels, 256^2, fp16 545
// us, 4.0 TB/s against 5.1 of a copy (vector instructions 67 % of the issue slots in the
// backward, half of them GELU's derivative and the split of gz), bf16 559 us; 16 x 32 x 32,
// 128^2, fp32 70 us, 3.4 TB/s; 16 x 128 x 128, 128^2, fp32 502 us: 206 us forward, 1.9 TB/s and 27 %
// of the fp32 matrix rate (154 TFLOP/s of a library product), backward 297 us, 57 % of it: two
// waves a SIMD that wait at the same barriers, nothing loaded ahead.

#include <algorithm>

#include "mix_train.hpp"

namespace fno {

namespace {

template <int OT, int IT>
struct MtGeom {
  static constexpr int WAVES = OT == 8 ? 8 : 4, THREADS = 64 * WAVES;
  static constexpr int WO = OT, WP = WAVES / WO, WI = IT < WAVES ? IT : WAVES, ITW = IT / WI;
  static constexpr int PT = 64 * WP, PITCH = PT + 4;   // floats
  static constexpr int XS = IT * 16 * PITCH * 4, GS = OT * 16 * PITCH * 4;
  static constexpr int UNITS = IT * 16 * (PT / 16), NU = (UNITS + THREADS - 1) / THREADS;
  // A tile's inputs are loaded a tile ahead (16 x 128 x 128 pixels, 32 channels: 83
  // us a step instead of 89) where they fit the registers, and the forward's second
  // buffer the LDS, at the same occupancy (128 channels: 550 us instead of 508).
  static constexpr bool AHEAD = NU <= 2 && OT * IT <= 16;
  static constexpr int LDS_FWD = (AHEAD ? 2 : 1) * XS;
};

// A[o][i], 0 past the channels; the address is clamped and the value selected, so
// that a wave's loads follow each other without a wait
__device__ __forceinline__ float mt_weight(const MixTrainArgs &a, int o, int i) {
  const float v = mt_load1<DT_F32>(a.A, (size_t)min(o, a.O - 1) * a.I + min(i, a.I - 1));
  return o < a.O && i < a.I ? v : 0.f;
}

// z of 16 pixels of the wave's output channels: zv[m][4 j + pt], without bias
template <int OT, int IT>
__device__ __forceinline__ void mt_z(const float *xs, int pb, int lane, const float (&wf)[IT * 4],
                                     v4f (&z)[4]) {
  using G = MtGeom<OT, IT>;
  const int g = lane >> 4, n = lane & 15;
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) z[pt] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kk = 0; kk < IT * 4; ++kk) {
    const float4 a = *reinterpret_cast<const float4 *>(xs + (4 * kk + g) * G::PITCH + pb + 4 * n);
    const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int pt = 0; pt < 4; ++pt)
        z[pt] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[pt], wf[kk], z[pt], 0, 0, 0);
  }
}

}  // namespace

template <int OT, int IT>
__global__ __launch_bounds__((MtGeom<OT, IT>::THREADS)) void fno_mix_save(MixTrainArgs a) {
  using G = MtGeom<OT, IT>;
  extern __shared__ float4 lds4[];
  float *xs0 = reinterpret_cast<float *>(lds4);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, n = lane & 15;
  const int ow = wave % G::WO, pb = 64 * (wave / G::WO);
  const long P = a.P, nb = (P + kCkBlock - 1) / kCkBlock;
  float wf[IT * 4], bias;
  {
    const int o = 16 * (ow) + n;
    bias = mt_bias<DT_F32>(a, o);
#pragma unroll
    for (int kk = 0; kk < IT * 4; ++kk) {
      const int i = 4 * kk + g;
      wf[kk] = mt_weight(a, o, i);
    }
  }
  const int t0 = blockIdx.x * a.per, t1 = min(a.tiles, t0 + a.per);
  Px16<DT_F32> xv[G::NU], nadd;
#pragma unroll
  for (int q = 0; q < 4; ++q) nadd.r[q] = ck_u32x4{0u, 0u, 0u, 0u};
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
        for (int q = 0; q < 4; ++q)
          if (!ok) xv[k].r[q] = ck_u32x4{0u, 0u, 0u, 0u};
      } else {
        xv[k].load(a.x, row * P + p0 + pu, ok ? P - p0 - pu : 0);
      }
    }
    if (a.add) {
      const int o = 16 * ow + n;
      const long p = p0 + pb + 16 * g;
      const size_t row = (size_t)b * a.O + min(o, a.O - 1);
      if (p0 + G::PT <= P) nadd.load64(a.add, row * P + p0 + pb, lane);
      else nadd.load(a.add, row * P + p, o < a.O ? P - p : 0);
    }
  };
  if (G::AHEAD && t0 < t1) fetch(t0);
  for (int t = t0; t < t1; ++t) {
    const int b = t / a.tpb;
    const long p0 = (long)(t - b * a.tpb) * G::PT;
    const bool whole = p0 + G::PT <= P;
    if (!G::AHEAD) fetch(t);
    // the other buffer may still be read by a slower wave
    float *xs = xs0 + (G::AHEAD && (t & 1) ? G::XS / 4 : 0);
#pragma unroll
    for (int k = 0; k < G::NU; ++k) {
      const int u = tid + k * G::THREADS, i = u / (G::PT / 16), pu = 16 * (u % (G::PT / 16));
      if (G::UNITS % G::THREADS != 0 && u >= G::UNITS) break;  // whole pairs of lanes
      const long p = p0 + pu;
      const size_t row = (size_t)b * a.I + i;
      uint32_t key = xv[k].key();
      key = max(key, ck_dpp<kDppXor1>(key));
      const int e = ck_exponent<DT_F32>(key);
      if (i < a.I && p < nb * kCkBlock) {
        *reinterpret_cast<ck_u32x4 *>(a.xq + row * nb * kCkBlock + p) = xv[k].codes(e);
        if (p % kCkBlock == 0) a.xe[row * nb + p / kCkBlock] = (int8_t)e;
      }
      float *d = xs + i * G::PITCH + pu;
#pragma unroll
      for (int q = 0; q < 4; ++q) reinterpret_cast<ck_u32x4 *>(d)[q] = xv[k].r[q];
    }
    Px16<DT_F32> ad = nadd;
    if (whole) mt_exchange(ad.r);
    __syncthreads();
    if (G::AHEAD && t + 1 < t1) fetch(t + 1);
    v4f z[4];
    mt_z<OT, IT>(xs, pb, lane, wf, z);
    const long p = p0 + pb + 16 * g;
    {
      const int o = 16 * (ow) + n;
      const bool ok = o < a.O;
      const size_t row = (size_t)b * a.O + o;
      if (a.aq) {
        uint32_t key = ad.key();
        const auto s = __builtin_amdgcn_permlane16_swap(key, key, false, false);  // the block's other 16 pixels
        const int e = ck_exponent<DT_F32>(max(s[0], s[1]));
        if (ok && p < nb * kCkBlock) {
          *reinterpret_cast<ck_u32x4 *>(a.aq + row * nb * kCkBlock + p) = ad.codes(e);
          if (p % kCkBlock == 0) a.ae[row * nb + p / kCkBlock] = (int8_t)e;
        }
      }
      float y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float v = z[e & 3][e >> 2] + bias + ad.get(e);
        y[e] = a.act ? gelu_train(v) : v;
      }
      if (ok) {
        if (whole) store64(a.y, row * P + p0 + pb, lane, y);
        else store16<DT_F32>(a.y, row * P + p, P - p, y);
      }
    }
    if (!G::AHEAD) __syncthreads();
  }
}

template <int OT, int IT>
__global__ __launch_bounds__((MtGeom<OT, IT>::THREADS)) void fno_mix_bwd(MixTrainArgs a) {
  using G = MtGeom<OT, IT>;
  extern __shared__ float4 lds4[];
  float *xs = reinterpret_cast<float *>(lds4), *gs = xs + G::XS / 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, n = lane & 15;
  const int ow = wave % G::WO, pb = 64 * (wave / G::WO), iw = wave % G::WI;
  const long P = a.P, nb = (P + kCkBlock - 1) / kCkBlock;
  float wf[IT * 4], wt[G::ITW][OT * 4], bias, gb;
  v4f ga[IT];
  {
    const int o = 16 * (ow) + n;
    gb = 0.f;
    bias = mt_bias<DT_F32>(a, o);
#pragma unroll
    for (int kk = 0; kk < IT * 4; ++kk) {
      const int i = 4 * kk + g;
      wf[kk] = mt_weight(a, o, i);
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) ga[it] = v4f{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int m = 0; m < G::ITW; ++m)
#pragma unroll
    for (int kk = 0; kk < OT * 4; ++kk) {
      const int o = 4 * kk + g, i = 16 * (iw + G::WI * m) + n;
      wt[m][kk] = mt_weight(a, o, i);
    }
  const int t0 = blockIdx.x * a.per, t1 = min(a.tiles, t0 + a.per);
  Code16 xc[G::NU], nac;
  Px16<DT_F32> ngy;
  auto fetch = [&](int t) {
    const int b = t / a.tpb;
    const long p0 = (long)(t - b * a.tpb) * G::PT;
#pragma unroll
    for (int k = 0; k < G::NU; ++k) {
      const int u = tid + k * G::THREADS, i = u / (G::PT / 16), pu = 16 * (u % (G::PT / 16));
      xc[k].load(a.xq, a.xe, (size_t)b * a.I + i, p0 + pu, nb, (G::UNITS % G::THREADS == 0 || u < G::UNITS) && i < a.I);
    }
    const long p = p0 + pb + 16 * g;
    const int o = 16 * ow + n;
    const size_t row = (size_t)b * a.O + min(o, a.O - 1);
    if (p0 + G::PT <= P) {
      ngy.load64(a.gy, row * P + p0 + pb, lane);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (o >= a.O) ngy.r[q] = ck_u32x4{0u, 0u, 0u, 0u};
    } else {
      ngy.load(a.gy, row * P + p, o < a.O ? P - p : 0);
    }
    nac.load(a.aq, a.ae, row, p, nb, a.aq && o < a.O);
  };
  if (G::AHEAD && t0 < t1) fetch(t0);
  for (int t = t0; t < t1; ++t) {
    const int b = t / a.tpb;
    const long p0 = (long)(t - b * a.tpb) * G::PT;
    const bool whole = p0 + G::PT <= P;
    if (!G::AHEAD) fetch(t);
    Px16<DT_F32> gy = ngy;
    if (whole) mt_exchange(gy.r);
    const Code16 ac = nac;
#pragma unroll
    for (int k = 0; k < G::NU; ++k) {
      const int u = tid + k * G::THREADS, i = u / (G::PT / 16), pu = 16 * (u % (G::PT / 16));
      if (G::UNITS % G::THREADS != 0 && u >= G::UNITS) break;
      const Code16 &c = xc[k];
      const float s = ck_step(c.e);
      float *d = xs + i * G::PITCH + pu;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        reinterpret_cast<float4 *>(d)[q] =
            make_float4(c.get(4 * q, s), c.get(4 * q + 1, s), c.get(4 * q + 2, s), c.get(4 * q + 3, s));
    }
    __syncthreads();
    if (G::AHEAD && t + 1 < t1) fetch(t + 1);
    v4f z[4];
    if (a.act) mt_z<OT, IT>(xs, pb, lane, wf, z);
    const long p = p0 + pb + 16 * g;
    {
      const int o = 16 * (ow) + n;
      const bool ok = o < a.O;
      const size_t row = (size_t)b * a.O + o;
      float gz[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) gz[e] = gy.get(e);
      if (a.act) {
        const float s = ck_step(ac.e);
#pragma unroll
        for (int e = 0; e < 16; ++e) gz[e] *= gelu_slope(z[e & 3][e >> 2] + bias + ac.get(e, s));
      }
      if (a.gadd && ok) {
        const size_t at = row * P + p0 + pb;
        if (whole) store64(a.gadd, at, lane, gz);
        else store16<DT_F32>(a.gadd, at + 16 * g, P - p, gz);
      }
      float *d = gs + (16 * (ow) + n) * G::PITCH + pb + 16 * g;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        reinterpret_cast<float4 *>(d)[q] = make_float4(gz[4 * q], gz[4 * q + 1], gz[4 * q + 2], gz[4 * q + 3]);
      if (a.part) {
#pragma unroll
        for (int e = 0; e < 16; ++e) gb += gz[e];
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 xv = *reinterpret_cast<const float4 *>(xs + (16 * it + n) * G::PITCH + pb + 16 * g + 4 * q);
            ga[it] = __builtin_amdgcn_mfma_f32_16x16x4f32(gz[4 * q], xv.x, ga[it], 0, 0, 0);
            ga[it] = __builtin_amdgcn_mfma_f32_16x16x4f32(gz[4 * q + 1], xv.y, ga[it], 0, 0, 0);
            ga[it] = __builtin_amdgcn_mfma_f32_16x16x4f32(gz[4 * q + 2], xv.z, ga[it], 0, 0, 0);
            ga[it] = __builtin_amdgcn_mfma_f32_16x16x4f32(gz[4 * q + 3], xv.w, ga[it], 0, 0, 0);
          }
      }
    }
    __syncthreads();
    if (a.gx) {
#pragma unroll
      for (int m = 0; m < G::ITW; ++m) {
        const int i = 16 * (iw + G::WI * m) + n;
        for (int sb = 64 * (wave / G::WI); sb < G::PT; sb += 64 * (G::WAVES / G::WI)) {
          v4f acc[4] = {v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}, v4f{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int kk = 0; kk < OT * 4; ++kk) {
            const float4 v = *reinterpret_cast<const float4 *>(gs + (4 * kk + g) * G::PITCH + sb + 4 * n);
            const float av[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int pt = 0; pt < 4; ++pt)
              acc[pt] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[pt], wt[m][kk], acc[pt], 0, 0, 0);
          }
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = acc[e & 3][e >> 2];
          const long q = p0 + sb + 16 * g;
          if (i < a.I) {
            const size_t at = ((size_t)b * a.I + i) * P + p0 + sb;
            if (whole) store64(a.gx, at, lane, v);
            else store16<DT_F32>(a.gx, at + 16 * g, P - q, v);
          }
        }
      }
    }
    // the next tile's channels overwrite xs, last read before the barrier above;
    // its gz overwrite gs only after the next barrier
  }
  if (!a.part) return;
  mt_finish<OT, IT, G::WP, G::THREADS>(a, ga, gb, xs, wave, lane);
}

// gA and gbias from the workgroups' sums part[S][O I + O]: 32 elements a
// workgroup, 32 slices of the S.
template <int DT>
__global__ __launch_bounds__(1024) void fno_mix_params(MixTrainArgs a, int S) {
  __shared__ float red[32][33];
  const int l = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const long na = (long)a.O * a.I, ne = na + a.O, e = blockIdx.x * 32L + l;
  float v = 0.f;
  if (e < ne) {
#pragma unroll 8
    for (int s = sl; s < S; s += 32) v += a.part[(size_t)s * ne + e];
  }
  red[sl][l] = v;
  __syncthreads();
  if (threadIdx.x >= 32 || e >= ne) return;
  v = 0.f;
  for (int s = 0; s < 32; ++s) v += red[s][l];
  void *d = e < na ? a.gA : a.gbias;
  const long i = e < na ? e : e - na;
  if (!d) return;
  if constexpr (DT == DT_F32) reinterpret_cast<float *>(d)[i] = v;
  else if constexpr (DT == DT_F16) reinterpret_cast<_Float16 *>(d)[i] = (_Float16)v;
  else reinterpret_cast<uint16_t *>(d)[i] = (uint16_t)f32_to_bf16(v);
}

// ------------------------------------------------------------------ launch

namespace {

template <int OT, int IT>
MtPick mt_pick3() {
  using G = MtGeom<OT, IT>;
  return {(const void *)fno_mix_save<OT, IT>, (const void *)fno_mix_bwd<OT, IT>, G::PT, G::PT, (size_t)G::LDS_FWD,
          (size_t)(G::XS + G::GS), G::THREADS, G::THREADS, 1024 / G::WAVES * 2};
}
template <int OT>
MtPick mt_pick2(int I) {
  return I <= 16 ? mt_pick3<OT, 1>() : I <= 32 ? mt_pick3<OT, 2>() : I <= 64 ? mt_pick3<OT, 4>() : mt_pick3<OT, 8>();
}
MtPick mt_pick(int O, int I, int dtype) {
  if (dtype == DT_F16) return mix_train_f16(O, I);
  if (dtype == DT_BF16) return mix_train_bf16(O, I);
  return O <= 16 ? mt_pick2<1>(I) : O <= 32 ? mt_pick2<2>(I) : O <= 64 ? mt_pick2<4>(I) : mt_pick2<8>(I);
}

// Workgroups of a call, each a contiguous run of tiles; fills the tiling in. The
// backward takes as many as the chip holds at once: with a few more, the last
// ones run alone (1024 of 768: 382 us against 300 at 32 x 64 x 64 channels, 256^2, fp16).
// fp32: two workgroups of four waves a CU, one of eight. Where registers or LDS hold one of the
// former only (eight tiles of c_in, or four and one of c_out) these are two full rounds, and one round is no
// better on the whole (16 x 128^2 pixels: 128 x 16 channels 84 us, 88 in one; 128 x 64 174, 167 in one).
int mt_runs(MixTrainArgs &a, int pt, long most) {
  a.tpb = (int)((a.P + pt - 1) / pt);
  a.tiles = a.B * a.tpb;
  const int m = (int)std::min((long)a.tiles, most);
  a.per = (a.tiles + m - 1) / m;
  return (a.tiles + a.per - 1) / a.per;
}

constexpr long kMtForward = 2048;

}  // namespace

size_t mix_train_workspace_bytes(int B, int I, int O, long P, int dtype) {
  MixTrainArgs a{};
  a.B = B, a.P = P;
  const MtPick k = mt_pick(O, I, dtype);
  return (size_t)mt_runs(a, k.pt_bwd, k.resident) * ((size_t)O * I + O) * 4;
}

hipError_t launch_mix_save(const MixTrainArgs &a, int dtype, hipStream_t s) {
  const MtPick k = mt_pick(a.O, a.I, dtype);
  MixTrainArgs arg = a;
  const int S = mt_runs(arg, k.pt_fwd, kMtForward);
  FNO_BOUNDS(check_mix_train(arg, true, S, k.lds_fwd, dtype, k.pt_fwd, k.threads_fwd);)
  if (hipError_t e = raise_lds_cap(k.fwd, k.lds_fwd); e != hipSuccess) return e;
  void *args[] = {(void *)&arg};
  return hipLaunchKernel(k.fwd, dim3((unsigned)S), dim3((unsigned)k.threads_fwd), args, k.lds_fwd, s);
}

hipError_t launch_mix_bwd(const MixTrainArgs &a, int dtype, hipStream_t s) {
  const MtPick k = mt_pick(a.O, a.I, dtype);
  MixTrainArgs arg = a;
  int S = mt_runs(arg, k.pt_bwd, k.resident);
  FNO_BOUNDS(check_mix_train(arg, false, S, k.lds_bwd, dtype, k.pt_bwd, k.threads_bwd);)
  if (hipError_t e = raise_lds_cap(k.bwd, k.lds_bwd); e != hipSuccess) return e;
  void *args[] = {(void *)&arg};
  hipError_t e = hipLaunchKernel(k.bwd, dim3((unsigned)S), dim3((unsigned)k.threads_bwd), args, k.lds_bwd, s);
  if (e != hipSuccess || !a.part) return e;
  void *pargs[] = {(void *)&arg, (void *)&S};
  const void *pk = dtype == DT_F32 ? (const void *)fno_mix_params<DT_F32>
                   : dtype == DT_F16 ? (const void *)fno_mix_params<DT_F16>
                                     : (const void *)fno_mix_params<DT_BF16>;
  const long ne = (long)a.O * a.I + a.O;
  return hipLaunchKernel(pk, dim3((unsigned)((ne + 31) / 32)), dim3(1024), pargs, 0, s);
}

}  // namespace fno
