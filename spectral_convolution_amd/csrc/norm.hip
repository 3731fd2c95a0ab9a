// norm.hip - the norms before and after a block, fused with its gate and
// residual scale, forward and backward.
//
// For every sample b and pixel p, over the channels c (C of them):
//   N(v)[c] = (v[c] - m) r w_post[c] + b_post[c]
//   y[c]    = x[c] + scale[c] gate[b][c] N(v)[c]
//   u[c]    = (y[c] - m') r' w_pre[c] + b_pre[c]
// with m the mean over c (layer norm; 0 for the root-mean-square norm), r =
// 1 / sqrt(mean((v - m)^2) + eps), and m', r' the same of y. v is a block's
// branch output, y the residual stream and u the next block's input.
//
// Backward, at gy = dL/dy and gu = dL/du: with a unit-scale norm h^ = (h - m) r
// and g = dL/dh^, dL/dh = r (g - h^ mean(g h^) - [layer] mean(g)). So
//   gx = gy + [that of y at g = gu w_pre],
//   gv = [that of v at g = gx scale gate w_post],
// and with the per-(b, c) sums over pixels
//   T = sum gx v^,  G = sum gx,  U = sum gu y^,  V = sum gu:
//   g_gate = scale (w_post T + b_post G),  g_scale = sum_b gate (w_post T + b_post G),
//   g_w_post = scale sum_b gate T,  g_b_post = scale sum_b gate G,
//   g_w_pre = sum_b U,  g_b_pre = sum_b V.
//
// Statistics, sums and everything between load and store are fp32; the
// variance is the mean of squared deviations from the mean already known, so
// a large mean costs no digits. Means are divided, not multiplied by 1 / C: with
// equal channels h - m is then 0, where an m one rounding off times r = eps^-1/2
// would not be. y's statistics are those of the unrounded y.
//
// Fields ([B][C][P], P > 1; fno_norm_fwd / fno_norm_bwd): a tile is all
// channels of 128 bytes of each row (64 pixels in 16 bits, 32 in fp32), one
// checkpoint block or two. A wave holds 8 CPT channels of it in registers: lane l
// owns 16 bytes of pixels (l % 8) of the channels l / 8 + 8 k, so every
// access covers 8 whole 128-byte lines, each input is read once and each
// output written once. The sums over channels are folded across the wave with
// row and half swaps that halve the values held with each step (14 operations for 8
// pixels instead of the 24 of a butterfly) and, where the channels need more
// than one wave, joined through LDS. Bound by memory.
//
// Token layout (P = 1; fno_norm_tok_fwd / _bwd): channels are contiguous and a
// row is held by one wave or by a workgroup (norm_token.hpp).
//
// The backward's sums over pixels stay with their thread (in LDS, from three
// channels a lane on; tokens: in registers) over a workgroup's run and go to the
// workspace once; fno_norm_params adds them in a fixed order, so results do not
// change from run to run.
//
// Measured (MI355X; a 1 GiB copy runs at 5.1 TB/s): forward of 32 x 64 x 256^2 fp16
// 199 us, 5.4 TB/s; backward of 4 x 32 x 64^3 fp32 161 us (5.0 TB/s) in a loop of its own,
// 176 among others; forward with checkpoints and backward from them of 20 x 64 x
// 256^2 fp16 144 + 164 us, 5.4 TB/s (layer norm: 368 for both, its backward spills 44 bytes a lane).
// 8192 x 1024 bf16 tokens, their fields (67 MB) from memory: forward 23 us (24 in a kernel trace;
// 18 to 19 with up to three sets of fields in turn, which the 256 MB cache partly holds), backward 43 (38 in a trace).

#include <algorithm>

#include "norm_common.hpp"

namespace fno {

// Parameter gradients of a field from the runs' sums part[4][C][B][S]: one
// workgroup per channel. A sample has 16 / B of its 16 waves, or a wave has a sample
// in turn; four loads of each sum are in flight (one wave a sample and one load: 9.5
// us instead of 5 at 20 samples of 171 runs).
template <int DT>
__global__ __launch_bounds__(1024) void fno_norm_params(NormArgs a, int S) {
  __shared__ float red[16][5];
  __shared__ float4 joint[16];
  const int c = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int share = a.B < 16 ? 16 / a.B : 1, slots = 16 / share, part = wave % share;
  const uint32_t wb = param_bits<DT>(a.w_post, a.gy, c), bb = param_bits<DT>(a.b_post, a.gy, c),
                 sb = param_bits<DT>(a.scale, a.gy, c);
  const size_t kstep = (size_t)a.C * a.B * S;
  const float w = param_value<DT>(a.w_post, wb, 1.f), bp = param_value<DT>(a.b_post, bb, 0.f),
              sc = param_value<DT>(a.scale, sb, 1.f);
  float t[5] = {0.f, 0.f, 0.f, 0.f, 0.f};  // sums over b of gate T, gate G, U, V and gate (w_post T + b_post G)
  for (int b0 = 0; b0 < a.B; b0 += slots) {  // once where waves share a sample
    const int b = b0 + wave / share;
    const bool ok = b < a.B;
    const uint32_t gb = param_bits<DT>(a.gate, a.gy, (size_t)min(b, a.B - 1) * a.C + c);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok) {
      const float *src = a.part + ((size_t)c * a.B + b) * S;
      for (int i = 64 * part + lane; i < S; i += 256 * share) {
        float l[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int j = i + 64 * share * r;
            l[r][q] = j < S ? src[q * kstep + j] : 0.f;
          }
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += (l[0][q] + l[1][q]) + (l[2][q] + l[3][q]);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = sum64(v[q]);
    if (share > 1) {
      if (lane == 0) joint[wave] = make_float4(v[0], v[1], v[2], v[3]);
      __syncthreads();
      if (part != 0 || !ok) break;
      for (int r = 1; r < share; ++r) {
        const float4 o = joint[wave + r];
        v[0] += o.x, v[1] += o.y, v[2] += o.z, v[3] += o.w;
      }
    }
    if (!ok) break;
    const float g = param_value<DT>(a.gate, gb, 1.f), n = fmaf(w, v[0], bp * v[1]);
    if (lane == 0) put<DT>(a.g_gate, (size_t)b * a.C + c, sc * n);
    t[0] = fmaf(g, v[0], t[0]);
    t[1] = fmaf(g, v[1], t[1]);
    t[2] += v[2];
    t[3] += v[3];
    t[4] = fmaf(g, n, t[4]);
  }
  if (lane == 0)
#pragma unroll
    for (int q = 0; q < 5; ++q) red[wave][q] = t[q];
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int q = 0; q < 5; ++q) {
    t[q] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t[q] += red[i][q];
  }
  put<DT>(a.g_w_post, c, sc * t[0]);
  put<DT>(a.g_b_post, c, sc * t[1]);
  put<DT>(a.g_w_pre, c, t[2]);
  put<DT>(a.g_b_pre, c, t[3]);
  put<DT>(a.g_scale, c, t[4]);
}

// Parameter gradients of tokens from part[S][4][C]: 32 channels and two of the
// four sums a workgroup, 32 slices of the runs.
template <int DT>
__global__ __launch_bounds__(1024) void fno_norm_tok_params(NormArgs a, int S) {
  __shared__ float red[2][32][33];
  const int l = threadIdx.x & 31, sl = threadIdx.x >> 5, c = blockIdx.x * 32 + l, half = blockIdx.y;
  float v[2] = {0.f, 0.f};
  if (c < a.C) {
#pragma unroll 8
    for (int i = sl; i < S; i += 32)
#pragma unroll
      for (int q = 0; q < 2; ++q) v[q] += a.part[((size_t)i * 4 + 2 * half + q) * a.C + c];
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) red[q][sl][l] = v[q];
  __syncthreads();
  if (threadIdx.x >= 32 || c >= a.C) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    v[q] = 0.f;
    for (int i = 0; i < 32; ++i) v[q] += red[q][i][l];
  }
  if (half == 1) {
    put<DT>(a.g_w_pre, c, v[0]);
    put<DT>(a.g_b_pre, c, v[1]);
    return;
  }
  const float w = param(a.w_post, DT, c, 1.f), bp = param(a.b_post, DT, c, 0.f), sc = param(a.scale, DT, c, 1.f);
  put<DT>(a.g_w_post, c, sc * v[0]);
  put<DT>(a.g_b_post, c, sc * v[1]);
  put<DT>(a.g_scale, c, fmaf(w, v[0], bp * v[1]));
}

// ------------------------------------------------------------------ launch

NormPick norm_kernel_f32(bool tok, int kind, bool fwd, int C, long tiles);
NormPick norm_kernel_f16(bool tok, int kind, bool fwd, int C, long tiles);
NormPick norm_kernel_bf16(bool tok, int kind, bool fwd, int C, long tiles);

namespace {

NormPick pick(const NormArgs &a, bool fwd, int dtype) {
  const bool tok = a.P == 1;
  const long px = dtype == DT_F32 ? 32 : 64, tiles = a.B * ((a.P + px - 1) / px);
  if (dtype == DT_F32) return norm_kernel_f32(tok, a.kind, fwd, a.C, tiles);
  if (dtype == DT_F16) return norm_kernel_f16(tok, a.kind, fwd, a.C, tiles);
  return norm_kernel_bf16(tok, a.kind, fwd, a.C, tiles);
}

// Runs per sample (fields) or in all (tokens): at most `most` of them. A
// field's run is a whole number of rounds of the workgroup's waves and short,
// so that the last workgroups to finish are not far behind the rest (the chip
// holds 512 of the backward's: 1040 long ones took three rounds, not two). Tokens:
// as many as the chip holds at two waves a SIMD; each leaves 4 C sums to be added.
constexpr long kFieldRuns = 4096, kTokenRuns = 512;
long norm_runs(const NormArgs &a, int dtype, const NormPick &k, long most, int *per = nullptr) {
  const int rpg = k.rpg;
  if (a.P == 1) return std::min((a.B + (long)rpg - 1) / rpg, most * 256 / k.threads);
  const long px = dtype == DT_F32 ? 32 : 64, nt = (a.P + px - 1) / px;
  const long s = std::max(1L, most / a.B), p = ((nt + s - 1) / s + rpg - 1) / rpg * rpg;
  if (per) *per = (int)p;
  return (nt + p - 1) / p;
}

}  // namespace

size_t norm_workspace_bytes(int B, int C, long P, int dtype) {
  NormArgs a{};
  a.B = B, a.C = C, a.P = P;
  const long S = norm_runs(a, dtype, pick(a, false, dtype), P == 1 ? kTokenRuns : kFieldRuns);
  return (size_t)4 * C * S * (P == 1 ? 1 : B) * 4;
}

hipError_t launch_norm_fwd(const NormArgs &a, int dtype, hipStream_t s) {
  const NormPick k = pick(a, true, dtype);
  NormArgs arg = a;
  const long S = norm_runs(a, dtype, k, kFieldRuns, &arg.per);
  FNO_BOUNDS(check_norm(arg, true, (int)S, dtype, k.threads, k.rpg, k.lds, k.wide, k.deep);)
  const dim3 grid((unsigned)S, a.P == 1 ? 1u : (unsigned)a.B);
  void *args[] = {(void *)&arg};
  return hipLaunchKernel(k.kernel, grid, dim3((unsigned)k.threads), args, k.lds, s);
}

hipError_t launch_norm_bwd(const NormArgs &a, int dtype, hipStream_t s) {
  const NormPick k = pick(a, false, dtype);
  NormArgs arg = a;
  int S = (int)norm_runs(a, dtype, k, a.P == 1 ? kTokenRuns : kFieldRuns, &arg.per);
  FNO_BOUNDS(check_norm(arg, false, S, dtype, k.threads, k.rpg, k.lds, k.wide, k.deep);)
  const bool tok = a.P == 1;
  const dim3 grid((unsigned)S, tok ? 1u : (unsigned)a.B);
  void *args[] = {(void *)&arg};
  if (hipError_t e = raise_lds_cap(k.kernel, k.lds); e != hipSuccess) return e;
  hipError_t e = hipLaunchKernel(k.kernel, grid, dim3((unsigned)k.threads), args, k.lds, s);
  if (e != hipSuccess || !a.part) return e;
  void *pargs[] = {(void *)&arg, (void *)&S};
#define FNO_PICK(DT) (tok ? (const void *)fno_norm_tok_params<DT> : (const void *)fno_norm_params<DT>)
  const void *pk = dtype == DT_F32 ? FNO_PICK(DT_F32) : dtype == DT_F16 ? FNO_PICK(DT_F16) : FNO_PICK(DT_BF16);
#undef FNO_PICK
  const dim3 pgrid(tok ? (a.C + 31) / 32 : a.C, tok ? 2 : 1);
  return hipLaunchKernel(pk, pgrid, dim3(1024), pargs, 0, s);
}

}  // namespace fno
