// gelu.hpp - GELU (the erf form v Phi(v), Phi the normal distribution function)
// and its derivative Phi(v) + v phi(v).
#pragma once

#include <hip/hip_runtime.h>

namespace fno {

__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)); }

// GELU for the half-precision kernels, whose outputs are rounded to 11 (fp16)
// or 8 (bf16) significant bits: erf from Abramowitz & Stegun, Handbook of
// Mathematical Functions, formula 7.1.28, erf(x) = 1 - (1 + a1 x + ... +
// a6 x^6)^-16 for x >= 0 (absolute error below 3e-7; evaluated in fp32 it
// stays below 2e-6), odd symmetry for x < 0. With r = 1 - erf(|v| / sqrt 2),
// GELU(v) = max(v, 0) - |v| r / 2. One reciprocal on the transcendental
// unit; formula 7.1.26 needs an exponential as well, which made the
// projection (128 hidden GELUs per pixel) 21 us slower at B = 20, 256^2.
__device__ __forceinline__ float gelu_half(float v) {
  const float x = fabsf(v) * 0.70710678118654752f;
  float p = fmaf(0.0000430638f, x, 0.0002765672f);
  p = fmaf(p, x, 0.0001520143f);
  p = fmaf(p, x, 0.0092705272f);
  p = fmaf(p, x, 0.0422820123f);
  p = fmaf(p, x, 0.0705230784f);
  p = fmaf(p, x, 1.0f);
  p = p * p;  // ^16 by four squarings; overflows to inf for large x, so r = 0
  p = p * p;
  p = p * p;
  p = p * p;
  const float r = __builtin_amdgcn_rcpf(p);
  return fmaf(-0.5f * fabsf(v), r, fmaxf(v, 0.0f));
}

// GELU and its derivative for the training kernels of all types, both from the normal
// distribution's upper tail q = 1 - Phi(|v|) = exp(-v^2 / 2) t P(t), t = 1 / (1 + 0.39 |v|),
// P of degree 5 fitted here by weighted least squares. Absolute errors of q: the fit below 1e-8,
// with everything in fp32 1.4e-7 (erff and expf: 6e-8, in five times the operations: a step
// on 16 x 32 x 32 channels, 128^2, fp32 took 82 us with them and 76 without). Relative to q the
// fit is off by 6e-8 up to |v| = 1, 3e-6 up to 3, 2e-4 up to 5 and 4e-4 up to 6, which no
// fp16 result shows; gelu_half() above (1e-6 of absolute error) is off by several fp16 steps from
// -3 on and no faster in a training step (32 x 64 x 64 channels, 256^2: within 1 us of 535).
// |v| is cut off at 100 where it multiplies a vanished tail: infinities stay what they are.
__device__ __forceinline__ float normal_tail(float a, float e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.39f, a, 1.0f));
  float p = fmaf(0.053847310403341085f, t, -0.2582449235385277f);
  p = fmaf(p, t, 0.3751703021987614f);
  p = fmaf(p, t, -0.016637008264066055f);
  p = fmaf(p, t, 0.19443737777823863f);
  p = fmaf(p, t, 0.1514269511269713f);
  return p * t * e;
}
__device__ __forceinline__ float normal_bell(float v) {  // exp(-v^2 / 2)
  return __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);
}
__device__ __forceinline__ float gelu_train(float v) {
  const float a = fabsf(v), q = normal_tail(a, normal_bell(v));
  return fmaf(-fminf(a, 100.0f), q, fmaxf(v, 0.0f));
}
__device__ __forceinline__ float gelu_slope(float v) {
  const float e = normal_bell(v), q = normal_tail(fabsf(v), e);
  return fmaf(__builtin_amdgcn_fmed3f(v, -100.0f, 100.0f) * 0.39894228040143268f, e, v >= 0.0f ? 1.0f - q : q);
}

}  // namespace fno
