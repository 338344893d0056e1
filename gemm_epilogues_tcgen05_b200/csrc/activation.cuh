// activation.cuh -- the activations that the epilogues evaluate without
// branches: GELU through the tail of the normal distribution, and those of a
// gated layer with their derivatives.
#pragma once

#include <stdint.h>

namespace ge {

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// h(a) = Phi(-a) = 2^q(a) of two values in [0, 13], the tail of the normal
// distribution: GELU(z) = z Phi(z) = max(z, 0) - |z| h(|z|), so that the negative
// tail keeps its relative accuracy (an approximation of h itself, off by 2e-7
// everywhere, was 0.2 % off at z = -4 and of the wrong sign at -5.2). q(a) = -1 + a (s(a) - a / (2 ln 2)): the Gaussian's exponent apart, s
// stays between -1.2 and -0.3, a polynomial of degree 14 in u = 2 a / 13 - 1
// (a weighted least-maximum fit on [0, 13], off by less than 2e-8 max(1, |q| / 2) /
// max(a, 0.3)), and the form is exact at a = 0. Measured over half a million
// points: |error| <= 9.3e-8 |z|, and relative to the result of a negative z at
// most 8e-7 down to -4, 2e-6 down to -6, 9e-6 down to -12.9, where h leaves the
// normal numbers and becomes 0 (ex2's flush); a is held at 13 beyond, so
// infinities give inf and 0, and max.NaN keeps NaN. Multiply-adds on two values an
// instruction and one ex2 each: with erff (an exponential and its branches) a 256
// x 256 tile's epilogue outlasted its products (microscaled T = 4096, N = 11008, K
// = 4096: 150 us, 96.5 with this, 74 without an activation; a polynomial for h
// took 92.3. E = 16, T = 1003, K = 2048, N = 5000: 23 us with either, 20.4 without).
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void phi_tail2(float a0, float a1, float& h0, float& h1) {
  constexpr float kS = 2.0f / 13.0f, kHalfLog2e = 0.72134752f;
  constexpr float kC[15] = {-0.47054109f, 0.258029431f, -0.160296753f, 0.102642007f, -0.0657589659f,
                            0.0410890728f, -0.0249870718f, 0.0165973958f, -0.00968039781f, -0.000120837707f,
                            0.00111253548f, 0.00610661181f, -0.00311078061f, -0.00396853918f, 0.00253350381f};
  const uint64_t a = pack_f32x2(a0, a1);
  const uint64_t u = fma_f32x2(a, pack_f32x2(kS, kS), pack_f32x2(-1.f, -1.f));
  uint64_t s = pack_f32x2(kC[14], kC[14]);
#pragma unroll
  for (int k = 13; k >= 0; --k) s = fma_f32x2(s, u, pack_f32x2(kC[k], kC[k]));
  s = fma_f32x2(a, pack_f32x2(-kHalfLog2e, -kHalfLog2e), s);
  const uint64_t q = fma_f32x2(a, s, pack_f32x2(-1.f, -1.f));
  float q0, q1;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(q0), "=f"(q1) : "l"(q));
  h0 = exp2_ftz(q0);
  h1 = exp2_ftz(q1);
}

constexpr float kPhiTailEnd = 13.0f;  // h is 0 in fp32 from here on

__device__ __forceinline__ float max0_nan(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
  return r;
}

__device__ __forceinline__ void gelu32(float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float a0 = fminf(fabsf(v[j]), kPhiTailEnd), a1 = fminf(fabsf(v[j + 1]), kPhiTailEnd);
    float h0, h1;
    phi_tail2(a0, a1, h0, h1);
    v[j] = fmaf(-a0, h0, max0_nan(v[j]));
    v[j + 1] = fmaf(-a1, h1, max0_nan(v[j + 1]));
  }
}

// The activations of a gated layer's gate (the values of gemm_epi_act).
enum ActKind : int { ACT_SILU = 0, ACT_GELU = 1, ACT_RELU = 2 };

// act(z) of an even number of values into a, and (DERIV) its derivative into d.
//   SILU  a = z p, p = 1 / (1 + e^-z);  d = p (1 + z (1 - p)) = p + a (1 - p)
//   GELU  a = max(z, 0) - |z| h(|z|);   d = Phi(z) + z phi(z), Phi(z) = h(-z) or 1 - h(z)
//   RELU  a = max(z, 0), of NaN 0;      d = 1 where z > 0
// With e = 2^-24: the exponential is off by 4 e (2 ulp) and its rounded argument's 1.22 |z| e, the
// sum by e, the reciprocal by 2 e, so p by (1 - p) (4 + 1.22 |z|) e + 3 e of itself: a keeps its relative
// accuracy in the negative tail (7e-6 at -88), and so does d beyond its zero at -1.28. p is 0
// below z = -88.72, where e^-z leaves fp32; -inf gives NaN, as -inf x 0 does, and so does d at an infinity.
__device__ __forceinline__ float reciprocal(float x) {  // (__fdividef gives 0 from 2^126 on)
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <int M, bool DERIV>
__device__ __forceinline__ void act_values(int act, const float (&z)[M], float (&a)[M], float (&d)[M]) {
  if (act == ACT_SILU) {
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const float p = reciprocal(1.f + exp2_ftz(-1.44269504f * z[j]));
      a[j] = z[j] * p;
      if constexpr (DERIV) d[j] = fmaf(a[j], 1.f - p, p);
    }
  } else if (act == ACT_GELU) {
#pragma unroll
    for (int j = 0; j < M; j += 2) {
      const float a0 = fminf(fabsf(z[j]), kPhiTailEnd), a1 = fminf(fabsf(z[j + 1]), kPhiTailEnd);
      float h0, h1;
      phi_tail2(a0, a1, h0, h1);
      a[j] = fmaf(-a0, h0, max0_nan(z[j]));
      a[j + 1] = fmaf(-a1, h1, max0_nan(z[j + 1]));
      if constexpr (DERIV) {
        const float p0 = 0.39894228f * exp2_ftz(-0.72134752f * z[j] * z[j]);
        const float p1 = 0.39894228f * exp2_ftz(-0.72134752f * z[j + 1] * z[j + 1]);
        d[j] = fmaf(z[j], p0, z[j] > 0.f ? 1.f - h0 : h0);
        d[j + 1] = fmaf(z[j + 1], p1, z[j + 1] > 0.f ? 1.f - h1 : h1);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < M; ++j) {
      a[j] = z[j] > 0.f ? z[j] : 0.f;
      if constexpr (DERIV) d[j] = z[j] > 0.f ? 1.f : 0.f;
    }
  }
}

}  // namespace ge
