// Activations of a projection's epilogue and their slopes, in fp32.
//
// Five functions in three forms, chosen by uniform branches:
//   clamp  z < a ? 0 : z                  none (a = -inf), relu (a = 0)
//   gate   z / (1 + exp(-u)), u = z (a + b z^2)
//                                         silu (1, 0), gelu_tanh (2 sqrt(2/pi) (1, 0.044715),
//                                         since 1 + tanh v = 2 / (1 + exp(-2 v)))
//   erf    z Phi(z)                       gelu
// Phi(-|z|) = exp(-z^2/2) erfcx(x) / 2 with x = |z| / sqrt 2 and erfcx(x) = exp(x^2)
// erfc(x) as t P(t), t = 1 / (1 + 0.4 x): P of degree 8 fitted to erfcx over the
// half line by least squares of the relative error, reweighted towards the
// largest; off by 1.5e-7 at most, and by 5e-7 as fp32 evaluates it.  A NaN stays one.
#pragma once

#include <cuda_runtime.h>

namespace dmuon {

enum ActKind { kActClamp, kActGate, kActErf };
struct Act {
  int kind;
  float a, b;
};

// Act of a code of include/dmuon.h (checked by the caller).
inline Act act_of(int code) {
  const float lowest = -__builtin_huge_valf();
  switch (code) {
    case 1: return {kActClamp, 0.f, 0.f};
    case 2: return {kActGate, 1.f, 0.f};
    case 3: return {kActErf, 0.f, 0.f};
    case 4: return {kActGate, 1.5957691216057308f, 0.07135481282556f};
    default: return {kActClamp, lowest, 0.f};
  }
}

// Past +-1e4 every one of them is 0 or z to the last bit: what would overflow
// there is taken at the border.
__device__ __forceinline__ float act_inside(float z) { return z > 1e4f ? 1e4f : z < -1e4f ? -1e4f : z; }

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// exp(-z^2/2) and Phi(z).
__device__ __forceinline__ float normal_below(float z, float& bell) {
  const float t = rcp_fast(fmaf(fabsf(z), 0.28284271f, 1.f));
  float p = 0.05026565119624138f;
  p = fmaf(p, t, -0.182915598154068f);
  p = fmaf(p, t, 0.169108584523201f);
  p = fmaf(p, t, -0.0056274873204529285f);
  p = fmaf(p, t, 0.14144112169742584f);
  p = fmaf(p, t, 0.16853934526443481f);
  p = fmaf(p, t, 0.20784308016300201f);
  p = fmaf(p, t, 0.22566957771778107f);
  p = fmaf(p, t, 0.22567586600780487f);
  bell = exp2_fast(z * z * (-0.5f * kLog2e));
  const float below = 0.5f * (p * t) * bell;  // Phi(-|z|)
  return z > 0.f ? 1.f - below : below;
}

// f[i] = act(f[i])
template <int N>
__device__ __forceinline__ void act_values(float (&f)[N], const Act& act) {
  if (act.kind == kActClamp) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = f[i] < act.a ? 0.f : f[i];
  } else if (act.kind == kActGate) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = act_inside(f[i]);
      f[i] *= rcp_fast(1.f + exp2_fast(-kLog2e * (z * fmaf(act.b * z, z, act.a))));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float bell;
      f[i] *= normal_below(act_inside(f[i]), bell);
    }
  }
}

// g[i] *= act'(z[i]); relu has slope 0 at 0, and where z is below it the
// product is 0 whatever g is.
template <int N>
__device__ __forceinline__ void act_slopes(float (&g)[N], const float (&z)[N], const Act& act) {
  if (act.kind == kActClamp) {
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = z[i] <= act.a ? 0.f : g[i];
  } else if (act.kind == kActGate) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = act_inside(z[i]), bv2 = act.b * v * v;
      const float s = rcp_fast(1.f + exp2_fast(-kLog2e * (v * (act.a + bv2))));
      g[i] *= s * fmaf(v * (1.f - s), fmaf(3.f, bv2, act.a), 1.f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = act_inside(z[i]);
      float bell;
      const float below = normal_below(v, bell);
      g[i] *= fmaf(v * 0.3989422804014327f, bell, below);
    }
  }
}

}  // namespace dmuon
