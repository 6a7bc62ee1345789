// Activations of a projection's epilogue and their slopes, in fp32.
//
// Five functions in three forms, chosen by uniform branches, two values at a time:
//   clamp  z < a ? 0 : z                  none (a = -inf), relu (a = 0)
//   gate   z / (1 + exp(-u)), u = z (a + b z^2), kept as -log2(e) a and b
//                                         silu (1, 0), gelu_tanh (2 sqrt(2/pi) (1, 0.044715),
//                                         since 1 + tanh v = 2 / (1 + exp(-2 v)))
//   erf    z Phi(z)                       gelu
// Phi(-|z|) = exp(-z^2/2) erfcx(x) / 2 with x = |z| / sqrt 2 and erfcx(x) = exp(x^2)
// erfc(x) as t P(t), t = 1 / (1 + 0.4 x): P of degree 8 fitted to erfcx over the
// half line by least squares of the relative error, reweighted towards the
// largest; off by 1.5e-7 at most, and by 5e-7 as fp32 evaluates it.  exp2's argument is
// rounded besides, so a value has 2^-21 (2 + |u|) of itself (u the exponent: z^2/2 for
// gelu), and what exp2 or the reciprocal would make subnormal is 0: silu and gelu_tanh
// below 2^-119, gelu below 2^-127, slopes below 2^-118.  A NaN stays one.
#pragma once

#include <cuda_runtime.h>

#include "f32x2.cuh"

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
    case 2: return {kActGate, -1.4426950408889634f, 0.f};
    case 3: return {kActErf, 0.f, 0.f};
    case 4: return {kActGate, -2.302208198144325f, -0.1029432395800235f};
    default: return {kActClamp, lowest, 0.f};
  }
}

// Past +-1e4 every one of them is 0 or z to the last bit: what would overflow
// there is taken at the border.
__device__ __forceinline__ float act_inside(float z) {  // the smaller magnitude, with z's sign; NaN stays
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(1e4f));
  return r;
}
__device__ __forceinline__ f2 act_inside2(f2 z) {
  const float2 p = unpack2(z);
  return pack2(act_inside(p.x), act_inside(p.y));
}

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
__device__ __forceinline__ f2 exp2_fast2(f2 x) {
  const float2 p = unpack2(x);
  return pack2(exp2_fast(p.x), exp2_fast(p.y));
}
__device__ __forceinline__ f2 rcp_fast2(f2 x) {
  const float2 p = unpack2(x);
  return pack2(rcp_fast(p.x), rcp_fast(p.y));
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// exp(-z^2/2) and Phi(z) of two values.
__device__ __forceinline__ f2 normal_below2(f2 z, f2& bell) {
  const float2 p = unpack2(z);
  const f2 t = rcp_fast2(fma2(pack2(fabsf(p.x), fabsf(p.y)), both(0.28284271f), both(1.f)));
  f2 q = both(0.05026565119624138f);
  q = fma2(q, t, both(-0.182915598154068f));
  q = fma2(q, t, both(0.169108584523201f));
  q = fma2(q, t, both(-0.0056274873204529285f));
  q = fma2(q, t, both(0.14144112169742584f));
  q = fma2(q, t, both(0.16853934526443481f));
  q = fma2(q, t, both(0.20784308016300201f));
  q = fma2(q, t, both(0.22566957771778107f));
  q = fma2(q, t, both(0.22567586600780487f));
  bell = exp2_fast2(mul2(mul2(z, z), both(-0.5f * kLog2e)));
  const float2 below = unpack2(mul2(mul2(mul2(q, t), both(0.5f)), bell));  // Phi(-|z|)
  return pack2(p.x > 0.f ? 1.f - below.x : below.x, p.y > 0.f ? 1.f - below.y : below.y);
}

// f[i] = act(f[i])
template <int KIND, int N>
__device__ __forceinline__ void act_values_of(f2 (&f)[N], const Act& act) {
  const f2 a = both(act.a), b = both(act.b);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (KIND == kActClamp) {
      const float2 p = unpack2(f[i]);
      f[i] = pack2(p.x < act.a ? 0.f : p.x, p.y < act.a ? 0.f : p.y);
    } else if constexpr (KIND == kActGate) {
      const f2 z = act_inside2(f[i]);
      f[i] = mul2(f[i], rcp_fast2(add2(exp2_fast2(mul2(z, fma2(b, mul2(z, z), a))), both(1.f))));
    } else {
      f2 bell;
      f[i] = mul2(f[i], normal_below2(act_inside2(f[i]), bell));
    }
  }
}
template <int N>
__device__ __forceinline__ void act_values(f2 (&f)[N], const Act& act) {
  if (act.kind == kActClamp) act_values_of<kActClamp>(f, act);
  else if (act.kind == kActGate) act_values_of<kActGate>(f, act);
  else act_values_of<kActErf>(f, act);
}

// g[i] *= act'(z[i]); relu has slope 0 at 0, and where z is below it the
// product is 0 whatever g is.  With s = 1 / (1 + exp(-u)) a gate's slope is
// s + s (1 - s) z u'; u, u' come scaled by -log2 e, undone by -ln 2.
template <int KIND, int N>
__device__ __forceinline__ void act_slopes(f2 (&g)[N], const f2 (&z)[N], const Act& act) {
  const f2 a = both(act.a), b = both(act.b), b3 = both(3.f * act.b);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (KIND == kActClamp) {
      const float2 p = unpack2(z[i]), q = unpack2(g[i]);
      g[i] = pack2(p.x <= act.a ? 0.f : q.x, p.y <= act.a ? 0.f : q.y);
    } else if constexpr (KIND == kActGate) {
      const f2 v = act_inside2(z[i]), vv = mul2(v, v);
      const f2 s = rcp_fast2(add2(exp2_fast2(mul2(v, fma2(b, vv, a))), both(1.f)));
      const f2 m = mul2(mul2(v, fma2(b3, vv, a)), fma2(s, both(kLn2), both(-kLn2)));
      g[i] = mul2(g[i], fma2(s, m, s));
    } else {
      const f2 v = act_inside2(z[i]);
      f2 bell;
      const f2 below = normal_below2(v, bell);
      g[i] = mul2(g[i], fma2(mul2(v, both(0.3989422804014327f)), bell, below));
    }
  }
}

}  // namespace dmuon
