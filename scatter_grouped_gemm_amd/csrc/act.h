// Activations of the products with an epilogue and their derivatives, in fp32.
//
// All but the exact GELU and the squared ReLU are x sigma(z) with z = alpha x
// (SiLU; the clamped gate with its own alpha) or z = 2 sqrt(2/pi) (x + 0.044715
// x^3) (GELU by tanh: (1 + tanh y) / 2 = sigma(2 y)), so one body with two
// factors serves them: p1 x + p3 x^3 is -z log2 e, and sigma = 1 / (1 + 2^that).
// Exponential and reciprocal are the hardware's (within about one fp32 place each); the
// exponential's argument is rounded, which costs up to about |z| 2^-22 of sigma.
//
// The exact GELU is x Phi(x).  Phi of a negative number is exp(-x^2/2) h(-x), with
// h(t) = exp(t^2/2) Phi(-t), which falls slowly like 1 / t: a polynomial of degree
// 8 in k = 1 / (1 + 0.305 t), without a constant term, fitted by weighted least
// squares to the smallest relative error (1.3e-7 for t up to 14; h in fp32 4e-7), so
// that the tail stays in proportion.  The exponential's argument is rounded here too:
// Phi is off by up to 4e-7 + 1.4 t^2 2^-24 of its value and a few places (5e-7 for t
// up to 2, 2e-6 up to 6, 8e-6 up to 13).  No branch, one reciprocal, one
// exponential: in a product's epilogue the library's erfc would take several times
// as long.
#pragma once

#include "common.h"

namespace moe {

constexpr int kActNone = 0, kActSigmoid = 1, kActErf = 2, kActRelu2 = 3;

// Activation of a call, worked out on the host from the public name.
struct ActArgs {
  int kind;
  int gated;      // gate and up halves: act(gate) * (up + offset)
  float p1, p3;   // kActSigmoid: see above
  float z1, z3;   // the same for z itself: its derivative is z1 + 3 z3 x^2
  float limit;    // gate cut at limit, up at -limit and limit; infinity: not cut
  float offset;
};

namespace act {

typedef __attribute__((ext_vector_type(4))) float f4;

// Far out sigma is 0 or 1 whatever x; cut there, x^3 stays finite and 0 times it 0.  By
// the minimum and maximum that keep a NaN (one instruction each, as fminf and fmaxf are,
// which drop it): the derivative is made of nothing but the value cut here.
__device__ __forceinline__ float bounded(float x) {
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(x, -1e12f), 1e12f);
}

__device__ __forceinline__ float sigmoid(const ActArgs& a, float x) {
  const float xb = bounded(x);
  const float e = __builtin_amdgcn_exp2f(xb * __builtin_fmaf(a.p3 * xb, xb, a.p1));
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// Phi(x); g receives exp(-x^2 / 2).
__device__ __forceinline__ float normal_cdf(float x, float& g) {
  const float t = fabsf(x);
  const float k = __builtin_amdgcn_rcpf(__builtin_fmaf(0.305f, t, 1.0f));
  float q = 0.0366993025f;
  q = __builtin_fmaf(q, k, -0.152988777f);
  q = __builtin_fmaf(q, k, 0.185717687f);
  q = __builtin_fmaf(q, k, -0.0379775651f);
  q = __builtin_fmaf(q, k, 0.121022068f);
  q = __builtin_fmaf(q, k, 0.103420749f);
  q = __builtin_fmaf(q, k, 0.12246684f);
  q = __builtin_fmaf(q, k, 0.121639736f);
  g = __builtin_amdgcn_exp2f(t * t * -0.7213475204f);  // log2(e) / 2
  q = q * k * g;
  return x < 0.0f ? q : 1.0f - q;
}

// act(x), without an up part.
__device__ __forceinline__ f4 value4(const ActArgs& a, f4 x) {
  f4 r = x;
  if (a.kind == kActSigmoid) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = x[e] * sigmoid(a, x[e]);
  } else if (a.kind == kActErf) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float g;
      r[e] = x[e] * normal_cdf(x[e], g);
    }
  } else if (a.kind == kActRelu2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = x[e] <= 0.0f ? 0.0f : x[e] * x[e];  // NaN stays NaN
  }
  return r;
}

// Comparisons, not fminf: a NaN has to stay one.
__device__ __forceinline__ float cut_gate(const ActArgs& a, float g) { return g > a.limit ? a.limit : g; }
__device__ __forceinline__ float cut_up(const ActArgs& a, float u) {
  return u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
}

__device__ __forceinline__ f4 gated4(const ActArgs& a, f4 g, f4 u) {
#pragma unroll
  for (int e = 0; e < 4; ++e) g[e] = cut_gate(a, g[e]);
  f4 r = value4(a, g);
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] *= cut_up(a, u[e]) + a.offset;
  return r;
}

// act(x) and its derivative.
__device__ __forceinline__ void slope(const ActArgs& a, float x, float& v, float& d) {
  if (a.kind == kActSigmoid) {
    const float s = sigmoid(a, x), xb = bounded(x);
    v = x * s;
    // where sigma is 0 or 1, s (1 - s) is 0 and has to make the product 0
    d = __builtin_fmaf(xb * __builtin_fmaf(3.0f * a.z3 * xb, xb, a.z1), s * (1.0f - s), s);
  } else if (a.kind == kActErf) {
    float g;
    const float c = normal_cdf(x, g);
    v = x * c;
    d = __builtin_fmaf(bounded(x) * 0.3989422804f, g, c);
  } else if (a.kind == kActRelu2) {
    v = x <= 0.0f ? 0.0f : x * x;
    d = x <= 0.0f ? 0.0f : 2.0f * x;
  } else {
    v = x;
    d = 1.0f;
  }
}

}  // namespace act

// The public name with its parameters -> the arguments of a launch.  False: no such
// activation, or parameters that it cannot take.
inline bool make_act(int32_t name, float alpha, float limit, ActArgs& a) {
  constexpr float kLog2e = 1.4426950408889634f, kInf = __builtin_inff();
  constexpr float kTanh1 = 1.5957691216057308f, kTanh3 = 0.07135481627159600f;  // 2 sqrt(2/pi), times 0.044715
  a = ActArgs{kActNone, 0, 0.0f, 0.0f, 0.0f, 0.0f, kInf, 0.0f};
  int base = name;
  if (name == MOE_ACT_SILU_MUL || name == MOE_ACT_GELU_MUL || name == MOE_ACT_GELU_TANH_MUL) {
    a.gated = 1;
    base = name == MOE_ACT_SILU_MUL ? MOE_ACT_SILU : name == MOE_ACT_GELU_MUL ? MOE_ACT_GELU : MOE_ACT_GELU_TANH;
  }
  switch (base) {
    case MOE_ACT_NONE: return true;
    case MOE_ACT_SILU: a.kind = kActSigmoid; a.z1 = 1.0f; break;
    case MOE_ACT_GELU: a.kind = kActErf; return true;
    case MOE_ACT_GELU_TANH: a.kind = kActSigmoid; a.z1 = kTanh1; a.z3 = kTanh3; break;
    case MOE_ACT_RELU2: a.kind = kActRelu2; return true;
    case MOE_ACT_SWIGLU_CLAMP:
      // a slope within what bounded() leaves saturated, a limit above 0
      if (!(alpha >= 1e-3f && alpha <= 1e3f) || !(limit > 0.0f)) return false;
      a.kind = kActSigmoid;
      a.gated = 1;
      a.z1 = alpha;
      a.limit = limit;
      a.offset = 1.0f;
      break;
    default: return false;
  }
  a.p1 = -a.z1 * kLog2e;
  a.p3 = -a.z3 * kLog2e;
  return true;
}

}  // namespace moe
