// gl_act.cuh -- the activations that products apply in their epilogues, and
// their slopes, on fp32 values.
//
//   relu2  max(u, 0)^2
//   silu   u q(u),                q(v) = 1 / (1 + e^-v)
//   gelu   u q(2c (u + a u^3)),   c = sqrt(2 / pi), a = 0.044715 (the tanh form:
//          0.5 (1 + tanh v) = q(2v))
// The gated forms act on pairs: swiglu silu(u0) * u1, geglu gelu(u0) * u1.
//
// e^x and the reciprocal are the fast forms (a few units in the last place
// of fp32, and results go to bf16).  A NaN stays a NaN in every value
// and slope.
#pragma once

#include <cuda_runtime.h>

#include "gl.h"

namespace gl {

__host__ __device__ constexpr bool act_gated(int act) { return act == GL_ACT_SWIGLU || act == GL_ACT_GEGLU; }

// The activation of one argument inside a (possibly gated) activation.
__host__ __device__ constexpr int act_inner(int act) {
  return act == GL_ACT_SWIGLU ? GL_ACT_SILU : act == GL_ACT_GEGLU ? GL_ACT_GELU : act;
}

// 1 / (1 + e^-v) from t = e^-|v| <= 1, which keeps the denominator in [1, 2]:
// 1 / (1 + t), or t / (1 + t) below 0.  From 1 / (1 + e^-v) the fast division
// gives 0 where its denominator is past 2^126, and e^-v overflows behind
// -88.7, while silu stays in bf16's normal range down to -91.8.
__device__ __forceinline__ float act_sigmoid(float v) {
  const float t = __expf(-fabsf(v));
  float r;  // of 1 .. 2: no subnormal on either side
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return v < 0.0f ? t * r : r;
}

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// One inner activation, known at compile time.
template <int ACT>
__device__ __forceinline__ float act_of(float u) {
  if (ACT == GL_ACT_RELU) return u < 0.0f ? 0.0f : u;
  if (ACT == GL_ACT_RELU2) return u < 0.0f ? 0.0f : u * u;
  if (ACT == GL_ACT_GELU) return u * act_sigmoid(u * fmaf(kGelu2C * kGeluA, u * u, kGelu2C));
  if (ACT == GL_ACT_SILU) return u * act_sigmoid(u);
  return u;
}

// Its value and slope.
template <int ACT>
__device__ __forceinline__ float slope_of(float u, float& value) {
  if (ACT == GL_ACT_RELU) {
    value = u < 0.0f ? 0.0f : u;
    return u > 0.0f ? 1.0f : u <= 0.0f ? 0.0f : u;
  }
  if (ACT == GL_ACT_RELU2) {
    value = u < 0.0f ? 0.0f : u * u;
    return u < 0.0f ? 0.0f : 2.0f * u;
  }
  if (ACT == GL_ACT_GELU) {
    const float u2 = u * u;
    const float q = act_sigmoid(u * fmaf(kGelu2C * kGeluA, u2, kGelu2C));
    value = u * q;
    const float w = q * (1.0f - q);
    // far out w is 0 and u2 may be infinite: the product's limit is 0
    return w == 0.0f ? q : fmaf(u * w, fmaf(3.0f * kGelu2C * kGeluA, u2, kGelu2C), q);
  }
  if (ACT == GL_ACT_SILU) {
    const float q = act_sigmoid(u);
    value = u * q;
    float slope;  // 0 where q is below the normal range (it is under 2^-119 there)
    asm("mul.ftz.f32 %0, %1, %2;" : "=f"(slope) : "f"(q), "f"(fmaf(u, 1.0f - q, 1.0f)));
    return slope;
  }
  value = u;
  return 1.0f;
}

// f.template operator()<ACT>() for the launch's inner activation: one branch
// around a loop instead of a chain of them per element.
template <typename Fn>
__device__ __forceinline__ void act_dispatch(int act, Fn f) {
  switch (act) {
    case GL_ACT_RELU: f.template operator()<GL_ACT_RELU>(); break;
    case GL_ACT_RELU2: f.template operator()<GL_ACT_RELU2>(); break;
    case GL_ACT_GELU: f.template operator()<GL_ACT_GELU>(); break;
    case GL_ACT_SILU: f.template operator()<GL_ACT_SILU>(); break;
    default: f.template operator()<GL_ACT_NONE>(); break;
  }
}

template <int N>
struct ActValues {
  float (&u)[N];
  template <int ACT>
  __device__ __forceinline__ void operator()() {
#pragma unroll
    for (int j = 0; j < N; ++j) u[j] = act_of<ACT>(u[j]);
  }
};
// u[] <- act(u[])
template <int N>
__device__ __forceinline__ void act_values(int act, float (&u)[N]) {
  act_dispatch(act, ActValues<N>{u});
}

template <int N>
struct ActSlopes {
  float (&u)[N];
  float (&value)[N];
  template <int ACT>
  __device__ __forceinline__ void operator()() {
#pragma unroll
    for (int j = 0; j < N; ++j) u[j] = slope_of<ACT>(u[j], value[j]);
  }
};
// u[] <- act'(u[]), value[] <- act(u[])
template <int N>
__device__ __forceinline__ void act_slopes(int act, float (&u)[N], float (&value)[N]) {
  act_dispatch(act, ActSlopes<N>{u, value});
}

}  // namespace gl
