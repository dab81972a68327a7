// gl_act.cuh -- the activations that products apply in their epilogues, and
// their slopes, on fp32 values.
//
//   relu2  max(u, 0)^2
//   silu   u q(u),                q(v) = 1 / (1 + e^-v)
//   gelu   u q(2c (u + a u^3)),   c = sqrt(2 / pi), a = 0.044715 (the tanh form:
//          0.5 (1 + tanh v) = q(2v))
// The gated forms act on pairs: swiglu silu(u0) * u1, geglu gelu(u0) * u1.
//
// e^x and the division are CUDA's fast forms (a few units in the last place
// of fp32, and results go to bf16).  A NaN stays a NaN in every value.
#pragma once

#include <cuda_runtime.h>

#include "gl.h"

namespace gl {

__host__ __device__ constexpr bool act_gated(int act) { return act == GL_ACT_SWIGLU || act == GL_ACT_GEGLU; }

// The activation of one argument inside a (possibly gated) activation.
__host__ __device__ constexpr int act_inner(int act) {
  return act == GL_ACT_SWIGLU ? GL_ACT_SILU : act == GL_ACT_GEGLU ? GL_ACT_GELU : act;
}

__device__ __forceinline__ float act_sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// Value of an inner activation.  `act` is the same for the whole launch.
__device__ __forceinline__ float act_value(int act, float u) {
  switch (act) {
    case GL_ACT_RELU: return u < 0.0f ? 0.0f : u;
    case GL_ACT_RELU2: return u < 0.0f ? 0.0f : u * u;
    case GL_ACT_GELU: return u * act_sigmoid(kGelu2C * (u + kGeluA * u * u * u));
    case GL_ACT_SILU: return u * act_sigmoid(u);
  }
  return u;
}

// Value and slope of an inner activation.
__device__ __forceinline__ float act_slope(int act, float u, float& value) {
  switch (act) {
    case GL_ACT_RELU:
      value = u < 0.0f ? 0.0f : u;
      return u > 0.0f ? 1.0f : 0.0f;
    case GL_ACT_RELU2:
      value = u < 0.0f ? 0.0f : u * u;
      return u < 0.0f ? 0.0f : 2.0f * u;
    case GL_ACT_GELU: {
      const float u2 = u * u;
      const float q = act_sigmoid(kGelu2C * (u + kGeluA * u2 * u));
      value = u * q;
      const float w = q * (1.0f - q);
      // far out w is 0 and u2 may be infinite: the product's limit is 0
      return w == 0.0f ? q : fmaf(u * w, kGelu2C * fmaf(3.0f * kGeluA, u2, 1.0f), q);
    }
    case GL_ACT_SILU: {
      const float q = act_sigmoid(u);
      value = u * q;
      return q * fmaf(u, 1.0f - q, 1.0f);
    }
  }
  value = u;
  return 1.0f;
}

}  // namespace gl
