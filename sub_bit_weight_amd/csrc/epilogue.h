// Epilogue of a packed linear on one output element, shared by the kernels that
// apply it, and the gradients of it.
#pragma once

#include <hip/hip_runtime.h>

#include "nq_internal.h"

namespace nq {

__device__ inline float epi_load(const void* p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

// Round to nearest even; NaN stays NaN.
__device__ inline uint16_t bf16_round(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ inline void epi_store(void* p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t*>(p)[i] = bf16_round(v);
  else
    static_cast<float*>(p)[i] = v;
}

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

__device__ inline float sigmoid_f(float z) { return 1.0f / (1.0f + expf(-z)); }

// act(z).  The logistic of tanh's form: 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u)), which keeps
// its relative accuracy where tanh is near -1.
__device__ inline float act_value(int act, float z) {
  switch (act) {
    case NQ_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays
    case NQ_ACT_GELU: return 0.5f * z * erfcf(-0.70710678f * z);
    case NQ_ACT_GELU_TANH: return z * sigmoid_f(2.0f * kGeluA * (z + kGeluB * z * z * z));
    case NQ_ACT_SILU: return z * sigmoid_f(z);
    default: return z;
  }
}

// act(z) and its derivative (relu's is 0 at 0).
__device__ inline void act_value_grad(int act, float z, float& a, float& da) {
  switch (act) {
    case NQ_ACT_RELU:
      a = z < 0.0f ? 0.0f : z;
      da = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
      return;
    case NQ_ACT_GELU: {
      const float cdf = 0.5f * erfcf(-0.70710678f * z);
      a = z * cdf;
      da = cdf + z * 0.3989422804f * expf(-0.5f * z * z);
      return;
    }
    case NQ_ACT_GELU_TANH: {
      const float q = sigmoid_f(2.0f * kGeluA * (z + kGeluB * z * z * z));
      a = z * q;
      da = q + a * (1.0f - q) * 2.0f * kGeluA * (1.0f + 3.0f * kGeluB * z * z);
      return;
    }
    case NQ_ACT_SILU: {
      const float q = sigmoid_f(z);
      a = z * q;
      da = q + a * (1.0f - q);
      return;
    }
    default:
      a = z;
      da = 1.0f;
  }
}

// What a kernel needs of an nq_epilogue and its output, for element i = t * d_out + o.
struct Epilogue {
  const float* bias;
  const void* mul;
  const void* residual;
  void* z;
  void* y;
  int act;
  int mul_bf16, residual_bf16, z_bf16, y_bf16;
};

// v: the layer's output W x before the bias.
__device__ inline void epilogue_store(const Epilogue& E, int64_t i, int64_t o, float v) {
  if (E.bias) v += E.bias[o];
  if (E.z) epi_store(E.z, E.z_bf16, i, v);
  float a = act_value(E.act, v);
  if (E.mul) a *= epi_load(E.mul, E.mul_bf16, i);
  if (E.residual) a += epi_load(E.residual, E.residual_bf16, i);
  epi_store(E.y, E.y_bf16, i, a);
}

}  // namespace nq
