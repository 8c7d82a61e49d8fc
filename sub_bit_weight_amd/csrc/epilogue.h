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

// exp(x) and 1 / (1 + exp(-x)) by the hardware's 2^x and reciprocal, one unit in the last place each and 0
// where the result is below 2^-126; the exponent's two roundings are felt |x| times.  At -inf: 0; NaN stays.
__device__ inline float exp_f(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ inline float sigmoid_f(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_f(-x)); }

// act(z).  The logistic of tanh's form: 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u)), which keeps
// its relative accuracy where tanh is near -1.
template <int ACT>
__device__ inline float act_value(float z) {
  if constexpr (ACT == NQ_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays
  if constexpr (ACT == NQ_ACT_GELU) return 0.5f * z * erfcf(-0.70710678f * z);
  if constexpr (ACT == NQ_ACT_GELU_TANH) return z * sigmoid_f(2.0f * kGeluA * (z + kGeluB * z * z * z));
  if constexpr (ACT == NQ_ACT_SILU) return z * sigmoid_f(z);
  return z;
}

// act(z) and its derivative (relu's is 0 at 0).
template <int ACT>
__device__ inline void act_value_grad(float z, float& a, float& da) {
  if constexpr (ACT == NQ_ACT_RELU) {
    a = z < 0.0f ? 0.0f : z;
    da = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  } else if constexpr (ACT == NQ_ACT_GELU) {
    const float cdf = 0.5f * erfcf(-0.70710678f * z);
    a = z * cdf;
    da = cdf + z * 0.3989422804f * exp_f(-0.5f * z * z);
  } else if constexpr (ACT == NQ_ACT_GELU_TANH) {
    const float q = sigmoid_f(2.0f * kGeluA * (z + kGeluB * z * z * z));
    a = z * q;
    da = q + a * (1.0f - q) * 2.0f * kGeluA * (1.0f + 3.0f * kGeluB * z * z);
  } else if constexpr (ACT == NQ_ACT_SILU) {
    const float q = sigmoid_f(z);
    a = z * q;
    da = q + a * (1.0f - q);
  } else {
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

// v: the layer's output W x before the bias.  One uniform branch for the activation.
__device__ inline float epilogue_act(int act, float v) {
  switch (act) {
    case NQ_ACT_RELU: return act_value<NQ_ACT_RELU>(v);
    case NQ_ACT_GELU: return act_value<NQ_ACT_GELU>(v);
    case NQ_ACT_GELU_TANH: return act_value<NQ_ACT_GELU_TANH>(v);
    case NQ_ACT_SILU: return act_value<NQ_ACT_SILU>(v);
    default: return v;
  }
}
__device__ inline void epilogue_store(const Epilogue& E, int64_t i, int64_t o, float v) {
  if (E.bias) v += E.bias[o];
  if (E.z) epi_store(E.z, E.z_bf16, i, v);
  float a = epilogue_act(E.act, v);
  if (E.mul) a *= epi_load(E.mul, E.mul_bf16, i);
  if (E.residual) a += epi_load(E.residual, E.residual_bf16, i);
  epi_store(E.y, E.y_bf16, i, a);
}

}  // namespace nq
