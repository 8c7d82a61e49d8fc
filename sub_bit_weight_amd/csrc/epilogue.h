// Epilogue of a packed linear on one output element, shared by the kernels that
// apply it, and the gradients of it.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "elements.h"
#include "nq_internal.h"

namespace nq {

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// exp(x), x <= 0: the hardware's 2^x (one unit in the last place) of what x log2(e) is from the nearest
// whole number, which two constants give with one rounding, so that the result is within two units at any x;
// ldexp keeps what is below the hardware's smallest, 2^-126 (silu of -88 to -104).  One 2^x of the rounded
// product is off by up to |x| roundings more and 0 there; the linear of 2048 x 28672 x 8192, rank 6336, with
// silu, gate and z takes 737 us with it, 749 so.
__device__ inline float exp_f(float x) {
  x = fmaxf(x, -256.0f);  // 0 all the same (NaN too: the callers' products keep it)
  const float w = rintf(x * 1.44269502f);
  return ldexpf(__builtin_amdgcn_exp2f(fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -w))), (int)w);
}
// q = 1 / (1 + exp(-u)) and p = 1 - q = 1 / (1 + exp(u)), each to its own last places.
struct Logistic {
  float q, p;
};
__device__ inline Logistic logistic(float u) {
  const float e = exp_f(-fabsf(u)), r = __builtin_amdgcn_rcpf(1.0f + e), s = e * r;
  return u < 0.0f ? Logistic{s, r} : Logistic{r, s};
}

// act(z).  The logistic of tanh's form: 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u)), which keeps
// its relative accuracy where tanh is near -1.
template <int ACT>
__device__ inline float act_value(float z) {
  if constexpr (ACT == NQ_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays
  if constexpr (ACT == NQ_ACT_GELU) return 0.5f * z * erfcf(-0.70710678f * z);
  if constexpr (ACT == NQ_ACT_GELU_TANH) return z * logistic(2.0f * kGeluA * (z + kGeluB * z * z * z)).q;
  if constexpr (ACT == NQ_ACT_SILU) return z * logistic(z).q;
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
    const Logistic l = logistic(2.0f * kGeluA * (z + kGeluB * z * z * z));
    a = z * l.q;
    // a p is 0 where z^2 overflows, and its product with an infinity would be NaN
    da = l.q + a * l.p * 2.0f * kGeluA * (1.0f + fminf(3.0f * kGeluB * z * z, __FLT_MAX__));
  } else if constexpr (ACT == NQ_ACT_SILU) {
    const Logistic l = logistic(z);
    a = z * l.q;
    da = l.q + a * l.p;
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

// What a kernel without an epilogue takes in its place, so that a plain linear carries nothing of it.
struct NoEpilogue {};
template <typename E>
constexpr bool is_epilogue = std::is_same<E, Epilogue>::value;

// f(the activation), by one uniform branch.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case NQ_ACT_RELU: return f([](float z) { return act_value<NQ_ACT_RELU>(z); });
    case NQ_ACT_GELU: return f([](float z) { return act_value<NQ_ACT_GELU>(z); });
    case NQ_ACT_GELU_TANH: return f([](float z) { return act_value<NQ_ACT_GELU_TANH>(z); });
    case NQ_ACT_SILU: return f([](float z) { return act_value<NQ_ACT_SILU>(z); });
    default: return f([](float z) { return z; });
  }
}

// N outputs of one column (bias: the column's, or 0): v, W x before the bias, at elements at(j).  The
// operands of all are loaded ahead of the first store, which no load can be moved across (y may be one of
// them): an element at a time pays a memory latency each (8 tokens of an 11008 x 4096 layer of rank 2368:
// 45.7 us instead of 33.3).
// kAtOnce activations are computed side by side (all of them at once spilled registers).
constexpr int kAtOnce = 2;
template <int N, typename At>
__device__ __forceinline__ void epilogue_store(const Epilogue& E, float bias, const float (&v)[N], At at) {
  float mul[N], res[N];
  if (E.mul)
#pragma unroll
    for (int j = 0; j < N; ++j) mul[j] = load_element(E.mul, E.mul_bf16, at(j));
  if (E.residual)
#pragma unroll
    for (int j = 0; j < N; ++j) res[j] = load_element(E.residual, E.residual_bf16, at(j));
  with_act(E.act, [&](auto act) __attribute__((always_inline)) {
    // v is rounded before the bias is added: the layer's output, as without an epilogue
#pragma clang fp contract(off)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j % kAtOnce == 0) __builtin_amdgcn_sched_barrier(0);
      const float z = v[j] + bias;
      float a = act(z);
      if (E.mul) a *= mul[j];
      if (E.residual) a += res[j];
      if (E.z) store_element(E.z, E.z_bf16, at(j), z);
      store_element(E.y, E.y_bf16, at(j), a);
    }
  });
}

// n (at most 8) outputs v of one row from column o on, at elements i ...: whole rows of 8 as 16-byte pieces,
// the operands and results of fewer one by one.  The activations of both are the same code: each behind the
// store before it, as its operands are, a ragged end's took longer (92 tokens of 1813 x 1716, rank 259, bf16:
// silu and gate 54.2 us, 49.3 so, gelu 58.7 and 48.9).
__device__ __forceinline__ void epilogue_store8(const Epilogue& E, int64_t i, int64_t o, int n, Elements<8>& v) {
#pragma clang fp contract(off)
  Elements<8> mul, res;
  if (n == 8) {
    if (E.mul) mul.load(E.mul, E.mul_bf16, i);
    if (E.residual) res.load(E.residual, E.residual_bf16, i);
    if (E.bias) {
      Elements<8> bias;
      bias.load(E.bias, false, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) v.v[j] += bias.v[j];
    }
    if (E.z) v.store(E.z, E.z_bf16, i);
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < n) {
        if (E.bias) v.v[j] += E.bias[o + j];
        if (E.z) store_element(E.z, E.z_bf16, i + j, v.v[j]);
      }
  }
  with_act(E.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j % kAtOnce == 0) __builtin_amdgcn_sched_barrier(0);
      v.v[j] = act(v.v[j]);
    }
  });
  if (n == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (E.mul) v.v[j] *= mul.v[j];
      if (E.residual) v.v[j] += res.v[j];
    }
    v.store(E.y, E.y_bf16, i);
  } else {
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < n) {
        float a = v.v[j];
        if (E.mul) a *= load_element(E.mul, E.mul_bf16, i + j);
        if (E.residual) a += load_element(E.residual, E.residual_bf16, i + j);
        store_element(E.y, E.y_bf16, i + j, a);
      }
  }
}

}  // namespace nq
