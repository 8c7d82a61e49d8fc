// Epilogue of a packed linear on one output element, shared by the kernels that
// apply it, and the gradients of it.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

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

// N elements of an operand from element i on, at any alignment of its elements.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <int N>
struct Elements {
  float v[N];
  __device__ void load(const void* p, bool bf16, int64_t i) {
    if (bf16) {
      const uint16_t* q = static_cast<const uint16_t*>(p) + i;
      uint32_t w[N / 2];
      if constexpr (N == 8) {
        const u32x4 d = *reinterpret_cast<const u32x4_a2*>(q);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = d[j];
      } else {
        const u32x2 d = *reinterpret_cast<const u32x2_a2*>(q);
        w[0] = d[0], w[1] = d[1];
      }
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
      const float* q = static_cast<const float*>(p) + i;
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const u32x4 d = *reinterpret_cast<const u32x4_a4*>(q + j);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j + k] = __uint_as_float(d[k]);
      }
    }
  }
  __device__ void store(void* p, bool bf16, int64_t i) const {
    if (bf16) {
      uint16_t* q = static_cast<uint16_t*>(p) + i;
      uint32_t w[N / 2];
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * j], v[2 * j + 1]}, bf16x2));
      if constexpr (N == 8)
        *reinterpret_cast<u32x4_a2*>(q) = u32x4{w[0], w[1], w[2], w[3]};
      else
        *reinterpret_cast<u32x2_a2*>(q) = u32x2{w[0], w[1]};
    } else {
      float* q = static_cast<float*>(p) + i;
#pragma unroll
      for (int j = 0; j < N; j += 4)
        *reinterpret_cast<u32x4_a4*>(q + j) = u32x4{__float_as_uint(v[j]), __float_as_uint(v[j + 1]),
                                                   __float_as_uint(v[j + 2]), __float_as_uint(v[j + 3])};
    }
  }
};

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// exp(x), x <= 0, as m 2^n: the hardware's 2^x (one unit in the last place) of what x log2(e) is from the
// nearest whole number, which two constants give with one rounding.  So m is within two units at any x, and
// ldexp keeps results below the hardware's smallest, 2^-126 (silu of -88 to -104).  One 2^x of the rounded
// product is off by up to |x| roundings more and 0 there; the linear of 2048 x 28672 x 8192, rank 6336, with
// silu, gate and z takes 737 us with it, 749 so.
__device__ inline float exp_parts(float x, int& n) {
  x = fmaxf(x, -256.0f);  // 0 all the same (NaN too: the callers' products keep it)
  const float w = rintf(x * 1.44269502f);
  n = (int)w;
  return __builtin_amdgcn_exp2f(fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -w)));
}
__device__ inline float exp_f(float x) {
  int n;
  const float m = exp_parts(x, n);
  return ldexpf(m, n);
}
// q = 1 / (1 + exp(-u)) and p = 1 - q = 1 / (1 + exp(u)), each to its own last places.
struct Logistic {
  float q, p;
};
__device__ inline Logistic logistic(float u) {
  int n;
  const float m = exp_parts(-fabsf(u), n), r = __builtin_amdgcn_rcpf(1.0f + ldexpf(m, n)), s = ldexpf(m * r, n);
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
    for (int j = 0; j < N; ++j) mul[j] = epi_load(E.mul, E.mul_bf16, at(j));
  if (E.residual)
#pragma unroll
    for (int j = 0; j < N; ++j) res[j] = epi_load(E.residual, E.residual_bf16, at(j));
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
      if (E.z) epi_store(E.z, E.z_bf16, at(j), z);
      epi_store(E.y, E.y_bf16, at(j), a);
    }
  });
}

// n (at most 8) outputs v of one row from column o on, at elements i ...: whole rows of 8 as 16-byte pieces.
__device__ __forceinline__ void epilogue_store8(const Epilogue& E, int64_t i, int64_t o, int n, Elements<8>& v) {
#pragma clang fp contract(off)
  if (n == 8) {
    Elements<8> mul, res, bias;
    if (E.mul) mul.load(E.mul, E.mul_bf16, i);
    if (E.residual) res.load(E.residual, E.residual_bf16, i);
    if (E.bias) {
      bias.load(E.bias, false, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) v.v[j] += bias.v[j];
    }
    if (E.z) v.store(E.z, E.z_bf16, i);
    with_act(E.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j % kAtOnce == 0) __builtin_amdgcn_sched_barrier(0);
        v.v[j] = act(v.v[j]);
      }
    });
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (E.mul) v.v[j] *= mul.v[j];
      if (E.residual) v.v[j] += res.v[j];
    }
    v.store(E.y, E.y_bf16, i);
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) {
      const float one[1] = {v.v[j]};
      epilogue_store<1>(E, E.bias ? E.bias[o + j] : 0.0f, one, [&](int) { return i + j; });
    }
}

}  // namespace nq
