// fp32 and bf16 elements of an operand, one at a time and in pieces of up to 16 bytes at any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nq {

__device__ inline float load_element(const void* p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

// Round to nearest even; NaN stays NaN.
__device__ inline uint16_t bf16_round(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ inline void store_element(void* p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t*>(p)[i] = bf16_round(v);
  else
    static_cast<float*>(p)[i] = v;
}

// 8 and 16 bytes at the alignment of their elements.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ inline uint32_t bf16_pair(float a, float b) {  // one conversion for both
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// N elements of an operand from element i on, at any alignment of its elements.
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
      for (int j = 0; j < N / 2; ++j) w[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
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

}  // namespace nq
