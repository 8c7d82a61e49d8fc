// Orthogonalised updates by Newton-Schulz: from X0 = X / ||X||_F the iteration
//
//     X <- a X + (b G + c G^2) X,   G = X X^T  (the shorter side first)
//
// maps every singular value s of X to a s + b s^3 + c s^5 and leaves the
// singular vectors alone.  With p the shorter and q the longer side:
//
//  * p <= 64 (ortho_gram / solve / apply): all iterates are polynomials of the
//    first Gram matrix, X_n = Q X0 with Q a p x p matrix, so the iteration runs
//    on p x p matrices and X is read twice and written once, instead of 3 passes
//    a step.  G squares the singular values and Q multiplies the small ones by
//    up to a^steps, so this form needs twice the digits: everything is fp64
//    (X0 enters exactly, one rounding at the end).  Rounding errors of the Gram
//    matrix, negative eigenvalues among them, grow by a^2 a step, since nothing
//    ties it to X again: after as many steps as that growth allows (five of the
//    default quintic) Q is applied, the iterate kept in fp64, and its Gram matrix
//    formed anew (segment_steps).  Bound by the launches and by
//    the bytes of X for p <= 16 (64 matrices of 16 x 4096: 8 + 14 us, 33 MB), by
//    the small products' chain as p nears 64 (one of 64 x 1024: 96 us) and then by
//    the fp64 matrix rate (60 TFLOP/s measured on a large product).  p = 65 takes
//    125 us for 1024 columns the other way, so the boundary costs nothing.
//  * p > 64: the iteration as written, on the fp16 matrix cores with fp32
//    accumulation, all three products as C = P Q^T of row-major operands.  The
//    state X is fp32 and a X is added in fp32; only the operands of products are
//    fp16.  Their rounding errors sit in the spaces that G spans with weight, so
//    the iteration does not blow them up as it does a rounding of X itself.  An
//    operand is two fp16 terms (hi + lo, 22 bits) and a product three fp16
//    products; one term and one product for a bf16 result of kOneTerm rows or more
//    in few steps (ortho_terms).
//    Operands are scaled by powers of two into fp16's range: bounds on x and G are
//    known because the host checks that the polynomial keeps singular values there,
//    roundings included.  Bound by how the tiles fill the chip and by the epilogues
//    behind the products: 4096 x 11008 in one term 4.1 ms (3.1 TFLOP by symmetric
//    halves, 0.76 PFLOP/s over the call).  Its symmetric products (gram 260,
//    polynomial 106 us) are 136 tiles on 256 CUs, whose matrix cores are busy 60 %
//    of the time; the step (435 us) is 688 tiles in three rounds, busy 46 %, with
//    540 MB of epilogue.  Two of 1371 x 2203 in two terms 0.84 ms.
#include <type_traits>

#include "nq_internal.h"

namespace nq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kGramMax = 64;  // shorter sides up to this take the fp64 form

// Shorter sides from kOneTerm on take one fp16 term for a bf16 result, in as many
// steps as kOneTermGain allows.  One term moves a result by 2e-4 of its norm (a
// rounding to 11 bits) times what B multiplies it by, its largest eigenvalue (2.8 of
// the default quintic), once per step whose singular values have grown to one.  At five
// default steps, beside a rounding to bf16 of 1.7e-3: 1.9e-3 for 65 x 300, 1.6e-3 for
// 256 x 256, 1.3e-3 for 512 x 700, 1.1e-3 for 2000 x 8000; in all 1.5, 1.4, 1.3 and
// 1.2 times the rounding alone.  At 512 x 700 twelve steps are off by 2.7 times the
// rounding and twenty by 5, so the square of that factor times the steps is bounded:
// 40, five default steps, 64 of 1.5, -0.5.  Two terms are off by 1.00 times the
// rounding.  They cost 1.2 to 1.8 times the call below 512 (us, one / two terms: 65 x
// 300 90 / 109, 256 x 1024 110 / 146, 500 x 700 117 / 184) and up to three times above
// it (4 of 768 x 4096 527 / 1193).
constexpr int kOneTerm = 512;
constexpr double kOneTermGain = 40.0;  // 512 x 700, twelve steps: 511 us; 4096 x 11008, five 4.1 ms, six 13.3

// Element types are fp32, bf16 bits and, of iterates between segments, fp64.
template <typename E>
struct ValueOf {
  typedef float type;
};
template <>
struct ValueOf<double> {
  typedef double type;
};

__device__ inline double load1(const double* p) { return *p; }
__device__ inline float load1(const float* p) { return *p; }
__device__ inline float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef double f64x4u __attribute__((ext_vector_type(4), aligned(8)));
__device__ inline void load4(const double* p, double (&v)[4]) {
  const f64x4u a = *reinterpret_cast<const f64x4u*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = a[e];
}
__device__ inline void load4(const float* p, float (&v)[4]) {
  const f32x4 a = *reinterpret_cast<const f32x4u*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = a[e];
}
__device__ inline void load4(const uint16_t* p, float (&v)[4]) {
  const u16x4u a = *reinterpret_cast<const u16x4u*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float((uint32_t)a[e] << 16);
}

// The sum over a workgroup of 256 threads, in a fixed order, to every thread.
__device__ inline double block_sum(double v, double* red) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
  __syncthreads();
  return ((red[0] + red[1]) + red[2]) + red[3];
}

__device__ inline uint16_t bf16_bits(float v) {  // round to nearest even
  const uint32_t u = __float_as_uint(v);
  if (v != v) return (uint16_t)((u >> 16) | 0x40);
  return (uint16_t)((u + 0x7FFF + ((u >> 16) & 1)) >> 16);
}
__device__ inline void store1(void* y, int bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t*>(y)[i] = bf16_bits(v);
  else
    static_cast<float*>(y)[i] = v;
}

// The first `count` of 4 consecutive results.
__device__ inline void store4(void* y, int bf16, int64_t at, const float (&v)[4], int64_t count) {
  if (count >= 4 && bf16) {
    *reinterpret_cast<u16x4u*>(static_cast<uint16_t*>(y) + at) =
        u16x4u{bf16_bits(v[0]), bf16_bits(v[1]), bf16_bits(v[2]), bf16_bits(v[3])};
  } else if (count >= 4) {
    *reinterpret_cast<f32x4u*>(static_cast<float*>(y) + at) = f32x4{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < count) store1(y, bf16, at + e, v[e]);
  }
}

__device__ inline void store4(double* y, int64_t at, const double (&v)[4], int64_t count) {
  if (count >= 4) {
    *reinterpret_cast<f64x4u*>(y + at) = f64x4u{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < count) y[at + e] = v[e];
  }
}

// ---------------------------------------------------------------- p <= 64
// One 16x16x4 fp64 instruction: lane l holds row l % 16, reduction l / 16 of
// each operand and rows 4 i + l / 16 (i = 0..3) of column l % 16 of the result.
struct SmallArgs {
  const void* x;
  int64_t ldx, stride_x;
  int p, tall;       // tall: the shorter side is the columns
  int64_t q;         // longer side
  int64_t span;      // longer-side elements of a workgroup
  double* gpart;     // [batch][spans][P][P], P = p rounded up to 16
  double* qmat;      // [batch][P][P]
  void* y;
  int y_bf16;
  double* it;        // [batch][rows][cols] the iterate between segments; may be x
  int spans, steps;  // steps: of this segment
  int normed;        // x is an iterate, not to be divided by its norm
  double a, b, c;
};

// Element (i, j) of the matrix with the shorter side first.
template <typename E>
__device__ inline const E* elem(const SmallArgs& s, const E* x, int64_t i, int64_t j) {
  return s.tall ? x + j * s.ldx + i : x + i * s.ldx + j;
}

// A lane's operands of a 32-deep step of the longer side from j: rows 16t + c,
// elements j + 8q + e (e-th instruction), zero from j1 on.
template <typename E, int PT>
__device__ inline void load_step(const SmallArgs& s, const E* x, int64_t j, int64_t j1, int q, int c,
                                 typename ValueOf<E>::type (&v)[PT][8]) {
  typedef typename ValueOf<E>::type V;
  const bool full = j + 32 <= j1;
#pragma unroll
  for (int t = 0; t < PT; ++t) {
    const int64_t i = min(16 * t + c, s.p - 1);
    const E* at = elem(s, x, i, j + 8 * q);
    if (full && !s.tall) {
      V lo[4], hi[4];
      load4(at, lo);
      load4(at + 4, hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[t][e] = lo[e], v[t][4 + e] = hi[e];
    } else if (full) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[t][e] = load1(at + e * s.ldx);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t jj = j + 8 * q + e;
        v[t][e] = jj < j1 ? load1(elem(s, x, i, jj)) : V(0);
      }
    }
  }
}

template <typename E, int PT>
__global__ __launch_bounds__(256) void ortho_gram_kernel(SmallArgs s) {
  __shared__ double part[4][4][64];
  constexpr int P = 16 * PT, NPAIR = PT * (PT + 1) / 2;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, c = lane % 16;
  const E* x = static_cast<const E*>(s.x) + (int64_t)blockIdx.y * s.stride_x;
  f64x4 acc[NPAIR];
#pragma unroll
  for (int k = 0; k < NPAIR; ++k) acc[k] = f64x4{0, 0, 0, 0};
  const int64_t j0 = (int64_t)blockIdx.x * s.span, j1 = imin(s.q, j0 + s.span);
  typedef typename ValueOf<E>::type V;
  V next[PT][8];
  int64_t j = j0 + 32 * wave;
  if (j < j1) load_step<E, PT>(s, x, j, j1, q, c, next);
  for (; j < j1; j += 128) {
    V v[PT][8];
#pragma unroll
    for (int t = 0; t < PT; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[t][e] = next[t][e];
    if (j + 128 < j1) load_step<E, PT>(s, x, j + 128, j1, q, c, next);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int k = 0;
#pragma unroll
      for (int t = 0; t < PT; ++t)
#pragma unroll
        for (int u = 0; u <= t; ++u, ++k)
          acc[k] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)v[t][e], (double)v[u][e], acc[k], 0, 0, 0);
    }
  }
  double* g = s.gpart + ((int64_t)blockIdx.y * s.spans + blockIdx.x) * P * P;
  int k = 0;
#pragma unroll
  for (int t = 0; t < PT; ++t)
#pragma unroll
    for (int u = 0; u <= t; ++u, ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][i][lane] = acc[k][i];
      __syncthreads();
      const int i = wave;  // this wave's register of the block
      const double sum = ((part[0][i][lane] + part[1][i][lane]) + part[2][i][lane]) + part[3][i][lane];
      const int row = 16 * t + 4 * i + q, col = 16 * u + c;
      const double out = row < s.p && col < s.p ? sum : 0.0;
      g[row * P + col] = out;
      if (t != u) g[col * P + row] = out;
    }
}

// 1 / ||X||_F^2 and 1 / ||X||_F from the trace of the Gram matrix.  A zero matrix
// stays zero; one that is not finite gives NaN.  An iterate is taken as it is.
__device__ inline void inverse_trace(double t, int normed, double& inv, double& root) {
  if (normed) {
    inv = root = 1.0;
    return;
  }
  inv = t > 0.0 && isfinite(t) ? 1.0 / t : (t == 0.0 ? 0.0 : __builtin_nan(""));
  root = t > 0.0 && isfinite(t) ? 1.0 / sqrt(t) : inv;
}

// The iteration on p x p matrices, one workgroup per matrix and a wave per 16x16
// block of them.  A (the Gram matrix of the iterate), P = a I + b A + c A^2 and Q
// (the product of the P so far) commute and are symmetric: every product reads both
// operands by rows, and P and the last Q are made in the registers of the products
// they come from.  A becomes P A^T P^T: with P on one side twice, A P^T P^T, what
// rounding leaves beside the diagonal grows by a^2 a step instead of a.  Bound by the
// chain of 19 products of five steps, about half of it the fp64 rate of one CU (a call
// of 64 x 1024: 96 us, with four waves 107).
template <int PT>
__global__ __launch_bounds__(64 * PT * PT) void ortho_solve_kernel(SmallArgs s) {
  constexpr int P = 16 * PT, S = P + 4, NTH = 64 * PT * PT;
  extern __shared__ double lds64[];
  double *A = lds64, *B = lds64 + P * S, *Q = lds64 + 2 * P * S;
  __shared__ double inv_sh[2];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, q = lane / 16, c = lane % 16;
  const double* g = s.gpart + (int64_t)blockIdx.x * s.spans * P * P;
  for (int i = tid; i < P * P; i += NTH) {
    double v = 0.0;
#pragma unroll 8
    for (int k = 0; k < s.spans; ++k) v += g[(int64_t)k * P * P + i];
    A[i / P * S + i % P] = v;
  }
  __syncthreads();
  if (wave == 0) {  // ||X||_F^2 is the trace
    double t = lane < P ? A[lane * S + lane] : 0.0;
    for (int off = 32; off > 0; off >>= 1) t += __shfl_xor(t, off);
    if (lane == 0) inverse_trace(t, s.normed, inv_sh[0], inv_sh[1]);
  }
  __syncthreads();
  const double inv = inv_sh[0];
  for (int i = tid; i < P * P; i += NTH) A[i / P * S + i % P] *= inv;
  __syncthreads();
  const int row = wave / PT * 16, col = wave % PT * 16;
  const int at = (row + q) * S + col + c;  // this lane's values: rows row + q + 4 i of column col + c
  auto product = [&](const double* L, const double* R) {  // this wave's block of L R^T
    f64x4 acc = {0, 0, 0, 0};
    const double* l = L + (row + c) * S + q;
    const double* r = R + (col + c) * S + q;
#pragma unroll
    for (int k = 0; k < P; k += 4) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(l[k], r[k], acc, 0, 0, 0);
    return acc;
  };
  auto store = [&](double* D, const f64x4& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) D[at + 4 * i * S] = v[i];
  };
  for (int step = 0; step < s.steps; ++step) {
    f64x4 v = product(A, A);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = s.c * v[i] + s.b * A[at + 4 * i * S] + (row + q + 4 * i == col + c ? s.a : 0.0);
    store(B, v);
    __syncthreads();
    const bool more = step + 1 < s.steps;
    f64x4 w = v;
    if (step > 0) w = product(Q, B);
    if (more) v = product(B, A);
    __syncthreads();  // every wave has read its operands
    store(Q, w);
    if (more) {
      store(A, v);
      __syncthreads();
      v = product(A, B);
      __syncthreads();
      store(A, v);
    }
    __syncthreads();
  }
  double* out = s.qmat + (int64_t)blockIdx.x * P * P;
  for (int i = tid; i < P * P; i += NTH) out[i] = Q[i / P * S + i % P] * inv_sh[1];
}

// The same for p <= 16 in the registers of a wave: its lanes hold a symmetric
// matrix M as M[c][4i + q], which is both how the instruction takes either operand
// (step i) and how it returns M[4i + q][c].
__device__ inline void solve16(const SmallArgs& s, double (&A)[4], double (&Q)[4], int q, int c) {
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) t += c == 4 * i + q ? A[i] : 0.0;
  for (int off = 32; off > 0; off >>= 1) t += __shfl_xor(t, off);
  double inv, root;
  inverse_trace(t, s.normed, inv, root);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] *= inv;
  auto product = [&](const double (&L)[4], const double (&R)[4], double (&D)[4]) {
    f64x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(L[i], R[i], acc, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) D[i] = acc[i];
  };
  for (int step = 0; step < s.steps; ++step) {
    double B[4];
    product(A, A, B);
#pragma unroll
    for (int i = 0; i < 4; ++i) B[i] = s.c * B[i] + s.b * A[i] + (c == 4 * i + q ? s.a : 0.0);
    if (step == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) Q[i] = B[i];
    } else {
      product(Q, B, Q);
    }
    if (step + 1 < s.steps) {
      product(A, B, A);
      product(A, B, A);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) Q[i] *= root;
}

// Y = Q X: a wave takes 64 elements of the longer side.  For p <= 16 every
// workgroup computes Q itself, from the spans' Gram matrices (a launch of its own
// for a few thousand operations would cost more).  IT: Y is the iterate in fp64; X
// may be the same one, since a wave stores only what it alone has loaded.
template <typename E, int PT, bool IT>
__global__ __launch_bounds__(256) void ortho_apply_kernel(SmallArgs s) {
  constexpr int P = 16 * PT, S = P + 4;
  extern __shared__ double lds64[];
  const int tid = threadIdx.x, lane = tid % 64, q = lane / 16, c = lane % 16;
  const int64_t j0 = ((int64_t)blockIdx.x * 4 + tid / 64) * 64;
  const E* x = static_cast<const E*>(s.x) + (int64_t)blockIdx.y * s.stride_x;
  // block v of the four holds longer-side elements j0 + 4c + v (wide: 16 bytes
  // of a row) or j0 + 16v + c (tall); e-th reduction step: shorter-side index
  // 16u + 4e + q (wide), 16u + 4q + e (tall)
  const bool full = j0 + 64 <= s.q;
  typedef typename ValueOf<E>::type V;
  auto load = [&](int u, V (&v)[4][4]) {
    if (full && !s.tall) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        V a[4];
        load4(x + (int64_t)min(16 * u + 4 * e + q, s.p - 1) * s.ldx + j0 + 4 * c, a);
#pragma unroll
        for (int b = 0; b < 4; ++b) v[b][e] = 16 * u + 4 * e + q < s.p ? a[b] : V(0);
      }
    } else if (full && 16 * u + 16 <= s.p) {
#pragma unroll
      for (int b = 0; b < 4; ++b) load4(x + (j0 + 16 * b + c) * s.ldx + 16 * u + 4 * q, v[b]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 16 * u + (s.tall ? 4 * q + e : 4 * e + q);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int64_t j = imin(s.tall ? j0 + 16 * b + c : j0 + 4 * c + b, s.q - 1);
          v[b][e] = k < s.p ? load1(elem(s, x, k, j)) : V(0);
        }
      }
    }
  };
  V first[4][4];
  if (j0 < s.q) load(0, first);
  if constexpr (PT == 1) {
    const double* g = s.gpart + (int64_t)blockIdx.y * s.spans * P * P;
    double v = 0.0;
#pragma unroll 8
    for (int k = 0; k < s.spans; ++k) v += g[(int64_t)k * P * P + tid];
    lds64[tid / P * S + tid % P] = v;
    __syncthreads();
    if (tid < 64) {
      double A[4], Q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) A[i] = lds64[c * S + 4 * i + q];
      solve16(s, A, Q, q, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) lds64[c * S + 4 * i + q] = Q[i];
    }
  } else {
    const double* qm = s.qmat + (int64_t)blockIdx.y * P * P;
    for (int i = tid; i < P * P; i += 256) lds64[i / P * S + i % P] = qm[i];
  }
  __syncthreads();
  if (j0 >= s.q) return;
  f64x4 acc[PT][4];
#pragma unroll
  for (int t = 0; t < PT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[t][v] = f64x4{0, 0, 0, 0};
  // tall: result row 4i + q of a block is stored as shorter-side index 4q + i, so
  // that a lane ends with 4 consecutive ones
  const int row = s.tall ? 4 * (c % 4) + c / 4 : c;
#pragma unroll
  for (int u = 0; u < PT; ++u) {
    V v[4][4];
    if (u == 0) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[b][e] = first[b][e];
    } else {
      load(u, v);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = 16 * u + (s.tall ? 4 * q + e : 4 * e + q);
#pragma unroll
      for (int t = 0; t < PT; ++t) {
        const double m = lds64[(16 * t + row) * S + k];
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[t][b] = __builtin_amdgcn_mfma_f64_16x16x4f64(m, (double)v[b][e], acc[t][b], 0, 0, 0);
      }
    }
  }
  const int64_t base = (int64_t)blockIdx.y * s.p * s.q;
#pragma unroll
  for (int t = 0; t < PT; ++t)
#pragma unroll
    for (int a = 0; a < 4; ++a) {  // four results side by side: of block a (tall), of register a (wide)
      typename std::conditional<IT, double, float>::type v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = s.tall ? acc[t][a][e] : acc[t][e][a];
      const int64_t j = s.tall ? j0 + 16 * a + c : j0 + 4 * c;
      const int i = 16 * t + (s.tall ? 4 * q : 4 * a + q);
      if (j >= s.q || i >= s.p) continue;
      const int64_t at = base + (s.tall ? j * s.p + i : (int64_t)i * s.q + j), count = s.tall ? s.p - i : s.q - j;
      if constexpr (IT)
        store4(s.it, at, v, count);
      else
        store4(s.y, s.y_bf16, at, v, count);
    }
}

// ---------------------------------------------------------------- p > 64
constexpr int kBK = 64;  // operand rows are padded to this: every tile shape is a multiple of it
constexpr float kScaleX = 16384.0f;  // operand scale of x: |x| <= kOrthoRange
constexpr int kSumBlocks = 512;  // partial sums of ||X||_F^2 per matrix

template <typename E>
__global__ __launch_bounds__(256) void ortho_sumsq_kernel(const E* __restrict__ x, int64_t rows, int64_t cols, int64_t ldx,
                                                          int64_t stride_x, double* __restrict__ part) {
  __shared__ double red[4];
  x += (int64_t)blockIdx.y * stride_x;
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const E* row = x + r * ldx;
#pragma unroll 4
    for (int64_t j = 4 * threadIdx.x; j + 4 <= cols; j += 1024) {
      float v[4];
      load4(row + j, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += (double)v[e] * v[e];
    }
    const int64_t j = cols / 4 * 4 + threadIdx.x;
    if (j < cols) {
      const double v = load1(row + j);
      sum[0] += v * v;
    }
  }
  const double t = block_sum((sum[0] + sum[1]) + (sum[2] + sum[3]), red);
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * kSumBlocks + blockIdx.x] = t;
}

// 1 / ||X||_F as f 2^e with f in (0.5, 1]: the norm of fp32 values may lie
// outside fp32.  Zero matrix: 0; a sum that is not finite: NaN.  Every thread of
// the workgroup (256) gets it.
__device__ inline float inverse_norm(const double* __restrict__ part, double* red, int& e) {
  double t = block_sum(part[threadIdx.x] + part[threadIdx.x + 256], red);
  e = 0;
  if (t == 0.0) return 0.0f;
  if (!isfinite(t)) return __builtin_nanf("");
  return (float)frexp(1.0 / sqrt(t), &e);
}

// An operand value as fp16 terms: hi, and for two terms the rest.
__device__ inline uint16_t half_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ inline void split_half(float v, int terms, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)v;
  hi = __builtin_bit_cast(uint16_t, h);
  lo = terms > 1 ? half_bits(v - (float)h) : 0;
}

// 8 values as fp16 terms, times a power of two.
__device__ inline void store_terms(uint16_t* out, int64_t term, int terms, const float (&v)[8], float scale) {
  f16x8 hi, lo;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = v[e] * scale;
    hi[e] = (_Float16)x;
    lo[e] = (_Float16)(x - (float)hi[e]);
  }
  *reinterpret_cast<f16x8*>(out) = hi;
  if (terms > 1) *reinterpret_cast<f16x8*>(out + term) = lo;
}

// The first `count` of 8 consecutive results.
__device__ inline void store8(void* y, int bf16, int64_t at, const float (&v)[8], int count) {
  if (count >= 8) {
    if (bf16) {
      typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
      u32x4u w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = (uint32_t)bf16_bits(v[2 * e]) | ((uint32_t)bf16_bits(v[2 * e + 1]) << 16);
      *reinterpret_cast<u32x4u*>(static_cast<uint16_t*>(y) + at) = w;
    } else {
      f32x4u* o = reinterpret_cast<f32x4u*>(static_cast<float*>(y) + at);
      o[0] = f32x4{v[0], v[1], v[2], v[3]};
      o[1] = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < count) store1(y, bf16, at + e, v[e]);
  }
}

struct LargeArgs {
  int p, pp;           // shorter side, and rounded up to kBK
  int q, qp;           // longer side
  int terms;
  float* xf;           // [batch][p][qp] state
  uint16_t* x16;       // [batch][terms][p][qp]
  uint16_t* xt16;      // [batch][terms][q][pp]
  const double* part;  // [batch][kSumBlocks]
  float* bad;          // [batch]: 0, or NaN for a matrix that is not finite
  float sx;            // operand scale of x
  int* arrived;        // counters of the split products, cleared here
  int64_t counters;
};

// Rows j0 .. of the transposed operand, columns i0 .., from a tile [i][j] of x.
__device__ inline void store_transposed(const LargeArgs& s, int64_t bi, int i0, int j0, const float (&tile)[64][65]) {
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  const int64_t ts = (int64_t)s.q * s.pp;
  for (int k = ty; k < 64; k += 4) {
    const int j = j0 + k, i = i0 + tx;
    if (j < s.q) {
      uint16_t hi, lo;
      split_half(tile[tx][k] * s.sx, s.terms, hi, lo);
      uint16_t* d = s.xt16 + bi * s.terms * ts + (int64_t)j * s.pp + i;
      d[0] = hi;
      if (s.terms > 1) d[ts] = lo;
    }
  }
}

// X0 in all its forms, with zeros in the padding.  A workgroup
// takes 64 x 64 elements (shorter side by longer side) through LDS.
template <typename E>
__global__ __launch_bounds__(256) void ortho_prepare_kernel(LargeArgs s, const E* __restrict__ x, int64_t ldx,
                                                            int64_t stride_x, int tall) {
  __shared__ float tile[64][65];
  __shared__ double red[4];
  const int64_t bi = blockIdx.z;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;  // i < pp, j < qp
  x += bi * stride_x;
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  int ex;
  const float f = inverse_norm(s.part + bi * kSumBlocks, red, ex);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) s.bad[bi] = f * 0.0f;
    for (int64_t i = threadIdx.x + 256 * bi; i < s.counters; i += 256 * (int64_t)gridDim.z) s.arrived[i] = 0;
  }
  for (int k = ty; k < 64; k += 4) {
    const int i = i0 + (tall ? tx : k), j = j0 + (tall ? k : tx);
    float v = 0.0f;
    if (i < s.p && j < s.q) v = ldexpf(load1(tall ? x + (int64_t)j * ldx + i : x + (int64_t)i * ldx + j), ex) * f;
    tile[tall ? tx : k][tall ? k : tx] = v;
  }
  __syncthreads();
  const int64_t xs = (int64_t)s.p * s.qp;
  for (int k = ty; k < 64; k += 4) {
    const int i = i0 + k, j = j0 + tx;
    if (i < s.p) {
      const float v = tile[k][tx];
      s.xf[(bi * s.p + i) * s.qp + j] = v;
      uint16_t hi, lo;
      split_half(v * s.sx, s.terms, hi, lo);
      uint16_t* d = s.x16 + bi * s.terms * xs + (int64_t)i * s.qp + j;
      d[0] = hi;
      if (s.terms > 1) d[xs] = lo;
    }
  }
  store_transposed(s, bi, i0, j0, tile);
}

// The transposed operand of an iterate, where there is room for one copy of it only: a
// step reads it whole and cannot write the next one beside.  Bound by its bytes (8 for
// each value; 512 x 700 to bf16, twelve steps: 511 us, to fp32 with two copies 421).
__global__ __launch_bounds__(256) void ortho_transpose_kernel(LargeArgs s) {
  __shared__ float tile[64][65];
  const int64_t bi = blockIdx.z;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;  // i < pp, j < qp
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
  for (int k = ty; k < 64; k += 4) {
    const int i = i0 + k;
    tile[k][tx] = i < s.p ? s.xf[(bi * s.p + i) * s.qp + j0 + tx] : 0.0f;
  }
  __syncthreads();
  store_transposed(s, bi, i0, j0, tile);
}

// Wait until at most N vector-memory operations of this wave are outstanding,
// and none of its LDS reads.
template <int N>
__device__ inline void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}

enum Mode { kGram = 0, kPoly = 1, kStep = 2, kLast = 3, kStepRows = 4 };

struct GemmArgs {
  const uint16_t *A, *B;   // [batch][terms][rows][K] fp16
  int64_t stride_a, stride_b, term_a, term_b;  // elements
  int M, N, K;             // K a multiple of kBK
  int tiles_m, tiles_n;    // sym: tiles with row block >= column block
  int sym, nseg;           // nseg: 1, or 3 products of two-term operands
  float s_acc, s_aux;
  int terms;
  // kGram, kPoly: out16 [batch][terms][M][ldo]; kPoly: aux16 as out16
  // kStep: xf (rows of ldo), out16 (x16), outt16 (the transpose); kStepRows: without
  // the transpose; kLast: xf, y
  uint16_t* out16;
  uint16_t* outt16;
  const uint16_t* aux16;
  int64_t ldo, ldt, term_o, term_t;
  float* xf;
  void* y;
  int y_bf16, y_t;         // y_t: store transposed
  const float* bad;
  int per;                 // reduction tiles of a split (gridDim.z of them)
  float* part;             // [batch][tiles][splits][registers][threads]
  int* arrived;            // [batch][tiles], zero before and after
};

// A split's partial sums: agent-scope stores, which write through by themselves (a
// release fence would write back the XCD's whole L2), then, once every thread's
// have completed, a relaxed count; the last workgroup acquires before it reads.
__device__ inline void store_agent(float* p, float v) {
  typedef __attribute__((address_space(1))) float* gptr;
  __hip_atomic_store((gptr)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline bool last_to_arrive(int* ctr, int n, int* s_last) {
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0) {
    typedef __attribute__((address_space(1))) int* gptr;
    *s_last = __hip_atomic_fetch_add((gptr)ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
    if (*s_last) {
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      __hip_atomic_store((gptr)ctr, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next product
    }
  }
  __syncthreads();
  return *s_last != 0;
}

// C = A B^T, workgroup tile BM x BN x BK: WM x WN waves of 32x32x16 fp16
// instructions.  Both operands stream into a ring of S LDS stages by direct
// global->LDS loads; rows of 2 BK bytes, 16-byte chunk c of row r stored at
// chunk c ^ swizzle(r), so that the 16 rows that a fragment read takes at once
// meet 16 different bank groups.
template <int BK>
__device__ constexpr int swizzle(int r) {
  return BK == 64 ? (r >> 1) & 7 : (r >> 2) & 3;
}

template <int BM, int BN, int BK, int WM, int WN, int S, bool SPREAD, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void ortho_gemm_kernel(GemmArgs p) {
  constexpr int NW = WM * WN, MB = BM / WM / 32, NB = BN / WN / 32;
  constexpr int ROW = 2 * BK, RPL = 1024 / ROW, CH = BK / 8;  // row bytes, rows of a load, chunks of a row
  constexpr bool STEP = MODE == kStep || MODE == kStepRows;
  constexpr int STAGE = (BM + BN) * ROW, LOADS_A = BM / RPL / NW, LOADS_B = BN / RPL / NW;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wave / WN, wn = wave % WN, l32 = lane % 32, h = lane / 32;
  // each XCD (workgroup index modulo 8) takes a contiguous range of tiles
  const int ntiles = p.sym ? p.tiles_m * (p.tiles_m + 1) / 2 : p.tiles_m * p.tiles_n;
  const int per = (ntiles + 7) / 8;
  const int t = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if ((int)(blockIdx.x / 8) >= per || t >= ntiles) return;
  int tm, tn;
  if (p.sym) {
    tm = (int)((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
    while (tm * (tm + 1) / 2 > t) --tm;
    tn = t - tm * (tm + 1) / 2;
  } else {
    tm = t / p.tiles_n;
    tn = t % p.tiles_n;
  }
  const int m0 = tm * BM, n0 = tn * BN;
  const int64_t bi = blockIdx.y;
  const uint16_t* A = p.A + bi * p.stride_a + (int64_t)m0 * p.K;
  const uint16_t* B = p.B + bi * p.stride_b + (int64_t)n0 * p.K;
  // rows past the matrix load its last row; they are not stored
  const int drow = lane / CH, dchunk = lane % CH;
  uint32_t oa[LOADS_A], ob[LOADS_B];  // bytes: a row of a tile lies below 2^25
#pragma unroll
  for (int j = 0; j < LOADS_A; ++j) {
    const int r = (wave * LOADS_A + j) * RPL + drow;
    oa[j] = 2 * ((uint32_t)min(r, p.M - 1 - m0) * p.K + (dchunk ^ swizzle<BK>(r)) * 8);
  }
#pragma unroll
  for (int j = 0; j < LOADS_B; ++j) {
    const int r = (wave * LOADS_B + j) * RPL + drow;
    ob[j] = 2 * ((uint32_t)min(r, p.N - 1 - n0) * p.K + (dchunk ^ swizzle<BK>(r)) * 8);
  }
  const int nk = p.K / BK, kbase = (int)blockIdx.z * p.per, total = min(p.per, nk * p.nseg - kbase);
  // product terms, the smallest first: hi lo, lo hi, hi hi; a stage's loads in
  // STEPS parts
  constexpr int STEPS = BK / 16, PER = LOADS_A + LOADS_B, PART = (PER + STEPS - 1) / STEPS;
  auto issue = [&](int k, int st, int part) {
    const int kt = kbase + min(k, total - 1);
    const int seg = kt / nk, kk = kt - seg * nk;
    const int ta = p.nseg == 1 ? 0 : (seg == 1), tb = p.nseg == 1 ? 0 : (seg == 0);
    const char* a = reinterpret_cast<const char*>(A + ta * p.term_a + (int64_t)kk * BK);
    const char* b = reinterpret_cast<const char*>(B + tb * p.term_b + (int64_t)kk * BK);
    char* dst = lds + st * STAGE;
#pragma unroll
    for (int l = part * PART; l < (part + 1) * PART && l < PER; ++l) {
      const int j = l / 2;  // A and B in turn
      const bool of_a = LOADS_A == LOADS_B ? l % 2 == 0 : l < LOADS_A;
      const int i = LOADS_A == LOADS_B ? j : (of_a ? l : l - LOADS_A);
      if (of_a)
        __builtin_amdgcn_global_load_lds((const void*)(a + oa[i < LOADS_A ? i : 0]),
                                         (__attribute__((address_space(3))) void*)(dst + (wave * LOADS_A + i) * 1024), 16, 0,
                                         0);
      else
        __builtin_amdgcn_global_load_lds(
            (const void*)(b + ob[i < LOADS_B ? i : 0]),
            (__attribute__((address_space(3))) void*)(dst + BM * ROW + (wave * LOADS_B + i) * 1024), 16, 0, 0);
    }
  };
  f32x16 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  uint32_t sw[STEPS];  // chunk 2s + h of this lane's row, swizzled
#pragma unroll
  for (int s = 0; s < STEPS; ++s) sw[s] = (uint32_t)l32 * ROW + (((2 * s + h) ^ swizzle<BK>(l32)) * 16);
  const uint32_t fa = wm * (BM / WM) * ROW, fb = BM * ROW + wn * (BN / WN) * ROW;
  // The fragments of a 16-deep step are read while the one before it is
  // multiplied, across stages too: once a wave holds the last step's fragments
  // it has no more use for the stage, so the barrier that frees it stands before
  // that step's products.
  f16x8 af[2][MB], bf[2][NB];
  auto read = [&](const char* stage, int s) {
#pragma unroll
    for (int i = 0; i < MB; ++i) af[s & 1][i] = *reinterpret_cast<const f16x8*>(stage + fa + i * 32 * ROW + sw[s]);
#pragma unroll
    for (int j = 0; j < NB; ++j) bf[s & 1][j] = *reinterpret_cast<const f16x8*>(stage + fb + j * 32 * ROW + sw[s]);
  };
  auto issue_all = [&](int kt, int st) {
#pragma unroll
    for (int part = 0; part < STEPS; ++part) issue(kt, st, part);
  };
  static_assert(STEPS % 2 == 0, "fragment buffers alternate across stages");
  if constexpr (SPREAD) {
    // the loads of stage kt + S follow in parts, one beside each step's products.
    // There are no branches: past the end the last stage is loaded and read again
    // (a branch would have the compiler wait for the reads on both its sides).
    // 128 x 128 tiles of 2 x 1371 x 1371 x 2203: 59 us, at once 75.
    // wait for the stage after this one (the S - 2 younger ones may stay in
    // flight) and for this wave's fragment reads, then meet the other waves
    auto landed = [&] {
      wait_loads<(S - 2) * PER>();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
#pragma unroll
    for (int kt = 0; kt < S - 1; ++kt)
#pragma unroll
      for (int part = 0; part < STEPS; ++part) issue(kt, kt, part);
    landed();
    issue(S - 1, S - 1, 0);
    read(lds, 0);
    for (int kt0 = 0; kt0 < total; kt0 += S) {
#pragma unroll
      for (int st = 0; st < S; ++st) {
        const int kt = kt0 + st;
        if (kt >= total) break;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          __builtin_amdgcn_sched_barrier(0);
          if (s + 1 < STEPS) {
            read(lds + st * STAGE, s + 1);
            issue(kt + S - 1, (st + S - 1) % S, s + 1);
          } else {
            landed();
            __builtin_amdgcn_sched_barrier(0);
            read(lds + (st + 1) % S * STAGE, 0);
            issue(kt + S, st, 0);
          }
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[s & 1][i], bf[s & 1][j], acc[i][j], 0, 0, 0);
          // one matrix instruction, then a share of the next step's fragment reads
          // and of the loads
#pragma unroll
          for (int i = 0; i < MB * NB; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (i < MB + NB) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if (i >= MB * NB - PART) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    wait_loads<0>();  // no load may land in LDS that the next workgroup owns
  } else {
    // the loads of stage kt + S at once behind the barrier: faster where two stages
    // are all that LDS holds (256 x 256: 276 us, spread 308; 4096 x 4096 x 11008)
    // wait for stage kt (later stages, S - 1 at most, may stay in flight) and for
    // this wave's fragment reads, then meet the other waves
    auto landed = [&](int later) {
      if (later >= S - 2)
        wait_loads<(S - 2) * PER>();
      else if (S > 3 && later == 1)
        wait_loads<PER>();
      else
        wait_loads<0>();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
#pragma unroll
    for (int kt = 0; kt < S; ++kt)
      if (kt < total) issue_all(kt, kt);
    if (total > S - 1)
      wait_loads<(S - 1) * PER>();
    else
      wait_loads<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(lds, 0);
    for (int kt0 = 0; kt0 < total; kt0 += S) {
#pragma unroll
      for (int st = 0; st < S; ++st) {
        const int kt = kt0 + st;
        if (kt >= total) break;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const bool more = s + 1 < STEPS || kt + 1 < total;
          __builtin_amdgcn_sched_barrier(0);
          if (s + 1 < STEPS) {
            read(lds + st * STAGE, s + 1);
          } else if (kt + 1 < total) {
            landed(total - 2 - kt);
            if (kt + S < total) issue_all(kt + S, st);
            __builtin_amdgcn_sched_barrier(0);
            read(lds + (st + 1) % S * STAGE, 0);
          } else {  // as on the other path, so that no wait for the reads above comes before the products
            wait_loads<0>();
          }
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[s & 1][i], bf[s & 1][j], acc[i][j], 0, 0, 0);
          // one matrix instruction, then a share of the next step's fragment reads
          if (more) {
#pragma unroll
            for (int i = 0; i < MB * NB; ++i) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              if (i < MB + NB) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  if constexpr (MODE == kGram || MODE == kPoly) {
    // few tiles over a long axis: the splits' sums are added in their order by the
    // workgroup that comes last (nobody waits)
    if (gridDim.z > 1) {
      constexpr int NT = 64 * NW, REGS = MB * NB * 16;
      __shared__ int last;
      float* part = p.part + (bi * ntiles + t) * gridDim.z * (REGS * NT) + threadIdx.x;
      float* mine = part + (int64_t)blockIdx.z * (REGS * NT);
#pragma unroll
      for (int b = 0; b < MB * NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) store_agent(mine + (b * 16 + r) * NT, acc[b / NB][b % NB][r]);
      if (!last_to_arrive(p.arrived + bi * ntiles + t, (int)gridDim.z, &last)) return;
#pragma unroll
      for (int b = 0; b < MB * NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[b / NB][b % NB][r] = part[(b * 16 + r) * NT];
      for (int z = 1; z < (int)gridDim.z; ++z) {
        part += REGS * NT;
#pragma unroll
        for (int b = 0; b < MB * NB; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[b / NB][b % NB][r] += part[(b * 16 + r) * NT];
      }
    }
  }
  // Epilogue, 32 rows at a time through the wave's part of LDS: lane l, register
  // 4a + c of a block holds row 8a + 4(l / 32) + c of column l % 32; read back, a
  // lane holds 8 consecutive columns of a row, and for a transposed result 8
  // consecutive rows of a column.  So everything moves 16 bytes a lane, in runs of
  // 64 bytes or more (two bytes a lane, straight from the registers, took 75 us of
  // the 150 us of a 256 x 256 tile with two terms).  Values past the matrix are
  // zero: they are the padding of the next product's operands.
  constexpr int CW = BN / WN, CS = CW + 4, CH8 = CW / 8, RPI = 64 / CH8;  // columns, LDS row, pieces, rows at once
  static_assert(NW * 32 * CS * 4 <= S * STAGE, "the ring holds the waves' blocks");
  float* blk = reinterpret_cast<float*>(lds) + wave * 32 * CS;
  uint16_t* out = p.out16 + bi * p.terms * p.term_o;
  uint16_t* outt = p.outt16 + bi * p.terms * p.term_t;
  const uint16_t* aux = p.aux16 + bi * p.terms * p.term_o;
  float* xf = p.xf + bi * p.M * p.ldo;
  const int64_t ybase = bi * p.M * (int64_t)p.N;
  const bool mirror = (MODE == kGram || MODE == kPoly) && p.sym && tm != tn;
  const bool transposed = MODE == kStep || (MODE == kLast && p.y_t) || mirror;
  const float bad = MODE == kLast ? p.bad[bi] : 0.0f;
  const int nb = n0 + wn * CW;
  // a transposed operand has padding along this tile's rows, too
  const int64_t rows_end = MODE == kStep ? p.ldt : (mirror ? p.ldo : p.M);
  __syncthreads();  // every wave is done with the ring
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int mr = m0 + wm * (BM / WM) + i * 32;
    if (mr >= rows_end) break;
    // what the block reads: 8 columns of rows lane / CH8 + RPI t
    float x[32 / RPI][8];
    const int n = nb + lane % CH8 * 8;
    if constexpr (MODE != kGram) {
#pragma unroll
      for (int t = 0; t < 32 / RPI; ++t) {
        const int64_t at = (int64_t)min(mr + lane / CH8 + RPI * t, p.M - 1) * p.ldo + min((int64_t)n, p.ldo - 8);
        if constexpr (MODE == kPoly) {
          const f16x8 g = *reinterpret_cast<const f16x8*>(aux + at);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[t][e] = (float)g[e];
          if (p.terms > 1) {
            const f16x8 l = *reinterpret_cast<const f16x8*>(aux + at + p.term_o);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[t][e] += (float)l[e];
          }
        } else {
          const f32x4 lo = *reinterpret_cast<const f32x4*>(xf + at), hi = *reinterpret_cast<const f32x4*>(xf + at + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][e] = lo[e], x[t][4 + e] = hi[e];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) blk[(8 * (r / 4) + 4 * h + r % 4) * CS + j * 32 + l32] = acc[i][j][r];
#pragma unroll
    for (int t = 0; t < 32 / RPI; ++t) {
      const int row = lane / CH8 + RPI * t, m = mr + row;
      float* cell = blk + row * CS + lane % CH8 * 8;
      float v[8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4 c = *reinterpret_cast<const f32x4*>(cell + 4 * u);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * u + e] = c[e] * p.s_acc;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (MODE != kGram) v[e] = fmaf(p.s_aux, x[t][e], v[e]);
        if constexpr (MODE == kLast) v[e] += bad;
        if (m >= p.M || n + e >= p.N) v[e] = 0.0f;
      }
      if (transposed) {
        *reinterpret_cast<f32x4*>(cell) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(cell + 4) = f32x4{v[4], v[5], v[6], v[7]};
      }
      if (m >= p.M) continue;
      if constexpr (MODE == kLast) {
        if (!p.y_t) store8(p.y, p.y_bf16, ybase + (int64_t)m * p.N + n, v, p.N - n);
      } else if (n < p.ldo) {
        if constexpr (STEP) {
          float* at = xf + (int64_t)m * p.ldo + n;
          *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<f32x4*>(at + 4) = f32x4{v[4], v[5], v[6], v[7]};
        }
        store_terms(out + (int64_t)m * p.ldo + n, p.term_o, p.terms, v, STEP ? kScaleX : 1.0f);
      }
    }
    if (transposed) {  // 8 rows of column lane / 4 + 16 t
#pragma unroll
      for (int t = 0; t < CW / 16; ++t) {
        const int col = lane / 4 + 16 * t, nn = nb + col, m = mr + lane % 4 * 8;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = blk[(lane % 4 * 8 + e) * CS + col];
        if (nn >= p.N) continue;
        if constexpr (MODE == kLast) {
          store8(p.y, p.y_bf16, ybase + (int64_t)nn * p.M + m, v, p.M - m);
        } else {
          const int64_t ld = MODE == kStep ? p.ldt : p.ldo;
          if (m < ld)
            store_terms((MODE == kStep ? outt : out) + (int64_t)nn * ld + m, MODE == kStep ? p.term_t : p.term_o, p.terms, v,
                        MODE == kStep ? kScaleX : 1.0f);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host side

struct OrthoLayout {
  bool small;
  int p, P, pp, qp, terms, copies, spans;  // copies: of the transposed operand
  int64_t q, span;
  size_t off_g, off_q, off_it, off_part, off_bad, off_xf, off_x16, off_xt[2], off_g16, off_b16, off_sums, off_arr, bytes;
  int64_t counters;
};

// Symmetric products of few tiles: the reduction is split, 16 tiles of it or more
// each, until a workgroup runs on every CU.  One matrix of 128 x 16384 has 3 tiles
// of 64 x 64: 229 us a call in fp32, unsplit 989; 128 x 4096 156 (splits of 8 tiles
// or more, two workgroups a CU: 171), unsplit 323.  64 matrices of 128 x 1024
// have 192: in one term 378 us whole, 415 in two splits.
int square_splits(int64_t batch, int64_t p, int64_t k, int terms) {
  const int64_t t = cdiv(p, 64), tiles = batch * t * (t + 1) / 2, all = k / kBK * (terms > 1 ? 3 : 1);
  const int64_t n = imax(1, imin(imin(256 / tiles, all / 16), 32));
  return (int)cdiv(all, cdiv(all, n));
}

// terms: of the operands (of a shorter side past kGramMax)
OrthoLayout ortho_layout(int64_t batch, int64_t rows, int64_t cols, nq_dtype yd, int terms) {
  OrthoLayout L{};
  L.p = (int)imin(rows, cols);
  L.q = imax(rows, cols);
  L.small = L.p <= kGramMax;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  if (L.small) {
    L.P = (int)round_up(L.p, 16);
    L.spans = (int)imax(1, imin(imin(cdiv(1024, batch), cdiv(L.q, 256)), 32));
    L.span = round_up(cdiv(L.q, L.spans), 128);
    L.spans = (int)cdiv(L.q, L.span);
    L.off_g = take((size_t)batch * L.spans * L.P * L.P * sizeof(double));
    L.off_q = take((size_t)batch * L.P * L.P * sizeof(double));
    L.off_it = take((size_t)batch * rows * cols * sizeof(double));  // the query does not know the steps: always
  } else {
    L.terms = terms;
    L.copies = yd == NQ_BF16 && L.p >= kOneTerm && terms == 2 ? 1 : 2;  // no more than a quarter over one term
    L.pp = (int)round_up(L.p, kBK);
    L.qp = (int)round_up(L.q, kBK);
    L.off_part = take((size_t)batch * kSumBlocks * sizeof(double));
    L.off_bad = take((size_t)batch * sizeof(float));
    L.off_xf = take((size_t)batch * L.p * L.qp * sizeof(float));
    L.off_x16 = take((size_t)batch * L.terms * L.p * L.qp * 2);
    for (int i = 0; i < L.copies; ++i) L.off_xt[i] = take((size_t)batch * L.terms * L.q * L.pp * 2);
    L.off_g16 = take((size_t)batch * L.terms * L.p * L.pp * 2);
    L.off_b16 = take((size_t)batch * L.terms * L.p * L.pp * 2);
    const int splits = (int)imax(square_splits(batch, L.p, L.qp, L.terms), square_splits(batch, L.p, L.pp, L.terms));
    if (splits > 1) {
      L.counters = batch * cdiv(L.p, 64) * (cdiv(L.p, 64) + 1) / 2;
      L.off_sums = take((size_t)L.counters * splits * 64 * 64 * sizeof(float));
      L.off_arr = take((size_t)L.counters * sizeof(int));
    }
  }
  L.bytes = off;
  return L;
}

// Steps on one Gram matrix.  Its rounding errors, 2^-53 n of the largest value,
// grow by at most the polynomial's largest square a step: by 2^20 in all, 2^-33 n,
// far below the result's rounding (five steps of the default quintic, 17 of 1.5,
// -0.5).  With more, a gradient of rank 4 (fewer tokens than rows) loses every digit
// from 20 steps on and is NaN at 30; in segments it stays as near the definition as
// the iteration as written in fp64 (2e-6 at 20 steps, 6e-6 as written).
int segment_steps(double ca, double cb, double cc) {
  const double top = 1.25 * 1.25;
  double m = fmax(fabs(ca), fabs(ca + cb * top + cc * top * top));
  const double v = cc != 0.0 ? -cb / (2.0 * cc) : 0.0;
  if (v > 0.0 && v < top) m = fmax(m, fabs(ca + cb * v + cc * v * v));
  return m * m <= 1.25 ? 64 : (int)imax(1, (int64_t)floor(20.0 / log2(m * m)));
}

template <typename E, int PT>
hipError_t launch_small(const SmallArgs& a, int64_t batch, bool last, hipStream_t s) {
  constexpr int P = 16 * PT, S = P + 4;
  hipLaunchKernelGGL((ortho_gram_kernel<E, PT>), dim3((unsigned)a.spans, (unsigned)batch), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if constexpr (PT > 1) {
    static std::atomic<uint64_t> done{0};
    if (e == hipSuccess)
      e = allow_lds(reinterpret_cast<const void*>(ortho_solve_kernel<PT>), 3 * P * S * sizeof(double), done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ortho_solve_kernel<PT>), dim3((unsigned)batch), dim3(64 * PT * PT), 3 * P * S * sizeof(double), s, a);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)cdiv(a.q, 256), (unsigned)batch);
  if (last)
    hipLaunchKernelGGL((ortho_apply_kernel<E, PT, false>), grid, dim3(256), P * S * sizeof(double), s, a);
  else
    hipLaunchKernelGGL((ortho_apply_kernel<E, PT, true>), grid, dim3(256), P * S * sizeof(double), s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_small_p(const SmallArgs& a, int64_t batch, bool last, hipStream_t s) {
  switch (cdiv(a.p, 16)) {
    case 1: return launch_small<E, 1>(a, batch, last, s);
    case 2: return launch_small<E, 2>(a, batch, last, s);
    case 3: return launch_small<E, 3>(a, batch, last, s);
    default: return launch_small<E, 4>(a, batch, last, s);
  }
}

template <int BM, int BN, int BK, int WM, int WN, int S, bool SPREAD, int MODE>
hipError_t launch_gemm_tile(GemmArgs g, int64_t batch, hipStream_t s, int splits = 1) {
  constexpr size_t lds = (size_t)S * (BM + BN) * BK * 2;
  const auto kernel = ortho_gemm_kernel<BM, BN, BK, WM, WN, S, SPREAD, MODE>;
  static std::atomic<uint64_t> done{0};
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), lds, done);
  if (e != hipSuccess) return e;
  g.tiles_m = (int)cdiv(g.M, BM);
  g.tiles_n = (int)cdiv(g.N, BN);
  g.per = (int)cdiv(g.K / BK * g.nseg, splits);
  const int64_t tiles = g.sym ? (int64_t)g.tiles_m * (g.tiles_m + 1) / 2 : (int64_t)g.tiles_m * g.tiles_n;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(8 * cdiv(tiles, 8)), (unsigned)batch, (unsigned)splits), dim3(64 * WM * WN), lds, s, g);
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_ortho_gemm(GemmArgs g, int64_t batch, hipStream_t s) {
  constexpr bool square = MODE == kGram || MODE == kPoly;
  // The largest tile that still occupies most of the chip: per product, smaller
  // tiles move more operand bytes and take more of the power the matrix cores run
  // on (4096 x 4096 x 11008, symmetric: 256 us with 256 x 256 tiles, 300 with
  // 128 x 128), but a launch of few large tiles leaves CUs idle (2 x 1371 x 1371 x
  // 2203, two terms: 108 tiles of 256 x 256 107 us, 198 of 128 x 256 75 us; 42 /
  // 132 / 552 tiles of 256 / 128 / 64 in the symmetric product of p x p matrices
  // 101 / 45 / 39 us).
  auto tiles = [&](int64_t bm, int64_t bn) {
    const int64_t tm = cdiv(g.M, bm), tn = cdiv(g.N, bn);
    return batch * (g.sym ? tm * (tm + 1) / 2 : tm * tn);
  };
  g.sym = square;  // a symmetric result: tiles on and below the diagonal, stored twice
  if (tiles(256, 256) >= (square ? 128 : 224)) return launch_gemm_tile<256, 256, 64, 2, 4, 2, false, MODE>(g, batch, s);
  if constexpr (!square)
    if (tiles(128, 256) >= 128) return launch_gemm_tile<128, 256, 64, 2, 4, 3, true, MODE>(g, batch, s);
  if (tiles(128, 128) >= 192) return launch_gemm_tile<128, 128, 64, 2, 2, 4, true, MODE>(g, batch, s);
  const int splits = square ? square_splits(batch, g.M, g.K, g.terms) : 1;
  return launch_gemm_tile<64, 64, 64, 2, 2, 4, true, MODE>(g, batch, s, splits);
}

// The largest |b l + c l^2| for l in [0, top].
double poly_bound(double b, double c, double top) {
  double m = fabs(b * top + c * top * top);
  if (c != 0.0) {
    const double v = -b / (2.0 * c);
    if (v > 0.0 && v < top) m = fmax(m, fabs(b * v + c * v * v));
  }
  return m;
}

// The operands' terms (of a shorter side past kGramMax): see kOneTerm.
int ortho_terms(int64_t rows, int64_t cols, nq_dtype yd, int steps, double cb, double cc) {
  if (yd == NQ_F32 || imin(rows, cols) < kOneTerm) return 2;
  const double gain = poly_bound(cb, cc, 1.25 * 1.25);
  return gain * gain * steps <= kOneTermGain ? 1 : 2;
}

}  // namespace

double ortho_rounding(int64_t rows, int64_t cols, nq_dtype yd, int steps, double cb, double cc) {
  if (imin(rows, cols) <= kGramMax) return 0x1p-33;  // what a segment may grow to
  return ortho_terms(rows, cols, yd, steps, cb, cc) == 2 ? 0x1p-21 : 0x1p-11 / sqrt(3.0);
}

size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols, nq_dtype yd) {
  const size_t two = ortho_layout(batch, rows, cols, yd, 2).bytes;
  if (yd == NQ_F32 || imin(rows, cols) < kOneTerm) return two;
  const size_t one = ortho_layout(batch, rows, cols, yd, 1).bytes;  // the steps are not known here
  return one > two ? one : two;
}

hipError_t launch_ortho(const void* x, nq_dtype xd, int64_t batch, int64_t rows, int64_t cols, int64_t ldx,
                        int64_t stride_x, int steps, double ca, double cb, double cc, void* y, nq_dtype yd, void* workspace,
                        hipStream_t s) {
  const OrthoLayout L = ortho_layout(batch, rows, cols, yd, ortho_terms(rows, cols, yd, steps, cb, cc));
  char* ws = static_cast<char*>(workspace);
  const int tall = rows > cols;
  if (L.small) {
    SmallArgs a;
    a.x = x;
    a.ldx = ldx;
    a.stride_x = stride_x;
    a.p = L.p;
    a.tall = tall;
    a.q = L.q;
    a.span = L.span;
    a.gpart = reinterpret_cast<double*>(ws + L.off_g);
    a.qmat = reinterpret_cast<double*>(ws + L.off_q);
    a.y = y;
    a.y_bf16 = yd == NQ_BF16;
    a.spans = L.spans;
    a.it = reinterpret_cast<double*>(ws + L.off_it);
    a.a = ca;
    a.b = cb;
    a.c = cc;
    const int most = segment_steps(ca, cb, cc);
    for (int done = 0; done < steps; done += a.steps) {
      a.steps = (int)imin(most, steps - done);
      a.normed = done > 0;
      const bool last = done + a.steps == steps;
      hipError_t e;
      if (done > 0)
        e = launch_small_p<double>(a, batch, last, s);
      else
        e = xd == NQ_BF16 ? launch_small_p<uint16_t>(a, batch, last, s) : launch_small_p<float>(a, batch, last, s);
      if (e != hipSuccess) return e;
      a.x = a.it;
      a.ldx = cols;
      a.stride_x = rows * cols;
    }
    return hipSuccess;
  }
  double* part = reinterpret_cast<double*>(ws + L.off_part);
  LargeArgs l;
  l.p = L.p;
  l.pp = L.pp;
  l.q = (int)L.q;
  l.qp = L.qp;
  l.terms = L.terms;
  l.xf = reinterpret_cast<float*>(ws + L.off_xf);
  l.x16 = reinterpret_cast<uint16_t*>(ws + L.off_x16);
  uint16_t* const xt16[2] = {reinterpret_cast<uint16_t*>(ws + L.off_xt[0]),
                             reinterpret_cast<uint16_t*>(ws + L.off_xt[L.copies - 1])};
  uint16_t* const g16 = reinterpret_cast<uint16_t*>(ws + L.off_g16);
  uint16_t* const b16 = reinterpret_cast<uint16_t*>(ws + L.off_b16);
  l.xt16 = xt16[0];
  l.part = part;
  l.bad = reinterpret_cast<float*>(ws + L.off_bad);
  l.arrived = reinterpret_cast<int*>(ws + L.off_arr);
  l.counters = L.counters;
  // |x| <= kOrthoRange, |G| <= its square and the polynomial's bound, each times its
  // scale below 65504
  const float sx = kScaleX, sg = 16384.0f;
  l.sx = sx;
  const double bound = poly_bound(cb, cc, kOrthoRange * kOrthoRange);
  const float sb = ldexpf(1.0f, bound > 0.0 ? (int)imax(-40, imin(14, (int64_t)floor(log2(60000.0 / bound)))) : 0);
  const dim3 pgrid((unsigned)(L.qp / 64), (unsigned)(L.pp / 64), (unsigned)batch);
  if (xd == NQ_BF16)
    hipLaunchKernelGGL((ortho_sumsq_kernel<uint16_t>), dim3(kSumBlocks, (unsigned)batch), dim3(256), 0, s,
                       static_cast<const uint16_t*>(x), rows, cols, ldx, stride_x, part);
  else
    hipLaunchKernelGGL((ortho_sumsq_kernel<float>), dim3(kSumBlocks, (unsigned)batch), dim3(256), 0, s,
                       static_cast<const float*>(x), rows, cols, ldx, stride_x, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (xd == NQ_BF16)
    hipLaunchKernelGGL((ortho_prepare_kernel<uint16_t>), pgrid, dim3(256), 0, s, l, static_cast<const uint16_t*>(x), ldx,
                       stride_x, tall);
  else
    hipLaunchKernelGGL((ortho_prepare_kernel<float>), pgrid, dim3(256), 0, s, l, static_cast<const float*>(x), ldx,
                       stride_x, tall);
  if ((e = hipGetLastError()) != hipSuccess) return e;

  const int64_t xs = (int64_t)L.p * L.qp, ts = L.q * L.pp, gs = (int64_t)L.p * L.pp;
  GemmArgs gram{}, poly{}, step{};
  gram.nseg = poly.nseg = step.nseg = L.terms == 2 ? 3 : 1;
  gram.terms = poly.terms = step.terms = L.terms;
  gram.A = gram.B = l.x16;
  gram.stride_a = gram.stride_b = L.terms * xs;
  gram.term_a = gram.term_b = xs;
  gram.M = gram.N = L.p;
  gram.K = L.qp;
  gram.out16 = g16;
  gram.ldo = L.pp;
  gram.term_o = gs;
  gram.s_acc = sg / (sx * sx);
  gram.part = reinterpret_cast<float*>(ws + L.off_sums);
  gram.arrived = l.arrived;
  poly = gram;
  poly.A = poly.B = g16;
  poly.stride_a = poly.stride_b = L.terms * gs;
  poly.term_a = poly.term_b = gs;
  poly.K = L.pp;
  poly.out16 = b16;
  poly.aux16 = g16;
  poly.s_acc = (float)(cc * sb / ((double)sg * sg));
  poly.s_aux = (float)(cb * sb / sg);
  step.A = b16;
  step.stride_a = L.terms * gs;
  step.term_a = gs;
  step.stride_b = L.terms * ts;
  step.term_b = ts;
  step.M = L.p;
  step.N = (int)L.q;
  step.K = L.pp;
  step.s_acc = 1.0f / (sb * sx);
  step.s_aux = (float)ca;
  step.xf = l.xf;
  step.out16 = l.x16;
  step.ldo = L.qp;
  step.term_o = xs;
  step.ldt = L.pp;
  step.term_t = ts;
  step.y = y;
  step.y_bf16 = yd == NQ_BF16;
  step.y_t = tall;
  step.bad = l.bad;
  for (int i = 0; i < steps; ++i) {
    if ((e = launch_ortho_gemm<kGram>(gram, batch, s)) != hipSuccess) return e;
    if ((e = launch_ortho_gemm<kPoly>(poly, batch, s)) != hipSuccess) return e;
    step.B = xt16[i % 2];
    step.outt16 = xt16[1 - i % 2];
    if (i + 1 == steps) {
      e = launch_ortho_gemm<kLast>(step, batch, s);
    } else if (L.copies == 2) {
      e = launch_ortho_gemm<kStep>(step, batch, s);
    } else {
      if ((e = launch_ortho_gemm<kStepRows>(step, batch, s)) != hipSuccess) return e;
      hipLaunchKernelGGL(ortho_transpose_kernel, pgrid, dim3(256), 0, s, l);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nq
