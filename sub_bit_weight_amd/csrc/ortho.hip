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
//    (X0 enters exactly, one rounding at the end).  HBM-bound for small p,
//    bound by the fp64 matrix rate (60 TFLOP/s measured on a large product)
//    as p nears 64.
//  * p > 64: the iteration as written, on the fp16 matrix cores with fp32
//    accumulation, all three products as C = P Q^T of row-major operands.  The
//    state X is fp32 and a X is added in fp32; only the operands of products are
//    fp16.  Their rounding errors sit in the spaces that G spans with weight, so
//    the iteration does not blow them up as it does a rounding of X itself.  For
//    an fp32 result each operand is two fp16 terms (hi + lo, 22 bits) and a
//    product three fp16 products.  Operands are scaled by powers of two into
//    fp16's range: |x| <= |G| bounds are known because the host checks that the
//    polynomial maps [0, 1.25] into [-1.25, 1.25].
#include "nq_internal.h"

namespace nq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

constexpr int kGramMax = 64;  // shorter sides up to this take the fp64 form

__device__ inline float load1(const float* p) { return *p; }
__device__ inline float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));
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
  int spans, steps;
  double a, b, c;
};

// Element (i, j) of the matrix with the shorter side first.
template <typename E>
__device__ inline const E* elem(const SmallArgs& s, const E* x, int64_t i, int64_t j) {
  return s.tall ? x + j * s.ldx + i : x + i * s.ldx + j;
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
  for (int64_t j = j0 + 32 * wave; j < j1; j += 128) {
    // lane group q takes elements j + 8q .. of the longer side, step e the e-th
    float v[PT][8];
#pragma unroll
    for (int t = 0; t < PT; ++t) {
      const int64_t i = min(16 * t + c, s.p - 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t jj = j + 8 * q + e;
        v[t][e] = jj < j1 ? load1(elem(s, x, i, jj)) : 0.0f;
      }
    }
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

// The iteration on p x p matrices, one workgroup per matrix.  A (the Gram
// matrix of the iterate), P = a I + b A + c A^2 and Q (the product of the P so
// far) commute and are symmetric: every product reads both operands by rows.
template <int PT>
__global__ __launch_bounds__(256) void ortho_solve_kernel(SmallArgs s) {
  constexpr int P = 16 * PT, S = P + 4, NT = (PT * PT + 3) / 4;
  extern __shared__ double lds64[];
  double *A = lds64, *B = lds64 + P * S, *Q = lds64 + 2 * P * S;
  __shared__ double inv_sh[2];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, q = lane / 16, c = lane % 16;
  const double* g = s.gpart + (int64_t)blockIdx.x * s.spans * P * P;
  for (int i = tid; i < P * P; i += 256) {
    double v = g[i];
    for (int k = 1; k < s.spans; ++k) v += g[(int64_t)k * P * P + i];
    A[i / P * S + i % P] = v;
  }
  __syncthreads();
  if (wave == 0) {  // ||X||_F^2 is the trace
    double t = lane < P ? A[lane * S + lane] : 0.0;
    for (int off = 32; off > 0; off >>= 1) t += __shfl_xor(t, off);
    if (lane == 0) {
      // a zero matrix stays zero; a matrix that is not finite gives NaN
      inv_sh[0] = t > 0.0 && isfinite(t) ? 1.0 / t : (t == 0.0 ? 0.0 : __builtin_nan(""));
      inv_sh[1] = t > 0.0 && isfinite(t) ? 1.0 / sqrt(t) : inv_sh[0];
    }
  }
  __syncthreads();
  const double inv = inv_sh[0];
  for (int i = tid; i < P * P; i += 256) A[i / P * S + i % P] *= inv;
  __syncthreads();
  f64x4 acc[NT];
  auto product = [&](const double* L, const double* R) {  // acc = this wave's blocks of L R
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      acc[n] = f64x4{0, 0, 0, 0};
      const int blk = wave + 4 * n;
      if (blk >= PT * PT) continue;
      const double* l = L + (blk / PT * 16 + c) * S + q;
      const double* r = R + (blk % PT * 16 + c) * S + q;
#pragma unroll
      for (int k = 0; k < P; k += 4) acc[n] = __builtin_amdgcn_mfma_f64_16x16x4f64(l[k], r[k], acc[n], 0, 0, 0);
    }
  };
  auto store = [&](double* D) {
    __syncthreads();  // every wave has read its operands
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int blk = wave + 4 * n;
      if (blk >= PT * PT) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) D[(blk / PT * 16 + 4 * i + q) * S + blk % PT * 16 + c] = acc[n][i];
    }
    __syncthreads();
  };
  for (int step = 0; step < s.steps; ++step) {
    product(A, A);
    store(B);
    for (int i = tid; i < P * P; i += 256) {
      const int at = i / P * S + i % P;
      const double v = s.c * B[at] + s.b * A[at] + (i / P == i % P ? s.a : 0.0);
      B[at] = v;
      if (step == 0) Q[at] = v;
    }
    __syncthreads();
    if (step > 0) {
      product(Q, B);
      store(Q);
    }
    if (step + 1 < s.steps) {
      product(A, B);
      store(A);
      product(A, B);
      store(A);
    }
  }
  double* out = s.qmat + (int64_t)blockIdx.x * P * P;
  for (int i = tid; i < P * P; i += 256) out[i] = Q[i / P * S + i % P] * inv_sh[1];
}

// Y = Q X: a wave takes 64 elements of the longer side.
template <typename E, int PT>
__global__ __launch_bounds__(256) void ortho_apply_kernel(SmallArgs s) {
  constexpr int P = 16 * PT, S = P + 4;
  extern __shared__ double lds64[];
  const int tid = threadIdx.x, lane = tid % 64, q = lane / 16, c = lane % 16;
  const double* qm = s.qmat + (int64_t)blockIdx.y * P * P;
  for (int i = tid; i < P * P; i += 256) lds64[i / P * S + i % P] = qm[i];
  __syncthreads();
  const int64_t j0 = ((int64_t)blockIdx.x * 4 + tid / 64) * 64;
  if (j0 >= s.q) return;
  const E* x = static_cast<const E*>(s.x) + (int64_t)blockIdx.y * s.stride_x;
  f64x4 acc[PT][4];
#pragma unroll
  for (int t = 0; t < PT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[t][v] = f64x4{0, 0, 0, 0};
  // block v of the four holds longer-side elements j0 + 4c + v (wide: 16 bytes
  // of a row) or j0 + 16v + c (tall)
  int64_t j[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) j[v] = imin(s.tall ? j0 + 16 * v + c : j0 + 4 * c + v, s.q - 1);
  // tall: result row 4i + q of a block is stored as shorter-side index 4q + i, so
  // that a lane ends with 4 consecutive ones
  const int row = s.tall ? 4 * (c % 4) + c / 4 : c;
#pragma unroll
  for (int u = 0; u < PT; ++u) {
    float v[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // reduction order: wide 16u + 4e + q, tall 16u + 4q + e
      const int k = 16 * u + (s.tall ? 4 * q + e : 4 * e + q);
#pragma unroll
      for (int b = 0; b < 4; ++b) v[b][e] = k < s.p ? load1(elem(s, x, k, j[b])) : 0.0f;
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
    for (int b = 0; b < 4; ++b) {
      const int64_t jj = s.tall ? j0 + 16 * b + c : j0 + 4 * c + b;
      if (jj >= s.q) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ii = 16 * t + (s.tall ? 4 * q + i : 4 * i + q);
        if (ii < s.p) store1(s.y, s.y_bf16, base + (s.tall ? jj * s.p + ii : ii * s.q + jj), (float)acc[t][b][i]);
      }
    }
}

// ---------------------------------------------------------------- p > 64
constexpr int kBK = 64;
constexpr float kScaleX = 16384.0f;  // operand scale of x: |x| <= 1.25
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

struct LargeArgs {
  int p, pp;           // shorter side, and rounded up to kBK
  int q, qp;           // longer side
  int terms;
  float* xf;           // [batch][p][q] state
  uint16_t* x16;       // [batch][terms][p][qp]
  uint16_t* xt16[2];   // [batch][terms][q][pp]
  uint16_t* g16;       // [batch][terms][p][pp]
  uint16_t* b16;       // [batch][terms][p][pp]
  const double* part;  // [batch][kSumBlocks]
  float* bad;          // [batch]: 0, or NaN for a matrix that is not finite
  float sx;            // operand scale of x
};

// X0 in all its forms, and zeros in the padding of every operand.  A workgroup
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
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) s.bad[bi] = f * 0.0f;
  for (int k = ty; k < 64; k += 4) {
    const int i = i0 + (tall ? tx : k), j = j0 + (tall ? k : tx);
    float v = 0.0f;
    if (i < s.p && j < s.q) v = ldexpf(load1(tall ? x + (int64_t)j * ldx + i : x + (int64_t)i * ldx + j), ex) * f;
    tile[tall ? tx : k][tall ? k : tx] = v;
  }
  __syncthreads();
  const int64_t xs = (int64_t)s.p * s.qp, ts = (int64_t)s.q * s.pp, gs = (int64_t)s.p * s.pp;
  for (int k = ty; k < 64; k += 4) {
    {
      const int i = i0 + k, j = j0 + tx;
      if (i < s.p) {
        const float v = tile[k][tx];
        if (j < s.q) s.xf[(bi * s.p + i) * s.q + j] = v;
        uint16_t hi, lo;
        split_half(v * s.sx, s.terms, hi, lo);
        uint16_t* d = s.x16 + bi * s.terms * xs + (int64_t)i * s.qp + j;
        d[0] = hi;
        if (s.terms > 1) d[xs] = lo;
      }
    }
    {
      const int j = j0 + k, i = i0 + tx;
      if (j < s.q) {
        uint16_t hi, lo;
        split_half(tile[tx][k] * s.sx, s.terms, hi, lo);
        for (int b = 0; b < (i < s.p ? 1 : 2); ++b) {
          uint16_t* d = s.xt16[b] + bi * s.terms * ts + (int64_t)j * s.pp + i;
          d[0] = hi;
          if (s.terms > 1) d[ts] = lo;
        }
      }
    }
  }
  if (blockIdx.x == 0 && i0 + 64 > s.p)  // the last rows' block: padding columns of G and B
    for (int64_t e = threadIdx.x; e < (int64_t)s.p * (s.pp - s.p); e += 256) {
      const int64_t at = bi * s.terms * gs + e / (s.pp - s.p) * s.pp + s.p + e % (s.pp - s.p);
      for (int t = 0; t < s.terms; ++t) s.g16[at + t * gs] = s.b16[at + t * gs] = 0;
    }
}

enum Mode { kGram = 0, kPoly = 1, kStep = 2, kLast = 3 };

struct GemmArgs {
  const uint16_t *A, *B;   // [batch][terms][rows][K] fp16
  int64_t stride_a, stride_b, term_a, term_b;  // elements
  int M, N, K;             // K a multiple of kBK
  int tiles_m, tiles_n;    // sym: tiles with row block >= column block
  int sym, nseg;           // nseg: 1, or 3 products of two-term operands
  float s_acc, s_aux;
  int terms;
  // kGram, kPoly: out16 [batch][terms][M][ldo]; kPoly: aux16 as out16
  // kStep: xf, out16 (x16), outt16 (the transpose); kLast: y
  uint16_t* out16;
  uint16_t* outt16;
  const uint16_t* aux16;
  int64_t ldo, ldt, term_o, term_t;
  float* xf;
  void* y;
  int y_bf16, y_t;         // y_t: store transposed
  const float* bad;
};

// C = A B^T, workgroup tile BM x BN x 64: WM x WN waves of 32x32x16 fp16
// instructions.  Both operands stream into a ring of S LDS stages by direct
// global->LDS loads; rows of 128 bytes, 16-byte chunk c of row r stored at
// chunk c ^ ((r >> 1) & 7), so that fragment reads (32 rows at one chunk) meet
// no bank twice in a group of 8 lanes.
template <int BM, int BN, int WM, int WN, int S, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void ortho_gemm_kernel(GemmArgs p) {
  constexpr int NW = WM * WN, MB = BM / WM / 32, NB = BN / WN / 32;
  constexpr int STAGE = (BM + BN) * 128, LOADS_A = BM / 8 / NW, LOADS_B = BN / 8 / NW;
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
  const int drow = lane / 8, dchunk = lane % 8;
  uint32_t oa[LOADS_A], ob[LOADS_B];
#pragma unroll
  for (int j = 0; j < LOADS_A; ++j) {
    const int r = (wave * LOADS_A + j) * 8 + drow;
    oa[j] = (uint32_t)min(r, p.M - 1 - m0) * p.K + ((dchunk ^ ((r >> 1) & 7)) * 8);
  }
#pragma unroll
  for (int j = 0; j < LOADS_B; ++j) {
    const int r = (wave * LOADS_B + j) * 8 + drow;
    ob[j] = (uint32_t)min(r, p.N - 1 - n0) * p.K + ((dchunk ^ ((r >> 1) & 7)) * 8);
  }
  const int nk = p.K / kBK, total = nk * p.nseg;
  // product terms, the smallest first: hi lo, lo hi, hi hi
  auto issue = [&](int kt, int st) {
    const int seg = kt / nk, kk = kt - seg * nk;
    const int ta = p.nseg == 1 ? 0 : (seg == 1), tb = p.nseg == 1 ? 0 : (seg == 0);
    const uint16_t* a = A + ta * p.term_a + (int64_t)kk * kBK;
    const uint16_t* b = B + tb * p.term_b + (int64_t)kk * kBK;
    char* dst = lds + st * STAGE;
#pragma unroll
    for (int j = 0; j < LOADS_A; ++j)
      __builtin_amdgcn_global_load_lds((const void*)(a + oa[j]),
                                       (__attribute__((address_space(3))) void*)(dst + (wave * LOADS_A + j) * 1024), 16, 0, 0);
#pragma unroll
    for (int j = 0; j < LOADS_B; ++j)
      __builtin_amdgcn_global_load_lds(
          (const void*)(b + ob[j]), (__attribute__((address_space(3))) void*)(dst + BM * 128 + (wave * LOADS_B + j) * 1024),
          16, 0, 0);
  };
  f32x16 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  uint32_t sw[4];  // chunk 2s + h of this lane's row, swizzled
#pragma unroll
  for (int s = 0; s < 4; ++s) sw[s] = (uint32_t)l32 * 128 + (((2 * s + h) ^ ((l32 >> 1) & 7)) * 16);
  const uint32_t fa = wm * (BM / WM) * 128, fb = BM * 128 + wn * (BN / WN) * 128;
#pragma unroll
  for (int kt = 0; kt < S - 1; ++kt)
    if (kt < total) issue(kt, kt);
  for (int kt0 = 0; kt0 < total; kt0 += S) {
#pragma unroll
    for (int st = 0; st < S; ++st) {
      const int kt = kt0 + st;
      if (kt >= total) break;
      // wait for stage kt; up to S - 2 later ones stay in flight
      const int ahead = min(total - 1 - kt, S - 2);
      constexpr int PER = LOADS_A + LOADS_B;
      if (S > 2 && ahead == S - 2)
        __builtin_amdgcn_s_waitcnt((((S - 2) * PER) & 15) | (7 << 4) | (15 << 8) | ((((S - 2) * PER) >> 4) << 14));
      else
        __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();  // every wave's loads of stage kt have landed, stage kt - 1 is consumed
      asm volatile("" ::: "memory");
      if (kt + S - 1 < total) issue(kt + S - 1, (st + S - 1) % S);
      const char* stage = lds + st * STAGE;
      f16x8 af[2][MB], bf[2][NB];
      auto read = [&](int s) {
#pragma unroll
        for (int i = 0; i < MB; ++i) af[s & 1][i] = *reinterpret_cast<const f16x8*>(stage + fa + i * 32 * 128 + sw[s]);
#pragma unroll
        for (int j = 0; j < NB; ++j) bf[s & 1][j] = *reinterpret_cast<const f16x8*>(stage + fb + j * 32 * 128 + sw[s]);
      };
      read(0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        __builtin_amdgcn_sched_barrier(0);
        if (s < 3) read(s + 1);
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af[s & 1][i], bf[s & 1][j], acc[i][j], 0, 0, 0);
        // one matrix instruction, then a share of the next step's fragment reads
#pragma unroll
        for (int i = 0; i < MB * NB; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (s < 3 && i < MB + NB) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // lane l, register 4a + c of a block: row 8a + 4(l / 32) + c, column l % 32
  uint16_t* out = p.out16 + bi * p.terms * p.term_o;
  uint16_t* outt = p.outt16 + bi * p.terms * p.term_t;
  const uint16_t* aux = p.aux16 + bi * p.terms * p.term_o;
  const bool mirror = (MODE == kGram || MODE == kPoly) && p.sym && tm != tn;
  const float bad = MODE == kLast ? p.bad[bi] : 0.0f;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int mr = m0 + wm * (BM / WM) + i * 32 + 4 * h;
    // what the block row reads, ahead of its stores (the compiler keeps their
    // order: one load at a time cost 70 us a round of tiles); elements past the
    // matrix repeat its last
    float x[NB][16];
    if constexpr (MODE != kGram) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int n = min(n0 + wn * (BN / WN) + j * 32 + l32, p.N - 1);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = min(mr + 8 * (r / 4) + r % 4, p.M - 1);
          if constexpr (MODE == kPoly) {
            x[j][r] = (float)__builtin_bit_cast(_Float16, aux[(int64_t)m * p.ldo + n]);
            if (p.terms > 1) x[j][r] += (float)__builtin_bit_cast(_Float16, aux[(int64_t)m * p.ldo + n + p.term_o]);
          } else {
            x[j][r] = p.xf[(bi * p.M + m) * (int64_t)p.N + n];
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = n0 + wn * (BN / WN) + j * 32 + l32;
      if (n >= p.N) continue;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int mb = mr + 8 * a;
        uint16_t hi[4], lo[4];
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[c] = acc[i][j][4 * a + c] * p.s_acc;
          if constexpr (MODE != kGram) v[c] = fmaf(p.s_aux, x[j][4 * a + c], v[c]);
          if constexpr (MODE != kLast) split_half(MODE == kStep ? v[c] * kScaleX : v[c], p.terms, hi[c], lo[c]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int m = mb + c;
          if (m >= p.M) continue;
          if constexpr (MODE == kStep) p.xf[(bi * p.M + m) * (int64_t)p.N + n] = v[c];
          if constexpr (MODE == kLast) {
            store1(p.y, p.y_bf16, bi * p.M * (int64_t)p.N + (p.y_t ? (int64_t)n * p.M + m : (int64_t)m * p.N + n), v[c] + bad);
          } else {
            const int64_t at = (int64_t)m * p.ldo + n;
            out[at] = hi[c];
            if (p.terms > 1) out[at + p.term_o] = lo[c];
          }
        }
        if constexpr (MODE != kLast) {
          if ((MODE == kStep || mirror) && mb < p.M) {
            uint16_t* d = (MODE == kStep ? outt : out) + (int64_t)n * (MODE == kStep ? p.ldt : p.ldo) + mb;
            const int64_t term = MODE == kStep ? p.term_t : p.term_o;
            if (mb + 4 <= p.M) {
              *reinterpret_cast<u16x4*>(d) = u16x4{hi[0], hi[1], hi[2], hi[3]};
              if (p.terms > 1) *reinterpret_cast<u16x4*>(d + term) = u16x4{lo[0], lo[1], lo[2], lo[3]};
            } else {
              for (int c = 0; c < p.M - mb; ++c) {
                d[c] = hi[c];
                if (p.terms > 1) d[term + c] = lo[c];
              }
            }
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host side

struct OrthoLayout {
  bool small;
  int p, P, pp, qp, terms, spans;
  int64_t q, span;
  size_t off_g, off_q, off_part, off_bad, off_xf, off_x16, off_xt[2], off_g16, off_b16, bytes;
};

OrthoLayout ortho_layout(int64_t batch, int64_t rows, int64_t cols, nq_dtype yd) {
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
    L.spans = (int)imax(1, imin(imin(cdiv(512, batch), cdiv(L.q, 512)), 64));
    L.span = round_up(cdiv(L.q, L.spans), 128);
    L.spans = (int)cdiv(L.q, L.span);
    L.off_g = take((size_t)batch * L.spans * L.P * L.P * sizeof(double));
    L.off_q = take((size_t)batch * L.P * L.P * sizeof(double));
  } else {
    L.terms = yd == NQ_F32 ? 2 : 1;
    L.pp = (int)round_up(L.p, kBK);
    L.qp = (int)round_up(L.q, kBK);
    L.off_part = take((size_t)batch * kSumBlocks * sizeof(double));
    L.off_bad = take((size_t)batch * sizeof(float));
    L.off_xf = take((size_t)batch * L.p * L.q * sizeof(float));
    L.off_x16 = take((size_t)batch * L.terms * L.p * L.qp * 2);
    for (auto& o : L.off_xt) o = take((size_t)batch * L.terms * L.q * L.pp * 2);
    L.off_g16 = take((size_t)batch * L.terms * L.p * L.pp * 2);
    L.off_b16 = take((size_t)batch * L.terms * L.p * L.pp * 2);
  }
  L.bytes = off;
  return L;
}

template <typename E, int PT>
hipError_t launch_small(const SmallArgs& a, int64_t batch, hipStream_t s) {
  constexpr int P = 16 * PT, S = P + 4;
  hipLaunchKernelGGL((ortho_gram_kernel<E, PT>), dim3((unsigned)a.spans, (unsigned)batch), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  static std::atomic<uint64_t> done{0};
  if (e == hipSuccess)
    e = allow_lds(reinterpret_cast<const void*>(ortho_solve_kernel<PT>), 3 * P * S * sizeof(double), done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((ortho_solve_kernel<PT>), dim3((unsigned)batch), dim3(256), 3 * P * S * sizeof(double), s, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((ortho_apply_kernel<E, PT>), dim3((unsigned)cdiv(a.q, 256), (unsigned)batch), dim3(256),
                     P * S * sizeof(double), s, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_small_p(const SmallArgs& a, int64_t batch, hipStream_t s) {
  switch (cdiv(a.p, 16)) {
    case 1: return launch_small<E, 1>(a, batch, s);
    case 2: return launch_small<E, 2>(a, batch, s);
    case 3: return launch_small<E, 3>(a, batch, s);
    default: return launch_small<E, 4>(a, batch, s);
  }
}

template <int BM, int BN, int WM, int WN, int S, int MODE>
hipError_t launch_gemm_tile(GemmArgs g, int64_t batch, hipStream_t s) {
  constexpr size_t lds = (size_t)S * (BM + BN) * 128;
  const auto kernel = ortho_gemm_kernel<BM, BN, WM, WN, S, MODE>;
  static std::atomic<uint64_t> done{0};
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), lds, done);
  if (e != hipSuccess) return e;
  g.tiles_m = (int)cdiv(g.M, BM);
  g.tiles_n = (int)cdiv(g.N, BN);
  const int64_t tiles = g.sym ? (int64_t)g.tiles_m * (g.tiles_m + 1) / 2 : (int64_t)g.tiles_m * g.tiles_n;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(8 * cdiv(tiles, 8)), (unsigned)batch), dim3(64 * WM * WN), lds, s, g);
  return hipGetLastError();
}

template <int MODE>
hipError_t launch_ortho_gemm(GemmArgs g, int64_t batch, hipStream_t s) {
  constexpr bool square = MODE == kGram || MODE == kPoly;
  // 256 x 256 tiles (one workgroup per CU) once they fill the chip; symmetric
  // results skip the tiles above the diagonal where that saves whole rounds
  const int64_t t256 = cdiv(g.M, 256), big = t256 * cdiv(g.N, 256) * batch;
  if (big >= 192) {
    const int64_t half = t256 * (t256 + 1) / 2 * batch;
    g.sym = square && cdiv(half, 256) < cdiv(big, 256);
    return launch_gemm_tile<256, 256, 2, 4, 2, MODE>(g, batch, s);
  }
  g.sym = square;
  return launch_gemm_tile<128, 128, 2, 2, 2, MODE>(g, batch, s);
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

}  // namespace

size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols, nq_dtype yd) {
  return ortho_layout(batch, rows, cols, yd).bytes;
}

hipError_t launch_ortho(const void* x, nq_dtype xd, int64_t batch, int64_t rows, int64_t cols, int64_t ldx,
                        int64_t stride_x, int steps, double ca, double cb, double cc, void* y, nq_dtype yd, void* workspace,
                        hipStream_t s) {
  const OrthoLayout L = ortho_layout(batch, rows, cols, yd);
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
    a.steps = steps;
    a.a = ca;
    a.b = cb;
    a.c = cc;
    return xd == NQ_BF16 ? launch_small_p<uint16_t>(a, batch, s) : launch_small_p<float>(a, batch, s);
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
  for (int i = 0; i < 2; ++i) l.xt16[i] = reinterpret_cast<uint16_t*>(ws + L.off_xt[i]);
  l.g16 = reinterpret_cast<uint16_t*>(ws + L.off_g16);
  l.b16 = reinterpret_cast<uint16_t*>(ws + L.off_b16);
  l.part = part;
  l.bad = reinterpret_cast<float*>(ws + L.off_bad);
  // |x| <= 1.25, |G| <= 1.25^2 and the polynomial's bound, each times its scale
  // below 65504
  const float sx = kScaleX, sg = 16384.0f;
  l.sx = sx;
  const double bound = poly_bound(cb, cc, 1.25 * 1.25);
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
  gram.out16 = l.g16;
  gram.ldo = L.pp;
  gram.term_o = gs;
  gram.s_acc = sg / (sx * sx);
  poly = gram;
  poly.A = poly.B = l.g16;
  poly.stride_a = poly.stride_b = L.terms * gs;
  poly.term_a = poly.term_b = gs;
  poly.K = L.pp;
  poly.out16 = l.b16;
  poly.aux16 = l.g16;
  poly.s_acc = (float)(cc * sb / ((double)sg * sg));
  poly.s_aux = (float)(cb * sb / sg);
  step.A = l.b16;
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
    step.B = l.xt16[i % 2];
    step.outt16 = l.xt16[1 - i % 2];
    e = i + 1 < steps ? launch_ortho_gemm<kStep>(step, batch, s) : launch_ortho_gemm<kLast>(step, batch, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nq
