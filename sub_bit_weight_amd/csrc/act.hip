// Gradients of a packed linear's epilogue.
//
// The layer y = s1 (.) U (V^T (s2 (.) x)) (research.samsung.com NanoQuant blog, section 2 "Low-Rank
// Binary Factorization") stands in a block between a bias, an activation, a gate and a residual:
//     z = W x + bias,   y = act(z) (.) mul + residual.
// Its gradients for dy = dL/dy:
//     dz = dy (.) mul (.) act'(z),   dmul = dy (.) act(z),   dbias = sum_t dz,   dresidual = dy,
// and dz is the output gradient that the scale gradients take.
#include "epilogue.h"

namespace nq {
namespace {

struct ActGrads {
  const void *z, *mul, *dy;
  void *dz, *dmul;
  int z_bf16, mul_bf16, dy_bf16, dz_bf16, dmul_bf16;
};

// One element's gradients.
template <int ACT>
__device__ inline void element_grads(float z, float mul, float dy, float& dz, float& dmul) {
  float a, da;
  act_value_grad<ACT>(z, a, da);
  dz = dy * da * mul;
  dmul = dy * a;
}

// A workgroup takes kCols pieces of N columns and tc tokens; each of its kRows rows of threads walks every
// kRows-th token, and the rows' sums of dz are added in order, in fp64, through LDS into sums[chunk][d].  The d % N
// columns past the last whole piece are pieces of one column (all of them one thread's took longer than
// everything else: 256 x 1117 bf16, gelu, 30 us, 17.8 so).  Bound by the loads and stores where the chip is
// full (2048 x 28672 bf16, silu and gate: 119 us, 4.9 TB/s), else by the chain of a thread's tokens.
constexpr int kCols = 16;
template <int ACT, int N, int kRows>
__global__ __launch_bounds__(kCols* kRows) void act_grads_kernel(const ActGrads G, int64_t T, int64_t tc, int64_t d,
                                                                 float* __restrict__ sums) {
  __shared__ float part[kRows][kCols * N];
  const int col = threadIdx.x % kCols, row = threadIdx.x / kCols;
  const int64_t np = d / N, first = (int64_t)blockIdx.x * kCols;
  const bool whole = first + col < np;
  const int64_t c0 = whole ? (first + col) * N : np * N + (first + col - np);
  const int64_t t0 = (int64_t)blockIdx.y * tc, t1 = imin(t0 + tc, T);
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  if (whole) {
    // two tokens at a time, all their loads ahead of their stores (a result may be in place)
    constexpr int U = 2;
    for (int64_t t = t0 + row; t < t1; t += U * kRows) {
      Elements<N> z[U], mul[U], dy[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = imin(t + u * kRows, t1 - 1) * d + c0;
        dy[u].load(G.dy, G.dy_bf16, i);
        if (G.z) z[u].load(G.z, G.z_bf16, i);
        if (G.mul) mul[u].load(G.mul, G.mul_bf16, i);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u * kRows >= t1) break;
        const int64_t i = (t + u * kRows) * d + c0;
        Elements<N> dz, dmul;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          element_grads<ACT>(G.z ? z[u].v[j] : 0.0f, G.mul ? mul[u].v[j] : 1.0f, dy[u].v[j], dz.v[j], dmul.v[j]);
          acc[j] += dz.v[j];
        }
        dz.store(G.dz, G.dz_bf16, i);
        if (G.dmul) dmul.store(G.dmul, G.dmul_bf16, i);
      }
    }
  } else if (c0 < d) {
    constexpr int U = 4;
    for (int64_t t = t0 + row; t < t1; t += U * kRows) {
      float z[U], mul[U], dy[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = imin(t + u * kRows, t1 - 1) * d + c0;
        dy[u] = load_element(G.dy, G.dy_bf16, i);
        z[u] = G.z ? load_element(G.z, G.z_bf16, i) : 0.0f;
        mul[u] = G.mul ? load_element(G.mul, G.mul_bf16, i) : 1.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u * kRows >= t1) break;
        const int64_t i = (t + u * kRows) * d + c0;
        float dz, dmul;
        element_grads<ACT>(z[u], mul[u], dy[u], dz, dmul);
        acc[0] += dz;
        store_element(G.dz, G.dz_bf16, i, dz);
        if (G.dmul) store_element(G.dmul, G.dmul_bf16, i, dmul);
      }
    }
  }
  if (!sums) return;
#pragma unroll
  for (int j = 0; j < N; ++j) part[row][col * N + j] = acc[j];
  __syncthreads();
  for (int c = threadIdx.x; c < kCols * N; c += kCols * kRows) {
    const int64_t piece = first + c / N, at = piece < np ? piece * N + c % N : np * N + (piece - np);
    if (at >= d || (piece >= np && c % N)) continue;
    double s = part[0][c];
#pragma unroll
    for (int r = 1; r < kRows; ++r) s += part[r][c];
    sums[(int64_t)blockIdx.y * d + at] = (float)s;
  }
}

__global__ __launch_bounds__(256) void chunk_sums_kernel(const float* __restrict__ sums, int64_t n, int64_t d,
                                                         float* __restrict__ out) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  double acc = 0.0;
#pragma unroll 8
  for (int64_t q = 0; q < n; ++q) acc += sums[q * d + c];
  out[c] = (float)acc;
}

// Tokens of a chunk: all up to 256 (no second launch for their sums), else 128, more when T has more
// than 1024 such chunks.
int64_t chunk_tokens(int64_t T) { return T <= 256 ? T : imax(128, cdiv(T, 1024)); }

template <int N, int kRows>
void launch_act_grads_t(int act, const ActGrads& G, int64_t T, int64_t tc, int64_t d, float* sums, hipStream_t s) {
  const dim3 grid((unsigned)cdiv(d / N + d % N, kCols), (unsigned)cdiv(T, tc));
  const auto kernel = act == NQ_ACT_RELU        ? act_grads_kernel<NQ_ACT_RELU, N, kRows>
                      : act == NQ_ACT_GELU      ? act_grads_kernel<NQ_ACT_GELU, N, kRows>
                      : act == NQ_ACT_GELU_TANH ? act_grads_kernel<NQ_ACT_GELU_TANH, N, kRows>
                      : act == NQ_ACT_SILU      ? act_grads_kernel<NQ_ACT_SILU, N, kRows>
                                                : act_grads_kernel<NQ_ACT_NONE, N, kRows>;
  hipLaunchKernelGGL(kernel, grid, dim3(kCols * kRows), 0, s, G, T, tc, d, sums);
}
// Rows of threads: 16, or 64 where that leaves the chip (256 units) with few workgroups and a thread with
// many tokens (us with 16 / 64, gelu; bf16: 77 tokens of 4096 9.0 / 6.4, 256 of 11008, 86 workgroups,
// 24.0 / 15.8, 2048 of 4096, 512 workgroups, 22.2 / 23.7; fp32: 16 tokens of 1117 3.5 / 3.8, 2048 of 4096,
// 1024 workgroups, 22.0 / 25.6).
template <int N>
void launch_act_grads_n(int act, const ActGrads& G, int64_t T, int64_t tc, int64_t d, float* sums, hipStream_t s) {
  if (tc > 16 && cdiv(d, kCols * N) * cdiv(T, tc) < 512)
    launch_act_grads_t<N, 64>(act, G, T, tc, d, sums, s);
  else
    launch_act_grads_t<N, 16>(act, G, T, tc, d, sums, s);
}

}  // namespace

size_t act_grads_workspace(int64_t T, int64_t d) {
  const int64_t n = cdiv(T, chunk_tokens(T));
  return n > 1 ? (size_t)n * d * sizeof(float) : 0;
}

hipError_t launch_act_grads(int act, const void* z, nq_dtype zd, const void* mul, nq_dtype md, const void* dy,
                            nq_dtype dyd, int64_t T, int64_t d, void* dz, nq_dtype dzd, void* dmul, nq_dtype dmd,
                            float* dbias, void* ws, hipStream_t s) {
  const ActGrads G{z,   mul,           dy,            dz,             dmul,
                   zd == NQ_BF16, md == NQ_BF16, dyd == NQ_BF16, dzd == NQ_BF16, dmd == NQ_BF16};
  const int64_t tc = chunk_tokens(T), n = cdiv(T, tc);
  float* sums = !dbias ? nullptr : n > 1 ? static_cast<float*>(ws) : dbias;
  // pieces of 16 bytes of dy
  if (dyd == NQ_BF16)
    launch_act_grads_n<8>(act, G, T, tc, d, sums, s);
  else
    launch_act_grads_n<4>(act, G, T, tc, d, sums, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dbias || n == 1) return e;
  hipLaunchKernelGGL(chunk_sums_kernel, dim3((unsigned)cdiv(d, 256)), dim3(256), 0, s, sums, n, d, dbias);
  return hipGetLastError();
}

}  // namespace nq
