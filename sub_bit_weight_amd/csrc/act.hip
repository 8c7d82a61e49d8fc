// Epilogue of a packed linear and its gradients.
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

__global__ __launch_bounds__(256) void epilogue_kernel(const float* __restrict__ v, int64_t n, int64_t d,
                                                       const Epilogue E) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    epilogue_store(E, i, i % d, v[i]);
}

struct ActGrads {
  const void *z, *mul, *dy;
  void *dz, *dmul;
  int act, z_bf16, mul_bf16, dy_bf16, dz_bf16, dmul_bf16;
};

// One thread per column walks a chunk of tc tokens; the chunk's sum of dz goes to sums[chunk][d].
__global__ __launch_bounds__(256) void act_grads_kernel(const ActGrads G, int64_t T, int64_t tc, int64_t d,
                                                        float* __restrict__ sums) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  const int64_t t0 = (int64_t)blockIdx.y * tc, t1 = imin(t0 + tc, T);
  float acc = 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t i = t * d + c;
    const float dy = epi_load(G.dy, G.dy_bf16, i);
    float a = 0.0f, da = 1.0f;
    if (G.z) act_value_grad(G.act, epi_load(G.z, G.z_bf16, i), a, da);
    float dz = dy * da;
    if (G.mul) dz *= epi_load(G.mul, G.mul_bf16, i);
    if (G.dmul) epi_store(G.dmul, G.dmul_bf16, i, dy * a);
    epi_store(G.dz, G.dz_bf16, i, dz);
    acc += dz;
  }
  if (sums) sums[(int64_t)blockIdx.y * d + c] = acc;
}

__global__ __launch_bounds__(256) void chunk_sums_kernel(const float* __restrict__ sums, int64_t n, int64_t d,
                                                         float* __restrict__ out) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float acc = 0.0f;
  for (int64_t q = 0; q < n; ++q) acc += sums[q * d + c];
  out[c] = acc;
}

// Tokens of a chunk: 64, more when T has more than 1024 such chunks.
int64_t chunk_tokens(int64_t T) { return imax(64, cdiv(T, 1024)); }

}  // namespace

hipError_t launch_epilogue(const float* v, int64_t T, int64_t d, const Epilogue& E, hipStream_t s) {
  const int64_t n = T * d;
  hipLaunchKernelGGL(epilogue_kernel, dim3((unsigned)imin(cdiv(n, 256), 8192)), dim3(256), 0, s, v, n, d, E);
  return hipGetLastError();
}

size_t act_grads_workspace(int64_t T, int64_t d) {
  const int64_t n = cdiv(T, chunk_tokens(T));
  return n > 1 ? (size_t)n * d * sizeof(float) : 0;
}

hipError_t launch_act_grads(int act, const void* z, nq_dtype zd, const void* mul, nq_dtype md, const void* dy,
                            nq_dtype dyd, int64_t T, int64_t d, void* dz, nq_dtype dzd, void* dmul, nq_dtype dmd,
                            float* dbias, void* ws, hipStream_t s) {
  const ActGrads G{z,   mul,           dy,            dz,             dmul,           act,
                   zd == NQ_BF16, md == NQ_BF16, dyd == NQ_BF16, dzd == NQ_BF16, dmd == NQ_BF16};
  const int64_t tc = chunk_tokens(T), n = cdiv(T, tc);
  float* sums = !dbias ? nullptr : n > 1 ? static_cast<float*>(ws) : dbias;
  hipLaunchKernelGGL(act_grads_kernel, dim3((unsigned)cdiv(d, 256), (unsigned)n), dim3(256), 0, s, G, T, tc, d, sums);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dbias || n == 1) return e;
  hipLaunchKernelGGL(chunk_sums_kernel, dim3((unsigned)cdiv(d, 256)), dim3(256), 0, s, sums, n, d, dbias);
  return hipGetLastError();
}

}  // namespace nq
