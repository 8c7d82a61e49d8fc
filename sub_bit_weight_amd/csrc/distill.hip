// Distillation from a teacher's top logits: the objective of scale-only reconstruction
// (research.samsung.com NanoQuant blog, section 3, "Phase 3: Scale-Only Model Reconstruction": the
// KL divergence of the quantized model's outputs from the full-precision model's) with the teacher
// kept as its k most likely tokens per position and the mass of the others.
//
// Per row, with q = softmax(s / tau) and K the listed tokens:
//   lse_K, lse_R   log-sum-exps of s / tau over the listed tokens and over the rest,
//   lse = log(exp(lse_K) + exp(lse_R)),  log q_v = s_v / tau - lse,  log q_rest = lse_R - lse,
//   loss = sum_e p_e (log p_e - log q_e) + r (log r - log q_rest),
//   dloss/ds_v = ((P + r) q_v - sum_{e: id_e = v} p_e) / tau                       v listed,
//              = exp(s_v / tau - lse_R) ((P + r) exp(lse_R - lse) - r) / tau        otherwise.
// The rest has a maximum and a sum of its own, so that neither its mass nor its gradient is the
// difference of two larger numbers.  One workgroup per row.
#include "nq_internal.h"

namespace nq {
namespace {

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.4426950408889634;

__device__ inline float row_load(const void* p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}
__device__ inline void row_store(void* p, bool bf16, int64_t i, float v) {
  if (bf16)
    static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    static_cast<float*>(p)[i] = v;
}

// exp(d / tau) for d <= 0 as 2^(d c), c = log2(e) / tau in two parts: one part's rounding
// would grow with |d|.  Both parts are above zero, so that d = -inf gives 0.
struct ExpScale {
  float hi, lo;
};
__device__ inline float exp_scaled(float d, ExpScale c) { return exp2f(fmaf(d, c.hi, d * c.lo)); }
ExpScale exp_scale(float tau) {
  const double c = kLog2e / (double)tau;
  float hi = (float)c;
  if ((double)hi > c) hi = nextafterf(hi, 0.0f);
  return {hi, fmaxf((float)(c - (double)hi), __FLT_MIN__)};
}

// Workgroup reductions in a fixed order; `red` holds one double per wave and is free again after
// the second barrier of the next use.
template <int NT>
__device__ inline float wg_max(float x, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = (double)x;
  __syncthreads();
  x = (float)red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) x = fmaxf(x, (float)red[w]);
  return x;
}
template <int NT>
__device__ inline double wg_sum(double x, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) x += red[w];
  return x;
}

// A running maximum and the sum of exponentials below it.
struct MaxSum {
  float m = -kInf, s = 0.0f;
  __device__ inline void add(float x, ExpScale c) {
    if (x > m) {
      s *= exp_scaled(m == -kInf ? -kInf : m - x, c);
      m = x;
    }
    s += exp_scaled(x - (m == -kInf ? 0.0f : m), c);  // -inf adds 0, NaN stays
  }
};

// ------------------------------------------------------------------ the divergence and its gradient

constexpr int kDistillThreads = 512;
constexpr int kEntries = (NQ_TOP_MAX + kDistillThreads - 1) / kDistillThreads;  // per thread

struct RowConsts {  // of one row, for every thread
  double base, lse, total, scale;
  float ref, coef;
  int zero;
};

// LDS: [bitmap of the listed tokens, V bits][ids][logits][probabilities of the k entries].
// An entry's id is -1 where there is none, and -2 - id for a repetition of an earlier entry.
template <bool GRADS>
__global__ __launch_bounds__(kDistillThreads) void distill_kernel(const nq_teacher P, ExpScale c, const void* logits,
                                                                  int bf16, int V, int64_t ld,
                                                                  const float* __restrict__ weight,
                                                                  float* __restrict__ loss, void* dlogits, int d_bf16,
                                                                  int64_t ldd) {
  constexpr int NT = kDistillThreads;
  extern __shared__ uint32_t lds[];
  __shared__ double red[NT / 64];
  __shared__ RowConsts row;
  __shared__ int s_bad, s_dup;
  const int tid = threadIdx.x, k = (int)P.k, nw = (V + 31) / 32;
  uint32_t* listed = lds;
  int* ids = reinterpret_cast<int*>(lds + nw);
  float* sv = reinterpret_cast<float*>(ids + k);
  float* ps = sv + k;
  const int64_t t = blockIdx.x;
  const char* x = static_cast<const char*>(logits) + t * ld * (bf16 ? 2 : 4);
  char* dx = GRADS ? static_cast<char*>(dlogits) + t * ldd * (d_bf16 ? 2 : 4) : nullptr;
  const float w = weight ? weight[t] : 1.0f;
  auto constant_row = [&](float v) {
    if (tid == 0 && loss) loss[t] = v;
    if (GRADS)
      for (int i = tid; i < V; i += NT) row_store(dx, d_bf16, i, v);
  };
  if (w == 0.0f) return constant_row(0.0f);

  if (tid == 0) s_bad = s_dup = 0;
  for (int i = tid; i < nw; i += NT) listed[i] = 0;
  __syncthreads();
  const int32_t* gid = P.ids + t * k;
  const float* glp = P.logp + t * k;
  for (int e = tid; e < k; e += NT) {
    const int id = gid[e];
    float s = -kInf, p = 0.0f;
    if (id >= V) {
      s_bad = 1;
    } else if (id >= 0) {
      if (atomicOr(&listed[id / 32], 1u << (id % 32)) >> (id % 32) & 1u) s_dup = 1;
      s = row_load(x, bf16, id);
      p = expf(glp[e]);
    }
    ids[e] = id < 0 ? -1 : id;
    sv[e] = s;
    ps[e] = p;
  }
  __syncthreads();
  if (s_bad) return constant_row(__builtin_nanf(""));
  if (s_dup) {  // the first of equal entries takes the probabilities of all
    float sum[kEntries];
    bool again[kEntries];
    for (int i = 0, e = tid; i < kEntries; ++i, e += NT) {
      sum[i] = 0.0f;
      again[i] = false;
      if (e >= k || ids[e] < 0) continue;
      for (int f = 0; f < k; ++f)
        if (ids[f] == ids[e]) {
          again[i] |= f < e;
          sum[i] += ps[f];
        }
    }
    __syncthreads();
    for (int i = 0, e = tid; i < kEntries; ++i, e += NT)
      if (e < k && ids[e] >= 0) {
        ps[e] = sum[i];
        if (again[i]) ids[e] = -2 - ids[e];
      }
    __syncthreads();
  }

  MaxSum rest;
  for (int i = tid; i < V; i += NT)
    if (!(listed[i / 32] >> (i % 32) & 1u)) rest.add(row_load(x, bf16, i), c);
  const float m_r = wg_max<NT>(rest.m, red);
  const float ref = m_r == -kInf ? 0.0f : m_r;
  const double s_r = wg_sum<NT>((double)rest.s * (double)exp_scaled(rest.m == -kInf ? 0.0f : rest.m - ref, c), red);

  float m_k = -kInf;
  for (int e = tid; e < k; e += NT)
    if (ids[e] != -1) m_k = fmaxf(m_k, sv[e]);
  m_k = wg_max<NT>(m_k, red);
  // everything relative to the row's largest logit, at which an fp64 number of its own size may not
  // hold the logarithms
  const float top = fmaxf(m_r, m_k);
  const double base = top == -kInf ? 0.0 : (double)top, rtau = 1.0 / (double)P.temperature;
  double s_k = 0.0, mass = 0.0, cross = 0.0;  // sum p, sum p (log p - s / tau)
  for (int e = tid; e < k; e += NT) {
    if (ids[e] == -1) continue;
    const double sx = ((double)sv[e] - base) * rtau;
    if (ids[e] >= 0) s_k += exp(sx);
    const double lp = glp[e], p = exp(lp);
    if (p == 0.0) continue;
    mass += p;
    cross += p * (lp - sx);
  }
  s_k = wg_sum<NT>(s_k, red);
  mass = wg_sum<NT>(mass, red);
  cross = wg_sum<NT>(cross, red);

  if (tid == 0) {
    const double ref_r = ((double)ref - base) * rtau, lse_r = ref_r + log(s_r);
    const double lse = log(s_k + s_r * exp(ref_r));
    const double lr = P.rest ? (double)P.rest[t] : -(double)kInf, r = exp(lr);
    const double total = P.rest ? mass + r : 1.0;
    RowConsts R;
    R.zero = P.rest ? total == 0.0 : mass == 0.0;
    double L = P.rest ? cross + mass * lse : cross / mass - log(mass) + lse;
    if (P.rest && r != 0.0) L += r * (lr - (lse_r - lse));
    if (loss) loss[t] = R.zero ? 0.0f : (float)((double)w * L);
    R.base = base;
    R.lse = lse;
    R.total = total;
    R.scale = P.rest ? 1.0 : 1.0 / mass;  // of the listed probabilities
    R.ref = ref;
    // the gradient of a token not listed is coef * exp((s - ref) / tau)
    double coef = total * exp(ref_r - lse);
    if (r != 0.0) coef -= r / s_r;
    R.coef = s_r == 0.0 && lse > -(double)kInf ? 0.0f : (float)((double)w * rtau * coef);
    row = R;
  }
  if (!GRADS) return;
  __syncthreads();
  const RowConsts R = row;
  if (R.zero) {
    for (int i = tid; i < V; i += NT) row_store(dx, d_bf16, i, 0.0f);
    return;
  }
  for (int i = tid; i < V; i += NT)
    if (!(listed[i / 32] >> (i % 32) & 1u))
      row_store(dx, d_bf16, i, R.coef * exp_scaled(row_load(x, bf16, i) - R.ref, c));
  for (int e = tid; e < k; e += NT)
    if (ids[e] >= 0) {
      const double q = exp(((double)sv[e] - R.base) * rtau - R.lse);
      row_store(dx, d_bf16, ids[e], (float)((double)w * rtau * (R.total * q - R.scale * (double)ps[e])));
    }
}

// ------------------------------------------------------------------ a teacher's top logits

// Keys in the order of the logits: -0 equals +0, NaN lies above +inf.
__device__ inline uint32_t logit_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kFirstKey = 0x00800000u;  // the lowest above -inf's

constexpr int kTopThreads = 1024;
constexpr int kCandidates = 2 * NQ_TOP_MAX;

template <int NT>
__device__ inline int wg_count(int n, int* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) n += red[w];
  return n;
}

// The k-th largest of the threads' maxima is a lower bound of the k-th largest logit, and nearly
// equal to it where the largest are spread over the row: the logits from it on (candidates) are few
// more than k and go to LDS, where each one's place is the number of candidates before it.  A row
// whose candidates are too many (long runs of equal logits, or the largest in few threads'
// elements) finds the k-th logit by its bits instead.
__global__ __launch_bounds__(kTopThreads) void logits_top_kernel(const void* __restrict__ logits, int bf16, int V,
                                                                 int64_t ld, int k, double rtau, ExpScale c,
                                                                 int32_t* __restrict__ ids, float* __restrict__ logp,
                                                                 float* __restrict__ rest_out) {
  constexpr int NT = kTopThreads;
  __shared__ uint32_t ckey[kCandidates];  // the threads' maxima at first
  __shared__ int cidx[kCandidates];
  __shared__ float top_z[NQ_TOP_MAX];
  __shared__ int top_i[NQ_TOP_MAX];
  __shared__ double red[NT / 64];
  __shared__ int s_n, s_last_i;
  __shared__ uint32_t s_last_key;
  int* ired = reinterpret_cast<int*>(red);
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  const char* x = static_cast<const char*>(logits) + t * ld * (bf16 ? 2 : 4);

  uint32_t mine = 0;
  for (int i = tid; i < V; i += NT) mine = max(mine, logit_key(row_load(x, bf16, i)));
  ckey[tid] = mine;
  if (tid == 0) {
    s_n = 0;
    s_last_key = kFirstKey - 1;  // everything finite is listed
    s_last_i = 0x7fffffff;
  }
  __syncthreads();
  uint32_t bound = 0;
  if (tid < 64) {  // one wave: the largest value that at least k of the maxima reach
    uint32_t v[NT / 64];
#pragma unroll
    for (int j = 0; j < NT / 64; ++j) v[j] = ckey[tid + 64 * j];
    for (int b = 31; b >= 0; --b) {
      const uint32_t at = bound | 1u << b;
      int n = 0;
#pragma unroll
      for (int j = 0; j < NT / 64; ++j) n += __popcll(__ballot(v[j] >= at));
      if (n >= k) bound = at;
    }
    if (tid == 0) s_last_i = (int)max(bound, kFirstKey);
  }
  __syncthreads();
  bound = (uint32_t)s_last_i;
  __syncthreads();
  if (tid == 0) s_last_i = 0x7fffffff;
  int last_i = 0x7fffffff;  // candidates equal to the bound: indices up to this
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = tid; i < V; i += NT) {
      const uint32_t key = logit_key(row_load(x, bf16, i));
      if (key > bound || (key == bound && i <= last_i)) {
        const int n = atomicAdd(&s_n, 1);
        if (n < kCandidates) {
          ckey[n] = key;
          cidx[n] = i;
        }
      }
    }
    __syncthreads();
    if (s_n <= kCandidates) break;
    // too many: the k-th largest key bit by bit (at least k keys reach the bound), then the last
    // of the equal ones by index; exactly k candidates are left
    uint32_t at = 0;
    for (int b = 31; b >= 0; --b) {
      const uint32_t key = at | 1u << b;
      int n = 0;
      for (int i = tid; i < V; i += NT) n += logit_key(row_load(x, bf16, i)) >= key;
      if (wg_count<NT>(n, ired) >= k) at = key;
    }
    int above = 0;
    for (int i = tid; i < V; i += NT) above += logit_key(row_load(x, bf16, i)) > at;
    const int need = k - wg_count<NT>(above, ired);
    int lo = 0, hi = V - 1;  // the smallest index up to which `need` keys equal the bound
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      int n = 0;
      for (int i = tid; i <= mid; i += NT) n += logit_key(row_load(x, bf16, i)) == at;
      if (wg_count<NT>(n, ired) >= need)
        hi = mid;
      else
        lo = mid + 1;
    }
    bound = at;
    last_i = lo;
    __syncthreads();
    if (tid == 0) s_n = 0;
    __syncthreads();
  }
  const int n = s_n;
  for (int e = tid; e < n; e += NT) {
    const uint32_t key = ckey[e];
    const int idx = cidx[e];
    int place = 0;
    for (int f = 0; f < n; ++f) place += ckey[f] > key || (ckey[f] == key && cidx[f] < idx);
    if (place < k) {
      top_z[place] = row_load(x, bf16, idx);
      top_i[place] = idx;
      if (place == k - 1) {
        s_last_key = key;
        s_last_i = idx;
      }
    }
  }
  __syncthreads();
  const int m = min(n, k);  // listed
  const uint32_t lkey = s_last_key;
  const int li = s_last_i;
  MaxSum rest;
  for (int i = tid; i < V; i += NT) {
    const float v = row_load(x, bf16, i);
    const uint32_t key = logit_key(v);
    if (key < lkey || (key == lkey && i > li)) rest.add(v, c);
  }
  const float m_r = wg_max<NT>(rest.m, red);
  const float ref = m_r == -kInf ? 0.0f : m_r;
  const double s_r = wg_sum<NT>((double)rest.s * (double)exp_scaled(rest.m == -kInf ? 0.0f : rest.m - ref, c), red);
  const double ref_k = m > 0 ? (double)top_z[0] : 0.0;
  double s_k = 0.0;
  for (int e = tid; e < m; e += NT) s_k += exp(((double)top_z[e] - ref_k) * rtau);
  s_k = wg_sum<NT>(s_k, red);
  // relative to ref_k / tau; an empty row has nothing listed and rest -inf
  const double lse = log(s_k + s_r * exp(((double)ref - ref_k) * rtau));
  for (int e = tid; e < k; e += NT) {
    ids[t * k + e] = e < m ? top_i[e] : -1;
    logp[t * k + e] = e < m ? (float)(((double)top_z[e] - ref_k) * rtau - lse) : -kInf;
  }
  if (tid == 0 && rest_out) rest_out[t] = s_r == 0.0 && lse == lse ? -kInf : (float)(((double)ref - ref_k) * rtau + log(s_r) - lse);
}

}  // namespace

hipError_t launch_logits_top(const void* logits, nq_dtype dt, int64_t T, int64_t V, int64_t ld, int k, float temperature,
                             int32_t* ids, float* logp, float* rest, hipStream_t s) {
  hipLaunchKernelGGL(logits_top_kernel, dim3((unsigned)T), dim3(kTopThreads), 0, s, logits, (int)(dt == NQ_BF16), (int)V,
                     ld, k, 1.0 / (double)temperature, exp_scale(temperature), ids, logp, rest);
  return hipGetLastError();
}

hipError_t launch_distill(const nq_teacher& P, const void* logits, nq_dtype dt, int64_t T, int64_t V, int64_t ld,
                          const float* weight, float* loss, void* dlogits, nq_dtype dd, int64_t ldd, hipStream_t s) {
  const size_t lds = (size_t)cdiv(V, 32) * 4 + (size_t)P.k * 12;
  static std::atomic<uint64_t> done[2];
  const bool grads = dlogits != nullptr;
  const void* kernel = grads ? reinterpret_cast<const void*>(distill_kernel<true>)
                             : reinterpret_cast<const void*>(distill_kernel<false>);
  // the largest call: 2^20 tokens and NQ_TOP_MAX entries
  const hipError_t e = allow_lds(kernel, (size_t)(1 << 15) * 4 + (size_t)NQ_TOP_MAX * 12, done[grads]);
  if (e != hipSuccess) return e;
  if (grads)
    hipLaunchKernelGGL(distill_kernel<true>, dim3((unsigned)T), dim3(kDistillThreads), lds, s, P, exp_scale(P.temperature),
                       logits, (int)(dt == NQ_BF16), (int)V, ld, weight, loss, dlogits, (int)(dd == NQ_BF16), ldd);
  else
    hipLaunchKernelGGL(distill_kernel<false>, dim3((unsigned)T), dim3(kDistillThreads), lds, s, P, exp_scale(P.temperature),
                       logits, (int)(dt == NQ_BF16), (int)V, ld, weight, loss, dlogits, 0, ldd);
  return hipGetLastError();
}

}  // namespace nq
