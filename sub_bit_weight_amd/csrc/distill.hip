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
#include "elements.h"
#include "nq_internal.h"

namespace nq {
namespace {

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.4426950408889634;

// exp(d / tau) for d <= 0, c = log2(e) / tau: the hardware's 2^x, one unit in the last place and 0 below
// 2^-126.  c's rounding and the product's are felt |d / tau| times each, as is the difference's.
__device__ inline float exp_scaled(float d, float c) { return __builtin_amdgcn_exp2f(d * c); }
float exp_scale(float tau) { return (float)(kLog2e / (double)tau); }

// The largest of three; a library maximum would quiet its operands first, an instruction each.
__device__ inline float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Reductions over a wave by lane moves within rows of 16 and four lane reads; over a workgroup's waves
// in a row of 16.
template <int CTRL>
__device__ inline float lane_move(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ inline double lane_move(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
__device__ inline float lane_read(float x, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), l));
}
__device__ inline double lane_read(double x, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l) << 32 |
                                        (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l));
}
__device__ inline float row_max(float x) {  // of 16 lanes, to all of them
  x = fmaxf(x, lane_move<kXor1>(x));
  x = fmaxf(x, lane_move<kXor2>(x));
  x = fmaxf(x, lane_move<kHalfMirror>(x));
  return fmaxf(x, lane_move<kMirror>(x));
}
__device__ inline double row_sum(double x) {
  x += lane_move<kXor1>(x);
  x += lane_move<kXor2>(x);
  x += lane_move<kHalfMirror>(x);
  return x + lane_move<kMirror>(x);
}
__device__ inline float wave_max(float x) {
  x = row_max(x);
  return fmaxf(fmaxf(lane_read(x, 0), lane_read(x, 16)), fmaxf(lane_read(x, 32), lane_read(x, 48)));
}
__device__ inline double wave_sum(double x) {
  x = row_sum(x);
  return (lane_read(x, 0) + lane_read(x, 16)) + (lane_read(x, 32) + lane_read(x, 48));
}

// A running maximum and the sum of exponentials below it.
struct MaxSum {
  float m = -kInf, s = 0.0f;
  __device__ inline void add(float x, float c) {
    if (x > m) {
      s *= exp_scaled(m == -kInf ? -kInf : m - x, c);
      m = x;
    }
    s += exp_scaled(x - (m == -kInf ? 0.0f : m), c);  // -inf adds 0, NaN stays
  }
};

// ------------------------------------------------------------------ the divergence and its gradient

struct DistillArgs {
  nq_teacher P;
  float c;
  const void* logits;
  int64_t ld;
  const float* weight;
  float* loss;
  void* dlogits;
  int64_t ldd;
  int V;
};

struct RowConsts {  // of one row, for every thread
  double base, inv, total, scale, w;
  float ref, coef;
  int zero;
};

// LDS of a row: [probabilities][ids][logits of the k entries][bitmap of the listed tokens, whole words].
// An entry's id is -1 where there is none, and -2 - id for a repetition of an earlier entry.
struct RowLds {
  double* ps;
  int* ids;
  float* sv;
  uint32_t* listed;
  __device__ RowLds(double* lds, int k) {
    ps = lds;
    ids = reinterpret_cast<int*>(lds + k);
    sv = reinterpret_cast<float*>(ids + k);
    listed = reinterpret_cast<uint32_t*>(sv + k);
  }
};
size_t row_lds_bytes(int64_t V, int64_t k) { return (size_t)cdiv(V, 32) * 4 + (size_t)k * 16; }

template <int NT>
struct RowShared {
  float max[NT / 64][2];
  double sum[NT / 64][4];
  RowConsts row;
  int bad, dup;
};

template <bool BF16>
__device__ inline const char* row_at(const void* p, int64_t t, int64_t ld) {
  return static_cast<const char*>(p) + t * ld * (BF16 ? 2 : 4);
}

// The entries of row t into LDS and the bitmap; this thread's part of sum p and of sum p log p.  False:
// an id is out of range.
template <int NT, bool BF16>
__device__ bool row_entries(const DistillArgs& A, int64_t t, const char* x, const RowLds& L, RowShared<NT>& S,
                            double& mass, double& plogp) {
  const int tid = threadIdx.x, k = (int)A.P.k, V = A.V;
  if (tid == 0) S.bad = S.dup = 0;
#pragma unroll 1
  for (int i = tid; i < (V + 31) / 32; i += NT) L.listed[i] = 0;
  __syncthreads();
  mass = plogp = 0.0;
#pragma unroll 1
  for (int e = tid; e < k; e += NT) {
    const int id = A.P.ids[t * k + e];
    float s = -kInf;
    double p = 0.0;
    if (id >= V) {
      S.bad = 1;
    } else if (id >= 0) {
      if (atomicOr(&L.listed[id / 32], 1u << (id % 32)) >> (id % 32) & 1u) S.dup = 1;
      s = load_element(x, BF16, id);
      const double lp = A.P.logp[t * k + e];
      p = exp(lp);
      mass += p;
      if (p != 0.0) plogp += p * lp;
    }
    L.ids[e] = id < 0 ? -1 : id;
    L.sv[e] = s;
    L.ps[e] = p;
  }
  __syncthreads();
  return !S.bad;
}

// Where a token is listed more than once: the first of its entries takes the probabilities of all.
// (NT entries at a time: the first of a token's entries keeps its id, so later ones find it.)
template <int NT>
__device__ void row_repetitions(const DistillArgs& A, const RowLds& L) {
  const int k = (int)A.P.k;
#pragma unroll 1
  for (int e0 = 0; e0 < k; e0 += NT) {
    const int e = e0 + (int)threadIdx.x, id = e < k ? L.ids[e] : -1;
    double sum = 0.0;
    bool again = false;
    if (id >= 0)
#pragma unroll 1
      for (int f = 0; f < k; ++f)
        if (L.ids[f] == id) {
          again |= f < e;
          sum += L.ps[f];
        }
    __syncthreads();
    if (id >= 0) {
      L.ps[e] = again ? 0.0 : sum;
      if (again) L.ids[e] = -2 - id;
    }
    __syncthreads();
  }
}

// The row's loss and the constants of its gradient, from each thread's maximum m and sum s (relative
// to its maximum) over the tokens not listed that it has read, and its parts of sum p and sum p log p.
template <int NT, bool GRADS>
__device__ RowConsts row_finish(const DistillArgs& A, int64_t t, float w, float m, float s, double mass, double plogp,
                                const RowLds& L, RowShared<NT>& S) {
  constexpr int W = NT / 64;  // waves, at most 16
  const int tid = threadIdx.x, k = (int)A.P.k, lane = tid % 64, wave = tid / 64;
  const bool entries = wave * 64 < k;  // the waves that have entries
  float m_k = -kInf;
  if (entries) {
#pragma unroll 1
    for (int e = tid; e < k; e += NT)
      if (L.ids[e] != -1) m_k = fmaxf(m_k, L.sv[e]);
    m_k = wave_max(m_k);
  }
  float m_r = wave_max(m);
  if (lane == 0) {
    S.max[wave][0] = m_r;
    S.max[wave][1] = m_k;
  }
  __syncthreads();
  m_r = row_max(S.max[lane % W][0]);
  m_k = row_max(S.max[lane % W][1]);
  // everything relative to the row's largest logit, at which an fp64 number of its own size may not
  // hold the logarithms
  const float ref = m_r == -kInf ? 0.0f : m_r, top = fmaxf(m_r, m_k);
  const double base = top == -kInf ? 0.0 : (double)top, rtau = 1.0 / (double)A.P.temperature;
  // sums: of the rest, of the listed tokens' exponentials, of p and of p (log p - s / tau)
  double sum[4] = {(double)s * (double)exp_scaled(m == -kInf ? 0.0f : m - ref, A.c), 0.0, mass, plogp};
  sum[0] = wave_sum(sum[0]);
  if (entries) {
#pragma unroll 1
    for (int e = tid; e < k; e += NT) {
      if (L.ids[e] < 0) continue;  // a repetition's probability is with the first
      const double p = L.ps[e], sx = ((double)L.sv[e] - base) * rtau;
      sum[1] += exp(sx);
      if (p != 0.0) sum[3] -= p * sx;
    }
#pragma unroll
    for (int j = 1; j < 4; ++j) sum[j] = wave_sum(sum[j]);
  }
  if (lane == 0)
#pragma unroll
    for (int j = 0; j < 4; ++j) S.sum[wave][j] = sum[j];
  __syncthreads();
  if (GRADS && wave == 0) {
#pragma unroll
    for (int j = 0; j < 3; ++j) sum[j] = row_sum(lane % 16 < W ? S.sum[lane % 16][j] : 0.0);
    if (tid == 0) {
      const double e_r = exp(((double)ref - base) * rtau), all = sum[1] + sum[0] * e_r;
      const double r = A.P.rest ? exp((double)A.P.rest[t]) : 0.0, total = A.P.rest ? sum[2] + r : 1.0;
      RowConsts R;
      R.zero = (A.P.rest ? total : sum[2]) == 0.0;
      R.base = base;
      R.inv = 1.0 / all;
      R.total = total;
      R.scale = A.P.rest ? 1.0 : 1.0 / sum[2];  // of the listed probabilities
      R.w = (double)w * rtau;
      R.ref = ref;
      // the gradient of a token not listed is coef * exp((s - ref) / tau)
      double coef = total * e_r * R.inv;
      if (r != 0.0) coef -= r / sum[0];
      R.coef = sum[0] == 0.0 && all > 0.0 ? 0.0f : (float)(R.w * coef);
      S.row = R;
    }
  }
  if (GRADS) __syncthreads();
  if (A.loss && wave == W - 1) {  // its logarithms are not waited for by the gradient
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = row_sum(lane % 16 < W ? S.sum[lane % 16][j] : 0.0);
    if (lane == 0) {
      const double ref_r = ((double)ref - base) * rtau, lse = log(sum[1] + sum[0] * exp(ref_r));
      double loss = A.P.rest ? sum[3] + sum[2] * lse : sum[3] / sum[2] - log(sum[2]) + lse;
      double all = sum[2];
      if (A.P.rest) {
        const double lr = A.P.rest[t], r = exp(lr);
        all += r;
        if (r != 0.0) loss += r * (lr - (ref_r + log(sum[0]) - lse));
      }
      A.loss[t] = all == 0.0 ? 0.0f : (float)((double)w * loss);
    }
  }
  if (!GRADS) return {};
  return S.row;
}

// The listed tokens' gradients, over what was stored for them before the last barrier.
template <int NT, bool DBF16>
__device__ inline void row_listed_grads(const DistillArgs& A, char* dx, const RowConsts& R, const RowLds& L) {
  const double rtau = 1.0 / (double)A.P.temperature;
#pragma unroll 1
  for (int e = threadIdx.x; e < (int)A.P.k; e += NT)
    if (L.ids[e] >= 0) {
      const double q = exp(((double)L.sv[e] - R.base) * rtau) * R.inv;
      store_element(dx, DBF16, L.ids[e], (float)(R.w * (R.total * q - R.scale * L.ps[e])));
    }
}

template <int NT, bool GRADS, bool DBF16>
__device__ inline void constant_row(const DistillArgs& A, int64_t t, char* dx, float v) {
  if (threadIdx.x == 0 && A.loss) A.loss[t] = v;
  if (GRADS)
#pragma unroll 1
    for (int i = threadIdx.x; i < A.V; i += NT) store_element(dx, DBF16, i, v);
}

// 16 bytes of a row at any alignment of its elements.
template <bool BF16>
struct Piece {
  static constexpr int N = BF16 ? 8 : 4;  // elements
  uint32_t v[4];
  __device__ void load(const char* row, int j) {
    u32x4 d;
    if (BF16)
      d = *reinterpret_cast<const u32x4_a2*>(row + (uint32_t)j * 16u);
    else
      d = *reinterpret_cast<const u32x4_a4*>(row + (uint32_t)j * 16u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = d[i];
  }
  __device__ void fill() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = BF16 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  }
  __device__ float at(int i) const {
    if (!BF16) return __uint_as_float(v[i]);
    return __uint_as_float(i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
  }
  // Keeps the compiler from holding the unpacked elements across a pass beside the packed ones.
  __device__ void packed() { asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3])); }
  // bit i of `m`: element i becomes -inf
  __device__ void mask(uint32_t m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        const uint32_t lo = __builtin_amdgcn_sbfe(m, 2 * i, 1), hi = __builtin_amdgcn_sbfe(m, 2 * i + 1, 1);
        const uint32_t on = (lo & 0xFFFFu) | (hi & 0xFFFF0000u);
        v[i] = (v[i] & ~on) | (on & 0xFF80FF80u);
      } else {
        const uint32_t on = __builtin_amdgcn_sbfe(m, i, 1);
        v[i] = (v[i] & ~on) | (on & 0xFF800000u);
      }
    }
  }
  __device__ void choose(bool other, const Piece& o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = v[i], b = o.v[i];
      v[i] = other ? b : a;
    }
  }
  // element i of a lane's own choice (by masks: a choice of array elements would put the piece in memory)
  __device__ float pick(int i) const {
    const int w = BF16 ? i / 2 : i;
    const uint32_t odd = __builtin_amdgcn_sbfe(w, 0, 1), up = __builtin_amdgcn_sbfe(w, 1, 1);
    const uint32_t lo = v[0] ^ ((v[0] ^ v[1]) & odd), hi = v[2] ^ ((v[2] ^ v[3]) & odd), u = lo ^ ((lo ^ hi) & up);
    return __uint_as_float(!BF16 ? u : i & 1 ? u & 0xFFFF0000u : u << 16);
  }
  // the bits of piece j in the bitmap
  __device__ static uint32_t bits(const uint32_t* listed, int j) {
    if (BF16) return reinterpret_cast<const uint8_t*>(listed)[j];
    return reinterpret_cast<const uint8_t*>(listed)[j / 2] >> (4 * (j % 2)) & 15u;
  }
};
// N results as piece j of a row, past the caches: a gradient's rows are not read again by the call, and
// what they would push out of the caches is (4096 rows of 131072 bf16: 522 us with plain stores, 456).
template <int N, bool BF16>
__device__ inline void store_piece(char* row, int j, const float (&g)[N]) {
  char* p = row + (uint32_t)j * (uint32_t)(N * (BF16 ? 2 : 4));
  if constexpr (BF16 && N == 8) {
    const u32x4_a2 d = u32x4{bf16_pair(g[0], g[1]), bf16_pair(g[2], g[3]), bf16_pair(g[4], g[5]), bf16_pair(g[6], g[7])};
    __builtin_nontemporal_store(d, reinterpret_cast<u32x4_a2*>(p));
  } else if constexpr (BF16) {
    const u32x2_a2 d = u32x2{bf16_pair(g[0], g[1]), bf16_pair(g[2], g[3])};
    __builtin_nontemporal_store(d, reinterpret_cast<u32x2_a2*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4_a4 d = u32x4{__float_as_uint(g[i]), __float_as_uint(g[i + 1]), __float_as_uint(g[i + 2]),
                               __float_as_uint(g[i + 3])};
      __builtin_nontemporal_store(d, reinterpret_cast<u32x4_a4*>(p + 4 * i));
    }
  }
}

// A workgroup reads its row once, U pieces per thread at a time, each thread with a maximum and the sum
// below it (rescaled once for the U pieces).  For the gradient it goes over the row a second time,
// backwards: the last pieces are still in registers and those before them in the caches.  Tokens past
// the last whole piece are one each of the first threads'.  Bound by memory where the rows are many and
// long: a loss of 2048 rows of 131072 bf16 98 us (5.5 TB/s read), a gradient of 4096 of them 453 us (4.7 TB/s,
// a large copy's rate is 4.9); 2048 rows of 32000 are all under way at once and read and write in turns
// (gradient 67 us, 3.9 TB/s).  Few short rows are a chain of a read, two exchanges and the logarithms (8
// rows of 4096: 6.1 us).
template <bool GRADS, bool BF16, bool DBF16, int NT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(8))) void distill_kernel(const DistillArgs A) {
  using Pc = Piece<BF16>;
  constexpr int N = Pc::N, U = 4;
  extern __shared__ double lds[];
  __shared__ RowShared<NT> S;
  const int tid = threadIdx.x, V = A.V, np = V / N;
  const int64_t t = blockIdx.x;
  const RowLds L(lds, (int)A.P.k);
  const char* x = row_at<BF16>(A.logits, t, A.ld);
  char* dx = GRADS ? static_cast<char*>(A.dlogits) + t * A.ldd * (DBF16 ? 2 : 4) : nullptr;
  const float w = A.weight ? A.weight[t] : 1.0f;
  if (w == 0.0f) return constant_row<NT, GRADS, DBF16>(A, t, dx, 0.0f);
  double mass, plogp;
  if (!row_entries<NT, BF16>(A, t, x, L, S, mass, plogp))
    return constant_row<NT, GRADS, DBF16>(A, t, dx, __builtin_nanf(""));
  if (S.dup) row_repetitions<NT>(A, L);
  const int it = np * N + tid;
  float xt = it < V ? load_element(x, BF16, it) : -kInf;
  if (it < V && (L.listed[it / 32] >> (it % 32) & 1u)) xt = -kInf;
  float m = xt, s = exp_scaled(xt - (xt == -kInf ? 0.0f : xt), A.c);
  Pc pc[U];
  auto load = [&](int j0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * NT;
      if (j < np)
        pc[i].load(x, j);
      else
        pc[i].fill();
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * NT;
      pc[i].packed();
      const uint32_t b = j < np ? Pc::bits(L.listed, j) : 0;
      if (b) pc[i].mask(b);
      pc[i].packed();
    }
  };
  int j0 = tid;
  for (;; j0 += NT * U) {
    load(j0);
    float mm = m;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int q = 0; q < N; q += 2) mm = max3(mm, pc[i].at(q), pc[i].at(q + 1));
    const float ref = mm == -kInf ? 0.0f : mm;
    s *= exp_scaled(m - ref, A.c);
    m = mm;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int q = 0; q < N; ++q) s += exp_scaled(pc[i].at(q) - ref, A.c);
      pc[i].packed();
    }
    if (j0 - tid + NT * U >= np) break;
  }
  const RowConsts R = row_finish<NT, GRADS>(A, t, w, m, s, mass, plogp, L, S);
  if (!GRADS) return;
  if (R.zero) return constant_row<NT, GRADS, DBF16>(A, t, dx, 0.0f);
  if (it < V) store_element(dx, DBF16, it, R.coef * exp_scaled(xt - R.ref, A.c));
  for (;; j0 -= NT * U) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * NT;
      pc[i].packed();
      float g[N];
#pragma unroll
      for (int q = 0; q < N; ++q) g[q] = R.coef * exp_scaled(pc[i].at(q) - R.ref, A.c);
      if (j < np) store_piece<N, DBF16>(dx, j, g);
    }
    if (j0 == tid) break;
    load(j0 - NT * U);
  }
  __syncthreads();  // the listed tokens' places are written
  row_listed_grads<NT, DBF16>(A, dx, R, L);
}

// ------------------------------------------------------------------ a teacher's top logits

// Keys in the order of the logits: -0 equals +0, NaN lies above +inf.
__device__ inline uint32_t logit_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ inline float key_logit(uint32_t key) { return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }
constexpr uint32_t kFirstKey = 0x00800000u;  // the lowest above -inf's

// Candidates a row has room for (twice the k that a workgroup's size serves), and each wave of it.
template <int NT>
constexpr int kCandidates = 2 * NT;
constexpr int kWaveCandidates = 256;

struct TopArgs {
  const void* logits;
  int64_t ld;
  int V, k;
  float c;
  double rtau;
  int32_t* ids;
  float *logp, *rest;
};

// A candidate: its key above its index's complement, so that the larger comes first and, of equal ones,
// the lower index.
__device__ inline uint64_t top_place_key(uint32_t key, int idx) { return (uint64_t)key << 32 | ~(uint32_t)idx; }

template <int NT>
struct TopShared {
  uint64_t cand[kCandidates<NT>];
  uint64_t own[NT / 64][kWaveCandidates];
  float top_z[kCandidates<NT>];  // by place
  int top_i[NT];
  double sum[NT / 64][2];
  float max[NT / 64];
  int count[NT / 64], bound[NT / 64];
  int n, over;
};

template <int NT>
__device__ inline int wg_count(int n, int* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = n;
  __syncthreads();
  n = 0;
#pragma unroll 1
  for (int w = 0; w < NT / 64; ++w) n += red[w];
  return n;
}

// Places of the candidates (each one's is the number of those before it); the first k are listed, the
// others belong to the rest.  (The candidates' own order changes from run to run, their places do not.)
template <int NT>
__device__ void top_places(const TopArgs& A, TopShared<NT>& S, int n, MaxSum& rest) {
  for (int e = threadIdx.x; e < n; e += NT) {
    const uint64_t mine = S.cand[e];
    int place = 0;
#pragma unroll 8
    for (int f = 0; f < n; ++f) place += S.cand[f] > mine;
    S.top_z[place] = key_logit((uint32_t)(mine >> 32));
    if (place < A.k) S.top_i[place] = (int)~(uint32_t)mine;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += NT)
    if (e >= A.k) rest.add(S.top_z[e], A.c);
}

// The record of row t from the m listed tokens and each thread's part of the rest.  False: there is NaN
// in the rest (nothing is written then).
template <int NT>
__device__ bool top_record(const TopArgs& A, TopShared<NT>& S, int64_t t, int m, const MaxSum& rest, bool even_nan) {
  constexpr int W = NT / 64;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  float m_r = wave_max(rest.m);
  if (lane == 0) S.max[wave] = m_r;
  __syncthreads();
  m_r = row_max(S.max[lane % W]);
  const float ref = m_r == -kInf ? 0.0f : m_r;
  const double ref_k = m > 0 ? (double)S.top_z[0] : 0.0;
  double s_r = wave_sum((double)rest.s * (double)exp_scaled(rest.m == -kInf ? 0.0f : rest.m - ref, A.c)), s_k = 0.0;
  if (wave * 64 < m) {
#pragma unroll 1
    for (int e = tid; e < m; e += NT) s_k += exp(((double)S.top_z[e] - ref_k) * A.rtau);
    s_k = wave_sum(s_k);
  }
  if (lane == 0) {
    S.sum[wave][0] = s_r;
    S.sum[wave][1] = s_k;
  }
  __syncthreads();
  s_r = row_sum(lane % 16 < W ? S.sum[lane % 16][0] : 0.0);
  if (s_r != s_r && !even_nan) return false;
  if (wave * 64 >= A.k && tid != 0) return true;
  s_k = row_sum(lane % 16 < W ? S.sum[lane % 16][1] : 0.0);
  // relative to ref_k / tau; an empty row has nothing listed and rest -inf
  const double ref_r = ((double)ref - ref_k) * A.rtau, lse = log(s_k + s_r * exp(ref_r));
#pragma unroll 1
  for (int e = tid; e < A.k; e += NT) {
    A.ids[t * A.k + e] = e < m ? S.top_i[e] : -1;
    A.logp[t * A.k + e] = e < m ? (float)(((double)S.top_z[e] - ref_k) * A.rtau - lse) : -kInf;
  }
  if (tid == 0 && A.rest) A.rest[t] = s_r == 0.0 && lse == lse ? -kInf : (float)(ref_r + log(s_r) - lse);
  return true;
}

// Any row, NaN and long runs of equal logits among them: the k-th largest key bit by bit, then the last
// of the equal ones by index, so that exactly the listed tokens are candidates.
template <int NT>
__device__ void top_by_bits(const TopArgs& A, TopShared<NT>& S, int64_t t, const char* x, bool bf16) {
  const int tid = threadIdx.x, V = A.V, k = A.k;
  int* red = S.count;
  uint32_t at = 0;
#pragma unroll 1
  for (int b = 31; b >= 0; --b) {
    const uint32_t key = at | 1u << b;
    int n = 0;
#pragma unroll 1
    for (int i = tid; i < V; i += NT) n += logit_key(load_element(x, bf16, i)) >= key;
    if (wg_count<NT>(n, red) >= k) at = key;
  }
  int last = 0x7fffffff;
  if (at < kFirstKey) {  // fewer than k above -inf: all of those
    at = kFirstKey;
  } else {
    int above = 0;
#pragma unroll 1
    for (int i = tid; i < V; i += NT) above += logit_key(load_element(x, bf16, i)) > at;
    const int need = k - wg_count<NT>(above, red);
    int lo = 0, hi = V - 1;  // the smallest index up to which `need` keys equal the k-th
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      int n = 0;
#pragma unroll 1
      for (int i = tid; i <= mid; i += NT) n += logit_key(load_element(x, bf16, i)) == at;
      if (wg_count<NT>(n, red) >= need)
        hi = mid;
      else
        lo = mid + 1;
    }
    last = lo;
  }
  __syncthreads();
  if (tid == 0) S.n = 0;
  __syncthreads();
  MaxSum rest;
#pragma unroll 1
  for (int i = tid; i < V; i += NT) {
    const float v = load_element(x, bf16, i);
    const uint32_t key = logit_key(v);
    if (key > at || (key == at && i <= last))
      S.cand[atomicAdd(&S.n, 1)] = top_place_key(key, i);  // at most k
    else
      rest.add(v, A.c);
  }
  __syncthreads();
  const int n = S.n;
  top_places<NT>(A, S, n, rest);
  top_record<NT>(A, S, t, n, rest, true);
}

// Order of floats as integers (-0 below 0; a bound of 0 takes both).
__device__ inline int float_order(float v) {
  const int i = __float_as_int(v);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ inline float order_float(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// A value that at least k logits reach, and few more where the largest are spread over the row: each of
// the `waves` waves that have logits finds one that `quota` of its groups' maxima reach (each thread has
// G), quota * waves >= k, and the lowest of them is taken.  The lowest finite value where a wave has too
// few finite groups.
template <int NT, int G>
__device__ float top_bound(TopShared<NT>& S, const float (&gm)[G], int quota, int waves) {
  constexpr int W = NT / 64;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  int lo = 0x7fffffff;
  if (wave < waves) {
    // between lo, which at least quota reach (the least of the lanes' largest, or of all groups, or the
    // lowest finite value), and hi, which fewer do
    float most = gm[0], least = gm[0];
#pragma unroll
    for (int i = 1; i < G; ++i) {
      most = fmaxf(most, gm[i]);
      least = fminf(least, gm[i]);
    }
    lo = max(float_order(-wave_max(-(quota <= 64 ? most : least))), float_order(-__FLT_MAX__));
    int hi = float_order(wave_max(most)) + 1, g[G];
#pragma unroll
    for (int i = 0; i < G; ++i) g[i] = float_order(gm[i]);
    while (hi > lo && (uint32_t)hi - (uint32_t)lo > 1) {
      const int mid = (int)((uint32_t)lo + ((uint32_t)hi - (uint32_t)lo) / 2);
      int n = 0;
#pragma unroll
      for (int i = 0; i < G; ++i) n += __popcll(__ballot(g[i] >= mid));
      if (n >= quota) {
        lo = mid;
        if (n <= quota + quota / 8 + 1) break;
      } else {
        hi = mid;
      }
    }
  }
  __syncthreads();  // an earlier call's values have been read
  if (lane == 0) S.bound[wave] = lo;
  __syncthreads();
  int b = S.bound[lane % W];
  b = min(b, __builtin_amdgcn_mov_dpp(b, kXor1, 0xF, 0xF, true));
  b = min(b, __builtin_amdgcn_mov_dpp(b, kXor2, 0xF, 0xF, true));
  b = min(b, __builtin_amdgcn_mov_dpp(b, kHalfMirror, 0xF, 0xF, true));
  b = min(b, __builtin_amdgcn_mov_dpp(b, kMirror, 0xF, 0xF, true));
  return order_float(b);
}

// One pass over the row.  The maxima of the first step's groups give a bound that at least k logits
// reach; from there on logits that reach it are candidates, which each wave keeps in LDS in the order it
// meets them, and the others are the rest, whose sum is taken as in distill_kernel.  The bound is taken
// anew where the steps double and at the end, and what no longer reaches it joins the rest.  Bound by vector
// instructions, 2900 a wave: 2048 rows of 32000 bf16, k 64, 51 us where their reads alone are 27; one row is
// a chain of dependent steps, 11.4 us.
// Rows with more candidates than there is room for or with NaN are done by bits instead: long runs of equal
// logits, the largest in few groups, and short rows whose last wave has fewer groups than its quota, which
// makes the bound the lowest finite value (fewer pieces than threads, and not a multiple of 64 of them, or
// nearly).  us for one row / 2048 of them, bf16: 520, k 64, 42 / 60 where 512 take 9.4 / 15; 1544, k 32,
// 58 / 89 where 1536 take 9.3 / 17; 3153, k 217, 71 / 193.  A constant row of 32000, k 64, takes 224 alone
// and 1600 with 256 threads, and a call of 2048 rows as long with one such row in 16 as with nothing else.
template <bool BF16, int NT>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(8))) void logits_top_kernel(const TopArgs A) {
  using Pc = Piece<BF16>;
  constexpr int N = Pc::N, U = 4;
  __shared__ TopShared<NT> S;
  const int tid = threadIdx.x, V = A.V, np = V / N, lane = tid % 64, k = A.k;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int64_t t = blockIdx.x;
  const char* x = row_at<BF16>(A.logits, t, A.ld);
  if (tid == 0) S.n = S.over = 0;
  const int it = np * N + tid;
  float xt = it < V ? load_element(x, BF16, it) : -kInf;
  constexpr int H = BF16 ? 2 : 1, G = U * H;  // groups: quarters of a step's pieces, 4 logits each
  float gm[G], bound = 0.0f;
#pragma unroll
  for (int i = 0; i < G; ++i) gm[i] = -kInf;
  gm[0] = xt;
  const int waves = max(1, (min(np, NT) + 63) / 64), quota = (k + waves - 1) / waves;
  MaxSum rest;
  int mine = 0;  // this wave's candidates
  // takes the logits of those lanes, one of each; all lanes of the wave come here
  auto take = [&](uint64_t lanes, bool on, float v, int idx) {
    const int at = mine + __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0));
    if (on && at < kWaveCandidates) S.own[wave][at] = top_place_key(logit_key(v), idx);
    mine += __popcll(lanes);
  };
  // what of this wave's candidates no longer reaches the bound joins the rest
  auto prune = [&] {
    int kept = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < mine; e0 += 64) {
      const uint64_t c = S.own[wave][min(e0 + lane, kWaveCandidates - 1)];
      const float v = key_logit((uint32_t)(c >> 32));
      const bool on = e0 + lane < mine, keep = on && v >= bound;
      const uint64_t lanes = __ballot(keep);
      const int at = kept + __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0));
      if (keep) S.own[wave][at] = c;
      if (on && !keep) rest.add(v, A.c);
      kept += __popcll(lanes);
    }
    mine = kept;
  };
  int steps = 0, next_bound = 0, last_bound = 0;
#pragma unroll 1
  for (int j0 = tid; j0 - tid < np || steps == 0; j0 += NT * U, ++steps) {
    Pc pc[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = j0 + i * NT;
      if (j < np)
        pc[i].load(x, j);
      else
        pc[i].fill();
    }
    float pm[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      pm[i] = -kInf;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float m = pc[i].at(4 * h);
        m = max3(m, pc[i].at(4 * h + 1), pc[i].at(4 * h + 2));
        m = fmaxf(m, pc[i].at(4 * h + 3));
        gm[i * H + h] = fmaxf(gm[i * H + h], m);
        pm[i] = fmaxf(pm[i], m);
      }
      pc[i].packed();
    }
    if (steps == next_bound) {
      bound = top_bound<NT>(S, gm, quota, waves);
      last_bound = steps;
      next_bound = 2 * steps + 1;
      if (mine > kWaveCandidates) S.over = 1, mine = kWaveCandidates;
      prune();
    }
    if (steps == 0) {
      const bool on = xt >= bound;
      if (const uint64_t lanes = __ballot(on)) take(lanes, on, xt, it);
      rest.add(on ? -kInf : xt, A.c);
    }
    // Pieces with candidates, one of each lane in turn (of 64 lanes' 4 pieces two thirds have one when 64 of
    // 32000 are wanted, but hardly a lane has it in two of its own): the lane's element by element in turn.
    for (;;) {
      int which = -1;
#pragma unroll
      for (int i = U - 1; i >= 0; --i) which = pm[i] >= bound ? i : which;
      if (!__any(which >= 0)) break;
      Pc p = pc[0];
#pragma unroll
      for (int i = 1; i < U; ++i) p.choose(which == i, pc[i]);
      uint32_t bits = 0;
#pragma unroll
      for (int q = 0; q < N; ++q) bits |= p.at(q) >= bound ? 1u << q : 0u;
      if (which < 0) bits = 0;
      uint32_t left = bits;
      while (const uint64_t lanes = __ballot(left != 0)) {
        const int q = __builtin_ctz(left | 1u << 31);
        take(lanes, left != 0, p.pick(q), (j0 + which * NT) * N + q);
        left &= left - 1;
      }
      p.mask(bits);
      float m = -kInf;
#pragma unroll
      for (int q = 0; q < N; q += 2) m = max3(m, p.at(q), p.at(q + 1));
#pragma unroll
      for (int i = 0; i < U; ++i) {
        pc[i].choose(which == i, p);
        pm[i] = which == i ? m : pm[i];
      }
    }
    float mm = rest.m;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      pc[i].packed();
      mm = fmaxf(mm, pm[i]);
    }
    const float ref = mm == -kInf ? 0.0f : mm;
    rest.s *= exp_scaled(rest.m - ref, A.c);
    rest.m = mm;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int q = 0; q < N; ++q) rest.s += exp_scaled(pc[i].at(q) - ref, A.c);
  }
  if (mine > kWaveCandidates) S.over = 1, mine = kWaveCandidates;
  if (last_bound < steps - 1) {
    bound = top_bound<NT>(S, gm, quota, waves);
    prune();
  }
  int first = 0;
  if (lane == 0) first = atomicAdd(&S.n, mine);
  first = __builtin_amdgcn_readfirstlane(first);
#pragma unroll 1
  for (int e = lane; e < mine; e += 64)
    if (first + e < kCandidates<NT>) S.cand[first + e] = S.own[wave][e];
  __syncthreads();
  const int n = S.n;
  if (n <= kCandidates<NT> && !S.over) {
    top_places<NT>(A, S, n, rest);
    if (top_record<NT>(A, S, t, min(n, k), rest, false)) return;
  }
  __syncthreads();
  top_by_bits<NT>(A, S, t, x, BF16);
}

}  // namespace

hipError_t launch_logits_top(const void* logits, nq_dtype dt, int64_t T, int64_t V, int64_t ld, int k, float temperature,
                             int32_t* ids, float* logp, float* rest, hipStream_t s) {
  const TopArgs A{logits, ld, (int)V, k, exp_scale(temperature), 1.0 / (double)temperature, ids, logp, rest};
  const bool bf16 = dt == NQ_BF16;
  const int64_t np = V / (bf16 ? 8 : 4);
  // as for the loss (launch_distill_t); a larger k needs the larger workgroups' room for candidates
  int nt = np <= 1024 || T > 1024 ? 256 : np <= 2048 ? 512 : 1024;
  if (k > 128) nt = k > 256 ? 1024 : nt < 512 ? 512 : nt;
  const auto kernel = nt == 256   ? (bf16 ? logits_top_kernel<true, 256> : logits_top_kernel<false, 256>)
                      : nt == 512 ? (bf16 ? logits_top_kernel<true, 512> : logits_top_kernel<false, 512>)
                                  : (bf16 ? logits_top_kernel<true, 1024> : logits_top_kernel<false, 1024>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)T), dim3(nt), 0, s, A);
  return hipGetLastError();
}

namespace {

// kernel<<<T, NT, lds of the row>>>; the largest row's LDS is allowed once per device
template <typename K>
hipError_t launch_rows(K kernel, int64_t T, int nt, const DistillArgs& A, std::atomic<uint64_t>& done, hipStream_t s) {
  const size_t lds = row_lds_bytes(A.V, A.P.k);
  if (lds > 48 * 1024) {
    const hipError_t e =
        allow_lds(reinterpret_cast<const void*>(kernel), row_lds_bytes(int64_t{1} << 20, NQ_TOP_MAX), done);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)T), dim3(nt), lds, s, A);
  return hipGetLastError();
}
// Threads per row, by its 16-byte pieces and the number of rows (us with 256 / 512 / 1024 threads):
//   up to 1024 pieces, one step of 256 threads: a row costs by its threads more than by its length
//     (8192 rows of 8192 bf16: loss 39 / 63 / 105, gradient 60 / 83 / 138; 16 rows: 6.3 / 6.5 / 6.8);
//   a loss of many rows needs no more than 256 either, the rows fill the chip (2048 rows of 32000: 28 /
//     29 / 37, of 131072: 100 / 109 / 102), one of few needs them (16 of 131072: 22 / 14 / 13);
//   a gradient reads back what its threads' registers do not hold, and the fewer rows are under way at
//     once the more of that is still in the caches (2048 of 131072: 283 / 267 / 241; 16: 41 / 26 / 22; 2048
//     of 32000: 61.7 / 61.2 / 60.3, 4096 of them 124 / 123 / 133, 512 22 / 18 / 18); rows of up to 2048
//     pieces fit 512 threads' (512 rows of 16384: 12.9 / 12.0 / 14.4).
template <bool GRADS, bool BF16, bool DBF16>
hipError_t launch_distill_t(int64_t T, const DistillArgs& A, hipStream_t s) {
  static std::atomic<uint64_t> done[3];
  const int64_t np = A.V / Piece<BF16>::N;
  if (np <= 1024 || (!GRADS && T > 1024)) return launch_rows(distill_kernel<GRADS, BF16, DBF16, 256>, T, 256, A, done[0], s);
  if (np <= 2048) return launch_rows(distill_kernel<GRADS, BF16, DBF16, 512>, T, 512, A, done[1], s);
  return launch_rows(distill_kernel<GRADS, BF16, DBF16, 1024>, T, 1024, A, done[2], s);
}

}  // namespace

hipError_t launch_distill(const nq_teacher& P, const void* logits, nq_dtype dt, int64_t T, int64_t V, int64_t ld,
                          const float* weight, float* loss, void* dlogits, nq_dtype dd, int64_t ldd, hipStream_t s) {
  const DistillArgs A{P, exp_scale(P.temperature), logits, ld, weight, loss, dlogits, ldd, (int)V};
  if (!dlogits) return dt == NQ_BF16 ? launch_distill_t<false, true, true>(T, A, s) : launch_distill_t<false, false, false>(T, A, s);
  if (dt == NQ_BF16)
    return dd == NQ_BF16 ? launch_distill_t<true, true, true>(T, A, s) : launch_distill_t<true, true, false>(T, A, s);
  return dd == NQ_BF16 ? launch_distill_t<true, false, true>(T, A, s) : launch_distill_t<true, false, false>(T, A, s);
}

}  // namespace nq
