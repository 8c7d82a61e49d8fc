// Low-rank adapters of many requests beside a shared projection, and their
// gradients.  Token t with adapter a = ids[t] adds a rank-r product to its row:
//
//     h_t  = A_a x_t                    y_t  = base_t + scale_a B_a h_t
//     dh_t = scale_a B_a^T g_t          dx_t = dx_base_t + A_a^T dh_t
//     dA_a = sum_t dh_t x_t^T           dB_a = scale_a sum_t g_t h_t^T
//
// with A_a [r][d_in] and B_a [d_out][r].  A negative id takes no adapter.
//
// What bounds it: the rows.  r is far below d_in and d_out, so each product
// reads or writes T x d values for 2 T r d operations; the kernels are built
// around streaming x, g, base, y once with the factors in registers or cache.
//
// Tokens are grouped by adapter (lora_route_kernel) into tiles of 32 slots of
// one adapter each, so that every matrix product of a tile has one adapter's
// factors; slots past an adapter's last token hold no row.  Calls of up to 64
// tokens find their groups with one ballot per workgroup instead.
//
// One fragment layout serves every product and both arithmetics: lane l =
// (q = l / 16, c = l % 16) holds 8 elements 8q .. 8q+7 of a 32-deep reduction
// step, for row (or column) c.  bf16 operands take one 16x16x32 bf16 matrix
// instruction; fp32 operands take eight 16x16x4 fp32 ones, step e using element
// e of each lane.  Which 8 elements of the reduction a lane's slots hold does
// not matter as long as both operands agree, so lanes load 16 bytes of
// consecutive elements.  The result's lane (q, c) holds rows 4q .. 4q+3 of
// column c.
//
// h and dh are kept in fp32.  Beside bf16 factors they enter the matrix cores
// as three bf16 terms that carry all 24 bits (split3), so nothing is rounded to
// fewer bits than fp32 anywhere.  Sums have a fixed order; there are no
// atomics on floating data.
//
// Rows and columns of a matrix product do not mix: slots without a row and
// rank rows past r load some valid address and are set to zero when stored;
// only tails of a reduction need zero operands.
#include "nq_internal.h"

namespace nq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = kLoraTile;   // slots per tile
constexpr int kRouteThreads = 1024;

struct Bf16 {  // storage of a bf16 element
  uint16_t u;
};
__device__ inline float to_f32(float v) { return v; }
__device__ inline float to_f32(Bf16 v) { return __uint_as_float((uint32_t)v.u << 16); }

// ---------------------------------------------------------------- fragments
// 8 elements of a lane, as bf16 (one matrix instruction) or fp32 (eight).
template <typename E>
struct Frag;
template <>
struct Frag<Bf16> {
  u32x4 d;
};
template <>
struct Frag<float> {
  float v[8];
};

__device__ inline void mma(const Frag<Bf16>& a, const Frag<Bf16>& b, f32x4& c) {
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.d), __builtin_bit_cast(bf16x8, b.d), c, 0, 0,
                                              0);
}
__device__ inline void mma(const Frag<float>& a, const Frag<float>& b, f32x4& c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
}

// An fp32 operand beside fragments of E: itself, or three bf16 terms.
template <typename E>
struct Wide;
template <>
struct Wide<float> {
  Frag<float> f;
};
template <>
struct Wide<Bf16> {
  Frag<Bf16> t[3];
};

__device__ inline uint32_t high_halves(uint32_t lo, uint32_t hi) {  // (hi's upper 16) << 16 | lo's upper 16
  return __builtin_amdgcn_perm(hi, lo, 0x07060302);
}

// v = t0 + t1 + t2 exactly: each term takes the next 8 bits of the significand
// (truncated, so no term rounds).  An infinity is its own first term; a NaN that
// arithmetic made has its quiet bit in the upper half and stays one.
__device__ inline void split3(float v, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  t0 = __float_as_uint(v) & 0xFFFF0000u;
  float rest = v - __uint_as_float(t0);
  if (__builtin_isinf(v)) rest = 0.0f;
  t1 = __float_as_uint(rest) & 0xFFFF0000u;
  t2 = __float_as_uint(rest - __uint_as_float(t1));
}

__device__ inline void widen(const float (&v)[8], Wide<float>& w) {
#pragma unroll
  for (int e = 0; e < 8; ++e) w.f.v[e] = v[e];
}
__device__ inline void widen(const float (&v)[8], Wide<Bf16>& w) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t a[3], b[3];
    split3(v[2 * p], a[0], a[1], a[2]);
    split3(v[2 * p + 1], b[0], b[1], b[2]);
#pragma unroll
    for (int k = 0; k < 3; ++k) w.t[k].d[p] = high_halves(a[k], b[k]);
  }
}
// a: factor or activation, w: the fp32 side (smallest terms first)
__device__ inline void mma(const Frag<float>& a, const Wide<float>& w, f32x4& c) { mma(a, w.f, c); }
__device__ inline void mma(const Frag<Bf16>& a, const Wide<Bf16>& w, f32x4& c) {
#pragma unroll
  for (int k = 2; k >= 0; --k) mma(a, w.t[k], c);
}
__device__ inline void mma(const Wide<float>& w, const Frag<float>& a, f32x4& c) { mma(w.f, a, c); }
__device__ inline void mma(const Wide<Bf16>& w, const Frag<Bf16>& a, f32x4& c) {
#pragma unroll
  for (int k = 2; k >= 0; --k) mma(w.t[k], a, c);
}

// A fragment of 8 elements from 8 consecutive ones in memory, the first nv of
// them valid (zero past them).  F is the fragment's element type: E itself, or
// fp32 from bf16 in memory.
template <typename F, typename E>
__device__ inline Frag<F> load8(const E* p, int64_t nv);

template <>
__device__ inline Frag<Bf16> load8<Bf16, Bf16>(const Bf16* p, int64_t nv) {
  Frag<Bf16> f;
  if (nv >= 8) {
    f.d = *reinterpret_cast<const u32x4u*>(p);
  } else if (nv > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < nv ? p[2 * i].u : 0, hi = 2 * i + 1 < nv ? p[2 * i + 1].u : 0;
      f.d[i] = lo | (hi << 16);
    }
  } else {
    f.d = u32x4{0, 0, 0, 0};
  }
  return f;
}
template <>
__device__ inline Frag<float> load8<float, float>(const float* p, int64_t nv) {
  Frag<float> f;
  if (nv >= 8) {
    const f32x4 a = *reinterpret_cast<const f32x4u*>(p), b = *reinterpret_cast<const f32x4u*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = a[e], f.v[4 + e] = b[e];
  } else if (nv > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = e < nv ? p[e] : 0.0f;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = 0.0f;
  }
  return f;
}
template <>
__device__ inline Frag<float> load8<float, Bf16>(const Bf16* p, int64_t nv) {
  const Frag<Bf16> b = load8<Bf16, Bf16>(p, nv);
  Frag<float> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[2 * i] = __uint_as_float(b.d[i] << 16);
    f.v[2 * i + 1] = __uint_as_float(b.d[i] & 0xFFFF0000u);
  }
  return f;
}

// The same from 8 elements `stride` apart.
template <typename F, typename E>
__device__ inline Frag<F> load8s(const E* p, int64_t stride, int64_t nv) {
  Frag<F> f;
  if constexpr (sizeof(F) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < nv ? p[2 * i * stride].u : 0, hi = 2 * i + 1 < nv ? p[(2 * i + 1) * stride].u : 0;
      f.d[i] = lo | (hi << 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = e < nv ? to_f32(p[e * stride]) : 0.0f;
  }
  return f;
}

// in[e] holds elements 0..7 of row e: out[v] takes element v of each row.
__device__ inline void transpose8(const Frag<Bf16> (&in)[8], Frag<Bf16> (&out)[8]) {
#pragma unroll
  for (int v = 0; v < 8; ++v)
#pragma unroll
    for (int p = 0; p < 4; ++p)
      out[v].d[p] = __builtin_amdgcn_perm(in[2 * p + 1].d[v / 2], in[2 * p].d[v / 2], v % 2 ? 0x07060302 : 0x05040100);
}
__device__ inline void transpose8(const Frag<float> (&in)[8], Frag<float> (&out)[8]) {
#pragma unroll
  for (int v = 0; v < 8; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) out[v].v[e] = in[e].v[v];
}

__device__ inline f32x4 zero4() { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }

// ---------------------------------------------------------------- routing
// One workgroup per group: adapters 0..n-1, then the tokens without an adapter
// (n) and those whose id is out of range (n + 1).  Each counts every group
// (integer counters in LDS), which gives its first tile, and then lists its own
// tokens in order.
__global__ __launch_bounds__(kRouteThreads) void lora_route_kernel(const int32_t* __restrict__ ids, int T, int n,
                                                                   int* __restrict__ tile_off, int* __restrict__ tile_ad,
                                                                   int* __restrict__ slot_row) {
  extern __shared__ int hist[];  // [n + 2] counts, then [16] per-wave sums
  constexpr int NW = kRouteThreads / 64;
  int* red = hist + n + 2;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int me = blockIdx.x;
  for (int i = tid; i < n + 2; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  auto group = [&](int id) { return id < 0 ? n : (id >= n ? n + 1 : id); };
  for (int t = tid; t < T; t += kRouteThreads) atomicAdd(&hist[group(ids[t])], 1);
  __syncthreads();
  int before = 0;
  for (int i = tid; i < me; i += kRouteThreads) before += (hist[i] + kTile - 1) / kTile;
  for (int off = 32; off > 0; off >>= 1) before += __shfl_xor(before, off);
  if (lane == 0) red[wave] = before;
  __syncthreads();
  int tile0 = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) tile0 += red[w];
  const int count = hist[me], tiles = (count + kTile - 1) / kTile;
  if (tid == 0) {
    tile_off[me] = tile0;
    if (me == n + 1) tile_off[n + 2] = tile0 + tiles;
  }
  for (int i = tid; i < tiles; i += kRouteThreads) tile_ad[tile0 + i] = me < n ? me : n - 1 - me;  // -1, -2
  for (int i = count + tid; i < tiles * kTile; i += kRouteThreads) slot_row[(int64_t)tile0 * kTile + i] = -1;
  // each wave lists the tokens of its own stretch behind those of the waves before it
  const int per = ((T + NW - 1) / NW + 63) / 64 * 64;
  const int t0 = wave * per, t1 = min(T, t0 + per);
  int mine = 0;
  for (int t = t0; t < t1; t += 64) mine += __popcll(__ballot(t + lane < t1 && group(ids[t + lane]) == me));
  __syncthreads();  // red is read above
  if (lane == 0) red[wave] = mine;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < wave; ++w) at += red[w];
  for (int t = t0; t < t1; t += 64) {
    const bool hit = t + lane < t1 && group(ids[t + lane]) == me;
    const unsigned long long m = __ballot(hit);
    if (hit) slot_row[(int64_t)tile0 * kTile + at + __popcll(m & ((1ull << lane) - 1))] = t + lane;
    at += __popcll(m);
  }
}

// The rows of a tile as a workgroup sees them.
struct Rows {
  int ad;    // the adapter, -1: none, -2: an id out of range
  int row;   // this lane's row (slot lane % 16 of the 16-slot group), -1: none
};

// Calls of up to 64 tokens: token t stands for its group when its place among
// the tokens of the same adapter is a multiple of 16; the group's rows are that
// token and the next 15 of them.  False: another token stands for t's group.
__device__ inline bool direct_rows(const int32_t* __restrict__ ids, int T, int n, int t, Rows& g) {
  const int lane = threadIdx.x % 64;
  const int id = lane < T ? ids[lane] : 0;
  const int key = lane >= T ? -3 : (id < 0 ? -1 : (id >= n ? -2 : id));
  const int mykey = __builtin_amdgcn_readlane(key, t);
  unsigned long long m = __ballot(key == mykey);
  if (__popcll(m & ((1ull << t) - 1)) % 16 != 0) return false;
  m &= ~0ull << t;
  g.ad = mykey;
  g.row = -1;
  const int c = lane % 16;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int b = m ? (int)__ffsll(m) - 1 : -1;
    if (k == c) g.row = b;
    m &= m - 1;
  }
  return true;
}

// ---------------------------------------------------------------- shrink
// h[slot][k] = sum_j W[k][j] x[row][j] over a span of j (TW: W stored [j][k]).
// A workgroup takes MT groups of 16 slots of one adapter and 16 NT rank rows;
// its four waves take 64-deep steps of the span in turn and add their sums
// through LDS in wave order.
struct ShrinkArgs {
  const void* x;       // [T][d]
  const void* w;       // adapters stride_w apart, rows ldw apart
  int64_t d, ldw, stride_w;
  const int32_t* ids;
  const int* tile_ad;   // null: direct (T <= 64)
  const int* tile_off;  // [n + 3]
  const int* slot_row;
  int T, n, r, rp;
  int64_t span;        // reduction span of a workgroup (a multiple of 256, or all)
  int64_t nslots;
  float* hpart;        // [spans][nslots][rp]
};

template <typename F, typename EX, typename EW, bool TW, int MT, int NT, bool TAIL>
__device__ inline void shrink_step(const EX* (&xp)[MT], const EW* (&wp)[NT], int64_t ldw, int64_t j, int64_t j1, int q,
                                   f32x4 (&acc)[MT][NT]) {
  // 64-deep step: lane group q takes elements 16q .. 16q+15 as two fragments
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t at = j + 16 * q + 8 * s;
    const int64_t nv = TAIL ? j1 - at : 8;
    Frag<F> xf[MT], wf[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xf[m] = load8<F, EX>(xp[m] + at, nv);
#pragma unroll
    for (int k = 0; k < NT; ++k)
      wf[k] = TW ? load8s<F, EW>(wp[k] + at * ldw, ldw, nv) : load8<F, EW>(wp[k] + at, nv);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int k = 0; k < NT; ++k) mma(wf[k], xf[m], acc[m][k]);
  }
}

template <typename EX, typename EW>
struct FragOf {
  typedef float type;
};
template <>
struct FragOf<Bf16, Bf16> {
  typedef Bf16 type;
};

template <typename EX, typename EW, bool TW, int MT, int NT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(ShrinkArgs p) {
  typedef typename FragOf<EX, EW>::type F;
  __shared__ float part[4][MT * NT][4][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, c = lane % 16;
  Rows g[MT];
  int64_t slot0;
  if (MT == 1) {  // direct: slots are the tokens themselves
    if (!direct_rows(p.ids, p.T, p.n, (int)blockIdx.x, g[0]) || g[0].ad < 0) return;
    slot0 = 0;
  } else {
    const int tile = (int)blockIdx.x;
    if (tile >= p.tile_off[p.n]) return;  // tiles without an adapter have no h
    slot0 = (int64_t)tile * kTile;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      g[m].ad = p.tile_ad[tile];
      g[m].row = p.slot_row[slot0 + 16 * m + c];
    }
  }
  const int ad = __builtin_amdgcn_readfirstlane(g[0].ad);
  const int first = __builtin_amdgcn_readfirstlane(g[0].row);  // slot 0 always has a row
  const int k0 = (int)blockIdx.z * 16 * NT;
  const EX* xp[MT];
  const EW* wp[NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = static_cast<const EX*>(p.x) + (int64_t)(g[m].row < 0 ? first : g[m].row) * p.d;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const int kr = min(k0 + 16 * k + c, p.r - 1);
    wp[k] = static_cast<const EW*>(p.w) + ad * p.stride_w + (TW ? (int64_t)kr : kr * p.ldw);
  }
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int k = 0; k < NT; ++k) acc[m][k] = zero4();
  const int64_t j0 = (int64_t)blockIdx.y * p.span, j1 = imin(p.d, j0 + p.span);
  int64_t j = j0 + 64 * wave;
#pragma unroll 2
  for (; j + 64 <= j1; j += 256) shrink_step<F, EX, EW, TW, MT, NT, false>(xp, wp, p.ldw, j, j1, q, acc);
  if (j < j1) shrink_step<F, EX, EW, TW, MT, NT, true>(xp, wp, p.ldw, j, j1, q, acc);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][m * NT + k][i][lane] = acc[m][k][i];
  __syncthreads();
  // the wave's share of the MT x NT blocks
  float* out = p.hpart + (int64_t)blockIdx.y * p.nslots * p.rp;
#pragma unroll
  for (int b = 0; b < MT * NT; ++b) {
    if (b % 4 != wave) continue;
    const int m = b / NT, k = b % NT;
    const int kr = k0 + 16 * k + 4 * q;
    if (kr >= p.rp) continue;
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = ((part[0][b][i][lane] + part[1][b][i][lane]) + part[2][b][i][lane]) + part[3][b][i][lane];
      v[i] = g[m].row >= 0 && kr + i < p.r ? s : 0.0f;
    }
    if (MT == 1) {
      if (g[0].row >= 0) *reinterpret_cast<f32x4*>(out + (int64_t)g[0].row * p.rp + kr) = v;
    } else {
      *reinterpret_cast<f32x4*>(out + (slot0 + 16 * m + c) * p.rp + kr) = v;
    }
  }
}

// ---------------------------------------------------------------- join
// h[slot][k] = scale * sum over spans, in order; ht is its transpose.  Either
// may be null.
__global__ __launch_bounds__(256) void lora_join_kernel(const float* __restrict__ hpart, int spans, int64_t nslots, int rp,
                                                        const float* __restrict__ scale, const int* __restrict__ tile_ad,
                                                        const int* __restrict__ tile_off, int n, float* __restrict__ h,
                                                        float* __restrict__ ht) {
  const int tile = (int)blockIdx.x;
  if (tile >= tile_off[n]) return;
  const float sc = scale[tile_ad[tile]];
  for (int i = threadIdx.x; i < kTile * rp / 4; i += 256) {
    const int64_t slot = (int64_t)tile * kTile + i % kTile;
    const int k = i / kTile * 4;
    f32x4 v = *reinterpret_cast<const f32x4*>(hpart + slot * rp + k);
    for (int s = 1; s < spans; ++s) v += *reinterpret_cast<const f32x4*>(hpart + ((int64_t)s * nslots + slot) * rp + k);
    v *= sc;
    if (h) *reinterpret_cast<f32x4*>(h + slot * rp + k) = v;
    if (ht)
#pragma unroll
      for (int e = 0; e < 4; ++e) ht[(int64_t)(k + e) * nslots + slot] = v[e];
  }
}

// ---------------------------------------------------------------- expand
// y[row][j] = base[row][j] + sum_k W[j][k] h[slot][k] (TW: W stored [k][j]).
// A wave takes 128 columns: eight 16x16 tiles, tile v holding columns 8c + v,
// so that lane (q, c) ends with 8 consecutive columns of row c for each i.
struct ExpandArgs {
  const float* h;       // [nslots][rp]; direct: [spans][nslots][rp] partial sums
  const void* w;
  int64_t d, ldw, stride_w;
  const float* scale;   // direct only
  const int32_t* ids;
  const int* tile_ad;
  const int* tile_off;
  const int* slot_row;
  int T, n, r, rp, spans;
  int64_t nslots;
  int tiles_per_wg;
  const float* base;    // [T][d] or null
  float* y;             // [T][d]
};

template <typename EW, bool TW>
__device__ inline void expand_weights(const ExpandArgs& p, int ad, int64_t n0, int kb, int q, int c, Frag<EW> (&w)[8]) {
  const EW* base = static_cast<const EW*>(p.w) + ad * p.stride_w;
  const int k = 32 * kb + 8 * q;
  if constexpr (TW) {  // rows k, columns j consecutive: 8 rows of 8 columns, transposed in registers
    Frag<EW> in[8];
    const int64_t j = n0 + 8 * c;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t nv = k + e < p.r ? p.d - j : 0;
      in[e] = load8<EW, EW>(base + (k + e) * p.ldw + j, nv);
    }
    transpose8(in, w);
  } else {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const int64_t j = n0 + 8 * c + v;
      w[v] = load8<EW, EW>(base + j * p.ldw + k, j < p.d ? p.r - k : 0);
    }
  }
}

template <typename EW, bool TW, bool DIRECT>
__global__ __launch_bounds__(256) void lora_expand_kernel(ExpandArgs p) {
  const int lane = threadIdx.x % 64, q = lane / 16, c = lane % 16;
  const int64_t n0 = ((int64_t)blockIdx.y * 4 + threadIdx.x / 64) * 128;
  if (n0 >= p.d) return;
  const int kbs = (p.r + 31) / 32;
  Frag<EW> w[8];
  int have = -1;  // adapter whose factors w holds (one 32-deep block only)
  const int ntiles = DIRECT ? 1 : p.tile_off[p.n + 2];
  const int t_begin = DIRECT ? 0 : (int)blockIdx.x * p.tiles_per_wg;
  const int t_end = DIRECT ? 1 : min(ntiles, t_begin + p.tiles_per_wg);
  for (int tile = t_begin; tile < t_end; ++tile) {
#pragma unroll 1
    for (int sub = 0; sub < (DIRECT ? 1 : kTile / 16); ++sub) {
      Rows g;
      int64_t slot;
      if (DIRECT) {
        if (!direct_rows(p.ids, p.T, p.n, (int)blockIdx.x, g)) return;
        slot = imax(g.row, 0);
      } else {
        slot = (int64_t)tile * kTile + 16 * sub + c;
        g.ad = p.tile_ad[tile];
        g.row = p.slot_row[slot];
        if (__ballot(g.row >= 0) == 0) break;
      }
      const int ad = __builtin_amdgcn_readfirstlane(g.ad);
      f32x4 acc[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) acc[v] = zero4();
      if (ad >= 0) {
        for (int kb = 0; kb < kbs; ++kb) {
          if (kbs > 1 || have != ad) expand_weights<EW, TW>(p, ad, n0, kb, q, c, w);
          have = ad;
          float hv[8];
          const int k = 32 * kb + 8 * q;
#pragma unroll
          for (int e = 0; e < 8; ++e) hv[e] = 0.0f;
          if (k < p.rp && g.row >= 0) {
            for (int s = 0; s < (DIRECT ? p.spans : 1); ++s) {
              const float* hp = p.h + (s * p.nslots + slot) * p.rp + k;
              const f32x4 a = *reinterpret_cast<const f32x4*>(hp), b = *reinterpret_cast<const f32x4*>(hp + 4);
#pragma unroll
              for (int e = 0; e < 4; ++e) hv[e] += a[e], hv[4 + e] += b[e];
            }
            if (DIRECT) {
              const float sc = p.scale[ad];
#pragma unroll
              for (int e = 0; e < 8; ++e) hv[e] *= sc;
            }
          }
          Wide<EW> hw;
          widen(hv, hw);
#pragma unroll
          for (int v = 0; v < 8; ++v) mma(w[v], hw, acc[v]);
        }
      }
      if (g.row < 0) continue;
      const float* bp = p.base ? p.base + (int64_t)g.row * p.d : nullptr;
      float* yp = p.y + (int64_t)g.row * p.d;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t j = n0 + (4 * q + i) * 8;
        float o[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) o[v] = ad == -2 ? __builtin_nanf("") : acc[v][i];
        if (j + 8 <= p.d) {
          f32x4 lo = {o[0], o[1], o[2], o[3]}, hi = {o[4], o[5], o[6], o[7]};
          if (bp) {
            lo += *reinterpret_cast<const f32x4u*>(bp + j);
            hi += *reinterpret_cast<const f32x4u*>(bp + j + 4);
          }
          *reinterpret_cast<f32x4u*>(yp + j) = lo;
          *reinterpret_cast<f32x4u*>(yp + j + 4) = hi;
        } else {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            if (j + v < p.d) yp[j + v] = (bp ? bp[j + v] : 0.0f) + o[v];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- factor gradients
// The sum over an adapter's tokens of x_t (128 columns of a workgroup) times
// ht (16 NT rank rows).  Lane (q, c) loads 8 consecutive columns 8c .. of the
// rows of slots 8q .. 8q+7 of a tile and transposes them in registers, so tile v
// of the eight holds columns 8c + v.  The four waves take tiles in turn and add
// their sums through LDS in wave order.
// DB false: out[k][j] (dA: x and dh), true: out[j][k] (dB: g and h).
struct WgradArgs {
  const void* x;     // [T][d]
  const float* ht;   // [rp][nslots]
  const int* tile_off;
  const int* slot_row;
  int64_t d, nslots;
  int n, r;
  int chunks;        // token chunks (blockIdx.z / rank blocks)
  float* out;        // [chunks][n][r][d] or [chunks][n][d][r]
};

template <typename EX, int NT, bool DB>
__global__ __launch_bounds__(256) void lora_wgrad_kernel(WgradArgs p) {
  __shared__ float part[4][8][4][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, q = lane / 16, c = lane % 16;
  const int64_t n0 = (int64_t)blockIdx.x * 128;
  const int ad = (int)blockIdx.y;
  const int chunk = (int)blockIdx.z % p.chunks, k0 = (int)blockIdx.z / p.chunks * 16 * NT;
  const int a0 = p.tile_off[ad], a1 = p.tile_off[ad + 1];
  const int per = (a1 - a0 + p.chunks - 1) / p.chunks;
  const int t0 = a0 + chunk * per, t1 = min(a1, t0 + per);
  f32x4 acc[8][NT];
#pragma unroll
  for (int v = 0; v < 8; ++v)
#pragma unroll
    for (int k = 0; k < NT; ++k) acc[v][k] = zero4();
  const int64_t j = n0 + 8 * c;
  for (int tile = t0 + wave; tile < t1; tile += 4) {
    const int* rows = p.slot_row + (int64_t)tile * kTile + 8 * q;
    Frag<EX> in[8], xf[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int row = rows[e];
      in[e] = load8<EX, EX>(static_cast<const EX*>(p.x) + (int64_t)row * p.d + j, row >= 0 ? p.d - j : 0);
    }
    transpose8(in, xf);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int kr = min(k0 + 16 * k + c, p.r - 1);
      const float* hp = p.ht + (int64_t)kr * p.nslots + (int64_t)tile * kTile + 8 * q;
      float hv[8];
      const f32x4 a = *reinterpret_cast<const f32x4*>(hp), b = *reinterpret_cast<const f32x4*>(hp + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) hv[e] = a[e], hv[4 + e] = b[e];
      Wide<EX> hw;
      widen(hv, hw);
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        if constexpr (DB)
          mma(hw, xf[v], acc[v][k]);
        else
          mma(xf[v], hw, acc[v][k]);
      }
    }
  }
  float* out = p.out + ((int64_t)chunk * p.n + ad) * p.r * p.d;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    if (k > 0) __syncthreads();
#pragma unroll
    for (int v = 0; v < 8; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][v][i][lane] = acc[v][k][i];
    __syncthreads();
    auto sum = [&](int v, int i) {
      return ((part[0][v][i][lane] + part[1][v][i][lane]) + part[2][v][i][lane]) + part[3][v][i][lane];
    };
    if constexpr (DB) {  // lane: column 8c + v, ranks 4q .. 4q+3; wave: two of the v
      const int kr = k0 + 16 * k + 4 * q;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int v = 2 * wave + u;
        if (j + v >= p.d) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (kr + i < p.r) out[(j + v) * p.r + kr + i] = sum(v, i);
      }
    } else {  // lane: rank c, columns 8 (4q + i) ..; wave: one of the i
      const int kr = k0 + 16 * k + c;
      const int64_t jj = n0 + (4 * q + wave) * 8;
      if (kr < p.r)
#pragma unroll
        for (int v = 0; v < 8; ++v)
          if (jj + v < p.d) out[(int64_t)kr * p.d + jj + v] = sum(v, wave);
    }
  }
}

// out[i] = sum over chunks of part[chunk][i], in order
__global__ __launch_bounds__(256) void lora_sum_kernel(const float* __restrict__ part, int chunks, int64_t count,
                                                       float* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    float v = part[i];
    for (int s = 1; s < chunks; ++s) v += part[(int64_t)s * count + i];
    out[i] = v;
  }
}

// ---------------------------------------------------------------- host side

int64_t max_tiles(int64_t n, int64_t T) { return T / kTile + imin(n + 2, T); }

// Spans of a shrink's reduction: enough workgroups for the chip, at least 256
// elements (one 64-deep step per wave) each.
constexpr int64_t kWantGroups = 768;
int shrink_spans(int64_t groups, int64_t d) {
  return (int)imax(1, imin(imin(cdiv(kWantGroups, groups), cdiv(d, 512)), 16));
}
int64_t span_len(int64_t d, int spans) { return round_up(cdiv(d, spans), 256); }

struct LoraLayout {
  bool direct;
  int64_t tiles, nslots;
  int rp, nt, kblocks, spans_x, spans_g, chunks_a, chunks_b;
  size_t off_toff, off_tad, off_rows, off_hp, off_h, off_gp, off_dh, off_ht, off_dht, off_pa, off_pb, bytes;
};

int wgrad_chunks(int64_t n, int64_t d, int64_t T, int kblocks) {
  const int64_t wgs = n * cdiv(d, 128) * kblocks;
  return (int)imax(1, imin(imin(512 / wgs, T / (n * 8 * kTile)), 16));
}

LoraLayout lora_layout(const nq_lora& P, int64_t T, bool grads) {
  LoraLayout L{};
  L.direct = !grads && T <= 64;
  L.tiles = max_tiles(P.n, T);
  L.nslots = L.direct ? T : L.tiles * kTile;
  L.rp = (int)round_up(P.r, 16);
  L.nt = (int)imin(L.rp / 16, 4);
  if (L.nt == 3) L.nt = 4;
  L.kblocks = (int)cdiv(L.rp, 16 * L.nt);
  // tiles in use lie between T / 32 and the maximum: the spans go by the former
  const int64_t groups = (L.direct ? T : cdiv(T, kTile)) * L.kblocks;
  L.spans_x = shrink_spans(groups, P.d_in);
  L.spans_g = shrink_spans(groups, P.d_out);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  if (!L.direct) {
    L.off_toff = take((size_t)(P.n + 3) * sizeof(int));
    L.off_tad = take((size_t)L.tiles * sizeof(int));
    L.off_rows = take((size_t)L.nslots * sizeof(int));
  }
  const size_t hb = (size_t)L.nslots * L.rp * sizeof(float);
  L.off_hp = take(L.spans_x * hb);
  if (!grads) {
    if (!L.direct) L.off_h = take(hb);
  } else {
    L.off_gp = take(L.spans_g * hb);
    L.off_dh = take(hb);
    L.off_ht = take(hb);
    L.off_dht = take(hb);
    L.chunks_a = wgrad_chunks(P.n, P.d_in, T, L.kblocks);
    L.chunks_b = wgrad_chunks(P.n, P.d_out, T, L.kblocks);
    const size_t per = (size_t)P.n * P.r * sizeof(float);
    if (L.chunks_a > 1) L.off_pa = take(L.chunks_a * per * P.d_in);
    if (L.chunks_b > 1) L.off_pb = take(L.chunks_b * per * P.d_out);
  }
  L.bytes = off;
  return L;
}

template <typename EX, typename EW, bool TW>
hipError_t launch_shrink(const ShrinkArgs& a, const LoraLayout& L, int spans, hipStream_t s) {
  const dim3 grid((unsigned)(L.direct ? L.nslots : L.tiles), (unsigned)spans, (unsigned)L.kblocks);
#define NQ_SHRINK(MT, NT) hipLaunchKernelGGL((lora_shrink_kernel<EX, EW, TW, MT, NT>), grid, dim3(256), 0, s, a)
  if (L.direct) {
    if constexpr (!TW) {
      if (L.nt == 1)
        NQ_SHRINK(1, 1);
      else if (L.nt == 2)
        NQ_SHRINK(1, 2);
      else
        NQ_SHRINK(1, 4);
    }
  } else {
    if (L.nt == 1)
      NQ_SHRINK(2, 1);
    else if (L.nt == 2)
      NQ_SHRINK(2, 2);
    else
      NQ_SHRINK(2, 4);
  }
#undef NQ_SHRINK
  return hipGetLastError();
}

template <bool TW>
hipError_t launch_shrink_types(const ShrinkArgs& a, const LoraLayout& L, int spans, nq_dtype xd, nq_dtype wd,
                               hipStream_t s) {
  if (xd == NQ_BF16)
    return wd == NQ_BF16 ? launch_shrink<Bf16, Bf16, TW>(a, L, spans, s) : launch_shrink<Bf16, float, TW>(a, L, spans, s);
  return wd == NQ_BF16 ? launch_shrink<float, Bf16, TW>(a, L, spans, s) : launch_shrink<float, float, TW>(a, L, spans, s);
}

template <bool TW, bool DIRECT>
hipError_t launch_expand(ExpandArgs a, const LoraLayout& L, nq_dtype wd, hipStream_t s) {
  const int64_t cols = cdiv(a.d, 512);
  // tiles of a workgroup: more keep the factors in registers for longer, fewer
  // fill the chip
  a.tiles_per_wg = (int)imax(1, imin(4, L.tiles * cols / 1024));
  const dim3 grid((unsigned)(DIRECT ? a.T : cdiv(L.tiles, a.tiles_per_wg)), (unsigned)cols);
  if (wd == NQ_BF16)
    hipLaunchKernelGGL((lora_expand_kernel<Bf16, TW, DIRECT>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((lora_expand_kernel<float, TW, DIRECT>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <bool DB>
hipError_t launch_wgrad(const WgradArgs& a, const LoraLayout& L, nq_dtype xd, hipStream_t s) {
  const dim3 grid((unsigned)cdiv(a.d, 128), (unsigned)a.n, (unsigned)(L.kblocks * a.chunks));
#define NQ_WGRAD(E, NT) hipLaunchKernelGGL((lora_wgrad_kernel<E, NT, DB>), grid, dim3(256), 0, s, a)
  if (xd == NQ_BF16) {
    if (L.nt == 1)
      NQ_WGRAD(Bf16, 1);
    else if (L.nt == 2)
      NQ_WGRAD(Bf16, 2);
    else
      NQ_WGRAD(Bf16, 4);
  } else {
    if (L.nt == 1)
      NQ_WGRAD(float, 1);
    else if (L.nt == 2)
      NQ_WGRAD(float, 2);
    else
      NQ_WGRAD(float, 4);
  }
#undef NQ_WGRAD
  return hipGetLastError();
}

hipError_t launch_route(const int32_t* ids, int64_t T, int64_t n, const LoraLayout& L, char* ws, hipStream_t s) {
  hipLaunchKernelGGL(lora_route_kernel, dim3((unsigned)(n + 2)), dim3(kRouteThreads),
                     (size_t)(n + 2 + kRouteThreads / 64) * sizeof(int), s, ids, (int)T, (int)n,
                     reinterpret_cast<int*>(ws + L.off_toff), reinterpret_cast<int*>(ws + L.off_tad),
                     reinterpret_cast<int*>(ws + L.off_rows));
  return hipGetLastError();
}

ShrinkArgs shrink_args(const nq_lora& P, const LoraLayout& L, char* ws, const void* x, const void* w, int64_t d,
                       int64_t ldw, int64_t stride_w, const int32_t* ids, int64_t T, int spans, size_t off_out) {
  ShrinkArgs a;
  a.x = x;
  a.w = w;
  a.d = d;
  a.ldw = ldw;
  a.stride_w = stride_w;
  a.ids = ids;
  a.tile_ad = reinterpret_cast<const int*>(ws + L.off_tad);
  a.tile_off = reinterpret_cast<const int*>(ws + L.off_toff);
  a.slot_row = reinterpret_cast<const int*>(ws + L.off_rows);
  a.T = (int)T;
  a.n = (int)P.n;
  a.r = (int)P.r;
  a.rp = L.rp;
  a.span = span_len(d, spans);
  a.nslots = L.nslots;
  a.hpart = reinterpret_cast<float*>(ws + off_out);
  return a;
}

hipError_t launch_join(const nq_lora& P, const LoraLayout& L, char* ws, size_t off_part, int spans, float* h, float* ht,
                       hipStream_t s) {
  hipLaunchKernelGGL(lora_join_kernel, dim3((unsigned)L.tiles), dim3(256), 0, s,
                     reinterpret_cast<const float*>(ws + off_part), spans, L.nslots, L.rp, P.scale,
                     reinterpret_cast<const int*>(ws + L.off_tad), reinterpret_cast<const int*>(ws + L.off_toff), (int)P.n,
                     h, ht);
  return hipGetLastError();
}

ExpandArgs expand_args(const nq_lora& P, const LoraLayout& L, char* ws, const float* h, const void* w, int64_t d,
                       int64_t ldw, int64_t stride_w, const int32_t* ids, int64_t T, const float* base, float* y) {
  ExpandArgs a;
  a.h = h;
  a.w = w;
  a.d = d;
  a.ldw = ldw;
  a.stride_w = stride_w;
  a.scale = P.scale;
  a.ids = ids;
  a.tile_ad = reinterpret_cast<const int*>(ws + L.off_tad);
  a.tile_off = reinterpret_cast<const int*>(ws + L.off_toff);
  a.slot_row = reinterpret_cast<const int*>(ws + L.off_rows);
  a.T = (int)T;
  a.n = (int)P.n;
  a.r = (int)P.r;
  a.rp = L.rp;
  a.spans = L.spans_x;
  a.nslots = L.nslots;
  a.tiles_per_wg = 1;
  a.base = base;
  a.y = y;
  return a;
}

}  // namespace

size_t lora_workspace(const nq_lora& P, int64_t T, bool grads) { return lora_layout(P, T, grads).bytes; }

hipError_t launch_lora_linear(const nq_lora& P, const void* x, nq_dtype xd, const int32_t* ids, int64_t T,
                              const float* base, float* y, void* workspace, hipStream_t s) {
  const LoraLayout L = lora_layout(P, T, false);
  char* ws = static_cast<char*>(workspace);
  hipError_t e = hipSuccess;
  if (!L.direct) e = launch_route(ids, T, P.n, L, ws, s);
  if (e != hipSuccess) return e;
  const ShrinkArgs sa =
      shrink_args(P, L, ws, x, P.a, P.d_in, P.lda, P.stride_a, ids, T, L.spans_x, L.off_hp);
  if ((e = launch_shrink_types<false>(sa, L, (int)cdiv(P.d_in, sa.span), xd, P.dtype, s)) != hipSuccess) return e;
  const float* h = sa.hpart;
  if (!L.direct) {
    float* hj = reinterpret_cast<float*>(ws + L.off_h);
    if ((e = launch_join(P, L, ws, L.off_hp, (int)cdiv(P.d_in, sa.span), hj, nullptr, s)) != hipSuccess) return e;
    h = hj;
  }
  ExpandArgs ea = expand_args(P, L, ws, h, P.b, P.d_out, P.ldb, P.stride_b, ids, T, base, y);
  ea.spans = (int)cdiv(P.d_in, sa.span);
  return L.direct ? launch_expand<false, true>(ea, L, P.dtype, s) : launch_expand<false, false>(ea, L, P.dtype, s);
}

hipError_t launch_lora_grads(const nq_lora& P, const void* x, nq_dtype xd, const void* g, nq_dtype gd,
                             const int32_t* ids, int64_t T, const float* dx_base, float* dx, float* da, float* db,
                             void* workspace, hipStream_t s) {
  const LoraLayout L = lora_layout(P, T, true);
  char* ws = static_cast<char*>(workspace);
  float* ht = reinterpret_cast<float*>(ws + L.off_ht);
  float* dh = reinterpret_cast<float*>(ws + L.off_dh);
  float* dht = reinterpret_cast<float*>(ws + L.off_dht);
  hipError_t e = launch_route(ids, T, P.n, L, ws, s);
  if (e != hipSuccess) return e;
  const ShrinkArgs sx =
      shrink_args(P, L, ws, x, P.a, P.d_in, P.lda, P.stride_a, ids, T, L.spans_x, L.off_hp);
  if ((e = launch_shrink_types<false>(sx, L, (int)cdiv(P.d_in, sx.span), xd, P.dtype, s)) != hipSuccess) return e;
  const ShrinkArgs sg =
      shrink_args(P, L, ws, g, P.b, P.d_out, P.ldb, P.stride_b, ids, T, L.spans_g, L.off_gp);
  if ((e = launch_shrink_types<true>(sg, L, (int)cdiv(P.d_out, sg.span), gd, P.dtype, s)) != hipSuccess) return e;
  if ((e = launch_join(P, L, ws, L.off_hp, (int)cdiv(P.d_in, sx.span), nullptr, ht, s)) != hipSuccess) return e;
  if ((e = launch_join(P, L, ws, L.off_gp, (int)cdiv(P.d_out, sg.span), dh, dht, s)) != hipSuccess) return e;
  const ExpandArgs ea = expand_args(P, L, ws, dh, P.a, P.d_in, P.lda, P.stride_a, ids, T, dx_base, dx);
  if ((e = launch_expand<true, false>(ea, L, P.dtype, s)) != hipSuccess) return e;
  WgradArgs wa;
  wa.tile_off = ea.tile_off;
  wa.slot_row = ea.slot_row;
  wa.nslots = L.nslots;
  wa.n = (int)P.n;
  wa.r = (int)P.r;
  for (int side = 0; side < 2; ++side) {
    float* out = side ? db : da;
    wa.d = side ? P.d_out : P.d_in;
    wa.x = side ? g : x;
    wa.ht = side ? ht : dht;
    wa.chunks = side ? L.chunks_b : L.chunks_a;
    float* part = reinterpret_cast<float*>(ws + (side ? L.off_pb : L.off_pa));
    wa.out = wa.chunks > 1 ? part : out;
    e = side ? launch_wgrad<true>(wa, L, gd, s) : launch_wgrad<false>(wa, L, xd, s);
    if (e != hipSuccess) return e;
    if (wa.chunks > 1) {
      const int64_t count = P.n * P.r * wa.d;
      hipLaunchKernelGGL(lora_sum_kernel, dim3((unsigned)imin(cdiv(count, 256), 2048)), dim3(256), 0, s, part, wa.chunks,
                         count, out);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace nq
