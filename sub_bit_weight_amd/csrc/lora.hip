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
// fewer bits than fp32 (but for values below 2^-110, whose bits under bf16's
// smallest, 2^-133, are lost).  Sums have a fixed order; there are no
// atomics on floating data.
//
// A load of 16 bytes per lane costs a cache access per line that 16 neighbouring
// lanes touch, and a fragment's 16 neighbours lie in 16 different rows.  Rows
// therefore go through LDS (shrink, expand) or are loaded along columns and
// transposed in registers (factor gradients), and the hidden vectors are stored
// in the order in which fragments read them.
//
// Rows and columns of a matrix product do not mix: slots without a row and
// rank rows past r load some valid address and are set to zero when stored;
// only tails of a reduction need zero operands.  A 16x16 tile's rows may stand
// for any rows of the operand, so each kernel assigns them such that lanes load
// and store 8 or 16 consecutive bytes.
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

// v = t0 + t1 + t2 exactly for |v| >= 2^-110: each term takes the next 8 bits of the
// significand (truncated, so no term rounds and all have v's sign).  From 2^-100 on
// no term is zero, which an infinite factor would turn into NaN where the product is
// infinite: a value of fewer bits is cut into halves.  An infinity is three; a NaN
// that arithmetic made has its quiet bit in the upper half and stays one.
__device__ inline void split3(float v, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  float a = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), rest = v - a;
  float b = __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u), c = rest - b;
  if (__builtin_isinf(v)) {
    b = c = v;
  } else if (__builtin_fabsf(v) >= 0x1p-100f) {
    if (rest == 0.0f) {
      a = 0.5f * v;
      b = c = 0.25f * v;
    } else if (c == 0.0f) {
      b = c = 0.5f * b;
    }
  }
  t0 = __float_as_uint(a);
  t1 = __float_as_uint(b);
  t2 = __float_as_uint(c);
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

// Elements k .. k + 7 of a row of r, zero past its end.  bf16 whose end lies among
// them (and r > 8): the row's last eight, shifted into place, one load instead of
// one per element (2048 tokens, rank 12, 4096 x 4096: 36 us, by elements 41).  fp32
// by elements: shifting its eight words costs more (133 tokens, rank 18, 64 ->
// 5616: 25 us, shifted 28).
__device__ inline Frag<float> load8_row(const float* row, int k, int r) { return load8<float, float>(row + k, r - k); }
__device__ inline Frag<Bf16> load8_row(const Bf16* row, int k, int r) {
  if (r % 8 == 0 || r < 8) return load8<Bf16, Bf16>(row + k, r - k);
  if (k >= r) return load8<Bf16, Bf16>(row, 0);
  const int at = min(k, r - 8), n = k - at;
  Frag<Bf16> f = load8<Bf16, Bf16>(row + at, 8);
  uint64_t lo = (uint64_t)f.d[1] << 32 | f.d[0], hi = (uint64_t)f.d[3] << 32 | f.d[2];
  if (n & 1) lo = lo >> 16 | hi << 48, hi >>= 16;
  if (n & 2) lo = lo >> 32 | hi << 32, hi >>= 32;
  if (n & 4) lo = hi, hi = 0;
  f.d = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  return f;
}

__device__ inline float element(const Frag<float>& f, int e) { return f.v[e]; }
__device__ inline float element(const Frag<Bf16>& f, int e) {
  return __uint_as_float(e % 2 ? f.d[e / 2] & 0xFFFF0000u : f.d[e / 2] << 16);
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
// tokens in order.  A wave owns a stretch of tokens, whose groups stay in
// registers between the two passes (up to 16384 tokens; the rest is read again).
// A chain of round trips: 5 us for 2048 tokens, 10 us for 8192.
__global__ __launch_bounds__(kRouteThreads) void lora_route_kernel(const int32_t* __restrict__ ids, int T, int n,
                                                                   int* __restrict__ tile_off, int* __restrict__ tile_ad,
                                                                   int* __restrict__ slot_row, int* __restrict__ arrived,
                                                                   int per_tile) {
  extern __shared__ int hist[];  // [n + 2] counts, then [16] per-wave sums
  constexpr int NW = kRouteThreads / 64, HELD = 16;
  int* red = hist + n + 2;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int me = blockIdx.x;
  const int per = ((T + NW - 1) / NW + 63) / 64 * 64;
  const int t0 = wave * per, t1 = min(T, t0 + per);
  auto group = [&](int id) { return id < 0 ? n : (id >= n ? n + 1 : id); };
  int held[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int t = t0 + 64 * i + lane;
    held[i] = t < t1 ? group(ids[t]) : -1;
  }
  for (int i = tid; i < n + 2; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  int mine = 0;
  auto count = [&](int g) {
    // neighbours usually share a group: the first lane's is counted at once
    const int g0 = __builtin_amdgcn_readfirstlane(g);
    const unsigned long long same = __ballot(g == g0);
    if (lane == 0 && g0 >= 0) atomicAdd(&hist[g0], __popcll(same));
    if (g != g0 && g >= 0) atomicAdd(&hist[g], 1);
    mine += __popcll(__ballot(g == me));
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (t0 + 64 * i < t1) count(held[i]);
  for (int t = t0 + 64 * HELD; t < t1; t += 64) count(t + lane < t1 ? group(ids[t + lane]) : -1);
  __syncthreads();
  int before = 0;
  for (int i = tid; i < me; i += kRouteThreads) before += (hist[i] + kTile - 1) / kTile;
  for (int off = 32; off > 0; off >>= 1) before += __shfl_xor(before, off);
  if (lane == 0) red[wave] = before;
  __syncthreads();
  int tile0 = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) tile0 += red[w];
  __syncthreads();
  if (lane == 0) red[wave] = mine;
  __syncthreads();
  const int total = hist[me], tiles = (total + kTile - 1) / kTile;
  if (tid == 0) {
    tile_off[me] = tile0;
    if (me == n + 1) tile_off[n + 2] = tile0 + tiles;
  }
  for (int i = tid; i < tiles; i += kRouteThreads) tile_ad[tile0 + i] = me < n ? me : n - 1 - me;  // -1, -2
  for (int64_t i = tid; i < (int64_t)tiles * per_tile; i += kRouteThreads) arrived[(int64_t)tile0 * per_tile + i] = 0;
  int* rows = slot_row + (int64_t)tile0 * kTile;
  for (int i = total + tid; i < tiles * kTile; i += kRouteThreads) rows[i] = -1;
  int at = 0;
  for (int w = 0; w < wave; ++w) at += red[w];
  auto list = [&](int g, int t) {
    const unsigned long long m = __ballot(g == me);
    const int place = at + __popcll(m & ((1ull << lane) - 1));
    if (g == me && place < tiles * kTile) rows[place] = t;  // ids read again: see routed_row
    at += __popcll(m);
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (t0 + 64 * i < t1) list(held[i], t0 + 64 * i + lane);
  for (int t = t0 + 64 * HELD; t < t1; t += 64) list(t + lane < t1 ? group(ids[t + lane]) : -1, t + lane);
}

// Every routing workgroup reads ids for itself.  If a caller changes them meanwhile
// (which it must not), workgroups disagree, tiles overlap and slots or adapters of
// others are never written: whatever stands there must not become an address.  The
// number of tiles is in range all the same, since each workgroup counts T tokens.
__device__ inline int routed_row(int row, int T) { return (unsigned)row < (unsigned)T ? row : -1; }
__device__ inline bool routed_adapter(int ad, int n) { return (unsigned)ad < (unsigned)n; }

// The rows of a tile as a workgroup sees them.
struct Rows {
  int ad;    // the adapter, -1: none, -2: an id out of range
  int row;   // this lane's row (slot lane % 16 of the 16-slot group), -1: none
};

// Calls of up to 64 tokens: token t stands for its group when its place among
// the tokens of the same adapter is a multiple of G; the group's rows are that
// token and the next G - 1 of them.  False: another token stands for t's group.
template <int G>
__device__ inline bool direct_rows(const int32_t* __restrict__ ids, int T, int n, int t, Rows& g) {
  const int lane = threadIdx.x % 64;
  const int id = lane < T ? ids[lane] : 0;
  const int key = lane >= T ? -3 : (id < 0 ? -1 : (id >= n ? -2 : id));
  const int mykey = __builtin_amdgcn_readlane(key, t);
  unsigned long long m = __ballot(key == mykey);
  if (__popcll(m & ((1ull << t) - 1)) % G != 0) return false;
  m &= ~0ull << t;
  g.ad = mykey;
  g.row = -1;
  const int c = lane % 16;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int b = m ? (int)__ffsll(m) - 1 : -1;
    if (k == c) g.row = b;
    m &= m - 1;
  }
  return true;
}

// ---------------------------------------------------------------- shrink
// h[slot][k] = scale * sum_j W[k][j] x[row][j] (TW: W stored [j][k]).
// A workgroup takes MT groups of 16 slots of one adapter, 16 NT rank rows and a
// span of the reduction.  bf16 operands stream through LDS (staged_steps);
// otherwise its eight waves take 64-deep steps of the span in turn, straight
// from memory.  The waves' sums are added through LDS in wave order.  With several
// spans, each writes its sum and counts itself in; the workgroup that comes last
// adds them in span order (nobody waits).  Direct calls leave that sum to the reader.
// Bound by the rows' bytes and, for few tokens, by the chain load - multiply - sum:
// 2048 tokens of 8192, bf16, rank 16 13 us (2.6 TB/s); 8192 tokens, rank 64 53 us
// (2.5 TB/s, one workgroup of 147 KB LDS a CU); 777 tokens of 4099, fp32, rank 41
// 18 us (loads straight from rows of odd length in eight dependent steps a wave; the
// matrix cores of its 248 CUs are busy 29 % of the time, and its waves wait half of
// it; fp32 rows through LDS by loads of 4 bytes a lane: 22 us).
//
// Rank rows of the NT tiles: 16n + row, or (TW) NT * row + n, so that a lane's
// NT ranks are consecutive in a row of W.
struct ShrinkArgs {
  const void* x;       // [T][d]
  const void* w;       // adapters stride_w apart, rows ldw apart
  int64_t d, ldw, stride_w;
  const int32_t* ids;
  const int* tile_ad;
  const int* tile_off;  // [n + 3]
  const int* slot_row;
  const float* scale;
  int T, n, r, rp;     // rp: r rounded up to 32
  int64_t span;        // reduction span of a workgroup (a multiple of 64)
  int spans;
  int64_t nslots;
  float* hpart;        // [spans][nslots][rp] (spans > 1, and direct)
  int* arrived;        // [tiles][rank blocks][2], this side's (spans > 1); zeroed by the routing
  // the results as the fragments of their readers, 8 elements a lane, in fp32 or
  // as three bf16 terms (`..._term` elements apart); either may be null
  void* h;             // [16-slot groups][32-rank blocks][lane]: slot c, ranks 8q ..
  void* ht;            // [tiles][16-rank blocks][lane]: rank c, slots 8q ..
  int h_bf16, ht_bf16;
  int64_t h_term, ht_term;
  int staged;          // rows are 16-byte aligned and of whole 16-byte chunks
};

constexpr int kShrinkWaves = 8;

// Partial sums that another workgroup of the launch reads: agent-scope stores
// (they write through by themselves, where a release fence would write back
// the XCD's whole L2: 90 us instead of 13 for 2048 tokens of 8192), then, once
// every thread's stores have completed and the workgroup has met, a relaxed
// count; the last workgroup acquires before it reads.
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
    if (*s_last) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  }
  __syncthreads();
  return *s_last != 0;
}

template <typename EX, typename EW>
struct FragOf {
  typedef float type;
};
template <>
struct FragOf<Bf16, Bf16> {
  typedef Bf16 type;
};

// Ranks k .. k + NT - 1 of 8 rows of W (reduction rows at .. at + 7): one
// fragment per rank tile.  whole: those ranks exist; otherwise ranks past r
// repeat the last, loaded one by one.
template <typename F, typename E, int NT, bool TAIL>
__device__ inline void load_ranks(const E* w, int64_t ldw, int64_t at, int64_t nv, int k, int r, bool whole,
                                  Frag<F> (&f)[NT]) {
  if constexpr (sizeof(E) == 2) {
    constexpr int ND = (NT + 1) / 2;  // words of a lane's ranks
    uint32_t d[8][ND];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int i = 0; i < ND; ++i) d[e][i] = 0;
      if (TAIL && e >= nv) continue;
      const E* p = w + (at + e) * ldw;
      if (NT > 1 && whole) {
        typedef uint32_t words __attribute__((ext_vector_type(ND), aligned(2)));
        const words v = *reinterpret_cast<const words*>(p + k);
        if constexpr (ND == 1)
          d[e][0] = v[0];
        else
          d[e][0] = v[0], d[e][1] = v[1];
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) d[e][n / 2] |= (uint32_t)p[min(k + n, r - 1)].u << (16 * (n % 2));
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = __builtin_amdgcn_perm(d[2 * i + 1][n / 2], d[2 * i][n / 2], n % 2 ? 0x07060302 : 0x05040100);
        if constexpr (sizeof(F) == 2)
          f[n].d[i] = v;
        else
          f[n].v[2 * i] = __uint_as_float(v << 16), f[n].v[2 * i + 1] = __uint_as_float(v & 0xFFFF0000u);
      }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n] = 0.0f;
      if (!TAIL || e < nv) {
        const E* p = w + (at + e) * ldw;
        if (whole) {
          struct __attribute__((packed, aligned(4))) Pack {
            float v[NT];
          };
          const Pack a = *reinterpret_cast<const Pack*>(p + k);
#pragma unroll
          for (int n = 0; n < NT; ++n) v[n] = a.v[n];
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n) v[n] = to_f32(p[min(k + n, r - 1)]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) f[n].v[e] = v[n];
    }
  }
}

template <typename F, typename EX, typename EW, bool TW, int MT, int NT, bool TAIL>
__device__ inline void shrink_step(const EX* (&xp)[MT], const EW* w, const int (&wrow)[NT], const ShrinkArgs& p, int k,
                                   bool whole, int64_t j, int64_t j1, int q, f32x4 (&acc)[MT][NT]) {
  // 64-deep step: lane group q takes elements 16q .. 16q+15 as two fragments
  Frag<F> xf[2][MT], wf[2][NT];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t at = j + 16 * q + 8 * s;
    const int64_t nv = TAIL ? j1 - at : 8;
#pragma unroll
    for (int m = 0; m < MT; ++m) xf[s][m] = load8<F, EX>(xp[m] + at, nv);
    if constexpr (TW) {
      load_ranks<F, EW, NT, TAIL>(w, p.ldw, at, nv, k, p.r, whole, wf[s]);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) wf[s][n] = load8<F, EW>(w + (int64_t)wrow[n] * p.ldw + at, nv);
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) mma(wf[s][n], xf[s][m], acc[m][n]);
}

// Whole chunks of kChunk reduction elements of bf16 operands: the rows of x and
// W (nt) or rows of R ranks (TW) come by direct global->LDS loads of 1 KB a wave,
// two chunks ahead, and wave w multiplies 32-deep step w of each chunk.  A row of
// 512 bytes keeps its 16-byte piece i at i ^ (row % 16), so that the 16 rows of a
// fragment read meet 16 different bank groups.  Straight from memory the same
// loads took 68 us, this way 53 (8192 tokens of 8192, rank 64); chunks of 128 for
// the wider rank tiles, so that two workgroups share a CU, 55.
constexpr int kChunk = 256, kStages = 3;

template <bool TW, int NT>
constexpr int stage_bytes() {
  return (kTile + 16 * NT) * 512;
}

template <bool TW, int NT>
__device__ inline void staged_steps(const ShrinkArgs& p, const Bf16* x, const int* rows, const Bf16* w, int k0, int64_t j0,
                                    int chunks, char* lds, f32x4 (&acc)[2][NT]) {
  constexpr int R = 16 * NT, NW = kShrinkWaves, XL = kTile / 2 / NW, WL = R / 2 / NW, STAGE = stage_bytes<TW, NT>();
  static_assert(XL >= 1 && WL >= 1 && XL + WL < 16, "a load per wave and operand, and the wait's range");
  const int tid = threadIdx.x, lane = tid % 64, q = lane / 16, c = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const Bf16 *xa[XL], *wa[WL];
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int r = (wave * XL + i) * 2 + lane / 32;
    xa[i] = x + (int64_t)rows[r] * p.d + j0 + ((lane % 32) ^ (r % 16)) * 8;
  }
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int o = (wave * WL + i) * 1024 + lane * 16;  // byte of the staged block
    if constexpr (TW) {  // [kChunk][R ranks]; ranks past r repeat the last eight
      wa[i] = w + (j0 + o / (2 * R)) * p.ldw + min(k0 + o % (2 * R) / 2, p.r - 8);
    } else {
      const int r = o / 512;
      wa[i] = w + (int64_t)min(k0 + r, p.r - 1) * p.ldw + j0 + ((o % 512 / 16) ^ (r % 16)) * 8;
    }
  }
  const int64_t wstep = TW ? kChunk * p.ldw : kChunk;
  auto issue = [&](int ch, int st) {
    char* dst = lds + st * STAGE;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_global_load_lds((const void*)(xa[i] + (int64_t)ch * kChunk),
                                       (__attribute__((address_space(3))) void*)(dst + (wave * XL + i) * 1024), 16, 0, 0);
#pragma unroll
    for (int i = 0; i < WL; ++i)
      __builtin_amdgcn_global_load_lds(
          (const void*)(wa[i] + ch * wstep),
          (__attribute__((address_space(3))) void*)(dst + kTile * 512 + (wave * WL + i) * 1024), 16, 0, 0);
  };
  for (int ch = 0; ch < kStages - 1 && ch < chunks; ++ch) issue(ch, ch);
  int st = 0;
  for (int ch = 0; ch < chunks; ++ch) {
    // vmcnt: this chunk has landed, the next may stay in flight; lgkmcnt(0): this
    // wave's reads of the last chunk have returned, whose stage is loaded anew below
    if (ch + 1 < chunks)
      __builtin_amdgcn_s_waitcnt((XL + WL) | (7 << 4));
    else
      __builtin_amdgcn_s_waitcnt(7 << 4);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();  // the same of every wave
    asm volatile("" ::: "memory");
    if (ch + kStages - 1 < chunks) issue(ch + kStages - 1, st + kStages - 1 < kStages ? st + kStages - 1 : st - 1);
    const char* stage = lds + st * STAGE;
    Frag<Bf16> xf[2], wf[NT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
      xf[m].d = *reinterpret_cast<const u32x4*>(stage + (16 * m + c) * 512 + (((4 * wave + q) ^ c) * 16));
    const char* ws = stage + kTile * 512;
    if constexpr (TW) {
      load_ranks<Bf16, Bf16, NT, false>(reinterpret_cast<const Bf16*>(ws), R, 32 * wave + 8 * q, 8, NT * c, R, true, wf);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        wf[n].d = *reinterpret_cast<const u32x4*>(ws + (16 * n + c) * 512 + (((4 * wave + q) ^ c) * 16));
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) mma(wf[n], xf[m], acc[m][n]);
    st = st + 1 < kStages ? st + 1 : 0;
  }
  __syncthreads();  // the stages are reused
}

// v[0..7] in fp32, or as bf16 terms `term` elements apart
__device__ inline void store_frag(void* out, int bf16, int64_t term, int64_t frag, const float (&v)[8]) {
  if (bf16) {
    Wide<Bf16> w;
    widen(v, w);
#pragma unroll
    for (int t = 0; t < 3; ++t)
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + t * term + frag * 8) = w.t[t].d;
  } else {
    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + frag * 8);
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
}

template <typename EX, typename EW, bool TW, int MT, int NT>
__device__ inline void shrink(const ShrinkArgs& p, int span, float* lds) {
  typedef typename FragOf<EX, EW>::type F;
  constexpr int NW = kShrinkWaves, R = 16 * NT;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, q = lane / 16, c = lane % 16;
  Rows g[MT];
  int64_t slot0 = 0;
  int tile = 0;
  if (MT == 1) {  // direct: slots are the tokens themselves
    if (!direct_rows<16>(p.ids, p.T, p.n, (int)blockIdx.x, g[0]) || g[0].ad < 0) return;
  } else {
    tile = (int)blockIdx.x;
    if (tile >= p.tile_off[p.n]) return;  // tiles without an adapter have no h
    slot0 = (int64_t)tile * kTile;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      g[m].ad = p.tile_ad[tile];
      g[m].row = routed_row(p.slot_row[slot0 + 16 * m + c], p.T);
    }
  }
  const int ad = __builtin_amdgcn_readfirstlane(g[0].ad);
  if (MT == 2 && !routed_adapter(ad, p.n)) return;
  const int first = max(__builtin_amdgcn_readfirstlane(g[0].row), 0);  // slot 0 always has a row
  const int k0 = (int)blockIdx.z * R;
  const EX* xp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xp[m] = static_cast<const EX*>(p.x) + (int64_t)(g[m].row < 0 ? first : g[m].row) * p.d;
  const EW* w = static_cast<const EW*>(p.w) + ad * p.stride_w;
  int wrow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) wrow[n] = min(k0 + 16 * n + c, p.r - 1);
  __shared__ int rows[16 * MT];
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = zero4();
  const int64_t j0 = (int64_t)span * p.span, j1 = imin(p.d, j0 + p.span);
  int64_t js = j0;
  // a lane's NT ranks exist, or (r a multiple of NT) none does and it repeats the
  // last: no load per rank (gradients of 2048 tokens, rank 20, 4096 -> 11008: 60 us,
  // by ranks 89)
  const bool whole = k0 + R <= p.r || p.r % NT == 0;
  const int k = whole ? min(k0 + NT * c, p.r - NT) : k0 + NT * c;
  if constexpr (MT == 2 && sizeof(F) == 2) {
    const int chunks = p.staged ? (int)((j1 - j0) / kChunk) : 0;
    if (chunks > 0) {  // slots without a row load the tile's first one
      if (tid < 16 * MT) {
        const int row = routed_row(p.slot_row[slot0 + tid], p.T);
        rows[tid] = row < 0 ? first : row;
      }
      __syncthreads();
      staged_steps<TW, NT>(p, static_cast<const Bf16*>(p.x), rows, w, k0, j0, chunks, reinterpret_cast<char*>(lds), acc);
      js += (int64_t)chunks * kChunk;
    }
  }
  int64_t j = js + 64 * wave;
  if (whole || !TW) {
#pragma unroll(TW || NT == 4 ? 1 : 2)
    for (; j + 64 <= j1; j += 64 * NW)
      shrink_step<F, EX, EW, TW, MT, NT, false>(xp, w, wrow, p, k, true, j, j1, q, acc);
  }
  for (; j < j1; j += 64 * NW) shrink_step<F, EX, EW, TW, MT, NT, true>(xp, w, wrow, p, k, whole, j, j1, q, acc);
  // [wave][block][i][lane], then the sums as [slot][rank] in the same memory
#pragma unroll
  for (int b = 0; b < MT * NT; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) lds[((wave * MT * NT + b) * 4 + i) * 64 + lane] = acc[b / NT][b % NT][i];
  __syncthreads();
  float sum[(MT * NT * 4 + NW - 1) / NW];
#pragma unroll
  for (int u = 0; u < (MT * NT * 4 + NW - 1) / NW; ++u) {
    const int bi = wave + NW * u;  // block and register
    float v = 0.0f;
    if (bi < MT * NT * 4)
#pragma unroll
      for (int ww = 0; ww < NW; ++ww) v += lds[(ww * MT * NT * 4 + bi) * 64 + lane];
    sum[u] = v;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < (MT * NT * 4 + NW - 1) / NW; ++u) {
    const int bi = wave + NW * u;
    if (bi < MT * NT * 4) {
      const int b = bi / 4, row = 4 * q + bi % 4, n = b % NT, m = b / NT;
      const int rank = TW ? NT * row + n : 16 * n + row;
      const int have = MT == 1 ? g[0].row : (m == 0 ? g[0].row : g[MT - 1].row);
      lds[(16 * m + c) * (R + 1) + rank] = have >= 0 && k0 + rank < p.r ? sum[u] : 0.0f;
    }
  }
  __syncthreads();
  constexpr int SLOTS = 16 * MT, COUNT = SLOTS * R;
  if (MT == 1) {
    float* out = p.hpart + (int64_t)span * p.nslots * p.rp;
    if (tid < 16) rows[tid] = g[0].row;
    __syncthreads();
    for (int i = tid; i < COUNT; i += 64 * NW) {
      const int s = i / R, rank = i % R;
      if (rows[s] >= 0 && k0 + rank < p.rp) out[(int64_t)rows[s] * p.rp + k0 + rank] = lds[s * (R + 1) + rank];
    }
    return;
  }
  if (p.spans > 1) {
    __shared__ int last;
    for (int i = tid; i < COUNT; i += 64 * NW)
      if (k0 + i % R < p.rp)
        store_agent(p.hpart + ((int64_t)span * p.nslots + slot0 + i / R) * p.rp + k0 + i % R,
                    lds[i / R * (R + 1) + i % R]);
    if (!last_to_arrive(p.arrived + 2 * ((int64_t)tile * gridDim.z + blockIdx.z), p.spans, &last)) return;
    for (int i = tid; i < COUNT; i += 64 * NW) {
      if (k0 + i % R >= p.rp) continue;
      const float* hp = p.hpart + (slot0 + i / R) * p.rp + k0 + i % R;
      float v = 0.0f;
#pragma unroll 4
      for (int s = 0; s < p.spans; ++s) v += hp[(int64_t)s * p.nslots * p.rp];
      lds[i / R * (R + 1) + i % R] = v;
    }
    __syncthreads();
  }
  const float sc = p.scale[ad];
  if (p.h) {  // a rank block of 16 fills its 32-rank block with zeros
    constexpr int KB = R < 32 ? 1 : R / 32;
    for (int i = tid; i < MT * KB * 64; i += 64 * NW) {
      const int m = i / (KB * 64), kb = i / 64 % KB, fq = i / 16 % 4, fc = i % 16;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int rank = 32 * kb + 8 * fq + e;
        v[e] = rank < R ? lds[(16 * m + fc) * (R + 1) + rank] * sc : 0.0f;
      }
      const int64_t group = slot0 / 16 + m, block = k0 / 32 + kb;
      if (block * 32 < p.rp) store_frag(p.h, p.h_bf16, p.h_term, (group * (p.rp / 32) + block) * 64 + i % 64, v);
    }
  }
  if (p.ht) {
    for (int i = tid; i < NT * 64; i += 64 * NW) {
      const int n = i / 64, fq = i / 16 % 4, fc = i % 16;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = lds[(8 * fq + e) * (R + 1) + 16 * n + fc] * sc;
      const int64_t block = k0 / 16 + n;
      if (block * 16 < p.rp) store_frag(p.ht, p.ht_bf16, p.ht_term, ((int64_t)tile * (p.rp / 16) + block) * 64 + i % 64, v);
    }
  }
}

// LDS of a shrink workgroup: the stages, or the waves' sums
template <typename EX, typename EW, int MT, int NT>
constexpr int shrink_lds() {
  const int sums = 4 * kShrinkWaves * MT * NT * 256, out = 4 * 16 * MT * (16 * NT + 1);
  const int stages = MT == 2 && sizeof(typename FragOf<EX, EW>::type) == 2 ? kStages * stage_bytes<false, NT>() : 0;
  return stages > sums ? stages : (sums > out ? sums : out);
}

template <typename EX, typename EW, int MT, int NT>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink_kernel(ShrinkArgs p) {
  extern __shared__ __attribute__((aligned(16))) float shrink_mem[];
  shrink<EX, EW, false, MT, NT>(p, (int)blockIdx.y, shrink_mem);
}

// Both hidden vectors of the gradients in one launch: g with B (the slower one,
// first), then x with A.
template <typename EX, typename EG, typename EW, int NT>
__global__ __launch_bounds__(64 * kShrinkWaves) void lora_shrink2_kernel(ShrinkArgs px, ShrinkArgs pg) {
  extern __shared__ __attribute__((aligned(16))) float shrink_mem[];
  const int y = (int)blockIdx.y;
  if (y < pg.spans)
    shrink<EG, EW, true, 2, NT>(pg, y, shrink_mem);
  else
    shrink<EX, EW, false, 2, NT>(px, y - pg.spans, shrink_mem);
}

// ---------------------------------------------------------------- expand
// y[row][j] = base[row][j] + sum_k W[j][k] h[slot][k] (TW: W stored [k][j]).
// A wave takes 128 columns as eight 16x16 tiles and keeps their factors (32 KB
// rank rows) in registers while consecutive groups of 16 slots have the same
// adapter.  The product of a group goes through the wave's part of LDS, so that
// rows of base and y move as 512 consecutive bytes; base of the next group is
// loaded before this one is stored.
// Columns: tile v, row p holds 16v + p, or (TW) tile 2u + b holds 32u + 2p + b,
// so that a lane loads two consecutive columns of a row of W; either way a
// lane's results are eight float4 pieces.
// Bound by the bytes of base and y: 2048 x 8192, rank 16 27 us (4.9 TB/s), 8192 x
// 28672, rank 64 415 us (4.5 TB/s); a large copy runs at 5.2.
struct ExpandArgs {
  const void* h;        // fragments as shrink stores them; direct calls: fp32 [spans][nslots][rp] unscaled sums
  int64_t h_term;
  const void* w;
  int64_t d, ldw, stride_w;
  const float* scale;   // direct calls
  const int32_t* ids;   // direct calls
  const int* tile_ad;
  const int* tile_off;
  const int* slot_row;
  int T, n, r, rp, spans;
  int64_t nslots;
  int per_wg;           // 16-slot groups of a workgroup
  const float* base;    // [T][d] or null
  float* y;             // [T][d]
};

template <typename EW, bool TW>
__device__ inline void expand_weights(const ExpandArgs& p, int ad, int64_t n0, int kb, int q, int c, Frag<EW> (&w)[8]) {
  const EW* base = static_cast<const EW*>(p.w) + ad * p.stride_w;
  const int k = 32 * kb + 8 * q;
  if constexpr (TW) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t j = n0 + 32 * u + 2 * c;
      EW v[8][2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const EW* a = base + (int64_t)(k + e) * p.ldw + j;
        if (k + e < p.r && j + 2 <= p.d) {
          struct __attribute__((packed, aligned(sizeof(EW)))) Pair {
            EW v[2];
          };
          const Pair t = *reinterpret_cast<const Pair*>(a);
          v[e][0] = t.v[0], v[e][1] = t.v[1];
        } else {
          v[e][0] = k + e < p.r && j < p.d ? a[0] : EW{};
          v[e][1] = EW{};
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if constexpr (sizeof(EW) == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[2 * u + b].d[i] = (uint32_t)v[2 * i][b].u | ((uint32_t)v[2 * i + 1][b].u << 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[2 * u + b].v[e] = v[e][b];
        }
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const EW* row = base + imin(n0 + 16 * v + c, p.d - 1) * p.ldw;  // columns past the last are not stored
      w[v] = load8_row(row, k, p.r);
    }
  }
}

// A fragment of hidden vectors as shrink stored it.
template <typename E>
__device__ inline void load_wide(const void* h, int64_t term, int64_t frag, Wide<E>& w);
template <>
__device__ inline void load_wide<float>(const void* h, int64_t term, int64_t frag, Wide<float>& w) {
  w.f = load8<float, float>(static_cast<const float*>(h) + frag * 8, 8);
}
template <>
__device__ inline void load_wide<Bf16>(const void* h, int64_t term, int64_t frag, Wide<Bf16>& w) {
#pragma unroll
  for (int t = 0; t < 3; ++t) w.t[t].d = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(h) + t * term + frag * 8);
}

// Row 2t + lane / 32 of a group (row: lane c's), as two scalars and a choice.
__device__ inline int group_row(int row, int t, int lane) {
  const int a = __builtin_amdgcn_readlane(row, 2 * t), b = __builtin_amdgcn_readlane(row, 2 * t + 1);
  return lane < 32 ? a : b;
}

// Columns n0 + 4 (lane % 32) .. of the group's rows.
__device__ inline void load_base(const ExpandArgs& p, int row, int64_t n0, int lane, f32x4 (&b)[8]) {
  const int64_t j = n0 + lane % 32 * 4;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int rt = group_row(row, t, lane);
    b[t] = zero4();
    if (!p.base || rt < 0) continue;
    const float* at = p.base + (int64_t)rt * p.d + j;
    if (j + 4 <= p.d) {
      b[t] = *reinterpret_cast<const f32x4u*>(at);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < p.d) b[t][e] = at[e];
    }
  }
}

constexpr int kOutRow = 132;  // floats of a row in LDS: 128 and a pad of one float4

template <bool TW>
__device__ inline void store_rows(const ExpandArgs& p, int row, int64_t n0, int lane, const f32x4 (&acc)[8],
                                  const f32x4 (&b)[8], bool bad, float* lds) {
  const int q = lane / 16, c = lane % 16;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if constexpr (TW) {
      const int u = t / 2, i = 2 * (t % 2);
      *reinterpret_cast<f32x4*>(lds + c * kOutRow + 32 * u + 8 * q + 2 * i) =
          f32x4{acc[2 * u][i], acc[2 * u + 1][i], acc[2 * u][i + 1], acc[2 * u + 1][i + 1]};
    } else {
      *reinterpret_cast<f32x4*>(lds + c * kOutRow + 16 * t + 4 * q) = acc[t];
    }
  }
  const int64_t j = n0 + lane % 32 * 4;
  const float nan = __builtin_nanf("");
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(lds + (2 * t + lane / 32) * kOutRow + lane % 32 * 4);
    const int rt = group_row(row, t, lane);
    if (rt < 0) continue;
    const f32x4 v = bad ? f32x4{nan, nan, nan, nan} : a + b[t];
    float* at = p.y + (int64_t)rt * p.d + j;
    if (j + 4 <= p.d) {
      *reinterpret_cast<f32x4u*>(at) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < p.d) at[e] = v[e];
    }
  }
}

// Workgroup bx along the slots (per_wg 16-slot groups each), by along the columns
// (512 each).
template <typename EW, bool TW, int KB>
__device__ inline void expand(const ExpandArgs& p, int bx, int by, float (*out)[16 * kOutRow]) {
  const int lane = threadIdx.x % 64, q = lane / 16, c = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t n0 = ((int64_t)by * 4 + wave) * 128;
  if (n0 >= p.d) return;
  const int kbs = p.rp / 32;
  Frag<EW> w[KB][8];
  f32x4 acc[8], bcur[8], bnext[8];
  constexpr int SUB = kTile / 16;
  const int begin = bx * p.per_wg;
  const int end = min(p.tile_off[p.n + 2] * SUB, begin + p.per_wg);
  if (begin >= end) return;
  int have = -1;  // adapter whose factors w holds
  int row = routed_row(p.slot_row[(int64_t)begin * 16 + c], p.T);
  load_base(p, row, n0, lane, bcur);
  for (int it = begin; it < end; ++it) {
    const int ad = __builtin_amdgcn_readfirstlane(p.tile_ad[it / SUB]);
    const int next = it + 1 < end ? routed_row(p.slot_row[(int64_t)it * 16 + 16 + c], p.T) : -1;
    const bool any = __ballot(row >= 0) != 0;
#pragma unroll
    for (int v = 0; v < 8; ++v) acc[v] = zero4();
    if (any && routed_adapter(ad, p.n)) {
      for (int kb0 = 0; kb0 < kbs; kb0 += KB) {
        Wide<EW> hw[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b)
          if (b == 0 || kb0 + b < kbs) load_wide<EW>(p.h, p.h_term, ((int64_t)it * kbs + kb0 + b) * 64 + lane, hw[b]);
        if (have != ad || kbs > KB)
#pragma unroll
          for (int b = 0; b < KB; ++b)
            if (b == 0 || kb0 + b < kbs) expand_weights<EW, TW>(p, ad, n0, kb0 + b, q, c, w[b]);
#pragma unroll
        for (int b = 0; b < KB; ++b)
          if (b == 0 || kb0 + b < kbs)
#pragma unroll
            for (int v = 0; v < 8; ++v) mma(w[b][v], hw[b], acc[v]);
      }
      have = ad;
    }
    load_base(p, next, n0, lane, bnext);
    if (any) store_rows<TW>(p, row, n0, lane, acc, bcur, ad == -2, out[wave]);
#pragma unroll
    for (int t = 0; t < 8; ++t) bcur[t] = bnext[t];
    row = next;
  }
}

template <typename EW, int KB>
__global__ __launch_bounds__(256, sizeof(EW) == 4 ? 1 : (KB == 1 ? 3 : 2)) void lora_expand_kernel(ExpandArgs p) {
  __shared__ __attribute__((aligned(16))) float out[4][16 * kOutRow];
  expand<EW, false, KB>(p, (int)blockIdx.x, (int)blockIdx.y, out);
}

// Calls of up to 64 tokens: most groups hold a token or two, where 16-wide
// tiles would leave the matrix cores and the lanes that load rows mostly idle.
// Two columns of W per thread instead, whose rank rows it reads whole, and fp32
// products with the hidden vectors of up to four tokens, which lie in LDS.  Bound
// by the factors' bytes where tokens have adapters of their own (48 mixed tokens,
// rank 16, 8192 -> 28672: 14 us for 42 MB, 3.0 TB/s).  As tiles: 34 us against 26
// for 64 tokens, 15 against 10 for 16 of 4096 x 4096; only 64 tokens of one adapter
// are faster as tiles, 16 against 18.
//
// FUSED: the workgroup computes the hidden vectors itself, four ranks a wave, in
// one launch; for calls so small that a second launch costs more than the longer
// chain of one workgroup (rank 16 in us, one launch / two: 1 token 512 wide 5.2 /
// 6.5, 2048 wide 7.3 / 7.8, 4096 wide 9.7 / 7.3; 4 tokens 1024 wide 6.2 / 7.5; 16
// tokens 256 wide 8.8 / 7.1; rank 64, 1 token 256 wide 11.2 / 8.1).
constexpr int kDirectTokens = 4, kDirectRanks = 64;  // tokens of a group, ranks held in LDS at a time
constexpr int64_t kFusedTokens = 4, kFusedRanks = 16, kFusedWidth = 2048;  // of a fused call, at most

struct DirectArgs {
  ExpandArgs e;
  const void* x;  // fused
  const void* a;
  int64_t d_in, lda, stride_a;
};

template <typename EX, typename EW, bool FUSED>
__global__ __launch_bounds__(256) void lora_direct_kernel(DirectArgs f) {
  constexpr int NC = 2, G = kDirectTokens;  // columns of a thread, 256 apart
  const ExpandArgs& p = f.e;
  __shared__ float hs[G][kDirectRanks];
  __shared__ int rows[G];
  const int tid = threadIdx.x;
  Rows g;
  if (!direct_rows<G>(p.ids, p.T, p.n, (int)blockIdx.x, g)) return;
  const int ad = __builtin_amdgcn_readfirstlane(g.ad);
  const int count = __popcll(__ballot(g.row >= 0) & 0xFFFF);
  int row[G];
#pragma unroll
  for (int t = 0; t < G; ++t) row[t] = __builtin_amdgcn_readlane(g.row, t);
  int64_t j[NC], jc[NC];  // columns past the last are not stored
  const EW* w[NC];
#pragma unroll
  for (int u = 0; u < NC; ++u) {
    j[u] = (int64_t)blockIdx.y * 256 * NC + 256 * u + tid;
    jc[u] = imin(j[u], p.d - 1);
    w[u] = static_cast<const EW*>(p.w) + imax(ad, 0) * p.stride_w + jc[u] * p.ldw;
  }
  Frag<EW> wf[NC][2];
  auto load = [&](int k) {
#pragma unroll
    for (int u = 0; u < NC; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) wf[u][i] = load8_row(w[u], k + 8 * i, p.r);
  };
  float acc[G][NC], b[G][NC];
#pragma unroll
  for (int t = 0; t < G; ++t)
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      acc[t][u] = 0.0f;
      b[t][u] = p.base && t < count ? p.base[(int64_t)row[t] * p.d + jc[u]] : 0.0f;
    }
  if (ad >= 0) {
    load(0);
    const float sc = p.scale[ad];
#pragma unroll 1
    for (int k0 = 0; k0 < p.r; k0 += kDirectRanks) {
      const int kn = min(p.r - k0, kDirectRanks);
      if (k0 > 0) __syncthreads();
      if constexpr (FUSED) {
        const int lane = tid % 64, wave = tid / 64;
        const EW* A = static_cast<const EW*>(f.a) + ad * f.stride_a;
        const int kb = 4 * wave;
        static_assert(kFusedRanks == 16 && kFusedTokens <= G, "four waves of four ranks");
        float h[4][G];
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int t = 0; t < G; ++t) h[v][t] = 0.0f;
        if (kb < kn)
#pragma unroll 1
          for (int64_t i = 8 * lane; i < f.d_in; i += 512) {
            Frag<float> af[4], xf[G];
#pragma unroll
            for (int v = 0; v < 4; ++v)
              af[v] = load8<float, EW>(A + (int64_t)min(kb + v, p.r - 1) * f.lda + i, f.d_in - i);
#pragma unroll
            for (int t = 0; t < G; ++t)
              if (t < count) xf[t] = load8<float, EX>(static_cast<const EX*>(f.x) + (int64_t)row[t] * f.d_in + i, f.d_in - i);
#pragma unroll
            for (int t = 0; t < G; ++t)
              if (t < count)
#pragma unroll
                for (int v = 0; v < 4; ++v)
#pragma unroll
                  for (int e = 0; e < 8; ++e) h[v][t] = fmaf(af[v].v[e], xf[t].v[e], h[v][t]);
          }
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int t = 0; t < G; ++t) {
            if (t >= count) break;
            for (int off = 32; off > 0; off >>= 1) h[v][t] += __shfl_xor(h[v][t], off);
            if (lane == 0) hs[t][kb + v] = kb + v < kn ? h[v][t] * sc : 0.0f;
          }
      } else {
        if (tid < G) rows[tid] = g.row;
        __syncthreads();
        for (int i = tid; i < count * kDirectRanks; i += 256) {
          const int t = i / kDirectRanks, k = i % kDirectRanks;
          float v = 0.0f;
          if (k < kn) {
            const float* hp = static_cast<const float*>(p.h) + (int64_t)rows[t] * p.rp + k0 + k;
#pragma unroll 8
            for (int s = 0; s < p.spans; ++s) v += hp[(int64_t)s * p.nslots * p.rp];
          }
          hs[t][k] = v * sc;  // ranks past r: zero, beside a zero factor
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int kk = 0; kk < kn; kk += 16) {
        Frag<EW> cur[NC][2];
#pragma unroll
        for (int u = 0; u < NC; ++u) cur[u][0] = wf[u][0], cur[u][1] = wf[u][1];
        if (k0 + kk + 16 < p.r) load(k0 + kk + 16);
#pragma unroll
        for (int t = 0; t < G; ++t) {
          if (t >= count) break;
#pragma unroll
          for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int u = 0; u < NC; ++u) acc[t][u] = fmaf(element(cur[u][e / 8], e % 8), hs[t][kk + e], acc[t][u]);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < G; ++t) {
    if (t >= count) break;
#pragma unroll
    for (int u = 0; u < NC; ++u)
      if (j[u] < p.d) p.y[(int64_t)row[t] * p.d + j[u]] = ad == -2 ? __builtin_nanf("") : b[t][u] + acc[t][u];
  }
}

// ---------------------------------------------------------------- factor gradients
// The sum over an adapter's tokens of x_t (128 columns of a workgroup) times
// ht (16 NT RW rank rows).  Lane (q, c) loads 8 consecutive columns 8c .. of the
// rows of slots 8q .. 8q+7 of a tile and transposes them in registers, so tile v
// of the eight holds columns 8c + v.  The four waves are 4 / RW that take tiles
// in turn times RW that take 16 NT ranks each (RW = 2 for more than 32 ranks: four
// rank tiles a wave leave no registers for the next tile's rows, 222 us against 129
// for both gradients of 8192 tokens, rank 64, 8192 x 8192); each loads the next
// tile's rows before it multiplies.  Their sums are added through LDS in wave order.
// DB false: out[k][j] (dA: x and dh), true: out[j][k] (dB: g and h).
struct WgradArgs {
  const void* x;     // [T][d]
  const void* ht;    // fragments as shrink stores them
  int64_t ht_term;
  const int* tile_off;
  const int* slot_row;
  int64_t d, nslots;
  int T, n, r, rp;
  int chunks;        // token chunks
  float* out;        // [chunks][n][r][d] or [chunks][n][d][r]
  int64_t chunk_stride;
};

constexpr int kWgradWaves = 4;

template <typename EX, int NT, int RW, bool DB>
__device__ inline void wgrad(const WgradArgs& p, int64_t block, int ad, int z, float (*part)[8][4][64]) {
  constexpr int TWN = kWgradWaves / RW;
  const int lane = threadIdx.x % 64, q = lane / 16, c = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), tw = wave / RW;
  const int64_t n0 = block * 128;
  const int chunk = z % p.chunks, kb = z / p.chunks * 16 * NT * RW;
  const int k0 = kb + wave % RW * 16 * NT;
  const int a0 = p.tile_off[ad], a1 = p.tile_off[ad + 1];
  const int per = (a1 - a0 + p.chunks - 1) / p.chunks;
  const int t0 = a0 + chunk * per, t1 = min(a1, t0 + per);
  f32x4 acc[8][NT];
#pragma unroll
  for (int v = 0; v < 8; ++v)
#pragma unroll
    for (int k = 0; k < NT; ++k) acc[v][k] = zero4();
  const int64_t j = n0 + 8 * c;
  const bool full = n0 + 128 <= p.d;
  Frag<EX> in[8];
  auto load = [&](int tile) {
    const int* rows = p.slot_row + (int64_t)tile * kTile + 8 * q;
    int row[8], all = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      row[e] = routed_row(rows[e], p.T);
      all |= row[e];
    }
    const EX* x = static_cast<const EX*>(p.x) + j;
    if (full && __ballot(all < 0) == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) in[e] = load8<EX, EX>(x + (int64_t)row[e] * p.d, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) in[e] = load8<EX, EX>(x + (int64_t)row[e] * p.d, row[e] >= 0 ? p.d - j : 0);
    }
  };
  if (t0 + tw < t1) load(t0 + tw);
  for (int tile = t0 + tw; tile < t1; tile += TWN) {
    Frag<EX> xf[8];
    transpose8(in, xf);
    Wide<EX> hw[NT];
#pragma unroll
    for (int k = 0; k < NT; ++k)
      load_wide<EX>(p.ht, p.ht_term, ((int64_t)tile * (p.rp / 16) + min(k0 / 16 + k, p.rp / 16 - 1)) * 64 + lane, hw[k]);
    if (tile + TWN < t1) load(tile + TWN);
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        if constexpr (DB)
          mma(hw[k], xf[v], acc[v][k]);
        else
          mma(xf[v], hw[k], acc[v][k]);
      }
  }
  float* out = p.out + chunk * p.chunk_stride + (int64_t)ad * p.r * p.d;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    if (k > 0) __syncthreads();
#pragma unroll
    for (int v = 0; v < 8; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][v][i][lane] = acc[v][k][i];
    __syncthreads();
    auto sum = [&](int rw, int v, int i) {
      float s = part[rw][v][i][lane];
#pragma unroll
      for (int w = 1; w < TWN; ++w) s += part[w * RW + rw][v][i][lane];
      return s;
    };
#pragma unroll
    for (int u = 0; u < 8 * RW / kWgradWaves; ++u) {
      const int unit = wave + kWgradWaves * u, rw = unit / 8;
      if constexpr (DB) {  // lane: column 8c + v, ranks 4q .. 4q+3
        const int v = unit % 8, kr = kb + rw * 16 * NT + 16 * k + 4 * q;
        if (j + v >= p.d) continue;
        float* at = out + (j + v) * p.r + kr;
        const f32x4 s = {sum(rw, v, 0), sum(rw, v, 1), sum(rw, v, 2), sum(rw, v, 3)};
        if (kr + 4 <= p.r) {
          *reinterpret_cast<f32x4u*>(at) = s;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (kr + i < p.r) at[i] = s[i];
        }
      } else {  // lane: rank c, columns 8 (4q + i) + 4 half ..
        const int half = unit % 2, i = unit / 2 % 4, kr = kb + rw * 16 * NT + 16 * k + c;
        const int64_t jj = n0 + (4 * q + i) * 8 + 4 * half;
        if (kr >= p.r) continue;
        float* at = out + (int64_t)kr * p.d + jj;
        const f32x4 s = {sum(rw, 4 * half, i), sum(rw, 4 * half + 1, i), sum(rw, 4 * half + 2, i), sum(rw, 4 * half + 3, i)};
        if (jj + 4 <= p.d) {
          *reinterpret_cast<f32x4u*>(at) = s;
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (jj + v < p.d) at[v] = s[v];
        }
      }
    }
  }
}

// What follows the hidden vectors of the gradients, in one launch, so that the
// parts fill each other's tails: dB (g and h), dA (x and dh), then dx (dh and A).
// Bound by the rows' bytes: 196 us for 8192 tokens, 16 adapters of rank 64, 8192 x
// 8192 (838 MB, 4.3 TB/s; as two launches 34 us more), 27 us for 2048 tokens, 4 adapters
// of rank 16, 4096 -> 11008.
// Grid: z below `parts` the factor gradients (x: 128-column blocks of both, y:
// adapters), z = parts the output product (x * y: its workgroups).
struct BackArgs {
  WgradArgs a, b;
  ExpandArgs dx;
  int parts, groups, cols;  // dx: workgroups along the slots and the columns
};

template <typename EX, typename EG, typename EW, int NT, int RW, int KB>
__global__ __launch_bounds__(64 * kWgradWaves, sizeof(EW) == 2 ? 2 : 1) void lora_back_kernel(BackArgs p) {
  static_assert(kWgradWaves == 4, "the output product takes four waves");
  union Shared {
    float part[kWgradWaves][8][4][64];
    float out[4][16 * kOutRow];
  };
  __shared__ __attribute__((aligned(16))) Shared lds;
  const int z = (int)blockIdx.z, y = (int)blockIdx.y;
  if (z == p.parts) {
    const int64_t i = (int64_t)y * gridDim.x + blockIdx.x;
    if (i < (int64_t)p.groups * p.cols)
      expand<EW, true, KB>(p.dx, (int)(i % p.groups), (int)(i / p.groups), lds.out);
    return;
  }
  const int64_t blocks_b = cdiv(p.b.d, 128), b = blockIdx.x;
  if (y >= p.a.n) return;
  if (b < blocks_b)
    wgrad<EG, NT, RW, true>(p.b, b, y, z, lds.part);
  else if (b < blocks_b + cdiv(p.a.d, 128))
    wgrad<EX, NT, RW, false>(p.a, b - blocks_b, y, z, lds.part);
}

// da and db: the sums over chunks, in order (both lie one after the other in a chunk)
__global__ __launch_bounds__(256) void lora_sum_kernel(const float* __restrict__ part, int chunks, int64_t count_a,
                                                       int64_t count, float* __restrict__ da, float* __restrict__ db) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    float v = part[i];
    for (int s = 1; s < chunks; ++s) v += part[(int64_t)s * count + i];
    (i < count_a ? da[i] : db[i - count_a]) = v;
  }
}

// ---------------------------------------------------------------- host side

int64_t max_tiles(int64_t n, int64_t T) { return T / kTile + imin(n + 2, T); }

// Spans of a shrink's reduction, 512 elements (one 64-deep step a wave) or more
// each, until the launch has `want` workgroups.  bf16 factors: 128, since a
// workgroup streams its rows and every span adds partial sums to write and read
// back (in us for 64 / 128 / 192 / 384: 512 tokens of 8192, rank 64 30.8 / 30.8 /
// 32.7 / 36.6; 2048 tokens, rank 16 49.5 / 46.2 / 47.5 / 50.4).  fp32 factors: 384,
// since their matrix instructions and scattered loads need more waves (777 tokens
// of 4099, rank 41 50.5 / 37.7 / 36.5 / 34.2).
int shrink_spans(int64_t groups, int64_t d, int64_t want) {
  return (int)imax(1, imin(imin(want / groups, d / 512), 16));
}
int64_t span_len(int64_t d, int spans) { return round_up(cdiv(d, spans), 64); }

struct LoraLayout {
  bool direct, fused;
  int64_t tiles, nslots;
  int rp, nt, kblocks, spans_x, spans_g, chunks;
  int64_t span_x, span_g;
  size_t off_toff, off_tad, off_rows, off_arr, off_hp, off_h, off_gp, off_dh, off_dht, off_part, bytes;
};

LoraLayout lora_layout(const nq_lora& P, int64_t T, bool grads) {
  LoraLayout L{};
  L.direct = !grads && T <= 64;
  L.fused = L.direct && T <= kFusedTokens && P.r <= kFusedRanks && P.d_in <= kFusedWidth;
  L.tiles = max_tiles(P.n, T);
  L.nslots = L.direct ? T : L.tiles * kTile;
  L.rp = (int)round_up(P.r, 32);
  L.nt = P.r <= 16 ? 1 : (P.r <= 32 ? 2 : 4);
  L.kblocks = (int)cdiv(P.r, 16 * L.nt);
  // tiles in use lie between T / 32 and the maximum: the spans go by the former
  const int64_t groups = (L.direct ? cdiv(T, 4) : cdiv(T, kTile)) * L.kblocks;
  auto spans = [&](int64_t d, int64_t* len) {
    const int s = L.direct ? (int)imin(shrink_spans(groups, d, 384), 8)
                           : shrink_spans(groups, d, P.dtype == NQ_BF16 ? 128 : 384);
    *len = span_len(d, s);
    return (int)cdiv(d, *len);
  };
  L.spans_x = spans(P.d_in, &L.span_x);
  if (grads) L.spans_g = spans(P.d_out, &L.span_g);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  const size_t hb = (size_t)L.nslots * L.rp * sizeof(float);
  if (L.fused) {
    take(1);  // no workspace, but a call is given one all the same
  } else if (L.direct) {
    L.off_hp = take(L.spans_x * hb);
  } else {
    L.off_toff = take((size_t)(P.n + 3) * sizeof(int));
    L.off_tad = take((size_t)L.tiles * sizeof(int));
    L.off_rows = take((size_t)L.nslots * sizeof(int));
    L.off_arr = take((size_t)L.tiles * L.kblocks * 2 * sizeof(int));
    if (L.spans_x > 1) L.off_hp = take(L.spans_x * hb);
    L.off_h = take(hb / 4 * 6);  // three bf16 terms at most
  }
  if (grads) {
    if (L.spans_g > 1) L.off_gp = take(L.spans_g * hb);
    L.off_dh = take(hb / 4 * 6);
    L.off_dht = take(hb / 4 * 6);
    const int64_t wgs = P.n * (cdiv(P.d_in, 128) + cdiv(P.d_out, 128)) * L.kblocks;
    // Few adapters leave CUs idle: their tokens are then split, 16 tiles or more of
    // an adapter each, and the parts added by a launch of their own (one adapter of
    // rank 64, 2048 x 2048 in us, split / whole: 8192 tokens 87 / 201, 2048 tokens
    // 49 / 72, 1024 tokens 35 / 41; two adapters of rank 16, 4096 x 4096, 1024
    // tokens: 31 split by 8 tiles, 28 whole).
    L.chunks = (int)imax(1, imin(imin(256 / wgs, T / (P.n * 16 * kTile)), 16));
    if (L.chunks > 1) L.off_part = take((size_t)L.chunks * P.n * P.r * (P.d_in + P.d_out) * sizeof(float));
  }
  L.bytes = off;
  return L;
}

hipError_t launch_route(const int32_t* ids, int64_t T, int64_t n, const LoraLayout& L, char* ws, hipStream_t s) {
  hipLaunchKernelGGL(lora_route_kernel, dim3((unsigned)(n + 2)), dim3(kRouteThreads),
                     (size_t)(n + 2 + kRouteThreads / 64) * sizeof(int), s, ids, (int)T, (int)n,
                     reinterpret_cast<int*>(ws + L.off_toff), reinterpret_cast<int*>(ws + L.off_tad),
                     reinterpret_cast<int*>(ws + L.off_rows), reinterpret_cast<int*>(ws + L.off_arr), 2 * L.kblocks);
  return hipGetLastError();
}

// side 0: h of x with A, 1: dh of g with B
ShrinkArgs shrink_args(const nq_lora& P, const LoraLayout& L, char* ws, int side, const void* x, const int32_t* ids,
                       int64_t T) {
  ShrinkArgs a{};
  a.x = x;
  a.w = side ? P.b : P.a;
  a.d = side ? P.d_out : P.d_in;
  a.ldw = side ? P.ldb : P.lda;
  a.stride_w = side ? P.stride_b : P.stride_a;
  a.ids = ids;
  a.tile_ad = reinterpret_cast<const int*>(ws + L.off_tad);
  a.tile_off = reinterpret_cast<const int*>(ws + L.off_toff);
  a.slot_row = reinterpret_cast<const int*>(ws + L.off_rows);
  a.scale = P.scale;
  a.T = (int)T;
  a.n = (int)P.n;
  a.r = (int)P.r;
  a.rp = L.rp;
  a.span = side ? L.span_g : L.span_x;
  a.spans = side ? L.spans_g : L.spans_x;
  a.nslots = L.nslots;
  a.hpart = reinterpret_cast<float*>(ws + (side ? L.off_gp : L.off_hp));
  a.arrived = reinterpret_cast<int*>(ws + L.off_arr) + side;
  a.h_term = a.ht_term = L.nslots * L.rp;
  a.staged = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && a.d % 8 == 0 &&
             a.ldw % 8 == 0 && a.stride_w % 8 == 0 && (side == 0 || P.r % 8 == 0);
  return a;
}

template <typename EX, typename EW>
hipError_t launch_shrink(const ShrinkArgs& a, const LoraLayout& L, hipStream_t s) {
  const dim3 grid((unsigned)(L.direct ? L.nslots : L.tiles), (unsigned)a.spans, (unsigned)L.kblocks);
  hipError_t e = hipSuccess;
#define NQ_SHRINK(MT, NT)                                                                                  \
  {                                                                                                        \
    constexpr size_t lds = shrink_lds<EX, EW, MT, NT>();                                                   \
    static std::atomic<uint64_t> done{0};                                                                  \
    e = allow_lds(reinterpret_cast<const void*>(lora_shrink_kernel<EX, EW, MT, NT>), lds, done);           \
    if (e != hipSuccess) return e;                                                                         \
    hipLaunchKernelGGL((lora_shrink_kernel<EX, EW, MT, NT>), grid, dim3(64 * kShrinkWaves), lds, s, a);    \
  }
  if (L.direct) {
    if (L.nt == 1)
      NQ_SHRINK(1, 1)
    else if (L.nt == 2)
      NQ_SHRINK(1, 2)
    else
      NQ_SHRINK(1, 4)
  } else {
    if (L.nt == 1)
      NQ_SHRINK(2, 1)
    else if (L.nt == 2)
      NQ_SHRINK(2, 2)
    else
      NQ_SHRINK(2, 4)
  }
#undef NQ_SHRINK
  return hipGetLastError();
}

template <typename EX, typename EG, typename EW>
hipError_t launch_shrink2(const ShrinkArgs& x, const ShrinkArgs& g, const LoraLayout& L, hipStream_t s) {
  const dim3 grid((unsigned)L.tiles, (unsigned)(x.spans + g.spans), (unsigned)L.kblocks);
  hipError_t e = hipSuccess;
#define NQ_SHRINK(NT)                                                                                      \
  {                                                                                                        \
    constexpr size_t lx = shrink_lds<EX, EW, 2, NT>(), lg = shrink_lds<EG, EW, 2, NT>();                   \
    constexpr size_t lds = lx > lg ? lx : lg;                                                              \
    static std::atomic<uint64_t> done{0};                                                                  \
    e = allow_lds(reinterpret_cast<const void*>(lora_shrink2_kernel<EX, EG, EW, NT>), lds, done);          \
    if (e != hipSuccess) return e;                                                                         \
    hipLaunchKernelGGL((lora_shrink2_kernel<EX, EG, EW, NT>), grid, dim3(64 * kShrinkWaves), lds, s, x, g); \
  }
  if (L.nt == 1)
    NQ_SHRINK(1)
  else if (L.nt == 2)
    NQ_SHRINK(2)
  else
    NQ_SHRINK(4)
#undef NQ_SHRINK
  return hipGetLastError();
}

// Workgroups along the slots of an output product: more 16-slot groups each keep
// an adapter's factors in registers for longer, fewer leave a shorter tail behind
// the last round (two workgroups a CU), and an odd number splits tiles.  2 or 4
// groups while 1024 workgroups are left, 8 while 2048 are (us for 1 / 2 / 4 / 8
// groups: 2048 tokens of rank 64, 8192 x 8192 72 / 66 / - / -; 8192 tokens of rank
// 16, 8192 x 8192 - / 164 / 160 / 179; 8192 tokens of rank 64, 8192 -> 28672 - /
// 537 / 491 / 475).
int expand_groups(ExpandArgs* a, const LoraLayout& L) {
  const int64_t groups = L.tiles * (kTile / 16), all = groups * cdiv(a->d, 512);
  // never more than 65536 of them: the gradients' grid folds them into y
  const int64_t want = all >= 16384 ? 8 : (all >= 4096 ? 4 : (all >= 2048 ? 2 : 1));
  a->per_wg = (int)imax(want, cdiv(groups, 65536));
  return (int)cdiv(groups, a->per_wg);
}

hipError_t launch_expand(ExpandArgs a, const LoraLayout& L, nq_dtype wd, hipStream_t s) {
  const int groups = expand_groups(&a, L);
  const dim3 grid((unsigned)groups, (unsigned)cdiv(a.d, 512));
#define NQ_EXPAND(E, KB) hipLaunchKernelGGL((lora_expand_kernel<E, KB>), grid, dim3(256), 0, s, a)
  if (wd == NQ_BF16) {
    if (a.r <= 32)
      NQ_EXPAND(Bf16, 1);
    else
      NQ_EXPAND(Bf16, 2);
  } else {
    NQ_EXPAND(float, 1);  // factors of 64 ranks would leave registers for one wave a SIMD
  }
#undef NQ_EXPAND
  return hipGetLastError();
}

template <typename EX, typename EG, typename EW>
hipError_t launch_back(const WgradArgs& wa, const WgradArgs& wb, const ExpandArgs& ea, const LoraLayout& L, hipStream_t s) {
  BackArgs a;
  a.a = wa;
  a.b = wb;
  a.dx = ea;
  a.parts = L.kblocks * L.chunks;
  a.groups = expand_groups(&a.dx, L);
  a.cols = (int)cdiv(ea.d, 512);
  // x: the column blocks of both gradients (two or more for each of its own); y:
  // the adapters, or more where the output product needs them
  const int64_t gx = cdiv(wa.d, 128) + cdiv(wb.d, 128), gy = imax(wa.n, cdiv((int64_t)a.groups * a.cols, gx));
  const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)(a.parts + 1));
#define NQ_BACK(NT, RW, KB) \
  hipLaunchKernelGGL((lora_back_kernel<EX, EG, EW, NT, RW, KB>), grid, dim3(64 * kWgradWaves), 0, s, a)
  if (L.nt == 1)
    NQ_BACK(1, 1, 1);
  else if (L.nt == 2)
    NQ_BACK(2, 1, 1);
  else
    NQ_BACK(2, 2, (sizeof(EW) == 2 ? 2 : 1));
#undef NQ_BACK
  return hipGetLastError();
}

// h: the hidden vectors' fragments, or (direct) their sums per span
ExpandArgs expand_args(const nq_lora& P, const LoraLayout& L, char* ws, bool grads, const void* h, const int32_t* ids,
                       int64_t T, const float* base, float* y) {
  ExpandArgs a{};
  a.h = h;
  a.h_term = L.nslots * L.rp;
  a.w = grads ? P.a : P.b;
  a.d = grads ? P.d_in : P.d_out;
  a.ldw = grads ? P.lda : P.ldb;
  a.stride_w = grads ? P.stride_a : P.stride_b;
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
  a.base = base;
  a.y = y;
  return a;
}

template <typename EX, typename EG>
hipError_t launch_lora_grads_types(const nq_lora& P, const LoraLayout& L, const ShrinkArgs& sx, const ShrinkArgs& sg,
                                   const ExpandArgs& ea, const WgradArgs& wa, const WgradArgs& wb, float* da, float* db,
                                   hipStream_t s) {
  hipError_t e = P.dtype == NQ_BF16 ? launch_shrink2<EX, EG, Bf16>(sx, sg, L, s) : launch_shrink2<EX, EG, float>(sx, sg, L, s);
  if (e == hipSuccess)
    e = P.dtype == NQ_BF16 ? launch_back<EX, EG, Bf16>(wa, wb, ea, L, s) : launch_back<EX, EG, float>(wa, wb, ea, L, s);
  if (e != hipSuccess || L.chunks == 1) return e;
  const int64_t count_a = P.n * P.r * P.d_in, count = count_a + P.n * P.r * P.d_out;
  hipLaunchKernelGGL(lora_sum_kernel, dim3((unsigned)imin(cdiv(count, 256), 2048)), dim3(256), 0, s, wa.out, L.chunks,
                     count_a, count, da, db);
  return hipGetLastError();
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
  ShrinkArgs sa = shrink_args(P, L, ws, 0, x, ids, T);
  sa.h = ws + L.off_h;
  sa.h_bf16 = P.dtype == NQ_BF16;
  if (!L.fused) {
    if (xd == NQ_BF16)
      e = P.dtype == NQ_BF16 ? launch_shrink<Bf16, Bf16>(sa, L, s) : launch_shrink<Bf16, float>(sa, L, s);
    else
      e = P.dtype == NQ_BF16 ? launch_shrink<float, Bf16>(sa, L, s) : launch_shrink<float, float>(sa, L, s);
    if (e != hipSuccess) return e;
  }
  const ExpandArgs ea =
      expand_args(P, L, ws, false, L.direct ? static_cast<const void*>(sa.hpart) : sa.h, ids, T, base, y);
  if (!L.direct) return launch_expand(ea, L, P.dtype, s);
  const DirectArgs da{ea, x, P.a, P.d_in, P.lda, P.stride_a};
  const dim3 grid((unsigned)T, (unsigned)cdiv(P.d_out, 512));
#define NQ_DIRECT(EX, EW, FUSED) hipLaunchKernelGGL((lora_direct_kernel<EX, EW, FUSED>), grid, dim3(256), 0, s, da)
  const bool xb = xd == NQ_BF16, wb = P.dtype == NQ_BF16;
  if (!L.fused) {  // x is not read
    if (wb)
      NQ_DIRECT(float, Bf16, false);
    else
      NQ_DIRECT(float, float, false);
  } else if (xb) {
    if (wb)
      NQ_DIRECT(Bf16, Bf16, true);
    else
      NQ_DIRECT(Bf16, float, true);
  } else if (wb) {
    NQ_DIRECT(float, Bf16, true);
  } else {
    NQ_DIRECT(float, float, true);
  }
#undef NQ_DIRECT
  return hipGetLastError();
}

hipError_t launch_lora_grads(const nq_lora& P, const void* x, nq_dtype xd, const void* g, nq_dtype gd,
                             const int32_t* ids, int64_t T, const float* dx_base, float* dx, float* da, float* db,
                             void* workspace, hipStream_t s) {
  const LoraLayout L = lora_layout(P, T, true);
  char* ws = static_cast<char*>(workspace);
  const hipError_t e = launch_route(ids, T, P.n, L, ws, s);
  if (e != hipSuccess) return e;
  ShrinkArgs sx = shrink_args(P, L, ws, 0, x, ids, T), sg = shrink_args(P, L, ws, 1, g, ids, T);
  sx.ht = ws + L.off_h;  // h beside g; dh beside A and x
  sx.ht_bf16 = gd == NQ_BF16;
  sg.h = ws + L.off_dh;
  sg.h_bf16 = P.dtype == NQ_BF16;
  sg.ht = ws + L.off_dht;
  sg.ht_bf16 = xd == NQ_BF16;
  const ExpandArgs ea = expand_args(P, L, ws, true, sg.h, ids, T, dx_base, dx);
  const int64_t count_a = P.n * P.r * P.d_in, count = count_a + P.n * P.r * P.d_out;
  float* part = reinterpret_cast<float*>(ws + L.off_part);
  WgradArgs wa{};
  wa.x = x;
  wa.ht = sg.ht;
  wa.ht_term = sg.ht_term;
  wa.tile_off = sx.tile_off;
  wa.slot_row = sx.slot_row;
  wa.d = P.d_in;
  wa.nslots = L.nslots;
  wa.T = (int)T;
  wa.n = (int)P.n;
  wa.r = (int)P.r;
  wa.rp = L.rp;
  wa.chunks = L.chunks;
  wa.out = L.chunks > 1 ? part : da;
  wa.chunk_stride = count;
  WgradArgs wb = wa;
  wb.x = g;
  wb.ht = sx.ht;
  wb.d = P.d_out;
  wb.out = L.chunks > 1 ? part + count_a : db;
  if (xd == NQ_BF16)
    return gd == NQ_BF16 ? launch_lora_grads_types<Bf16, Bf16>(P, L, sx, sg, ea, wa, wb, da, db, s)
                         : launch_lora_grads_types<Bf16, float>(P, L, sx, sg, ea, wa, wb, da, db, s);
  return gd == NQ_BF16 ? launch_lora_grads_types<float, Bf16>(P, L, sx, sg, ea, wa, wb, da, db, s)
                       : launch_lora_grads_types<float, float>(P, L, sx, sg, ea, wa, wb, da, db, s);
}

}  // namespace nq
