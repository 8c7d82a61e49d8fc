/*
 * nq.h -- C ABI of libnq, the MI355X (gfx950) library for NanoQuant's
 * low-rank binary (LRB) linear layer.
 *
 * The layer (research.samsung.com blog "NanoQuant: Efficient Sub-1-Bit
 * Quantization of Large Language Models", section 2 "Problem Formulation and
 * Background", subsection "Low-Rank Binary Factorization", the factorization
 * equation) approximates a weight matrix W (d_out x d_in) by
 *
 *     W[i,j] = s1[i] * (sum_k U[i,k] * V[j,k]) * s2[j],
 *
 * with U in {-1,+1}^(d_out x r), V in {-1,+1}^(d_in x r) and real scale vectors
 * s1 (d_out) and s2 (d_in).  The library evaluates y = W x for T tokens in the
 * factored order y = s1 (.) U (V^T (s2 (.) x)) without forming W.
 *
 * Conventions shared by every call:
 *  - Every pointer argument except `const nq_lrb*`, `nq_seq*` and the arrays of
 *    nq_seq_create is DEVICE memory of the current HIP device.  The caller
 *    allocates and frees all device buffers; libnq keeps no device allocation.
 *  - Every call that launches work enqueues it on `stream` (a hipStream_t
 *    passed as void*; NULL is the default stream) and returns without waiting.
 *    Device faults surface at the caller's next synchronisation.
 *  - Arguments are validated on the host before any HIP call.  A failed check
 *    returns a non-zero status, launches nothing, and sets a thread-local
 *    message readable with nq_last_error().  No C++ exception crosses the ABI.
 *  - Buffers passed to one call must not overlap unless stated.
 *  - Calls are re-entrant; different streams may be used concurrently.
 *
 * Sign-word layout (the "packed integer format"; the pages say only that the
 * frozen binary factors are packed into integer formats, section 3 "Phase 3:
 * Scale-Only Model Reconstruction"):
 *  A stage with n_out outputs and a reduction of length n_red is stored as
 *  words[w][o], w < ceil(n_red/32), o < n_out, with row stride ld >= n_out
 *  (in 32-bit words).  Bit b of words[w][o] is 1 exactly when the sign of
 *  element (o, 32w+b) is -1.  Bits for 32w+b >= n_red are 0.
 *    U   is stored with outputs i < d_out and reduction k < r    (words along r),
 *    V^T is stored with outputs k < r     and reduction j < d_in (words along d_in).
 *  With dimensions that are multiples of 32 and ld = n_out the two buffers hold
 *  exactly r(d_out+d_in) bits, the storage the pages give for the signs
 *  (section 2, the sentence after the factorization equation).
 */
#ifndef NQ_H
#define NQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NQ_OK = 0,
  NQ_ERR_ARG = 1,         /* invalid argument (null pointer, bad size, bad stride) */
  NQ_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. a shape limit)        */
  NQ_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required           */
  NQ_ERR_HIP = 4          /* a HIP runtime call or kernel launch failed           */
} nq_status;

/* Element type of an activation buffer: NQ_F32 or NQ_BF16.  A plain 32-bit
   integer rather than an enum type, so that any value a caller passes is
   well defined in the library (anything else is rejected with NQ_ERR_ARG). */
typedef int32_t nq_dtype;
enum { NQ_F32 = 0, NQ_BF16 = 1 };

/* One packed LRB matrix.  A host struct, read only during a call. */
typedef struct {
  int64_t d_out, d_in, r;   /* all >= 1 */
  const uint32_t* u_bits;   /* [ceil(r/32)][ldu] words, ldu >= d_out   */
  int64_t ldu;
  const uint32_t* vt_bits;  /* [ceil(d_in/32)][ldv] words, ldv >= r    */
  int64_t ldv;
  const float* s1;          /* [d_out] fp32 */
  const float* s2;          /* [d_in]  fp32 */
} nq_lrb;

/*
 * nq_pack_signs -- pack the signs of a real matrix into sign words.
 * The binary factors are sign(U) and sign(V) of real latent factors (section 3
 * "Step 3: Factorized Component Refinement"); once frozen they are packed into
 * integer formats (section 3 "Phase 3").
 *   dst[w*ld + o] bit b = (src[o*stride_out + (32w+b)*stride_red] < 0.0f)
 * for o < n_out, 32w+b < n_red; padding bits are 0; dst columns n_out..ld-1 are
 * not written.  sign() reads -1 only for values < 0 under IEEE comparison:
 * +0, -0 and NaN pack as +1.
 *   U latent [d_out][r]:  n_out=d_out, n_red=r,    stride_out=r, stride_red=1
 *   V latent [d_in][r]:   n_out=r,     n_red=d_in, stride_out=1, stride_red=r
 * Errors: NQ_ERR_ARG for null pointers, n_out or n_red < 1, strides < 1,
 * ld < n_out.
 */
nq_status nq_pack_signs(const float* src, int64_t n_out, int64_t n_red,
                        int64_t stride_out, int64_t stride_red,
                        uint32_t* dst, int64_t ld, void* stream);

/*
 * nq_unpack_signs -- inverse of nq_pack_signs for checking the layout.
 *   dst[o*n_red + e] = bit(words[e/32][o], e%32) ? -1.0f : +1.0f
 * dst is [n_out][n_red] fp32, row-major.  Padding bits are ignored.
 * Errors: NQ_ERR_ARG as for nq_pack_signs.
 */
nq_status nq_unpack_signs(const uint32_t* bits, int64_t n_out, int64_t n_red, int64_t ld,
                          float* dst, void* stream);

/*
 * nq_lrb_workspace_bytes -- device workspace nq_lrb_linear needs for T tokens
 * (the rank-r intermediate t and split-reduction partial sums).  Returns 0 if
 * the arguments are invalid (see nq_lrb_linear).
 */
size_t nq_lrb_workspace_bytes(const nq_lrb* L, int64_t T);

/*
 * nq_lrb_linear -- y = s1 (.) U (V^T (s2 (.) x)) for T tokens.
 * The pages run binary GEMV kernels for token-by-token decoding and binary GEMM
 * kernels for batches (section 4 "Results", subsection "Inference Performance").
 *   x: [T][d_in] row-major, fp32 or bf16 (x_dtype);  y: [T][d_out] fp32.
 *   workspace: at least nq_lrb_workspace_bytes(L, T) bytes, 256-byte aligned.
 * Regimes: T <= 8 runs the decode kernels: each token's stage input is scaled
 * per chunk of 1024 elements by a power of two and split into four fp8 pieces
 * that carry it to within 2^-16 of the chunk's largest value (about 2^-20 in
 * practice, ~4e-7 relative per stage), multiplied by
 * the exact +-1 signs on the matrix cores with fp32 accumulation;
 * T > 8 runs the GEMM kernels: each token row of a stage's activations
 * is scaled by an exact power of two and rounded to fp16 (two fp16 terms for
 * fp32 x), multiplied by the exact +-1 signs with fp32 accumulation, and
 * scaled back.
 * Small layers at T <= 8 (T*d_in <= 2048 and T*r <= 512 with both rounded up
 * to whole words, d_out <= 1024) run in one workgroup instead: z, t and y as
 * fp32 sums in index order with the exact signs (set NQ_DECODE_TINY=0 in the
 * environment to keep them on the decode kernels above; sequence plans always
 * use those, so a sequence entry and a single call of such a layer may differ
 * in the last bits).
 * y is fully overwritten.  Summation order is fixed: results are run-to-run
 * deterministic, but not bitwise equal across regimes.
 * The decode kernels of a single call keep their dependency counters in a
 * small array of the library, one slot per stream (up to 64 streams per
 * device; each launch leaves its slot cleared, so calls need no clearing
 * launch): calls on different streams may overlap, and a call captured into a
 * graph keeps the slot of the stream it was captured on, so its replays must
 * not overlap other calls made on that stream.
 * Errors: NQ_ERR_ARG for null pointers, dims < 1, ldu < d_out, ldv < r, T < 1,
 * an unknown dtype or a misaligned pointer (x, y: 4 bytes; bits, scales: 4
 * bytes); NQ_ERR_UNSUPPORTED when r > 2^24, d_out or d_in > 2^31, or a
 * sign-word buffer exceeds 2 GiB; NQ_ERR_WORKSPACE when workspace_bytes is too
 * small; NQ_ERR_HIP when a launch fails.
 */
nq_status nq_lrb_linear(const nq_lrb* L, const void* x, nq_dtype x_dtype, int64_t T,
                        float* y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nq_reconstruct -- the dense W for checking (the factorization equation):
 *   w[i*d_in + j] = fl32( fl32(s1[i] * m) * s2[j] ),  m = sum_k U[i,k] V[j,k]
 * with m an exact integer and both products rounded to nearest even, so the
 * result is unique bit for bit.  w is [d_out][d_in] fp32.
 * Errors: NQ_ERR_ARG as for nq_lrb_linear; NQ_ERR_UNSUPPORTED for r > 2^24.
 */
nq_status nq_reconstruct(const nq_lrb* L, float* w, void* stream);

/*
 * nq_storage_bits -- storage of one LRB matrix in bits: r(d_out+d_in) signs
 * plus (d_out+d_in) fp32 scales (section 2, the sentence after the
 * factorization equation).  Returns 0 for non-positive arguments.  Host only.
 */
uint64_t nq_storage_bits(int64_t d_out, int64_t d_in, int64_t r);

/*
 * Sequences of independent LRB linears (e.g. every linear of a decoder stack)
 * run as one schedule.  Running the sequence is equivalent to calling
 * nq_lrb_linear on each entry in order, except that entries may run
 * concurrently (no entry's input may be another entry's output, and no two
 * entries' outputs may overlap) and that in the matrix-core regime an entry
 * never splits its reduction, so its sums may be ordered differently from a
 * single call (equal up to rounding; each plan is run-to-run deterministic).
 *
 * nq_seq_create: host-only planning.  `layers`, `xs`, `ys` are host arrays of
 *   n entries (the nq_lrb structs are copied; xs[i], ys[i] are device
 *   pointers).  All entries share T and x_dtype.  The decode regime (T <= 8)
 *   runs as one persistent kernel; T > 8 runs the per-entry kernels
 *   round-robin on three streams owned by the plan (created on the first run
 *   on the device current then), each entry with its own part of the
 *   workspace.  Errors: as for nq_lrb_linear, per entry.
 * nq_seq_workspace_bytes: device workspace the plan needs.
 * nq_seq_run: runs the whole sequence, ordered after the work already on
 *   `stream`; work queued on `stream` afterwards waits for all of it.  The
 *   workspace must stay the same buffer across runs of one plan (the first
 *   decode-regime run uploads the schedule into it, synchronising `stream`
 *   once) and must not be shared by plans running concurrently.  In the decode
 *   regime the first 4 bytes of the workspace are a device error word: 0, or
 *   non-zero (sticky) if a dependency wait inside the kernel gave up; read it
 *   after synchronising.
 * nq_seq_destroy: frees the plan (and its streams).
 */
typedef struct nq_seq nq_seq;
nq_status nq_seq_create(const nq_lrb* layers, const void* const* xs, float* const* ys, int64_t n,
                        nq_dtype x_dtype, int64_t T, nq_seq** out);
size_t nq_seq_workspace_bytes(const nq_seq* s);
nq_status nq_seq_run(nq_seq* s, void* workspace, size_t workspace_bytes, void* stream);
void nq_seq_destroy(nq_seq* s);

/*
 * Scale-only reconstruction (section 3 "Phase 3: Scale-Only Model
 * Reconstruction": with the binary factors frozen only s1 and s2 are tuned).
 *
 * nq_transpose_signs -- sign words of the transposed sign matrix.  src holds an
 *   n_out x n_red sign matrix S in the layout above (row stride ld); dst
 *   receives S^T, i.e. n_red outputs with a reduction over n_out:
 *     bit b of dst[w*ldt + e] = bit (e%32) of src[(e/32)*ld + 32w+b]
 *   for e < n_red, 32w+b < n_out; padding bits are 0; columns n_red..ldt-1 are
 *   not written.  dst is [ceil(n_out/32)][ldt] words, ldt >= n_red, and must
 *   not overlap src.  The transposed layer's words are
 *     ut_bits = nq_transpose_signs(u_bits,  n_out=d_out, n_red=r,    ld=ldu)  [ceil(d_out/32)][ldut >= r]
 *     v_bits  = nq_transpose_signs(vt_bits, n_out=r,     n_red=d_in, ld=ldv)  [ceil(r/32)][ldvv >= d_in]
 *   Errors: NQ_ERR_ARG for null pointers, sizes < 1, ld < n_out, ldt < n_red,
 *   misaligned pointers; NQ_ERR_UNSUPPORTED if a buffer exceeds 2 GiB.
 *
 * nq_lrb_scale_grads -- for y = W x (W as in nq_lrb_linear) and the gradient
 *   g = dL/dy of a loss, the gradients with respect to the input and the scales:
 *     dx[t][j] = sum_i W[i][j] g[t][i]
 *     ds1[i]   = sum_t g[t][i] * (U V^T (s2 (.) x_t))_i
 *     ds2[j]   = sum_t x[t][j] * (V U^T (s1 (.) g_t))_j
 *   x: [T][d_in] fp32 or bf16 (x_dtype); g: [T][d_out] fp32 or bf16
 *   (g_dtype); dx: [T][d_in] fp32; ds1: [d_out] fp32; ds2: [d_in] fp32
 *   (overwritten, not accumulated).
 *   ut_bits/v_bits: the transposed layer's words from nq_transpose_signs.
 *   Both products run through the kernels of nq_lrb_linear (decode regime for
 *   T <= 8, GEMM regime above, with the same arithmetic); the token sums are
 *   fp32 in token order (deterministic).  The two products run concurrently:
 *   the transposed one on a second stream that the library makes on a
 *   device's first call and keeps, forked from and joined back to `stream`
 *   (all of the call's work is ordered after what `stream` holds at the call,
 *   and what is queued on `stream` afterwards is ordered after all of it).
 *   workspace: at least nq_lrb_scale_grads_workspace_bytes(L, T) bytes,
 *   256-byte aligned.  Errors: as for nq_lrb_linear, for L and for the
 *   transposed layer's words; NQ_ERR_ARG for an unknown g_dtype or a null or
 *   misaligned g, ds1 or ds2.
 */
nq_status nq_transpose_signs(const uint32_t* src, int64_t n_out, int64_t n_red, int64_t ld,
                             uint32_t* dst, int64_t ldt, void* stream);
size_t nq_lrb_scale_grads_workspace_bytes(const nq_lrb* L, int64_t T);
nq_status nq_lrb_scale_grads(const nq_lrb* L, const uint32_t* ut_bits, int64_t ldut,
                             const uint32_t* v_bits, int64_t ldvv, const void* x, nq_dtype x_dtype,
                             const void* g, nq_dtype g_dtype, int64_t T, float* dx, float* ds1,
                             float* ds2, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nq_lrb_scale_grads_batch -- nq_lrb_scale_grads for n independent linears in
 * one call (the linears of a decoder layer, say: section 3 "Phase 3: Scale-Only
 * Model Reconstruction" tunes every layer's scales against the model's
 * outputs).  Linear i takes L[i], ut_bits[i]/ldut[i], v_bits[i]/ldvv[i], x[i],
 * g[i] and writes dx[i], ds1[i], ds2[i], each as in nq_lrb_scale_grads; all
 * share T, x_dtype and g_dtype.  The results equal n calls of
 * nq_lrb_scale_grads bit for bit.  With T > 8 the 2n products (forward and
 * transposed of each linear) run round-robin on three streams that the library
 * makes on a device's first such call and keeps, forked from and joined back
 * to `stream`, so that one product's prep kernels and partly filled GEMM waves
 * run beside another's GEMMs; with T <= 8 the linears run one after another.
 *   workspace: at least nq_lrb_scale_grads_batch_workspace_bytes(n, L, T)
 *   bytes, 256-byte aligned; the query returns 0 for invalid arguments.
 * Errors: as for nq_lrb_scale_grads, for each linear (the message names it);
 * NQ_ERR_ARG for n < 1 or a null array.
 */
size_t nq_lrb_scale_grads_batch_workspace_bytes(int64_t n, const nq_lrb* L, int64_t T);
nq_status nq_lrb_scale_grads_batch(int64_t n, const nq_lrb* L, const uint32_t* const* ut_bits,
                                   const int64_t* ldut, const uint32_t* const* v_bits, const int64_t* ldvv,
                                   const void* const* x, nq_dtype x_dtype, const void* const* g,
                                   nq_dtype g_dtype, int64_t T, float* const* dx, float* const* ds1,
                                   float* const* ds2, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nq_lrb_linear_latent -- the layer with the signs taken from real latent
 *   factors at the call: y = s1 (.) sign(U)(sign(V)^T (s2 (.) x)), the forward
 *   pass of the factorized component refinement (section 3 "Step 3:
 *   Factorized Component Refinement", where the binary factors are sign(U) and
 *   sign(V) of latents that the refinement keeps updating).  sign() as in
 *   nq_pack_signs (-1 only for values < 0).  T <= 8: the two stages read the
 *   fp32 latents once and apply sign() as they load (no packed words), fp32
 *   sums in a fixed order.  T > 8: the latents are packed into the workspace,
 *   then the packed layer runs as in nq_lrb_linear: y equals nq_pack_signs
 *   followed by nq_lrb_linear bit for bit.
 *   u_lat: [d_out][ldu_lat] fp32 (row i's r entries first), v_lat:
 *   [d_in][ldv_lat] fp32; s1, s2, x, x_dtype, T, y as for nq_lrb_linear.
 *   workspace: at least nq_lrb_latent_workspace_bytes(d_out, d_in, r, T)
 *   bytes, 256-byte aligned.  Errors: NQ_ERR_ARG for null or misaligned
 *   latents, sizes < 1, ldu_lat or ldv_lat < r; NQ_ERR_UNSUPPORTED at T <= 8
 *   for shapes whose launch grid would exceed 65535 reduction spans;
 *   otherwise as nq_lrb_linear.
 */
size_t nq_lrb_latent_workspace_bytes(int64_t d_out, int64_t d_in, int64_t r, int64_t T);
nq_status nq_lrb_linear_latent(const float* u_lat, int64_t ldu_lat, const float* v_lat,
                               int64_t ldv_lat, int64_t d_out, int64_t d_in, int64_t r,
                               const float* s1, const float* s2, const void* x, nq_dtype x_dtype,
                               int64_t T, float* y, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * Magnitude balancing and scale extraction (section 3, "Magnitude Balancing
 * and Scale Extraction"): the step between the ADMM factorization and the
 * sign packing.  The latent factors can be rescaled inversely without
 * changing their product; balancing equalises their Frobenius norms and the
 * scale vectors are the balanced factors' per-row mean absolute values.
 *
 * nq_balance_factors --
 *     eta = sqrt(||V_hat||_F / ||U_hat||_F)      (1 if either norm is 0)
 *     U = eta * U_hat,   V = V_hat / eta
 *     s1[i] = mean_k |U[i][k]|,   s2[j] = mean_k |V[j][k]|
 *   u_hat: [d_out][ldu] fp32, row i's r entries first (the U latent layout of
 *   nq_pack_signs when ldu = r); v_hat: [d_in][ldv] likewise.  u_out, v_out:
 *   both null (scales only) or both given, with the inputs' strides; each may
 *   be its input (in place) but must not otherwise overlap anything.  s1:
 *   [d_out], s2: [d_in], eta: [1] fp32 device.  Sums of |.| are fp32, sums of
 *   squares and the norms fp64 (every finite fp32 latent), all in a fixed order
 *   (deterministic).  Signs are unchanged (eta > 0), so
 *   nq_pack_signs may read either the latents or the balanced factors.
 *   workspace: at least nq_balance_workspace_bytes(d_out, d_in) bytes,
 *   256-byte aligned.  Errors: NQ_ERR_ARG for null inputs, scales or eta,
 *   sizes < 1, ldu or ldv < r, only one of u_out / v_out, pointers not 4-byte
 *   aligned; NQ_ERR_WORKSPACE for a missing or short workspace.
 */
size_t nq_balance_workspace_bytes(int64_t d_out, int64_t d_in);
nq_status nq_balance_factors(const float* u_hat, int64_t d_out, int64_t ldu, const float* v_hat,
                             int64_t d_in, int64_t ldv, int64_t r, float* u_out, float* v_out,
                             float* s1, float* s2, float* eta, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Low-rank adapters of many requests beside a shared projection: adapter a of
 * a pool adds scale[a] * B_a A_a to a linear, A_a [r][d_in], B_a [d_out][r]
 * real (an adapter of a smaller rank has zero rows in A_a or zero columns in
 * B_a).  Tokens of one call may take different adapters.
 */
typedef struct {
  int64_t n;               /* adapters in the pool, 1 .. NQ_LORA_MAX_ADAPTERS */
  int64_t d_out, d_in, r;  /* all >= 1 */
  nq_dtype dtype;          /* of a and b: NQ_F32 or NQ_BF16 */
  const void* a;           /* A_a[k][j] at a[a*stride_a + k*lda + j], lda >= d_in */
  int64_t lda, stride_a;   /* in elements */
  const void* b;           /* B_a[i][k] at b[a*stride_b + i*ldb + k], ldb >= r */
  int64_t ldb, stride_b;
  const float* scale;      /* [n] fp32 */
} nq_lora;
#define NQ_LORA_MAX_ADAPTERS 8192
#define NQ_LORA_MAX_RANK 1024

/*
 * nq_lora_linear -- y[t] = base[t] + scale[a] * B_a (A_a x[t]),  a = ids[t].
 *   x: [T][d_in] row-major, fp32 or bf16 (x_dtype); ids: [T] int32 device;
 *   base: [T][d_out] fp32, the shared projection's output, or null (zeros);
 *   y: [T][d_out] fp32, fully overwritten; y may be base (in place).
 *   ids[t] < 0: no adapter, y[t] = base[t].  ids[t] >= n: row t of y is NaN
 *   (ids is device data, which a call cannot check on the host).  A call reads
 *   ids more than once: they must be final when it starts on `stream` (work of
 *   another stream that writes them must be waited for) and must not change while
 *   it runs (results are undefined then; no address is made of them).
 * The hidden vectors A_a x[t] and all sums are fp32: nothing is rounded to
 * fewer bits, whatever the types of x and of the factors (beside bf16 factors
 * hidden values below 2^-110 lose what lies under 2^-133).  Values that are not
 * finite stay within the rows whose x, base or adapter holds them, and are
 * infinite or NaN as the products and sums of the formula are (NaN beside a hidden
 * value below 2^-100).  Summation
 * order is fixed: results are run-to-run deterministic, but the order depends
 * on T and n.
 *   workspace: at least nq_lora_workspace_bytes(P, T) bytes, 256-byte aligned;
 *   calls that may overlap (streams, graphs replayed beside other calls) need a
 *   workspace each.
 * Errors: NQ_ERR_ARG for null pointers, sizes < 1, lda < d_in, ldb < r, a
 * negative adapter stride, T < 1, an unknown dtype or a pointer not aligned to
 * its elements; NQ_ERR_UNSUPPORTED for n > NQ_LORA_MAX_ADAPTERS,
 * r > NQ_LORA_MAX_RANK, d_out or d_in > 2^24 or T > 2^24; NQ_ERR_WORKSPACE when
 * workspace_bytes is too small; NQ_ERR_HIP when a launch fails.  The size query
 * returns 0 for invalid arguments.
 */
size_t nq_lora_workspace_bytes(const nq_lora* P, int64_t T);
nq_status nq_lora_linear(const nq_lora* P, const void* x, nq_dtype x_dtype, const int32_t* ids, int64_t T,
                         const float* base, float* y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nq_lrb_lora_linear -- nq_lrb_linear followed by nq_lora_linear on its output:
 *   y = W x (W the packed layer L) plus each token's adapter.  P's d_out and
 *   d_in must be L's.  The same y as the two calls, bit for bit.
 *   workspace: at least nq_lrb_lora_workspace_bytes(L, P, T) bytes, 256-byte
 *   aligned.  Errors: as for the two calls; NQ_ERR_ARG if the sizes differ.
 */
size_t nq_lrb_lora_workspace_bytes(const nq_lrb* L, const nq_lora* P, int64_t T);
nq_status nq_lrb_lora_linear(const nq_lrb* L, const nq_lora* P, const void* x, nq_dtype x_dtype, const int32_t* ids,
                             int64_t T, float* y, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nq_lora_grads -- the gradients of nq_lora_linear for g = dL/dy:
 *     dx[t]   = dx_base[t] + scale[a] * A_a^T (B_a^T g[t])
 *     da[a]   = scale[a] * sum over a's tokens of (B_a^T g[t]) x[t]^T    [r][d_in]
 *     db[a]   = scale[a] * sum over a's tokens of g[t] (A_a x[t])^T      [d_out][r]
 *   x: [T][d_in] (x_dtype), g: [T][d_out] (g_dtype), fp32 or bf16; dx_base:
 *   [T][d_in] fp32 (the shared projection's dx, as from nq_lrb_scale_grads) or
 *   null (zeros); dx: [T][d_in] fp32, may be dx_base (in place); da:
 *   [n][r][d_in] and db: [n][d_out][r] fp32, contiguous and fully overwritten
 *   (zeros for adapters without tokens).  ids as in nq_lora_linear: a token
 *   without an adapter has dx[t] = dx_base[t], one with an id out of range a NaN
 *   row of dx, and neither enters da or db.  Arithmetic, determinism and errors
 *   as for nq_lora_linear.
 *   workspace: at least nq_lora_grads_workspace_bytes(P, T) bytes, 256-byte
 *   aligned.
 */
size_t nq_lora_grads_workspace_bytes(const nq_lora* P, int64_t T);
nq_status nq_lora_grads(const nq_lora* P, const void* x, nq_dtype x_dtype, const void* g, nq_dtype g_dtype,
                        const int32_t* ids, int64_t T, const float* dx_base, float* dx, float* da, float* db,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * nq_orthogonalize -- Newton-Schulz orthogonalisation of a batch of matrices:
 * the update that takes a factor's gradient (latent U or V, an adapter's A or
 * B) and sets its singular values near one.  From X0 = X / ||X||_F, `steps`
 * times
 *     X <- ca X + (cb G + cc G^2) X,   G = X X^T
 * (X^T in place of X where rows > cols: the same result), that is, every
 * singular value s becomes ca s + cb s^3 + cc s^5.
 *   x: [batch] matrices of rows x cols, element (i, j) of matrix k at
 *   x[k*stride_x + i*ldx + j], fp32 or bf16; y: [batch][rows][cols] contiguous,
 *   fp32 or bf16 (y_dtype), must not overlap x.
 * A zero matrix gives zeros; one with a value that is not finite gives NaN
 * throughout and leaves the other matrices of the batch alone.  Entries of any
 * size are fine (the norm is fp64).
 * Arithmetic: a shorter side up to 64 is computed in fp64 and rounded once.  (Where
 * X has no singular value, in a matrix of fewer independent rows than rows, what
 * rounding leaves there grows by |ca| a step, as in any evaluation: 2^-53 |ca|^steps
 * of the result, below its own rounding up to 15 steps of 3.4445.)  A
 * longer one keeps the iterate in fp32 (what rounding leaves without a singular
 * value: 2^-24 |ca|^steps) and multiplies fp16 operands with fp32 accumulation:
 * two terms each (22 bits), or one (11 bits) for y in bf16, a shorter side of 512
 * or more and few steps: while the square of the largest |cb l + cc l^2|, l in [0,
 * 1.25^2], times the steps is at most 40 (five steps of 3.4445, -4.7750, 2.0315; 64
 * of 1.5, -0.5, 0).  One term costs a third of the products.  Its error is below the
 * rounding of y to bf16 (at five steps 1.3e-3 of the norm beside 1.7e-3 at 512 x 700,
 * 1.1e-3 at 2000 x 8000) but passes it for matrices of rank one (up to 1e-2): take y
 * in fp32 and round it where that matters.  Deterministic.
 *   steps: 1 .. 64; the coefficients must be finite and must map [0, 1.25] into
 *   [-1.25, 1.25], and the largest singular value, one at first, must stay below
 *   1.3125 when every step adds its operands' roundings (up to 0.02 with one term
 *   and 3.4445, -4.7750, 2.0315; 2e-5 with two), so that no iterate leaves the
 *   operands' range.  3.4445, -4.7750, 2.0315 and 1.5, -0.5, 0 do in any form; a
 *   polynomial that touches 1.25 and rises steeply behind it does not.
 *   workspace: at least nq_orthogonalize_workspace_bytes(batch, rows, cols,
 *   y_dtype) bytes, 256-byte aligned (the query returns 0 for invalid
 *   arguments).
 * Errors: NQ_ERR_ARG for null or misaligned pointers, sizes < 1, ldx < cols, a
 * negative stride_x, unknown dtypes, steps or coefficients outside the above;
 * NQ_ERR_UNSUPPORTED for batch > 65535, a side above 2^24 or both sides above
 * 65536; NQ_ERR_WORKSPACE; NQ_ERR_HIP.
 */
size_t nq_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols, nq_dtype y_dtype);
nq_status nq_orthogonalize(const void* x, nq_dtype x_dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ldx,
                           int64_t stride_x, int32_t steps, double ca, double cb, double cc, void* y, nq_dtype y_dtype,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * The packed layer inside a block: bias, activation, gate and residual in the
 * epilogue of the product, and the gradients of that epilogue.
 */
typedef int32_t nq_act;
enum {
  NQ_ACT_NONE = 0,      /* z */
  NQ_ACT_RELU = 1,      /* max(z, 0) */
  NQ_ACT_GELU = 2,      /* z Phi(z), Phi the normal distribution's cdf */
  NQ_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
  NQ_ACT_SILU = 4       /* z / (1 + exp(-z)) */
};
typedef struct {
  nq_act act;
  const float* bias;    /* [d_out] fp32, or null */
  const void* mul;      /* [T][d_out], or null: what act(z) is multiplied by (a gated layer's other projection) */
  nq_dtype mul_dtype;   /* read only with mul; likewise below */
  const void* residual; /* [T][d_out], or null */
  nq_dtype residual_dtype;
  void* z;              /* [T][d_out], or null: receives z, for the backward pass */
  nq_dtype z_dtype;
} nq_epilogue;

/*
 * nq_lrb_linear_act -- nq_lrb_linear with an epilogue:
 *     z[t] = W x[t] + bias,   y[t] = act(z[t]) (.) mul[t] + residual[t]
 *   (a factor or term that is null is left out).  x, T: as in nq_lrb_linear;
 *   y: [T][d_out], fp32 or bf16 (y_dtype).  W x is computed as by nq_lrb_linear
 *   (the same regimes and arithmetic); the epilogue is fp32 and rounds once, to
 *   y's type (and z to its own).  mul and residual may be x; y may be mul or residual
 *   where the types are equal (in place), but not x; z may not be any of them.  z
 *   and an fp32 y carry the error of W x: of bf16 x at T > 8 that of fp16 operands
 *   (3e-4 normwise).  silu and gelu of -inf are NaN, the products -inf * 0 of their
 *   formulas.
 *   workspace: at least nq_lrb_act_workspace_bytes(L, T) bytes, 256-byte aligned
 *   (0 bytes: none, it may be null: small layers at T <= 8).  Streams, graphs and
 *   determinism: as for nq_lrb_linear (NQ_DECODE_TINY does not count here).
 * Errors: as for nq_lrb_linear; NQ_ERR_ARG for a null epilogue, an unknown
 * activation or dtype, or a pointer not aligned to its elements.
 */
size_t nq_lrb_act_workspace_bytes(const nq_lrb* L, int64_t T);
nq_status nq_lrb_linear_act(const nq_lrb* L, const void* x, nq_dtype x_dtype, int64_t T, const nq_epilogue* E, void* y,
                            nq_dtype y_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * nq_act_grads -- the gradients of that epilogue for dy = dL/dy:
 *     dz = dy (.) mul (.) act'(z),   dmul = dy (.) act(z),   dbias[i] = sum_t dz[t][i]
 *   (the residual's gradient is dy itself; dz is the g of nq_lrb_scale_grads).
 *   z, mul, dy, dz, dmul: [T][d] contiguous, fp32 or bf16 each; mul null: ones, and
 *   dmul must be null; dmul and dbias may be null (not computed); z may be null
 *   where neither act' nor dmul needs it (NQ_ACT_NONE without dmul).  dz may be dy
 *   or z and dmul may be mul where the types are equal (in place).  fp32
 *   arithmetic, each result rounded once; relu'(0) = 0; silu' and gelu' of +-inf are
 *   NaN, as their formulas' products inf * 0; dbias sums the unrounded dz in a fixed
 *   order (deterministic), in fp32 per thread and fp64 across threads and chunks.
 *   workspace: at least nq_act_grads_workspace_bytes(T, d) bytes, 256-byte aligned
 *   (0 bytes, or dbias null: none, it may be null); calls that may overlap need one
 *   each.
 * Errors: NQ_ERR_ARG for null or misaligned pointers, sizes < 1, unknown
 * activations or dtypes; NQ_ERR_UNSUPPORTED for T or d > 2^24; NQ_ERR_WORKSPACE;
 * NQ_ERR_HIP.  The size query also returns 0 for invalid arguments.
 */
size_t nq_act_grads_workspace_bytes(int64_t T, int64_t d);
nq_status nq_act_grads(nq_act act, const void* z, nq_dtype z_dtype, const void* mul, nq_dtype mul_dtype, const void* dy,
                       nq_dtype dy_dtype, int64_t T, int64_t d, void* dz, nq_dtype dz_dtype, void* dmul,
                       nq_dtype dmul_dtype, float* dbias, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Distillation from a teacher's top logits: the objective of scale-only
 * reconstruction (section 3 "Phase 3: Scale-Only Model Reconstruction": the
 * divergence KL of the quantized model's outputs from the full-precision
 * model's), with the teacher kept as its k most likely tokens per position.
 *
 * nq_logits_top -- a teacher's record: of each row's V logits, at a temperature,
 *   the k largest (largest first; equal ones by index) with their log-probabilities
 *   and the log-probability of all the others together:
 *     l = log sum_v exp(z[v] / temperature)
 *     logp[t][e] = z[ids[t][e]] / temperature - l
 *     rest[t] = log sum over the v not in ids[t] of exp(z[v] / temperature) - l
 *   logits: [T] rows of V, row stride ld >= V elements, fp32 or bf16; ids: [T][k]
 *   int32, logp: [T][k] fp32, rest: [T] fp32 (may be null).  Logits of -inf (masked
 *   tokens) are not listed: where fewer than k remain, ids is -1 and logp -inf from
 *   there on, and rest is -inf where nothing else is left (a row of -inf alone: an
 *   empty record).  A row with NaN or +inf has NaN logp and rest (NaN counts as the
 *   largest logit).
 *   A row is read once; one whose logits are largely equal (padding rows of one
 *   value, say) or NaN, and some rows of fewer than 8 NQ_TOP_MAX logits, are read
 *   some 34 + log2 V times instead: a call waits for its slowest row (V = 32000,
 *   bf16: 0.2 ms for one such row, 1.6 ms among more than 1024 rows; 11 and 53 us
 *   a call without).
 *
 * nq_distill_loss -- the divergence of a student from the record, row by row.  With
 *   q = softmax(s[t] / temperature), p_e = exp(logp[t][e]), r = exp(rest[t]) and
 *   q_rest = the sum of q over the tokens not listed:
 *     loss[t] = weight[t] * ( sum_e p_e (logp[t][e] - log q[ids[t][e]]) + r (rest[t] - log q_rest) )
 *   rest null: r = 0 and the p_e are divided by their sum.  Entries with ids < 0
 *   are not there, those of probability 0 add nothing to the sum (but are listed); a
 *   token listed more than once counts once in q_rest and each of its entries in the
 *   sum.  An id >= V: NaN for that row.  Nothing listed and r = 0: 0 for that row.
 *   weight[t] = 0: the row's logits are not read, its loss and gradient are 0; weight
 *   null: ones.
 *   logits: [T] rows of V, row stride ld >= V elements, fp32 or bf16; weight, loss:
 *   [T] fp32.
 *
 * nq_distill_grads -- the same and its gradient, dlogits[t][v] = d loss[t] / d s[t][v]:
 *     v listed:      weight/temperature * ( (P + r) q_v - sum of p_e over ids[t][e] = v ),  P = sum_e p_e
 *     v not listed:  weight/temperature * ( (P + r) q_v - r q_v / q_rest )
 *   dlogits: [T] rows of V, row stride ldd >= V elements, fp32 or bf16
 *   (dlogits_dtype); columns past V are not written; it may be logits itself with
 *   the same type and stride (in place).  loss may be null.
 * The loss reads the logits once; the gradient goes over a row a second time, at once,
 * while the last of it is in registers and the rest in the caches.  Exponentials are fp32, the sums over a row fp32 per thread and fp64 across, the
 * loss is formed in fp64 and rounded once, each gradient rounded once.  Deterministic;
 * the order of the sums depends on T, V and the call, so the two calls' losses agree
 * to rounding.
 * Logits that are not finite stay within their row, infinite or NaN as the formulas
 * are (a row of -inf alone has no softmax: NaN; a token of logit -inf has q = 0).
 * No workspace.
 * Errors: NQ_ERR_ARG for null or misaligned pointers, T < 1, V < 1, k < 1, ld < V,
 * ldd < V, unknown dtypes, a temperature outside [2^-20, 2^20], or dlogits
 * equal to logits with another type or stride; NQ_ERR_UNSUPPORTED for k >
 * NQ_TOP_MAX, V > 2^20 or T > 2^21; NQ_ERR_HIP.
 */
#define NQ_TOP_MAX 1024
typedef struct {
  int64_t k;            /* entries per row, 1 .. NQ_TOP_MAX */
  const int32_t* ids;   /* [T][k] device */
  const float* logp;    /* [T][k] device: log-probabilities at `temperature` */
  const float* rest;    /* [T] device, or null */
  float temperature;    /* 2^-20 .. 2^20 */
} nq_teacher;
nq_status nq_logits_top(const void* logits, nq_dtype logits_dtype, int64_t T, int64_t V, int64_t ld, int64_t k,
                        float temperature, int32_t* ids, float* logp, float* rest, void* stream);
nq_status nq_distill_loss(const nq_teacher* P, const void* logits, nq_dtype logits_dtype, int64_t T, int64_t V,
                          int64_t ld, const float* weight, float* loss, void* stream);
nq_status nq_distill_grads(const nq_teacher* P, const void* logits, nq_dtype logits_dtype, int64_t T, int64_t V,
                           int64_t ld, const float* weight, float* loss, void* dlogits, nq_dtype dlogits_dtype,
                           int64_t ldd, void* stream);

/*
 * nq_fill_random_words -- synthetic sign words for large benchmark matrices:
 *   dst[i] = low 32 bits of SplitMix64(seed, i), i < n, where SplitMix64(seed,
 *   i) is output number i+1 of the SplitMix64 stream started at `seed`
 *   (Steele, Lea, Flood 2014).  Uniform words give iid +-1 signs.  This is an
 *   input generator, not part of the layer.  Errors: NQ_ERR_ARG for a null
 *   dst or n < 0.
 */
nq_status nq_fill_random_words(uint32_t* dst, int64_t n, uint64_t seed, void* stream);

/*
 * nq_lrb_linear_noalloc -- nq_lrb_linear without a caller workspace and
 *   without any device allocation, for callers that cannot allocate device
 *   memory: code under HIP graph capture, tight serving loops, harnesses that
 *   forbid hipMalloc.  The caller still passes x and y; the workspace is a
 *   fixed array of NQ_NOALLOC_SCRATCH_BYTES bytes inside the library, one copy
 *   per GPU, held from the first use on that GPU until the process ends.
 *   Arguments, results and regimes are those of nq_lrb_linear (same kernels,
 *   bit-identical y).  Every call on one GPU uses that GPU's one array, so
 *   calls on one GPU whose executions overlap (different streams or threads
 *   without ordering between them) race and give wrong results; order them.
 *   The decode regime clears the array's counters with a fill kernel at the
 *   start of each call (no memset).  16 MiB covers the decode regime (T <= 8)
 *   at every Llama-2-70B linear shape up to 2 bits/weight and small GEMM
 *   batches.  Errors: as for nq_lrb_linear; NQ_ERR_UNSUPPORTED when the call
 *   needs more workspace than the array holds (nq_lrb_workspace_bytes(L, T) >
 *   NQ_NOALLOC_SCRATCH_BYTES), checked before any HIP call.
 */
#define NQ_NOALLOC_SCRATCH_BYTES (16u << 20)
nq_status nq_lrb_linear_noalloc(const nq_lrb* L, const void* x, nq_dtype x_dtype, int64_t T, float* y,
                                void* stream);

/* Thread-local message for the last non-OK status of this thread ("" if none). */
const char* nq_last_error(void);

/* Library version string. */
const char* nq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NQ_H */
