/*
 * gdn.h -- C ABI of the MI355X (gfx950) Gated DeltaNet library, CPR schedule.
 *
 * The layer is Gated DeltaNet, named in the IsoExec write-up on agentlenshq.com
 * (section "Chunkwise-Parallel Recurrent (CPR) Gated DeltaNet"), whose pages
 * do not write its equations.  The definition implemented is the gated delta
 * rule in the form in which the problem this library solves is stated, per
 * sequence and value head h, with S a d_v x d_k fp32 matrix:
 *
 *     alpha_t = exp(g_t)
 *     S_t     = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t     = S_t q_t
 *
 * where q_t, k_t are the query/key head h / (H_v / H_qk) vectors, normalised
 * to unit length (x / sqrt(sum x^2 + 1e-6)) when qk_l2norm is set, and q is
 * then multiplied by `scale`.
 *
 * CPR ("chunkwise-parallel recurrent": the same section of the write-up, and
 * the daily.dev digest's Q&A on CPR) keeps the token recurrence as the main
 * computation, evaluated in parallel across C-token chunks, and has decode
 * resynchronise its state every C tokens.  This library's reading:
 *   - every chunk-start state comes from the chunk (WY) form of the
 *     recurrence, scanned sequentially over the chunks of a sequence;
 *   - every output o_t, and the state inside a chunk, comes from the token
 *     recurrence started from that chunk's start state;
 *   - decode runs the same token step and, after the C-th token of a chunk,
 *     replaces its running state by the chunk form applied to the chunk-start
 *     state and the chunk's buffered tokens.
 * Chunks are counted from each sequence's first token.  Because all three
 * entry points run the same device code on the same values, prefill, decode
 * and the trainer forward give bit-identical o and final states, for any
 * batch composition, run after run.
 *
 * Conventions for every call
 *   - All tensors are dense, row-major, on the current HIP device, and start
 *     at 16-byte aligned addresses (else GDN_ERR_INVALID_ARG); the caller
 *     owns every buffer.  The library never allocates or frees device memory
 *     in these calls; scratch comes from `ws`, sized by gdn_workspace_bytes.
 *   - Packed layouts: q, k [T, H_qk, d_k]; v [T, H_v, d_v] in in_dtype;
 *     beta, g [T, H_v] fp32; o [T, H_v, d_v] fp32.  States are fp32
 *     [N, H_v, d_k, d_v] with d_v fastest, i.e. the transpose of S.
 *   - cu_seqlens [N+1] int32: sequence n is tokens [cu[n], cu[n+1]).  It must
 *     start at 0 and be non-decreasing.  Calls take a device copy (read by the
 *     kernels) and a host copy (validated and used to size the launches); both
 *     must hold the same values.  Kernels clamp every index to the buffers'
 *     extents, so a mismatch gives wrong values but no out-of-bounds access.
 *     The host copy may be NULL: the call then first copies the device copy
 *     to the host on `stream` and waits for it (the library's only host
 *     synchronisation; a call made so cannot be captured in a graph).
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = default stream) and
 *     the call returns without waiting.
 *   - Every argument is validated on the host before any launch; on a
 *     validation error nothing is enqueued and nothing is written.  Shapes
 *     outside the compiled claims return GDN_ERR_UNSUPPORTED -- they are never
 *     run through a different arithmetic.
 *   - Supported: d_k == d_v == 128 with C == 64, or d_k == d_v == 16 with
 *     C == 16; H_v a multiple of H_qk with at most 8 value heads per q/k
 *     head; in_dtype fp32 or bf16.
 *   - Calls that overlap on the same workspace or cache race; calls on
 *     separate buffers may run concurrently.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = -1, /* NULL pointer, bad cu_seqlens, negative size, ... */
  GDN_ERR_UNSUPPORTED = -2, /* shape outside the compiled claims              */
  GDN_ERR_WORKSPACE = -3,   /* ws NULL or smaller than gdn_workspace_bytes     */
  GDN_ERR_HIP = -4          /* a HIP runtime call failed                       */
} gdn_status_t;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype_t;

typedef enum {
  GDN_OP_PREFILL = 0,
  GDN_OP_DECODE = 1,
  GDN_OP_FWD_BWD = 2,
  GDN_OP_PREFILL_CHUNKED = 3,
  GDN_OP_PREFILL_CONTINUE = 4
} gdn_op_t;

/* Problem shape.  beta, g, states, o and gradients are always fp32. */
typedef struct {
  int32_t H_qk;      /* query/key heads                                     */
  int32_t H_v;       /* value heads; value head h reads q/k head h/(H_v/H_qk) */
  int32_t d_k, d_v;  /* head dimensions                                     */
  int32_t C;         /* chunk length                                        */
  int32_t in_dtype;  /* gdn_dtype_t of q, k, v                              */
  int32_t qk_l2norm; /* 1: normalise q and k in-kernel; 0: use as given     */
  float scale;       /* multiplies the (normalised) query                   */
} gdn_shape_t;

/*
 * Decode cache of N sequences: the resumable state of token-by-token decode.
 * It is plain device memory owned by the caller: copying it out and back in
 * resumes decode bit-exactly.
 */
typedef struct {
  float* S_run;   /* [N, H_v, d_k, d_v] running state after the last token      */
  float* S_chunk; /* [N, H_v, d_k, d_v] state at the start of the current chunk */
  float* kbuf;    /* [N, C, H_qk, d_k] normalised keys of the current chunk     */
  void* vbuf;     /* [N, C, H_v, d_v] values of the current chunk, in_dtype     */
  float* bbuf;    /* [N, C, H_v] beta of the current chunk                      */
  float* gbuf;    /* [N, C, H_v] g of the current chunk                         */
  int32_t* pos;   /* [N, H_v] tokens of the current chunk absorbed, 0..C-1     */
} gdn_cache_t;

/* Bytes of workspace `op` needs for n_seqs sequences of total_tokens tokens
 * (decode: total_tokens is ignored).  0 for an invalid or unsupported shape. */
size_t gdn_workspace_bytes(const gdn_shape_t* shape, int32_t n_seqs,
                           int64_t total_tokens, int32_t op);

/* Decode cache for n_seqs sequences with nothing decoded yet: S_run = S_chunk
 * = h0 (or zero when h0 is NULL), pos = 0.  h0 is [N, H_v, d_k, d_v] fp32. */
int gdn_cache_init(const gdn_shape_t* shape, int32_t n_seqs, const float* h0,
                   gdn_cache_t* cache, void* stream);

/*
 * Rollout prefill (case "engine_prefill" in the write-up's contract section).
 * h0 [N, H_v, d_k, d_v] nullable (zero).  Writes o; hT [N, H_v, d_k, d_v]
 * (nullable) receives each sequence's final state.  If `cache` is non-NULL it
 * is filled so that gdn_decode_step continues every sequence exactly where
 * this prefill stopped (each sequence's current chunk is its last, possibly
 * partial, chunk).
 */
int gdn_prefill(const gdn_shape_t* shape, int32_t n_seqs,
                const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                const void* q, const void* k, const void* v, const float* beta,
                const float* g, const float* h0, float* o, float* hT,
                gdn_cache_t* cache, void* ws, size_t ws_bytes, void* stream);

/*
 * Rollout decode: one token for each of n_seqs sequences (case "engine
 * decode").  q, k [N, H_qk, d_k], v [N, H_v, d_v] in in_dtype; beta, g
 * [N, H_v] fp32; o [N, H_v, d_v] fp32.  Runs the token step on cache->S_run,
 * appends the token to the chunk buffers and, for every sequence whose chunk
 * is now complete, resynchronises S_run = S_chunk = chunk-form state and sets
 * pos to 0.  pos_host ([N, H_v] mirror of cache->pos, nullable) only lets the
 * host skip the resync launch when no sequence completes a chunk; with NULL
 * the decision is taken on the device.  Out-of-range device pos values are
 * clamped into [0, C).
 */
int gdn_decode_step(const gdn_shape_t* shape, int32_t n_seqs, const void* q,
                    const void* k, const void* v, const float* beta,
                    const float* g, gdn_cache_t* cache, const int32_t* pos_host,
                    float* o, void* ws, size_t ws_bytes, void* stream);

/* Bytes of the fixed device scratch of gdn_decode_step_noalloc, per GPU. */
#define GDN_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/*
 * gdn_decode_step for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments and the same bits as gdn_decode_step, without the workspace:
 * the resync's chunk factors go to a fixed device array of
 * GDN_NOALLOC_SCRATCH_BYTES that the library holds on every GPU it runs on
 * until the process ends.  The resync runs in groups of sequences whose
 * factors fit that array together (H_v * C * (2 d_k + 1) * 4 bytes per
 * sequence: 15 sequences at H_v = 32, d = 128, C = 64), so a batch larger
 * than one group costs two launches per extra group on the steps that
 * resync (every step when pos_host is NULL).  No hipMalloc, hipFree or other
 * allocating call is made.  GDN_ERR_WORKSPACE if a single sequence's factors
 * do not fit.  Every call on a GPU shares that GPU's array: calls that
 * overlap on one GPU (e.g. on two streams) race and must not be issued; the
 * array keeps the last call's contents, which no call reads before writing.
 */
int gdn_decode_step_noalloc(const gdn_shape_t* shape, int32_t n_seqs, const void* q,
                            const void* k, const void* v, const float* beta,
                            const float* g, gdn_cache_t* cache,
                            const int32_t* pos_host, float* o, void* stream);

/*
 * Chunked-prefill continuation: n_seqs sequences whose decode cache stands
 * anywhere inside a chunk (cache->pos = p, the same for every head of a
 * sequence) take their next tokens q, k, v, beta, g (packed by cu_seqlens, as
 * in gdn_prefill) in one call.  The result is bit-identical to having run
 * the whole history and these tokens through one gdn_prefill, or token by
 * token through gdn_decode_step (chunk grid anchored at each sequence's
 * first token, as everywhere): the current chunk is prefilled again from
 * its start state cache->S_chunk, its p buffered tokens (cache->kbuf, vbuf,
 * bbuf, gbuf) followed by the new ones, and the outputs of the new tokens
 * only are written to o [T, H_v, d_v].  hT (nullable) receives each
 * sequence's final state; the cache is left where the sequence now stands.
 * pos_host [n_seqs] (host memory) must hold each sequence's cache->pos; it
 * sizes the launches (a value that disagrees with the device gives wrong
 * results for that sequence, never an access outside the buffers).
 * GDN_ERR_INVALID_ARG if some pos_host value is outside [0, C).  Workspace
 * from gdn_workspace_bytes(..., T, GDN_OP_PREFILL_CONTINUE); it covers the
 * up to n_seqs * (C - 1) buffered tokens.
 */
int gdn_prefill_continue(const gdn_shape_t* shape, int32_t n_seqs,
                         const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                         const int32_t* pos_host, const void* q, const void* k,
                         const void* v, const float* beta, const float* g,
                         gdn_cache_t* cache, float* o, float* hT, void* ws,
                         size_t ws_bytes, void* stream);

/*
 * Trainer forward + backward (case "trainer_fwd" and its gradient).  The
 * forward runs exactly the prefill launches, so o and hT are bit-identical to
 * gdn_prefill's.  dO [T, H_v, d_v] fp32; dhT [N, H_v, d_k, d_v] nullable
 * (zero).  Writes dq, dk [T, H_qk, d_k], dv [T, H_v, d_v], dbeta, dg [T, H_v],
 * dh0 [N, H_v, d_k, d_v], all fp32.  h0 nullable (zero).  The backward
 * recomputes nothing it can keep: chunk-start states and chunk factors of the
 * forward stay in `ws`.  No atomics: results are bitwise reproducible.
 */
int gdn_fwd_bwd(const gdn_shape_t* shape, int32_t n_seqs,
                const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                const void* q, const void* k, const void* v, const float* beta,
                const float* g, const float* h0, const float* dO,
                const float* dhT, float* o, float* hT, float* dq, float* dk,
                float* dv, float* dbeta, float* dg, float* dh0, void* ws,
                size_t ws_bytes, void* stream);

/*
 * gdn_fwd_bwd with the input-shaped gradients dq, dk [T, H_qk, d_k] and dv
 * [T, H_v, d_v] written in grad_dtype: GDN_F32 (then identical to
 * gdn_fwd_bwd) or GDN_BF16, the fp32 result rounded to nearest even (the
 * trainer that keeps its parameters and activations in bf16).  dbeta, dg and
 * dh0 stay fp32.  GDN_ERR_INVALID_ARG for any other grad_dtype.
 */
int gdn_fwd_bwd_ex(const gdn_shape_t* shape, int32_t n_seqs,
                   const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                   const void* q, const void* k, const void* v, const float* beta,
                   const float* g, const float* h0, const float* dO,
                   const float* dhT, float* o, float* hT, int32_t grad_dtype,
                   void* dq, void* dk, void* dv, float* dbeta, float* dg,
                   float* dh0, void* ws, size_t ws_bytes, void* stream);

/*
 * Native-mixed baseline (not the CPR contract): prefill whose outputs come
 * from the chunk form instead of the token recurrence,
 *     o_p = exp(G_p) S_c q_p + sum_{r<=p} (q_p . k_r) exp(G_p - G_r) Delta_r
 * for each chunk with start state S_c (the same chunk-state scan as
 * gdn_prefill, run over every chunk including a partial last one).  This is
 * the "native mixed" prefill of the write-up's stage table (CPR section):
 * the same function as gdn_prefill within the parity tolerance, but its bits
 * are NOT those of gdn_prefill / gdn_decode_step.  It exists to measure what
 * the bitwise guarantee costs.  hT (nullable) gets each sequence's final
 * state from the chunk form.  Same argument conventions as gdn_prefill, no
 * cache; workspace from gdn_workspace_bytes(..., GDN_OP_PREFILL_CHUNKED).
 * Supported at d_k = d_v = 128 only (GDN_ERR_UNSUPPORTED otherwise).
 */
int gdn_prefill_chunked(const gdn_shape_t* shape, int32_t n_seqs,
                        const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                        const void* q, const void* k, const void* v, const float* beta,
                        const float* g, const float* h0, float* o, float* hT, void* ws,
                        size_t ws_bytes, void* stream);

/*
 * Native-mixed baseline trainer step (not the CPR contract): gdn_fwd_bwd whose
 * forward outputs o, and the final state of a sequence whose last chunk is
 * partial, come from the chunk form (as in gdn_prefill_chunked) instead of
 * the token recurrence; the backward is gdn_fwd_bwd's.  The same function
 * within the parity tolerance, other bits.  It exists to measure what the
 * bitwise guarantee costs the trainer (the write-up's stage table, CPR
 * section: native mixed against CPR trainer fwd+bwd).  Arguments as
 * gdn_fwd_bwd (fp32 gradients); workspace from gdn_workspace_bytes(...,
 * GDN_OP_FWD_BWD).  d_k = d_v = 128 only (GDN_ERR_UNSUPPORTED otherwise).
 */
int gdn_fwd_bwd_chunked(const gdn_shape_t* shape, int32_t n_seqs,
                        const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                        const void* q, const void* k, const void* v, const float* beta,
                        const float* g, const float* h0, const float* dO,
                        const float* dhT, float* o, float* hT, float* dq, float* dk,
                        float* dv, float* dbeta, float* dg, float* dh0, void* ws,
                        size_t ws_bytes, void* stream);

/*
 * Native-mixed baseline decode (not the CPR contract): the plain recurrent
 * token step on the running state S [N, H_v, d_k, d_v] (in-out), with no
 * chunk buffers, no position and no resync.  Its arithmetic per token is
 * gdn_decode_step's token step, but without the resync its state leaves the
 * prefill's bits after the first completed chunk.  It exists to measure what
 * the bitwise guarantee costs decode (the write-up's stage table, CPR
 * section: native mixed against CPR rollout decode).  q, k, v, beta, g, o as
 * in gdn_decode_step; no workspace.
 */
int gdn_decode_step_native(const gdn_shape_t* shape, int32_t n_seqs, const void* q,
                           const void* k, const void* v, const float* beta,
                           const float* g, float* S, float* o, void* stream);

/*
 * ---- Gated linear recurrence ------------------------------------------------
 *
 * The layer with a vector for a state: per sequence and channel,
 *
 *     alpha_t = exp(g_t)
 *     h_t     = alpha_t h_{t-1} + b_t x_t
 *     o_t     = h_t
 *
 * with b_t = 1 (GDN_LRU_GATE_NONE), 1 - alpha_t (GDN_LRU_GATE_COMPLEMENT) or
 * sqrt(max(0, 1 - alpha_t^2)) (GDN_LRU_GATE_NORM; 0 where 1 - alpha_t^2 <
 * 2^-126, that is for g_t above -2^-127).  g_t = -inf resets a finite state.
 *
 * As above, chunks are counted from each sequence's first token, here of
 * GDN_LRU_CHUNK tokens, whatever the batch.  Within a chunk
 *     A_p = alpha_p A_{p-1},  B_p = fma(alpha_p, B_{p-1}, b_p x_p),
 *     h_p = fma(A_p, S, B_p)
 * from A = 1, B = 0 and the state S at the chunk's start; the next chunk
 * starts from its last h.  Prefill, continuation, decode and the trainer's
 * forward run these operations in this order, so they give bit-identical o and
 * states, for any batch composition.
 *
 * Range: g_t <= 0 is meant.  Where g_t > 0, the sum of g over a chunk's tokens
 * up to any of them has to stay below 88.7: past that A_p is infinite in fp32,
 * and A_p S is NaN (S = 0) or infinite whatever the state.  At the other end
 * A_p has fewer bits below 2^-126 and none below 2^-150, so that what is left
 * of a state S that a chunk takes down so far is off by up to 2^-145 |S|: for
 * |S| < 2^19 less than fp32's smallest normal number.  The gradient's products
 * are these A_p too.
 *
 * Rows: x, o, dO and dx hold D channels in in_dtype, g and dg in g_dtype; ldx,
 * ldg, ... is the distance between tokens' rows in elements (0 = D, and at
 * least D otherwise), so that they may be slices of wider rows.  h0, hT, dhT,
 * dh0 are fp32 [N, D] and dense.  o may be x itself (same ld); no other buffers
 * may overlap.  Rows past cu_seqlens[N] are neither read nor written.  The
 * conventions at the top hold (16-byte aligned starts, cu_seqlens in a device
 * and a host copy, host copy nullable); a host copy that disagrees with the
 * device copy gives wrong values, never an access outside the rows [0, T).
 * A batch whose launches would hold 2^32 threads is refused
 * (GDN_ERR_UNSUPPORTED); none is where N max(D, 64) <= 2^24 and T max(D, 64)
 * <= 2^35.
 */
#define GDN_LRU_CHUNK 32

typedef enum {
  GDN_LRU_GATE_NONE = 0,
  GDN_LRU_GATE_COMPLEMENT = 1,
  GDN_LRU_GATE_NORM = 2
} gdn_lru_gate_t;

typedef struct {
  int32_t D;        /* channels, 1 .. 2^20                */
  int32_t in_dtype; /* gdn_dtype_t of x, o, dO, dx        */
  int32_t g_dtype;  /* gdn_dtype_t of g, dg               */
  int32_t gate;     /* gdn_lru_gate_t                     */
} gdn_lru_shape_t;

/* Decode cache of N sequences, plain device memory owned by the caller: the
 * state of sequence n is h = A S + B.  pos counts the tokens that the current
 * chunk has taken, 0..GDN_LRU_CHUNK-1, once for each 256 channels (all equal);
 * values outside are clamped. */
typedef struct {
  float* S;     /* [N, D] state at the start of the current chunk      */
  float* A;     /* [N, D] product of the current chunk's alpha         */
  float* B;     /* [N, D] the current chunk's state from a zero start  */
  int32_t* pos; /* [N, ceil(D / 256)]                                  */
} gdn_lru_cache_t;

/* Cache of n_seqs sequences with nothing decoded yet: S = h0 (or zero when h0
 * is NULL), A = 1, B = 0, pos = 0. */
int gdn_lru_cache_init(const gdn_lru_shape_t* shape, int32_t n_seqs, const float* h0,
                       gdn_lru_cache_t* cache, void* stream);

/* Bytes of workspace of `op` (GDN_OP_PREFILL, GDN_OP_PREFILL_CONTINUE or
 * GDN_OP_FWD_BWD); 0 for an invalid shape or another op.  A prefill or
 * continuation of at most GDN_LRU_SMALL tokens needs none: ws may be NULL.
 * Above it the need follows from the sizes alone, and holds also where a call
 * then runs in one pass and leaves the workspace untouched. */
#define GDN_LRU_SMALL 2048
size_t gdn_lru_workspace_bytes(const gdn_lru_shape_t* shape, int32_t n_seqs, int64_t total_tokens,
                               int32_t op);

/* Packed prefill from h0 (nullable: zero).  Writes o and, where given, each
 * sequence's final state hT and the cache from which decode or continuation
 * goes on. */
int gdn_lru_prefill(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                    const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g,
                    int64_t ldg, const float* h0, void* o, int64_t ldo, float* hT,
                    gdn_lru_cache_t* cache, void* ws, size_t ws_bytes, void* stream);

/* The next tokens of sequences whose cache stands anywhere inside a chunk: the
 * same bits as one prefill of the whole history.  The cache is left where the
 * sequences now stand.  Unlike gdn_prefill_continue it needs no host copy of
 * the positions. */
int gdn_lru_prefill_continue(const gdn_lru_shape_t* shape, int32_t n_seqs,
                             const int32_t* cu_seqlens_dev, const int32_t* cu_seqlens_host,
                             const void* x, int64_t ldx, const void* g, int64_t ldg,
                             gdn_lru_cache_t* cache, void* o, int64_t ldo, float* hT, void* ws,
                             size_t ws_bytes, void* stream);

/* One token for each of n_seqs sequences (at most 65535): x, o and g hold
 * n_seqs rows. */
int gdn_lru_decode_step(const gdn_lru_shape_t* shape, int32_t n_seqs, const void* x, int64_t ldx,
                        const void* g, int64_t ldg, gdn_lru_cache_t* cache, void* o, int64_t ldo,
                        void* stream);

/*
 * Trainer forward + backward.  o (nullable) and hT (nullable) are gdn_lru_prefill's
 * bits; without them the call is the backward alone.  dhT nullable (zero).
 * With delta_t the gradient of h_t,
 *     delta_t = dO_t + alpha_{t+1} delta_{t+1}        (+ dhT at the last token)
 *     dx_t    = b_t delta_t
 *     dg_t    = delta_t (alpha_t h_{t-1} + b'_t x_t)
 *     dh0     = alpha_1 delta_1                        (dhT for an empty sequence)
 * where b' = db/dg is 0, -alpha or -alpha^2 / b (0 where b = 0: for g above
 * -2^-127, and at g = 0 the derivative has no finite value).  No atomics:
 * bitwise reproducible.
 */
int gdn_lru_fwd_bwd(const gdn_lru_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens_dev,
                    const int32_t* cu_seqlens_host, const void* x, int64_t ldx, const void* g,
                    int64_t ldg, const float* h0, const void* dO, int64_t lddo, const float* dhT,
                    void* o, int64_t ldo, float* hT, void* dx, int64_t lddx, void* dg,
                    int64_t lddg, float* dh0, void* ws, size_t ws_bytes, void* stream);

/*
 * ---- Norms of q and k per head, with rotary positions -----------------------
 *
 * What a layer does to q and k before it (with gdn_prefill's qk_l2norm = 0), in
 * one pass.  Per token and head, on a vector x of d elements:
 *
 *     n = 1 / sqrt(sum x^2 + eps)   (GDN_NORM_L2),  1 / sqrt(mean x^2 + eps)
 *         (GDN_NORM_RMS),  1 (GDN_NORM_NONE)
 *     z = x n                        (L2, NONE),   x n (weight_offset + w)  (RMS)
 *     y = z, its first r elements turned in pairs (z_a, z_b):
 *         y_a = c (z_a cos - z_b sin),  y_b = c (z_b cos + z_a sin),
 *         angle = pos inv_freq[i],  c = rope_scale,
 *         pair i: (i, i + r/2) for GDN_ROPE_HALF, (2i, 2i + 1) for
 *         GDN_ROPE_INTERLEAVED
 *     q is multiplied by `scale` besides.
 *
 * Angles are formed in fp64 and reduced there, so far positions lose nothing;
 * sums are fp32, and each output is rounded once.  With eps = 0 a head whose
 * fp32 sum of squares is 0 has an infinite n.
 *
 * Rows: token t's heads are H_q (H_k) vectors of d elements one after another,
 * at q + t ldq (ld in elements; 0 = dense; a multiple of 8), so that q and k
 * may be slices of one projection's rows.  qo may be q and ko may be k (same
 * type and ld); no other overlap.  Every start is 16-byte aligned.
 *
 * Positions: pos [T] int32 on the device if given; else token t of sequence n
 * stands at start[n] + t - cu_seqlens[n] (start NULL = 0; all on the device),
 * and rows past cu_seqlens[n_seqs] are neither read nor written.
 *
 * Supported: d a multiple of 8 up to 512, r a multiple of 8 up to d (0: no
 * rotation, inv_freq may be NULL), H_q >= 1, H_k >= 0 (0: k is not touched),
 * together at most 4096, fp32 or bf16 on either side.
 */
typedef enum { GDN_NORM_NONE = 0, GDN_NORM_L2 = 1, GDN_NORM_RMS = 2 } gdn_norm_t;
typedef enum { GDN_ROPE_HALF = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_layout_t;

typedef struct {
  int32_t H_q, H_k;
  int32_t d, r;
  int32_t in_dtype;    /* gdn_dtype_t of q, k (and dq, dk)             */
  int32_t out_dtype;   /* gdn_dtype_t of qo, ko (and dqo, dko)         */
  int32_t norm;        /* gdn_norm_t                                   */
  int32_t layout;      /* gdn_rope_layout_t                            */
  float eps;
  float scale;         /* multiplies q                                 */
  float rope_scale;    /* multiplies cos and sin                       */
  float weight_offset; /* RMS: the factor is weight_offset + w         */
} gdn_qk_shape_t;

/* w_q, w_k: fp32 [d], RMS only (NULL: w = 0 with weight_offset as given). */
int gdn_qk_rotary(const gdn_qk_shape_t* shape, int64_t n_tokens, const int32_t* pos,
                  int32_t n_seqs, const int32_t* cu_seqlens, const int32_t* start,
                  const float* inv_freq, const float* w_q, const float* w_k, const void* q,
                  int64_t ldq, const void* k, int64_t ldk, void* qo, int64_t ldqo, void* ko,
                  int64_t ldko, void* stream);

/* Bytes of workspace of gdn_qk_rotary_bwd; 0 for an invalid shape. */
size_t gdn_qk_workspace_bytes(const gdn_qk_shape_t* shape, int64_t n_tokens);

/* Its gradient, from the inputs q, k and the gradients dqo, dko of qo, ko:
 * with dz the turned-back dy times scale, u = dz (weight_offset + w) and m = d
 * (RMS) or 1 (L2),
 *     dx = n (u - x (n^2 / m) sum(u x)),   dw = sum over tokens and heads of dz x n.
 * n^2 has to be finite in fp32: with eps = 0 heads of elements below 1e-19 may
 * get infinite or NaN gradients.
 * dw_q, dw_k: fp32 [d], RMS only, nullable; their sums run in a fixed order
 * for given sizes (no atomics). */
int gdn_qk_rotary_bwd(const gdn_qk_shape_t* shape, int64_t n_tokens, const int32_t* pos,
                      int32_t n_seqs, const int32_t* cu_seqlens, const int32_t* start,
                      const float* inv_freq, const float* w_q, const float* w_k, const void* q,
                      int64_t ldq, const void* k, int64_t ldk, const void* dqo, int64_t lddqo,
                      const void* dko, int64_t lddko, void* dq, int64_t lddq, void* dk,
                      int64_t lddk, float* dw_q, float* dw_k, void* ws, size_t ws_bytes,
                      void* stream);

/* Frequencies of the r/2 pairs, base^(-2i/r), scaled for contexts longer than
 * trained on: `factor` times longer than orig_len tokens.
 *   NONE    as they are
 *   LINEAR  divided by factor
 *   NTK     base replaced by base factor^(r / (r - 2))
 *   YARN    a pair that turns more than `high` times in orig_len tokens stays,
 *           one that turns fewer than `low` times is divided by factor, and
 *           between the (whole) pair indices where that is so the two are
 *           blended in proportion to the index; rope_scale = 0.1 ln factor + 1
 *           unless attn > 0 gives it
 *   BANDS   as YARN, blended in proportion to the number of turns, with
 *           rope_scale 1 (or attn)
 * Writes inv_freq [r/2] and *rope_scale in host memory; formed in fp64 and
 * rounded once.  Host only. */
typedef enum {
  GDN_ROPE_NONE = 0,
  GDN_ROPE_LINEAR = 1,
  GDN_ROPE_NTK = 2,
  GDN_ROPE_YARN = 3,
  GDN_ROPE_BANDS = 4
} gdn_rope_scaling_kind_t;

typedef struct {
  int32_t kind;     /* gdn_rope_scaling_kind_t                 */
  double factor;    /* >= 1; not read for NONE                 */
  double orig_len;  /* > 0; YARN and BANDS                     */
  double low, high; /* 0 < low < high; YARN and BANDS          */
  double attn;      /* YARN, BANDS: rope_scale, 0 = as above   */
} gdn_rope_scaling_t;

int gdn_rope_freqs(int32_t r, double base, const gdn_rope_scaling_t* scaling, float* inv_freq,
                   float* rope_scale);

/*
 * ---- Softmax attention -------------------------------------------------------
 *
 * The other mixer of stacks that interleave it with the layers above.  Query head
 * h reads key/value head h / (H_q / H_kv).  Sequence n has the queries [cu_q[n],
 * cu_q[n+1]) and the keys [cu_k[n], cu_k[n+1]), aligned at their ends: query i of
 * L_q sees keys j <= i + L_k - L_q, and
 *
 *     s_ij = scale q_i . k_j,  lse_i = log sum_j exp(s_ij),
 *     o_i  = sum_j exp(s_ij - lse_i) v_j
 *
 * A query that sees nothing (L_k < L_q) has o = 0 and lse = -inf.  Products and
 * sums are fp32; bf16 inputs go into the products as they are, and exp(s - max)
 * is rounded to bf16 there (not in its own sum), with fp32 inputs nothing is.
 * Forward, a sequence's bits do not depend on the batch.
 *
 * Rows as for gdn_qk_rotary: token t's heads are d elements each, one after
 * another, at q + t ldq (ld in elements; 0 = dense; a multiple of 8, at most 2^22).
 * All cu_* are on the device and read there; they, and lse and the int32 arrays
 * below, start at multiples of 4 bytes, everything else at multiples of 16.  cu_* must
 * start at 0 and be non-decreasing (values outside the T rows are clamped: wrong
 * values, no access outside).  Rows past cu[n_seqs] are neither read nor written.
 * No output may overlap an input.
 *
 * One sequence's infinities and NaN reach no other's rows; within the sequence they
 * reach the rows that see them, forward (an infinite v as infinities or NaN), and
 * any, in the gradient.  fp32 inputs over 3.39e38 (the largest bf16) count as
 * infinite.  Scores s_ij hold up to 2^30 in magnitude; beyond that a row may become
 * NaN.
 *
 * Supported: d 64, 128 or 256; H_q a multiple of H_kv, at most 4096; 0 < scale <=
 * 2^126.  A batch whose launches would hold 2^32 threads is refused
 * (GDN_ERR_UNSUPPORTED); none is where (T / 128 + n_seqs) max(H_q, 64) <= 2^21, T the
 * larger of T_q and T_k (for the cache (T / 32 + 2 n_seqs) max(H_q, 64) <= 2^23,
 * whatever max_len is).
 */
typedef struct {
  int32_t H_q, H_kv;
  int32_t d;
  int32_t in_dtype; /* gdn_dtype_t of q, k, v, o and the gradients */
  float scale;
} gdn_attn_shape_t;

/* Prefill and the trainer's forward.  cu_k NULL: cu_q, and T_k = T_q.  lse fp32
 * [T_q, H_q], nullable. */
int gdn_attn_prefill(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_q,
                     const int32_t* cu_k, int64_t T_q, int64_t T_k, const void* q, int64_t ldq,
                     const void* k, int64_t ldk, const void* v, int64_t ldv, void* o, int64_t ldo,
                     float* lse, void* stream);

/* Bytes of workspace of gdn_attn_bwd; 0 for an invalid shape. */
size_t gdn_attn_workspace_bytes(const gdn_attn_shape_t* shape, int64_t T_q, int64_t T_k);

/* Its gradient, from what gdn_attn_prefill took and gave and the gradient dO of o
 * (in in_dtype, as dq, dk, dv): with p = exp(s - lse),
 *     dS_ij = p_ij (dO_i . v_j - dO_i . o_i),   dv_j = sum p_ij dO_i,
 *     dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum dS_ij q_i,
 * the sums of dk and dv over the queries of all heads of the group.  Keys that no
 * query sees get 0.  lse is fp32: its rounding, 2^-24 |lse|, is an error of s in p.
 * Of bf16 inputs p goes into dv and dS into dk rounded to bf16, and dS into dq in two
 * bf16 parts; o's own rounding is in dq's dO_i . o_i, not in dk's.  Of fp32 inputs all go
 * in as they are.  No atomics: bitwise reproducible, and T_q and T_k decide the parts
 * that the sums are cut into. */
int gdn_attn_bwd(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_q,
                 const int32_t* cu_k, int64_t T_q, int64_t T_k, const void* q, int64_t ldq,
                 const void* k, int64_t ldk, const void* v, int64_t ldv, const void* o,
                 int64_t ldo, const float* lse, const void* dO, int64_t lddo, void* dq,
                 int64_t lddq, void* dk, int64_t lddk, void* dv, int64_t lddv, void* ws,
                 size_t ws_bytes, void* stream);

/*
 * Key/value cache in 8 bits, plain device memory owned by the caller: pages of
 * page_tokens tokens (a multiple of GDN_KV_BLOCK), anywhere in one pool.  Token t
 * of sequence n stands in page block_table[n * max_pages + t / page_tokens], place
 * t % page_tokens.  An element is an e4m3 code (fn: no infinity) times the scale
 * that GDN_KV_BLOCK neighbouring tokens of a head share, one for keys and one for
 * values: the least power of two s >= 2^-117 with max |x| <= 448 s over the finite
 * elements.  Codes are x / s rounded to nearest even; infinities and NaN become
 * NaN.  (At s = 2^120 codes end at 240.)  Entries of block_table outside [0, pages)
 * hold no tokens: writes to them are dropped, reads leave the rows as they are,
 * attention passes over them.
 */
#define GDN_KV_BLOCK 32

typedef struct {
  void* k;             /* [pages, H_kv, page_tokens, d] e4m3                       */
  void* v;
  float* k_scale;      /* [pages, H_kv, page_tokens / GDN_KV_BLOCK], powers of two */
  float* v_scale;
  int32_t pages;
  int32_t page_tokens; /* at most 2^20                                             */
} gdn_kv_cache_t;

/* Writes the next tokens of n_seqs sequences, k, v [T, H_kv, d] packed by
 * cu_seqlens (device; NULL: one token a sequence, T = n_seqs), at the places
 * start[n], start[n] + 1, ... (device; NULL: 0).  A block that already holds tokens
 * before start[n] keeps its scale if it is the larger, else their codes go over to
 * the new one (exact, but for codes that become subnormal, which are rounded
 * again); places behind the written ones are left as they are and hold nothing.
 * Writing the same tokens again changes nothing.  No two sequences may write to
 * one page, and none may name a page twice where it writes; one without new tokens
 * touches no page, whatever its start. */
int gdn_kv_write(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens,
                 const int32_t* start, int64_t T, const void* k, int64_t ldk, const void* v,
                 int64_t ldv, const gdn_kv_cache_t* cache, const int32_t* block_table,
                 int32_t max_pages, void* stream);

/* Reads tokens back into rows of in_dtype, packed by cu_seqlens, from the places
 * start[n] on (arguments as gdn_kv_write). */
int gdn_kv_read(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens,
                const int32_t* start, int64_t T, const gdn_kv_cache_t* cache,
                const int32_t* block_table, int32_t max_pages, void* k, int64_t ldk, void* v,
                int64_t ldv, void* stream);

/* Attention of new tokens over the cache, which holds them already: q [T, H_q, d]
 * packed by cu_seqlens (NULL: one token a sequence).  kv_len[n] (device) counts the
 * sequence's cached tokens, its L_q new ones being the last of them; as above,
 * query i sees the tokens up to kv_len - L_q + i.  max_len, at least every
 * kv_len[n] (tokens past it are not seen), sizes the launches and the workspace:
 * a captured call holds for lengths up to it.  lse fp32 [T, H_q], nullable.  The
 * cache's values go into the products exactly, in bf16; of bf16 rows q does too, with
 * exp(s - max) in two bf16 parts for a sequence of fewer than 32 rows a key/value
 * head and in one for more; of fp32 rows both are three that sum to them.  No
 * atomics; a sequence's bits depend on neither batch, page size nor max_len. */
size_t gdn_attn_decode_workspace_bytes(const gdn_attn_shape_t* shape, int32_t n_seqs,
                                       int64_t T, int64_t max_len);
int gdn_attn_decode(const gdn_attn_shape_t* shape, int32_t n_seqs, const int32_t* cu_seqlens,
                    int64_t T, const void* q, int64_t ldq, const gdn_kv_cache_t* cache,
                    const int32_t* block_table, int32_t max_pages, const int32_t* kv_len,
                    int64_t max_len, void* o, int64_t ldo, float* lse, void* ws,
                    size_t ws_bytes, void* stream);

/*
 * Kernel timing (instrumentation).  While enabled, every launch the entry
 * points make is bracketed by HIP events recorded on the call's stream.
 * gdn_profile_read waits for the recorded events, returns the summed
 * duration (ms) and launch count of the kernels whose name contains `kernel`
 * (e.g. "k_rec"; NULL or "" = all), and forgets them.  Kernel names:
 * k_plan, k_prep, k_wy, k_scan, k_rec, k_decode, k_wy_resync, k_scan_resync,
 * k_cache_init, k_chunk_o (gdn_prefill_chunked, gdn_fwd_bwd_chunked),
 * k_decode_native (gdn_decode_step_native), k_cont_plan, k_cont_gather,
 * k_cont_scatter (gdn_prefill_continue), the k_bwd_* kernels of gdn_fwd_bwd,
 * the k_lru_* kernels of gdn_lru_*, the k_qk_* kernels of gdn_qk_*, the k_attn_*
 * kernels of gdn_attn_* and the k_kv_* kernels of gdn_kv_*.  Events are created
 * by the library on first use and reused; no device memory is allocated.
 * Thread-safe; records from concurrent calls are merged.
 */
int gdn_profile_enable(int on);
/* While timing is enabled, bracket only the launches whose kernel name
 * contains `kernel` (NULL or "" = all, the default): fewer events in a timed
 * loop.  Host only; GDN_OK. */
int gdn_profile_filter(const char* kernel);
int gdn_profile_read(const char* kernel, double* total_ms, int64_t* launches);

/* Identifier of the compiled arithmetic contract (chunk lengths, epsilon,
 * reduction orders, tiling) ending in "src=" and the first 16 hex digits of a
 * SHA-256 over this header, the library sources and the compile flags.  Two
 * builds give bit-identical results only if these strings are equal (the
 * write-up's contract section, identities: the engines that must agree carry
 * and compare such an identity). */
const char* gdn_contract_id(void);

/* Compares another build's gdn_contract_id() with this one's: GDN_OK if equal,
 * GDN_ERR_UNSUPPORTED if not (the two builds are not guaranteed to produce
 * the same bits, e.g. a trainer and a rollout engine built from different
 * sources), GDN_ERR_INVALID_ARG for NULL.  Host only. */
int gdn_contract_check(const char* id);

/* Human-readable text for a gdn_status_t. */
const char* gdn_error_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
