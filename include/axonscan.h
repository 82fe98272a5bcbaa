/*
 * libaxonscan — C ABI of the selective-scan hot path of the Axon-SSM layer on AMD Instinct
 * MI355X (gfx950).
 *
 * What is computed. The pages cited below are:
 *   [AXON] "Axon-SSM: Selective State Space Model for Apple Silicon" (bit-axon docs).
 *   [WIKI] "Selective State Space Models (Mamba)" (wiki note, "Selective scan (toy)" and
 *          "1M context inference" patterns).
 *
 * For every batch row b and channel e (d_inner = E channels) the layer carries a state
 * h[b,e,0..N-1] and runs, for t = 0..L-1:
 *
 *   u_t   = conv_b[e] + sum_{k=0}^{K-1} conv_w[e,k] * xx[t-(K-1)+k]
 *             [AXON "Key contributions": causal depthwise conv1d, kernel size 4, before the scan;
 *              xx[s] = x[b,s,e] for s >= 0, taken from conv_cache for s < 0]
 *   dt_t  = min(max(softplus(dt_raw[b,t,e] + dt_bias[e]), dt_min), dt_max)
 *             [AXON "Selective mechanism": softplus of the raw step plus a bias, clipped to
 *              [eps, dt_max] with eps = 1e-4, dt_max = 100]
 *   A_n   = -exp(A_log[e,n])                       [AXON "Diagonal state matrix"]
 *   h_n  <- exp(dt_t * A_n) * h_n + dt_t * B[b,t,n] * u_t
 *             [AXON "ZOH discretization": first-order form, Abar = exp(dt A), Bbar = dt B]
 *   y_t   = sum_n C[b,t,n] * h_n + D[e] * u_t      [AXON "Continuous-time SSM", readout]
 *   out[b,t,e] = y_t * z_t * sigmoid(z_t)          [AXON "Gating": y times SiLU(z)]
 *
 * There is no activation between the convolution and the scan (the Axon-SSM page applies SiLU
 * only on the z branch). B, C and dt_raw arrive already projected; the projections W_in,
 * f_proj and W_out are the caller's.
 *
 * Layouts (all row-major, contiguous, innermost index last):
 *   x, z, dt_raw, y : (batch, seqlen, d_inner), activation dtype
 *   B, C            : (batch, seqlen, d_state), activation dtype
 *   A_log           : (d_inner, d_state) fp32
 *   D, dt_bias      : (d_inner) fp32
 *   conv_w          : (d_inner, d_conv) fp32; tap d_conv-1 multiplies the current token
 *   conv_b          : (d_inner) fp32
 *   conv_cache      : (batch, d_conv-1, d_inner) fp32; the last d_conv-1 x-branch inputs seen
 *                     (before the convolution), oldest first [AXON "Autoregressive decoding"]
 *   ssm_state       : (batch, d_inner, d_state) fp32 [AXON "Autoregressive decoding"]
 *
 * Supported shapes: d_state == 16, d_conv == 4 (the layer configuration table of [AXON]);
 * batch >= 1, d_inner >= 1, seqlen >= 0 (else AXON_ERR_INVALID_ARGUMENT);
 * batch <= 65535 and d_inner <= 2^23 (else AXON_ERR_UNSUPPORTED);
 * batch*seqlen*d_inner*d_state <= 2^40 (else AXON_ERR_INVALID_ARGUMENT).
 * Activation dtype: fp32 or bf16 (bf16 outputs are rounded to nearest even from fp32).
 * State, cache and parameters are always fp32; the state recurrence runs in fp32.
 *
 * Ownership and memory: every tensor pointer is device memory owned by the caller, 16-byte
 * aligned. The library allocates nothing and keeps no mutable global state; scratch memory
 * is a caller-provided workspace. Calls are asynchronous on the given stream (a hipStream_t
 * passed as void*; NULL = the default stream); nothing is synchronised on the host.
 *
 * Errors: every argument is checked on the host before anything is launched. On any error
 * code other than AXON_ERR_HIP nothing has been enqueued and no memory was written.
 * AXON_ERR_HIP means a launch failed (hipGetLastError); outputs are then unspecified.
 * The functions are thread-safe.
 */
#ifndef AXONSCAN_H_
#define AXONSCAN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  AXON_OK = 0,
  AXON_ERR_INVALID_ARGUMENT = 1,  /* null/misaligned pointer, bad size, forbidden aliasing */
  AXON_ERR_UNSUPPORTED = 2,       /* d_state != 16, d_conv != 4, unknown dtype, size limits */
  AXON_ERR_WORKSPACE_TOO_SMALL = 3,
  AXON_ERR_HIP = 4                /* a HIP launch or runtime call failed */
} axon_status;

typedef enum { AXON_F32 = 0, AXON_BF16 = 1 } axon_dtype;
/* Enumerated fields of the structs below are int32_t holding these values, so that any integer a
 * caller stores is a defined value that the checks can reject. */

typedef struct {
  int64_t batch;      /* B */
  int64_t seqlen;     /* L (ignored by the decode step) */
  int64_t d_inner;    /* E, channels */
  int64_t d_state;    /* N, must be 16 */
  int64_t d_conv;     /* K, must be 4 */
  int32_t act_dtype;  /* an axon_dtype value */
} axon_ssm_shape;

typedef struct {
  const float* A_log;    /* (E, N) */
  const float* D;        /* (E)    */
  const float* dt_bias;  /* (E)    */
  const float* conv_w;   /* (E, K) */
  const float* conv_b;   /* (E)    */
  float dt_min;          /* lower clip of dt; the Axon-SSM page uses 1e-4 */
  float dt_max;          /* upper clip of dt; the Axon-SSM page uses 100  */
  /* Variants; zero (the default of a zero-initialised struct) is the Axon-SSM layer.
   *   conv_activation: AXON_CONV_NONE, or AXON_CONV_SILU: u = SiLU(conv(x)) before the scan
   *     (the Mamba block of "Selective State Space Models (Mamba)", pattern "Mamba block"); the
   *     skip term D u uses the same u, and conv_cache still holds the raw inputs.
   *   discretization: AXON_DISC_FIRST_ORDER (Bbar = dt B, [AXON "ZOH discretization"]), or
   *     AXON_DISC_ZOH: the exact zero-order hold for the diagonal A that the same section
   *     states first, Bbar = expm1(dt A) / A * B.
   * Other values: AXON_ERR_UNSUPPORTED. */
  int32_t conv_activation;
  int32_t discretization;
} axon_ssm_params;

enum { AXON_CONV_NONE = 0, AXON_CONV_SILU = 1 };
enum { AXON_DISC_FIRST_ORDER = 0, AXON_DISC_ZOH = 1 };

/* Library version as 10000*major + 100*minor + patch. */
int axon_version(void);

/* Static description of a status code (any int; unknown codes give "unknown status"); never
 * NULL. */
const char* axon_status_string(int status);

/* Bytes of device workspace axon_ssm_prefill needs for this shape (0 is possible). A pure
 * function of the shape: no device is queried. Returns 0 for an invalid shape as well, so call
 * axon_ssm_prefill for the diagnosis. */
size_t axon_ssm_prefill_workspace_bytes(const axon_ssm_shape* shape);

/* Prefill: runs the layer over seqlen tokens for every (b, e), continuing from the given cache.
 *
 * conv_cache_in (B, K-1, E) and ssm_state_in (B, E, N) may be NULL, meaning zeros (a fresh
 * sequence, as with state = None in the streaming loop of [WIKI "1M context inference"]).
 * conv_cache_out and ssm_state_out receive the cache after the last token; they may be equal to
 * the corresponding inputs (in-place update) but must not partially overlap them. y must not
 * overlap any input. Prefill(L1) followed by prefill(L2) from its caches equals prefill(L1+L2)
 * up to rounding.
 * seqlen == 0 copies the caches in to out unchanged (zeros for NULL inputs) and writes no y.
 * The conv cache after the call holds exact copies (fp32, exact widening for bf16) of the last
 * K-1 x-branch inputs of the concatenation [cache_in, x].
 * workspace: device memory of at least axon_ssm_prefill_workspace_bytes(shape) bytes, 16-byte
 * aligned; may be NULL when that size is 0. Its contents need no initialisation. */
axon_status axon_ssm_prefill(const axon_ssm_shape* shape, const axon_ssm_params* params,
                             const void* x, const void* z, const void* dt_raw,
                             const void* B, const void* C,
                             const float* conv_cache_in, const float* ssm_state_in,
                             void* y, float* conv_cache_out, float* ssm_state_out,
                             void* workspace, size_t workspace_bytes, void* stream);

/* The same prefill without allocating and without a caller workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation). The time-chunked scan's workspace is a 64 MiB scratch array the library
 * holds on each GPU it runs on until the process ends; for shapes whose chunked plan would need
 * more, the plan takes fewer time chunks (same results to rounding, possibly slower), so every
 * shape axon_ssm_prefill accepts is accepted. Arguments, checks and results otherwise as
 * axon_ssm_prefill; the stream must belong to the current device. Calls on one GPU share its
 * scratch: calls that overlap in time on the same GPU race (serialise them, e.g. on one
 * stream). AXON_ERR_HIP if the scratch's device address cannot be obtained. */
axon_status axon_ssm_prefill_noalloc(const axon_ssm_shape* shape, const axon_ssm_params* params,
                                     const void* x, const void* z, const void* dt_raw,
                                     const void* B, const void* C, const float* conv_cache_in,
                                     const float* ssm_state_in, void* y, float* conv_cache_out,
                                     float* ssm_state_out, void* stream);

/* Decode step: one token per batch row, with the caches updated in place
 * [AXON "Autoregressive decoding": the cache pair carries the convolution padding and the
 * hidden state from one step to the next].
 * x, z, dt_raw, y: (B, E) activation dtype; B, C: (B, N) activation dtype;
 * conv_cache (B, K-1, E) and ssm_state (B, E, N) fp32, read and then overwritten.
 * shape->seqlen is ignored. y must not overlap any input or cache. Equivalent to
 * axon_ssm_prefill with seqlen = 1 and in-place caches. */
axon_status axon_ssm_decode_step(const axon_ssm_shape* shape, const axon_ssm_params* params,
                                 const void* x, const void* z, const void* dt_raw,
                                 const void* B, const void* C,
                                 float* conv_cache, float* ssm_state,
                                 void* y, void* stream);

/* ---- The layer around the path ---------------------------------------------------------------
 * The whole Axon-SSM layer on (B, L, D) activations [AXON "Gating", "Selective mechanism",
 * "Code mapping"]:
 *   (x_branch, z_branch) = split(W_in x)                  W_in (2E, D): rows 0..E-1 give x_branch
 *   u = conv(x_branch) (+ SiLU with AXON_CONV_SILU)        causal depthwise, K = 4, with the cache
 *   (B_t, C_t, dt_raw_t) = f_proj(u_t)                    W_f (2N + E, E): rows 0..N-1 give B_t,
 *                                                           N..2N-1 C_t, 2N..2N+E-1 dt_raw_t
 *   y = the selective scan of u with B, C, dt_raw, gated by SiLU(z_branch) (as axon_ssm_prefill)
 *   out = W_out y                                         W_out (D, E)
 * READING: f_proj is one full-rank linear map from the E conv outputs to [B, C, dt_raw] (the page
 * states a linear projection and no rank bottleneck), with no bias.
 * The projections are dense GEMMs (hipBLASLt, fp32 accumulation) in the activation dtype; every
 * intermediate (x_branch, z_branch, u, B, C, dt_raw, y) is stored in the activation dtype, the
 * conv cache and the state in fp32. seqlen = 1 with in-place caches is the layer's decode step.
 *
 * A context owns the GEMM library handle and its cached GEMM plans; create one per thread (a
 * context is not safe for concurrent use). The forward call allocates nothing: all scratch is
 * the caller's workspace. */
typedef struct axon_layer_ctx axon_layer_ctx;

typedef struct {
  int64_t batch;      /* B */
  int64_t seqlen;     /* L >= 1 */
  int64_t d_model;    /* D */
  int64_t d_inner;    /* E */
  int64_t d_state;    /* N, must be 16 */
  int64_t d_conv;     /* K, must be 4 */
  int32_t act_dtype;  /* an axon_dtype: x_in, out, the three projection weights and the
                        * intermediates */
} axon_layer_shape;

typedef struct {
  const void* W_in;   /* (2E, D) activation dtype, row-major (output feature major) */
  const void* W_f;    /* (2N + E, E) activation dtype */
  const void* W_out;  /* (D, E) activation dtype */
  axon_ssm_params ssm;  /* A_log, D, dt_bias, conv_w, conv_b (fp32), dt clips, variants */
} axon_layer_weights;

/* Create / destroy a context (AXON_ERR_HIP if the GEMM library cannot be initialised). */
axon_status axon_layer_create(axon_layer_ctx** ctx);
void axon_layer_destroy(axon_layer_ctx* ctx);

/* Bytes of device workspace axon_layer_forward needs (0 for an invalid shape). */
size_t axon_layer_workspace_bytes(const axon_layer_shape* shape);

/* Forward over seqlen tokens: x_in (B, L, D) -> out (B, L, D), continuing from the caches as
 * axon_ssm_prefill does (NULL inputs = zeros). Aliasing: out, the workspace, conv_cache_out and
 * ssm_state_out must not overlap x_in, a weight, a parameter array or one another; out and the
 * workspace also not the cache / state inputs; conv_cache_out may equal conv_cache_in and
 * ssm_state_out may equal ssm_state_in exactly (in place), never overlap them partly; the cache
 * output must not overlap the state input nor the state output the cache input. Any violation:
 * AXON_ERR_INVALID_ARGUMENT, nothing written. workspace: axon_layer_workspace_bytes(shape) bytes,
 * 16-byte aligned, contents need no initialisation. */
axon_status axon_layer_forward(axon_layer_ctx* ctx, const axon_layer_shape* shape,
                               const axon_layer_weights* weights, const void* x_in,
                               const float* conv_cache_in, const float* ssm_state_in, void* out,
                               float* conv_cache_out, float* ssm_state_out, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The checks axon_layer_forward makes of its arguments before it launches anything (shape,
 * parameters, null and misaligned pointers, workspace size, aliasing), without a context and
 * without touching device memory: AXON_OK when the forward call with these arguments would run.
 * Pointers are only compared, never dereferenced. */
axon_status axon_layer_forward_check(const axon_layer_shape* shape,
                                     const axon_layer_weights* weights, const void* x_in,
                                     const float* conv_cache_in, const float* ssm_state_in,
                                     const void* out, const float* conv_cache_out,
                                     const float* ssm_state_out, const void* workspace,
                                     size_t workspace_bytes);

/* ---- Mamba-2 SSD core ------------------------------------------------------------------------
 * The state space duality (SSD) layer core of Mamba-2 ["Selective State Space Models (Mamba)",
 * pattern "Mamba-2 block": d_state 128, headdim 64; the SSD article, sections on the duality
 * with linear attention and on the chunked scan]. Heads of head_dim P channels share one scalar
 * decay; for every batch row b and head h, with a state h[p, n] (P x N), for t = 0..L-1:
 *
 *   dt_t      = min(max(softplus(dt_raw[b,t,h] + dt_bias[h]), dt_min), dt_max)
 *   A         = -exp(A_log[h])
 *   h[p, n]  <- exp(dt_t A) h[p, n] + dt_t x[b,t,h,p] B[b,t,n]
 *   y[b,t,h,p] = sum_n C[b,t,n] h[p, n] + D[h] x[b,t,h,p]
 *
 * READING: the first-order input term dt B and the step size of the Axon-SSM layer; B and C are
 * shared by all heads (one group); the convolution, gate and projections of the Mamba-2 block
 * are the caller's. The library computes it in chunks of 64 tokens: within a chunk as matrix
 * products on the matrix cores (the decay-masked C B^T times dt x, the chunk's state
 * contribution x^T diag(w) B and the readout of the incoming state C h^T), and across chunks as a
 * recurrence over the chunk states. fp32 arithmetic throughout (bf16 inputs are widened).
 *
 * Layouts (row-major, contiguous):
 *   x, y    : (batch, seqlen, n_heads, head_dim), activation dtype
 *   dt_raw  : (batch, seqlen, n_heads), activation dtype
 *   B, C    : (batch, seqlen, d_state), activation dtype
 *   A_log, D, dt_bias : (n_heads) fp32
 *   state   : (batch, n_heads, head_dim, d_state) fp32
 * Supported: head_dim == 64 and d_state == 128 (else AXON_ERR_UNSUPPORTED); batch and n_heads in
 * [1, 65535] (0 or negative: AXON_ERR_INVALID_ARGUMENT; larger: AXON_ERR_UNSUPPORTED);
 * seqlen >= 0; batch*seqlen*n_heads*head_dim <= 2^40. Pointers are device memory owned by the
 * caller, 16-byte aligned; errors as for axon_ssm_prefill. */
typedef struct {
  int64_t batch;     /* B */
  int64_t seqlen;    /* L */
  int64_t n_heads;   /* H */
  int64_t head_dim;  /* P, must be 64 */
  int64_t d_state;   /* N, must be 128 */
  int32_t act_dtype;  /* an axon_dtype value */
} axon_ssd_shape;

typedef struct {
  const float* A_log;    /* (H) */
  const float* D;        /* (H) */
  const float* dt_bias;  /* (H) */
  float dt_min;
  float dt_max;
} axon_ssd_params;

/* Bytes of device workspace axon_ssd_scan needs (0 for an invalid shape or seqlen == 0). */
size_t axon_ssd_scan_workspace_bytes(const axon_ssd_shape* shape);

/* Runs the SSD core over seqlen tokens. state_in (B, H, P, N) may be NULL (zeros); state_out
 * receives the state after the last token and may equal state_in (in place) but must not
 * partially overlap it. y must not overlap any input. seqlen == 0 copies state_in to state_out
 * (zeros for NULL) and writes no y. Running L1 tokens then L2 from the returned state equals
 * running L1 + L2 up to rounding. workspace: axon_ssd_scan_workspace_bytes(shape) bytes,
 * 16-byte aligned, no initialisation needed. */
axon_status axon_ssd_scan(const axon_ssd_shape* shape, const axon_ssd_params* params,
                          const void* x, const void* dt_raw, const void* B, const void* C,
                          const float* state_in, void* y, float* state_out, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ---- Packed sequences ------------------------------------------------------------------------
 * Requests of unequal length are packed one behind the other in one buffer of total_tokens rows.
 * axon_sequence_tables builds, on the GPU from the request lengths alone, where each sequence and
 * each block of `block` tokens begins. One int32 array `tables` holds, in this order,
 *   starts       (sequences + 1): starts[n] = min(total_tokens, sum of max(lengths, 0) before n)
 *   block_starts (sequences + 1): blocks of the sequences before n; the last entry is their number
 *   block_seq    (rows): the sequence of each block, -1 behind the last block
 *   block_first  (rows): its first packed token, -1 behind the last block
 * with rows = total_tokens / block + sequences, an upper bound of the number of blocks for any
 * lengths, so that neither a host nor a captured graph has to know the lengths. A sequence's last
 * block may be short; blocks never span two sequences. Lengths below zero count as zero; what goes
 * past total_tokens is cut off there.
 * Limits: sequences in [1, 65535], block >= 1, total_tokens in [0, 2^31), rows < 2^31 (else
 * AXON_ERR_INVALID_ARGUMENT below and AXON_ERR_UNSUPPORTED above them). lengths and tables are
 * device arrays, 4-byte aligned, that must not overlap. */

/* Number of int32 elements of `tables` (0 for invalid arguments). */
size_t axon_sequence_tables_count(int64_t sequences, int64_t total_tokens, int64_t block);

axon_status axon_sequence_tables(int64_t sequences, int64_t total_tokens, int64_t block,
                                 const int32_t* lengths, int32_t* tables, void* stream);

/* Zeros the rows of a packed buffer that lie behind its last sequence, for an output that nothing was
 * written to before (axon_gated_delta_scan leaves these rows as they were): rows starts[sequences] ..
 * total_tokens - 1 of `rows`, row_bytes each. tables: of axon_sequence_tables for these sequences (only
 * that entry is read; it is cut to [0, total_tokens]). Limits: sequences and total_tokens as above;
 * row_bytes a positive multiple of 16; total_tokens * row_bytes <= 2^42; rows 16-byte aligned and not
 * overlapping the tables' starts. */
axon_status axon_clear_behind_sequences(int64_t sequences, int64_t total_tokens, int64_t row_bytes,
                                        const int32_t* tables, void* rows, void* stream);

/* ---- Gated delta rule ------------------------------------------------------------------------
 * The scalar-decay recurrence of the SSD core with the delta rule's write: what the state already
 * answers for a key is taken off before the value is written. For every sequence and value head h
 * (key head h / (value_heads / key_heads)) with a state S[v, k] (V x K), per token:
 *
 *   dt    = min(max(softplus(dt_raw[h] + dt_bias[h]), dt_min), dt_max),  A = -exp(A_log[h])
 *   beta  = sigmoid(beta_raw[h])
 *   k^    = k / sqrt(sum k^2 + eps),   q^ = q / sqrt(sum q^2 + eps)
 *   S    <- exp(dt A) S
 *   S    <- S + beta (v - S k^) k^T
 *   y     = scale S q^
 *
 * The step size and decay are those of axon_ssd_scan; the convolution, gate, norm and projections
 * of the block are the caller's (axon_group_norm is the norm). axon_gated_delta_scan runs chunks of
 * 64 tokens on the matrix cores: with g the inclusive sum of dt A inside the chunk and S0 the
 * entering state, D = T (v - e^g S0 k^), T = (I + M)^-1 diag(beta), M[t,s] = beta_t e^(g_t - g_s)
 * k^_t.k^_s for s < t, are the chunk's corrected writes. axon_gated_delta_step is the recurrence
 * itself for one token a row. All sums, decays and states are fp32. The scan's products are off by
 * about 2^-23 of the largest entry of their row or column in a chunk, so that errors are relative to
 * the largest entries of a state's row (and of v's column) in a chunk, not to each. Squares of a row
 * of q or k must not sum beyond the range of fp32.
 *
 * Layouts: q, k (tokens, key_heads, K); v (tokens, value_heads, V); dt_raw, beta_raw
 * (tokens, value_heads); y (tokens, value_heads, V); activation dtype. The rows of q, k and v may
 * lie q_stride, k_stride, v_stride elements apart (parts of one projection's output; 0 = dense;
 * else a multiple of 8 elements, at least the row's own length); everything else is contiguous.
 *   A_log, dt_bias (value_heads) fp32;  pools of states (slots, value_heads, V, K) fp32.
 * Supported: K 64 or 128; V a multiple of 16 up to 256; value_heads a multiple of key_heads (else
 * AXON_ERR_UNSUPPORTED); sequences and heads in [1, 65535]; sequences * value_heads < 2^20;
 * tokens < 2^29; rows and their strides at most 2^22 elements; tokens * stride and slots *
 * value_heads * V * K <= 2^40. Device pointers 16-byte aligned, integer arrays 4-byte.
 *
 * Slots: sequence (or row) n uses state slots[n] of the pool, or state n where slots is NULL (the
 * pool then holds at least `sequences` states). A slot outside the pool means no state: a scan starts from
 * zeros (in_slots) or does not store the final state (out_slots), a step leaves the row's y as it
 * was and touches no state. The slots of one call that are written must be distinct, and no
 * sequence may read a slot that another one writes; else those states and outputs are
 * unspecified (no other memory is touched).
 *
 * NaN in a token's k, v, dt_raw or beta_raw makes the state NaN (that of v its own row v), and with
 * it the outputs of its head from there on (a scan: those of its 64-token chunk may be as well); so
 * does an infinity, unless dt_raw or beta_raw has it, where it is their limit. One exception: a long
 * sequence of few heads is walked in segments, and the state behind one forgets what decays have
 * since multiplied by less than 2^-160, NaN too. No other sequence or head sees it. */
typedef struct {
  int64_t sequences;    /* batch rows, or packed sequences */
  int64_t tokens;       /* rows of q, k, v: sequences * seqlen, or the packed buffer's rows */
  int64_t key_heads;
  int64_t value_heads;
  int64_t key_dim;      /* K */
  int64_t value_dim;    /* V */
  int64_t q_stride;     /* elements between the rows of q, k, v; 0 = dense */
  int64_t k_stride;
  int64_t v_stride;
  int64_t state_slots;  /* states of the pool state_in (of the step's pool) */
  int64_t out_slots;    /* states of the pool state_out; equal to state_slots in place; not read by
                           the step */
  int32_t act_dtype;    /* an axon_dtype value */
} axon_gated_delta_shape;

typedef struct {
  const float* A_log;    /* (value_heads) */
  const float* dt_bias;  /* (value_heads) */
  float dt_min;          /* as for axon_ssd_scan */
  float dt_max;
  float scale;           /* of the readout, finite; K^-0.5 is usual */
  float eps;             /* of the norms of q and k, finite and > 0 */
} axon_gated_delta_params;

/* Bytes of device workspace axon_gated_delta_scan needs (0 for an invalid shape or tokens == 0). */
size_t axon_gated_delta_scan_workspace_bytes(const axon_gated_delta_shape* shape);

/* Runs every sequence. tables: NULL for a uniform batch (tokens must be a multiple of sequences),
 * else the packed sequences' tables of axon_sequence_tables for these sequences, these tokens as
 * total_tokens and block 64 (other contents give unspecified results, but no access outside the
 * arrays). Rows of y behind the last sequence are left as they were. state_in NULL: zeros.
 * state_out NULL: the final states are not stored. state_out may equal state_in but must not
 * overlap it otherwise; y and state_out overlap nothing else. A sequence without tokens copies its
 * state. Running L1 tokens then L2 from the returned state equals running L1 + L2 up to rounding.
 * workspace: device memory, 16-byte aligned, no initialisation needed; two calls that may overlap
 * in time need one each. */
axon_status axon_gated_delta_scan(const axon_gated_delta_shape* shape,
                                  const axon_gated_delta_params* params, const void* q,
                                  const void* k, const void* v, const void* dt_raw,
                                  const void* beta_raw, const int32_t* tables,
                                  const float* state_in, const int32_t* in_slots, void* y,
                                  float* state_out, const int32_t* out_slots, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* One token for each of `sequences` rows (tokens == sequences), states updated in place. */
axon_status axon_gated_delta_step(const axon_gated_delta_shape* shape,
                                  const axon_gated_delta_params* params, const void* q,
                                  const void* k, const void* v, const void* dt_raw,
                                  const void* beta_raw, float* state, const int32_t* slots,
                                  void* y, void* stream);

/* ---- Group norm ------------------------------------------------------------------------------
 * The normalisation behind a scan, channels last, with its activation and gate in one pass. Every
 * row of x (rows, groups * width) is one token; every group of `width` channels has statistics of
 * its own (over time as well they would see the future of a causal layer):
 *
 *   u = x, or x SiLU(z)                                      (gate AXON_GATE_BEFORE)
 *   n = (u - mean(u)) / sqrt(var(u) + eps)    centered;  u / sqrt(mean(u^2) + eps)    otherwise
 *   y = n weight + bias;   y = SiLU(y) (activation AXON_ACT_SILU);   y = y SiLU(z) (AXON_GATE_AFTER)
 *
 * x, z, y: activation dtype, rows x_stride / z_stride elements apart (0 = dense; else at least
 * groups * width, any alignment of an element); y dense, fp32 statistics, rounded once. weight and
 * bias: fp32, (groups * width), or (width) where shared_weights is set; either may be NULL (ones,
 * zeros). y may equal x where x is dense; else y overlaps nothing. rows >= 0; groups, width >= 1;
 * groups * width <= 2^30; rows * groups < 2^31; rows * groups * width <= 2^40. x, z, y and the
 * parameters need the alignment of an element only. */
enum { AXON_ACT_NONE = 0, AXON_ACT_SILU = 1 };
enum { AXON_GATE_NONE = 0, AXON_GATE_BEFORE = 1, AXON_GATE_AFTER = 2 };

typedef struct {
  int64_t rows;
  int64_t groups;
  int64_t width;           /* channels of a group */
  int64_t x_stride;        /* elements between rows; 0 = dense */
  int64_t z_stride;
  float eps;               /* finite, >= 0 */
  int32_t act_dtype;       /* an axon_dtype value */
  int32_t centered;        /* 0 or 1 */
  int32_t activation;      /* AXON_ACT_* */
  int32_t gate;            /* AXON_GATE_*; z is not read with AXON_GATE_NONE */
  int32_t shared_weights;  /* 0 or 1 */
} axon_group_norm_desc;

axon_status axon_group_norm(const axon_group_norm_desc* desc, const void* x, const void* z,
                            const float* weight, const float* bias, void* y, void* stream);

/* ---- Gated linear recurrence -------------------------------------------------------------------
 * One state a channel, with a decay and an input that are gated by the token. For every sequence and
 * channel e, per token:
 *
 *   dt    = sigmoid(dt_raw + dt_bias[e])   (AXON_LINEAR_SIGMOID), or softplus(..) (AXON_LINEAR_SOFTPLUS)
 *   log a = -exp(A_log[e]) dt
 *   u     = x sigmoid(in_raw + in_bias[e]), or x where in_raw is NULL
 *   h    <- a h + m u,  m = 1 (AXON_INPUT_PLAIN), 1 - a (AXON_INPUT_COMPLEMENT),
 *                           sqrt(1 - a^2) (AXON_INPUT_SQRT)
 *   y     = h
 *
 * (With softplus, A_log = 0 and the complement, a = 1 - z and m = z for the gate z = sigmoid(dt_raw
 * + dt_bias).) Gates, decays and states are fp32, y is rounded once. Where a >= 1/2, states are handed
 * on as h + expm1(log a) h, so that slow decays lose nothing to the rounding of a, in a long scan as in many
 * short ones: from the state that a sequence begins with, every 16 tokens at most, to the one that it hands
 * back, which its last y shows, and so their gradients. The y between multiply by a (off by 32 2^-24 of h
 * at most, which does not add up).
 *
 * Layouts: x, dt_raw, in_raw, y (tokens, channels), activation dtype; the rows of x, dt_raw, in_raw
 * and dy may lie x_stride, dt_stride, in_stride, dy_stride elements apart (0 = dense, else at least
 * `channels`); y and the gradients are dense. A_log, dt_bias, in_bias (channels) fp32; the biases
 * may be NULL (zeros). Pools of states (slots, channels) fp32. Sequences (a uniform batch, or packed
 * with tables of block 64) and slots as for axon_gated_delta_scan. Activations need the alignment of an
 * element only, fp32 and integer arrays 4-byte.
 * Limits: sequences in [1, 65535]; channels in [1, 2^22]; tokens < 2^29; strides up to 2^22; tokens *
 * stride and slots * channels <= 2^40; (tokens / 64 + sequences) * channels < 2^37.
 *
 * A value that is not finite in a token's x, dt_raw or in_raw makes its channel's state not finite
 * from there on, unless a gate has an infinity, where it is the gate's limit. No other channel or
 * sequence sees it. */
enum { AXON_LINEAR_SIGMOID = 0, AXON_LINEAR_SOFTPLUS = 1 };
enum { AXON_INPUT_PLAIN = 0, AXON_INPUT_COMPLEMENT = 1, AXON_INPUT_SQRT = 2 };

typedef struct {
  int64_t sequences;    /* batch rows, or packed sequences; the step's rows */
  int64_t tokens;       /* rows of x: sequences * seqlen, or the packed buffer's rows */
  int64_t channels;     /* E */
  int64_t x_stride;     /* elements between rows; 0 = dense */
  int64_t dt_stride;
  int64_t in_stride;
  int64_t dy_stride;    /* read by the backward pass only */
  int64_t state_slots;  /* states of the pool state_in (of the step's pool); not read by the backward pass */
  int64_t out_slots;    /* states of the pool state_out; not read by the step and the backward pass */
  int32_t act_dtype;    /* an axon_dtype value */
  int32_t gate;         /* AXON_LINEAR_* */
  int32_t input_scale;  /* AXON_INPUT_* */
  int32_t clear_behind; /* 1: rows of y behind the last sequence get zeros; 0: they are left as they
                           were. Read by the scan only */
} axon_linear_shape;

typedef struct {
  const float* A_log;    /* (channels) */
  const float* dt_bias;  /* (channels) or NULL */
  const float* in_bias;  /* (channels) or NULL; not read where in_raw is NULL */
} axon_linear_params;

/* Rows of `checkpoints`: blocks of 64 tokens that sequences of these tokens can have, packed
 * (tokens / 64 + sequences) or uniform. 0 for invalid arguments. */
size_t axon_linear_checkpoint_rows(int64_t sequences, int64_t tokens, int32_t packed);

/* Bytes of device workspace axon_linear_scan needs (0 for an invalid shape; 0 is possible). */
size_t axon_linear_scan_workspace_bytes(const axon_linear_shape* shape);

/* Runs every sequence. tables, state_in, in_slots, state_out, out_slots and workspace as for
 * axon_gated_delta_scan, with the same rules of aliasing. checkpoints: NULL, or
 * (axon_linear_checkpoint_rows, channels) fp32, which receives the state that enters each block of
 * 64 tokens, for the backward pass (rows of blocks that no sequence has are left as they were). */
axon_status axon_linear_scan(const axon_linear_shape* shape, const axon_linear_params* params,
                             const void* x, const void* dt_raw, const void* in_raw,
                             const int32_t* tables, const float* state_in, const int32_t* in_slots,
                             void* y, float* state_out, const int32_t* out_slots,
                             float* checkpoints, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Bytes of device workspace axon_linear_scan_backward needs (0 for an invalid shape). */
size_t axon_linear_scan_backward_workspace_bytes(const axon_linear_shape* shape);

/* Gradients of axon_linear_scan: from dy (tokens, channels) and dstate_out (sequences, channels; the
 * gradient of each sequence's final state, NULL = zeros), with the inputs, tables and checkpoints of
 * the forward call, to
 *   dx, ddt_raw, din_raw (tokens, channels) activation dtype; zeros behind the last sequence
 *   dA_log, ddt_bias, din_bias (channels) fp32, summed over all tokens in an order of their own that
 *       does not change from call to call
 *   dstate_in (sequences, channels) fp32; NULL = not stored
 * din_raw and din_bias belong to in_raw: all three or none. Where m = sqrt(1 - a^2) is 0 the gradient
 * of its input term is taken as 0 (its limit for the gate). Outputs overlap nothing. */
axon_status axon_linear_scan_backward(const axon_linear_shape* shape,
                                      const axon_linear_params* params, const void* dy,
                                      const void* x, const void* dt_raw, const void* in_raw,
                                      const int32_t* tables, const float* checkpoints,
                                      const float* dstate_out, void* dx, void* ddt_raw,
                                      void* din_raw, float* dA_log, float* ddt_bias,
                                      float* din_bias, float* dstate_in, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* One token for each of `sequences` rows (tokens == sequences), states updated in place. A row whose
 * slot lies outside the pool is idle: its y stays as it was and no state is touched. */
axon_status axon_linear_step(const axon_linear_shape* shape, const axon_linear_params* params,
                             const void* x, const void* dt_raw, const void* in_raw, float* state,
                             const int32_t* slots, void* y, void* stream);

/* ---- Causal depthwise convolution --------------------------------------------------------------
 * The convolution in front of a scan, by itself: for every sequence and channel e
 *
 *   p_t = conv_b[e] + sum_k conv_w[e,k] xx[t - 3 + k],  k = 0 .. 3
 *   y_t = p_t, or SiLU(p_t) (AXON_CONV_SILU)
 *
 * xx[s] is x for s >= 0 and the sequence's cache (its last three inputs, oldest first) for s < 0, as in
 * axon_ssm_prefill. Layouts: x, y (tokens, channels), activation dtype, the rows of x and dy x_stride,
 * dy_stride elements apart (0 = dense); conv_w (channels, 4), conv_b (channels, or NULL = zeros)
 * fp32; pools of caches (slots, 3, channels) fp32. Sums are fp32 and rounded once. Sequences, tables
 * (block 64), slots, alignment and limits as for axon_linear_scan (slots * 3 * channels <= 2^40). */
typedef struct {
  int64_t sequences;
  int64_t tokens;
  int64_t channels;
  int64_t x_stride;
  int64_t dy_stride;    /* read by the backward pass only */
  int64_t cache_slots;  /* caches of the pool cache_in (of the step's pool); not read by the backward pass */
  int64_t out_slots;    /* caches of the pool cache_out; read by the forward pass only */
  int32_t act_dtype;
  int32_t activation;   /* AXON_CONV_NONE or AXON_CONV_SILU */
  int32_t clear_behind; /* as in axon_linear_shape */
} axon_conv_shape;

/* cache_in NULL: zeros. cache_out NULL: not stored. cache_out may equal cache_in (then with as many
 * slots) but must not overlap it otherwise; outputs overlap nothing else. A sequence without tokens
 * copies its cache. The cache holds exact copies of the inputs. */
axon_status axon_causal_conv(const axon_conv_shape* shape, const void* x, const float* conv_w,
                             const float* conv_b, const int32_t* tables, const float* cache_in,
                             const int32_t* in_slots, void* y, float* cache_out,
                             const int32_t* out_slots, void* stream);

/* Bytes of device workspace axon_causal_conv_backward needs (0 for an invalid shape). */
size_t axon_causal_conv_backward_workspace_bytes(const axon_conv_shape* shape);

/* Gradients of axon_causal_conv from dy (tokens, channels) and dcache_out (sequences, 3, channels, or
 * NULL = zeros), with the inputs of the forward call; cache_in is (sequences, 3, channels) or NULL.
 * dx (tokens, channels), zeros behind the last sequence; dconv_w (channels, 4), dconv_b (channels)
 * fp32, summed in an order that does not change from call to call; dcache_in (sequences, 3,
 * channels) or NULL. Outputs overlap nothing. */
axon_status axon_causal_conv_backward(const axon_conv_shape* shape, const void* dy, const void* x,
                                      const float* conv_w, const float* conv_b,
                                      const int32_t* tables, const float* cache_in,
                                      const float* dcache_out, void* dx, float* dconv_w,
                                      float* dconv_b, float* dcache_in, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* One token for each of `sequences` rows (tokens == sequences), caches updated in place; idle rows as
 * in axon_linear_step. */
axon_status axon_causal_conv_step(const axon_conv_shape* shape, const void* x, const float* conv_w,
                                  const float* conv_b, float* cache, const int32_t* slots, void* y,
                                  void* stream);

/* ---- Head norm with position rotation ----------------------------------------------------------
 * Queries and keys before attention or before axon_gated_delta_scan: every head of head_dim D
 * channels is normalised and its first rotary_dim R channels are turned by the token's position, in
 * one pass over both tensors. Per row (token) with position p and head:
 *
 *   n = x / sqrt(mean(x^2) + eps) w
 *   (n_i, n_j) <- (n_i cos - n_j sin, n_j cos + n_i sin) of the angle p freqs[c],  c = 0 .. R / 2 - 1
 *
 * where pair c is (c, c + R / 2), or (2 c, 2 c + 1) with `interleaved`. Angles are reduced in 64 bits,
 * so that far positions lose nothing; sums and products are fp32 and rounded once.
 *
 * q (rows, q_heads, D), k (rows, k_heads, D; k_heads = 0: none), activation dtype, rows q_stride /
 * k_stride elements apart (0 = dense, else at least heads * D); outputs dense. positions (rows) int32,
 * any sign; freqs (R / 2) fp64, radians a token; weights (D) fp32 or NULL (ones). q_out may equal q
 * (and k_out k) where that is dense, else outputs overlap nothing.
 * Limits: D even, in [2, 256]; R even, in [2, D]; q_heads in [1, 65535], k_heads in [0, 65535]; rows
 * < 2^31; strides up to 2^31; rows * stride <= 2^40. Activations need the alignment of an element
 * only, fp32 and int32 arrays 4-byte, freqs 8-byte. Squares of a head must not sum beyond fp32 nor, where eps
 * is 0, have a mean below its least normal number, 2^-126. */
typedef struct {
  int64_t rows;
  int64_t q_heads;
  int64_t k_heads;
  int64_t head_dim;     /* D */
  int64_t rotary_dim;   /* R */
  int64_t q_stride;     /* elements between the rows of q; 0 = dense */
  int64_t k_stride;
  int64_t dq_stride;    /* of the output gradients; read by the backward pass only */
  int64_t dk_stride;
  float eps;            /* finite, >= 0 */
  int32_t act_dtype;
  int32_t interleaved;  /* 0 or 1 */
} axon_norm_rotate_desc;

axon_status axon_norm_rotate(const axon_norm_rotate_desc* desc, const void* q, const void* k,
                             const int32_t* positions, const double* freqs, const float* q_weight,
                             const float* k_weight, void* q_out, void* k_out, void* stream);

/* Bytes of device workspace axon_norm_rotate_backward needs (0 for an invalid desc or no rows). */
size_t axon_norm_rotate_backward_workspace_bytes(const axon_norm_rotate_desc* desc);

/* Gradients from dq_out, dk_out (rows, heads, D) with the inputs of the forward call: dq, dk dense,
 * activation dtype; dq_weight, dk_weight (D) fp32, each NULL = not wanted, summed in an order that does
 * not change from call to call. dq may equal a dense dq_out (dk dk_out); else outputs overlap nothing. */
axon_status axon_norm_rotate_backward(const axon_norm_rotate_desc* desc, const void* dq_out,
                                      const void* dk_out, const void* q, const void* k,
                                      const int32_t* positions, const double* freqs,
                                      const float* q_weight, const float* k_weight, void* dq,
                                      void* dk, float* dq_weight, float* dk_weight,
                                      void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* AXONSCAN_H_ */
