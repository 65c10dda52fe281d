/*
 * ssm_mi355x.h -- C ABI of the MI355X (gfx950) selective-scan library.
 *
 * Three entry points, one per path of the Mamba-style selective state space
 * layer described by the pages:
 *
 *   ssm_scan_fwd        full-sequence (prefill) scan: causal depthwise conv1d
 *                       + SiLU, dt = clip(softplus(dt_proj + dt_bias)), the
 *                       diagonal recurrence h_t = exp(dt*A) h_{t-1} + dt*B_t*u_t,
 *                       y_t = C_t . h_t + D*u_t, gate y * SiLU(z).  Page
 *                       "Axon-SSM: selective state space model", sections
 *                       "Algorithm", "SSM scan", "Discretization", "JIT-compiled
 *                       kernels" and "Autoregressive decoding" (prefill,
 *                       cache = None).
 *   ssm_decode_step     one token of autoregressive decoding that updates
 *                       [conv_cache, ssm_state] in place.  Same page, section
 *                       "Autoregressive decoding" (decode, cache =
 *                       [conv_cache, ssm_state]).
 *   ssm_chunk_scan_fwd  multi-head chunked scan (scalar A per head): page "What
 *                       is the Mamba model?", sections "chunkscan" and
 *                       "chunkscan implementation", chunk output formula
 *                       out[l] = sum_{s<=l} cb[l,s] e^{dA[l]-dA[s]} dt[s] x[s]
 *                              + e^{dA[l]} C[l] prev_states + D x[l],
 *                       with the chunk-final state carried to the next chunk.
 *
 * Next to them: the multi-head scan's decode step, the scan's backward, the
 * layer's projections and the whole layer; the gated delta rule
 * (ssm_delta_chunk_fwd, ssm_delta_chunk_bwd, ssm_delta_decode_step), the
 * norms before and after a block (ssm_block_norm_fwd, ssm_block_norm_bwd) and
 * attention with a sliding window and sinks with its paged cache (ssm_attn_fwd,
 * ssm_attn_bwd, ssm_attn_cache_write, ssm_attn_decode_step).
 *
 * Conventions shared by every entry point
 *  - Every tensor pointer is a DEVICE pointer owned by the caller.  The scan,
 *    chunked-scan, decode and backward entry points allocate nothing, keep no
 *    per-call state, never copy between host and device and never
 *    synchronise.  The projection entry points (ssm_linear_fwd,
 *    ssm_layer_fwd) are the exception: the first call of a shape on a device
 *    creates that device's hipBLASLt handle and the shape's matmul plan, both
 *    of which allocate host and device memory inside the GEMM library, and
 *    keeps them until the process ends; later calls of the same shape
 *    allocate nothing.
 *  - Work is enqueued on `stream` (a hipStream_t passed as void*; NULL is the
 *    null stream) and the call returns at once.  Asynchronous kernel faults
 *    surface at the caller's next synchronisation.
 *  - Layouts are dense row-major in the order written next to each field, last
 *    index fastest.  Pointers must be aligned to their element size.
 *  - Every argument error is detected before anything is launched: the call
 *    returns SSM_ERR_INVALID_ARG or SSM_ERR_UNSUPPORTED and writes nothing;
 *    ssm_last_error() then names the field.  A failed launch returns
 *    SSM_ERR_HIP.  NaN/Inf inputs are not checked; they propagate.
 *  - Outputs (y, out) must not overlap any input.  State and cache outputs may
 *    alias their inputs exactly (in-place update).
 *  - Floating point: all arithmetic is fp32; bf16 inputs are widened exactly;
 *    bf16 outputs are rounded to nearest-even.
 */
#ifndef SSM_MI355X_H
#define SSM_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 2

/* element types (int32 fields in the structs below).  SSM_E4M3 (8 bits: sign, 4 of
 * exponent, 3 of fraction, largest 448, no infinity) only for the attention's cache. */
typedef enum { SSM_F32 = 0, SSM_BF16 = 1, SSM_E4M3 = 2 } ssm_dtype_t;

/* How B is discretized.  SSM_EULER: dB u = dt B u (the "dB * x_t" of the
 * Axon-SSM page's kernel section and the dt[s] x[s] of the velog page's chunk
 * formula).  SSM_ZOH: the zero-order hold of the molayo page's "Technical
 * details", dB u = ((e^{dt A} - 1) / A) B u.  The decay is e^{dt A} in both. */
typedef enum { SSM_EULER = 0, SSM_ZOH = 1 } ssm_discretization_t;

/* return codes */
typedef enum {
  SSM_OK = 0,
  SSM_ERR_INVALID_ARG = 1, /* a null required pointer, a negative size, bad bounds, wrong struct_size */
  SSM_ERR_UNSUPPORTED = 2, /* a valid request this build does not implement (e.g. d_state != 16) */
  SSM_ERR_WORKSPACE = 3,   /* workspace missing or smaller than the *_workspace_size query */
  SSM_ERR_HIP = 4,         /* the HIP runtime rejected a launch */
  SSM_ERR_INTERNAL = 5     /* debug builds only: a launch plan broke an invariant its kernels rely on */
} ssm_status_t;

/* ------------------------------------------------------------------------
 * Full-sequence scan (prefill).
 *
 * Shapes: Bt = batch, L = seqlen, E = dim (channels), N = d_state.
 *   x             (Bt, L, E) x_dtype     pre-conv x_branch when conv_w != NULL, else u itself
 *   conv_w        (E, K) f32 or NULL     causal depthwise conv; NULL skips conv and SiLU.
 *                                        xc[t] = sum_k conv_w[e,k] * xpad[t+k] (+ conv_b[e]),
 *                                        xpad = (conv_cache_in or zeros, x) along t, so
 *                                        conv_w[e,K-1] multiplies the current token;
 *                                        u = SiLU(xc).  K = conv_k must be 4.
 *   conv_b        (E) f32 or NULL
 *   conv_cache_in (Bt, E, K-1) f32 or NULL (zeros): raw pre-conv inputs before t=0, oldest first
 *   conv_cache_out(Bt, E, K-1) f32 or NULL: the last K-1 raw inputs (including cache_in
 *                                        values when L < K-1), oldest first; may alias conv_cache_in
 *   dt            dt_rank1 != 0: (Bt, L) f32 r, and pre = dt_w[e] * r[b,t] (dt_proj 1 -> E)
 *                 dt_rank1 == 0: (Bt, L, E) dt_dtype, and pre = dt[b,t,e]
 *   dt_w          (E) f32, required iff dt_rank1
 *   dt_bias       (E) f32 or NULL (zero)
 *   dt_softplus   nonzero: dt = clip(softplus(pre + dt_bias), dt_min, dt_max)
 *                 zero:    dt = clip(pre + dt_bias, dt_min, dt_max)
 *   dt_min/dt_max clip bounds (inclusive); -INFINITY / +INFINITY disable a side; dt_min <= dt_max
 *   A             (E, N) f32, the continuous-time diagonal (normally A = -exp(A_log) < 0)
 *   B, C          (Bt, L, N) bc_dtype
 *   D             (E) f32 or NULL (no skip term)
 *   z             (Bt, L, E) z_dtype or NULL (no gate); z_dtype must equal x_dtype
 *   ssm_state_in  (Bt, E, N) f32 or NULL (zeros, the prefill start)
 *   ssm_state_out (Bt, E, N) f32 or NULL; may alias ssm_state_in
 *   y             (Bt, L, E) y_dtype: y_t = (C_t . h_t + D*u_t) * SiLU(z_t)
 *   workspace     device scratch of at least ssm_scan_workspace_size(p) bytes (may be
 *                 NULL when that size is 0); 256-byte aligned; not touched by other calls
 *   time_split    0: the library chooses; >= 1: split the sequence into at most that
 *                 many segments scanned in parallel and combined (at most 32; every
 *                 segment but the last spans a multiple of 8 steps);
 *                 SSM_SCAN_BLOCKED (-1): one pass over 16-step blocks, 16 channels per
 *                 wave, blocks whose dt sits at dt_max in every channel computed as
 *                 matrix-core products of per-block tables (the chunk form of the
 *                 velog page's "chunkscan"); it takes bf16 x and z, an E-wide bf16
 *                 dt, no conv, SSM_EULER, dim % 64 == 0, x/z/dt/bf16 y 8-byte and
 *                 fp32 y and ssm_state_out 16-byte aligned (else SSM_ERR_UNSUPPORTED).
 *                 With 0 the library takes it for such calls when batch * dim / 64 >= 768.
 *   discretization SSM_EULER or SSM_ZOH (see ssm_discretization_t)
 * Supported: N = 16.  L = 0 only copies the state/cache inputs to the outputs.
 * ---------------------------------------------------------------------- */
#define SSM_SCAN_BLOCKED (-1) /* ssm_scan_params_t.time_split: the blocked single-pass scan */

typedef struct ssm_scan_params {
  uint32_t struct_size; /* = sizeof(ssm_scan_params_t) */
  int32_t batch, seqlen, dim, d_state;
  int32_t conv_k;
  const void *x;
  int32_t x_dtype;
  const float *conv_w;
  const float *conv_b;
  const float *conv_cache_in;
  float *conv_cache_out;
  const void *dt;
  int32_t dt_dtype;
  int32_t dt_rank1;
  const float *dt_w;
  const float *dt_bias;
  int32_t dt_softplus;
  float dt_min, dt_max;
  const float *A;
  const void *B;
  const void *C;
  int32_t bc_dtype;
  const float *D;
  const void *z;
  int32_t z_dtype;
  const float *ssm_state_in;
  float *ssm_state_out;
  void *y;
  int32_t y_dtype;
  int32_t time_split;
  void *workspace;
  size_t workspace_bytes;
  int32_t discretization; /* SSM_EULER (0): dB u = dt B u; SSM_ZOH (1): ((e^{dt A} - 1) / A) B u */
} ssm_scan_params_t;

ssm_status_t ssm_scan_fwd(const ssm_scan_params_t *p, void *stream);
size_t ssm_scan_workspace_size(const ssm_scan_params_t *p);
/* Validation only: the status ssm_scan_fwd would return before launching. */
ssm_status_t ssm_scan_check(const ssm_scan_params_t *p);

/* ------------------------------------------------------------------------
 * ssm_scan_fwd for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same computation, kernels and results as ssm_scan_fwd, with the
 * workspace taken from a scratch array inside the library instead of the
 * caller.  p->workspace must be NULL and p->workspace_bytes 0 (else
 * SSM_ERR_INVALID_ARG); every other field is as for ssm_scan_fwd, and the
 * caller still owns the inputs and outputs.  The call allocates nothing and
 * calls no allocating routine.
 *  - The scratch holds SSM_SCAN_NOALLOC_MAX_BYTES (64 MiB).  A call whose
 *    ssm_scan_workspace_size(p) exceeds it returns SSM_ERR_WORKSPACE, with the
 *    size in ssm_last_error(), before anything is launched.  (It covers, for
 *    example, batch 8 x 4096 tokens and batch 1 x 2048 tokens at E 7680 with
 *    the library's own time split.)
 *  - Each GPU the library runs on holds one copy of the scratch for the life
 *    of the process.  Its address on a device is looked up on the first call
 *    made there (with that device current); a failure of that lookup returns
 *    SSM_ERR_HIP.
 *  - Every call on one GPU uses that GPU's single copy: calls that may run at
 *    the same time on one GPU (different streams without ordering between
 *    them, or different threads) race on it and must not overlap.  Calls on
 *    one stream are ordered and safe.  Nothing in the scratch needs to start
 *    at zero; it keeps the last call's contents.
 * ---------------------------------------------------------------------- */
#define SSM_SCAN_NOALLOC_MAX_BYTES ((size_t)64 << 20)
ssm_status_t ssm_scan_fwd_noalloc(const ssm_scan_params_t *p, void *stream);

/* ------------------------------------------------------------------------
 * One decode step, in place.  Shapes as above with L = 1:
 *   x (Bt, E) x_dtype new token (pre-conv when conv_w != NULL); z (Bt, E) or NULL;
 *   dt: dt_rank1 ? (Bt) f32 r : (Bt, E) dt_dtype;  B, C (Bt, N) bc_dtype;
 *   conv_cache (Bt, E, K-1) f32, read then overwritten with the window shifted by one
 *   (required iff conv_w != NULL);  ssm_state (Bt, E, N) f32, read then overwritten;
 *   y (Bt, E) y_dtype.
 * ssm_state, A and conv_w must be 16-byte aligned, B and C aligned to 4
 * elements (16 bytes in f32, 8 in bf16); batch * dim < 2^31.
 * The result equals ssm_scan_fwd with L = 1, conv_cache_in = conv_cache_out =
 * conv_cache and ssm_state_in = ssm_state_out = ssm_state.
 * ---------------------------------------------------------------------- */
typedef struct ssm_decode_params {
  uint32_t struct_size; /* = sizeof(ssm_decode_params_t) */
  int32_t batch, dim, d_state, conv_k;
  const void *x;
  int32_t x_dtype;
  const float *conv_w;
  const float *conv_b;
  float *conv_cache;
  const void *dt;
  int32_t dt_dtype;
  int32_t dt_rank1;
  const float *dt_w;
  const float *dt_bias;
  int32_t dt_softplus;
  float dt_min, dt_max;
  const float *A;
  const void *B;
  const void *C;
  int32_t bc_dtype;
  const float *D;
  const void *z;
  int32_t z_dtype;
  float *ssm_state;
  void *y;
  int32_t y_dtype;
  int32_t discretization; /* as in ssm_scan_params_t */
} ssm_decode_params_t;

ssm_status_t ssm_decode_step(const ssm_decode_params_t *p, void *stream);
ssm_status_t ssm_decode_check(const ssm_decode_params_t *p);

/* ------------------------------------------------------------------------
 * Multi-head chunked scan (SSD form), scalar A per head.
 *   x         (Bt, L, H, P) x_dtype
 *   dt        (Bt, L, H) f32 raw; dt = clip(softplus(dt + dt_bias[h]), dt_min, dt_max)
 *             (softplus skipped when dt_softplus == 0)
 *   dt_bias   (H) f32 or NULL
 *   A         (H) f32 (negative)
 *   B, C      (Bt, L, G, N) bc_dtype; head h reads group h / (H / G)
 *   D         (H) f32 (d_per_channel == 0) or (H, P) f32 (d_per_channel != 0) or NULL
 *   state_in  (Bt, H, P, N) f32 or NULL (zeros); state_out (Bt, H, P, N) f32 or NULL
 *   out       (Bt, L, H, P) out_dtype
 *   dA[l] = sum_{i<=l} dt[i] A_h inside each chunk of chunk_size tokens (inclusive);
 *   state passing: S <- e^{dA[Q-1]} S + sum_s e^{dA[Q-1]-dA[s]} dt[s] x[s] (outer) B[s].
 * A sequence that is not a whole number of chunks ends with a shorter chunk
 * (the same formulas over its own length).
 * Supported: chunk_size up to 256, d_state up to 128, headdim up to 128, x,
 * B/C, z and out each in f32 or bf16, and seqlen * max(nheads * headdim,
 * ngroups * d_state) * 2 bytes (one batch row) below 4 GiB.  Two kernels
 * share the work: N = 64, chunk_size = 128, bf16 x and B/C and headdim a
 * multiple of 16 run the matrix-core kernel (x, B, C, out and z 16-byte
 * aligned; it may cut each sequence into segments, see `segments`); every
 * other shape runs chunk by chunk on the vector ALUs in fp32 (pointers
 * aligned to their element size; `segments` has no effect there: every chunk
 * already starts from the state composed ahead of it).  The result is the
 * same function either way, up to rounding order.
 * Workspace: ssm_chunk_scan_workspace_size() bytes of device memory, 256-byte
 * aligned, owned by the caller (zero for the matrix-core kernel when the
 * sequences are not cut into segments; batch * nchunks * nheads * (headdim *
 * d_state + 1) floats, rounded up, for the vector-ALU kernels); its contents
 * on entry do not matter.
 * ---------------------------------------------------------------------- */
typedef struct ssm_chunk_params {
  uint32_t struct_size; /* = sizeof(ssm_chunk_params_t) */
  int32_t batch, seqlen, nheads, headdim, ngroups, d_state, chunk_size;
  const void *x;
  int32_t x_dtype;
  const float *dt;
  const float *dt_bias;
  int32_t dt_softplus;
  float dt_min, dt_max;
  const float *A;
  const void *B;
  const void *C;
  int32_t bc_dtype;
  const float *D;
  int32_t d_per_channel;
  const float *state_in;
  float *state_out;
  void *out;
  int32_t out_dtype;
  void *workspace;
  size_t workspace_bytes;
  const void *z;        /* (Bt, L, H, P) z_dtype or NULL: out *= SiLU(z) after the D skip */
  int32_t z_dtype;
  int32_t segments;     /* 0: chosen by the library; else cut each sequence into this many
                           runs of whole chunks (at most 16, and at most one per chunk) that
                           start from states composed ahead of them; the result is the same
                           up to rounding order */
} ssm_chunk_params_t;

ssm_status_t ssm_chunk_scan_fwd(const ssm_chunk_params_t *p, void *stream);
size_t ssm_chunk_scan_workspace_size(const ssm_chunk_params_t *p);
ssm_status_t ssm_chunk_scan_check(const ssm_chunk_params_t *p);

/* ------------------------------------------------------------------------
 * Backward of ssm_scan_fwd (Euler form) with recomputation (page "Mamba/SSM
 * basics", the production recipe after "Technical details": intermediate
 * states are recomputed in the backward pass instead of being stored).  Given
 * dy = dL/dy (Bt, L, E) dy_dtype and optionally dstate_out = dL/dh_L
 * (Bt, E, N) f32, writes the gradients of L with respect to the forward's
 * inputs, all f32 and in the inputs' shapes:
 *   dx (Bt, L, E); dz (Bt, L, E) when z was given; ddt: (Bt, L) for a rank-1
 *   dt (gradient of r), else (Bt, L, E); ddt_w (E) for a rank-1 dt; ddt_bias (E);
 *   dA (E, N); dB, dC (Bt, L, N); dD (E); dconv_w (E, 4), dconv_b (E) and
 *   dconv_cache (Bt, E, 3) when there is a conv; dstate_in (Bt, E, N).
 * Any gradient pointer may be NULL (not written).  The forward inputs are the
 * fields of the same names in ssm_scan_params_t with the same rules; the
 * clip passes gradient strictly inside (dt_min, dt_max).  Sums over
 * channels and time are taken in a fixed order (results are deterministic).
 * The workspace holds ssm_scan_bwd_workspace_size(p) bytes (256-byte aligned).
 * Supported: N = 16, Euler discretization; dy_dtype f32 or bf16.
 * ---------------------------------------------------------------------- */
typedef struct ssm_scan_bwd_params {
  uint32_t struct_size; /* = sizeof(ssm_scan_bwd_params_t) */
  int32_t batch, seqlen, dim, d_state, conv_k;
  const void *x;
  int32_t x_dtype;
  const float *conv_w, *conv_b, *conv_cache_in;
  const void *dt;
  int32_t dt_dtype, dt_rank1;
  const float *dt_w, *dt_bias;
  int32_t dt_softplus;
  float dt_min, dt_max;
  const float *A;
  const void *B, *C;
  int32_t bc_dtype;
  const float *D;
  const void *z;
  int32_t z_dtype;
  const float *ssm_state_in;
  const void *dy;
  int32_t dy_dtype;
  const float *dstate_out;
  float *dx, *dz, *ddt, *ddt_w, *ddt_bias, *dA, *dB, *dC, *dD, *dconv_w, *dconv_b, *dconv_cache, *dstate_in;
  void *workspace;
  size_t workspace_bytes;
} ssm_scan_bwd_params_t;

ssm_status_t ssm_scan_bwd(const ssm_scan_bwd_params_t *p, void *stream);
size_t ssm_scan_bwd_workspace_size(const ssm_scan_bwd_params_t *p);
ssm_status_t ssm_scan_bwd_check(const ssm_scan_bwd_params_t *p);

/* ------------------------------------------------------------------------
 * One decode step of the multi-head scan, in place (page "What is the Mamba
 * model?", section "chunkscan": the state that the chunked scan passes from
 * chunk to chunk, advanced by a chunk of one token).  For each (b, h):
 *   dt = clip(softplus(dt_raw[b,h] + dt_bias[h]), dt_min, dt_max)   (softplus
 *        skipped when dt_softplus == 0)
 *   state[b,h,p,n] <- e^{dt A_h} state[b,h,p,n] + dt x[b,h,p] B[b,g,n]
 *   out[b,h,p] = (sum_n C[b,g,n] state[b,h,p,n] + D x[b,h,p]) * SiLU(z[b,h,p])
 * with g = h / (H / G) and the gate only when z != NULL.
 *   x         (Bt, H, P) x_dtype
 *   dt        (Bt, H) f32 raw;  dt_bias (H) f32 or NULL;  A (H) f32
 *   B, C      (Bt, G, N) bc_dtype
 *   D         (H) f32 (d_per_channel == 0) or (H, P) f32 or NULL
 *   z         (Bt, H, P) z_dtype or NULL
 *   state     (Bt, H, P, N) f32, read then overwritten (the layout of the
 *             chunked scan's state_in / state_out)
 *   out       (Bt, H, P) out_dtype; must not overlap any input
 * The result equals ssm_chunk_scan_fwd with L = 1 and state_in = state_out =
 * state.  state must be 16-byte aligned; B and C aligned to 8 elements (32
 * bytes in f32, 16 in bf16).  Supported: N in {16, 32, 64, 128};
 * batch * H * P < 2^31.  All dtypes f32 or bf16.
 * ---------------------------------------------------------------------- */
typedef struct ssm_chunk_decode_params {
  uint32_t struct_size; /* = sizeof(ssm_chunk_decode_params_t) */
  int32_t batch, nheads, headdim, ngroups, d_state;
  const void *x;
  int32_t x_dtype;
  const float *dt;
  const float *dt_bias;
  int32_t dt_softplus;
  float dt_min, dt_max;
  const float *A;
  const void *B;
  const void *C;
  int32_t bc_dtype;
  const float *D;
  int32_t d_per_channel;
  const void *z;
  int32_t z_dtype;
  float *state;
  void *out;
  int32_t out_dtype;
} ssm_chunk_decode_params_t;

ssm_status_t ssm_chunk_decode_step(const ssm_chunk_decode_params_t *p, void *stream);
ssm_status_t ssm_chunk_decode_check(const ssm_chunk_decode_params_t *p);

/* ------------------------------------------------------------------------
 * A projection of the layer (page "Axon-SSM: selective state space model",
 * section "Algorithm": in_proj D -> 2E and out_proj E -> D), no bias:
 *   out[r, o] = sum_i x[r, i] * weight[o, i]
 *   x       (rows, in_features) x_dtype: bf16 is used as it is; f32 enters the
 *           matrix cores as a bf16 pair (value and remainder), which keeps
 *           about 16 mantissa bits
 *   weight  (out_features, in_features) bf16 (the (out, in) layout of a weight)
 *   out     (rows, out_features) out_dtype; must not overlap x or weight
 *   workspace  device scratch of ssm_linear_workspace_size(p) bytes (256-byte
 *           aligned, owned by the caller, contents on entry irrelevant):
 *           none for a bf16 x; for an f32 x its bf16 value and remainder and
 *           an fp32 product.  Missing or short: SSM_ERR_WORKSPACE.
 * fp32 accumulation.  The products run in the ROCm GEMM library (hipBLASLt),
 * the same algorithm for a given shape and device, so results repeat bit for
 * bit.  x, weight and out must be 16-byte aligned; in_features % 8 == 0;
 * out_features % 4 == 0.
 * ---------------------------------------------------------------------- */
typedef struct ssm_linear_params {
  uint32_t struct_size; /* = sizeof(ssm_linear_params_t) */
  int32_t rows, in_features, out_features;
  const void *x;
  int32_t x_dtype;
  const void *weight;
  void *out;
  int32_t out_dtype;
  void *workspace;
  size_t workspace_bytes;
} ssm_linear_params_t;

ssm_status_t ssm_linear_fwd(const ssm_linear_params_t *p, void *stream);
size_t ssm_linear_workspace_size(const ssm_linear_params_t *p);
ssm_status_t ssm_linear_check(const ssm_linear_params_t *p);

/* ------------------------------------------------------------------------
 * The whole layer forward (page "Axon-SSM: selective state space model",
 * section "Algorithm"), T = batch * seqlen tokens:
 *   [x_branch | z] = in_proj(hidden)                   w_in (2E, D) bf16
 *   u = SiLU(causal depthwise conv1d(x_branch))        conv_w (E, K), conv_b (E) or NULL
 *   [B | C | dt_raw] = x_proj(u)                       w_x (2N+1, E) bf16, in that order
 *   dt = clip(softplus(dt_w * dt_raw + dt_bias), dt_min, dt_max)   dt_w, dt_bias (E)
 *   y = scan(u, dt, A, B, C) + D u, gated by SiLU(z)   A (E, N), D (E) or NULL
 *   out = out_proj(y)                                  w_out (D, E) bf16
 * hidden (Bt, L, D) hidden_dtype; out (Bt, L, D) out_dtype; conv caches
 * (Bt, E, K-1) f32 and states (Bt, E, N) f32 as in ssm_scan_fwd (each NULL-able;
 * in and out may be the same buffer).  The activations between the steps
 * (x_branch, z, y: fp32; B, C, dt_raw: fp32) live in the workspace, which
 * must hold ssm_layer_workspace_size(p) bytes (256-byte aligned).
 * Supported: N = 16, K = 4, E % 256 == 0, D % 8 == 0; hidden, the weights,
 * out, conv_w and A 16-byte aligned.
 * Timing events (ssm_set_timing_events) bracket the whole layer.
 * ---------------------------------------------------------------------- */
typedef struct ssm_layer_params {
  uint32_t struct_size; /* = sizeof(ssm_layer_params_t) */
  int32_t batch, seqlen, d_model, dim, d_state, conv_k;
  const void *hidden;
  int32_t hidden_dtype;
  const void *w_in;
  const float *conv_w, *conv_b;
  const void *w_x;
  const float *dt_w, *dt_bias;
  int32_t dt_softplus;
  float dt_min, dt_max;
  const float *A;
  const float *D;
  const void *w_out;
  const float *conv_cache_in;
  float *conv_cache_out;
  const float *ssm_state_in;
  float *ssm_state_out;
  void *out;
  int32_t out_dtype;
  void *workspace;
  size_t workspace_bytes;
} ssm_layer_params_t;

ssm_status_t ssm_layer_fwd(const ssm_layer_params_t *p, void *stream);
size_t ssm_layer_workspace_size(const ssm_layer_params_t *p);
ssm_status_t ssm_layer_check(const ssm_layer_params_t *p);

/* ------------------------------------------------------------------------
 * Gated delta rule: the multi-head linear recurrence whose input is the error
 * of the state's own prediction.  Per sequence and value head h, state S (V, K):
 *   S <- e^{g_t} S;  u_t = beta_t (v_t - S k_t);  S <- S + u_t k_t^T;  o_t = scale S q_t
 *   q, k      (Bt, L, Hk, K) x_dtype, v (Bt, L, H, V) x_dtype; head h reads key
 *             head h / (H / Hk).  *_stride: elements from one token to the next
 *             (the same across sequences), 0 for a dense tensor: rows of a
 *             wider projection are taken where they are
 *   g, beta   (Bt, L, H) f32: the log of the decay (<= 0 in a model; -inf forgets
 *             the state) and the write strength
 *   qk_norm   nonzero: q and k rows are first divided by sqrt(|row|^2 + eps)
 *   cu_seqlens (num_seqs + 1) int32 in DEVICE memory or NULL: packed sequences,
 *             Bt = 1, sequence i holds the tokens [cu[i], cu[i+1]); offsets rise
 *             from 0 to L (empty sequences allowed).  They are not read on the
 *             host; offsets out of range are clamped, tokens outside every
 *             sequence are not written.  NULL: num_seqs = Bt
 *   state_in  (num_seqs, H, V, K) f32 or NULL (zeros); state_out the same or NULL;
 *             may alias state_in exactly
 *   o         (Bt, L, H, V) o_dtype, dense
 * The sequence is taken in chunks of 64 tokens whose corrections u solve one
 * triangular system each, with matrix products throughout.  bf16 operands are
 * exact; 32-bit operands (f32 inputs, the state, u) enter the matrix cores as
 * three bf16 parts, so an f32 result carries f32 accuracy and a bf16 one is that
 * rounded once.  A NaN or infinity in k, v, g (g = -inf apart) or beta of a token may
 * reach the outputs of its whole chunk, earlier tokens included; other sequences are
 * never reached.
 * Workspace: ssm_delta_chunk_workspace_size() bytes, 256-byte aligned (39.7 kB per
 * chunk and head and 49.2 kB per chunk and key head at K = 128 in bf16).
 * Supported: K <= 128, any V, x_dtype f32 or bf16, L == 0 copies the state.
 * A launch's 2^32 threads bound num_seqs * H * ceil(V / 32) and the chunks times H
 * to below 2^24 (2^23 chunks times H in the backward with K > 64).
 * ---------------------------------------------------------------------- */
typedef struct ssm_delta_chunk_params {
  uint32_t struct_size; /* = sizeof(ssm_delta_chunk_params_t) */
  int32_t batch, seqlen, num_seqs, nkheads, nheads, d_key, d_value;
  const void *q, *k, *v;
  int32_t x_dtype;
  int64_t q_stride, k_stride, v_stride;
  const float *g, *beta;
  float scale;
  int32_t qk_norm;
  float eps;
  const int32_t *cu_seqlens;
  const float *state_in;
  float *state_out;
  void *o;
  int32_t o_dtype;
  void *workspace;
  size_t workspace_bytes;
} ssm_delta_chunk_params_t;

ssm_status_t ssm_delta_chunk_fwd(const ssm_delta_chunk_params_t *p, void *stream);
size_t ssm_delta_chunk_workspace_size(const ssm_delta_chunk_params_t *p);
ssm_status_t ssm_delta_chunk_check(const ssm_delta_chunk_params_t *p);

/* ------------------------------------------------------------------------
 * Backward of ssm_delta_chunk_fwd, recomputing the states of the chunks.  Given
 * dout = dL/do (Bt, L, H, V) x_dtype and optionally dstate_out (num_seqs, H, V, K)
 * f32, writes dq, dk (Bt, L, Hk, K) and dv (Bt, L, H, V) in grad_dtype, dense, and
 * dg, dbeta (Bt, L, H) and dstate_in (num_seqs, H, V, K) in f32; any may be NULL.
 * Key heads shared by several value heads receive the sum over them, in a fixed
 * order (no atomics: results repeat bit for bit).  The other fields are those of
 * the forward.  Workspace: ssm_delta_chunk_bwd_workspace_size() bytes (the
 * forward's, two (K, V) states and two (64, V) tiles in f32 per chunk and head, and
 * where value heads share key heads two (K) rows in f32 per token and value head).
 * ---------------------------------------------------------------------- */
typedef struct ssm_delta_chunk_bwd_params {
  uint32_t struct_size; /* = sizeof(ssm_delta_chunk_bwd_params_t) */
  int32_t batch, seqlen, num_seqs, nkheads, nheads, d_key, d_value;
  const void *q, *k, *v;
  int32_t x_dtype;
  int64_t q_stride, k_stride, v_stride;
  const float *g, *beta;
  float scale;
  int32_t qk_norm;
  float eps;
  const int32_t *cu_seqlens;
  const float *state_in;
  const void *dout;
  const float *dstate_out;
  void *dq, *dk, *dv;
  int32_t grad_dtype;
  float *dg, *dbeta, *dstate_in;
  void *workspace;
  size_t workspace_bytes;
} ssm_delta_chunk_bwd_params_t;

ssm_status_t ssm_delta_chunk_bwd(const ssm_delta_chunk_bwd_params_t *p, void *stream);
size_t ssm_delta_chunk_bwd_workspace_size(const ssm_delta_chunk_bwd_params_t *p);
ssm_status_t ssm_delta_chunk_bwd_check(const ssm_delta_chunk_bwd_params_t *p);

/* ------------------------------------------------------------------------
 * One token of the gated delta rule for each of Bt sequences, in place (the
 * result equals ssm_delta_chunk_fwd with L = 1 and state_in = state_out = state):
 *   q, k (Bt, Hk, K), v (Bt, H, V) x_dtype with *_stride elements from one
 *   sequence to the next (0: dense); g, beta (Bt, H) f32; state (Bt, H, V, K) f32,
 *   read then overwritten; o (Bt, H, V) o_dtype, dense.  All arithmetic is f32.
 * Supported: K <= 128; Bt * H * V < 2^27.
 * ---------------------------------------------------------------------- */
typedef struct ssm_delta_decode_params {
  uint32_t struct_size; /* = sizeof(ssm_delta_decode_params_t) */
  int32_t batch, nkheads, nheads, d_key, d_value;
  const void *q, *k, *v;
  int32_t x_dtype;
  int64_t q_stride, k_stride, v_stride;
  const float *g, *beta;
  float scale;
  int32_t qk_norm;
  float eps;
  float *state;
  void *o;
  int32_t o_dtype;
} ssm_delta_decode_params_t;

ssm_status_t ssm_delta_decode_step(const ssm_delta_decode_params_t *p, void *stream);
ssm_status_t ssm_delta_decode_check(const ssm_delta_decode_params_t *p);

/* ------------------------------------------------------------------------
 * The norms before and after a block, fused with its gate and residual scale.
 * On each of `rows` rows of `width` values, norm(r) = r / sqrt(mean(r^2) + eps):
 *   y = x              (y = x SiLU(z) with gate_first)
 *   a = norm(y) norm_w (in groups of group_size consecutive values each)
 *   a = a SiLU(z)      (without gate_first)
 *   t = residual + scale a,  residual_out = t
 *   out = norm(t) out_norm_w   (out = t without out_norm_w)
 * Every part may be left out (NULL): norm_w, z, residual, scale, out_norm_w.  The
 * mixer's gated norm is x, z and norm_w in groups of a head; the end of a block
 * with the next one's norm is all of it.
 *   x, z      (rows, width) x_dtype, *_stride elements between rows (0: dense)
 *   norm_w    f32, norm_w_len = group_size (shared by the groups) or width
 *   residual  (rows, width) res_dtype; residual_out the same, may alias residual
 *             exactly; NULL: not written
 *   scale, out_norm_w (width) f32;  out (rows, width) out_dtype or NULL
 * All arithmetic is f32; out is normalised from t before t is rounded to res_dtype.
 * Supported: group_size <= 16384, dividing width; group_size = width where
 * residual, scale or out_norm_w is given.
 * ---------------------------------------------------------------------- */
typedef struct ssm_block_norm_params {
  uint32_t struct_size; /* = sizeof(ssm_block_norm_params_t) */
  int64_t rows;
  int32_t width, group_size;
  const void *x;
  int32_t x_dtype;
  int64_t x_stride;
  const void *z;
  int64_t z_stride;
  int32_t gate_first;
  const float *norm_w;
  int32_t norm_w_len;
  const void *residual;
  int32_t res_dtype;
  const float *scale;
  void *residual_out;
  const float *out_norm_w;
  void *out;
  int32_t out_dtype;
  float eps;
} ssm_block_norm_params_t;

ssm_status_t ssm_block_norm_fwd(const ssm_block_norm_params_t *p, void *stream);
ssm_status_t ssm_block_norm_check(const ssm_block_norm_params_t *p);

/* ------------------------------------------------------------------------
 * Backward of ssm_block_norm_fwd from its inputs (nothing is saved by the
 * forward): dout = dL/dout and dresidual_out = dL/dresidual_out (either may be
 * NULL), in dout_dtype and dres_dtype.  Writes dx, dz (rows, width) in grad_dtype,
 * dresidual in res_dtype, and dnorm_w (norm_w_len), dscale, dout_norm_w (width) in
 * f32; any may be NULL.  Column sums are taken in a fixed order (results repeat
 * bit for bit).  The workspace holds ssm_block_norm_bwd_workspace_size(p) bytes
 * (256-byte aligned).  The other fields are those of the forward; a norm_w of the
 * whole width may hold at most 2^22 groups.
 * ---------------------------------------------------------------------- */
typedef struct ssm_block_norm_bwd_params {
  uint32_t struct_size; /* = sizeof(ssm_block_norm_bwd_params_t) */
  int64_t rows;
  int32_t width, group_size;
  const void *x;
  int32_t x_dtype;
  int64_t x_stride;
  const void *z;
  int64_t z_stride;
  int32_t gate_first;
  const float *norm_w;
  int32_t norm_w_len;
  const void *residual;
  int32_t res_dtype;
  const float *scale;
  const float *out_norm_w;
  float eps;
  const void *dout;
  int32_t dout_dtype;
  const void *dresidual_out;
  int32_t dres_dtype;
  void *dx, *dz;
  int32_t grad_dtype;
  void *dresidual;
  float *dnorm_w, *dscale, *dout_norm_w;
  void *workspace;
  size_t workspace_bytes;
} ssm_block_norm_bwd_params_t;

ssm_status_t ssm_block_norm_bwd(const ssm_block_norm_bwd_params_t *p, void *stream);
size_t ssm_block_norm_bwd_workspace_size(const ssm_block_norm_bwd_params_t *p);
ssm_status_t ssm_block_norm_bwd_check(const ssm_block_norm_bwd_params_t *p);

/* ------------------------------------------------------------------------
 * Causal attention with a sliding window and sinks, over whole sequences.  The query
 * at position p of its sequence sees the keys j <= p with j > p - window or j < sinks:
 *   s_pj = scale q_p.k_j,  lse_p = log sum_j e^{s_pj},  o_p = sum_j e^{s_pj - lse_p} v_j
 *   q         (Bt, L, H, D), k, v (Bt, Lk, Hk, D) x_dtype; head h reads key head
 *             h / (H / Hk).  *_stride: elements from one token to the next (the same
 *             across sequences), 0 for a dense tensor
 *   L, Lk     with more keys than queries the queries are the sequence's last positions
 *             (query i is at i + Lk - L); with fewer, the first see nothing
 *   window    keys that a query sees at most besides the sinks, itself among them; 0: all
 *   sinks     first keys of the sequence that stay visible behind the window
 *   scale     finite, not negative (less than 1e-30: the scores count as those of 1e-30)
 *   cu_seqlens (num_seqs + 1) int32 in DEVICE memory or NULL: packed sequences, Bt = 1,
 *             sequence i holds the queries [cu[i], cu[i+1]); offsets rise from 0 to L (empty
 *             sequences allowed).  They are not read on the host; offsets out of range are
 *             clamped, queries outside every sequence are not written.  NULL: num_seqs = Bt
 *   cu_seqlens_k  the same for the keys; NULL with cu_seqlens: the same offsets (L = Lk)
 *   lse       (Bt, L, H) f32 or NULL; -infinity where a query sees nothing (o is zero there)
 *   o         (Bt, L, H, D) o_dtype, dense
 *   o_rest    (Bt, L, H, D) bf16, dense, or NULL: what rounding took from an o in bf16
 *             (o + o_rest has 16 bits), for ssm_attn_bwd
 * Sums and the softmax's statistics are f32.  Scores are products of the inputs as they
 * are; their exponentials enter the product with v in f32 for f32 inputs, in three bf16
 * parts (24 bits) for bf16 inputs and an f32 o, in two (16 bits) for a bf16 o.
 * A NaN or infinity in a row of v that a query does not see may reach it where another
 * query of its tile of 128 (from the sequence's first query on) sees that row; rows that
 * none of these sees, and rows of other sequences, never do.  One in a row of k reaches
 * only the queries that see it.  An infinity in a row of v that a query sees gives it an
 * infinity or NaN.
 * Workspace: ssm_attn_workspace_size() bytes, 256-byte aligned.
 * Supported: D <= 128, x_dtype and o_dtype f32 or bf16, L and Lk up to 2^30; a launch's
 * 2^32 threads bound the tiles of 64 queries times H to below 2^24.
 * ---------------------------------------------------------------------- */
typedef struct ssm_attn_params {
  uint32_t struct_size; /* = sizeof(ssm_attn_params_t) */
  int32_t batch, seqlen, seqlen_k, num_seqs, nkheads, nheads, d_head;
  const void *q, *k, *v;
  int32_t x_dtype;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  int32_t window, sinks;
  const int32_t *cu_seqlens, *cu_seqlens_k;
  float *lse;
  void *o;
  int32_t o_dtype;
  void *o_rest;
  void *workspace;
  size_t workspace_bytes;
} ssm_attn_params_t;

ssm_status_t ssm_attn_fwd(const ssm_attn_params_t *p, void *stream);
size_t ssm_attn_workspace_size(const ssm_attn_params_t *p);
ssm_status_t ssm_attn_check(const ssm_attn_params_t *p);

/* ------------------------------------------------------------------------
 * Backward of ssm_attn_fwd from its inputs and its results o and lse: given dout = dL/do
 * (Bt, L, H, D) x_dtype, dense, writes dq (Bt, L, H, D), dk and dv (Bt, Lk, Hk, D) in
 * grad_dtype, dense; any may be NULL:
 *   P_pj = e^{s_pj - lse_p},  dS_pj = P_pj (dout_p.v_j - dout_p.o_p),
 *   dq_p = scale sum_j dS_pj k_j,  dk_j = scale sum_p dS_pj q_p,  dv_j = sum_p P_pj dout_p
 * Key heads shared by several heads receive the sum over them.  Sums are taken in a
 * fixed order, without atomics: results repeat bit for bit.  dout_p.o_p comes from o as
 * it is given: an o in bf16 moves dS_pj by P_pj |dout_p||o_p| 2^-8 at most, which is as
 * much as the gradients' rounding to bf16 or, where dS is small, several times that; with
 * its o_rest, or in f32, it does not.  P and dS enter their products as they do in the
 * forward (grad_dtype in the place of o_dtype).  A NaN or infinity in a row of k may
 * reach the dq of a query that does not see it where another query of its tile of 256 does,
 * and one in a row of q or dout the dk and dv of a key that this query does not see where
 * it sees another key of that key's tile of 64 (tiles from the sequence's first row on).
 * One in a row of v reaches only the dq of queries that see it and its own dk; rows of other
 * sequences never reach any.  Queries and keys outside every sequence are not written.
 * Workspace: ssm_attn_bwd_workspace_size() bytes, 256-byte aligned.
 * Supported: as in ssm_attn_fwd, and tiles of 64 keys (with the pieces of queries that the
 * sinks' tiles are cut into) times Hk and tiles of 64 queries times half of H, together
 * below 2^23.
 * ---------------------------------------------------------------------- */
typedef struct ssm_attn_bwd_params {
  uint32_t struct_size; /* = sizeof(ssm_attn_bwd_params_t) */
  int32_t batch, seqlen, seqlen_k, num_seqs, nkheads, nheads, d_head;
  const void *q, *k, *v;
  int32_t x_dtype;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  int32_t window, sinks;
  const int32_t *cu_seqlens, *cu_seqlens_k;
  const float *lse;
  const void *o;
  int32_t o_dtype;
  const void *o_rest;
  const void *dout;
  void *dq, *dk, *dv;
  int32_t grad_dtype;
  void *workspace;
  size_t workspace_bytes;
} ssm_attn_bwd_params_t;

ssm_status_t ssm_attn_bwd(const ssm_attn_bwd_params_t *p, void *stream);
size_t ssm_attn_bwd_workspace_size(const ssm_attn_bwd_params_t *p);
ssm_status_t ssm_attn_bwd_check(const ssm_attn_bwd_params_t *p);

/* ------------------------------------------------------------------------
 * The attention's cache lies in pages, in a pool (pages, Hk, page_size, D) for the keys
 * and one for the values, in f32, bf16 or SSM_E4M3; the token at position j of a sequence
 * is row j % page_size of page page_table[sequence][j / page_size].  A cache in SSM_E4M3
 * has a scale (pages, Hk) f32 beside each pool: a code c stands for c scale.
 *
 * ssm_attn_cache_write puts new tokens behind the lens[i] that sequence i holds:
 *   k, v      (Bt, L, Hk, D) x_dtype; *_stride elements from one token to the next (0:
 *             dense).  cu_seqlens as in ssm_attn_fwd, or NULL: L tokens of each of the
 *             num_seqs = Bt sequences
 *   lens      (num_seqs) int32 in DEVICE memory: tokens held before the call (not changed)
 *   page_table (num_seqs, table_rows) int32 in DEVICE memory.  Tokens whose page is not in
 *             [0, pages), or past the table, are not written: pages that no query sees any
 *             more may be given back and their entries set to -1
 *   cache_dtype  x_dtype, or SSM_E4M3
 * Scales are powers of two: for a page and head the least s with |x| <= 448 s for every
 * finite value put there (2^-100 at least); a page that holds tokens already keeps its
 * scale or takes a larger one, and its codes are put to that (exactly, but for codes that
 * become subnormal, which are rounded again).  Values are rounded to nearest even;
 * infinities and NaN become NaN.  Rows that no token is put to keep their contents.
 * A page whose first token here is not its row 0 is taken to hold the rows before, with its
 * scales: one that is new to the sequence there (its entry was out of range before) wants
 * scales of 0.
 * Pages that the call writes to belong to one sequence.
 * Supported: D <= 128; page_size up to 65536, table_rows * page_size up to 2^30; the pages
 * met (at most tokens / page_size + 2 num_seqs) times Hk below 2^24.
 * ---------------------------------------------------------------------- */
typedef struct ssm_attn_cache_params {
  uint32_t struct_size; /* = sizeof(ssm_attn_cache_params_t) */
  int32_t batch, seqlen, num_seqs, nkheads, d_head;
  const void *k, *v;
  int32_t x_dtype;
  int64_t k_stride, v_stride;
  const int32_t *cu_seqlens, *lens, *page_table;
  int32_t table_rows, pages, page_size;
  void *k_cache, *v_cache;
  int32_t cache_dtype;
  float *k_scale, *v_scale;
} ssm_attn_cache_params_t;

ssm_status_t ssm_attn_cache_write(const ssm_attn_cache_params_t *p, void *stream);
ssm_status_t ssm_attn_cache_check(const ssm_attn_cache_params_t *p);

/* ------------------------------------------------------------------------
 * One query of each of Bt sequences over its pages (the cache as above):
 *   q (Bt, H, D) x_dtype with q_stride elements from one sequence to the next (0: dense);
 *   lens (Bt) int32: tokens that the sequence holds, the query's own among them (the query
 *   is at position lens - 1; 0: o is zero); o (Bt, H, D) o_dtype, dense.
 * window, sinks and scale as in ssm_attn_fwd.  Entries of page_table that no visible key
 * needs are not read; keys whose page is not in [0, pages) are left out.  A lens past the
 * table counts as table_rows * page_size.  The result equals the last row of ssm_attn_fwd
 * over the values that the cache stands for.
 * cache_dtype: x_dtype, or SSM_E4M3, or bf16 beside an f32 x_dtype.
 * A key with infinite channels whose score is -infinity vanishes, but not from a bf16 cache
 * beside an f32 q, whose parts may be zero: there it may give NaN.  An infinity in a visible
 * row of v gives an infinity or NaN.
 * Workspace: ssm_attn_decode_workspace_size() bytes, 256-byte aligned.
 * Supported: D <= 128; Bt * H below 2^24; page_size up to 65536, table_rows * page_size up
 * to 2^30.
 * ---------------------------------------------------------------------- */
typedef struct ssm_attn_decode_params {
  uint32_t struct_size; /* = sizeof(ssm_attn_decode_params_t) */
  int32_t batch, nkheads, nheads, d_head;
  const void *q;
  int32_t x_dtype;
  int64_t q_stride;
  const void *k_cache, *v_cache;
  int32_t cache_dtype;
  const float *k_scale, *v_scale;
  const int32_t *page_table, *lens;
  int32_t table_rows, pages, page_size;
  float scale;
  int32_t window, sinks;
  void *o;
  int32_t o_dtype;
  void *workspace;
  size_t workspace_bytes;
} ssm_attn_decode_params_t;

ssm_status_t ssm_attn_decode_step(const ssm_attn_decode_params_t *p, void *stream);
size_t ssm_attn_decode_workspace_size(const ssm_attn_decode_params_t *p);
ssm_status_t ssm_attn_decode_check(const ssm_attn_decode_params_t *p);

/* ------------------------------------------------------------------------ */
const char *ssm_status_string(int32_t status);
/* Detail of the last non-OK return on the calling thread ("" if none). */
const char *ssm_last_error(void);
int32_t ssm_abi_version(void);
/* sizeof of a params struct: which = 0 scan, 1 decode, 2 chunk, 3 chunk
 * decode, 4 linear, 5 layer, 6 scan backward, 8 delta chunk, 9 delta chunk
 * backward, 10 delta decode, 11 block norm, 12 block norm backward, 13 attention,
 * 14 attention backward, 15 attention cache, 16 attention decode; 0 otherwise. */
size_t ssm_params_sizeof(int32_t which);

/* Kernel timing for measurement tools.  start and stop are hipEvent_t handles
 * owned by the caller (both NULL switches timing off).  While set, each entry
 * point called on this thread records start on its stream right before the
 * launch of its main kernel and stop right after it, so
 * hipEventElapsedTime(start, stop) is that kernel's duration.  Main kernels: the
 * full-segment scan kernel of ssm_scan_fwd; the walk over the chunks of
 * ssm_delta_chunk_fwd, without the kernel that forms its operands; the gradients'
 * kernel of ssm_delta_chunk_bwd, without operands, walks and the sums of shared
 * heads; the row kernel of ssm_block_norm_bwd, without the column sums; the
 * gradients' kernel of ssm_attn_bwd, without dout.o and the sums of the sinks'
 * pieces; the kernel over the cache of ssm_attn_decode_step, without the join of
 * its parts; all of ssm_layer_fwd; the main or only kernel of the others.  The events are only
 * recorded, never created, synchronised or destroyed by the library. */
void ssm_set_timing_events(void *start, void *stop);

/* ---- debug builds (SSM_DEBUG) ---------------------------------------------
 * For callers that want the host-side bounds checks: a build of the library
 * with SSM_DEBUG defined (libssm_mi355x_debug.so, the same kernels) checks,
 * before every launch of ssm_scan_fwd(_noalloc), ssm_chunk_scan_fwd and
 * ssm_scan_bwd, the launch plan against the buffers the call describes: each
 * grid's mapping from block ids to work items is a bijection onto the work,
 * the time segments, chunk segments and summary pieces tile the sequence as
 * the kernels assume, and every workspace region a kernel indexes is
 * 256-byte aligned, lies inside workspace_bytes and overlaps no other.  A
 * failure returns SSM_ERR_INTERNAL (ssm_last_error() names the check) and
 * launches nothing.
 * ssm_debug_checks: launch plans checked so far in this process (-1: a build
 *   without the checks).
 * ssm_debug_check_{scan,chunk,scan_bwd}: validation plus the plan checks of
 *   that entry point without launching anything (runs without a GPU; pointers
 *   are compared, never dereferenced); SSM_ERR_UNSUPPORTED in builds without
 *   the checks. */
long ssm_debug_checks(void);
ssm_status_t ssm_debug_check_scan(const ssm_scan_params_t *p);
ssm_status_t ssm_debug_check_chunk(const ssm_chunk_params_t *p);
ssm_status_t ssm_debug_check_scan_bwd(const ssm_scan_bwd_params_t *p);

#ifdef __cplusplus
}
#endif

#endif /* SSM_MI355X_H */
