/*
 * kda.h -- C ABI of the MI355X (gfx950) Kimi Delta Attention (KDA) core.
 *
 * What the library computes.  For every sequence and head, with raw per-token
 * projections q, k (dk channels per head), v (dv channels per head), a
 * per-channel decay input alpha and a per-head write-strength input b:
 *
 *   1. each q, k, v channel passes a depthwise causal conv1d of kernel 4,
 *      padding 3, no bias, then SiLU;  q and k are L2-normalised per head
 *      (AliceAI-Foundation-80B-A3B page, section 二);
 *   2. g = max(-exp(A_log[h]) * softplus(alpha + dt_bias[h]), lower_bound)
 *      (same page, section 二, gate formula; the -5.0 lower bound is the safe
 *      gate of the Ling-3.0-flash-VL page, section "KDA 层的安全门");
 *      beta = sigmoid(b) (AliceAI page, section 二: beta is not doubled);
 *   3. per token, with the dk x dv state S (rows = key channels):
 *        S <- Diag(exp(g)) S;  delta = beta (v - k^T S);  S <- S + k delta^T;
 *        o = q^T S   (the read uses the updated state)
 *      (AliceAI page, section 二, the delta-rule loop; state shape
 *      (batch, v_heads, k_dim, v_dim)).
 *
 * Prefill and decode share the state interface: a prefill's final state and
 * conv history are a decode step's input (AliceAI page, section 五).  The
 * conv history of a sequence is its last 3 raw (pre-conv) inputs per channel
 * (AliceAI page, section 四: kernel-1 = 3 history elements), stored oldest
 * first with channels ordered q | k | v:  Ctot = H * (2*dk + dv).
 *
 * Entry points: kda_prefill (B equal-length sequences) and kda_varlen_prefill
 * (packed sequences), each in the chunked form or, for gates below -5.4, the
 * token recurrence; kda_decode_step (one token per sequence, in place);
 * kda_decode_multi (K tokens per sequence through state / conv-history pools,
 * with commit counts for speculative decoding); kda_decode_step_gated and
 * kda_decode_multi_gated (the same with the output epilogue fused);
 * kda_output_gate (the layer's o_norm x sigmoid output epilogue).  Around the
 * core: kda_add_rmsnorm (the residual's addition and the norm in front of the
 * layer), kda_fp8_matmul (its projections, e4m3 operands with block scales),
 * kda_add_rmsnorm_fp8 and kda_output_gate_fp8 (the producers of such operands),
 * kda_add_rmsnorm_backward and kda_output_gate_backward.  For the decoder's
 * full-attention layers, which stand between the KDA layers: kda_qk_norm_rope
 * and its backward (norm and rotation of the query and key heads),
 * kda_append_kv and kda_read_kv (a paged cache of 4-bit keys and values) and
 * kda_paged_attention.  Plus the workspace queries, the version and status
 * strings.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers, contiguous, row-major in the
 *    layout given, 16-byte aligned.  The caller owns every buffer; the library
 *    allocates no device memory and keeps no mutable global state, so calls on
 *    different streams are independent.  The one exception is
 *    kda_varlen_prefill_noalloc, whose fixed per-GPU scratch array is shared
 *    by all its calls on that GPU (see there).
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream)
 *    and is asynchronous: the library never synchronises and never reads
 *    device data on the host.
 *  - Host-side validation runs before any launch.  On failure the call
 *    returns a nonzero kda_status_t, launches nothing and leaves every output
 *    untouched.  A launch failure returns KDA_ERR_HIP.  Faults inside kernels
 *    surface at the caller's next synchronisation.
 *  - NaN/Inf inputs propagate; they are not trapped.
 *  - B == 0 or N == 0 is a valid no-op returning KDA_OK.  A sequence of
 *    length 0 passes its initial state and conv history through unchanged.
 *  - Supported geometry: dk == dv, dk in {16, 32, 64, 128}; chunk_size 64.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1,    /* null required pointer, negative size, bad cu_seqlens length */
    KDA_ERR_UNSUPPORTED = 2,         /* geometry / dtype / flag combination not built */
    KDA_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes below the size query's answer */
    KDA_ERR_HIP = 4                  /* a HIP launch reported an error */
} kda_status_t;

typedef enum kda_dtype {
    KDA_BF16 = 0,
    KDA_FP32 = 1
} kda_dtype_t;

/* Test hooks; 0 for the method as described. */
#define KDA_FLAG_SKIP_CONV   (1u << 0) /* q, k, v are already conv + SiLU outputs           */
#define KDA_FLAG_SKIP_L2NORM (1u << 1) /* q, k are used without L2 normalisation           */
#define KDA_FLAG_RAW_GATE    (1u << 2) /* alpha holds g itself (no softplus, no clamp)      */
#define KDA_FLAG_RAW_BETA    (1u << 3) /* b holds beta itself (no sigmoid)                  */
#define KDA_FLAG_BETA_X2     (1u << 4) /* beta = 2 sigmoid(b): negative eigenvalues allowed */

/* Stages of a call, for the optional per-stage timing hook below. */
typedef enum kda_stage {
    KDA_STAGE_CHUNK_TABLE = 0,  /* packed-batch chunk table (device cu_seqlens scan)          */
    KDA_STAGE_CHUNK_PREP = 1,   /* preprocess + intra-chunk solve, parallel over chunks
                                   (recurrent form: the per-token preprocess)                 */
    KDA_STAGE_CHUNK_SCAN = 2,   /* inter-chunk state propagation + chunk output, sequential
                                   (recurrent form: the token-by-token state scan)            */
    KDA_STAGE_CONV_STATE = 3,   /* conv history out                                           */
    KDA_STAGE_DECODE = 4,       /* the decode step kernel (also kda_decode_multi)             */
    KDA_STAGE_OUTPUT_GATE = 5,  /* the o_norm + sigmoid output-gate epilogue                  */
    KDA_STAGE_BACKWARD = 6,     /* the backward pass's kernels (after its chunk table)        */
    KDA_STAGE_NORM = 7,         /* the residual's addition and the RMS norm                   */
    KDA_STAGE_MATMUL = 8,       /* the block-scaled e4m3 product                              */
    KDA_STAGE_ROPE = 9,         /* norm and rotation of query and key heads                   */
    KDA_STAGE_CACHE = 10,       /* kda_append_kv, kda_read_kv                                 */
    KDA_STAGE_ATTENTION = 11,   /* kda_paged_attention                                        */
    KDA_NUM_STAGES = 12
} kda_stage_t;

typedef struct kda_config {
    int32_t num_heads;        /* H                                                      */
    int32_t head_k_dim;       /* dk                                                     */
    int32_t head_v_dim;       /* dv (must equal dk)                                     */
    int32_t io_dtype;         /* kda_dtype_t of q, k, v, alpha, b, conv weights, conv history */
    int32_t out_dtype;        /* kda_dtype_t of o                                       */
    float scale;              /* multiplies the normalised q; 1.0 as on the pages       */
    float gate_lower_bound;   /* -5.0 (safe gate); any value, -INFINITY disabling the
                                 clamp.  It also picks the prefill's form: >= -5.4 the
                                 chunked form; below, the token-by-token recurrence
                                 (exact for any gate, ~2.3x slower; its workspace holds
                                 (4*dk + 4) fp32 per head and token).  With
                                 KDA_FLAG_RAW_GATE the bound is not applied to g but
                                 still picks the form: the chunked one needs every
                                 g >= -5.4                                            */
    float l2norm_eps;         /* q / sqrt(|q|^2 + eps); 1e-6                            */
    int32_t chunk_size;       /* 64                                                     */
    uint32_t flags;           /* KDA_FLAG_* test hooks, normally 0                      */
    const float *A_log;       /* [H] fp32, device                                       */
    const float *dt_bias;     /* [H*dk] fp32, device                                    */
    const void *conv_w_q;     /* [H*dk][4] io_dtype, device; tap 3 multiplies the current token */
    const void *conv_w_k;     /* [H*dk][4]                                              */
    const void *conv_w_v;     /* [H*dv][4]                                              */
    /* Optional timing hook, NULL for none: an array of 2*KDA_NUM_STAGES
     * hipEvent_t handles owned by the caller.  Entries 2*s and 2*s+1 (when
     * non-NULL) are recorded on the call's stream right before and right
     * after the launches of stage s. */
    void **stage_events;
} kda_config_t;

/* Library version, major*10000 + minor*100 + patch.  The operators around the
 * core (kda_add_rmsnorm and those after it) came without a new one: a caller
 * that opens the library at run time looks for their symbols.  The arrays of
 * stage_events that callers of the core made for 7 stages stay valid for its
 * calls, which record no others; those made for 9 for the calls up to
 * kda_fp8_matmul. */
int32_t kda_version(void);

/* Human-readable name of a status code (static storage). */
const char *kda_status_string(kda_status_t status);

/*
 * Workspace size in bytes for kda_prefill over B sequences of T tokens.
 * Returns 0 for an invalid or unsupported configuration.
 */
size_t kda_prefill_workspace_bytes(const kda_config_t *cfg, int32_t B, int32_t T);

/*
 * Chunked prefill of B equal-length sequences of T tokens.
 *   q, k           [B][T][H*dk]  io_dtype, raw projections (pre-conv)
 *   v              [B][T][H*dv]  io_dtype
 *   alpha          [B][T][H][dk] io_dtype, decay input
 *   b              [B][T][H]     io_dtype, pre-sigmoid write strength
 *   initial_state  [B][H][dk][dv] fp32, or NULL for zeros
 *   conv_state_in  [B][3][Ctot] io_dtype, oldest first, or NULL for zeros
 *   o              [B][T][H][dv] out_dtype (required)
 *   final_state    [B][H][dk][dv] fp32, or NULL; may alias initial_state
 *   conv_state_out [B][3][Ctot] io_dtype, or NULL; may alias conv_state_in
 *   workspace      device scratch of kda_prefill_workspace_bytes() for one pass
 *                  over the whole batch.  A smaller workspace runs the chunked
 *                  form (gate lower bound >= -5.4) in slabs: windows of the
 *                  longest multiple of 64 positions of every sequence whose
 *                  kda_prefill_slab_workspace_bytes() fits, one after the
 *                  other, with the state carried between them.  The results
 *                  are bit-identical to one pass.  KDA_ERR_WORKSPACE_TOO_SMALL
 *                  when not even a 64-token slab fits, or for the recurrent
 *                  form (bound below -5.4).  The per-stage timing events
 *                  (stage_events) are not recorded in slabs.
 * No other aliasing is allowed.
 */
kda_status_t kda_prefill(const kda_config_t *cfg, int32_t B, int32_t T,
                         const void *q, const void *k, const void *v,
                         const void *alpha, const void *b,
                         const float *initial_state, const void *conv_state_in,
                         void *o, float *final_state, void *conv_state_out,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * Workspace size in bytes for kda_varlen_prefill over N packed sequences
 * holding total_T tokens.  Returns 0 for an invalid configuration.
 */
size_t kda_varlen_workspace_bytes(const kda_config_t *cfg, int32_t N, int32_t total_T);

/*
 * Workspace size in bytes for the chunked prefill (kda_prefill with B = N, or
 * kda_varlen_prefill) run in slabs of slab_tokens positions per sequence
 * (rounded up to a multiple of 64): the chunk table and records of one slab
 * plus a carried state of [N][H][dk][dv] fp32.  It depends on neither T nor
 * total_T, which bounds the workspace of long prefills (4 x 32768 tokens at
 * H = 32, d = 128: 9.0 GiB in one pass, 2.3 GiB in slabs of 8192).  Returns 0
 * for an invalid configuration, N < 1, slab_tokens < 1 or a gate lower bound
 * below -5.4 (the recurrent form, which has no slabs).
 */
size_t kda_prefill_slab_workspace_bytes(const kda_config_t *cfg, int32_t N, int32_t slab_tokens);

/*
 * Chunked prefill of N sequences packed back to back (varlen).
 *   cu_seqlens     [N+1] int32, DEVICE; cu[0] = 0, cu[N] = total_T,
 *                  nondecreasing (zero-length sequences allowed).  The
 *                  library does not read it on the host; a malformed array
 *                  is undefined behaviour.
 *   q, k           [total_T][H*dk];  v [total_T][H*dv]
 *   alpha          [total_T][H][dk]; b [total_T][H]
 *   initial_state  [N][H][dk][dv] fp32 or NULL;  conv_state_in [N][3][Ctot] or NULL
 *   o              [total_T][H][dv]
 *   final_state    [N][H][dk][dv] or NULL;  conv_state_out [N][3][Ctot] or NULL
 * State and conv history restart at each sequence; chunks never straddle two
 * sequences.  Aliasing rules, and slabs for a smaller workspace, as for
 * kda_prefill (a slab is a window of positions of every sequence; the host
 * does not know the longest sequence, so it runs ceil(total_T / slab) of
 * them, the later ones empty for short sequences).
 */
kda_status_t kda_varlen_prefill(const kda_config_t *cfg, int32_t N, int32_t total_T,
                                const int32_t *cu_seqlens,
                                const void *q, const void *k, const void *v,
                                const void *alpha, const void *b,
                                const float *initial_state, const void *conv_state_in,
                                void *o, float *final_state, void *conv_state_out,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_varlen_prefill without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, serving loops and
 * harnesses that forbid hipMalloc.  The workspace is a fixed array of
 * KDA_NOALLOC_SCRATCH_BYTES in the library's device memory, one per GPU,
 * held from the first call on that GPU until the process ends; the call
 * allocates nothing.  Arguments, layouts and results as for
 * kda_varlen_prefill.
 *   - A batch whose workspace (kda_varlen_workspace_bytes) exceeds
 *     KDA_NOALLOC_SCRATCH_BYTES runs in slabs (as kda_varlen_prefill does
 *     with a small workspace); it is refused with KDA_ERR_WORKSPACE_TOO_SMALL,
 *     before any device call, when not even one slab of 64 tokens fits
 *     (kda_prefill_slab_workspace_bytes(cfg, N, 64) above the scratch: at
 *     H = 32, dk = dv = 128, bf16, 6.5 MB per sequence, a chunk's records for
 *     every head and the carried state, so N up to 39) or for the recurrent
 *     form.  One pass fits up to ~1800 (64-token chunk,
 *     head) pairs, e.g. 3 x 1024 tokens x 32 heads.
 *   - Every call on one GPU uses that GPU's single array: calls that overlap
 *     in time on one GPU (different streams, different threads) race and
 *     must be serialised by the caller.  Nothing from a previous call needs
 *     clearing: each call writes the scratch bytes it reads.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (256u << 20)

kda_status_t kda_varlen_prefill_noalloc(const kda_config_t *cfg, int32_t N, int32_t total_T,
                                        const int32_t *cu_seqlens,
                                        const void *q, const void *k, const void *v,
                                        const void *alpha, const void *b,
                                        const float *initial_state, const void *conv_state_in,
                                        void *o, float *final_state, void *conv_state_out,
                                        void *stream);

/*
 * Backward pass of kda_varlen_prefill: the gradient of a loss through o and
 * the final state with respect to every input and parameter (the models on
 * the Ling pages are trained natively with KDA layers; the pages give only
 * the forward, AliceAI page, section 二, whose reverse-mode derivative this
 * computes).  The forward is recomputed inside; nothing from a forward call
 * is needed.  Inputs are those of kda_varlen_prefill (same layouts, dtypes
 * and cu_seqlens rules) plus
 *   d_o            [total_T][H][dv] out_dtype: dLoss/do
 *   d_final_state  [N][H][dk][dv] fp32: dLoss/dfinal_state, or NULL (zero)
 * Outputs, all fp32 (every element written):
 *   dq, dk         [total_T][H*dk]   gradients of the raw (pre-conv) q, k
 *   dv             [total_T][H*dv]
 *   dalpha         [total_T][H][dk]  (0 where the safe gate clamped g)
 *   db             [total_T][H]
 *   d_initial_state [N][H][dk][dv], or NULL if not wanted
 *   d_conv_state_in [N][3][Ctot] gradient of the incoming conv history
 *                  (zeros when it was NULL), or NULL if not wanted
 *   dw_q, dw_k     [H*dk][4], dw_v [H*dv][4], ddt_bias [H*dk], dA_log [H]:
 *                  summed over all sequences of the batch
 * Supported: the chunked form's gates (gate_lower_bound >= -5.4) and
 * flags 0 or KDA_FLAG_BETA_X2; anything else is KDA_ERR_UNSUPPORTED.  The
 * workspace (kda_varlen_backward_workspace_bytes) holds per 16-token block
 * and head about 2 dk dv + 6 * 16 dk floats (~170 KB at dk = dv = 128).
 * Timing stages: KDA_STAGE_CHUNK_TABLE, then KDA_STAGE_BACKWARD.
 */
size_t kda_varlen_backward_workspace_bytes(const kda_config_t *cfg, int32_t N, int32_t total_T);

kda_status_t kda_varlen_backward(const kda_config_t *cfg, int32_t N, int32_t total_T,
                                 const int32_t *cu_seqlens,
                                 const void *q, const void *k, const void *v,
                                 const void *alpha, const void *b,
                                 const float *initial_state, const void *conv_state_in,
                                 const void *d_o, const float *d_final_state,
                                 float *dq, float *dk, float *dv, float *dalpha, float *db,
                                 float *d_initial_state, float *d_conv_state_in,
                                 float *dw_q, float *dw_k, float *dw_v, float *ddt_bias, float *dA_log,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * One decode step: one new token for each of N independent sequences
 * (the fused recurrent form; AliceAI page, section 五).
 *   q, k           [N][H*dk] io_dtype;  v [N][H*dv]
 *   alpha          [N][H][dk];          b [N][H]
 *   state          [N][H][dk][dv] fp32, read and updated in place (required)
 *   conv_state     [N][3][Ctot] io_dtype, read and shifted in place (required)
 *   o              [N][H][dv] out_dtype
 * Needs no workspace.
 */
kda_status_t kda_decode_step(const kda_config_t *cfg, int32_t N,
                             const void *q, const void *k, const void *v,
                             const void *alpha, const void *b,
                             float *state, void *conv_state, void *o, void *stream);

/*
 * Serving decode: K tokens for each of N sequences whose state and conv
 * history live in caller-owned pools (AliceAI page, section 五: the
 * recurrent state and the conv states are what decode carries; section 六:
 * speculative decoding with MTP drafts one extra token per forward, whose
 * outputs a verify pass needs before the accepted tokens are kept).
 *   slots          [N] int32, device: the pool row of each sequence; a
 *                  negative slot skips the sequence (its outputs are not
 *                  written).  NULL: sequence n uses row n.  Slots of one call
 *                  must be distinct.
 *   q, k           [N][K][H*dk]  io_dtype     v [N][K][H*dv]
 *   alpha          [N][K][H][dk] io_dtype     b [N][K][H]
 *   state_pool     [P][H][dk][dv] fp32, device (P > every slot)
 *   conv_pool      [P][3][Ctot] io_dtype, raw-input history, oldest first
 *   o              [N][K][H][dv] out_dtype: the outputs of all K tokens,
 *                  each reading the state updated by the tokens before it
 *   n_commit       [N] int32, device: keep the updates of the first
 *                  n_commit[n] tokens (clamped to 0..K): the pools receive
 *                  the state and conv history after them.  0 leaves the
 *                  pools untouched (a verify pass); NULL keeps all K.
 * The state is read once and written at most once per call, so K tokens cost
 * about the HBM traffic of one decode step.  A rejected draft is rolled back
 * by committing fewer tokens, e.g. a verify call with n_commit = 0 and then a
 * call over the accepted tokens only.  K in 1..64.  Needs no workspace.
 */
kda_status_t kda_decode_multi(const kda_config_t *cfg, int32_t N, int32_t K, const int32_t *slots,
                              const void *q, const void *k, const void *v,
                              const void *alpha, const void *b,
                              float *state_pool, void *conv_pool, void *o,
                              const int32_t *n_commit, void *stream);

/*
 * kda_decode_step and kda_decode_multi with the layer's output epilogue
 * (kda_output_gate below) fused into the step: each (sequence, head)
 * workgroup holds the whole row of dv outputs, so the row is normalised and
 * gated before it is stored and o never goes to memory
 * (AliceAI page, section 三: KDA's output goes through o_norm and a sigmoid
 * gate).  Arguments as for the plain calls, plus:
 *   gate           the output-gate projection before the sigmoid, io_dtype,
 *                  laid out like o: [N][H][dv] (step), [N][K][H][dv] (multi)
 *   o_norm_weight  [dv] fp32, one weight per channel shared by the heads
 *   eps            o_norm epsilon, >= 0 (NaN or negative, or a NULL gate or
 *                  weight: KDA_ERR_INVALID_ARGUMENT)
 *   y              out_dtype, in place of o: y = o / sqrt(mean(o^2) + eps)
 *                  * o_norm_weight * sigmoid(gate), per (token, head) row
 * The state and conv history are updated exactly as by the plain calls.
 */
kda_status_t kda_decode_step_gated(const kda_config_t *cfg, int32_t N,
                                   const void *q, const void *k, const void *v,
                                   const void *alpha, const void *b,
                                   float *state, void *conv_state,
                                   const void *gate, const float *o_norm_weight, float eps,
                                   void *y, void *stream);

kda_status_t kda_decode_multi_gated(const kda_config_t *cfg, int32_t N, int32_t K, const int32_t *slots,
                                    const void *q, const void *k, const void *v,
                                    const void *alpha, const void *b,
                                    float *state_pool, void *conv_pool,
                                    const void *gate, const float *o_norm_weight, float eps,
                                    void *y, const int32_t *n_commit, void *stream);

/*
 * The layer's output epilogue on n_tokens x H rows of dv outputs (AliceAI
 * page, section 三: KDA's output goes through o_norm and a sigmoid gate;
 * section 二: output_gate is one of the per-token control inputs):
 *   y[t][h][j] = o[t][h][j] / sqrt(mean_j' o[t][h][j']^2 + eps)
 *                * o_norm_weight[j] * sigmoid(gate[t][h][j])
 * The pages give neither the norm's epsilon nor its weight's shape: o_norm
 * is read as an RMS norm over one head's dv outputs with one weight per
 * channel shared by the heads (eps 1e-6 in the reference setting).
 *   o              [n_tokens][H][dv] out_dtype, as written by the calls above
 *   gate           [n_tokens][H][dv] io_dtype, the output-gate projection
 *                  before the sigmoid
 *   o_norm_weight  [dv] fp32
 *   eps            >= 0 (NaN or negative: KDA_ERR_INVALID_ARGUMENT)
 *   y              [n_tokens][H][dv] out_dtype; may alias o (in place)
 * Only num_heads, head_v_dim, io_dtype, out_dtype and stage_events of cfg
 * are used.  Needs no workspace.  n_tokens == 0 is a no-op.
 */
kda_status_t kda_output_gate(const kda_config_t *cfg, int64_t n_tokens,
                             const void *o, const void *gate,
                             const float *o_norm_weight, float eps,
                             void *y, void *stream);

/*
 * ---- The operators around the core ---------------------------------------
 *
 * A KDA layer adds its input to the residual stream, normalises it, projects
 * it to q, k, v, alpha, b and the output gate, runs the core and the output
 * epilogue, and projects back.  The entry points below are those steps, in
 * bf16 / fp32 or with 8-bit matrix operands:
 *
 *   e4m3 rows: K values of 1 byte (OCP e4m3: 3 mantissa bits, at most 448, no
 *   infinity) with one fp32 scale for every 128 consecutive values, the last
 *   block of a row being short when 128 does not divide K:  KB = ceil(K / 128),
 *   value k of a row stands for q[k] * scale[k / 128].  A row is written from
 *   fp32 values v as  scale = max(max|v| over the block, 1e-30) / 448,
 *   q = v / scale rounded to nearest even.  A NaN or an infinity in a block
 *   makes its scale NaN or infinite.
 *
 * Pointers are 16-byte aligned as everywhere (e4m3 outputs 8-byte, scales
 * 4-byte); one that is not is KDA_ERR_INVALID_ARGUMENT here.
 */

/*
 * The norm in front of a layer, with the residual's addition:
 *   h[t] = x[t] + residual[t], rounded to io_dtype
 *   y[t][j] = h[t][j] / sqrt(mean_j' h[t][j']^2 + eps) * weight[j]
 *   x, residual    [n_tokens][hidden] io_dtype; residual NULL: h = x
 *   weight         [hidden] fp32
 *   eps            >= 0 (NaN or negative: KDA_ERR_INVALID_ARGUMENT); with 0 a
 *                  row of zeros gives NaN
 *                  (the squares are summed in fp32: where the sum passes
 *                  3.4e38 the row's y is 0, squares below 1e-45 count as 0)
 *   h              [n_tokens][hidden] io_dtype, or NULL if not wanted; may
 *                  alias x or residual (in place)
 *   y              [n_tokens][hidden] out_dtype; with h NULL it may alias x
 *                  when both have the same type
 *   hidden         a multiple of 8, 8 .. 32768 (else KDA_ERR_UNSUPPORTED)
 * No other aliasing.  Only io_dtype, out_dtype and stage_events of cfg are
 * used.  Needs no workspace.  n_tokens == 0 is a no-op.
 */
kda_status_t kda_add_rmsnorm(const kda_config_t *cfg, int64_t n_tokens, int32_t hidden,
                             const void *x, const void *residual, const float *weight, float eps,
                             void *h, void *y, void *stream);

/*
 * The same with y as e4m3 rows: y [n_tokens][hidden] e4m3, y_scale
 * [n_tokens][ceil(hidden / 128)] fp32.  y aliases nothing; out_dtype of cfg
 * is not used, but has to be a known type.
 */
kda_status_t kda_add_rmsnorm_fp8(const kda_config_t *cfg, int64_t n_tokens, int32_t hidden,
                                 const void *x, const void *residual, const float *weight, float eps,
                                 void *h, void *y, float *y_scale, void *stream);

/*
 * Gradient of kda_add_rmsnorm (of kda_add_rmsnorm_fp8 with the rounding taken
 * as the identity).  With n = h / sqrt(mean h^2 + eps) and g = dy * weight:
 *   dx = (g - n * mean(g * n)) / sqrt(mean h^2 + eps) + d_h
 *   dweight[j] = sum over tokens of dy * n
 *   h              [n_tokens][hidden] io_dtype, as the forward wrote it
 *   dy             [n_tokens][hidden] out_dtype: dLoss/dy
 *   d_h            [n_tokens][hidden] fp32: the gradient that reaches h by the
 *                  residual stream, or NULL (zero)
 *   dx             [n_tokens][hidden] fp32: the gradient of x, and of residual
 *                  alike; may alias d_h.  On a row whose squares sum to more
 *                  than 3.4e38 (its y is 0) it is d_h
 *   dweight        [hidden] fp32; zeros when n_tokens == 0
 *   workspace      kda_add_rmsnorm_backward_workspace_bytes(); calls that
 *                  overlap in time need one each
 * The same inputs give the same bits on every run.
 */
size_t kda_add_rmsnorm_backward_workspace_bytes(const kda_config_t *cfg, int64_t n_tokens, int32_t hidden);

kda_status_t kda_add_rmsnorm_backward(const kda_config_t *cfg, int64_t n_tokens, int32_t hidden,
                                      const void *h, const float *weight, float eps,
                                      const void *dy, const float *d_h,
                                      float *dx, float *dweight,
                                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_output_gate with its output as e4m3 rows, the operand of the projection
 * that follows: a token's heads are one row of num_heads * head_v_dim values.
 *   y              [n_tokens][H * dv] e4m3
 *   y_scale        [n_tokens][ceil(H * dv / 128)] fp32
 * With heads of 128, o * o_norm_weight has to stay inside fp32's range, else
 * the block's scale is infinite or NaN (below 1e-38 it keeps a denormal's
 * bits); narrower heads are normalised before the weight and have no such
 * limit.  A row whose squares sum to more than 3.4e38 has y 0.
 * The other arguments as for kda_output_gate; nothing aliases.
 */
kda_status_t kda_output_gate_fp8(const kda_config_t *cfg, int64_t n_tokens,
                                 const void *o, const void *gate,
                                 const float *o_norm_weight, float eps,
                                 void *y, float *y_scale, void *stream);

/*
 * Gradient of kda_output_gate (of kda_output_gate_fp8 with the rounding taken
 * as the identity).  Per (token, head) row, with n = o / sqrt(mean o^2 + eps),
 * s = sigmoid(gate) and g = dy * o_norm_weight * s:
 *   d_o = (g - n * mean(g * n)) / sqrt(mean o^2 + eps)
 *   d_gate = dy * o_norm_weight * n * s * (1 - s)
 *   d_weight[j] = sum over tokens and heads of dy * n * s
 *   o              [n_tokens][H][dv] out_dtype; gate [n_tokens][H][dv] io_dtype
 *   dy             [n_tokens][H][dv] out_dtype: dLoss/dy
 *   d_o            [n_tokens][H][dv] out_dtype, as kda_varlen_backward takes it
 *   d_gate         [n_tokens][H][dv] fp32, as the other input gradients
 *   d_weight       [dv] fp32; zeros when n_tokens == 0
 *   workspace      kda_output_gate_backward_workspace_bytes(); calls that
 *                  overlap in time need one each
 * Nothing aliases.  The same inputs give the same bits on every run.
 */
size_t kda_output_gate_backward_workspace_bytes(const kda_config_t *cfg, int64_t n_tokens);

kda_status_t kda_output_gate_backward(const kda_config_t *cfg, int64_t n_tokens,
                                      const void *o, const void *gate,
                                      const float *o_norm_weight, float eps, const void *dy,
                                      void *d_o, float *d_gate, float *d_weight,
                                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * A projection with 8-bit operands:
 *   y[m][n] = sum over b of a_scale[m][b] * w_scale[n / 128][b]
 *                           * sum over k in block b of a[m][k] * w[n][k]
 * summed in fp32 (for bf16 y but for the cut described below) and rounded once
 * to out_dtype.
 *   a              [M][K] e4m3 rows, a_scale [M][KB] fp32, KB = ceil(K / 128)
 *   w              [N][K] e4m3 (row n holds the weights of output n)
 *   w_scale        [ceil(N / 128)][KB] fp32, one scale per 128 x 128 block
 *   y              [M][N] out_dtype
 * K is a multiple of 16; K, N up to 2^20, M below 2^31 (else
 * KDA_ERR_UNSUPPORTED).  M == 0 is a no-op; M == 1 is the single-token form.
 * A NaN scale or value reaches the outputs of its row (of its 128 columns for
 * a w_scale).  Nothing aliases.  Only out_dtype and stage_events of cfg are
 * used.  Needs no workspace.  The same inputs give the same bits on every run.
 *
 * The products of a scale block are exact and summed by the matrix cores.  For
 * fp32 y in fp32.  For bf16 y in their e4m3 form: of each 8 neighbouring
 * channels (8 i .. 8 i + 7) the products are summed in units of 2^-13 of the
 * power of two of the largest (an operand below 2^-6 counting as one of 2^-6),
 * what lies below a unit is cut, and the sums of the eights are added in fp32.
 * An eight so loses less than 7 units: over a row at most 2^-10 of the sum of
 * |a w|, a quarter of half a step of bf16 (2^-7 in an eight whose largest
 * product has an operand below 2^-6).  That is not small against the result
 * where large products cancel: 448 * 448 - 448 * 448 + 126 ones gives 112 or
 * 120.  Measured against the result's norm, in front of the rounding to bf16
 * (1.7e-3): 1.3e-5 on Gaussian operands, 4.2e-5 with two channels in 128 a
 * hundred times larger; 1.1% to 2.8% of the values are then a neighbour of the
 * nearest bf16 value.  A caller who needs fp32's sums on any operands takes y
 * in fp32 and rounds it.
 */
kda_status_t kda_fp8_matmul(const kda_config_t *cfg, int64_t M, int32_t N, int32_t K,
                            const void *a, const float *a_scale,
                            const void *w, const float *w_scale,
                            void *y, void *stream);

/*
 * ---- The full-attention layers -------------------------------------------
 *
 * In the hybrid decoders every fourth to sixth layer is full attention
 * (AliceAI page, section 三: 16 query and 2 key / value heads, an RMS norm of q
 * and k per head, rotary positions on a quarter of the channels, base 1e6).
 * The entry points below are that layer's steps between its projections.  Of
 * cfg they use num_heads (the query heads Hq), head_k_dim (the size d of every
 * head, query, key and value: 64, 128 or 256, else KDA_ERR_UNSUPPORTED),
 * head_v_dim (the same), io_dtype, out_dtype and stage_events.
 */

/* A rotation of the first rotary_dim channels of a head in pairs (a, b):
 *   (a cos t - b sin t, a sin t + b cos t),
 *   t = positions[axis[i]][token] * inv_freq[i]  for pair i < rotary_dim / 2.
 * The product is formed in 64 bits, so far positions keep their angle. */
typedef struct kda_rope {
    int32_t rotary_dim;      /* a multiple of 16, 0 .. d; 0 rotates nothing            */
    int32_t interleaved;     /* 0: pair i is channels (i, i + rotary_dim / 2);
                                1: channels (2 i, 2 i + 1)                             */
    int32_t num_axes;        /* position axes, 1 .. 4 (text has one; images time,
                                height and width)                                      */
    const float *inv_freq;   /* [rotary_dim / 2] fp32, device                          */
    const int32_t *axis;     /* [rotary_dim / 2] int32, device: the axis of each pair
                                (clamped to 0 .. num_axes - 1), or NULL: axis 0        */
} kda_rope_t;

/*
 * Norm of each query and key head, and its rotation:
 *   y = rotate(x / sqrt(mean x^2 + eps) * weight)   over the d channels of a head
 *   q              [n_tokens] rows of [Hq][d] io_dtype, q_stride elements apart
 *                  (a multiple of 8, >= Hq * d: a view into a wider projection)
 *   k              [n_tokens] rows of [num_kv_heads][d], k_stride apart; unused
 *                  with num_kv_heads == 0
 *   q_weight, k_weight  [d] fp32, or NULL: no norm of q / of k, the rotation alone.
 *                  They multiply as they are: of a zero-centred norm, as the page's,
 *                  whose factor is 1 + w, 1 + w is what goes here (here, in the
 *                  backward, where the gradient is the same, and in kda_append_kv)
 *   eps            >= 0 (NaN or negative: KDA_ERR_INVALID_ARGUMENT); with 0 a row
 *                  of zeros gives NaN.  A row whose squares sum to more than
 *                  3.4e38 gives 0
 *   rope           host struct; NULL rotates nothing
 *   positions      [num_axes][n_tokens] int32 (any value); unused without rotation
 *   q_out          [n_tokens][Hq][d] out_dtype; may alias q when q_stride ==
 *                  Hq * d and both have the same type
 *   k_out          [n_tokens][num_kv_heads][d], likewise
 * num_kv_heads 0 .. 65535.  Needs no workspace.  n_tokens == 0 is a no-op.
 */
kda_status_t kda_qk_norm_rope(const kda_config_t *cfg, const kda_rope_t *rope, int64_t n_tokens,
                              int32_t num_kv_heads, const void *q, int64_t q_stride,
                              const void *k, int64_t k_stride,
                              const float *q_weight, const float *k_weight, float eps,
                              const int32_t *positions, void *q_out, void *k_out, void *stream);

/*
 * Gradient of kda_qk_norm_rope.  With n = x / sqrt(mean x^2 + eps), g the
 * upstream gradient rotated back and u = g * weight, per head:
 *   dx = (u - n * mean(u * n)) / sqrt(mean x^2 + eps)   (without a weight: dx = g)
 *   dweight[j] = sum over tokens and heads of g * n
 *   q, k, weights, eps, rope, positions   as given to the forward
 *   dq_out, dk_out  [n_tokens][heads][d] out_dtype: dLoss/dq_out, dLoss/dk_out
 *   dq, dk          [n_tokens][heads][d] fp32; alias nothing.  0 on a row whose
 *                   squares sum to more than 3.4e38 (its y is 0)
 *   d_weight        [2][d] fp32, of q_weight then of k_weight; zeros where the
 *                   weight is NULL or there is no head or token
 *   workspace       kda_qk_norm_rope_backward_workspace_bytes(); calls that
 *                   overlap in time need one each
 * The same inputs give the same bits on every run.
 */
size_t kda_qk_norm_rope_backward_workspace_bytes(const kda_config_t *cfg, int64_t n_tokens, int32_t num_kv_heads);

kda_status_t kda_qk_norm_rope_backward(const kda_config_t *cfg, const kda_rope_t *rope, int64_t n_tokens,
                                       int32_t num_kv_heads, const void *q, int64_t q_stride,
                                       const void *k, int64_t k_stride,
                                       const float *q_weight, const float *k_weight, float eps,
                                       const int32_t *positions, const void *dq_out, const void *dk_out,
                                       float *dq, float *dk, float *d_weight,
                                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * A paged cache of keys and values in 4 bits (OCP microscaling fp4): e2m1
 * values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign; code 0 .. 7, bit 3 the sign)
 * and one e8m0 scale 2^(byte - 127) for each 32 channels of a head,
 *   E = the least with max|x| <= 6 * 2^(E - 127), at least 1;
 *   value = x / 2^(E - 127) rounded to nearest even.
 * A NaN or a magnitude of 2^127 or more in a block makes its byte 255, and the
 * block reads as NaN (253 and 254 are not written; their values may overflow).
 * A page holds page_size positions of one sequence, for all heads:
 *   k, v           [num_pages][num_kv_heads][page_size][d / 2]   two values a
 *                  byte, the even channel in the low half
 *   k_scale, v_scale  [num_pages][num_kv_heads][d / 32][page_size]
 * (16-byte aligned, e8m0 bytes 8-byte).  Position p of sequence n is position
 * p % page_size of page page_table[n * max_pages + p / page_size].  Table
 * entries outside 0 .. num_pages - 1 hold nothing: nothing is written there,
 * and attention leaves their positions out.
 */
typedef struct kda_kv_cache {
    void *k;
    void *k_scale;
    void *v;
    void *v_scale;
    int32_t num_pages;       /* any pages of one call's sequences; 0 .. 2^31 - 1       */
    int32_t page_size;       /* 32, 64, 128 or 256                                     */
    int32_t num_kv_heads;    /* 1 .. 65535; for attention a divisor of num_heads       */
    int32_t max_pages;       /* entries of a row of page_table, >= 0                   */
    const int32_t *page_table;   /* [N][max_pages], device                             */
    const int32_t *lengths;      /* [N], device: positions held of each sequence, the
                                    call's own tokens among them (what lies behind
                                    max_pages * page_size is not held)                 */
    const int32_t *cu_seqlens;   /* [N + 1], device, 0 first, nondecreasing: sequence
                                    n's tokens are rows cu[n] .. cu[n + 1] - 1 of the
                                    call's tensors; NULL: row n alone.  Rows from
                                    cu[N] on belong to no sequence and stay as they
                                    were                                               */
} kda_kv_cache_t;

/*
 * Appends keys and values: token j of the q_n tokens of sequence n goes to
 * position lengths[n] - q_n + j (a negative one is left out).
 *   k, v           [n_tokens] rows of [num_kv_heads][d] io_dtype, k_stride and
 *                  v_stride elements apart (multiples of 8, >= num_kv_heads * d)
 *   k_weight, eps, rope, positions  norm and rotation of the keys, as in
 *                  kda_qk_norm_rope; positions NULL: the cache position, on every
 *                  axis.  Keys are computed in 64 bits, so each is held as the
 *                  nearest value of its block's scale
 * Two tokens of one call must not go to one position of one page (a page that
 * two sequences share is appended to by one of them).  N == 0 or n_tokens == 0
 * is a no-op.  N up to 2^24.  Needs no workspace.
 */
kda_status_t kda_append_kv(const kda_config_t *cfg, const kda_rope_t *rope, const kda_kv_cache_t *cache, int32_t N,
                           int64_t n_tokens, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                           const float *k_weight, float eps, const int32_t *positions, void *stream);

/*
 * Reads rows back: k_out, v_out [n_tokens][num_kv_heads][d] out_dtype (either
 * may be NULL), token j of sequence n from position lengths[n] - q_n + j.  Rows
 * of positions that are not held are 0.
 */
kda_status_t kda_read_kv(const kda_config_t *cfg, const kda_kv_cache_t *cache, int32_t N, int64_t n_tokens,
                         void *k_out, void *v_out, void *stream);

/*
 * Attention of each sequence's newest tokens over its cache, causal among them:
 *   token j of the q_n tokens of sequence n sees positions 0 .. lengths[n] - q_n + j,
 *   those of them that are held (also where lengths[n] passes the table)
 *   o = sum_p w_p v_p,  w = softmax over those positions of scale * q . k_p
 * where query head h reads key / value head h * num_kv_heads / num_heads.
 *   q              [n_tokens][Hq][d] io_dtype (16-byte aligned)
 *   scale          finite, e.g. 1 / sqrt(d)
 *   max_q          at least the largest q_n, or 0 if not known: only the choice
 *                  of the kernel (0: by the mean n_tokens / N) and the workspace
 *                  (0: of the most that it can be) go by it
 *   o              [n_tokens][Hq][d] out_dtype; 0 for a token that sees nothing
 *   lse            [n_tokens][Hq] fp32: log(sum exp(scale * q . k_p)), -infinity
 *                  for a token that sees nothing; or NULL
 *   workspace      kda_paged_attention_workspace_bytes(); calls that overlap in
 *                  time need one each.  Nothing in it is kept between calls.  The
 *                  bytes grow with n_tokens, N and max_q (0 counts as n_tokens):
 *                  one that is right for a call is enough for every smaller one
 *                  of the same heads and types.  At most 18 MB without, and 204
 *                  MB (103 at d 128, 52 at 64) with chunks of many rows, plus 32
 *                  bytes for each tile of up to 256 rows of a sequence and key head
 * Positions that a token does not see, whatever their bytes, have no effect on
 * it, and a token's precision does not go by what else is in the call.  Sums and
 * the softmax are fp32, queries and keys exact.  Weights meet the values to within
 * 2^-16 of themselves for bf16 outputs, and for fp32 outputs to within fp32's
 * rounding.  N up to 4096 (else KDA_ERR_UNSUPPORTED).  Nothing aliases.  The
 * same inputs give the same bits on every run.
 */
size_t kda_paged_attention_workspace_bytes(const kda_config_t *cfg, int32_t num_kv_heads, int32_t N,
                                           int64_t n_tokens, int32_t max_q);

kda_status_t kda_paged_attention(const kda_config_t *cfg, const kda_kv_cache_t *cache, int32_t N, int64_t n_tokens,
                                 int32_t max_q, const void *q, float scale, void *o, float *lse,
                                 void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
