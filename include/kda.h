/*
 * kda.h -- C ABI of libkda, the Kimi Delta Attention (KDA) operator for
 * AMD Instinct MI355X (gfx950).
 *
 * KDA is a gated delta-rule linear attention ("Kimi K3" explainer, "Across
 * the sequence"): per head it keeps a fixed-size state S[d_k][d_v] and, for
 * each token t in order,
 *     S   <- Diag(exp(g_t)) S                 channel-wise forgetting
 *     u_t  = beta_t (v_t - S^T k_t)
 *     S   <- S + k_t u_t^T
 *     o_t  = S^T q_t
 * with the bounded log-decay g_t = KDA_G_MIN * sigmoid(theta_t)
 * ("Architecture Deep Dive: Kimi K3...", section 3.2, equation 1; "Kimi K3
 * Deep Dive...", "The Design: Putting a Lower Bound on Log-Decay").
 *
 * Conventions shared by every call:
 *  - Pointers are DEVICE pointers into memory the caller owns (for instance
 *    torch tensors).  The library never allocates, frees or retains them.
 *    Its only global state is a thread-local error string and, for
 *    kda_chunk_fwd_noalloc, one static device scratch array per device.
 *  - Tensors are dense and row-major in the layouts stated per argument; the
 *    innermost dimension is contiguous.  Every pointer must be 16-byte aligned.
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *    Work is enqueued asynchronously on it; KDA_OK means "validated and
 *    enqueued".  Faults inside kernels surface at the caller's next
 *    synchronisation of that stream.
 *  - All argument checks run on the host before any HIP call, so every error
 *    return leaves device memory untouched and enqueues nothing.
 *  - Non-finite inputs are not checked; they propagate into the outputs.
 *  - Results are deterministic run to run (no floating-point atomics).
 *  - Supported head sizes: d_k = d_v in {16, 32, 64, 128}.
 *  - dtype of q, k, v and o: KDA_BF16 (bf16 storage, bf16 matrix-core
 *    operands, fp32 accumulation and fp32 state) or KDA_F32 (fp32 storage and
 *    fp32 arithmetic throughout; a validation mode).  fp16 is not offered:
 *    exp(16 * 5) = 5.5e34 exceeds its range.  theta, beta and the states are
 *    always fp32.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens per chunk of the chunked evaluation (the pages' 16-token tile). */
#define KDA_CHUNK 16
/* Fixed lower bound of the log-decay g (the pages set it to -5). */
#define KDA_G_MIN (-5.0f)
/* Version of this ABI; bumped on any incompatible change. */
#define KDA_ABI_VERSION 1

typedef enum kda_dtype { KDA_BF16 = 0, KDA_F32 = 1 } kda_dtype;

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_NULL = 1,       /* a required pointer is NULL                         */
    KDA_ERR_SHAPE = 2,      /* a size is out of range or unsupported              */
    KDA_ERR_DTYPE = 3,      /* unknown dtype code                                 */
    KDA_ERR_ALIGN = 4,      /* a pointer is not 16-byte aligned                   */
    KDA_ERR_WORKSPACE = 5,  /* workspace missing or smaller than required         */
    KDA_ERR_ALIAS = 6,      /* an output overlaps memory it must not overlap      */
    KDA_ERR_HIP = 7         /* the HIP runtime reported an error at launch        */
} kda_status;

/* ---------------------------------------------------------------------------
 * kda_chunk_fwd: chunked prefill ("Kimi K3 Deep Dive...", "The Problem: The
 * Diagonal-Block Dilemma": 16-token chunks with intra-chunk (diagonal) and
 * inter-chunk causal paths; the bounded gate lets both run as dense matrix
 * products, "Architecture Deep Dive", section 3.2).
 *
 * Runs the recurrence over T tokens for every (batch, head) from the start
 * state S0 and returns every output o_t and the final state S_T.
 *
 *   dtype        KDA_BF16 or KDA_F32 (storage of q, k, v, o)
 *   B, T, H      batch, tokens (T >= 1), heads; B, H >= 1
 *   dk, dv       head sizes, equal, in {16, 32, 64, 128}
 *   segments     how many pieces each sequence is cut into along T for
 *                parallel evaluation (each piece's affine state map is
 *                composed afterwards); 0 = the library's choice, which is
 *                what kda_chunk_fwd_auto_segments returns.  Any value from 1
 *                to ceil(T/16) gives the same result up to rounding.
 *   q, k         [B, T, H, dk]   dtype
 *   v            [B, T, H, dv]   dtype
 *   theta        [B, T, H, dk]   fp32; the gate applies KDA_G_MIN*sigmoid
 *   beta         [B, T, H]       fp32, used as given (no sigmoid applied)
 *   S0           [B, H, dk, dv]  fp32 start state, or NULL for zero
 *   o            [B, T, H, dv]   dtype, written
 *   S_T          [B, H, dk, dv]  fp32 final state, written; or NULL to skip.
 *                S_T may be the same pointer as S0 (in-place update); any
 *                other overlap between an output and an input is rejected.
 *   workspace    device scratch of at least kda_chunk_fwd_workspace_size
 *                bytes (may be NULL when that size is 0); contents on entry
 *                are ignored, on exit unspecified.
 *   stream       hipStream_t as void*
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_chunk_fwd(int dtype, int B, int T, int H, int dk, int dv, int segments,
                  const void* q, const void* k, const void* v,
                  const float* theta, const float* beta, const float* S0,
                  void* o, float* S_T,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device scratch that kda_chunk_fwd_noalloc holds per device. */
#define KDA_NOALLOC_SCRATCH_BYTES (128u << 20)

/* ---------------------------------------------------------------------------
 * kda_chunk_fwd_noalloc: kda_chunk_fwd for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  It takes no workspace: a segmented call uses a static
 * device array of KDA_NOALLOC_SCRATCH_BYTES (128 MiB) that each device the
 * library runs on holds from its first call there until the process ends.
 * The call itself allocates and frees nothing.
 *
 *   Every argument and the result are those of kda_chunk_fwd, without
 *   workspace and workspace_bytes.  The scratch is the one of the calling
 *   thread's current device; `stream` must belong to that device.
 *   Errors: those of kda_chunk_fwd, and KDA_ERR_WORKSPACE when the segment
 *   count (given, or the automatic one for segments = 0) needs more than
 *   KDA_NOALLOC_SCRATCH_BYTES (kda_chunk_fwd_workspace_size gives the need;
 *   one segment needs none).  The 64K-token prefill of 16 heads at d = 128
 *   with its automatic 16 segments needs 110 MiB and fits.
 *   The scratch holds nothing that must start at zero and keeps the last
 *   call's contents.  Every call on one device shares that device's scratch:
 *   calls that overlap in time on one device (several streams or threads)
 *   race and give undefined results; serialise them.
 * ------------------------------------------------------------------------- */
int kda_chunk_fwd_noalloc(int dtype, int B, int T, int H, int dk, int dv, int segments,
                          const void* q, const void* k, const void* v,
                          const float* theta, const float* beta, const float* S0,
                          void* o, float* S_T, void* stream);

/* ---------------------------------------------------------------------------
 * kda_chunk_fwd_gated: kda_chunk_fwd with the output gate applied to o
 * ("Kimi K3" explainer, "Across the sequence": in the model, the attention
 * output is multiplied channel by channel, token by token, by a sigmoid of a
 * pre-activation computed from the layer's input):
 *     o_t[j] = sigmoid(z_t[j]) * (S_t^T q_t)[j]
 * The gate acts on the output only; S_T is the same as kda_chunk_fwd's.
 *
 *   z            [B, T, H, dv]   dtype, the gate's pre-activation; must be
 *                non-NULL and 16-byte aligned, and must not overlap o, S_T or
 *                the workspace.
 *   Every other argument, the workspace size and the errors are those of
 *   kda_chunk_fwd.  The ungated output is rounded to dtype, multiplied by the
 *   gate in fp32 and rounded again.
 * ------------------------------------------------------------------------- */
int kda_chunk_fwd_gated(int dtype, int B, int T, int H, int dk, int dv, int segments,
                        const void* q, const void* k, const void* v,
                        const float* theta, const float* beta, const float* S0,
                        const void* z, void* o, float* S_T,
                        void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * kda_chunk_fwd_unbounded: the ablation of the bound.  The same recurrence
 * with the conventional unbounded log-decay that the bounded gate replaces
 * ("Kimi K3 Deep Dive...", "The Design: Putting a Lower Bound on Log-Decay"):
 *     g = -softplus(theta) = -ln(1 + e^theta),   range (-inf, 0)
 * instead of KDA_G_MIN*sigmoid(theta).  The inverse cumulative decay inside a
 * chunk is then unbounded and can overflow any floating-point type, so the two
 * diagonal tiles are formed position by position in fp32 ("Architecture Deep
 * Dive...", section 3.1) instead of as matrix products; everything else is the
 * chunked evaluation of kda_chunk_fwd.  It exists to measure what the bound
 * buys, not for use in a model.
 *
 *   Arguments as kda_chunk_fwd, without segments (always one: no workspace),
 *   with the same validation and errors.  Where the unbounded gate drives a
 *   decay below fp32's range the result is the limit (the state forgets).
 * ------------------------------------------------------------------------- */
int kda_chunk_fwd_unbounded(int dtype, int B, int T, int H, int dk, int dv,
                            const void* q, const void* k, const void* v,
                            const float* theta, const float* beta, const float* S0,
                            void* o, float* S_T, void* stream);

/* ---------------------------------------------------------------------------
 * kda_chunk_bwd: the backward pass of kda_chunk_fwd.  For the scalar
 *     L = sum_t <do_t, o_t> + <dS_T, S_T>
 * it writes the gradients of L with respect to q, k, v, theta, beta and S0, by
 * the chain rule through the recurrence taken chunk by chunk (the chunk form of
 * "Kimi K3 Deep Dive...", "The Problem: The Diagonal-Block Dilemma", run in
 * reverse; the training step the pages' kernel design serves, "Architecture
 * Deep Dive...", section 3.2).  dtheta includes the gate's derivative
 * KDA_G_MIN * sigmoid(theta) (1 - sigmoid(theta)).
 *
 *   dtype, B, T, H, dk, dv, q, k, v, theta, beta, S0   as kda_chunk_fwd
 *   do           [B, T, H, dv]   dtype, gradient of L with respect to o
 *   dS_T         [B, H, dk, dv]  fp32, gradient with respect to S_T, or NULL (zero)
 *   dq, dk       [B, T, H, dk]   fp32, written
 *   dv           [B, T, H, dv]   fp32, written
 *   dtheta       [B, T, H, dk]   fp32, written
 *   dbeta        [B, T, H]       fp32, written
 *   dS0          [B, H, dk, dv]  fp32, written; or NULL to skip
 *   workspace    kda_chunk_bwd_workspace_size bytes of device memory (every
 *                chunk's start state, and at dk = 64 and 128 its U and
 *                V - K+ S tiles and the segment maps and boundary values, fp32);
 *                contents on entry do not matter
 *   stream       hipStream_t the work is enqueued on
 * Returns KDA_OK once enqueued.  Errors (before any HIP call): as kda_chunk_fwd;
 * every gradient output must not overlap an input, another output or the
 * workspace.  One workgroup per (batch, head) walks the chunks in order; with
 * at most 64 (batch, head) pairs and at least 64 chunks (dk = 64 and 128) each
 * sequence is split into segments joined by their affine maps, as in the
 * forward.  Results are deterministic run to run.
 * ------------------------------------------------------------------------- */
int kda_chunk_bwd(int dtype, int B, int T, int H, int dk, int dv,
                  const void* q, const void* k, const void* v,
                  const float* theta, const float* beta, const float* S0,
                  const void* do_, const float* dS_T,
                  float* dq, float* dk_, float* dv_, float* dtheta, float* dbeta, float* dS0,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace kda_chunk_bwd needs.  Writes *bytes; returns a kda_status. */
int kda_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, size_t* bytes);

/* Bytes of workspace kda_chunk_fwd needs for these sizes and this segment
 * count (0 = automatic).  Writes *bytes; returns a kda_status. */
int kda_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int segments,
                                 size_t* bytes);

/* The segment count kda_chunk_fwd uses when passed 0 (depends on sizes only,
 * never on the device).  Returns it, or a value <= 0 for invalid sizes. */
int kda_chunk_fwd_auto_segments(int B, int T, int H, int dk, int dv);

/* ---------------------------------------------------------------------------
 * kda_decode_step: one token of the recurrence for every (batch, head), with
 * the fixed-size state updated in place ("Kimi K3" explainer, "Across the
 * sequence": the state does not grow with context length).
 *
 *   dtype        KDA_BF16 or KDA_F32 (storage of q, k, v, o)
 *   B, H         >= 1;  dk, dv as for kda_chunk_fwd
 *   q, k         [B, H, dk]      dtype
 *   v            [B, H, dv]      dtype
 *   theta        [B, H, dk]      fp32
 *   beta         [B, H]          fp32
 *   S            [B, H, dk, dv]  fp32, read and overwritten with the new state
 *   o            [B, H, dv]      dtype, written; must not overlap any input
 *   stream       hipStream_t as void*
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_decode_step(int dtype, int B, int H, int dk, int dv,
                    const void* q, const void* k, const void* v,
                    const float* theta, const float* beta,
                    float* S, void* o, void* stream);

/* ---------------------------------------------------------------------------
 * kda_decode_step_gated: kda_decode_step with the output gate of
 * kda_chunk_fwd_gated, o[j] = sigmoid(z[j]) * (S'^T q)[j], formed in fp32 and
 * rounded once to dtype.
 *
 *   z            [B, H, dv]      dtype; non-NULL, 16-byte aligned, and not
 *                overlapping o or S.
 *   Every other argument and the errors are those of kda_decode_step; the
 *   state update is the same.
 * ------------------------------------------------------------------------- */
int kda_decode_step_gated(int dtype, int B, int H, int dk, int dv,
                          const void* q, const void* k, const void* v,
                          const float* theta, const float* beta,
                          float* S, const void* z, void* o, void* stream);

/* ---------------------------------------------------------------------------
 * kda_gate: the bounded gate on its own ("Architecture Deep Dive", section 3.2,
 * equation 1; "Kimi K3 Deep Dive", illustrative code of the lower-bounded
 * log-decay).
 *
 *   B, T, H, dk  sizes (dk in {16, 32, 64, 128}), T >= 1
 *   theta        [B, T, H, dk] fp32
 *   g            [B, T, H, dk] fp32 or NULL: g = KDA_G_MIN * sigmoid(theta)
 *   g_cum        [B, T, H, dk] fp32 or NULL: inclusive prefix sum of g along T
 *                restarted at every 16-token chunk (t = 0, 16, 32, ...)
 *   At least one of g, g_cum must be non-NULL; neither may overlap theta or
 *   each other.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_gate(int B, int T, int H, int dk, const float* theta, float* g, float* g_cum,
             void* stream);

/* ===========================================================================
 * The gated delta rule with one decay a head.
 *
 * The sibling of KDA whose forgetting is one factor a token and head instead of
 * one a channel, given as a log-decay g_t <= 0 without a lower bound.  Per
 * value head h, whose key head is h / (Hv / Hk), with a state S[dk][dv]:
 *     S   <- exp(g_t) S
 *     e_t  = v_t - S^T k_t
 *     S   <- S + beta_t k_t e_t^T
 *     o_t  = scale S^T q_t
 * The entries below share the conventions above, and these:
 *  - Hv is a multiple of Hk; dk is 32, 64 or 128; dv a multiple of 32 from 32
 *    to 256, dk and dv independent of each other.
 *  - g below -120 (minus infinity included) forgets the state entirely; beta is used
 *    as given.  Positive g is used as it is (the state grows).
 *  - KDA_BF16 means bf16 storage of q, k, v, o (and of do, dq, dk, dv).  The state,
 *    g, beta and their gradients are fp32, and so is the arithmetic: products of
 *    intermediate results run on the bf16 matrix cores as sums over three parts of
 *    each factor, which keep all its 24 bits.  KDA_F32 keeps fp32 storage and the
 *    fp32 matrix cores throughout.
 * ------------------------------------------------------------------------- */

/* ---------------------------------------------------------------------------
 * kda_gdr_chunk_fwd: the rule over whole sequences in chunks of 64 tokens (prefill,
 * training), from a start state to a last state.  A value that is not finite may reach every
 * row of its chunk and head, the ones before it among them, and everything behind it in its
 * sequence; other sequences and heads never see it.
 *
 *   nseq, T      cu_seqlens NULL: nseq sequences of T tokens each, tensors [nseq, T, ...].
 *                Otherwise the sequences are packed into T rows, tensors [T, ...].
 *   cu_seqlens   [nseq + 1] int32, read on the device: sequence n has the rows from
 *                cu_seqlens[n] up to cu_seqlens[n + 1].  Offsets rise from at least 0
 *                to at most T; equal ones are a sequence of no tokens, whose S_T is its
 *                S0.  Rows of no sequence are neither read nor written.  Offsets out of order
 *                or range are held to both, so nothing outside the tensors is touched; the
 *                results are then unspecified.
 *   q, k         [.., Hk, dk]  dtype
 *   v            [.., Hv, dv]  dtype
 *   g, beta      [.., Hv]      fp32
 *   S0           [nseq, Hv, dk, dv]  fp32, or NULL for zero
 *   o            [.., Hv, dv]  dtype, written
 *   S_T          [nseq, Hv, dk, dv]  fp32, written; or NULL to skip.  May be S0 itself.
 *   workspace    kda_gdr_chunk_fwd_workspace_size bytes; contents on entry do not matter
 *   Any other overlap of an output with an input, an output or the workspace is rejected.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_gdr_chunk_fwd(int dtype, int nseq, int T, int Hk, int Hv, int dk, int dv, float scale,
                      const int* cu_seqlens, const void* q, const void* k, const void* v,
                      const float* g, const float* beta, const float* S0, void* o, float* S_T,
                      void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * kda_gdr_chunk_bwd: gradients of L = sum <do, o> + <dS_T, S_T> with respect to q, k, v,
 * g, beta and S0, from the forward's inputs (nothing of it is saved).
 *
 *   do           as o;  dS_T  as S_T, or NULL for zero
 *   dq, dk       as q, summed over the value heads of a key head; dv as v: dtype, written
 *   dg, dbeta    as g, fp32, written
 *   dS0          as S0, fp32, written; or NULL to skip
 *   workspace    kda_gdr_chunk_bwd_workspace_size bytes (at dk = dv = 128 206 KiB a chunk
 *                of 64 tokens and value head)
 *   Every other argument is that of kda_gdr_chunk_fwd; no output may overlap anything.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_gdr_chunk_bwd(int dtype, int nseq, int T, int Hk, int Hv, int dk, int dv, float scale,
                      const int* cu_seqlens, const void* q, const void* k, const void* v,
                      const float* g, const float* beta, const float* S0,
                      const void* do_, const float* dS_T,
                      void* dq, void* dk_, void* dv_, float* dg, float* dbeta, float* dS0,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of the two calls; packed: whether cu_seqlens is given.  Writes *bytes;
 * returns a kda_status. */
int kda_gdr_chunk_fwd_workspace_size(int nseq, int T, int Hv, int dk, int dv, int packed, size_t* bytes);
int kda_gdr_chunk_bwd_workspace_size(int nseq, int T, int Hv, int dk, int dv, int packed, size_t* bytes);

/* ---------------------------------------------------------------------------
 * kda_gdr_clear_rows: zeros in the rows of no sequence of packed tensors, which the two
 * calls above leave as they were: those before cu_seqlens[0] and from
 * cu_seqlens[nseq] on.  No other row is touched.
 *
 *   nseq, T, cu_seqlens   as above, cu_seqlens not NULL
 *   n            tensors, 1 to 8
 *   tensors      n device pointers, 16-byte aligned, that overlap nothing; read on the host
 *   row_bytes    the bytes of a row of each, a multiple of 4 below 2^31; read on the host
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_gdr_clear_rows(int nseq, int T, const int* cu_seqlens, int n, void* const* tensors,
                       const size_t* row_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * kda_gdr_step: T tokens of the rule for each of B rows, from and to a state in a
 * pool, in place (decode: T = 1; proposed tokens: T of a few).  The state is read
 * and written once a call.
 *
 *   nslot        states in the pool
 *   q, k         [B, T, Hk, dk]  dtype
 *   v            [B, T, Hv, dv]  dtype
 *   g, beta      [B, T, Hv]      fp32
 *   S            [nslot, Hv, dk, dv]  fp32, the rows' states read and overwritten
 *   slots        [B] int32, the state of each row, or NULL: row b has state b
 *                (nslot >= B).  A slot outside [0, nslot) marks a padded row.  Of the
 *                rows with tokens that name one slot the first has it and the others
 *                count as padded.
 *   ntok         [B] int32, how many of a row's T tokens are real (more than T counts
 *                as T), or NULL: all.  With none the row is padded.
 *   o            [B, T, Hv, dv]  dtype, written for the real tokens of rows that are not
 *                padded and left as it was elsewhere; must not overlap any input
 *   slots and ntok are read on the device, when the work runs.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_gdr_step(int dtype, int B, int T, int Hk, int Hv, int dk, int dv, int nslot, float scale,
                 const void* q, const void* k, const void* v, const float* g, const float* beta,
                 float* S, const int* slots, const int* ntok, void* o, void* stream);

/* ===========================================================================
 * The norms around a block, fused with its gate, residual scale and residual sum.
 *
 * Per row of D channels, every operand but y optional (NULL):
 *     n = y / sqrt(mean(y^2) + eps) * w_post     norm after the block   (w_post NULL: n = y)
 *     a = n * act(z) * s                         gate, residual scale   (z, s NULL: factor 1)
 *     r = x + a                                  residual stream        (x NULL: r = a)
 *     h = r / sqrt(mean(r^2) + eps) * w_pre      norm before the next block
 * With rows = tokens x heads and D = dv, y and z alone it is the output norm and gate of
 * a KDA or gated-delta-rule head; with rows = tokens it stands between two blocks.
 * All arithmetic is fp32; h is formed from r before r is rounded.
 *
 *   dtype        storage of y, x, z, r, h and of their gradients
 *   act          KDA_ACT_SIGMOID: act(z) = 1/(1+e^-z);  KDA_ACT_SILU: z/(1+e^-z)
 *   rows, D      rows >= 1; D a multiple of 8 from 8 to 8192
 *   eps          in [0, 1]; with 0 a row of zeros is 0 / 0, NaN.  The sum of a row's squares
 *                is fp32: values up to 1e19 / sqrt(D) are in its range, and with eps 0 a row
 *                of values all below 1e-19 loses digits
 *   y, x, z      [rows, D]  dtype
 *   w_post, s, w_pre   [D]  fp32
 *   r            [rows, D]  dtype, written; may be x itself
 *   h            [rows, D]  dtype, written; NULL exactly when w_pre is
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
typedef enum kda_act { KDA_ACT_SIGMOID = 0, KDA_ACT_SILU = 1 } kda_act;

int kda_block_norm_fwd(int dtype, int act, long long rows, int D, float eps,
                       const void* y, const void* x, const void* z,
                       const float* w_post, const float* s, const float* w_pre,
                       void* r, void* h, void* stream);

/* ---------------------------------------------------------------------------
 * kda_block_norm_bwd: gradients of L = sum <dr, r> + <dh, h>, from the inputs of the
 * forward alone (nothing of it is saved).
 *
 *   dr           [rows, D]  dtype, or NULL (zero);  dh  [rows, D]  dtype, NULL exactly
 *                when w_pre is; one of the two must be given
 *   dy           [rows, D]  dtype, written
 *   dx, dz       [rows, D]  dtype, written; or NULL to skip
 *   dw_post, ds, dw_pre   [D]  fp32, written (sums over the rows, in a fixed order);
 *                or NULL to skip
 *   workspace    kda_block_norm_bwd_workspace_size bytes when a weight's gradient is
 *                asked for; otherwise it may be NULL
 *   No output may overlap an input, another output or the workspace.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_block_norm_bwd(int dtype, int act, long long rows, int D, float eps,
                       const void* y, const void* x, const void* z,
                       const float* w_post, const float* s, const float* w_pre,
                       const void* dr, const void* dh,
                       void* dy, void* dx, void* dz, float* dw_post, float* ds, float* dw_pre,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace kda_block_norm_bwd needs.  Writes *bytes; returns a kda_status. */
int kda_block_norm_bwd_workspace_size(long long rows, int D, size_t* bytes);

/* ===========================================================================
 * The operators of a state-space block.
 *
 * Conventions as above; D, the channels, lie side by side in a row, a row a token.  Sequences
 * are nseq times T tokens, or packed as for kda_gdr_chunk_fwd (cu_seqlens, with what is said
 * there of offsets).  Rows of no sequence: the forward calls leave those of y alone, or zero
 * them with zero_rest = 1; the backward calls zero those of all gradients.  The step calls take
 * slots and ntok as kda_gdr_step does.
 * ------------------------------------------------------------------------- */

/* ---------------------------------------------------------------------------
 * kda_sel_scan_fwd: the selective scan, a state-space recurrence whose step size, input and output
 * vectors depend on the token.  Channel d keeps N states h_n and belongs to group d / (D / G):
 *     delta_t = softplus(dt_t + dt_bias)        (softplus = 0: dt_t + dt_bias)
 *     h_n    <- exp(delta_t A_n) h_n + delta_t x_t b_t,n
 *     y_t     = (sum_n c_t,n h_n + skip x_t) z_t / (1 + e^-z_t)
 *
 *   dtype        storage of x, dt, b, c, z and y; all arithmetic, A and the states are fp32
 *   T            at most 2^30;  D at most 2^20, D / G a multiple of 8;  N 8, 16, 32 or 64
 *   nseq         fewer than 2^24 workgroups a call, for which (nseq + 2048) G ceil(D / G / 64) < 2^24 is enough
 *   x, dt, z     [.., D]     dtype; z NULL: no gate
 *   A            [D, N]      fp32, used as given (negative in a model that forgets); finite.  Where states
 *                grow, exp(A sum delta) has to stay within fp32 over every part of a sequence
 *   b, c         [.., G, N]  dtype
 *   skip, dt_bias  [D]       fp32, or NULL for zero
 *   S0           [nseq, D, N]  fp32, or NULL for zero
 *   y            [.., D]     dtype, written
 *   S_T          [nseq, D, N]  fp32, written; or NULL to skip.  May be S0 itself.
 *   workspace    kda_sel_scan_fwd_workspace_size bytes (NULL where that is 0); contents on entry do not matter
 *   A value that is not finite reaches what follows it in its sequence (in b and c in all channels of the group, elsewhere in its own).
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_sel_scan_fwd(int dtype, int nseq, int T, int D, int N, int G, int softplus, const int* cu_seqlens,
                     int zero_rest, const void* x, const void* dt, const float* A, const void* b, const void* c, const float* skip,
                     const void* z, const float* dt_bias, const float* S0, void* y, float* S_T,
                     void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * kda_sel_scan_bwd: gradients of L = sum <dy, y> + <dS_T, S_T> with respect to every input, from
 * the forward's inputs (nothing of it is saved).
 *
 *   dy           as y;  dS_T  as S_T, or NULL for zero
 *   dx, ddt, dz  as x; dz goes with z;  db, dc  as b, summed over a group's channels: dtype, written
 *   dA           [D, N] fp32, written;  dskip, ddt_bias  [D] fp32, written, or NULL to skip
 *   dS0          as S0, fp32, written; or NULL to skip
 *   workspace    kda_sel_scan_bwd_workspace_size bytes: about D N / 4 + 8 N B a token, B = G ceil(D / G / 64); 24 D N
 *                a piece of sequences, which has at least 64 tokens (32 where none is longer; one piece at
 *                least); and (N + 2) / 2 MiB at most.  However many sequences the rows are
 *   No output may overlap anything.  Sums over rows and channels are in a fixed order.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_sel_scan_bwd(int dtype, int nseq, int T, int D, int N, int G, int softplus, const int* cu_seqlens,
                     const void* x, const void* dt, const float* A, const void* b, const void* c, const float* skip,
                     const void* z, const float* dt_bias, const float* S0, const void* dy, const float* dS_T,
                     void* dx, void* ddt, float* dA, void* db, void* dc, float* dskip, void* dz, float* ddt_bias,
                     float* dS0, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace of the two calls; packed: whether cu_seqlens is given.  Writes *bytes;
 * returns a kda_status. */
int kda_sel_scan_fwd_workspace_size(int nseq, int T, int D, int N, int G, int packed, size_t* bytes);
int kda_sel_scan_bwd_workspace_size(int nseq, int T, int D, int N, int G, int packed, size_t* bytes);

/* ---------------------------------------------------------------------------
 * kda_sel_scan_step: T tokens of the scan for each of B rows, from and to a state in a pool, in
 * place.  The state is read and written once a call.
 *
 *   x, dt, z     [B, T, D]  dtype;  b, c  [B, T, G, N]  dtype;  A, skip, dt_bias as above
 *   S            [nslot, D, N]  fp32, the rows' states read and overwritten
 *   slots, ntok  [B] int32, as for kda_gdr_step
 *   y            [B, T, D]  dtype, written for the real tokens of rows that are not padded
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_sel_scan_step(int dtype, int B, int T, int D, int N, int G, int nslot, int softplus, const void* x,
                      const void* dt, const float* A, const void* b, const void* c, const float* skip, const void* z,
                      const float* dt_bias, float* S, const int* slots, const int* ntok, void* y, void* stream);

/* ---------------------------------------------------------------------------
 * kda_short_conv_fwd: the short causal convolution of every channel over its own last W inputs,
 * before the scan or before the queries, keys and values of a delta rule:
 *     y_t = act(bias + sum_j w_j x_{t-W+1+j})
 * where inputs before the first are S0's (the last W - 1 before the sequence, oldest first).
 *
 *   act          KDA_CONV_LINEAR: the identity;  KDA_CONV_SILU: p / (1 + e^-p)
 *   T            at most 2^30;  D a multiple of 8, at most 2^20;  W 2, 3 or 4
 *   x            [.., D]   dtype
 *   w            [D, W]    fp32;  bias  [D] fp32, or NULL for zero
 *   S0           [nseq, W - 1, D]  dtype, or NULL for zero
 *   y            [.., D]   dtype, written
 *   S_T          [nseq, W - 1, D]  dtype, the last W - 1 inputs, S0's among them where a
 *                sequence is short; or NULL to skip.  May be S0 itself.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
typedef enum kda_conv_act { KDA_CONV_LINEAR = 0, KDA_CONV_SILU = 1 } kda_conv_act;

int kda_short_conv_fwd(int dtype, int act, int nseq, int T, int D, int W, const int* cu_seqlens, int zero_rest,
                       const void* x, const float* w, const float* bias, const void* S0, void* y, void* S_T, void* stream);

/* ---------------------------------------------------------------------------
 * kda_short_conv_bwd: gradients of L = sum <dy, y> + <dS_T, S_T>, from the forward's inputs.
 *
 *   dy           as y;  dS_T  as S_T, or NULL for zero
 *   dx           as x, dtype, written;  dw  [D, W] fp32, written
 *   dbias        [D] fp32, written, or NULL to skip;  dS0  as S0, dtype, written, or NULL to skip
 *   workspace    kda_short_conv_bwd_workspace_size bytes, rows being all rows of x
 *   No output may overlap anything.  Sums over rows are in a fixed order.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_short_conv_bwd(int dtype, int act, int nseq, int T, int D, int W, const int* cu_seqlens, const void* x,
                       const float* w, const float* bias, const void* S0, const void* dy, const void* dS_T,
                       void* dx, float* dw, float* dbias, void* dS0,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace kda_short_conv_bwd needs.  Writes *bytes; returns a kda_status. */
int kda_short_conv_bwd_workspace_size(long long rows, int D, int W, size_t* bytes);

/* ---------------------------------------------------------------------------
 * kda_short_conv_step: T tokens of the convolution for each of B rows, from and to a state in
 * a pool, in place.
 *
 *   x            [B, T, D]  dtype;  w, bias as above
 *   S            [nslot, W - 1, D]  dtype, the rows' states read and overwritten
 *   slots, ntok  [B] int32, as for kda_gdr_step
 *   y            [B, T, D]  dtype, written for the real tokens of rows that are not padded
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_short_conv_step(int dtype, int act, int B, int T, int D, int W, int nslot, const void* x, const float* w,
                        const float* bias, void* S, const int* slots, const int* ntok, void* y, void* stream);

/* ---------------------------------------------------------------------------
 * kda_layer_norm_fwd: the layer norm behind a residual sum, per row of D channels:
 *     r = x + y                                              (x NULL: r = y, not written)
 *     h = (r - mean(r)) / sqrt(mean((r - mean(r))^2) + eps) * w + b    (w, b NULL: 1 and 0)
 * All arithmetic is fp32; h is formed from r before r is rounded.
 *
 *   rows, D, eps as for kda_block_norm_fwd; with eps 0 a row of equal values has no
 *                direction and comes out as NaN or as rounding errors.  The sum of the squares
 *                is fp32: values within 1e19 / sqrt(D) of their mean are in its range
 *   y, x         [rows, D]  dtype;  w, b  [D] fp32
 *   r            [rows, D]  dtype, written; may be x itself; NULL exactly when x is
 *   h            [rows, D]  dtype, written
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_layer_norm_fwd(int dtype, long long rows, int D, float eps, const void* y, const void* x, const float* w,
                       const float* b, void* r, void* h, void* stream);

/* ---------------------------------------------------------------------------
 * kda_layer_norm_bwd: gradients of L = sum <dr, r> + <dh, h>, from the inputs of the forward alone.
 *
 *   dr           [rows, D]  dtype, or NULL (zero; it goes with x);  dh  [rows, D]  dtype
 *   dy           [rows, D]  dtype, written: the gradient of y, and of x, which has the same
 *   dw, db       [D] fp32, written (sums over the rows, in a fixed order); or NULL to skip
 *   workspace    kda_layer_norm_bwd_workspace_size bytes when dw or db is asked for
 *   No output may overlap an input, another output or the workspace.
 * Returns a kda_status.
 * ------------------------------------------------------------------------- */
int kda_layer_norm_bwd(int dtype, long long rows, int D, float eps, const void* y, const void* x, const float* w,
                       const void* dr, const void* dh, void* dy, float* dw, float* db,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace kda_layer_norm_bwd needs.  Writes *bytes; returns a kda_status. */
int kda_layer_norm_bwd_workspace_size(long long rows, int D, size_t* bytes);

/* Static description of a status code (never NULL). */
const char* kda_status_string(int status);

/* Thread-local detail about the last non-OK return on this thread ("" if none). */
const char* kda_last_error(void);

/* KDA_ABI_VERSION of the loaded library. */
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
