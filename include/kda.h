/*
 * kda.h — C ABI of libkda: the KDA gated delta-rule recurrence on AMD
 * Instinct MI355X (gfx950).
 *
 * The operation (per sequence n and head h; S is d_k x d_v, fp32):
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t ,          alpha_t = exp(log_alpha_t) in (0, 1]^{d_k}
 *
 * Closed form and operator order: "GLM-5.3-Flash Architecture Mastery",
 * course index, Course Outcomes; Module 11 — Correctness as Architecture
 * Mastery, §2 "The full correctness matrix", KDA row.  Two entry points, one
 * per request phase (Module 04 — KDA II: Chunked Parallelism & the Full
 * Sublayer, §2 "Why decode and prefill need different kernels"):
 *
 *   kda_prefill_chunked  many tokens per sequence; chunk-parallel: every
 *                        chunk's composed transition is built independently
 *                        in structured (diagonal + low-rank) form, then the
 *                        chunks are applied in order (Module 04, §1 "The
 *                        recurrence has affine form").
 *   kda_decode_step      one token per sequence, fused recurrent step, the
 *                        state updated in place.
 *   kda_decode           m >= 1 tokens per sequence in one launch (multi-token
 *                        decode / speculative verification), the state read
 *                        once and written once, optionally the state after
 *                        every token for rollback (Module 11, §2 "The full
 *                        correctness matrix", row "Serving state").
 *
 *   kda_short_conv       the short causal convolution that precedes the
 *                        recurrence in the sublayer, with its rolling state.
 *   kda_backward         gradients of the recurrence (reverse mode through the
 *                        chunked form, from the prefill's chunk checkpoints).
 *   kda_short_conv_backward  gradients of the short convolution.
 *   kda_ssm_prefill, kda_ssm_decode, kda_ssm_backward  the selective state
 *                        space scan for prompts, for a few tokens, and its
 *                        gradients.
 *   kda_block_norm, kda_block_norm_backward  the norm after a block with its
 *                        gate, the scaled residual and the norm before the
 *                        next block, and their gradients.
 *
 * Both recurrence families can fuse the stages that run just before the
 * recurrence (KDA_PROLOGUE_* flags below).
 *
 * Conventions common to all entry points
 *   - Pointers marked DEVICE are device memory owned by the caller; the
 *     library never allocates, frees or synchronises.  Scratch memory for
 *     prefill is a caller-provided workspace sized by
 *     kda_prefill_workspace_bytes(), or, for kda_prefill_chunked_noalloc, a
 *     fixed array the library's code holds on each GPU.
 *   - Tensors are contiguous, row-major, with the layouts given below, except
 *     where a stride argument is named.
 *   - Every argument is validated on the host before the first launch; on an
 *     error nothing is launched and nothing is written.  After the launches
 *     a launch failure maps to KDA_ERR_HIP.  Execution is asynchronous on
 *     the given stream (a hipStream_t passed as void*; NULL = default).
 *   - No query scale is applied: callers pre-scale q.
 *   - log_alpha must be <= 0 and all inputs finite; other values are not
 *     checked and propagate (NaN in, NaN out).
 *   - Apart from the fixed scratch of kda_prefill_chunked_noalloc, the
 *     library holds no mutable global state: concurrent calls on different
 *     streams with disjoint outputs and workspaces are safe.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 3

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL_ARG = 1,           /* a required pointer is NULL                 */
    KDA_ERR_BAD_SHAPE = 2,          /* sizes inconsistent or out of range         */
    KDA_ERR_UNSUPPORTED = 3,        /* valid but not implemented (dtype, d, C)    */
    KDA_ERR_WORKSPACE_TOO_SMALL = 4,
    KDA_ERR_HIP = 5,                /* a HIP launch failed                        */
    KDA_ERR_BAD_SEQLENS = 6,        /* host-visible cu_seqlens are malformed      */
    KDA_ERR_SCRATCH_LIMIT = 7,      /* needs more than the fixed scratch of
                                       kda_prefill_chunked_noalloc             */
    KDA_ERR_DEVICE_WAIT = 8         /* device-side only (*device_status): a
                                       hand-off between workgroups of the
                                       overlapped prefill failed; the call's
                                       results are undefined                  */
} kda_status;

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/*
 * Prologue flags (the `prologue` field of the argument structs).  The
 * executed sublayer runs Q/K normalisation, a learned decay gate producing
 * alpha and a learned write gate producing beta just before the recurrence
 * (Module 04 — KDA II, §3 "The sublayer is bigger than the recurrence");
 * each flag fuses one of them into the kernels, so that the argument holds
 * the pre-activation x instead of the value:
 *   GATE_SOFTPLUS  log_alpha holds x; the kernels use log alpha = -softplus(x)
 *                  = -log(1 + e^x) (alpha = 1 / (1 + e^x)), computed in fp32.
 *   BETA_SIGMOID   beta holds x; beta = 1 / (1 + e^-x).
 *   QK_L2NORM      q and k are divided by sqrt(sum_c x_c^2 + 1e-6) over their
 *                  d_k channels, per (token, head), in fp32 (the inputs are
 *                  not rounded again after the division).
 * The pages name the stages without formulas; these are the forms the
 * workload descriptions apply to their inputs.  Unknown bits are
 * KDA_ERR_UNSUPPORTED.
 */
#define KDA_PROLOGUE_GATE_SOFTPLUS 1u
#define KDA_PROLOGUE_BETA_SIGMOID 2u
#define KDA_PROLOGUE_QK_L2NORM 4u
#define KDA_PROLOGUE_ALL 7u

/*
 * Prefill arguments.  Sequences are either the B rows of a batch
 * (cu_seqlens == NULL, num_seqs == B) or documents packed along T
 * (B == 1, cu_seqlens != NULL, num_seqs == len(cu_seqlens) - 1); documents
 * never share state (Module 11, §2, row "Padding / packing").
 *
 *   q, k        DEVICE [B, T, H, d_k]  in_dtype
 *   v           DEVICE [B, T, H, d_v]  in_dtype
 *   beta        DEVICE [B, T, H]       in_dtype, expected in [0, 1]
 *   log_alpha   DEVICE [B, T, H, d_k]  in_dtype, <= 0
 *   cu_seqlens  DEVICE int32 [num_seqs + 1]: 0 = cu[0] <= cu[1] <= ... <=
 *               cu[num_seqs] = T.  Checked on the device before any other
 *               kernel reads it: if malformed, no kernel writes o or any
 *               state and *device_status (if given) is set to
 *               KDA_ERR_BAD_SEQLENS.
 *   cu_seqlens_host  HOST, optional copy of cu_seqlens; when given it is
 *               validated on the host as well (KDA_ERR_BAD_SEQLENS).
 *   initial_state DEVICE fp32 [num_seqs, H, d_k, d_v], NULL = zeros.
 *   final_state DEVICE fp32 [num_seqs, H, d_k, d_v], NULL = not written.
 *               May alias initial_state (in-place continuation).
 *   chunk_states DEVICE fp32, NULL = not written: the state ENTERING every
 *               chunk, documents in order, [sum_n ceil(len_n / C), H, d_k, d_v]
 *               (the chunk-boundary states of Module 04, §4 "The correctness
 *               invariant").  Its size is bounded by
 *               kda_prefill_max_chunks() * H * d_k * d_v floats.
 *   o           DEVICE [B, T, H, d_v]  out_dtype (fp32 recommended: a bf16
 *               output alone costs ~2^-9 relative per element).
 *   device_status DEVICE int32, NULL = not reported; written 0 or an error.
 *   workspace   DEVICE, >= kda_prefill_workspace_bytes(args), 256-byte aligned.
 *   timing_events  HOST, nullable: pointer to 3 hipEvent_t created by the
 *               caller; recorded on hip_stream before the first kernel
 *               (the chunk table), between the per-chunk kernel and the scan
 *               kernel (after the single kernel on the fp32 vector-ALU path)
 *               and after the last kernel.  A profiling hook; costs nothing
 *               when NULL.
 *   prologue    KDA_PROLOGUE_* bits, 0 = q, k, beta, log_alpha used as given.
 *
 * Supported: d_k, d_v in {16, 32, 64, 128}; chunk_size in {16, 32, 64};
 * in_dtype f32 or bf16; out_dtype f32 or bf16.  Paths (all with fp32 state
 * and accumulation): bf16 inputs with d_k == d_v in {64, 128} run on bf16
 * matrix cores, reading q, k, v and log_alpha as 128-bit vectors (each
 * must be 16-byte aligned there, else KDA_ERR_UNSUPPORTED); every other
 * case (fp32 inputs for the 1e-5 contract, other
 * bf16 head sizes) runs on the fp32 matrix cores, with a workspace of about
 * 209 KB (d_k = 128) per (chunk, head) whatever the chunk size
 * (chunk_size 16 only while that stays within 4 GiB); larger chunk-16 calls
 * run in fp32 on the vector ALUs.
 *
 * On the bf16 matrix-core path, one sequence (num_seqs == 1) whose
 * inter-chunk scan needs at most 16 workgroups per XCD (ceil(H / 8) *
 * d_v / 16 <= 16) with chunk_size 64 runs, on a device with 256 CUs, as one
 * launch in which the scan consumes each chunk's intermediate block as soon
 * as it is written (Module 04 — KDA II, §2: the per-chunk work is parallel,
 * only the composition across chunks is sequential).  fp32 inputs with
 * d_k = 128 on the fp32 matrix-core path (any chunk size) overlap the same
 * way when one sequence's scan needs at most 16 workgroups per XCD.
 * Results are bitwise those of the two-kernel launch, which
 * KDA_PREFILL_OVERLAP=0 in the environment forces.  Its cross-workgroup waits are bounded (1 s, or
 * KDA_PREFILL_WAIT_TICKS ticks of the device's 100 MHz real-time counter
 * from the environment, for tests of this path): a hand-off that does not
 * complete sets *device_status to KDA_ERR_DEVICE_WAIT, every kernel still
 * runs to its end, and the call's results are undefined.
 */
typedef struct kda_prefill_args {
    int32_t B, T, H, d_k, d_v;
    int32_t num_seqs;
    int32_t chunk_size;
    int32_t in_dtype;              /* kda_dtype */
    int32_t out_dtype;             /* kda_dtype */
    const void *q, *k, *v, *beta, *log_alpha;
    const int32_t *cu_seqlens;
    const int32_t *cu_seqlens_host;
    const float *initial_state;
    float *final_state;
    float *chunk_states;
    void *o;
    int32_t *device_status;
    void *workspace;
    size_t workspace_bytes;
    void *timing_events;
    uint32_t prologue;
} kda_prefill_args;

/* Workspace bytes the call described by *a needs (0 if a is NULL or
 * invalid).  Pure host function; depends only on sizes and dtypes. */
size_t kda_prefill_workspace_bytes(const kda_prefill_args *a);

/* Upper bound on sum_n ceil(len_n / C): ceil(T / C) + num_seqs for packed
 * input, B * ceil(T / C) otherwise.  Pure host function. */
int64_t kda_prefill_max_chunks(const kda_prefill_args *a);

/* Chunked prefill over all sequences and heads.  Returns KDA_OK once the
 * kernels are enqueued on hip_stream. */
kda_status kda_prefill_chunked(const kda_prefill_args *a, void *hip_stream);

/*
 * Allocation-free variant of kda_prefill_chunked, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  Same operation, arguments, validation
 * and results as kda_prefill_chunked, except that the scratch comes from a
 * fixed device array inside the library instead of a->workspace (which is
 * ignored, with a->workspace_bytes):
 *   - the array holds KDA_NOALLOC_SCRATCH_BYTES on every GPU the library runs
 *     on, from the load of the library's code on that GPU until the process
 *     ends; its device address is looked up once per GPU, on the first call
 *     for that GPU (the GPU owning hip_stream, or the current one for NULL);
 *   - a call whose scratch need (kda_prefill_workspace_bytes) exceeds it
 *     returns KDA_ERR_SCRATCH_LIMIT before anything is launched;
 *   - nothing is allocated or freed (no hipMalloc, hipFree or allocating
 *     library routine);
 *   - every call on one GPU shares that GPU's array and finds the previous
 *     call's contents there (each call rewrites all it reads): calls that
 *     overlap in time on one GPU (on different streams, or from threads
 *     without ordering) race and give undefined results; calls ordered on
 *     one stream are safe.
 * The caller still provides every input and output buffer.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (256u << 20)
kda_status kda_prefill_chunked_noalloc(const kda_prefill_args *a, void *hip_stream);

/*
 * One decode step for B independent sequences (one token each), fused:
 * the state is read once and written once per (sequence, head)
 * (Module 04, §2: decode uses a fused recurrent kernel).
 *
 *   q, k, log_alpha  DEVICE [B, H, d_k]  in_dtype
 *   v                DEVICE [B, H, d_v]  in_dtype
 *   beta             DEVICE [B, H]       in_dtype
 *   state            DEVICE fp32 [B, H, d_k, d_v], updated in place
 *   o                DEVICE [B, H, d_v]  out_dtype
 * Supported: d_k, d_v in {16, 32, 64, 128}; dtypes as for prefill.
 */
kda_status kda_decode_step(int32_t B, int32_t H, int32_t d_k, int32_t d_v,
                           int32_t in_dtype, int32_t out_dtype,
                           const void *q, const void *k, const void *v,
                           const void *beta, const void *log_alpha,
                           float *state, void *o, void *hip_stream);

/*
 * m >= 1 consecutive tokens for each of B independent sequences in one
 * launch: multi-token decode and speculative verification, where a rejected
 * suffix must be rolled back to the state after the last accepted token
 * (Module 11, §2 "The full correctness matrix", row "Serving state"; the
 * course index's module list, Module 08 "Vision, MTP, and Hybrid Serving
 * State", on why a rollback must restore the recurrent state).
 * Per (sequence, head) the state is read once, the m tokens are applied in
 * registers, and the results are written once.  With 2 <= m <= 4 and no
 * token_states the m tokens are applied in the chunked form of the
 * recurrence (Module 04 — KDA II, §1 "The recurrence has affine form"): one
 * pass of reductions over the state and a rank-m update, equal to applying
 * them one by one up to fp32 rounding; otherwise token by token with the
 * same fused step as kda_decode_step.
 *
 *   q, k, log_alpha  DEVICE [B, m, H, d_k]  in_dtype
 *   v                DEVICE [B, m, H, d_v]  in_dtype
 *   beta             DEVICE [B, m, H]       in_dtype
 *   initial_state    DEVICE fp32 [B, H, d_k, d_v]: the state before token 0.
 *   final_state      DEVICE fp32 [B, H, d_k, d_v], NULL = not written: the
 *                    state after token m - 1.  May alias initial_state (in
 *                    place); leave it NULL to keep initial_state for a
 *                    rollback to zero accepted tokens.
 *   token_states     DEVICE fp32 [B, m, H, d_k, d_v], NULL = not written:
 *                    the state after every token (m x the state traffic).
 *   o                DEVICE [B, m, H, d_v]  out_dtype; o[b, j] uses the
 *                    state after token j.
 *   prologue         KDA_PROLOGUE_* bits.
 * Supported: d_k, d_v in {16, 32, 64, 128}; 1 <= m; B * m * H < 2^31; the
 * three state pointers 16-byte aligned (the kernel moves state rows as
 * 128-bit vectors), else KDA_ERR_UNSUPPORTED.
 */
typedef struct kda_decode_args {
    int32_t B, H, d_k, d_v;
    int32_t n_tokens;
    int32_t in_dtype;              /* kda_dtype */
    int32_t out_dtype;             /* kda_dtype */
    uint32_t prologue;
    const void *q, *k, *v, *beta, *log_alpha;
    const float *initial_state;
    float *final_state;
    float *token_states;
    void *o;
} kda_decode_args;

kda_status kda_decode(const kda_decode_args *a, void *hip_stream);

/*
 * Short causal convolution with a rolling state: the small local mixing step
 * the executed sublayer applies to q, k and/or v before the recurrence
 * (Module 04 — KDA II, §3 "The sublayer is bigger than the recurrence").
 * Its state, the last W - 1 inputs of each sequence, is serving state that a
 * rollback restores (Module 11, §2, row "Serving state").  The pages give
 * neither its width nor its form; this is a depthwise causal filter:
 *
 *     y_t[c] = sum_{j=0}^{W-1} weight[c][j] * x_{t-W+1+j}[c]  (+ bias[c]),
 *     then y * sigmoid(y) if activation == KDA_CONV_SILU,
 *
 * taps ordered oldest input first; inputs before a sequence's first token
 * come from its initial state (zeros when NULL).  Prefill passes whole
 * sequences; decode passes B rows of m tokens with the state updated in
 * place (final_state == initial_state).
 *
 *   x             DEVICE [B, T, C]  in_dtype (C = channels, e.g. H * d)
 *   weight        DEVICE fp32 [C, W]
 *   bias          DEVICE fp32 [C], NULL = none
 *   cu_seqlens    DEVICE int32 [num_seqs + 1], NULL = the B rows are the
 *                 sequences; else B == 1 and documents are packed along T
 *                 (offsets are not validated: malformed offsets give
 *                 unspecified values, never an out-of-range access)
 *   initial_state DEVICE fp32 [num_seqs, C, W - 1], oldest input first,
 *                 NULL = zeros
 *   final_state   DEVICE fp32 [num_seqs, C, W - 1], NULL = not written: the
 *                 last W - 1 inputs of each sequence (from its initial state
 *                 where the sequence is shorter).  May alias initial_state.
 *   y             DEVICE [B, T, C]  out_dtype
 * Supported: 1 <= W <= 8; C a positive multiple of 8; B * T * C < 2^31;
 * x, y and the states 16-byte aligned.
 */
#define KDA_CONV_NONE 0
#define KDA_CONV_SILU 1
typedef struct kda_conv_args {
    int32_t B, T, C, W;
    int32_t num_seqs;
    int32_t in_dtype;              /* kda_dtype */
    int32_t out_dtype;             /* kda_dtype */
    int32_t activation;            /* KDA_CONV_NONE or KDA_CONV_SILU */
    const void *x;
    const float *weight;
    const float *bias;
    const int32_t *cu_seqlens;
    const float *initial_state;
    float *final_state;
    void *y;
} kda_conv_args;

kda_status kda_short_conv(const kda_conv_args *a, void *hip_stream);

/*
 * Backward pass: gradients of q, k, v, beta, log_alpha and the initial state
 * from the gradients of o and of the final state.  The pages call the affine
 * composition the argument for parallel training (course index, module
 * list, the Module 04 entry) but derive no backward; this is reverse-mode
 * differentiation, in fp32, of the chunked form (bf16 inputs: every chunk's
 * gradients from its structured matrices, the chunks coupled by a reverse
 * scan of the state gradient) or of the token operations (fp32 inputs, last
 * token first, states recomputed token by token).  Both start from
 * checkpoints: the state entering every chunk of chunk_size tokens, exactly
 * what kda_prefill_chunked writes to chunk_states when called with that
 * chunk_size on the same inputs and initial state.
 *
 *   chunk_size   the checkpoint spacing: 16, 32 or 64 for bf16 inputs (64
 *                recommended), 16 for fp32 inputs.
 *
 *   q, k, v, beta, log_alpha, cu_seqlens, B, T, H, d_k, d_v, num_seqs,
 *   in_dtype     as for kda_prefill_chunked (no prologue: the gradients are
 *                with respect to the recurrence's own inputs)
 *   checkpoints  DEVICE fp32 [sum_n ceil(len_n / chunk_size), H, d_k, d_v]
 *   d_o          DEVICE fp32 [B, T, H, d_v]
 *   d_final_state DEVICE fp32 [num_seqs, H, d_k, d_v], NULL = zeros
 *   dq, dk, dlog_alpha  DEVICE fp32 [B, T, H, d_k]    (written)
 *   dv           DEVICE fp32 [B, T, H, d_v]            (written)
 *   dbeta        DEVICE fp32 [B, T, H]                 (written)
 *   d_initial_state DEVICE fp32 [num_seqs, H, d_k, d_v], NULL = not written
 *   workspace    DEVICE, >= kda_backward_workspace_bytes(args), 256-aligned
 * With fp32 inputs dq, dk, dlog_alpha and dbeta are sums over the state's
 * column tiles taken with fp32 atomics: their rounding may differ from run to
 * run; the bf16 path is deterministic.
 * Supported: d_k, d_v in {16, 32, 64, 128}; in_dtype f32 or bf16; with bf16
 * inputs checkpoints and d_o must be 16-byte aligned (KDA_ERR_UNSUPPORTED
 * otherwise).
 * The first int32 word of the workspace holds the call's device status once
 * it has run (0, or KDA_ERR_BAD_SEQLENS for malformed cu_seqlens).
 */
typedef struct kda_backward_args {
    int32_t B, T, H, d_k, d_v;
    int32_t num_seqs;
    int32_t in_dtype;              /* kda_dtype */
    int32_t chunk_size;            /* checkpoint spacing */
    const void *q, *k, *v, *beta, *log_alpha;
    const int32_t *cu_seqlens;
    const float *checkpoints;
    const float *d_o;
    const float *d_final_state;
    float *dq, *dk, *dv, *dbeta, *dlog_alpha;
    float *d_initial_state;
    void *workspace;
    size_t workspace_bytes;
} kda_backward_args;

size_t kda_backward_workspace_bytes(const kda_backward_args *a);
kda_status kda_backward(const kda_backward_args *a, void *hip_stream);

/*
 * Selective state space scan: the other recurrence a hybrid model's sublayer
 * runs behind the same short convolution.  Per sequence and head h of group
 * g = h / (H / G), with state S [d_state, d_head] in fp32:
 *
 *     dt_t = dt[t, h] (+ dt_bias[h]), then log(1 + e^dt) with dt_softplus
 *     a_t  = exp(A[h] dt_t)
 *     S_t  = a_t S_{t-1} + dt_t B_t x_t^T ,   y_t = S_t^T C_t (+ D[h] x_t)
 *
 * A step of 0 leaves the state as it is; with dt_softplus a dt of the type's
 * lowest value or -infinity is such a step (x, B and C finite there: a NaN or
 * an infinity may reach all of its own sequence's chunk).
 *
 * x, B and C may be slices of one wider tensor (the convolution's output):
 * their token and batch strides are given in elements, the last two axes are
 * contiguous.
 *
 *   x            DEVICE [B, T, H, d_head]   in_dtype, strides x_stride_*
 *   Bm, Cm       DEVICE [B, T, G, d_state]  in_dtype, strides b_/c_stride_*
 *   dt           DEVICE [B, T, H]           in_dtype, contiguous
 *   A            DEVICE fp32 [H], <= 0, as every dt_t is >= 0 (not checked)
 *   D, dt_bias   DEVICE fp32 [H], NULL = none
 *   cu_seqlens   DEVICE int32 [num_seqs + 1], NULL = the B rows are the
 *                sequences; else B == 1 and documents are packed along T.
 *                Checked on the device before any other kernel reads it: if
 *                malformed, no kernel writes y or any state and
 *                *device_status (if given) is KDA_ERR_BAD_SEQLENS.
 *   initial_state DEVICE fp32 [num_seqs, H, d_state, d_head], NULL = zeros
 *   final_state  DEVICE fp32, same shape, NULL = not written; may alias
 *                initial_state
 *   chunk_states DEVICE fp32, NULL = not written: the state entering every
 *                chunk of KDA_SSM_CHUNK tokens, documents in order,
 *                [sum_n ceil(len_n / KDA_SSM_CHUNK), H, d_state, d_head]
 *   y            DEVICE [B, T, H, d_head]   out_dtype, contiguous
 *   device_status DEVICE int32, NULL = not reported; written 0 or an error
 *   workspace    DEVICE, >= kda_ssm_workspace_bytes(args), 256-byte aligned
 *
 * Supported: d_head, d_state in {16, 32, 64, 128}; G divides H; in_dtype and
 * out_dtype f32 or bf16; B * T * H < 2^31; strides multiples of 8, token strides
 * and H * d_head below 2^23;
 * x, Bm, Cm 16-byte aligned, the states too (else KDA_ERR_UNSUPPORTED).
 */
#define KDA_SSM_CHUNK 64
typedef struct kda_ssm_args {
    int32_t B, T, H, G, d_head, d_state;
    int32_t num_seqs;
    int32_t in_dtype;              /* kda_dtype */
    int32_t out_dtype;             /* kda_dtype */
    int32_t dt_softplus;           /* 0 or 1 */
    int64_t x_stride_b, x_stride_t;
    int64_t b_stride_b, b_stride_t;
    int64_t c_stride_b, c_stride_t;
    const void *x, *dt, *Bm, *Cm;
    const float *A, *D, *dt_bias;
    const int32_t *cu_seqlens;
    const float *initial_state;
    float *final_state;
    float *chunk_states;
    void *y;
    int32_t *device_status;
    void *workspace;
    size_t workspace_bytes;
} kda_ssm_args;

/* Workspace bytes the call needs (0 if a is NULL or invalid); upper bound of
 * the rows of chunk_states.  Pure host functions. */
size_t kda_ssm_workspace_bytes(const kda_ssm_args *a);
int64_t kda_ssm_max_chunks(const kda_ssm_args *a);
kda_status kda_ssm_prefill(const kda_ssm_args *a, void *hip_stream);

/*
 * m >= 1 consecutive tokens of the scan for each of B sequences in one
 * launch; the state is read once and written once.  Layouts as above with
 * T = n_tokens (x and y [B, m, H, d_head], Bm and Cm [B, m, G, d_state],
 * dt [B, m, H]).
 *   initial_state DEVICE fp32 [B, H, d_state, d_head]: the state before
 *   final_state   DEVICE fp32, same shape, NULL = not written; may alias
 *                 initial_state
 *   token_states  DEVICE fp32 [B, m, H, d_state, d_head], NULL = not written:
 *                 the state after every token (a rollback restores one)
 */
typedef struct kda_ssm_decode_args {
    int32_t B, H, G, d_head, d_state;
    int32_t n_tokens;
    int32_t in_dtype;              /* kda_dtype */
    int32_t out_dtype;             /* kda_dtype */
    int32_t dt_softplus;           /* 0 or 1 */
    int64_t x_stride_b, x_stride_t;
    int64_t b_stride_b, b_stride_t;
    int64_t c_stride_b, c_stride_t;
    const void *x, *dt, *Bm, *Cm;
    const float *A, *D, *dt_bias;
    const float *initial_state;
    float *final_state;
    float *token_states;
    void *y;
} kda_ssm_decode_args;
kda_status kda_ssm_decode(const kda_ssm_decode_args *a, void *hip_stream);

/*
 * Gradients of the scan: of x, dt (as given: through the softplus and the
 * bias), A, B, C, D, dt_bias and the initial state, from the gradients of y
 * and of the final state.
 *   x .. cu_seqlens  as for kda_ssm_prefill
 *   d_y           DEVICE [B, T, H, d_head] in_dtype, contiguous
 *   d_final_state DEVICE fp32 [num_seqs, H, d_state, d_head], NULL = zeros
 *   dx, ddt, dB, dC  DEVICE, shapes of x, dt, Bm, Cm, contiguous, in_dtype
 *   dA            DEVICE fp32 [H];  dD, ddt_bias DEVICE fp32 [H], NULL = not
 *                 written
 *   d_initial_state DEVICE fp32 [num_seqs, H, d_state, d_head], NULL = not
 *                 written
 *   workspace     DEVICE, >= kda_ssm_backward_workspace_bytes(args), 256-byte
 *                 aligned; its first int32 word holds the call's device
 *                 status once it has run
 * The states entering the chunks are recomputed from initial_state in the
 * workspace, whose size is about 2 fp32 states per 64 tokens (32 with fp32
 * inputs) and head.  With malformed cu_seqlens nothing is written.  Results
 * are the same from run to run (no floating-point atomics).
 */
typedef struct kda_ssm_backward_args {
    int32_t B, T, H, G, d_head, d_state;
    int32_t num_seqs;
    int32_t in_dtype;              /* kda_dtype */
    int32_t dt_softplus;           /* 0 or 1 */
    int64_t x_stride_b, x_stride_t;
    int64_t b_stride_b, b_stride_t;
    int64_t c_stride_b, c_stride_t;
    const void *x, *dt, *Bm, *Cm;
    const float *A, *D, *dt_bias;
    const int32_t *cu_seqlens;
    const float *initial_state;
    const void *d_y;
    const float *d_final_state;
    void *dx, *ddt, *dB, *dC;
    float *dA, *dD, *ddt_bias;
    float *d_initial_state;
    void *workspace;
    size_t workspace_bytes;
} kda_ssm_backward_args;
size_t kda_ssm_backward_workspace_bytes(const kda_ssm_backward_args *a);
kda_status kda_ssm_backward(const kda_ssm_backward_args *a, void *hip_stream);

/*
 * Gradients of kda_short_conv: of x, the weight, the bias and the initial
 * state, from the gradients of y and of the final state.
 *   x .. initial_state  as for kda_short_conv
 *   d_y           DEVICE [B, T, C] grad_dtype
 *   d_final_state DEVICE fp32 [num_seqs, C, W - 1], NULL = zeros
 *   dx            DEVICE [B, T, C] in_dtype
 *   dweight       DEVICE fp32 [C, W];  dbias DEVICE fp32 [C], NULL = not written
 *   d_initial_state DEVICE fp32 [num_seqs, C, W - 1], NULL = not written
 *   workspace     DEVICE, >= kda_short_conv_backward_workspace_bytes(args),
 *                 256-byte aligned
 * Supported sizes, alignment and the treatment of malformed offsets as for
 * kda_short_conv.  Results are the same from run to run.
 */
typedef struct kda_conv_backward_args {
    int32_t B, T, C, W;
    int32_t num_seqs;
    int32_t in_dtype;              /* kda_dtype */
    int32_t grad_dtype;            /* kda_dtype */
    int32_t activation;            /* KDA_CONV_NONE or KDA_CONV_SILU */
    const void *x;
    const float *weight;
    const float *bias;
    const int32_t *cu_seqlens;
    const float *initial_state;
    const void *d_y;
    const float *d_final_state;
    void *dx;
    float *dweight;
    float *dbias;
    float *d_initial_state;
    void *workspace;
    size_t workspace_bytes;
} kda_conv_backward_args;
size_t kda_short_conv_backward_workspace_bytes(const kda_conv_backward_args *a);
kda_status kda_short_conv_backward(const kda_conv_backward_args *a, void *hip_stream);

/*
 * The stages after a block and before the next one in a single pass over the
 * rows: the norm of the block's output with its gate (the sublayer's gated
 * output norm), the scaled residual, and the norm in front of the next block
 * (Module 04 — KDA II, §3 "The sublayer is bigger than the recurrence").
 * Per row of dim channels, rms(v) = v / sqrt(mean(v^2) + eps):
 *
 *     p      = rms_group(x) * post_weight   over groups of `group` channels
 *              (p = x when post_weight is NULL)
 *     p      = p * act(gate)                when gate is given; with gate_first
 *              the gate multiplies x before the norm instead
 *     out    = residual + scale * p         (residual NULL = none, scale NULL = 1)
 *     normed = rms(out) * pre_weight        when pre_weight is given; from out
 *              before its rounding to dtype
 *
 *   x, gate, residual  DEVICE [rows, dim] dtype, row strides *_stride in
 *                elements (channels contiguous); gate, residual nullable
 *   post_weight  DEVICE fp32 [group] (post_per_channel 0: shared by the groups)
 *                or [dim] (post_per_channel 1), NULL = no norm after the block
 *   scale        DEVICE fp32 [dim], NULL = 1
 *   pre_weight   DEVICE fp32 [dim], NULL = no second norm
 *   out          DEVICE [rows, dim] dtype, contiguous
 *   normed       DEVICE [rows, dim] dtype, contiguous; required with
 *                pre_weight, NULL without
 * out and normed may each be an input's own rows (contiguous); any other
 * overlap, of each other or of part of an input, is refused
 * (KDA_ERR_BAD_SHAPE).
 * Supported: 1 <= dim <= 16384, group divides dim, rows * dim < 2^40.  Rows
 * whose sizes, strides and addresses are multiples of 8 channels and 16 bytes
 * are moved as 128-bit vectors; any other row element by element.
 */
#define KDA_GATE_SIGMOID 0
#define KDA_GATE_SILU 1
typedef struct kda_block_norm_args {
    int64_t rows;
    int32_t dim, group;
    int32_t dtype;                 /* kda_dtype */
    int32_t gate_activation;       /* KDA_GATE_* */
    int32_t gate_first;            /* 0 or 1 */
    int32_t post_per_channel;      /* 0 or 1 */
    float eps;
    int64_t x_stride, gate_stride, residual_stride;
    const void *x, *gate, *residual;
    const float *post_weight, *scale, *pre_weight;
    void *out, *normed;
} kda_block_norm_args;
kda_status kda_block_norm(const kda_block_norm_args *a, void *hip_stream);

/*
 * Gradients of kda_block_norm with respect to everything it reads, from the
 * gradients of out and of normed; the forward's values are recomputed from
 * its inputs.
 *   f            the forward's arguments (out and normed are not read)
 *   d_out        DEVICE [rows, dim] dtype, contiguous, NULL = zeros
 *   d_normed     DEVICE [rows, dim] dtype, contiguous, NULL = zeros (needs
 *                f.pre_weight)
 *   dx           DEVICE [rows, dim] dtype, contiguous
 *   dgate, dresidual  DEVICE [rows, dim] dtype, contiguous, NULL = not written
 *   dpost_weight (shape of post_weight), dscale, dpre_weight [dim]  DEVICE
 *                fp32, NULL = not written
 *   workspace    DEVICE, >= kda_block_norm_backward_workspace_bytes(args),
 *                256-byte aligned
 * A gradient whose input is not given is refused (KDA_ERR_BAD_SHAPE).
 * Results are the same from run to run.
 */
typedef struct kda_block_norm_backward_args {
    kda_block_norm_args f;
    const void *d_out, *d_normed;
    void *dx, *dgate, *dresidual;
    float *dpost_weight, *dscale, *dpre_weight;
    void *workspace;
    size_t workspace_bytes;
} kda_block_norm_backward_args;
size_t kda_block_norm_backward_workspace_bytes(const kda_block_norm_backward_args *a);
kda_status kda_block_norm_backward(const kda_block_norm_backward_args *a, void *hip_stream);

/* Static description of a status code (never NULL). */
const char *kda_status_string(int32_t status);

/* KDA_ABI_VERSION of the loaded library. */
int32_t kda_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KDA_H */
