/*
 * libgdr — gated delta rule kernels for AMD Instinct MI355X (gfx950).
 *
 * The operation (Gated Delta Rule-2; Gated DeltaNet-2 Q&A page "Gated
 * DeltaNet-2 — decoupling erase and write in linear attention", Q3, and
 * "Gated DeltaNet-2 Review" §3-1), per independent (batch, head) pair:
 *
 *     S_t = (I - k_t (b_t ⊙ k_t)^T) D_t S_{t-1} + k_t (w_t ⊙ v_t)^T
 *     D_t = diag(alpha_t),  alpha_t = exp(log_alpha_t)
 *     o_t = S_t^T q_t                  (read-out after the write; "Gated
 *                                       DeltaNet" explainer, mechanism)
 *
 * S_t is d_k x d_v.  b_t in R^{d_k} is the key-side erase gate, w_t in
 * R^{d_v} the value-side write gate.  Tying b = w = beta·1 gives KDA; also
 * making D_t = alpha_t·I gives Gated DeltaNet (Q&A page Q3).  Gates are
 * neither clamped nor assumed to lie in [0,1]; the expanded erase range
 * [0,2] ("Gated DeltaNet-2 Review" §5 ablation; sungsoo commentary, state
 * tracking) works unchanged.  No query scaling and no normalisation of q, k
 * is applied: that is the caller's job.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers owned by the caller.  The
 *   library never allocates device memory (scratch space is passed in as a
 *   caller-owned workspace), never frees caller memory, and keeps no state
 *   besides a lazily cached device-property record and, once the backward
 *   has run on a device, one extra stream and two events there (kept until
 *   the process ends).
 * - Execution is asynchronous on `stream` (a hipStream_t passed as void*;
 *   NULL is the default stream).  No call synchronises.
 * - Arguments are validated before any launch.  An invalid argument returns
 *   a status and launches nothing.  Launch failures return GDR_ERR_LAUNCH.
 *   No exception, abort or exit crosses the ABI.
 * - Layouts are contiguous row-major.  "act" is the activation dtype chosen
 *   by flags (bf16 bit patterns as uint16, or fp32).  Pointers must be
 *   16-byte aligned.
 * - Gate modes (flags): each of log_alpha, b, w is either per channel
 *   ([..., d_k] / [..., d_k] / [..., d_v]) or one scalar per token ([...]).
 *   Gated DeltaNet passes scalar log_alpha and the same scalar buffer as b
 *   and w; KDA passes channel log_alpha and one scalar buffer as b and w;
 *   the b-only / w-only ablations ("Gated DeltaNet-2 Review" §5 gate
 *   ablation) are mixed modes.
 * - Precision: with bf16 activations the dense chunk contractions run on
 *   MFMA with f16 operands and fp32 accumulation; the state, log-decay and
 *   the cumulative decay stay fp32 (the log-decay path runs in fp32:
 *   "Gated DeltaNet-2 Review" §3-2 item 2).  With fp32 activations every
 *   contraction runs on fp32 MFMA.  Erase gates up to 2 (the expanded range,
 *   "Gated DeltaNet-2 Review" §5) keep the bf16 accuracy for ordinary keys;
 *   one key repeated through a chunk with an erase gate near 2 makes the
 *   in-chunk solve cancel by about two orders of magnitude, and such inputs
 *   need fp32 activations.
 * - Decay range: every call returns values for any decay an fp32 log_alpha
 *   can express.  The forward with a workspace (fixed-length and packed)
 *   references each 16-token block's decay so that no operand factor leaves
 *   the f16 range.  The other chunk kernels reference a chunk's decay to its
 *   end; a (sequence, head) whose in-chunk decay leaves their operand range
 *   (about 10 nats per chunk with f16 operands) is recomputed token by token
 *   in fp32 by a follow-up kernel of the same call, which costs one small
 *   launch when no head needs it.  That recompute is sequential over a unit's
 *   tokens: a backward at B=1, H=32, T=16384, d=128 whose heads all leave the
 *   chunk-64 range takes about 240 ms instead of 2 ms.  Callers with such decay
 *   should pass chunk 16 to gdr_chunk_bwd (about 10 nats per 16 tokens stay in
 *   range; the same backward then takes about 13 ms).
 */
#ifndef GDR_H
#define GDR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdr_status {
    GDR_OK = 0,
    GDR_ERR_INVALID_ARG = 1,     /* null pointer, bad size, misalignment, T % chunk != 0 */
    GDR_ERR_UNSUPPORTED = 2,     /* a valid request the library has no kernel for     */
    GDR_ERR_WORKSPACE = 3,       /* workspace pointer NULL or smaller than required   */
    GDR_ERR_LAUNCH = 4,          /* the HIP runtime rejected a launch                 */
    GDR_ERR_DEVICE = 5           /* no usable gfx950 device / device query failed     */
} gdr_status;

/* flags (bitwise OR) */
#define GDR_ACT_BF16      0x0u   /* q, k, v, b, w, dO are bf16 (uint16 bit patterns)  */
#define GDR_ACT_F32       0x1u   /* q, k, v, b, w, dO are fp32                        */
#define GDR_OUT_BF16      0x2u   /* o is bf16 (default fp32).  Forward/decode only.   */
#define GDR_ALPHA_SCALAR  0x4u   /* log_alpha is one fp32 per token                   */
#define GDR_B_SCALAR      0x8u   /* b is one value per token                          */
#define GDR_W_SCALAR      0x10u  /* w is one value per token                          */
#define GDR_FWD_GENERIC   0x20u  /* forward: use the single-role kernel even where the
                                    pipelined one applies (same results up to rounding
                                    order; for testing)                               */
#define GDR_FWD_SPLIT     0x80u  /* forward with a workspace: run the chunk producer and
                                    the state chains as two kernels, one after the
                                    other, instead of one persistent kernel (same
                                    results bit for bit; for testing)               */
#define GDR_GATE_LOGITS   0x40u  /* log_alpha, b and w hold logits: the kernels use
                                    log alpha = log(sigmoid(log_alpha)), b = sigmoid(b),
                                    w = sigmoid(w) in fp32 (the token mixer's gating,
                                    fused into the loads), and the backward returns the
                                    gradients of the logits.  Two-pass forward and
                                    backward (workspace, bf16, chunk 64) and decode only;
                                    GDR_ERR_UNSUPPORTED elsewhere.                      */

/* flags of the attention layer's calls (gdr_rope, gdr_attn_*, gdr_kv_append) */
#define GDR_TOKEN_MAJOR      0x1000u /* tensors are [B, T, H, d] ([T, H, d] packed) instead
                                        of [B, H, T, d] ([H, T, d])                  */
#define GDR_ROPE_INTERLEAVED 0x2000u /* pairs of channels (2i, 2i + 1) instead of
                                        (i, i + rot_dim / 2)                         */
#define GDR_ROPE_INVERSE     0x4000u /* turn back: the transpose, which is the gradient  */

/* flag of gdr_beam_select */
#define GDR_KEEP_SLOTS       0x8000u /* a beam's first continuation stays in the beam's row */

#define GDR_ABI_VERSION 2

int gdr_abi_version(void);
const char* gdr_status_string(gdr_status s);

/*
 * Chunkwise-parallel forward (the WY form: in-chunk cumulative log-decay is
 * absorbed into the rank-one erase factor, giving an asymmetric delta
 * recurrence solved per chunk; Q&A page Q4, "Gated DeltaNet-2 Review"
 * §3-2 item 5).
 *
 *   q, k       : act  [B, H, T, d_k]
 *   v          : act  [B, H, T, d_v]
 *   log_alpha  : fp32 [B, H, T, d_k]   or [B, H, T] with GDR_ALPHA_SCALAR
 *   b          : act  [B, H, T, d_k]   or [B, H, T] with GDR_B_SCALAR
 *   w          : act  [B, H, T, d_v]   or [B, H, T] with GDR_W_SCALAR
 *   S0         : fp32 [B, H, d_k, d_v] initial state; NULL means zeros
 *   o          : fp32 (or bf16 with GDR_OUT_BF16) [B, H, T, d_v], written
 *   S_final    : fp32 [B, H, d_k, d_v], written; NULL means not written.
 *                May alias S0 (each workgroup reads its block of S0 before
 *                writing the same block).  No other aliasing is allowed.
 *   chunk      : 16, 32 or 64; T must be a multiple of chunk.  The chunk is
 *                a blocking choice: results equal the token recurrence up to
 *                rounding for every chunk size.
 *   workspace  : optional device scratch owned by the caller, contents on
 *                entry ignored.  When it is non-NULL and
 *                gdr_chunk_fwd_workspace_bytes() is non-zero for the call, a
 *                persistent kernel runs (one workgroup per compute unit, after
 *                a small kernel that clears the call's flags): producer
 *                workgroups compute every chunk's state-independent operands
 *                into the workspace while per-head state chains consume them,
 *                each chunk handed over through a flag.  A chain waits for a
 *                flag with a bounded spin (seconds); if the call's producers
 *                cannot become resident meanwhile (another kernel holding the
 *                compute units for that long), the chain stops and its head's
 *                o and S_final are NaN.  workspace_bytes below the required
 *                size returns GDR_ERR_WORKSPACE.  With a NULL workspace (or a
 *                zero requirement) a single fused kernel runs.  Both paths
 *                give the same result up to rounding.
 * Supported: d_k, d_v in {16, 32, 64, 128}; B*H >= 1; T >= 0 (T == 0 copies
 * S0 to S_final).  Returns GDR_ERR_UNSUPPORTED for other head sizes.
 */
size_t gdr_chunk_fwd_workspace_bytes(int B, int H, int T, int d_k, int d_v,
                                     int chunk, uint32_t flags);

gdr_status gdr_chunk_fwd(const void* q, const void* k, const void* v,
                         const float* log_alpha, const void* b, const void* w,
                         const float* S0, void* o, float* S_final,
                         int B, int H, int T, int d_k, int d_v, int chunk,
                         uint32_t flags, void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * gdr_chunk_fwd without a caller workspace and without any allocation, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).  Arguments and
 * results are those of gdr_chunk_fwd.  Where gdr_chunk_fwd would take a
 * workspace, this call uses a library-owned device array of
 * GDR_NOALLOC_SCRATCH_BYTES on the current GPU instead (each GPU the library
 * runs on holds its own copy until the process ends; it is looked up once per
 * device at the first call there).  A call whose
 * gdr_chunk_fwd_workspace_bytes() exceeds GDR_NOALLOC_SCRATCH_BYTES returns
 * GDR_ERR_WORKSPACE and launches nothing (at d_k = d_v = 128 the array holds
 * the operands of 900 chunks of 64 tokens, e.g. B*H = 16 heads of T = 3584).
 * Every call on one GPU shares that GPU's array: calls that overlap on one
 * GPU (different streams, or different host threads) race and must be
 * ordered by the caller.  The array's contents between calls are never read
 * before being written.
 */
#define GDR_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

gdr_status gdr_chunk_fwd_noalloc(const void* q, const void* k, const void* v,
                                 const float* log_alpha, const void* b, const void* w,
                                 const float* S0, void* o, float* S_final,
                                 int B, int H, int T, int d_k, int d_v, int chunk,
                                 uint32_t flags, void* stream);

/*
 * The same forward over packed variable-length sequences: nseq sequences of
 * any lengths stored back to back (variable-length batches are the practical
 * extension the pages point to: "Gated DeltaNet study notes" §4-3).  Each
 * sequence runs its own recurrence from its own initial state; no state
 * crosses from one sequence to the next.
 *
 *   q, k       : act  [H, T, d_k]   (T = total tokens of all sequences)
 *   v          : act  [H, T, d_v]
 *   log_alpha  : fp32 [H, T, d_k]   or [H, T] with GDR_ALPHA_SCALAR
 *   b          : act  [H, T, d_k]   or [H, T] with GDR_B_SCALAR
 *   w          : act  [H, T, d_v]   or [H, T] with GDR_W_SCALAR
 *   cu_seqlens : int32 [nseq + 1], DEVICE memory: sequence s is tokens
 *                cu_seqlens[s] .. cu_seqlens[s+1]-1 of every head.  The
 *                caller guarantees cu_seqlens[0] = 0, non-decreasing values
 *                and cu_seqlens[nseq] = T (the library cannot check values in
 *                device memory).  Lengths need not be multiples of 64; a
 *                length of 0 copies that sequence's S0 to S_final.
 *   S0         : fp32 [nseq, H, d_k, d_v]; NULL means zeros
 *   o          : as gdr_chunk_fwd, [H, T, d_v]
 *   S_final    : fp32 [nseq, H, d_k, d_v]; NULL means not written; may alias S0
 *   workspace  : required, at least gdr_chunk_fwd_varlen_workspace_bytes()
 *                bytes (chunks of 64: a record per chunk for the producer and
 *                chain kernels of gdr_chunk_fwd, then the chunk tables; the
 *                tokens past a sequence's end in its last chunk are treated as
 *                absent).
 * Supported: bf16 activations, d_k and d_v in {64, 128}; nseq >= 1, H >= 1,
 * T >= 0.  Returns GDR_ERR_UNSUPPORTED otherwise.
 */
size_t gdr_chunk_fwd_varlen_workspace_bytes(int nseq, int H, int T, int d_k, int d_v,
                                            uint32_t flags);

gdr_status gdr_chunk_fwd_varlen(const void* q, const void* k, const void* v,
                                const float* log_alpha, const void* b, const void* w,
                                const float* S0, void* o, float* S_final,
                                const int* cu_seqlens, int nseq, int H, int T,
                                int d_k, int d_v, uint32_t flags, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * One recurrent decode step for N independent sequences (constant memory:
 * the state is updated in place; Q&A page introduction, "Gated DeltaNet-2
 * Review" §3-2 item 1).  Each (n, h) state is read once and written once.
 *
 *   q, k       : act  [N, H, d_k]
 *   v          : act  [N, H, d_v]
 *   log_alpha  : fp32 [N, H, d_k] or [N, H] with GDR_ALPHA_SCALAR
 *   b          : act  [N, H, d_k] or [N, H] with GDR_B_SCALAR
 *   w          : act  [N, H, d_v] or [N, H] with GDR_W_SCALAR
 *   S          : fp32 [N, H, d_k, d_v], read and overwritten with S_t
 *   o          : fp32 (or bf16) [N, H, d_v], written
 * Supported: d_k, d_v in {16, 32, 64, 128}.  All arithmetic is fp32.
 */
gdr_status gdr_decode_step(const void* q, const void* k, const void* v,
                           const float* log_alpha, const void* b, const void* w,
                           float* S, void* o, int N, int H, int d_k, int d_v,
                           uint32_t flags, void* stream);

/*
 * Gate-aware backward of gdr_chunk_fwd for the loss
 *     L = <dO, o> + <dS_final, S_final>,
 * with the erase-side gate gradient (db) and the write-side one (dw)
 * accumulated separately (Q&A page Q4).
 *
 *   inputs as gdr_chunk_fwd, plus
 *   dO         : act  [B, H, T, d_v]
 *   dS_final   : fp32 [B, H, d_k, d_v]; NULL means zero
 *   outputs (fp32, written, never accumulated into):
 *   dq, dk     : [B, H, T, d_k]       dv : [B, H, T, d_v]
 *   dlog_alpha : [B, H, T, d_k] (or [B, H, T] in scalar mode: the sum over
 *                channels)
 *   db         : [B, H, T, d_k] (or [B, H, T])   dw : [B, H, T, d_v] (or [B, H, T])
 *                When b and w are the same scalar buffer (tied gates), the
 *                gradient of that buffer is db + dw.
 *   dS0        : [B, H, d_k, d_v]; may be NULL when not needed.
 *   workspace  : device scratch of at least gdr_chunk_bwd_workspace_bytes()
 *                bytes, owned by the caller; contents on entry are ignored.
 * Part of the work may run on the library's second stream for the device; it
 * waits for the work queued on `stream` before the call and `stream` waits for
 * it before the call's last kernel (event fork and join), so every effect is
 * ordered on `stream` as if it ran there, also under graph capture.  Calls on
 * one device share that second stream.
 * Supported: bf16 or fp32 activations, d_k and d_v each in {16, 32, 64,
 * 128}, chunk 16, 32 or 64 (fp32 activations block with at most 32; results
 * do not depend on the blocking beyond rounding).  Returns
 * GDR_ERR_UNSUPPORTED otherwise.  GDR_GATE_LOGITS needs bf16 activations,
 * chunk 64 and d_k = d_v in {64, 128}.
 */
size_t gdr_chunk_bwd_workspace_bytes(int B, int H, int T, int d_k, int d_v,
                                     int chunk, uint32_t flags);

gdr_status gdr_chunk_bwd(const void* q, const void* k, const void* v,
                         const float* log_alpha, const void* b, const void* w,
                         const float* S0, const void* dO, const float* dS_final,
                         float* dq, float* dk, float* dv, float* dlog_alpha,
                         float* db, float* dw, float* dS0,
                         int B, int H, int T, int d_k, int d_v, int chunk,
                         uint32_t flags, void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * The backward of gdr_chunk_fwd_varlen (packed variable-length sequences,
 * "Gated DeltaNet study notes" §4-3), for the same loss: every sequence's
 * gradients depend only on its own tokens, initial state and dS_final.
 *
 *   inputs as gdr_chunk_fwd_varlen ([H, T, ...] token streams, cu_seqlens in
 *   DEVICE memory with the same guarantees), plus
 *   dO         : act  [H, T, d_v]
 *   dS_final   : fp32 [nseq, H, d_k, d_v]; NULL means zero
 *   outputs (fp32, written, never accumulated into):
 *   dq, dk     : [H, T, d_k]       dv : [H, T, d_v]
 *   dlog_alpha, db, dw : [H, T, d_k] / [H, T, d_k] / [H, T, d_v], or [H, T]
 *                in the scalar modes (as gdr_chunk_bwd)
 *   dS0        : [nseq, H, d_k, d_v]; may be NULL.  A sequence of length 0
 *                gets dS0 = dS_final (zero when dS_final is NULL).
 *   workspace  : required, at least gdr_chunk_bwd_varlen_workspace_bytes()
 *                bytes, owned by the caller; contents on entry are ignored.
 * Uses the library's second stream as gdr_chunk_bwd does.
 * Supported: bf16 activations, d_k = d_v = 128 or 64 (chunks of 64).
 * Returns GDR_ERR_UNSUPPORTED otherwise.
 */
size_t gdr_chunk_bwd_varlen_workspace_bytes(int nseq, int H, int T, int d_k, int d_v,
                                            uint32_t flags);

gdr_status gdr_chunk_bwd_varlen(const void* q, const void* k, const void* v,
                                const float* log_alpha, const void* b, const void* w,
                                const float* S0, const void* dO, const float* dS_final,
                                float* dq, float* dk, float* dv, float* dlog_alpha,
                                float* db, float* dw, float* dS0,
                                const int* cu_seqlens, int nseq, int H, int T,
                                int d_k, int d_v, uint32_t flags, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * Token-mixer prologue: the element-wise and short-window steps between the
 * caller's linear projections and the recurrence ("Gated DeltaNet study
 * notes" §2 token mixer block design; "Gated DeltaNet-2 Review" §4-3
 * engineering notes), in one pass:
 *   q = L2norm(SiLU(conv(q_pre))),  k = L2norm(SiLU(conv(k_pre))),
 *   v = SiLU(conv(v_pre)),  log_alpha = log(sigmoid(a_pre)) in fp32,
 *   b = sigmoid(b_pre),  w = sigmoid(w_pre).
 * conv is the depthwise causal convolution with 4 taps per channel, zero
 * before the first token of each sequence; L2norm(x) = x / sqrt(sum x^2 +
 * 1e-6) over the head's d_k channels.  All arithmetic is fp32.
 *
 *   q_pre, k_pre : bf16 [B, H, T, d_k]   v_pre : bf16 [B, H, T, d_v]
 *   conv_q, conv_k : fp32 [H, d_k, 4]    conv_v : fp32 [H, d_v, 4]
 *                  taps of channel c of head h: element j weights token t - j
 *   a_pre  : fp32 [B, H, T, d_k] (or [B, H, T] with GDR_ALPHA_SCALAR)
 *   b_pre  : bf16 [B, H, T, d_k] (or [B, H, T] with GDR_B_SCALAR)
 *   w_pre  : bf16 [B, H, T, d_v] (or [B, H, T] with GDR_W_SCALAR)
 *   outputs, written: q, k, v bf16 in the shapes of q_pre, k_pre, v_pre;
 *   log_alpha fp32 shaped as a_pre; b, w bf16 shaped as b_pre, w_pre.  These
 *   are exactly the inputs gdr_chunk_fwd takes with the same gate flags.
 * Outputs must not alias inputs.  Flags: the three gate modes only.
 * Supported: d_k, d_v in {64, 128}; GDR_ERR_UNSUPPORTED otherwise (also for
 * GDR_ACT_F32).
 */
gdr_status gdr_mixer_prologue(const void* q_pre, const void* k_pre, const void* v_pre,
                              const float* conv_q, const float* conv_k, const float* conv_v,
                              const float* a_pre, const void* b_pre, const void* w_pre,
                              void* q, void* k, void* v, float* log_alpha, void* b, void* w,
                              int B, int H, int T, int d_k, int d_v, uint32_t flags,
                              void* stream);

/*
 * Token-mixer epilogue: the recurrent output RMS-normalised and gated before
 * the caller's output projection ("Gated DeltaNet-2 Review" §4-3), per
 * (token, head):
 *   y = o / sqrt(mean(o^2) + 1e-6) * norm_weight * SiLU(g)
 * with the mean over the head's d_v channels, in fp32.
 *
 *   o           : fp32 [B, H, T, d_v] (gdr_chunk_fwd's output)
 *   g           : bf16 [B, H, T, d_v] output-gate logits
 *   norm_weight : fp32 [d_v], shared by the heads
 *   y           : bf16 [B, H, T, d_v], written; must not alias o or g
 * flags must be 0.  Supported: d_v in {64, 128}.
 */
gdr_status gdr_mixer_epilogue(const float* o, const void* g, const float* norm_weight, void* y,
                              int B, int H, int T, int d_v, uint32_t flags, void* stream);

/*
 * Backward of the token-mixer prologue's q, k and v paths and of the
 * epilogue, for training through the block.  (With GDR_GATE_LOGITS the
 * recurrence's backward already returns the gate logits' gradients, so the
 * gate paths need nothing here.)
 *
 * gdr_mixer_prologue_bwd: given dq, dk, dv (fp32 [B, H, T, d], the gradients
 * of the prologue's outputs, e.g. from gdr_chunk_bwd), writes the gradients
 * of the projection outputs dq_pre, dk_pre, dv_pre (fp32, shaped as q_pre,
 * k_pre, v_pre) and of the convolution taps dconv_q, dconv_k, dconv_v (fp32
 * [H, d, 4], summed over the batch and the tokens in a fixed order, so the
 * result is deterministic).  The forward's values are recomputed from q_pre,
 * k_pre, v_pre and the taps.
 * gdr_mixer_epilogue_bwd: given dy (fp32 [B, H, T, d_v]), writes d_o and dg
 * (fp32 [B, H, T, d_v]) and dnorm_weight (fp32 [d_v], summed over all rows
 * in a fixed order).
 * Both need a workspace of gdr_mixer_bwd_workspace_bytes() bytes (one buffer
 * serves both calls on one stream); outputs must not alias inputs; flags
 * must be 0.  Supported: d_k = d_v in {64, 128}, T >= 1.
 */
size_t gdr_mixer_bwd_workspace_bytes(int B, int H, int T, int d_k, int d_v);

gdr_status gdr_mixer_prologue_bwd(const void* q_pre, const void* k_pre, const void* v_pre,
                                  const float* conv_q, const float* conv_k, const float* conv_v,
                                  const float* dq, const float* dk, const float* dv,
                                  float* dq_pre, float* dk_pre, float* dv_pre,
                                  float* dconv_q, float* dconv_k, float* dconv_v,
                                  int B, int H, int T, int d_k, int d_v, uint32_t flags,
                                  void* workspace, size_t workspace_bytes, void* stream);

gdr_status gdr_mixer_epilogue_bwd(const float* o, const void* g, const float* norm_weight,
                                  const float* dy, float* d_o, float* dg, float* dnorm_weight,
                                  int B, int H, int T, int d_v, uint32_t flags,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * The attention layer of a hybrid stack.  Stacks of the gated delta rule put
 * softmax attention layers between the recurrent ones, over a window of about
 * 2,048 tokens ("Q&A page" Q5, "Gated DeltaNet-2 Review" hybrid cell) or over
 * the whole past ("Gated DeltaNet explainer", three recurrent layers to one).
 * The calls below are such a layer between the caller's projections: rotary
 * positions, causal attention and its gradients for training and prompts, and
 * for generation an 8-bit paged cache with its one-token attention.
 *
 * All of them: queries have Hq heads, keys and values Hkv heads, Hq a multiple
 * of Hkv; query head h reads key head h / (Hq / Hkv).  Indexes and lengths in
 * device memory (positions, cu_seqlens, block_table, cache_len) are not checked
 * on the host; no content of them makes a kernel read or write outside the
 * tensors.  Results do not depend on the order in which workgroups run.  A call
 * whose largest launch would pass 2^24 - 1 workgroups (one for 128 queries of a
 * head, say) is refused with GDR_ERR_INVALID_ARG.
 */

/*
 * Rotary positions of queries and keys.  For channel pairs (a, b) of the first
 * rot_dim channels, i < rot_dim / 2, at position t of the row:
 *   theta = t * inv_freq[i],  y_a = scale (x_a cos theta - x_b sin theta),
 *                             y_b = scale (x_b cos theta + x_a sin theta);
 * GDR_ROPE_INVERSE turns by -theta (with the same scale: the gradient).  The
 * other channels are copied.  Long contexts scale inv_freq and, where wanted,
 * `scale`; the angle is formed in 64 bits, so far positions keep their accuracy.
 *
 *   q, q_out   : act  [B, Hq, T, d]       k, k_out : act [B, Hk, T, d]
 *                (k and k_out are NULL when Hk = 0; q and q_out when Hq = 0;
 *                an output may be its input, no other aliasing)
 *   inv_freq   : fp32 [rot_dim / 2]
 *   positions  : int32 [B, T] in device memory, or NULL: token t stands at
 *                position0 + t
 * Packed sequences: B = 1 and their positions.  One token of N sequences: B = N,
 * T = 1.  Flags: GDR_ACT_F32, GDR_TOKEN_MAJOR, GDR_ROPE_INTERLEAVED,
 * GDR_ROPE_INVERSE.  Supported: d in {16, 32, 64, 128}, rot_dim a multiple of 16
 * up to d.
 */
gdr_status gdr_rope(const void* q, const void* k, void* q_out, void* k_out,
                    const float* inv_freq, const int* positions, int position0,
                    int B, int Hq, int Hk, int T, int d, int rot_dim, float scale,
                    uint32_t flags, void* stream);

/*
 * Causal attention, forward.  Query i of Tq stands at place i + Tk - Tq among the
 * Tk keys and sees the keys up to it, the last `window` of them when window > 0:
 *   s_ij = scale q_i . k_j,  lse_i = log sum_j exp(s_ij),  o_i = sum_j exp(s_ij - lse_i) v_j.
 * A query that sees no key (Tk < Tq) gets o = 0 and lse = -inf.  A key or value
 * that a query does not see has no effect on it, not on one bit when it is finite.
 * NaN and infinities reach only the queries that see them as well: where a tile of 64
 * keys that some query sees in part holds one among its values, the tile's 128 queries
 * are computed one by one, which is many times slower and rounds otherwise (the
 * weights stay fp32).
 *
 *   q, o : bf16 [B, Hq, Tq, d]      k, v : bf16 [B, Hkv, Tk, d]
 *   lse  : fp32 [B, Hq, Tq] in both layouts, written; NULL means not written
 *   window : 0 (none) or the number of keys; scale >= 1e-30, finite
 * Products run on bf16 MFMA with fp32 accumulation; the weights exp(s - m) are
 * rounded to bf16 for the product with v (m the running maximum), their sum is
 * kept in fp32.  Flags: GDR_TOKEN_MAJOR.  Supported: d in {64, 128};
 * GDR_ERR_UNSUPPORTED otherwise (also for GDR_ACT_F32).  No workspace.
 */
gdr_status gdr_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                        int B, int Hq, int Hkv, int Tq, int Tk, int d, int window,
                        float scale, uint32_t flags, void* stream);

/*
 * The same over packed sequences, as gdr_chunk_fwd_varlen packs them: q, o
 * [Hq, T, d], k, v [Hkv, T, d], lse [Hq, T]; a query sees keys of its own
 * sequence only.  cu_seqlens: int32 [nseq + 1] in device memory, non-decreasing
 * from 0 (nseq at most 2^30); rows from cu_seqlens[nseq] on (if it is below T) are not written.
 */
gdr_status gdr_attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                               const int* cu_seqlens, int nseq, int Hq, int Hkv, int T, int d,
                               int window, float scale, uint32_t flags, void* stream);

/*
 * Gradients of gdr_attn_fwd for the loss <dO, o>: the probabilities are
 * recomputed from lse, P = exp(s - lse), and
 *   D_i = sum_j P_ij dO_i . v_j = dO_i . o_i,  dS_ij = P_ij (dO_i . v_j - D_i),
 *   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i,
 * dk and dv summed over the query heads that share the key head, in a fixed order.
 *
 *   q, k, v, o, lse : as gdr_attn_fwd took and wrote them     dO : bf16, as o
 *   dq : bf16, as q     dk, dv : bf16, as k   (written, never accumulated into;
 *        keys that no query sees get 0)
 *   workspace : device scratch of at least gdr_attn_bwd_workspace_bytes() bytes,
 *        contents on entry ignored; calls that may overlap need one each
 * Sums are fp32; P and dS are rounded to bf16 as operands.  D is formed from the
 * keys for queries that see at most 32 of them (there o's rounding would show in dq
 * and dk), from o for the others.  A pair that is not
 * seen has no effect on a gradient, as in the forward (finite values near the
 * type's largest, whose products overflow, included; NaN and infinities in partly
 * seen tiles make the tile's keys or queries slow as there).  Supported as
 * gdr_attn_fwd.  The varlen call leaves rows from cu_seqlens[nseq] on unwritten.
 */
size_t gdr_attn_bwd_workspace_bytes(int B, int Hq, int Hkv, int Tq, int Tk, int d);

gdr_status gdr_attn_bwd(const void* q, const void* k, const void* v, const void* o,
                        const float* lse, const void* dO, void* dq, void* dk, void* dv,
                        int B, int Hq, int Hkv, int Tq, int Tk, int d, int window,
                        float scale, uint32_t flags, void* workspace,
                        size_t workspace_bytes, void* stream);

gdr_status gdr_attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                               const float* lse, const void* dO, void* dq, void* dk, void* dv,
                               const int* cu_seqlens, int nseq, int Hq, int Hkv, int T, int d,
                               int window, float scale, uint32_t flags, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * The paged 8-bit key/value cache.  A page holds GDR_KV_PAGE tokens of every
 * key head as e4m3 values:
 *   k_cache : uint8 [n_pages, Hkv, 64, d]      v_cache : uint8 [n_pages, Hkv, 4, d, 16]
 *             (value of token 16 g + i and channel c at [g][c][i])
 *   k_scale, v_scale : fp32 [n_pages, Hkv]; a value stands for e4m3 * scale
 *   block_table : int32 [nseq, max_pages]: sequence n's token t is in page
 *             block_table[n][t / 64], slot t % 64
 *   cache_len : int32 [nseq]: tokens of each sequence in the cache
 *
 * gdr_kv_append writes new tokens behind the cache_len tokens of each sequence
 * (cache_len itself is the caller's to raise).  Per touched page and head the
 * scale becomes max(old, s), s the smallest power of two >= 2^-96 with every new
 * finite |x| <= 448 s; old counts as 0 when the page's first slot is written.
 * Values are round_e4m3(x / scale), to nearest even; infinities and NaN become
 * NaN.  Where the scale grows, the page's older tokens are rounded again to it
 * (exact but for values that fall below the normal range).  Slots behind the new
 * tokens are left as they were.
 *   k, v : bf16 [Hkv, T, d] ([T, Hkv, d] with GDR_TOKEN_MAJOR), sequence n's new
 *          tokens cu_seqlens[n] .. cu_seqlens[n + 1] - 1; or cu_seqlens NULL:
 *          [nseq, Hkv, d], one token of each sequence (T = nseq)
 * Tokens past max_pages pages, or whose page is not in [0, n_pages), are dropped.
 * The caller keeps two sequences of one call from writing to the same page.
 * Supported: d in {64, 128}.
 */
#define GDR_KV_PAGE 64

gdr_status gdr_kv_append(const void* k, const void* v, void* k_cache, void* v_cache,
                         float* k_scale, float* v_scale, const int* block_table,
                         const int* cache_len, const int* cu_seqlens, int nseq, int Hkv, int T,
                         int d, int n_pages, int max_pages, uint32_t flags, void* stream);

/*
 * Attention of one query token per sequence over the cache: the query stands at
 * the last of the cache_len tokens (append first) and sees all of them, or the
 * last `window`.  A sequence of length 0 gets o = 0; tokens in pages outside
 * [0, n_pages) count as masked; bytes of masked slots have no effect.
 *   q : bf16 [N, Hq, d]       o : fp32 (or bf16 with GDR_OUT_BF16) [N, Hq, d]
 *   workspace : device scratch of gdr_attn_decode_workspace_bytes() bytes (0:
 *        none needed, may be NULL), contents on entry ignored; calls that may
 *        overlap need one each
 * Scores, weights and sums are fp32 (the weights enter the product as two f16
 * parts).  The work is dealt out by the table's width (or the window): a table much
 * wider than its sequences makes calls of few sequences slow (one of 8,192 tokens
 * behind 128 pages 16 us, behind 16,384 86), so pass its first columns as a table of
 * their own.  The cache is read once for each 16 query heads of a key head.
 * Flags: GDR_OUT_BF16.  Supported: d in {64, 128}.
 */
size_t gdr_attn_decode_workspace_bytes(int N, int Hq, int Hkv, int d, int max_pages, int window);

gdr_status gdr_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                           const float* k_scale, const float* v_scale, const int* block_table,
                           const int* cache_len, void* o, int N, int Hq, int Hkv, int d,
                           int n_pages, int max_pages, int window, float scale, uint32_t flags,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Several continuations of one prompt: samples, beams, or a batch behind a common
 * system prompt.  Their sequences share the prompt's pages of the cache, whose tokens
 * are then read once a group; their block tables are forked, and their recurrent
 * states moved, as beams go on or end.
 *
 * Indexes and lengths in device memory (group_start, shared_pages, block_table,
 * cache_len, parent, room) are not checked on the host; no content of them makes a
 * kernel read or write outside the tensors.  Results do not depend on the order in which
 * workgroups run.  A call whose largest launch would pass 2^24 - 1 workgroups is
 * refused with GDR_ERR_INVALID_ARG.
 */

/*
 * gdr_attn_decode for groups of sequences that share their first pages: group g is the
 * sequences group_start[g] .. group_start[g + 1] - 1, and their first
 * shared_pages[g] pages are those in the table's row of the group's first sequence
 * (the other rows' entries for them are not read, and of that row those entries whatever the
 * sequence's length: where it was dropped and its row emptied, as gdr_kv_fork does for a parent
 * outside the table, let the group begin behind it, or its shared tokens count as masked).  Their tokens are read once for every
 * 32 or 64 of the group's (sequence, query head) pairs on a key head, not once for
 * each sequence.  Lengths and windows are each sequence's own; a sequence may end inside
 * the shared pages.  Sequences in no group share nothing.
 *   group_start  : int32 [groups + 1] in device memory, non-decreasing, within 0 .. N
 *   shared_pages : int32 [groups] in device memory
 *   the rest as gdr_attn_decode
 *   workspace    : gdr_attn_decode_shared_workspace_bytes() bytes of device scratch,
 *        contents on entry ignored; calls that may overlap need one each
 * A token that a sequence does not see has no effect on it, NaN included.  Scores, softmax
 * statistics and sums are fp32 (the weights enter the product with v as two f16 parts, 22
 * bits); a bf16 result is the fp32 one rounded once.
 * Flags: GDR_OUT_BF16.  Supported: d in {64, 128}, groups <= 4096, N Hq <= 2^24 - 2^15,
 * max_pages <= 2^24.
 */
size_t gdr_attn_decode_shared_workspace_bytes(int N, int groups, int Hq, int Hkv, int d, int max_pages,
                                              int window);

gdr_status gdr_attn_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                  const float* k_scale, const float* v_scale, const int* block_table,
                                  const int* cache_len, const int* group_start, const int* shared_pages,
                                  void* o, int N, int groups, int Hq, int Hkv, int d, int n_pages,
                                  int max_pages, int window, float scale, uint32_t flags,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rows of the block table continued, forked, grown and dropped, in one call between two
 * tokens: row n of the new table continues row parent[n] of the old one, for the
 * room[n] tokens that it is about to append.  A row holds the pages of its cache_len
 * tokens, and a page that no row holds (and `held` does not mark) is free.
 *   - Pages that hold whole pages of tokens are shared by the rows that continue a row.
 *   - The page that row n is about to write on (cache_len % 64 tokens are in it) is copied
 *     for it, unless no other row holds that page, or all rows that do are about to write
 *     on it and n is the lowest of them.  It is copied too where `held` marks it.
 *   - Fresh pages follow for the tokens that do not fit, as far as max_pages: a row whose table has no
 *     place left wants none and misses none.
 * The j-th page wanted (row by row, a row's copy first) is the j-th lowest free one.
 * Nothing is kept between calls, so that a call made again gives the same again; pages
 * that a row was given for tokens that were never appended are free at the next call.
 *   block_table : int32 [N_in, max_pages]   cache_len : int32 [N_in]
 *   parent      : int32 [N], or NULL: row n (N_in = N); outside [0, N_in): row n becomes
 *                 empty, is given no page, and has length 0
 *   room        : int32 [N], or NULL: room_all for every row
 *   held        : uint8 [n_pages], or NULL: pages that others hold (other tables)
 *   table_out   : int32 [N, max_pages], written; -1 behind a row's pages
 *   len_out     : int32 [N], written: the tokens that row n has
 *   missing     : int32 [N], written: pages that were wanted and not free.  A row that
 *                 misses any must not be appended to (its page may still be shared).
 *   k_cache, v_cache, k_scale, v_scale : as gdr_kv_append; copied pages are written
 *   workspace   : gdr_kv_fork_workspace_bytes() bytes of device scratch, contents on
 *                 entry ignored; calls that may overlap need one each
 * table_out and len_out may be block_table and cache_len where parent is NULL; no other
 * aliasing.  Every table that holds pages of this cache is either in the call or in `held`.
 * A call copies the pages of one layer's cache.  Layers under one table take a call each, all
 * with the same old table, lengths, parent, room and held, which give the same new table: only the last of
 * them may write over the old one.
 * flags must be 0.  Supported: d in {64, 128}, N_in, N <= 2^20, Hkv <= 65535, n_pages <= 2^30,
 * max_pages <= 2^24, N_in max_pages and N max_pages < 2^31.
 */
size_t gdr_kv_fork_workspace_bytes(int N, int n_pages);

gdr_status gdr_kv_fork(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                       const int* block_table, const int* cache_len, const int* parent,
                       const int* room, const uint8_t* held, int* table_out, int* len_out,
                       int* missing, int N_in, int N, int room_all, int Hkv, int d, int n_pages,
                       int max_pages, uint32_t flags, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Pages in use moved to the lowest places, so that the cache's tail is free: the j-th lowest
 * free page takes the j-th highest page that rows hold, while that is the higher of the
 * two.  Pages that `held` marks stay.  (Pages, rows and free ones as in gdr_kv_fork: call it
 * where cache_len is up to date.)
 *   table_out : int32 [N, max_pages], written; -1 behind a row's pages; may be block_table
 *               (of layers under one table, which take a call each, in the last one only)
 *   used      : int32 [1], written: one past the last page in use afterwards
 *   workspace : gdr_kv_compact_workspace_bytes() bytes of device scratch, contents on
 *               entry ignored; calls that may overlap need one each
 * flags must be 0.  Supported: as gdr_kv_fork.
 */
size_t gdr_kv_compact_workspace_bytes(int n_pages);

gdr_status gdr_kv_compact(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                          const int* block_table, const int* cache_len, const uint8_t* held,
                          int* table_out, int* used, int N, int Hkv, int d, int n_pages,
                          int max_pages, uint32_t flags, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * Beam search: the best M continuations of each of G groups of K beams over a vocabulary
 * of V tokens.  Row r = g K + k of the logits is beam k of group g, and
 *   score(k, t) = scores[r] + x_rt - log sum_u exp x_ru.
 * A beam that has ended offers one candidate, end_token at its own score, and its logits
 * are not read; its other candidates have the score -inf.  So have those of a row without
 * a finite log-sum (every logit -inf, or one of them NaN or +inf) and of a beam whose
 * score is not finite.  Candidates are taken in the order: score from the highest; lower
 * beam; higher logit; lower token.  Equal ones thus go to the lowest (beam, token).
 *   logits : bf16, or fp32 with GDR_ACT_F32: [G K] rows of V, `stride` elements apart
 *   scores : fp32 [G, K]     ended : uint8 [G, K] (0 or 1), or NULL: none
 *   tokens, rows : int32 [G, M], written: the token, and the row g K + k it continues
 *   scores_out   : fp32 [G, M], written
 *   ended_out    : uint8 [G, M], written: 1 where the beam had ended or the token ends it
 *   end_token    : the token that ends a beam; -1: none does (ended is NULL then)
 *   workspace    : gdr_beam_select_workspace_bytes() bytes of device scratch, contents on
 *                  entry ignored; calls that may overlap need one each
 * Results stand in the order taken, or with GDR_KEEP_SLOTS (M = K): the first taken
 * continuation of a beam in the beam's own place, the others, in order, in the places
 * left: then what a beam has (its state, its table's row) moves only where it has to.
 * Log-sums are formed in fp32 from each row's maximum and joined in 64 bits; scores are
 * compared in 64 bits and rounded once.  Supported: K, M <= 64, M <= K V, V <= 2^26, G K <= 65535,
 * stride <= 2^40.
 */
size_t gdr_beam_select_workspace_bytes(int G, int K, int M, int V);

gdr_status gdr_beam_select(const void* logits, const float* scores, const uint8_t* ended,
                           int* tokens, int* rows, float* scores_out, uint8_t* ended_out, int G,
                           int K, int M, int V, long long stride, int end_token, uint32_t flags,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * States moved to the rows that continue them, in place: state[l][n] becomes what
 * state[l][parent[n]] was, for rows of any type.  Rows n = g K .. g K + K - 1 are a group,
 * and parent[n] is in n's group; a row whose parent is not, or is itself, stays as it is
 * and costs nothing.
 *   state  : [layers, N, row_bytes], row_bytes a multiple of 16
 *   parent : int32 [N] in device memory (gdr_beam_select's rows, M = K)
 * flags must be 0.  Supported: K <= 64, N a multiple of K, layers N <= 2^28, row_bytes <= 2^40.
 */
gdr_status gdr_state_reorder(void* state, const int* parent, int layers, int N, int K,
                             size_t row_bytes, uint32_t flags, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */
