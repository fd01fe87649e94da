/*
 * kda.h -- C ABI of the MI355X (gfx950) Kimi Delta Attention library
 *          (libkda.so, built from gated_delta_rule_27_amd/csrc).
 *
 * The operation.  Per head, on a d_k x d_v fp32 state S (row i = key
 * channel, column j = value channel), every token t applies
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,
 *     o_t = S_t^T q_t,          alpha_t = exp(log_alpha_t) per key channel,
 *
 * ("Kimi K3 Architecture Explained", Step 3 "Forgetting, Channel by
 * Channel", the KDA equation; "An infra-oriented diagram of Kimi K3", KDA
 * card).  Decay acts on the old state before the erase and the write, and
 * the read uses the state after the token's own update ("From GPT-2 to
 * Kimi K3, from first principles", ch. 5 "Read the recurrence as four
 * verbs" and ch. 6 "Chunkwise execution").  There is no 1/sqrt(d_k) factor
 * on the read (the pages give none; q and k are L2-normalised upstream).
 *
 * Two regimes, as in the pages' mode rule (ch. 6 "Training, prefill, and
 * decode use different paths"): multi-token prefill runs chunkwise
 * (kda_chunk_fwd), a single cached token runs one fused recurrent step
 * (kda_decode_step).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers to contiguous row-major
 *     memory, 16-byte aligned, except beta (aligned to its element size,
 *     since its rows are only H elements) and cu_seqlens (4-byte aligned).
 *     Every [.., 128] row is 16-byte aligned when its base is, so slices at
 *     any token offset stay valid.  The caller owns every buffer; the library
 *     never allocates or frees device memory and keeps no state between
 *     calls except a per-device property cache.
 *   - Work is enqueued on `stream` (NULL = the default stream); no call
 *     synchronises the stream.  Buffers must stay valid until the queued
 *     work has finished.
 *   - Arguments are validated on the host before any HIP call; on an error
 *     nothing is launched and the outputs are untouched.  KDA_ERR_DEVICE
 *     reports a launch failure (the outputs are then unspecified).
 *   - d_k = d_v = 128 (the K3 head shape, "An infra-oriented diagram of
 *     Kimi K3", KDA card).  Other sizes return KDA_ERR_BAD_SHAPE.  The
 *     number of heads H is at most KDA_MAX_HEADS (the kernels address a
 *     16-token chunk of one tensor with 32-bit offsets).
 *   - Input contract (not checked, never clamped): log_alpha in [-5, 0]
 *     (the K3 lower-bounded log-decay, "From GPT-2 to Kimi K3", ch. 5
 *     "K3's lower-bounded decay"), beta in [0, 1].  Inside the contract the
 *     chunk kernels' decay factors stay finite: 16 tokens at log_alpha >= -5
 *     give a log-decay >= -80, so no factor exceeds e^80.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 2

#define KDA_MAX_HEADS 65536

typedef enum {
    KDA_OK = 0,
    KDA_ERR_NULL_ARG = 1,   /* a required pointer is NULL                    */
    KDA_ERR_BAD_SHAPE = 2,  /* a size <= 0 (or < 0 where 0 is allowed),
                               d_k or d_v != 128, H > KDA_MAX_HEADS, N != 1
                               without cu_seqlens, or an unsupported chunk /
                               split override                                */
    KDA_ERR_BAD_DTYPE = 3,  /* dtype is not a kda_dtype                      */
    KDA_ERR_MISALIGNED = 4, /* a pointer breaks the alignment rules above    */
    KDA_ERR_ALIAS = 5,      /* an output overlaps an input or another output */
    KDA_ERR_WORKSPACE = 6,  /* workspace smaller than the size reported      */
    KDA_ERR_DEVICE = 7      /* a HIP call or kernel launch failed            */
} kda_status;

/* Storage type of q, k, v, log_alpha, beta and o.  States are always fp32. */
typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/* Bytes of device workspace kda_chunk_fwd needs for these sizes (0 means
 * workspace may be NULL).  Never fails; returns 0 for invalid sizes. */
size_t kda_chunk_fwd_workspace_size(int64_t T_total, int32_t N, int32_t H,
                                    int32_t Dk, int32_t Dv, kda_dtype dt);

/*
 * Chunkwise prefill over N packed sequences.
 *
 *   q, k, log_alpha : [T_total, H, Dk]  dt
 *   v               : [T_total, H, Dv]  dt
 *   beta            : [T_total, H]      dt
 *   h0              : [N, H, Dk, Dv] fp32, read only; NULL = zero state
 *   cu_seqlens      : [N + 1] int32 DEVICE offsets of the packed sequences
 *                     ("An infra-oriented diagram of Kimi K3": several
 *                     documents share the packed tokens, cumulative offsets
 *                     keep their boundaries); NULL = one sequence (N == 1).
 *                     Precondition (not checked): cu[0] = 0, non-decreasing,
 *                     cu[N] = T_total.  Zero-length sequences are allowed
 *                     (their h_T is h0).
 *   o               : [T_total, H, Dv]  dt (output; round-to-nearest-even
 *                     from fp32 for bf16)
 *   h_T             : [N, H, Dk, Dv] fp32 final states; NULL = not stored.
 *                     Must not overlap h0: a stored snapshot is never
 *                     mutated ("From GPT-2 to Kimi K3", ch. 14 "Serving a
 *                     hybrid cache": restored snapshots are read-only).
 *   workspace       : device scratch of at least
 *                     kda_chunk_fwd_workspace_size(...) bytes (may be NULL
 *                     when that size is 0).
 * The state resets to h0[n] (or zero) at every sequence start; chunks are
 * aligned to each sequence's first token and the last chunk may be partial.
 * T_total == 0 is allowed (only h_T is written).
 */
kda_status kda_chunk_fwd(const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta,
                         const float* h0, const int32_t* cu_seqlens, int32_t N,
                         int64_t T_total, int32_t H, int32_t Dk, int32_t Dv,
                         kda_dtype dt, void* o, float* h_T, void* workspace,
                         size_t workspace_bytes, hipStream_t stream);

/*
 * kda_chunk_fwd with explicit tuning choices.  chunk = tokens per chunk
 * (16 or 32; 0 = library choice); dv_split = number of workgroups that
 * share one head's value columns (1, 2 or 4; 0 = library choice).  The
 * chunk length is a tuning parameter, not a property of the recurrence
 * ("From GPT-2 to Kimi K3", ch. 6 "Chunkwise execution"): every choice
 * computes the same function up to rounding.  Unsupported combinations
 * return KDA_ERR_BAD_SHAPE.
 */
kda_status kda_chunk_fwd_ex(const void* q, const void* k, const void* v,
                            const void* log_alpha, const void* beta,
                            const float* h0, const int32_t* cu_seqlens,
                            int32_t N, int64_t T_total, int32_t H, int32_t Dk,
                            int32_t Dv, kda_dtype dt, void* o, float* h_T,
                            void* workspace, size_t workspace_bytes,
                            int32_t chunk, int32_t dv_split,
                            hipStream_t stream);

/*
 * kda_chunk_fwd that also writes prefix snapshots of the state, for a prefix
 * cache: sparse KDA snapshots stored only at token boundaries on a fixed
 * grid (512-token hash boundaries on the pages, "From GPT-2 to Kimi K3",
 * "Serving a hybrid cache").
 *
 *   interval : a positive multiple of 16 tokens (KDA_ERR_BAD_SHAPE otherwise)
 *   snap_cu  : [N + 1] int32 device, snap_cu[n] = sum over m < n of
 *              floor(len_m / interval) with len_m = cu_seqlens[m+1] -
 *              cu_seqlens[m]; may be NULL only for N == 1 (base 0)
 *   n_snap   : entries of snap (snap_cu[N] when it is consistent)
 *   snap     : [n_snap, H, Dk, Dv] fp32, 16-byte aligned, written: entry
 *              snap_cu[n] + j - 1 = the state of sequence n after its first
 *              j * interval tokens, j = 1 .. floor(len_n / interval)
 *
 * Entries at or past n_snap are never written, whatever snap_cu holds.  A
 * snapshot is meant to be read-only: restoring one (h0 = a snapshot entry in
 * kda_chunk_fwd, or a copy as the in-place S of kda_decode_step) resumes the
 * recurrence from that boundary, and replaying only the accepted prefix of a
 * speculative draft from the pre-draft state is the same call with T = the
 * accepted tokens ("Speculative decoding cannot naively roll KDA back").
 * Errors as kda_chunk_fwd, plus: n_snap > 0 with snap NULL, or with N > 1
 * and snap_cu NULL, is KDA_ERR_NULL_ARG; snap overlapping any other buffer
 * is KDA_ERR_ALIAS.
 */
kda_status kda_chunk_fwd_snap(const void* q, const void* k, const void* v,
                              const void* log_alpha, const void* beta,
                              const float* h0, const int32_t* cu_seqlens,
                              int32_t N, int64_t T_total, int32_t H, int32_t Dk,
                              int32_t Dv, kda_dtype dt, void* o, float* h_T,
                              int32_t interval, const int32_t* snap_cu,
                              int64_t n_snap, float* snap, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/*
 * One recurrent step for B independent sequences (single-token cached
 * decode; "From GPT-2 to Kimi K3", ch. 6, the fused recurrent path).
 *
 *   q, k, log_alpha : [B, H, Dk]  dt
 *   v               : [B, H, Dv]  dt
 *   beta            : [B, H]      dt
 *   S               : [B, H, Dk, Dv] fp32, updated IN PLACE to S_t
 *   o               : [B, H, Dv]  dt, o = S_t^T q
 * B == 0 is allowed (nothing is launched).
 */
kda_status kda_decode_step(const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta, float* S,
                           int32_t B, int32_t H, int32_t Dk, int32_t Dv,
                           kda_dtype dt, void* o, hipStream_t stream);

/*
 * Segment summaries for KDA context parallelism ("An infra-oriented diagram
 * of Kimi K3", "KDA Context Parallelism"; "From GPT-2 to Kimi K3", ch. 6):
 * a segment maps the state entering it affinely, S_out = M S_in + B.  For
 * every segment n (the packed sequences of cu_seqlens, as for
 * kda_chunk_fwd):
 *   B[n] : [H, Dk, Dv] fp32, the state reached from a zero start;
 *   M[n] : [H, Dk, Dk] fp32, the product of the segment's per-token
 *          transitions (I - beta k k^T) Diag(alpha), latest on the left.
 * Either output may be NULL (not computed), not both.  Each is one prefill
 * pass (M: V taken as zero from the identity, by column independence).
 * Neither pass reads q (it feeds only the outputs o = S^T q, which a summary
 * does not form), so q may be NULL.  Errors as kda_chunk_fwd (o and h0 are
 * not arguments); v may be NULL when only M is asked for; M overlapping B
 * is KDA_ERR_ALIAS.  Both passes are validated before either is launched.
 */
kda_status kda_segment_summary(const void* q, const void* k, const void* v,
                               const void* log_alpha, const void* beta,
                               const int32_t* cu_seqlens, int32_t N,
                               int64_t T_total, int32_t H, int32_t Dk,
                               int32_t Dv, kda_dtype dt, float* M, float* B,
                               void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

/*
 * The exclusive scan over R consecutive segments of one sequence, per head:
 *   S_in[0] = h0 (NULL = 0),  S_in[r + 1] = M[r] S_in[r] + B[r],
 * with M, B, S_in : [R, H, 128, 128] fp32 and S_final = M[R-1] S_in[R-1] +
 * B[R-1] : [H, 128, 128] (may be NULL).  Resuming each segment from
 * S_in[r] (kda_chunk_fwd with h0 = S_in) reproduces the uninterrupted run.
 * R == 0 writes S_final = h0.  All buffers 16-byte aligned; S_in or
 * S_final overlapping an input is KDA_ERR_ALIAS.
 */
kda_status kda_segment_scan(const float* M, const float* B, const float* h0,
                            int32_t R, int32_t H, int32_t Dk, int32_t Dv,
                            float* S_in, float* S_final, hipStream_t stream);

/*
 * Backward pass of kda_chunk_fwd (training runs the chunkwise mode: "From
 * GPT-2 to Kimi K3", ch. 6, "Training, prefill, and decode use different
 * paths").  For the loss  sum(dout * o) + sum(dhT * h_T)  of the forward
 * pass on the same inputs (same layouts, same packed sequences), writes
 *   dq, dk, dv, dlog_alpha : [T_total, H, D]  dt
 *   dbeta                  : [T_total, H]     dt
 *   dh0                    : [N, H, Dk, Dv]   fp32 (NULL: not written)
 * from dout [T_total, H, Dv] (dt) and dhT [N, H, Dk, Dv] fp32 (NULL: zero).
 * The pages give no gradient formulas; they are the reverse mode of the
 * recurrence, checked against a token-by-token reverse-mode oracle that is
 * itself pinned by finite differences.
 *
 * The workspace (kda_chunk_bwd_workspace_size bytes, 16-byte aligned,
 * required) holds the state after every 16-token chunk and its gradient
 * in the input dtype: 2 x (T_total / 16 + N + 1) x H x 128 x 128 elements
 * (bf16 tables for bf16 inputs: the products read them as bf16 operands).  Three launches on `stream`:
 * the forward state recursion again (storing those states), the reverse
 * recursion of the state gradient, and all per-chunk gradients at once.
 * Errors as kda_chunk_fwd; dout and the five token gradients are required
 * when T_total > 0 (KDA_ERR_NULL_ARG); no output may overlap an input,
 * another output or the workspace (KDA_ERR_ALIAS); a missing or short
 * workspace is KDA_ERR_WORKSPACE.
 */
size_t kda_chunk_bwd_workspace_size(int64_t T_total, int32_t N, int32_t H,
                                    int32_t Dk, int32_t Dv, kda_dtype dt);

kda_status kda_chunk_bwd(const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta,
                         const float* h0, const int32_t* cu_seqlens, int32_t N,
                         int64_t T_total, int32_t H, int32_t Dk, int32_t Dv,
                         kda_dtype dt, const void* dout, const float* dhT,
                         void* dq, void* dk, void* dv, void* dlog_alpha,
                         void* dbeta, float* dh0, void* workspace,
                         size_t workspace_bytes, hipStream_t stream);

/*
 * kda_chunk_bwd for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving or training loops, harnesses that forbid
 * hipMalloc): the same computation, the same kernels and the same arguments
 * minus the workspace.  The per-chunk tables live instead in a scratch array
 * of KDA_BWD_NOALLOC_MAX_BYTES that the library holds in device memory, one
 * copy per GPU it runs on, from this call's first use on that GPU until the
 * process ends.  The call allocates nothing (no hipMalloc, hipFree or
 * allocating library routine); its first call on a device looks the array
 * up once (hipGetSymbolAddress), after all arguments are validated.
 *
 * Limit: kda_chunk_bwd_workspace_size(T_total, N, H, 128, 128, dt) must not
 * exceed KDA_BWD_NOALLOC_MAX_BYTES (256 MiB: for bf16, (T_total / 16 + N +
 * 1) * H <= 4096, e.g. 1,024 tokens of 48 heads or 512 tokens of 96 heads);
 * larger problems return KDA_ERR_WORKSPACE before any HIP call.  Other
 * errors as kda_chunk_bwd (KDA_ERR_DEVICE also when the scratch array cannot
 * be found on the current device).
 *
 * Every call on one GPU uses that GPU's one array, which keeps whatever the
 * last call left there (no call needs it cleared).  Calls that overlap on
 * one GPU -- on different streams, or from different threads -- race on
 * it: serialise them (one stream, or events).
 */
#define KDA_BWD_NOALLOC_MAX_BYTES ((size_t)256 << 20)

kda_status kda_chunk_bwd_noalloc(const void* q, const void* k, const void* v,
                                 const void* log_alpha, const void* beta,
                                 const float* h0, const int32_t* cu_seqlens,
                                 int32_t N, int64_t T_total, int32_t H,
                                 int32_t Dk, int32_t Dv, kda_dtype dt,
                                 const void* dout, const float* dhT, void* dq,
                                 void* dk, void* dv, void* dlog_alpha,
                                 void* dbeta, float* dh0, hipStream_t stream);

/*
 * Prologue of a KDA layer: from the outputs of its input projections to the
 * inputs of kda_chunk_fwd / kda_decode_step ("From GPT-2 to Kimi K3", ch. 6,
 * "Where q, k, v, alpha, and beta come from"; "An infra-oriented diagram of
 * Kimi K3", Kimi Delta Attention card; "Kimi K3 Architecture Explained",
 * "Inside a KDA Layer").  Per packed sequence n of cu_seqlens (as for
 * kda_chunk_fwd; N = 1 and cu_seqlens NULL for one sequence) and head:
 *   q, k, v    = Swish(conv(x_q | x_k | x_v)), q and k then divided by
 *                sqrt(sum over the head's 128 channels of x^2 + l2_eps);
 *   log_alpha  = -5 sigmoid(a_raw + a_bias), in (-5, 0);
 *   beta       = sigmoid(b_raw).
 * conv is depthwise and causal over the tokens of a sequence, width 4:
 * y_t[c] = sum_{j=0..3} w[c][j] x_{t-3+j}[c] (w[c][3] on the current token),
 * no bias; inputs before the sequence start come from conv_state_in (the
 * last three inputs of the previous segment, oldest first) or are zero when
 * it is NULL.  conv_state_out, when not NULL, receives the last three inputs
 * of every sequence (an empty sequence carries its history over), ready as
 * conv_state_in of the next segment or decode step.
 *
 *   xq, xk, xv, a_raw, q, k, v, log_alpha : [T_total, H, D]  dt
 *   b_raw, beta                           : [T_total, H]     dt
 *   conv_w   : [3 (q, k, v), H, D, 4] fp32
 *   a_bias   : [H, D] fp32
 *   conv_state_in / conv_state_out : [N, 3 (q, k, v), 3 (tokens), H, D] dt
 * D must be 128.  l2_eps must be finite and >= 0 (KDA_ERR_BAD_SHAPE).
 * No output may overlap an input or another output (KDA_ERR_ALIAS; a
 * decode loop alternates two history buffers).  Pointers 16-byte aligned,
 * b_raw / beta element aligned.  Math in fp32, outputs rounded to dt.
 */
kda_status kda_prologue(const void* xq, const void* xk, const void* xv,
                        const void* a_raw, const void* b_raw,
                        const float* conv_w, const float* a_bias,
                        const int32_t* cu_seqlens, int32_t N, int64_t T_total,
                        int32_t H, int32_t D, kda_dtype dt,
                        const void* conv_state_in, void* conv_state_out,
                        float l2_eps, void* q, void* k, void* v,
                        void* log_alpha, void* beta, hipStream_t stream);

/*
 * Epilogue of a KDA layer ("From GPT-2 to Kimi K3", ch. 6, "A third gate:
 * control what leaves the module"): head-wise RMSNorm and the full-rank
 * output gate,
 *   y = o / sqrt(mean over the head's 128 channels of o^2 + eps)
 *       * norm_w[h] * sigmoid(g),
 * where g is the output of the gate projection.
 *
 *   o, g, y : [T_total, H, D] dt;  norm_w : [H, D] fp32;  D must be 128.
 * y may be o or g itself (in place); any other overlap is KDA_ERR_ALIAS.
 * eps must be finite and >= 0.  Pointers 16-byte aligned.
 */
kda_status kda_epilogue(const void* o, const void* g, const float* norm_w,
                        int64_t T_total, int32_t H, int32_t D, kda_dtype dt,
                        float eps, void* y, hipStream_t stream);

/*
 * Up to K recurrent steps for each of B sequences in one pass over their
 * states: a short window of tokens per cached sequence, such as a
 * speculative draft.  Verifying a draft must not move the cached state, and
 * after acceptance only the accepted updates are replayed, on chip, from
 * the pre-draft state ("From GPT-2 to Kimi K3", "Speculative decoding
 * cannot naively roll KDA back"); with update_state = 0 this call is the
 * verify pass (outputs only), with update_state = 1 and n_tok = the accepted
 * counts it is the replay.  Token t of sequence b gives what t + 1 calls of
 * kda_decode_step would, to rounding (the column sums over the state's rows
 * are accumulated in another order); verify and replay of the same tokens
 * give bit-identical outputs, being the same kernel.
 *
 *   q, k, log_alpha : [B, K, H, Dk]  dt   (sequence-major, then token)
 *   v               : [B, K, H, Dv]  dt
 *   beta            : [B, K, H]      dt
 *   S               : [B, H, Dk, Dv] fp32, read; written back (in place)
 *                     iff update_state != 0
 *   n_tok           : [B] int32 device, tokens to apply per sequence, clamped
 *                     to [0, K] by the kernel; NULL = K for every sequence
 *   o               : [B, K, H, Dv]  dt; rows t >= n_tok[b] are not written
 * B == 0 is allowed (nothing is launched); K >= 1.  Alignment and errors as
 * kda_decode_step (n_tok: 4-byte aligned; o overlapping S, n_tok or an
 * input, or S overlapping an input or n_tok, is KDA_ERR_ALIAS).
 */
kda_status kda_decode_multi(const void* q, const void* k, const void* v,
                            const void* log_alpha, const void* beta, float* S,
                            const int32_t* n_tok, int32_t B, int32_t K, int32_t H,
                            int32_t Dk, int32_t Dv, kda_dtype dt,
                            int32_t update_state, void* o, hipStream_t stream);

/*
 * Speculative decoding with a tree of drafted tokens.  The tokens of one
 * serving step are a tree of N nodes per sequence over its cached state:
 * node 0 is the pending token (sampled, not yet in the state), every other
 * node continues an earlier one.  A step of a layer is kda_tree_prologue ->
 * kda_tree_decode -> kda_epilogue over all nodes at once, with state and
 * convolution history left as they are; kda_tree_accept then chooses one
 * path from the target's probabilities, and kda_tree_commit moves state and
 * history of every layer along that path alone ("From GPT-2 to Kimi K3",
 * "Speculative decoding cannot naively roll KDA back").  A chain of drafts
 * is the tree with parent = NULL.
 *
 *   parent : [B, N] int32 device, parent[b][i] the node that node i
 *            continues; any value outside [0, i) makes node i a
 *            continuation of the cached state itself (-1 by custom).
 *            NULL = a chain (node i continues node i - 1).
 *   n_node : [B] int32 device, nodes of each sequence, clamped to [0, N] by
 *            the kernels; NULL = N for every sequence.  Nodes at or past it
 *            take no part and their output rows are not written.
 *   1 <= N <= KDA_MAX_TREE; B * H < 2^23 (kda_tree_accept: B < 2^22), else
 *   KDA_ERR_BAD_SHAPE.  B == 0 is allowed (nothing is launched).
 * No call keeps anything between calls or uses scratch memory: calls may run
 * at the same time on several streams, and in captured graphs.
 */
#define KDA_MAX_TREE 64

/*
 * The prologue of a KDA layer (kda_prologue) for the nodes of a tree: node i
 * convolves over itself and its three nearest ancestors, and where it has
 * fewer, over the end of the cached history.  For a chain the outputs are
 * the bits of kda_prologue on the same tokens.
 *
 *   xq, xk, xv, a_raw, q, k, v, log_alpha : [B, N, H, D]  dt
 *   b_raw, beta                           : [B, N, H]     dt
 *   conv_w : [3, H, D, 4] fp32;  a_bias : [H, D] fp32
 *   conv_state : [B, 3 (q, k, v), 3 (tokens), H, D] dt, read only; NULL =
 *                zero history
 * Errors, alignment and l2_eps as kda_prologue (parent, n_node: 4-byte
 * aligned; N out of range is KDA_ERR_BAD_SHAPE).
 */
kda_status kda_tree_prologue(const void* xq, const void* xk, const void* xv,
                             const void* a_raw, const void* b_raw,
                             const float* conv_w, const float* a_bias,
                             const int32_t* parent, const int32_t* n_node,
                             int32_t B, int32_t N, int32_t H, int32_t D,
                             kda_dtype dt, const void* conv_state, float l2_eps,
                             void* q, void* k, void* v, void* log_alpha,
                             void* beta, hipStream_t stream);

/*
 * The KDA outputs of every node of a tree from one read of the cached state,
 * which is not written: with S_i = (I - beta_i k_i k_i^T) Diag(alpha_i)
 * S_parent(i) + beta_i k_i v_i^T, o_i = S_i^T q_i.  Node i gives what
 * kda_decode_multi would on the path from the root to i, to the rounding of
 * an evaluation that holds 24 bits of every operand, whatever dt, and rounds
 * to dt once.  A NaN or infinity of node i reaches no other nodes than those
 * that descend from it: in k, log_alpha or beta it makes NaN of all outputs of
 * i and of its descendants, in v of that column of theirs, and in q it makes
 * i's own outputs non-finite.
 *
 *   q, k, log_alpha : [B, N, H, Dk]  dt
 *   v               : [B, N, H, Dv]  dt
 *   beta            : [B, N, H]      dt
 *   S               : [B, H, Dk, Dv] fp32, read only
 *   o               : [B, N, H, Dv]  dt
 * Alignment and errors as kda_decode_multi (o overlapping S, parent, n_node
 * or an input is KDA_ERR_ALIAS).
 */
kda_status kda_tree_decode(const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta,
                           const float* S, const int32_t* parent,
                           const int32_t* n_node, int32_t B, int32_t N,
                           int32_t H, int32_t Dk, int32_t Dv, kda_dtype dt,
                           void* o, hipStream_t stream);

/*
 * Verification of the drafted tokens against the target's probabilities:
 * the accepted path and the next token of every sequence.  The walk starts
 * at node 0.  At node r, with p the target's distribution after r and q the
 * draft distribution that r's children were drawn from, c = 0 and Z = 1 on
 * arrival, r's children x (token t, random number u_x) are tried in
 * ascending order:
 *     w = max(p(t) - c q(t), 0);  x is accepted iff  u_x q(t) Z < w;
 *     refused: c <- c + Z,  Z <- sum over v of max(p(v) - c q(v), 0).
 * Without q the drafts are certain (chosen, not drawn): w = p(t), 0 for a
 * token refused here before, x is accepted iff u_x Z < w, and a refusal
 * takes p(t) out: Z <- Z - w.  An accepted child is the next r; where no
 * child is accepted, the next token is drawn from what is left at r,
 *     w(v) = max(p(v) - c q(v), 0)   (without q: p without refused tokens),
 * as the smallest v with  sum of w over 0..v  >  u_0 * (sum of w)  (from p
 * itself where w has no mass left).  The tokens so emitted are distributed
 * as the target's own samples.  Sums and comparisons are in fp64.
 *
 *   p      : [B, N, V] dt, row i the target's distribution after node i
 *   q      : [B, N - 1, V] dt, row i the draft distribution of node i's
 *            children (the last node can have none); NULL = certain drafts
 *   tokens : [B, N] int32, the drafted tokens (tokens[b][0] is not read); a
 *            token outside [0, V) is refused and changes nothing else
 *   u      : [B, N] fp32 in [0, 1): u[b][i] tests node i >= 1, u[b][0]
 *            draws the next token
 *   path   : [B, N] int32 output, the accepted nodes in order (path[b][0] =
 *            0), then -1
 *   n_path : [B] int32 output, accepted nodes (>= 1; 0 for a sequence
 *            without nodes): n_tok of kda_decode_multi for a chain, n_path
 *            of kda_tree_commit
 *   next_token : [B] int32 output (-1 for a sequence without nodes)
 * A node whose parent lies outside [0, i) is never reached.  p and q are
 * probabilities: finite, >= 0, rows summing to 1 up to rounding (not
 * checked; a NaN or negative weight counts as 0, nothing out of range is
 * ever read or written, and the next token lies in [0, V)).
 * 1 <= V <= KDA_MAX_VOCAB.  p and q 16-byte aligned (their rows need not be;
 * a slice of a batch over an odd vocabulary may start where it is refused),
 * the int32 and fp32 arrays 4-byte aligned.  Any overlap of an output with
 * another buffer is KDA_ERR_ALIAS.
 */
#define KDA_MAX_VOCAB (1 << 22)

kda_status kda_tree_accept(const void* p, const void* q, const int32_t* tokens,
                           const int32_t* parent, const int32_t* n_node,
                           const float* u, int32_t B, int32_t N, int32_t V,
                           kda_dtype dt, int32_t* path, int32_t* n_path,
                           int32_t* next_token, hipStream_t stream);

/*
 * Moves cached states, and convolution histories, along one path of each
 * tree: the tokens of the nodes path[b][0], path[b][1], ... are applied in
 * that order, as kda_decode_step would one after the other.
 *
 *   k, log_alpha : [B, N, H, Dk]  dt  (N >= 1 nodes, here without a limit)
 *   v            : [B, N, H, Dv]  dt
 *   beta         : [B, N, H]      dt
 *   S            : [B, H, Dk, Dv] fp32, updated IN PLACE
 *   path         : [B, P] int32; a path ends before an entry outside [0, N)
 *                  (P > 16 runs the code of long paths, 1 to 2 us a call slower
 *                  on short ones in small batches, the same in large ones)
 *   n_path       : [B] int32, entries to apply, clamped to [0, P]; NULL = P
 *   xq, xk, xv   : [B, N, H, Dk]  dt, the inputs of the convolution
 *   conv_state   : [B, 3 (q, k, v), 3 (tokens), H, Dk] dt, updated IN PLACE
 *                  to the last three of (history, inputs along the path);
 *                  NULL = not kept (xq, xk, xv are then not read)
 * A sequence whose path is empty keeps its state and history untouched.
 * 1 <= P <= KDA_MAX_PATH.  Alignment and errors as kda_decode_multi; S or conv_state
 * overlapping another buffer is KDA_ERR_ALIAS.
 */
#define KDA_MAX_PATH (1 << 24)

kda_status kda_tree_commit(const void* k, const void* v, const void* log_alpha,
                           const void* beta, float* S, const int32_t* path,
                           const int32_t* n_path, int32_t B, int32_t N,
                           int32_t P, int32_t H, int32_t Dk, int32_t Dv,
                           kda_dtype dt, const void* xq, const void* xk,
                           const void* xv, void* conv_state,
                           hipStream_t stream);

/*
 * The state cache in 8 bits.  A cached state is held as codes in -127..127
 * and one scale per key channel,
 *
 *     codes : [.., H, Dv, Dk] int8   (value channel, then key channel)
 *     scale : [.., H, Dk] fp32       S[i][j] = scale[i] * codes[j][i],
 *
 * scale[i] = (largest |S[i][j]| over j) / 127 in fp32 and codes[j][i] = S[i][j]
 * times (127 / largest, in fp32), the exact product rounded to the nearest whole
 * number, ties to even: half a scale step off at the most.  A key channel without
 * a magnitude of 2^-100 or more is held as zeros; one with a NaN or an
 * infinity reads back as NaN.  The decay Diag(alpha) multiplies key channels,
 * so the scales take it up and the codes keep their bits.
 *
 * Beside the 8-bit state lies a window of up to W tokens whose rank-one
 * updates are not yet in it: the tokens' keys k_t and log-decays log alpha_t
 * and their updates u_t = beta_t (v_t - S'^T k_t), S' the state before token
 * t's write, decayed by it, so that after the window's first n tokens
 *
 *     S = Diag(e^(G_0)) Diag(scale) codes^T
 *         + sum over t < n of (e^(G_(t+1)) k_t) u_t^T,
 *     G_t = log alpha_t + ... + log alpha_(n-1).
 *
 *     win_k, win_log_alpha : [.., H, W, Dk] dt
 *     win_u                : [.., H, W, Dv] dt
 *     n_win : int32 device, tokens in each window.  The caller keeps it, one
 *             for all the layers of a model: kda_cache_decode puts its token
 *             at place n_win, after which the caller counts one more;
 *             kda_cache_fold empties a window, after which the caller sets 0.
 * 1 <= W <= KDA_MAX_WINDOW.  A state is rounded to its codes once per fold and
 * not once per token.  B * H < 2^24, else KDA_ERR_BAD_SHAPE; B == 0 is allowed
 * (nothing is launched).  Pointers are 16-byte aligned, n_win and page 4-byte.
 * No call keeps anything between calls or uses scratch memory.
 */
#define KDA_MAX_WINDOW 16

/*
 * fp32 states (final states of a prefill, prefix snapshots) into the cache.
 *
 *   S     : [B, H, Dk, Dv] fp32, read only
 *   page  : [B] int32 device, the page each state goes to; a state whose page
 *           lies outside [0, P) is left out, and of several states for one
 *           page the last one counts.  NULL = state b to page b (B <= P)
 *   codes : [P, H, Dv, Dk], scale : [P, H, Dk], outputs; pages not named are
 *           not written
 * Any overlap of an output with another buffer is KDA_ERR_ALIAS.
 */
kda_status kda_cache_store(const float* S, const int32_t* page, int32_t B, int32_t P,
                           int32_t H, int32_t Dk, int32_t Dv, int8_t* codes,
                           float* scale, hipStream_t stream);

/*
 * Pages of the cache back into fp32 states, with their windows' updates.
 *
 *   codes, scale : [P, ..]; win_k, win_log_alpha, win_u : [P, H, W, ..] dt,
 *           all three NULL = no windows (n_win, W and dt are then not looked at)
 *   page  : [B] int32, the page each state is read from (several may read the
 *           same one); outside [0, P) the state is not written.  NULL = page b
 *   n_win : [B] int32, the tokens to apply to each state, clamped to [0, W];
 *           NULL = W
 *   S     : [B, H, Dk, Dv] fp32, output
 * S overlapping another buffer is KDA_ERR_ALIAS.
 */
kda_status kda_cache_load(const int8_t* codes, const float* scale, const int32_t* page,
                          const void* win_k, const void* win_log_alpha,
                          const void* win_u, const int32_t* n_win, int32_t B,
                          int32_t P, int32_t H, int32_t W, int32_t Dk, int32_t Dv,
                          kda_dtype dt, float* S, hipStream_t stream);

/*
 * One recurrent step for a batch of states in the 8-bit cache: kda_decode_step
 * with the state read from codes, scale and window, and the token appended to
 * the window.  With S the state before, S' = Diag(alpha) S:
 *
 *     u = beta (v - S'^T k), held in dt,    o = S'^T q + (k . q) u.
 *
 *   q, k, log_alpha : [B, H, Dk]  dt;  v : [B, H, Dv] dt;  beta : [B, H] dt
 *   codes, scale    : [B, ..], read only
 *   win_k, win_log_alpha, win_u : [B, H, W, ..] dt, places below n_win[b]
 *                     read, place n_win[b] written
 *   n_win           : [B] int32, required; a sequence whose n_win lies outside
 *                     [0, W) is idle: nothing of it is read or written
 *   o               : [B, H, Dv]  dt
 * The reads of the state are sums over the key channels that are off by fp32
 * roundings of their own terms: k and q, times decay and scale in fp32, meet the codes
 * as whole numbers, with all their bits however much larger another channel is (down to
 * 2^-150 of the largest).  A NaN or infinity in q makes NaN of the head's outputs, one
 * in k, or a NaN or +infinity in log_alpha, of its outputs and its update; -infinity in
 * log_alpha, here and in a window, is a decay to 0 and empties the key channel.  Any
 * overlap of o or the window with another buffer is KDA_ERR_ALIAS.
 */
kda_status kda_cache_decode(const void* q, const void* k, const void* v,
                            const void* log_alpha, const void* beta,
                            const int8_t* codes, const float* scale, void* win_k,
                            void* win_log_alpha, void* win_u, const int32_t* n_win,
                            int32_t B, int32_t H, int32_t W, int32_t Dk, int32_t Dv,
                            kda_dtype dt, void* o, hipStream_t stream);

/*
 * The windows' updates into the 8-bit states, in place: what kda_cache_load
 * gives, rounded to codes and scales anew.
 *
 *   n_win : [B] int32, tokens to take in, clamped to [0, W]; NULL = W.  A
 *           sequence with none keeps its state untouched.
 * The windows are read only.  codes or scale overlapping another buffer is
 * KDA_ERR_ALIAS.
 */
kda_status kda_cache_fold(int8_t* codes, float* scale, const void* win_k,
                          const void* win_log_alpha, const void* win_u,
                          const int32_t* n_win, int32_t B, int32_t H, int32_t W,
                          int32_t Dk, int32_t Dv, kda_dtype dt, hipStream_t stream);

/*
 * Sampling: the next token of every row of logits, and the probabilities it is
 * drawn with (what kda_tree_accept takes as the target's p and, from a draft
 * model's logits, as q).  With T the row's temperature and M its largest
 * logit, a token weighs w_i = e^((l_i - M) / T); -infinity and NaN weigh 0 and
 * are never kept, and if M is infinite, what equals it weighs 1 and all else 0.
 * In the order of descending logits, equal ones by ascending index, what is
 * kept is the shortest of
 *     top-k : the first k tokens                 (off: k < 1 or k >= V)
 *     top-p : the smallest leading set whose weights sum to at least p times
 *             those of the first k               (off: p >= 1 or NaN; one
 *             token at least)
 *     min-p : the tokens of w_i >= min(m, 1)     (off: m <= 0 or NaN)
 * and T = 0 (or less, or NaN) keeps the first token alone.  The probabilities
 * are the kept tokens' weights over their sum, 0 elsewhere, rounded to dt
 * once.  The token drawn is the smallest kept i with
 *     (sum of the kept w over 0..i)  >  u * (sum of the kept w),
 * -1 where a row has no weight at all (its probabilities are then all 0).
 * Weights are e^x in 64 bits, added up as whole numbers of 2^-F of the largest
 * (F = 62 less the bits of V, 50 at most), so that results do not depend on the
 * launch or the order.  A token that weighs less than half of 2^-F counts for
 * nothing in them: the share of a nucleus and the place of u are met within
 * V * 2^-(F + 1) of the sum of the weights, 1.1e-10 for 32,000 tokens, 4.5e-9 for
 * 160,000 and 4e-6, which is more than a step of an fp32 u or top_p, for four
 * million.  Elsewhere tokens are what exact sums give.  Without a filter tiles of
 * 1024 tokens are counted so, not tokens: within a thousandth of that, and 1e-12.
 * What is drawn is always kept, and has a probability above 0.
 *
 *   logits, probs : [R, V] dt;  probs NULL = not wanted
 *   u             : [R] fp32 in [0, 1) (clamped; NaN counts as 0); NULL = no
 *                   token is wanted (token is then not looked at, probs is
 *                   required)
 *   temperature, top_p, min_p : [R] fp32;  top_k : [R] int32;  NULL = 1, off,
 *                   off, off for every row
 *   token         : [R] int32
 *   workspace     : kda_sample_workspace_size(R, V) bytes, 16-byte aligned,
 *                   for this call alone until it has run (calls that may run at
 *                   the same time, captured ones among them, need their own)
 * 1 <= V <= KDA_MAX_VOCAB, R < 2^22, R * ceil(V / 4096) < 2^24, else
 * KDA_ERR_BAD_SHAPE; R == 0 is allowed (nothing is launched).  logits and
 * probs 16-byte aligned (their rows need not be), the arrays 4-byte.  Any overlap of token, probs or
 * workspace with another buffer is KDA_ERR_ALIAS.
 */
size_t kda_sample_workspace_size(int32_t R, int32_t V);

kda_status kda_sample(const void* logits, const float* u, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p,
                      int32_t R, int32_t V, kda_dtype dt, int32_t* token, void* probs,
                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Static, human-readable name of a status code (never NULL). */
const char* kda_status_str(kda_status s);

/* KDA_ABI_VERSION of the built library. */
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* KDA_H */
