/*
 * kda.h -- C ABI of the MI355X (gfx950) KDA recurrent prefill forward.
 *
 * The operation is the Kimi Delta Attention prefill forward described by the
 * FlashInfer PR #4262 summary (section 1 "A Fused Recurrent-Prefill Kernel",
 * section 2 "Chunk-32 Through Fixed-Anchor Exponent Centering", section 3
 * "Intra-Chunk and Inter-Chunk Decomposition") with the call contract of
 * FlashKDA's `fwd` ("How FlashKDA Manages Recurrent State Across Sequences and
 * Batch Modes", the Python wrapper and both modes).  Per sequence n and head h
 * the V x K state S evolves token by token as
 *
 *     lam_t = lower_bound * sigmoid(exp(A_log[h]) * (g_t + dt_bias[h]))  (per key column)
 *     S     = S * diag(exp(lam_t))
 *     S     = S + sigmoid(beta_t) * (v_t - S kh_t) kh_t^T
 *     out_t = scale * S qh_t
 *
 * with qh, kh the L2-normalised q and k rows (x / sqrt(|x|^2 + 1e-6)).  The
 * library evaluates this in chunks of 32 or 16 tokens (fewer for strongly
 * negative lower bounds) with bf16 matrix-core products and an fp32 state that
 * stays on chip for the whole sequence.
 * Within a chunk the decayed operands are centred on a fixed exponent anchor
 * (section 2 of the PR #4262 summary); the state rows' 1-norms must stay below
 * 2^25 for the centred state products to stay inside fp32, and q and k rows
 * below an L2 norm of 1.8e19 (their sums of squares are fp32).
 *
 * Conventions for every entry point:
 *   - Every pointer argument except `stream` is a caller-owned DEVICE pointer
 *     to contiguous memory; the library never frees or retains it.
 *   - Kernels launch on the calling thread's current HIP device: the pointers
 *     and `stream` must belong to it (hipSetDevice before the call).
 *   - The library allocates nothing and keeps no global state; calls on
 *     different streams may run concurrently.  The one exception is
 *     kda_fwd_split_noalloc, whose scratch is a static device array per GPU.
 *   - kda_fwd is asynchronous: it validates on the host, enqueues one kernel on
 *     `stream` and returns.  It never reads device memory on the host (in
 *     particular not cu_seqlens) and never synchronises.
 *   - Errors are returned as negative status codes; nothing aborts or throws
 *     across this ABI.  On a validation error nothing is enqueued.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define KDA_OK 0
#define KDA_ERR_NULL_ARG (-1)        /* a required pointer is NULL (q, k, v, g, beta and */
                                     /* out may be NULL when B * T == 0)                */
#define KDA_ERR_BAD_SHAPE (-2)       /* B,T,H < 1 (T may be 0 only with cu_seqlens),     */
                                     /* D not in {32, 64, 128}, H * D >= 2^25,            */
                                     /* B * T > 2^40, num_seqs * H > 2^29, an activation  */
                                     /* tensor of more than 2^62 bytes, or a launch of    */
                                     /* more than 2^32 - 1 work-items (workgroups times   */
                                     /* their 128 to 768 threads)                         */
#define KDA_ERR_BAD_DTYPE (-3)       /* unknown state, weight or residual dtype, or gate */
                                     /* function code                                    */
#define KDA_ERR_BAD_VARLEN (-4)      /* cu_seqlens with B != 1, num_seqs < 1, or         */
                                     /* num_seqs != B without cu_seqlens                 */
#define KDA_ERR_BAD_ALIAS (-5)       /* an output overlaps an input or the other output; */
                                     /* only the exact in-place state alias is allowed   */
#define KDA_ERR_BAD_LOWER_BOUND (-6) /* lower_bound not finite, not < 0, below -2.35e38 */
                                     /* (lb log2(e) not a finite float), or too strong   */
                                     /* for a forced chunk size (see kda_fwd)            */
#define KDA_ERR_BAD_SCALE (-7)       /* scale not finite (kda_attn_fwd: its limits)      */
#define KDA_ERR_BAD_SCHEDULE (-8)    /* unsupported forced chunk size or value tile      */
#define KDA_ERR_HIP (-9)             /* the HIP runtime reported an error at launch      */
#define KDA_ERR_BAD_WORKSPACE (-10)  /* kda_fwd_split: workspace smaller than required   */
#define KDA_ERR_SCRATCH_TOO_SMALL (-11) /* kda_fwd_split_noalloc: the call's workspace   */
                                        /* exceeds kda_split_noalloc_max_bytes()         */
#define KDA_ERR_BAD_LAYOUT (-12)     /* serving operators: a pointer or row stride is    */
                                     /* not a multiple of 16 bytes, or a row stride is   */
                                     /* shorter than the row                             */

/* State dtype codes (initial_state_dtype, final_state_dtype); kda_norm's weights and residual. */
#define KDA_DTYPE_BF16 0
#define KDA_DTYPE_FP32 1
/* kda_norm's gate functions. */
#define KDA_GATE_SIGMOID 0
#define KDA_GATE_SILU 1

/*
 * kda_fwd -- the prefill forward (FlashKDA `fwd` contract: q, k, v, g, beta,
 * scale, out, A_log, dt_bias, lower_bound, initial_state, final_state,
 * cu_seqlens).
 *
 *   q, k, v, g     bf16 [B, T, H, D], contiguous (D fastest).  K = V = D.
 *   beta           bf16 [B, T, H], logits (the kernel applies the sigmoid).
 *   scale          output scale, folded into the normalised q; finite.
 *   out            bf16 [B, T, H, D], written for every token (padding-free).
 *   A_log          fp32 [H].
 *   dt_bias        fp32 [H, D].
 *   lower_bound    gate lower bound lb (finite, < 0); per-token decay lies in (lb, 0).
 *   initial_state  [num_seqs, H, D(v), D(k)] of initial_state_dtype, or NULL for zeros.
 *   final_state    [num_seqs, H, D(v), D(k)] of final_state_dtype, or NULL (not written).
 *                  It may be exactly the same allocation as initial_state (same
 *                  pointer and dtype: in-place update); any other overlap between
 *                  buffers is rejected.  Each workgroup reads all state rows it
 *                  owns before it writes any of them, which makes the alias safe.
 *   cu_seqlens     int64 [num_seqs + 1] device array, or NULL.
 *                  NULL: batched mode, num_seqs == B, sequence b is tokens
 *                  [b*T, (b+1)*T) of the flattened [B*T] axis, no resets.
 *                  Non-NULL: varlen mode, B == 1, sequence n is tokens
 *                  [cu[n], cu[n+1]); the state restarts from initial_state[n]
 *                  (or zeros) at every sequence.  Preconditions (not checked on
 *                  the host, which never reads device memory): cu[0] = 0,
 *                  non-decreasing, cu[num_seqs] = T.  The kernel clamps every
 *                  index into [0, T] so a malformed array cannot make it access
 *                  memory out of bounds; results are then unspecified.
 *                  An empty sequence passes its initial state (or zeros) through.
 *   num_seqs       N (see above).
 *   B, T, H, D     sizes; D in {32, 64, 128}.
 *   stream         a hipStream_t (NULL: the null stream).
 *
 * Scheduling: a packed batch of at most 256 sequences whose workgroups (num_seqs *
 * H * D / value tile) number between one and four times the device's compute
 * units is dispatched longest first: the kernel ranks the lengths itself, so the
 * host still reads nothing.  The order never changes the results (see
 * kda_fwd_ordered for a caller-chosen order).
 *
 * Returns KDA_OK or a negative status.  The decay span of a chunk is
 * chunk * |lower_bound| * log2(e); it must not exceed 236.  The library uses the
 * longest chunk whose span allows it: 32 tokens for |lb| <= 5.112, 16 for
 * |lb| <= 10.22, then 8, 4 and 2 tokens, and one token per chunk for every
 * stronger lower bound (chunks shorter than 16 tokens run in 16-row tiles, so each
 * halving of the chunk doubles the kernel's sequential steps).  Past
 * |lb| = 163.6 one token's decay can exceed the span: the kernel then floors each
 * token's decay factor at 2^-236 (about 1e-71), which differs from the exact
 * recurrence by less than 1e-71 times the state.  See kda_chunk_anchor.
 */
int kda_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
            float scale, void* out, const float* A_log, const float* dt_bias, float lower_bound,
            const void* initial_state, int initial_state_dtype, void* final_state,
            int final_state_dtype, const int64_t* cu_seqlens, int64_t num_seqs, int64_t B,
            int64_t T, int64_t H, int64_t D, void* stream);

/*
 * kda_fwd_sched -- kda_fwd with a forced schedule, for tests and tuning.
 *   chunk_size  0 (automatic), or tokens per chunk: 32, 16, 8, 4, 2 or 1
 *               (KDA_ERR_BAD_SCHEDULE otherwise).  A chunk of 2 or more tokens
 *               whose decay span exceeds 236 (see kda_fwd) is rejected with
 *               KDA_ERR_BAD_LOWER_BOUND, e.g. 32 when |lb| > 5.112; one-token
 *               chunks take every lower bound.
 *   v_tile      0 (automatic) or the number of value rows one workgroup owns:
 *               a divisor of D that is a multiple of 16 and at least 32
 *               (KDA_ERR_BAD_SCHEDULE otherwise).  Automatic: D, or D/2 for
 *               D = 128 with 32-token chunks when twice num_seqs * H workgroups
 *               still fit one per compute unit of the current device (queried
 *               on the host; the host never synchronises).
 * Everything else is exactly as kda_fwd.
 */
int kda_fwd_sched(const void* q, const void* k, const void* v, const void* g, const void* beta,
                  float scale, void* out, const float* A_log, const float* dt_bias,
                  float lower_bound, const void* initial_state, int initial_state_dtype,
                  void* final_state, int final_state_dtype, const int64_t* cu_seqlens,
                  int64_t num_seqs, int64_t B, int64_t T, int64_t H, int64_t D, void* stream,
                  int chunk_size, int v_tile);

/*
 * kda_fwd_ordered -- kda_fwd with a caller-chosen order of the sequences over
 * the workgroups (the sequence-order option of the FlashInfer PR #4262
 * summary's integration section, where it serves tail utilisation).
 *   seq_order  int32 [num_seqs] device array, a permutation of 0 .. num_seqs-1:
 *              the workgroups of sequence seq_order[0] are dispatched first,
 *              then those of seq_order[1], and so on.  Longest first (see
 *              kda_longest_first) keeps long sequences of a packed batch from
 *              starting last.  It must not overlap any output
 *              (KDA_ERR_BAD_ALIAS); NULL is KDA_ERR_NULL_ARG.
 * The results are bitwise those of kda_fwd: the order only changes which
 * workgroup starts when.  The host never reads seq_order; entries outside
 * [0, num_seqs) are clamped (in bounds, but the results are then unspecified).
 * Everything else is exactly as kda_fwd.
 */
int kda_fwd_ordered(const void* q, const void* k, const void* v, const void* g,
                    const void* beta, float scale, void* out, const float* A_log,
                    const float* dt_bias, float lower_bound, const void* initial_state,
                    int initial_state_dtype, void* final_state, int final_state_dtype,
                    const int64_t* cu_seqlens, int64_t num_seqs, int64_t B, int64_t T, int64_t H,
                    int64_t D, void* stream, const int32_t* seq_order);

/*
 * kda_fwd_bf16_state -- kda_fwd_sched with the recurrent state held in bf16 in
 * on-chip memory (LDS) instead of fp32 registers, as the page "How FlashKDA
 * Stores On-Chip Recurrent State in BF16 for Memory Efficiency" describes (its
 * sections "The BF16 State Layout in Shared Memory" and "State Updates with FP32
 * FMA"): each chunk's update widens the stored state to fp32, applies the decay
 * and adds the chunk's term in fp32, then rounds once back to bf16.  An fp32
 * initial state is rounded to bf16 on entry; the final state is the stored bf16
 * state (exact in either output dtype).
 * Runs D = 128 with 32-token chunks (chunk_size 0 or 32; the lower bound must
 * allow them, |lb| <= 5.112) at v_tile 0, 64 or 128; other schedules return
 * KDA_ERR_BAD_SCHEDULE.  States are [num_seqs, H, D(v), D(k)] as for kda_fwd;
 * everything else, including the exact in-place alias, is exactly as kda_fwd.
 * The results differ from kda_fwd by the per-chunk rounding of the state; it is
 * an opt-in mode and never chosen automatically.
 */
int kda_fwd_bf16_state(const void* q, const void* k, const void* v, const void* g,
                       const void* beta, float scale, void* out, const float* A_log,
                       const float* dt_bias, float lower_bound, const void* initial_state,
                       int initial_state_dtype, void* final_state, int final_state_dtype,
                       const int64_t* cu_seqlens, int64_t num_seqs, int64_t B, int64_t T,
                       int64_t H, int64_t D, void* stream, int chunk_size, int v_tile);

/*
 * kda_fwd_transposed_state -- kda_fwd with both states in the transposed,
 * key-major layout [num_seqs, H, D(k), D(v)]: element (v, k) of a head's
 * state sits at k * D + v (FlashKDA's alternative state layout, its
 * transpose-state-layout option).  Everything else, including the exact
 * in-place alias, is exactly as kda_fwd; the results equal those of kda_fwd on
 * transposed states bitwise.
 */
int kda_fwd_transposed_state(const void* q, const void* k, const void* v, const void* g,
                             const void* beta, float scale, void* out, const float* A_log,
                             const float* dt_bias, float lower_bound, const void* initial_state,
                             int initial_state_dtype, void* final_state, int final_state_dtype,
                             const int64_t* cu_seqlens, int64_t num_seqs, int64_t B, int64_t T,
                             int64_t H, int64_t D, void* stream);

/*
 * kda_split_workspace_bytes -- bytes of the workspace kda_fwd_split needs.
 *   T_total     tokens of the flattened batch (B * T).
 *   num_seqs    N, as for kda_fwd.
 *   H, D        heads and head dimension; the split runs D = 128 only.
 *   lower_bound, chunk_size  as for kda_fwd_sched (0: automatic chunk length); pass
 *               kda_fwd_split the same chunk_size.
 * One record per slot and head: the prepared operands of one chunk (Qc, Kc, Kr,
 * the solve operands, Mqk and the decay, in the layout the recurrent kernel copies
 * into LDS; 35,840 bytes at 32-token chunks).  A head has floor(T_total / chunk)
 * + num_seqs + 1 slots.  Returns the size, or a negative status
 * (KDA_ERR_BAD_SHAPE, also when a head's records reach 2^31 bytes or the prep
 * kernel's grid of slots times heads workgroups of 512 threads exceeds 2^32 - 1
 * work-items; KDA_ERR_BAD_LOWER_BOUND; KDA_ERR_BAD_SCHEDULE).
 */
int64_t kda_split_workspace_bytes(int64_t T_total, int64_t num_seqs, int64_t H, int64_t D,
                                  float lower_bound, int chunk_size);

/*
 * kda_fwd_split -- kda_fwd as two kernels, the organisation of FlashKDA's
 * prep and recurrent kernels that the FlashInfer PR #4262 summary describes
 * (its workspace of chunk-local matrices and transformed Q and K between them).
 * A token-parallel kernel prepares every chunk of every head (gate, prefix,
 * norms, centred operands, Mqk and the inverted diagonal blocks) and writes it to
 * `workspace`.  The recurrent kernel then reads those records back in chunk order
 * and runs only the state side, on value tiles of v_tile rows.
 *   workspace        caller-owned device memory of at least
 *                    kda_split_workspace_bytes(B * T, num_seqs, H, D, lower_bound,
 *                    chunk_size) bytes (KDA_ERR_BAD_WORKSPACE otherwise,
 *                    KDA_ERR_NULL_ARG when NULL).  It must not overlap any other
 *                    argument (KDA_ERR_BAD_ALIAS).  Its contents on entry do not
 *                    matter and are scratch on return.
 *   workspace_bytes  its size in bytes.
 *   chunk_size       0 (automatic) or a forced chunk length, as for kda_fwd_sched.
 *   v_tile           0 (automatic, as for kda_fwd), 128, or 64 at 32-token chunks;
 *                    other schedules are KDA_ERR_BAD_SCHEDULE, as is D != 128.
 * The results are bitwise those of kda_fwd_sched with the same chunk length and
 * value tile: both
 * kernels run the fused kernel's own preparation and state-side code.  Both are
 * enqueued on `stream`.  Everything else is exactly as kda_fwd.
 */
int kda_fwd_split(const void* q, const void* k, const void* v, const void* g, const void* beta,
                  float scale, void* out, const float* A_log, const float* dt_bias,
                  float lower_bound, const void* initial_state, int initial_state_dtype,
                  void* final_state, int final_state_dtype, const int64_t* cu_seqlens,
                  int64_t num_seqs, int64_t B, int64_t T, int64_t H, int64_t D, void* stream,
                  void* workspace, int64_t workspace_bytes, int chunk_size, int v_tile);

/*
 * kda_fwd_split_noalloc -- kda_fwd_split for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  The workspace is the library's own scratch: a static device
 * array of kda_split_noalloc_max_bytes() bytes (64 MiB) that each GPU the library
 * runs on holds until the process ends.  Its address is resolved once per device,
 * on the first call with that device current; the call allocates nothing.
 *   chunk_size, v_tile  as for kda_fwd_split.
 * A call whose kda_split_workspace_bytes(B * T, num_seqs, H, D, lower_bound,
 * chunk_size) exceeds the scratch returns KDA_ERR_SCRATCH_TOO_SMALL before
 * anything is enqueued (for example 96 heads hold 19 records of 35,840 bytes each:
 * T_total + 32 num_seqs below about 576 tokens at 32-token chunks).  Every call on a
 * GPU shares that GPU's array and leaves its records there; calls that overlap in
 * time on one GPU (concurrent streams, or threads) race on it and must be
 * serialised by the caller.  Nothing in the array needs to start at zero: every
 * record is written by the call's prep kernel before its recurrent kernel reads it.
 * The results are bitwise those of kda_fwd_split.  Returns KDA_OK, a kda_fwd_split
 * status, KDA_ERR_SCRATCH_TOO_SMALL, or KDA_ERR_HIP if the scratch address cannot
 * be resolved.
 */
int kda_fwd_split_noalloc(const void* q, const void* k, const void* v, const void* g,
                          const void* beta, float scale, void* out, const float* A_log,
                          const float* dt_bias, float lower_bound, const void* initial_state,
                          int initial_state_dtype, void* final_state, int final_state_dtype,
                          const int64_t* cu_seqlens, int64_t num_seqs, int64_t B, int64_t T,
                          int64_t H, int64_t D, void* stream, int chunk_size, int v_tile);

/* kda_split_noalloc_max_bytes -- bytes of kda_fwd_split_noalloc's scratch (64 MiB). */
int64_t kda_split_noalloc_max_bytes(void);

/*
 * kda_longest_first -- writes the longest-first order of a packed batch for
 * kda_fwd_ordered: seq_order[i] is the index of the sequence with the i-th
 * largest length cu_seqlens[n+1] - cu_seqlens[n] (equal lengths keep their
 * index order).  One small kernel on `stream`; the host reads nothing.
 *   cu_seqlens  int64 [num_seqs + 1] device array (as for kda_fwd).
 *   num_seqs    1 .. 8192 (KDA_ERR_BAD_VARLEN otherwise).
 *   seq_order   int32 [num_seqs] device array, written; must not overlap
 *               cu_seqlens (KDA_ERR_BAD_ALIAS).
 * Returns KDA_OK, KDA_ERR_BAD_VARLEN (checked first), KDA_ERR_NULL_ARG,
 * KDA_ERR_BAD_ALIAS or KDA_ERR_HIP.  An order depends only on the lengths, so one computation can
 * serve every layer of a model that shares the batch.
 */
int kda_longest_first(const int64_t* cu_seqlens, int64_t num_seqs, int32_t* seq_order,
                      void* stream);

/*
 * kda_fwd_check -- the host-side validation of kda_fwd_sched on its own: the
 * same arguments without the stream, returns the status kda_fwd_sched would
 * return before launching.  Pure host code (pointer values are compared, never
 * dereferenced); needs no GPU.
 */
int kda_fwd_check(const void* q, const void* k, const void* v, const void* g, const void* beta,
                  float scale, const void* out, const float* A_log, const float* dt_bias,
                  float lower_bound, const void* initial_state, int initial_state_dtype,
                  const void* final_state, int final_state_dtype, const int64_t* cu_seqlens,
                  int64_t num_seqs, int64_t B, int64_t T, int64_t H, int64_t D, int chunk_size,
                  int v_tile);

/*
 * kda_chunk_anchor -- the fixed exponent anchor Ca (base 2) the library centres a
 * chunk's operands on: the middle of the chunk's decay span,
 * chunk_size * lower_bound * log2(e) / 2 (-118 for one-token chunks whose span
 * exceeds 236, where the decay is floored).  For 32-token chunks this is section 2
 * of the PR #4262 summary's 16 * lower_bound * log2(e) (about -115.42 for
 * lower_bound = -5).  The centred operands then reach 2^(-Ca) at most and keep
 * as much room above the bf16 normal minimum as below its maximum, which the
 * most strongly decayed rows of a chunk need.  Pure host function.
 */
float kda_chunk_anchor(float lower_bound, int chunk_size);

/* ------------------------------------------------------------------------------
 * Serving operators: the single-token forms of the recurrences, on states kept in a
 * pool, and the other layers of a model that mixes KDA with them.  The conventions of
 * the header apply, and for these:
 *   - pointers are 16-byte aligned (KDA_ERR_BAD_LAYOUT), fp32 and int64 arrays
 *     naturally aligned;
 *   - a *_row argument is the distance in elements between the rows of consecutive
 *     tokens of that tensor (heads * D when it is contiguous; more when it is a view of
 *     wider rows, as of one projection's output): a multiple of 8 and at least
 *     heads * D (KDA_ERR_BAD_LAYOUT).  Heads and D are contiguous inside a row;
 *   - an output must not overlap any input or other output (KDA_ERR_BAD_ALIAS; the
 *     bytes from a strided tensor's first row to its last count as that tensor).
 * Each has a *_check function: the same arguments without the stream, returns the status
 * the operator would return before launching; host code that needs no GPU.
 * ------------------------------------------------------------------------------ */

/*
 * kda_step -- one token of each of N requests through the recurrence of kda_fwd, on
 * states kept in a pool.
 *   q, k, v, g     bf16 [N, H, D], contiguous; beta bf16 [N, H] (logits).
 *   out            bf16 [N, H, D].
 *   scale, A_log, dt_bias, lower_bound  as for kda_fwd (any finite lower bound below 0;
 *                  decay factors below the fp32 range are zero).
 *   state          [num_slots, H, D(v), D(k)] of state_dtype: the layout of kda_fwd's
 *                  final_state, so a prompt's final states are slots of the pool.
 *                  The update is fp32; out uses the fp32 state, before a bf16 slot is
 *                  rounded.
 *   slot_in        int64 [N] device array: request n's state is slot slot_in[n]; NULL: n.
 *                  An index outside [0, num_slots) reads zeros (a request's first token).
 *   slot_out       int64 [N] device array: where the new state goes; NULL: slot_in.  An
 *                  index outside [0, num_slots) stores no state (a padded row; its out row
 *                  is still written).  Slots that no request names are left as they were.
 *                  Several requests may read one slot; a slot that a request writes must be
 *                  named by no other request of the call (its contents, and the results of
 *                  the others that read it, are unspecified otherwise).
 *   N, H, D        requests (0: nothing is done), heads, D in {32, 64, 128};
 *                  N * H < 2^24.  Without slot_in N <= num_slots.
 * One kernel on `stream`.  Returns KDA_OK or a negative status.
 */
int kda_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
             float scale, void* out, const float* A_log, const float* dt_bias, float lower_bound,
             void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
             const int64_t* slot_out, int64_t N, int64_t H, int64_t D, void* stream);
int kda_step_check(const void* q, const void* k, const void* v, const void* g, const void* beta,
                   float scale, const void* out, const float* A_log, const float* dt_bias,
                   float lower_bound, const void* state, int state_dtype, int64_t num_slots,
                   const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H,
                   int64_t D);

/*
 * kda_la_step -- one token of each of N requests through linear attention with one
 * decay per head:
 *
 *     S = exp(g_n + decay) S + v k^T,    out = scale S q       (S: V x K)
 *
 *   q, k           bf16 [N, Hk, D]; head h of H uses q/k head h / (H / Hk).
 *   v, out         bf16 [N, H, D] (out contiguous).
 *   g              fp32 [N, H] natural-log decays, contiguous, or NULL.
 *   decay          fp32 [H] natural-log decays, or NULL (both NULL: no decay).  A sum
 *                  g + decay above zero counts as zero.
 *   state, slots, N, D  as for kda_step.  H % Hk == 0 (KDA_ERR_BAD_SHAPE).
 * One kernel on `stream`.
 */
int kda_la_step(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                int64_t v_row, const float* g, const float* decay, float scale, void* out,
                void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
                const int64_t* slot_out, int64_t N, int64_t H, int64_t Hk, int64_t D,
                void* stream);
int kda_la_step_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                      int64_t v_row, const float* g, const float* decay, float scale,
                      const void* out, const void* state, int state_dtype, int64_t num_slots,
                      const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H,
                      int64_t Hk, int64_t D);

/*
 * kda_la_fwd -- prompts through linear attention with one decay per head.  Per sequence
 * and head the V x K state S evolves token by token as
 *
 *     S = exp(g_t + decay) S + v_t k_t^T,    out_t = scale S q_t
 *
 * evaluated in chunks of 64 tokens with bf16 matrix-core products and an fp32 state.
 *   q, k           bf16 [B, T, Hk, D] with row strides q_row, k_row (below 2^24); head h of
 *                  H uses q/k head h / (H / Hk).  Batch rows follow each other: token t of
 *                  batch row b is row b * T + t.
 *   v              bf16 [B, T, H, D], row stride v_row (below 2^24).
 *   out            bf16 [B, T, H, D], contiguous.
 *   g              fp32 [B, T, H] natural-log decays, contiguous, or NULL.
 *   decay          fp32 [H] natural-log decays, or NULL (both NULL: no decay).  A sum
 *                  g + decay above zero counts as zero, and below -87.3 (a factor of
 *                  2^-126, minus infinity included) as -87.3; NaN reaches the outputs of
 *                  its head's chunk and all that follow.
 *   initial_state, final_state, cu_seqlens, num_seqs, B, T  as for kda_fwd, the in-place
 *                  state alias included.  An empty sequence passes its state through.
 *   H, Hk, D       H % Hk == 0, H * D < 2^24, D in {32, 64, 128}.  (num_seqs + 8) * H at
 *                  most 2^23 - 8, and the same for a workspace's slots (KDA_ERR_BAD_SHAPE).
 *   segment        0 (automatic), or tokens per segment: a multiple of 64, at most 2^20
 *                  (KDA_ERR_BAD_SCHEDULE).  A few long sequences do not fill the device
 *                  one workgroup per (sequence, head): their tokens are then split into
 *                  segments, whose own sums are formed first (four kernels instead of
 *                  one).  The state before a segment is then a sum in another order
 *                  (fp32 roundings of the state).
 *   workspace      caller-owned device memory, 16-byte aligned, of at least
 *                  kda_la_workspace_bytes(B * T, num_seqs, H, D, segment) bytes
 *                  (KDA_ERR_BAD_WORKSPACE), scratch on return: calls that may overlap in
 *                  time need one each.  With segment 0 it may be NULL: no segments then.
 * Roundings, relative to the sum of the absolute values of an output's (or state element's)
 * terms: the scores times their weights and the state as an operand of S q are rounded to bf16
 * once each, or held in two bf16 parts in calls of B * T * H <= 2048; the weighted v of the
 * state's update to 2^-17, or to 2^-25 in those calls and where final_state is fp32.  So a
 * sequence's results depend, by these roundings, on the size of its call, on segments (which the
 * automatic choice takes from the whole batch), and on final_state's type.  They never depend
 * on what the other sequences hold, and a call repeats itself bit for bit.
 * Infinities and NaN of one token reach outputs of that token and later ones of its sequence
 * only: those of q its own, of k all of its heads', of v its value's (as infinities or NaN,
 * whatever the decays since, in segments or without).
 */
int kda_la_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
               int64_t v_row, const float* g, const float* decay, float scale, void* out,
               const void* initial_state, int initial_state_dtype, void* final_state,
               int final_state_dtype, const int64_t* cu_seqlens, int64_t num_seqs, int64_t B,
               int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t segment, void* workspace,
               int64_t workspace_bytes, void* stream);
int kda_la_fwd_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                     int64_t v_row, const float* g, const float* decay, float scale,
                     const void* out, const void* initial_state, int initial_state_dtype,
                     const void* final_state, int final_state_dtype, const int64_t* cu_seqlens,
                     int64_t num_seqs, int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t D,
                     int64_t segment, const void* workspace, int64_t workspace_bytes);

/*
 * kda_la_workspace_bytes -- bytes of kda_la_fwd's workspace for T_total = B * T tokens of
 * num_seqs sequences: zero when the (automatic) schedule uses no segments, else one fp32
 * state and decay per head for each of T_total / segment + num_seqs + 1 slots.  Returns the
 * size or a negative status (KDA_ERR_BAD_SHAPE, KDA_ERR_BAD_SCHEDULE).
 */
int64_t kda_la_workspace_bytes(int64_t T_total, int64_t num_seqs, int64_t H, int64_t D,
                               int64_t segment);

/*
 * kda_attn_fwd -- causal softmax attention with grouped heads, for the layers of a model
 * that are not recurrent: whole prompts, prompts that continue earlier keys, and single
 * (or a few drafted) tokens over key/value caches.  Query i of a sequence with Lq queries
 * and Lk keys sees keys j <= i + Lk - Lq, its queries being the last Lq of its positions:
 *
 *     out_i = sum_j softmax_j(scale q_i . k_j) v_j,    lse_i = log sum_j exp(scale q_i . k_j)
 *
 * and a query that sees no key (Lk < Lq, or no keys), or only scores of minus infinity, gets out
 * 0 and lse minus infinity.
 *   q              bf16 [Bq, Tq, Hq, D], row stride q_row (below 2^24).
 *   k, v           bf16 [Bk, Tk, Hk, D], row strides k_row, v_row (below 2^24); query head h
 *                  uses key/value head h / (Hq / Hk).  Batch rows follow each other: token t
 *                  of batch row b is row b * T + t.
 *   scale          not negative; scale log2(e) a finite float (scale up to 2.35e38;
 *                  KDA_ERR_BAD_SCALE).  Zero gives the mean of the visible v.
 *   out            bf16 [Bq, Tq, Hq, D], contiguous.
 *   lse            fp32 [Bq, Tq, Hq], or NULL.
 *   cu_seqlens_q   int64 [num_seqs + 1] device array (Bq == 1): sequence n's queries are
 *                  tokens [cu[n], cu[n+1]); or NULL (Bq == num_seqs): batch row n, Tq each.
 *   cu_seqlens_k   the same for keys (Bk == 1); or NULL (Bk == num_seqs): batch row n, of
 *                  which the first k_lens[n] keys are in use.
 *   k_lens         int64 [num_seqs] device array, clamped into [0, Tk]; NULL: all Tk.  Not
 *                  with cu_seqlens_k (KDA_ERR_BAD_VARLEN).  Keys behind a sequence's last
 *                  are never used, whatever they hold.
 *                  Offsets as for kda_fwd's cu_seqlens: not checked on the host, clamped on
 *                  the device.  Query tokens outside every sequence keep their out and lse
 *                  rows as they were.
 *   Hq, Hk, D      Hq % Hk == 0, D in {64, 128}.  Tk <= 2^30, Tq * Hq / Hk <= 2^30.
 *   splits         0 (automatic), or 1 .. 64 parts of each row's keys
 *                  (KDA_ERR_BAD_SCHEDULE): few rows over long keys fill the device only
 *                  when several workgroups share a row.  Each writes a partial result and a
 *                  second kernel joins them.
 *   workspace      caller-owned device memory, 16-byte aligned, of at least
 *                  kda_attn_workspace_bytes(num_seqs, Bq, Tq, Bk, Tk, Hq, Hk, D, splits)
 *                  bytes (KDA_ERR_BAD_WORKSPACE), scratch on return: calls that may overlap
 *                  in time need one each.  With splits 0 it may be NULL: one part then.
 * Scores and sums are fp32.  For their product with v probabilities are rounded to bf16 once, or
 * held in two bf16 parts in calls of at most 64 rows (query tokens times Hq / Hk) a sequence on
 * average; splits sum in another order.  A sequence's results depend on its call by these
 * roundings, relative to the sum of the absolute values of its terms, and a call repeats itself
 * bit for bit.
 * Infinities and NaN reach the outputs of the queries that see them and no others.
 */
int kda_attn_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                 int64_t v_row, float scale, void* out, float* lse, const int64_t* cu_seqlens_q,
                 const int64_t* cu_seqlens_k, const int64_t* k_lens, int64_t num_seqs, int64_t Bq,
                 int64_t Tq, int64_t Bk, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D,
                 int64_t splits, void* workspace, int64_t workspace_bytes, void* stream);
int kda_attn_fwd_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                       int64_t v_row, float scale, const void* out, const float* lse,
                       const int64_t* cu_seqlens_q, const int64_t* cu_seqlens_k,
                       const int64_t* k_lens, int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Bk,
                       int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t splits,
                       const void* workspace, int64_t workspace_bytes);

/*
 * kda_attn_workspace_bytes -- bytes of kda_attn_fwd's workspace: zero when the (automatic)
 * schedule does not split the keys, else splits * Bq * Tq * Hq * (D + 2) floats.  Returns
 * the size or a negative status.
 */
int64_t kda_attn_workspace_bytes(int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Bk, int64_t Tk,
                                 int64_t Hq, int64_t Hk, int64_t D, int64_t splits);

/* ------------------------------------------------------------------------------
 * What such layers call around their attention and recurrences: norms with the block's gate and
 * the residual sum, rotary positions, and caches of keys and values in 4 bits with the attention
 * that reads them.  The conventions of the serving operators apply.
 * ------------------------------------------------------------------------------ */

/*
 * kda_norm -- the norms before and after a block, with its gate, the residual sum and its
 * scale, in one pass over the rows.  For each row of W channels, every part optional:
 *
 *     u = x
 *     u = u / sqrt(mean(u^2) + eps) post_weight        over each group of `group` channels
 *     u = u sigmoid(gate), or u gate sigmoid(gate)
 *     h = residual + residual_scale u                  -> residual_out     (without one h = u)
 *     out = h / sqrt(mean(h^2) + eps) weight           over the row        (without one out = h)
 *
 *   x              bf16 [R, W], row stride x_row.
 *   gate           bf16 [R, W], row stride gate_row, or NULL; gate_fn KDA_GATE_SIGMOID or
 *                  KDA_GATE_SILU (KDA_ERR_BAD_DTYPE).
 *   post_weight    [group] of weight_dtype, or NULL.  group: W, or 32, 64, 128, 256 or 512 and a
 *                  divisor of W (KDA_ERR_BAD_SHAPE): a head's output norm shares its weights
 *                  among the heads.
 *   weight         [W] of weight_dtype, or NULL.
 *   eps            finite, not negative (KDA_ERR_BAD_SCALE).
 *   residual, residual_out  [R, W] of residual_dtype, contiguous, both or neither
 *                  (KDA_ERR_NULL_ARG).  They may be exactly the same allocation (in place).
 *   residual_scale finite.
 *   out            bf16 [R, W], contiguous; may be NULL with a residual and without a weight.
 *   R, W           rows (0: nothing is done); W a multiple of 8, 8 .. 16384.  R below
 *                  2^32 / 4096 (KDA_ERR_BAD_SHAPE).
 * At least one of post_weight, gate, weight and residual (KDA_ERR_NULL_ARG).
 * Everything between loads and stores is fp32; the second norm takes h before residual_out is
 * rounded.  Squares and their sums are fp32: a group's L2 norm stays below 1.8e19, and values
 * whose squares underflow count as zero beside eps.  With eps zero squares below 2^-126 lose
 * digits, and a group of nothing but zeros and such values gives NaN and infinities.  One kernel
 * on `stream`.
 */
int kda_norm(const void* x, int64_t x_row, const void* gate, int64_t gate_row, int gate_fn,
             const void* post_weight, int64_t group, const void* weight, int weight_dtype,
             float eps, const void* residual, void* residual_out, int residual_dtype,
             float residual_scale, void* out, int64_t R, int64_t W, void* stream);
int kda_norm_check(const void* x, int64_t x_row, const void* gate, int64_t gate_row, int gate_fn,
                   const void* post_weight, int64_t group, const void* weight, int weight_dtype,
                   float eps, const void* residual, const void* residual_out, int residual_dtype,
                   float residual_scale, const void* out, int64_t R, int64_t W);

/*
 * kda_rope -- rotary positions of queries and keys: each pair (a, b) of a head's first rot
 * channels is turned by position times the pair's frequency,
 *
 *     (a, b) -> amplitude (a cos - b sin, a sin + b cos),
 *
 * the channels behind rot stay as they are.  inverse turns back (the gradient of the turn, or a
 * key on its way to another position).
 *   q, q_out       bf16 [B, T, Hq, D], row strides q_row, q_out_row.  In place where pointer and
 *                  row stride are the same; any other shared byte is refused
 *                  (KDA_ERR_BAD_ALIAS).  Rows of one stride in other columns of the same wider
 *                  rows, as of one projection, share none.
 *   k, k_out       the same with Hk heads; Hk 0 (NULL): queries alone.
 *   freqs          float64 [rot / 2], radians per position: plain powers of a base, or scaled for
 *                  long contexts.  Their product with the position is formed and reduced to a
 *                  turn in 64 bits, its sine and cosine and the products are fp32.
 *   rot            even, 2 .. D (KDA_ERR_BAD_SHAPE).  D a multiple of 8, up to 1024.
 *   amplitude      finite (KDA_ERR_BAD_SCALE); of the turned channels only.
 *   interleaved    0: pairs (i, i + rot / 2); else pairs (2 i, 2 i + 1).
 *   positions      int64 [B, T] device array, or NULL: token t of sequence n is at position
 *                  offsets[n] + t (int64 [num_seqs], NULL: 0), sequences as for kda_fwd
 *                  (cu_seqlens, num_seqs, B, T).  positions exclude the other two
 *                  (KDA_ERR_BAD_VARLEN).  Tokens outside every sequence keep their outputs.
 *   B * T          below 2^24 (KDA_ERR_BAD_SHAPE).
 * One kernel on `stream`.
 */
int kda_rope(const void* q, int64_t q_row, void* q_out, int64_t q_out_row, const void* k,
             int64_t k_row, void* k_out, int64_t k_out_row, const double* freqs, int64_t rot,
             float amplitude, int interleaved, int inverse, const int64_t* positions,
             const int64_t* offsets, const int64_t* cu_seqlens, int64_t num_seqs, int64_t B,
             int64_t T, int64_t Hq, int64_t Hk, int64_t D, void* stream);
int kda_rope_check(const void* q, int64_t q_row, const void* q_out, int64_t q_out_row,
                   const void* k, int64_t k_row, const void* k_out, int64_t k_out_row,
                   const double* freqs, int64_t rot, float amplitude, int interleaved, int inverse,
                   const int64_t* positions, const int64_t* offsets, const int64_t* cu_seqlens,
                   int64_t num_seqs, int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D);

/*
 * Caches in 4 bits.  A block of 32 channels of one token and head shares a power of two 2^e and
 * holds a code for each value: bit 3 the sign, bits 0-2 the magnitude 0, .5, 1, 1.5, 2, 3, 4 or 6
 * (the two-bit-exponent format with a scale per block of 32 that the device converts in
 * hardware).  The scale's byte is e + 127; 255 says that the block held an infinity or NaN, and
 * stands for NaN.  A cache has num_slots slots of Hk heads of cap positions, cap a multiple of 32:
 *   k4             uint8 [num_slots, Hk, cap, D / 2]: two codes a byte, the even channel's low.
 *   v4             uint8 [num_slots, Hk, cap / 32, 16 D]: tiles of 32 positions.  Position
 *                  16 j + 4 i + g of a tile (j < 2, i < 4, g < 4), channel d, two channels a byte:
 *                    D 128: byte 1024 j + 256 g + 16 (d / 8) + 4 i + d % 8 / 2,
 *                    D  64: byte 256 g + 16 (d / 4) + 8 j + 2 i + d % 4 / 2.
 *   ks, vs         uint8 [num_slots, Hk, cap / 32, D / 32, 32]: the scales of the tile's positions
 *                  for each block of channels, position 16 j + 4 i + g at 8 g + 2 i + j.
 * (These places are those of the matrix products' operands: kda_attn4_fwd brings 16 bytes a
 * lane and every lane uses its own, none is exchanged.)  D in {64, 128}; cap up to 2^30.  A slot is
 * contiguous in all four: copying it copies the cache of a request.
 *
 * kda_cache4_put -- new keys and values into such caches: token t of sequence n goes to
 * position offsets[n] + t of slot slots[n].  2^e is the smallest power with
 * max |x| <= 6 2^e over the block (not below 2^-127), a value takes the nearest code of x / 2^e,
 * of two the even one; nothing saturates, and every step is exact.
 *   k, v           bf16 [B, T, Hk, D], row strides k_row, v_row.
 *   k_out, v_out   bf16 [B, T, Hk, D], contiguous, or both NULL: what the codes stand for, for
 *                  attention over the prompt itself with the same keys as later tokens see.  (A
 *                  magnitude from 1.75 2^127 on rounds to infinity.)
 *   offsets        int64 [num_seqs] device array, NULL: 0.  Positions outside [0, cap) are not
 *                  stored (k_out and v_out are).
 *   slots          int64 [num_seqs] device array, NULL: n (num_seqs <= num_slots).  Sequences with
 *                  an index outside [0, num_slots) are not stored.  A slot must not be named by
 *                  two sequences whose positions meet.
 *   cu_seqlens, num_seqs, B, T  as for kda_fwd; tokens outside every sequence are left out.
 * Other positions keep what they hold.  One kernel on `stream`.
 */
int kda_cache4_put(const void* k, int64_t k_row, const void* v, int64_t v_row, void* k4, void* ks,
                   void* v4, void* vs, int64_t num_slots, int64_t cap, void* k_out, void* v_out,
                   const int64_t* offsets, const int64_t* slots, const int64_t* cu_seqlens,
                   int64_t num_seqs, int64_t B, int64_t T, int64_t Hk, int64_t D, void* stream);
int kda_cache4_put_check(const void* k, int64_t k_row, const void* v, int64_t v_row,
                         const void* k4, const void* ks, const void* v4, const void* vs,
                         int64_t num_slots, int64_t cap, const void* k_out, const void* v_out,
                         const int64_t* offsets, const int64_t* slots, const int64_t* cu_seqlens,
                         int64_t num_seqs, int64_t B, int64_t T, int64_t Hk, int64_t D);

/*
 * kda_attn4_fwd -- kda_attn_fwd over caches in 4 bits: the same formulas, masks and limits, with
 * keys and values the products of codes and scales (exact in bf16; beyond its range infinity).
 *   q, q_row, scale, out, lse, cu_seqlens_q, num_seqs, Bq, Tq, Hq, Hk, D  as for kda_attn_fwd.
 *   k4, ks, v4, vs, num_slots, cap  the caches.
 *   k_lens         int64 [num_seqs] device array, clamped into [0, cap]; NULL: all cap.  Positions
 *                  behind a sequence's last are never used, whatever they hold.
 *   slots          int64 [num_seqs] device array, NULL: n (num_seqs <= num_slots).  Several
 *                  sequences may read one slot.  An index outside [0, num_slots) has no keys.
 *   part           0 (automatic), or keys per part: a multiple of 32 with at most 64 parts in
 *                  cap (KDA_ERR_BAD_SCHEDULE).  Each part of a row's keys has a workgroup of its
 *                  own, and a second kernel joins them.  With many rows (prompts: more than 448
 *                  (query token, head) pairs a sequence and key/value head on average, and enough
 *                  of them to fill the device many times over) the automatic choice expands the
 *                  caches in use to bf16 once, where that takes 8 GiB at most, and runs
 *                  kda_attn_fwd's kernels over them.  The choice goes by the whole call, so a
 *                  prompt among many single tokens, or these beside a large prompt, are faster in
 *                  a call of their own; and the expanded caches' size by their capacity, not by
 *                  k_lens.
 *   workspace      caller-owned device memory, 16-byte aligned, of at least
 *                  kda_attn4_workspace_bytes(num_seqs, Bq, Tq, cap, Hq, Hk, D, part) bytes
 *                  (KDA_ERR_BAD_WORKSPACE), scratch on return: calls that may overlap in time
 *                  need one each.  With part 0 it may be NULL: one part straight from the caches
 *                  then.
 * Scores and sums are fp32.  For their product with v probabilities are held in two bf16 parts, or
 * rounded to bf16 once where the caches are expanded; parts sum in another order.  A sequence's
 * results depend on its call by these roundings, relative to the sum of the absolute values of its
 * terms, and a call repeats itself bit for bit.  Infinities and NaN reach the outputs of the
 * queries that see them and no others.
 */
int kda_attn4_fwd(const void* q, int64_t q_row, const void* k4, const void* ks, const void* v4,
                  const void* vs, int64_t num_slots, int64_t cap, float scale, void* out,
                  float* lse, const int64_t* cu_seqlens_q, const int64_t* k_lens,
                  const int64_t* slots, int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Hq,
                  int64_t Hk, int64_t D, int64_t part, void* workspace, int64_t workspace_bytes,
                  void* stream);
int kda_attn4_fwd_check(const void* q, int64_t q_row, const void* k4, const void* ks,
                        const void* v4, const void* vs, int64_t num_slots, int64_t cap,
                        float scale, const void* out, const float* lse,
                        const int64_t* cu_seqlens_q, const int64_t* k_lens, const int64_t* slots,
                        int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Hq, int64_t Hk,
                        int64_t D, int64_t part, const void* workspace, int64_t workspace_bytes);

/*
 * kda_attn4_workspace_bytes -- bytes of kda_attn4_fwd's workspace: zero when the keys are one part,
 * parts * Bq * Tq * Hq * (D + 2) floats for several, or num_seqs * cap * Hk * D * 4 bytes for
 * expanded caches, with their lengths and the parts of kda_attn_fwd.  Returns the size or a
 * negative status.
 */
int64_t kda_attn4_workspace_bytes(int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t cap,
                                  int64_t Hq, int64_t Hk, int64_t D, int64_t part);

/* kda_status_string -- a static, human-readable name for a status code. */
const char* kda_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
