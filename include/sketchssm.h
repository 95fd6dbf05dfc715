/*
 * sketchssm.h -- C ABI of libsketchssm.so: the SketchSSM windowed
 * linear-attention decode path on AMD Instinct MI355X (gfx950).
 *
 * Method (SketchSSM pages: readsearch.ai listing of arXiv 2609.33051,
 * "SketchSSM: Write to the Full State, Read from a Compact Sketch", Abstract;
 * agihunt.info summary, "Confirmed" bullets "Mechanism details" and
 * "Error control"):
 *   - keys, values and gates of the current window are buffered and the full
 *     recurrent state S (d_k x d_v, fp32, one per (sequence, head) unit) is
 *     written once per window;
 *   - the same pass that writes S also stores a compact sketch: the outputs of
 *     S for r fixed, offline basis vectors b_1..b_r;
 *   - every decode step in between reads only the sketch and the buffer and
 *     rebuilds the output from query-dependent coefficients; the sketch's
 *     approximation error never reaches S.
 *
 * Notation (per unit). Token i of the window has key k_i, value v_i, gate(s)
 * and, for the delta rules, a write strength beta_i. Its transition matrix M_i
 * and update S <- M_i S + b_i k_i v_i^T are:
 *   SSM_MAMBA2 : M = a I                         , b = 1      (scalar decay a)
 *   SSM_GDN    : M = alpha (I - beta k k^T)      , b = beta   (scalar gate alpha)
 *   SSM_KDA    : M = (I - beta k k^T) Diag(alpha), b = beta   (per-channel gate alpha[d_k])
 * With S_win the state at the window start, after tau buffered tokens
 *   S_tau = A S_win + R,  A = M_tau ... M_1,  R = sum_i M_tau..M_{i+1} b_i k_i v_i^T,
 * and the exact output is y = S_tau^T q = S_win^T (A^T q) + R^T q.
 * The sketch read replaces S_win^T q~ (q~ = A^T q) by Sk^T c with c = B q~.
 *
 * Memory layouts (row-major, every pointer a DEVICE pointer owned by the
 * caller; the library keeps no pointer after a call returns):
 *   state   S   fp32  [N][H][d_k][d_v]
 *   sketch  Sk  fp32 or bf16 (ssm_dims.sketch_dtype)  [N][H][r][d_v]
 *                                        row m = S^T b_m (the output for basis vector b_m)
 *   basis   B   fp32  [H][r][d_k]        row m = b_m; rows orthonormal (not checked)
 *   k_buf       in    [N][H][W][d_k]     window buffer, slot i = token i+1 of the window
 *   v_buf       in    [N][H][W][d_v]
 *   decay_buf   fp32  [N][H][W] (Mamba-2 a, GDN alpha) or [N][H][W][d_k] (KDA alpha)
 *   beta_buf    fp32  [N][H][W] (GDN, KDA); NULL for Mamba-2
 *   q, k_t      in    [N][H][d_k]        one token per unit
 *   v_t         in    [N][H][d_v]
 *   decay_t     fp32  [N][H] or [N][H][d_k];  beta_t fp32 [N][H] or NULL
 *   y           fp32  [N][H][d_v]
 * "in" is bf16 or fp32 as ssm_dims.in_dtype says. A unit is (n, h), flat
 * index n*H + h.
 *
 * Calls are asynchronous: arguments are checked on the host, then the work is
 * enqueued on `stream` (a hipStream_t; NULL = the default stream). No call
 * allocates, frees or synchronises. Invalid arguments return a non-zero
 * status before anything is enqueued; a failed launch returns SSM_E_LAUNCH.
 * Faults inside a kernel surface at the caller's next synchronisation. No C++
 * exception crosses this interface. The detail of the last failure on the
 * calling thread is in ssm_last_error().
 *
 * Supported shapes: d_k in {16, 32, 64, 128}; d_v in {16, 32, 64, 128}; 1 <= W <= 16;
 * 1 <= r <= min(d_k, 32); N >= 0 (N = 0 is a no-op); H >= 1; N*H < 2^24, which
 * keeps every grid (one workgroup of up to 256 threads per unit) below 2^32
 * threads. Every pointer must be 16-byte aligned. Outputs must not overlap any
 * input of the same call.
 */
#ifndef SKETCHSSM_H
#define SKETCHSSM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 5

typedef enum { SSM_MAMBA2 = 0, SSM_GDN = 1, SSM_KDA = 2 } ssm_rule;
typedef enum { SSM_IN_BF16 = 0, SSM_IN_F32 = 1 } ssm_in_dtype;
/* Storage type of the sketch. The pages leave its precision open: fp32 is the
 * default; bf16 halves the sketch bytes every decode step reads. A bf16 sketch
 * is computed in fp32 and rounded to nearest, ties to even, when it is stored. */
typedef enum { SSM_SKETCH_F32 = 0, SSM_SKETCH_BF16 = 1 } ssm_sketch_dtype;

typedef enum {
  SSM_OK = 0,
  SSM_E_NULL = 1,   /* a required pointer is NULL                          */
  SSM_E_SHAPE = 2,  /* unsupported or inconsistent dimensions               */
  SSM_E_ALIGN = 3,  /* a pointer is not 16-byte aligned                     */
  SSM_E_RANGE = 4,  /* an enum, a token count, tau or slot is out of range,
                       or beta is given for Mamba-2                         */
  SSM_E_ALIAS = 5,  /* an output overlaps an input                          */
  SSM_E_LAUNCH = 6  /* the HIP runtime refused the launch                   */
} ssm_status;

typedef struct {
  int32_t rule;      /* ssm_rule                          */
  int32_t in_dtype;  /* ssm_in_dtype of q, k, v           */
  int32_t batch;     /* N sequences                       */
  int32_t heads;     /* H heads                           */
  int32_t d_k;       /* key / state rows                  */
  int32_t d_v;       /* value / state columns             */
  int32_t window;    /* W buffered tokens per state write */
  int32_t rank;      /* r basis vectors (sketch rows)     */
  int32_t sketch_dtype; /* ssm_sketch_dtype of the sketch (0: fp32) */
} ssm_dims;

/* SSM_ABI_VERSION of the library. */
int32_t ssm_abi_version(void);

/* Static text for a status code. */
const char* ssm_status_string(int32_t status);

/* Detail of the last non-OK status returned on the calling thread ("" if none). */
const char* ssm_last_error(void);

/*
 * Token buffering. Copies the current token of every unit into window slot
 * `slot` (0-based, 0 <= slot < W): k_t -> k_buf, v_t -> v_buf,
 * decay_t -> decay_buf, beta_t -> beta_buf (beta_t and beta_buf NULL for
 * Mamba-2). Source: the pages' buffering of keys and values between state
 * writes (readsearch.ai listing, Abstract, on ReplaySSM; agihunt.info
 * "Confirmed", background bullet).
 */
ssm_status ssm_buffer_append(const ssm_dims* d,
                             const void* k_t, const void* v_t,
                             const float* decay_t, const float* beta_t,
                             void* k_buf, void* v_buf, float* decay_buf, float* beta_buf,
                             int32_t slot, void* stream);

/*
 * Window update fused with the sketch refresh. For every unit: reads S once,
 * applies the first n_tokens buffered tokens in order (S <- M_i S + b_i k_i v_i^T),
 * writes S back (only if n_tokens > 0), then, if `sketch` is not NULL, stores
 * Sk = B S (row m = S^T b_m) from the updated state. n_tokens = 0 with a sketch
 * is the refresh-only pass that creates the first sketch; sketch = NULL (basis
 * may then be NULL) is a plain windowed update with no refresh.
 * 0 <= n_tokens <= W. Source: readsearch.ai listing, Abstract (one full-state
 * read per update precomputes the basis outputs); agihunt.info "Error control"
 * (the full state is updated once per window and the sketch is refreshed in
 * the same kernel).
 * Outputs: state (in/out), sketch. Inputs: basis, the buffers.
 */
ssm_status ssm_window_update_refresh(const ssm_dims* d,
                                     float* state, void* sketch, const float* basis,
                                     const void* k_buf, const void* v_buf,
                                     const float* decay_buf, const float* beta_buf,
                                     int32_t n_tokens, void* stream);

/*
 * Sketch decode step (the per-step read). tau (1 <= tau <= W) tokens of the
 * window are valid, the current token included. For every unit:
 *   walk the buffer newest to oldest from u = q:  s_i = k_i . u,
 *   intra += b_i s_i v_i,  u <- M_i^T u;  then q~ = u, c = B q~ and
 *   y = Sk^T c + intra.
 * Reads only the sketch, the basis, q and the buffer; never the state.
 * Token append, fused: if k_t is not NULL, the current token (k_t, v_t,
 * decay_t, beta_t) is first written into slot tau-1 of the buffer and used
 * from there; if k_t is NULL, slot tau-1 must already hold it and v_t,
 * decay_t, beta_t must be NULL too. The buffers are written only in the
 * fused case. Source: readsearch.ai listing, Abstract (each decode step
 * combines the sketch vectors with query-dependent coefficients);
 * agihunt.info "Mechanism details" (within a window only the queries vary).
 * Output: y. The sketch and the state are never written.
 */
ssm_status ssm_sketch_decode_step(const ssm_dims* d,
                                  const void* sketch, const float* basis, const void* q,
                                  const void* k_t, const void* v_t,
                                  const float* decay_t, const float* beta_t,
                                  void* k_buf, void* v_buf, float* decay_buf, float* beta_buf,
                                  int32_t tau, float* y, void* stream);

/*
 * Exact full-read decode step (the comparison path: the buffered read that
 * still reads all of S each step; readsearch.ai listing, Abstract, on
 * ReplaySSM). Same walk as ssm_sketch_decode_step, then
 * y = S_win^T q~ + intra, reading the whole window-start state S_win = state.
 * Token append works as in ssm_sketch_decode_step. Output: y.
 */
ssm_status ssm_full_read_decode_step(const ssm_dims* d,
                                     const float* state, const void* q,
                                     const void* k_t, const void* v_t,
                                     const float* decay_t, const float* beta_t,
                                     void* k_buf, void* v_buf, float* decay_buf, float* beta_buf,
                                     int32_t tau, float* y, void* stream);

/*
 * Heterogeneous sketch ranks per head (the pages report an average sketch rank
 * of 8: agihunt.info "Results"), for ssm_window_update_refresh_ranked and
 * ssm_sketch_decode_step_ranked. rank_offsets is a HOST array of H + 1 int32
 * prefix offsets: head h has rank r_h = rank_offsets[h+1] - rank_offsets[h],
 * 1 <= r_h <= min(d_k, 32), rank_offsets[0] = 0, H <= 256; the array is read
 * during the call only. With R = rank_offsets[H]:
 *   basis   fp32 [R][d_k]       rows rank_offsets[h] .. +r_h are head h's basis
 *   sketch  [N][R][d_v] (fp32 or bf16) rows rank_offsets[h] .. +r_h of sequence n are
 *                               the outputs of head h's basis vectors
 * d->rank must still be a valid rank (the table decides the sizes). Every other
 * argument and behaviour is that of the uniform-rank entry point.
 */
ssm_status ssm_window_update_refresh_ranked(const ssm_dims* d, const int32_t* rank_offsets,
                                            float* state, void* sketch, const float* basis,
                                            const void* k_buf, const void* v_buf,
                                            const float* decay_buf, const float* beta_buf,
                                            int32_t n_tokens, void* stream);

ssm_status ssm_sketch_decode_step_ranked(const ssm_dims* d, const int32_t* rank_offsets,
                                         const void* sketch, const float* basis, const void* q,
                                         const void* k_t, const void* v_t,
                                         const float* decay_t, const float* beta_t,
                                         void* k_buf, void* v_buf, float* decay_buf,
                                         float* beta_buf, int32_t tau, float* y, void* stream);

/*
 * Variable-length batches over a pool of persistent slots (serving with
 * continuous batching: sequences join, leave and sit at different positions
 * of their windows). A call serves d->batch rows; row n uses slot[n] (a DEVICE
 * int32 array, or NULL for slot n) of a pool of num_slots slots:
 *   persistent, indexed by slot: state [num_slots][H][d_k][d_v], sketch
 *     [num_slots][H][r][d_v], k_buf/v_buf/decay_buf/beta_buf [num_slots][H][W]...
 *   per call, indexed by row: q, k_t, v_t, decay_t, beta_t, y [batch][H][...]
 * Per-row counts come from DEVICE int32 arrays:
 *   ssm_window_update_refresh_varlen: n_tokens[n] in [0, W] tokens to apply
 *     (0 = refresh only); any other value skips the row.
 *   ssm_sketch_decode_step_varlen: tau[n] in [1, W] as in ssm_sketch_decode_step;
 *     any other value skips the row (its y is not written).
 * A row whose slot is outside [0, num_slots) is skipped too. Rows of one call
 * must map to distinct slots (calls with repeated slots race); the device
 * arrays are not read on the host. Uniform sketch rank (d->rank). The slot and
 * count arrays need 4-byte alignment; everything else as the lockstep entry
 * points. Source: the pages' setting of large decode batches (readsearch.ai
 * listing, Abstract); the serving schedule itself is not on the pages.
 */
ssm_status ssm_window_update_refresh_varlen(const ssm_dims* d, int32_t num_slots,
                                            const int32_t* slot, const int32_t* n_tokens,
                                            float* state, void* sketch, const float* basis,
                                            const void* k_buf, const void* v_buf,
                                            const float* decay_buf, const float* beta_buf,
                                            void* stream);

ssm_status ssm_sketch_decode_step_varlen(const ssm_dims* d, int32_t num_slots,
                                         const int32_t* slot, const int32_t* tau,
                                         const void* sketch, const float* basis, const void* q,
                                         const void* k_t, const void* v_t,
                                         const float* decay_t, const float* beta_t,
                                         void* k_buf, void* v_buf, float* decay_buf,
                                         float* beta_buf, float* y, void* stream);

/*
 * One serving decode step over a slot pool in a single launch (ABI version 5).
 * Source: the pages' once-per-window state write and every-step sketch read
 * (readsearch.ai listing of arXiv 2609.33051, Abstract; agihunt.info summary,
 * "Mechanism details"), for a batch whose sequences sit at different window
 * positions; the schedule itself is not on the pages. For every batch row n
 * with slot s = slot[n] (or n when slot is NULL) and tau[n] in [1, W]:
 *   1. the current token (k_t, v_t, decay_t, beta_t of row n) is appended into
 *      window slot tau[n] - 1 of slot s;
 *   2. y[n] is the sketch read at window position tau[n], as
 *      ssm_sketch_decode_step, from sketch0 when parity[n] is 0 and from
 *      sketch1 otherwise;
 *   3. if n is one of the n_update rows listed in update_rows (DEVICE int32
 *      batch-row indices, distinct) and tau[n] == W, the window's W tokens (the
 *      current one included) are applied to state[s], and the refreshed sketch
 *      is stored in the other buffer (sketch1 when parity[n] is 0, else
 *      sketch0). A listed row with tau[n] != W is not updated.
 * The two sketch buffers let a row at tau = W read its window's sketch while
 * the same launch writes the next one; the caller flips parity[n] for the
 * row's next window. Rows with tau outside [1, W] or slot outside
 * [0, num_slots) are skipped (nothing is read for them and y[n] is not
 * written). slot, tau and parity are DEVICE int32 [batch] arrays (4-byte
 * aligned; parity required); the counts in them are not read on the host.
 * Rows must map to distinct slots. Layouts as the other _varlen entry points,
 * sketch0 and sketch1 each [num_slots][H][r][d_v] in d->sketch_dtype; uniform
 * rank. Outputs: y, state, sketch0, sketch1 and the window buffers, none of
 * which may overlap an input or each other.
 */
ssm_status ssm_decode_step_varlen(const ssm_dims* d, int32_t num_slots, const int32_t* slot,
                                  const int32_t* tau, const int32_t* parity, int32_t n_update,
                                  const int32_t* update_rows, float* state, void* sketch0,
                                  void* sketch1, const float* basis, const void* q,
                                  const void* k_t, const void* v_t, const float* decay_t,
                                  const float* beta_t, void* k_buf, void* v_buf,
                                  float* decay_buf, float* beta_buf, float* y, void* stream);

/*
 * Least-squares coefficients: the other reading of the pages' "low-rank
 * state-weighted query approximation" (readsearch.ai listing of arXiv
 * 2609.33051, Abstract). Instead of c = B q~, a step takes the c that minimises
 * || S_win^T q~ - Sk^T c || (the smallest such c when the sketch rows are
 * linearly dependent), so its output Sk^T c + R^T q is the orthogonal
 * projection of the exact window-start read on the span of the sketch rows.
 * It is never further from the exact read than the projection read, and it is
 * exact whenever S_win^T q~ lies in that span (e.g. a state of rank <= r whose
 * row space the sketch captures).
 *
 * ssm_window_update_refresh_ls: the window update as ssm_window_update_refresh,
 * then, from the updated state S and Sk = B S,
 *   sketch_q  fp32 [N][H][r][d_v]  rows orthonormal and spanning the rows of Sk
 *                                  (Gram-Schmidt; a row whose residual is below
 *                                  1e-5 of the largest Sk row norm is stored as zero)
 *   read_map  fp32 [N][H][r][d_k]  Y = sketch_q S^T
 * ssm_sketch_decode_step_ls: the step as ssm_sketch_decode_step, with
 * y = sketch_q^T (read_map q~) + R^T q. The basis is not read.
 * Requires sketch_dtype = SSM_SKETCH_F32 (else SSM_E_RANGE); uniform rank; all
 * sequences at the same window position. Outputs of the update: state,
 * sketch_q, read_map; of the step: y (and the buffers when the token is fused).
 * Per step the read moves r*(d_v + d_k)*4 bytes of sketch_q and read_map per
 * unit instead of r*d_v*4 of Sk.
 */
ssm_status ssm_window_update_refresh_ls(const ssm_dims* d, float* state, float* sketch_q,
                                        float* read_map, const float* basis, const void* k_buf,
                                        const void* v_buf, const float* decay_buf,
                                        const float* beta_buf, int32_t n_tokens, void* stream);
ssm_status ssm_sketch_decode_step_ls(const ssm_dims* d, const float* sketch_q,
                                     const float* read_map, const void* q, const void* k_t,
                                     const void* v_t, const float* decay_t,
                                     const float* beta_t, void* k_buf, void* v_buf,
                                     float* decay_buf, float* beta_buf, int32_t tau, float* y,
                                     void* stream);

/*
 * Per-token recurrent decode step (the standard decode SketchSSM is compared
 * against: readsearch.ai listing, Abstract, kernel speedups over the standard
 * vLLM baseline; agihunt.info "Confirmed", background bullet: every step reads
 * the full state). For every unit, with the current token (k_t, v_t, decay_t,
 * beta_t): S <- M S + b k v^T, S is written back, and y = S^T q is read from
 * the updated state. No window buffer and no sketch; d->window and d->rank are
 * checked but not used. Outputs: state (in/out), y.
 */
ssm_status ssm_recurrent_decode_step(const ssm_dims* d,
                                     float* state, const void* q,
                                     const void* k_t, const void* v_t,
                                     const float* decay_t, const float* beta_t,
                                     float* y, void* stream);

/*
 * Whole sequences at once: prompt processing, which makes the states that the
 * decode calls above start from, and its gradients. (Not on the pages, which
 * start at the decode: agihunt.info summary, "Confirmed", background bullet, on
 * the recurrent state; the recurrence is the one above.) A packed batch holds
 * d->batch sequences one after another:
 *   q, k        in    [total_tokens][H][d_k]       v  in  [total_tokens][H][d_v]
 *   decay       fp32  [total_tokens][H] or [total_tokens][H][d_k] (KDA)
 *   beta        fp32  [total_tokens][H] (GDN, KDA); NULL for Mamba-2
 *   y, dy       fp32  [total_tokens][H][d_v]
 *   plan        int32, as ssm_scan_plan writes it from the sequences' lengths:
 *               [seq_start (n + 1) | chunk_start (n + 1) | chunk_seq (total_tokens/64 + n)]
 *               with n = d->batch: sequence s owns tokens seq_start[s] .. seq_start[s+1] and
 *               the 64-token chunks chunk_start[s] .. chunk_start[s+1]; chunk_seq names a
 *               chunk's sequence, -1 past the last chunk. One plan serves every layer.
 * Sequences may be empty. Tokens behind the last sequence are neither read nor
 * written. A plan's entries are DEVICE data and are not read on the host; whatever
 * they hold, no token outside [0, total_tokens) is touched (an entry that no plan
 * has skips its chunk or sequence). Gates are meant to be in [0, 1]; 0 and 1 are exact.
 * Scalar decays, beta, their gradients and the plan need 4-byte alignment only.
 * A non-finite value of a token may reach outputs of its own sequence up to 15
 * tokens before it (tokens are taken 16 at a time), in the backward pass any gradient of
 * its own sequence; never another sequence or head. An infinity may come out as NaN.
 * Sums and states are fp32; a product of two fp32 values is taken to 2^-21 of itself, one
 * with a bf16 input exactly. d->window and d->rank are checked but not used.
 * heads <= 65536; (total_tokens/64 + batch)*heads < 2^22. Results are the same bits from run
 * to run. A sequence's depend on the rest of the batch only by rounding: batch*heads chooses
 * how a sum over d_k is divided.
 */

/* Sizes for a packed batch: int32 elements of the plan, and the bytes of the
 * workspace of ssm_scan_forward and ssm_scan_backward. Any output may be NULL. */
ssm_status ssm_scan_sizes(const ssm_dims* d, int32_t total_tokens, int64_t* plan_ints,
                          int64_t* forward_bytes, int64_t* backward_bytes);

/*
 * The plan of a packed batch, built on the device from the sequences' lengths
 * (DEVICE int32 [n_seqs], 0 <= n_seqs < 2^24). A negative length counts as 0;
 * sequences are cut where the arrays end (total_tokens). plan: int32, the size
 * that ssm_scan_sizes gives for batch = n_seqs. Both need 4-byte alignment.
 * n_seqs = 0 is a no-op. One launch.
 */
ssm_status ssm_scan_plan(const int32_t* lengths, int32_t n_seqs, int32_t total_tokens,
                         int32_t* plan, void* stream);

/*
 * For every sequence and head: S <- M_t S + b_t k_t v_t^T and y_t = S^T q_t over
 * its tokens, from the state in state_in (NULL: from zero), which ends in state.
 * Both states are pools [num_slots][H][d_k][d_v] indexed by slot[s] (DEVICE int32
 * [batch], NULL: slot s); state_in may be state itself, which continues a prompt
 * in place. A sequence whose slot is outside [0, num_slots) is skipped (its y and
 * state are not written); the sequences must map to distinct slots. An empty
 * sequence's state is its state_in. The workspace (16-byte aligned, at least
 * ssm_scan_sizes' forward_bytes) holds nothing between calls; calls that may run
 * at the same time, captured graphs among them, need one each.
 * Outputs: state, y, workspace.
 */
ssm_status ssm_scan_forward(const ssm_dims* d, int32_t total_tokens, const int32_t* plan,
                            int32_t num_slots, const int32_t* slot, const float* state_in,
                            const void* q, const void* k, const void* v, const float* decay,
                            const float* beta, float* state, float* y, void* workspace,
                            int64_t workspace_bytes, void* stream);

/*
 * Gradients of ssm_scan_forward (slots 0 .. batch-1) for a loss whose gradients
 * with respect to y and the final states are dy and dstate ([batch][H][d_k][d_v],
 * NULL: zero). dq, dk, dv have the inputs' type (bf16: rounded once, to nearest);
 * dbeta (NULL for Mamba-2) and dstate_in (NULL: not wanted) are fp32;
 * dlog_decay is fp32 in decay's shape and holds decay * dL/d(decay), the gradient
 * with respect to ln(decay), which stays finite at decay = 0 (where it is exactly 0).
 * It is the difference of sums over up to 64 tokens, so its rounding is relative to
 * their terms, |state * dL/d(state)| + |q dq| + |k dk|, not to the value: divided by a
 * small decay it is no accurate dL/d(decay). The states are computed again from the
 * inputs: nothing is kept from the forward call.
 * Gradients of tokens behind the last sequence are not written. The workspace as
 * in ssm_scan_forward, with backward_bytes.
 * Outputs: dq, dk, dv, dlog_decay, dbeta, dstate_in, workspace.
 */
ssm_status ssm_scan_backward(const ssm_dims* d, int32_t total_tokens, const int32_t* plan,
                             const float* state_in, const void* q, const void* k, const void* v,
                             const float* decay, const float* beta, const float* dy,
                             const float* dstate, void* dq, void* dk, void* dv,
                             float* dlog_decay, float* dbeta, float* dstate_in, void* workspace,
                             int64_t workspace_bytes, void* stream);

/*
 * The index arrays of ssm_decode_step_varlen, built on the device (so a serving
 * loop needs no host arithmetic per step and can be captured into a graph). For
 * every row n, from lengths[n] = the number of tokens the row has decoded before
 * this step (its prompt not counted; negative: a padding row):
 *   tau[n]    = lengths[n] mod W + 1   (0 for a padding row, which the step skips)
 *   parity[n] = (lengths[n] / W) mod 2 (0 for a padding row)
 *   update_rows: the rows with tau = W, in ascending order, then -1; *n_update of them.
 * d->batch rows; W = d->window; the other dims are checked but not used. All arrays
 * DEVICE int32 [batch] (n_update: one element), 4-byte aligned. A step that takes
 * n_update = d->batch with these update_rows updates exactly the listed rows: the
 * entries of -1 are skipped, but the listed rows, the first of a longer list, then share
 * fewer of the GPU's parts (256 rows of 32 heads, 128 x 128, W = 8, 32 rows listed: 125 us
 * a step, 40 us with n_update = 32). Where the host knows the count, pass it. One launch.
 */
ssm_status ssm_window_plan(const ssm_dims* d, const int32_t* lengths, int32_t* tau,
                           int32_t* parity, int32_t* update_rows, int32_t* n_update,
                           void* stream);

/*
 * Offline basis fit on the device. The pages fix the query basis offline
 * (readsearch.ai listing, Abstract; agihunt.info "Confirmed", mechanism bullet:
 * queries are compressed onto a small low-rank basis); the Mamba-2 workload's
 * recipe takes the top PCA directions of sampled queries and makes them
 * orthonormal. For every head h, with X_h = samples[h] (n_samples queries of
 * d_k entries), basis[h] receives the d->rank unit eigenvectors of the
 * uncentred second moment X_h^T X_h / n_samples with the largest eigenvalues,
 * one per row, in decreasing order of eigenvalue, orthonormal in fp32, each
 * signed so that its entry of largest magnitude (the first on a tie) is
 * positive. Rows for equal eigenvalues are some orthonormal basis of their
 * eigenspace.
 *   samples: [H][n_samples][d_k], d->in_dtype, device, read only;
 *   basis:   [H][rank][d_k] fp32, device, out: the layout the window and
 *            sketch calls read.
 * Uses heads, d_k, rank and in_dtype of d; the other fields are checked but
 * not used. 1 <= n_samples <= 2^24. The basis must not overlap the samples.
 * Setup-time work: one workgroup per head, nothing allocated.
 */
ssm_status ssm_fit_basis(const ssm_dims* d, const void* samples, int32_t n_samples,
                         float* basis, void* stream);

/*
 * Measurement aid, not a step of the method: the HBM rate that a state-sized
 * read + write reaches on this device, to set the window update's bandwidth
 * against. Streams buf in place: every value is read, multiplied by 1.0f and
 * written back, all of a thread's loads before its stores, non-temporal.
 *   buf:     fp32, device, n_tiles * 16384 floats (64 KB tiles), in/out;
 *   shape 0: the window update's access order: one 256-thread workgroup per
 *            tile seen as a 128 x 128 state; each wave holds 32 columns, lane
 *            group g of a wave the rows g, g + 8, ...; consecutive tiles go to
 *            one XCD;
 *   shape 1: two tiles per 512-thread workgroup, read as one flat run; each
 *            load instruction of the workgroup covers 8 KB contiguous.
 * 1 <= n_tiles < 2^24; shape 1 needs an even n_tiles (else SSM_E_SHAPE);
 * shape outside {0, 1} gives SSM_E_RANGE. One launch per call.
 */
ssm_status ssm_stream_probe(float* buf, int64_t n_tiles, int32_t shape, void* stream);

/*
 * What a layer does around its recurrence: the short convolution of its inputs, a recurrence whose
 * decay goes by channel and state, and the norm of its outputs, each for packed prompts (the plan of
 * ssm_scan_plan), for their gradients and for a batch of single tokens. (Not on the pages, which
 * start at the recurrence's inputs.)
 *
 * Token arrays are rows: row t is `width` elements from data + t * stride elements on, so that
 * an array may be a column range of a larger one (a fused projection, its gradient). A stride is at
 * least the width, a multiple of 8 and below 2^26. Outputs must not overlap inputs or each other;
 * column ranges of one array (the same stride) do not overlap. Weights are fp32.
 * Sums, states and statistics are fp32; results in bf16 are rounded once, to nearest. Results are the
 * same bits from run to run. A plan that ssm_scan_plan did not write gives wrong results, but nothing outside
 * the arrays is touched, whatever it holds.
 */
typedef struct {
  void* data;
  int64_t stride; /* elements from row to row */
} ssm_rows;

/*
 * The short causal convolution. Its channels come in 1 to 4 parts (queries, keys, values), each with
 * rows of its own; weights, bias and kept inputs hold the parts' channels one after another,
 * C = sum of channels[]. For token t of a sequence and channel c, with K = taps:
 *   u_t = bias[c] + sum_j weight[c][j] x_{t-(K-1)+j}[c],   a = silu(u) or u,
 * where x before the sequence is the kept state's (zero without one), and
 *   y = a,  or with norm[p] = n > 0, over each run of n channels of part p:
 *   y = scale[p] * a / sqrt(sum a^2 + eps)
 * (the l2 norm of queries and keys per head, n = d_k; a run whose sum of squares passes fp32's range
 * gives 0).
 *   x, y, dy, dx: parts arrays of rows, in_dtype;   weight fp32 [C][K], bias fp32 [C] or NULL;
 *   state: in_dtype [slots][K-1][C], a sequence's last K-1 inputs, oldest first.
 * A NaN or infinity in a token reaches the K tokens from it on (in the gradients the K-1 before them
 * too) of its own channel, or of its norm's run; dweight and dbias of the channel.
 * 2 <= K <= 4; channels[p] a multiple of 8, of norm[p] where that is set; norm[p] in {0, 16, 32, 64,
 * 128}; C <= 2^20; batch < 2^24; (total_tokens/64 + batch) * ceil(C/512) < 2^24.
 */
#define SSM_CONV_PARTS 4
typedef enum { SSM_ACT_NONE = 0, SSM_ACT_SILU = 1, SSM_ACT_SIGMOID = 2 } ssm_activation;
typedef struct {
  int32_t in_dtype;   /* ssm_in_dtype of x, y, the state and their gradients */
  int32_t batch;      /* sequences, or rows of a step                       */
  int32_t taps;       /* K                                                  */
  int32_t activation; /* SSM_ACT_NONE or SSM_ACT_SILU                       */
  int32_t parts;
  int32_t channels[SSM_CONV_PARTS];
  int32_t norm[SSM_CONV_PARTS];
  float scale[SSM_CONV_PARTS];
  float eps;          /* added to a run's sum of squares: at least 2^-126 with a norm */
} ssm_conv_dims;

/* Bytes of the workspace of ssm_conv_backward. */
ssm_status ssm_conv_sizes(const ssm_conv_dims* d, int32_t total_tokens, int64_t* backward_bytes);

/*
 * A packed batch of d->batch sequences. state_in (NULL: zero) and state (NULL: not wanted) are pools of
 * num_slots, indexed by slot[s] (DEVICE int32 [batch], NULL: slot s); state_in may be state itself,
 * which continues prompts in place. A sequence whose slot is outside [0, num_slots) is skipped; the
 * sequences must map to distinct slots. An empty sequence's state is its state_in. Rows behind the
 * last sequence are neither read nor written. num_slots and slot are ignored without a state.
 * Outputs: y, state.
 */
ssm_status ssm_conv_forward(const ssm_conv_dims* d, int32_t total_tokens, const int32_t* plan,
                            int32_t num_slots, const int32_t* slot, const void* state_in,
                            const ssm_rows* x, const float* weight, const float* bias, void* state,
                            const ssm_rows* y, void* stream);

/*
 * Gradients of ssm_conv_forward (slots 0 .. batch-1) for a loss whose gradients with respect to y and
 * the final states are dy and dstate (in_dtype [batch][K-1][C], NULL: zero). dweight, dbias (NULL:
 * not wanted) are fp32, sums over all tokens; dstate_in (NULL: not wanted) is in_dtype. Nothing is kept from
 * the forward call. dx behind the last sequence is not written.
 * Outputs: dx, dweight, dbias, dstate_in, workspace (16-byte aligned, ssm_conv_sizes' bytes; calls
 * that may run at the same time need one each).
 */
ssm_status ssm_conv_backward(const ssm_conv_dims* d, int32_t total_tokens, const int32_t* plan,
                             const void* state_in, const ssm_rows* x, const float* weight,
                             const float* bias, const ssm_rows* dy, const void* dstate,
                             const ssm_rows* dx, float* dweight, float* dbias, void* dstate_in,
                             void* workspace, int64_t workspace_bytes, void* stream);

/*
 * One token of every row: rows d->batch, the state (in/out) a pool as above. Outputs: y, state.
 */
ssm_status ssm_conv_step(const ssm_conv_dims* d, int32_t num_slots, const int32_t* slot,
                         const ssm_rows* x, const float* weight, const float* bias, void* state,
                         const ssm_rows* y, void* stream);

/*
 * The selective recurrence: a state of N = d_state values per channel, whose decay goes by channel and
 * state. For every token and channel d, with g the channel's group (channels/groups consecutive ones):
 *   delta = softplus(dt[d] + dt_bias[d])   (softplus = 0: dt[d] + dt_bias[d] itself)
 *   h[n] <- exp(delta A[d][n]) h[n] + delta x[d] B[g][n],     n = 0 .. N-1
 *   y[d] = sum_n C[g][n] h[n] + D[d] x[d],      out[d] = y[d] silu(z[d])
 *   x, dt, z, out   in_dtype rows of `channels`;  B, C  in_dtype rows of groups * d_state
 *   A  fp32 [channels][d_state] (finite; negative, so that the state decays);  D, dt_bias fp32 [channels]
 *   states  fp32 [slots][channels][d_state]
 * z.data, D and dt_bias may be NULL (no gate, no skip, no bias).
 * A NaN or infinity reaches what follows it in its own sequence (in the gradients all of its
 * sequence, and the sums over tokens); one in B or C every channel of its group.
 * d_state in {8, 16, 32, 64}; channels/groups a multiple of 16; channels <= 2^20; batch < 2^24;
 * (total_tokens/64 + batch) * channels/16 < 2^31; backward total_tokens * groups * d_state <= 2^31 - 128;
 * a step batch * channels * max(d_state, 16) < 2^34.
 */
typedef struct {
  int32_t in_dtype; /* ssm_in_dtype of x, dt, z, B, C, out */
  int32_t batch;    /* sequences, or rows of a step        */
  int32_t channels;
  int32_t d_state;
  int32_t groups;
  int32_t softplus; /* 0 or 1                              */
} ssm_selective_dims;

typedef struct {
  ssm_rows x, dt, z, B, C;
  const float *A, *D, *dt_bias;
} ssm_selective_inputs;

typedef struct {
  ssm_rows dx, ddt, dz, dB, dC;
  float *dA, *dD, *ddt_bias;
} ssm_selective_grads;

/*
 * Bytes of the workspaces of ssm_selective_forward and ssm_selective_backward. Either may be NULL. Forward: 22 MB at
 * the most. Backward: 8.5 bytes a token and channel with d_state = 8, 16.5 with 16 (8.3 times x in bf16; 5.6 GB for
 * 65,536 tokens of 5,120 channels), 48.5 with 32, 160.5 with 64: the state before every 8 tokens, and the sums for dB and
 * dC over a wave's channels, which are 16 with d_state up to 16, 8 with 32, 4 with 64.
 */
ssm_status ssm_selective_sizes(const ssm_selective_dims* d, int32_t total_tokens,
                               int64_t* forward_bytes, int64_t* backward_bytes);

/*
 * A packed batch; plan, slots and states as in ssm_conv_forward (state_in may be state itself), but the
 * final states are always written. The workspace holds nothing between calls; calls that may run at the
 * same time need one each. Outputs: state, out, workspace.
 */
ssm_status ssm_selective_forward(const ssm_selective_dims* d, int32_t total_tokens,
                                 const int32_t* plan, int32_t num_slots, const int32_t* slot,
                                 const float* state_in, const ssm_selective_inputs* in, float* state,
                                 const ssm_rows* out, void* workspace, int64_t workspace_bytes,
                                 void* stream);

/*
 * Gradients of ssm_selective_forward (slots 0 .. batch-1) for a loss whose gradients with respect to out
 * and the final states are dout and dstate (fp32 [batch][channels][d_state], NULL: zero). dx, ddt, dz,
 * dB, dC are in_dtype; dA [channels][d_state], dD, ddt_bias [channels] fp32, sums over all tokens, and
 * dstate_in (NULL: not wanted) fp32. dz, dD, ddt_bias are given where z, D, dt_bias are. The
 * states are computed again: nothing is kept from the forward call.
 * Outputs: the gradients, workspace.
 */
ssm_status ssm_selective_backward(const ssm_selective_dims* d, int32_t total_tokens,
                                  const int32_t* plan, const float* state_in,
                                  const ssm_selective_inputs* in, const ssm_rows* dout,
                                  const float* dstate, const ssm_selective_grads* grads,
                                  float* dstate_in, void* workspace, int64_t workspace_bytes,
                                  void* stream);

/* One token of every row: rows d->batch, the state (in/out) a pool. Outputs: state, out. */
ssm_status ssm_selective_step(const ssm_selective_dims* d, int32_t num_slots, const int32_t* slot,
                              const ssm_selective_inputs* in, float* state, const ssm_rows* out,
                              void* stream);

/*
 * The norm of a layer's outputs in groups of channels, with a gate. For every row and group of `width`
 * channels, with s(z) the activation z sigmoid(z) (SSM_ACT_SILU) or sigmoid(z) (SSM_ACT_SIGMOID):
 *   u = x (SSM_GATE_NONE, SSM_GATE_AFTER) or x s(z) (SSM_GATE_BEFORE)
 *   n = (u - mean) / sqrt(var + eps)      (centred = 0: the mean taken as zero)
 *   o = n weight + bias,     out = o, or o s(z) (SSM_GATE_AFTER)
 *   x        x_dtype, rows of groups * width;   z, out  in_dtype, the same shape
 *   weight   fp32 [groups][width], or [width] for all groups (shared = 1);  bias the same or NULL
 * width a multiple of 8, at most 8192; groups * width <= 2^20; rows * groups < 2^31;
 * eps >= 2^-126. A group whose sum of squares passes fp32's range has n = 0.
 */
typedef enum { SSM_GATE_NONE = 0, SSM_GATE_AFTER = 1, SSM_GATE_BEFORE = 2 } ssm_gate;
typedef struct {
  int32_t x_dtype;  /* ssm_in_dtype of x and dx              */
  int32_t in_dtype; /* ssm_in_dtype of z, out, dout and dz   */
  int32_t groups;
  int32_t width;
  int32_t gate;       /* ssm_gate                            */
  int32_t activation; /* of the gate                         */
  int32_t shared;     /* 1: one weight row for all groups    */
  int32_t centred;    /* 1: the mean is subtracted           */
  float eps;
} ssm_norm_dims;

ssm_status ssm_gated_norm(const ssm_norm_dims* d, int32_t rows, const ssm_rows* x, const ssm_rows* z,
                          const float* weight, const float* bias, const ssm_rows* out, void* stream);

/* Bytes of the workspace of ssm_gated_norm_backward. */
ssm_status ssm_gated_norm_sizes(const ssm_norm_dims* d, int32_t rows, int64_t* backward_bytes);

/*
 * Gradients of ssm_gated_norm for dout. dx is x_dtype, dz (NULL without a gate) in_dtype; dweight
 * and dbias (NULL: not wanted; bias, which they do without, is needed for dz with SSM_GATE_AFTER) fp32 in
 * the weights' shape, sums over all rows (shared: and groups).
 * Outputs: dx, dz, dweight, dbias, workspace (16-byte aligned; calls that may run at the same time
 * need one each).
 */
ssm_status ssm_gated_norm_backward(const ssm_norm_dims* d, int32_t rows, const ssm_rows* x,
                                   const ssm_rows* z, const float* weight, const float* bias,
                                   const ssm_rows* dout, const ssm_rows* dx, const ssm_rows* dz,
                                   float* dweight, float* dbias, void* workspace,
                                   int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SKETCHSSM_H */
