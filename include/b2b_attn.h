/*
 * b2b_attn.h -- attention operators of libb2b.so for AMD Instinct MI355X
 * (gfx950): cascades of two products whose second operands are activations,
 * with a mask, a softmax or a decay between the products.  As in the GEMM
 * cascades of b2b.h the intermediate never leaves the chip: the first
 * product's accumulator fragment becomes the second one's operand in place.
 * And what comes before them: norms and rotations of queries and keys, alone
 * or into the pages of a cache.
 *
 * Layouts: every operand is a set of rows (tokens) of heads, head_dim
 * elements contiguous, with a stride from row to row and one from head to
 * head (b2b_rows_t), so [tokens, heads, dim], [heads, tokens, dim] and slices
 * of a fused projection are all taken as they lie.  Base pointers are
 * 16-byte aligned and strides are multiples of 8 elements, from row to row up
 * to 2^23 (a single row's is not looked at).  Query head h reads key/value head
 * h / (heads / kv_heads).
 *
 * Sequence starts (cu_*), lengths (lens), tables of pages and positions are
 * read on the device, so a captured graph replays with new ones; the kernels
 * clamp them to the rows and pages that the call names, so no value of theirs
 * reaches outside the tensors.
 *
 * Plans hold host data only; any number of runs of one plan may overlap.  A
 * run that splits its keys or its sequences over workgroups needs a
 * workspace (the _workspace call says how many bytes), which belongs to that
 * run until it is over: runs that overlap, or graphs captured with one, each
 * need their own.  Errors as in b2b.h: a status, never an abort; runs only
 * enqueue kernels on the stream.
 */
#ifndef B2B_ATTN_H_
#define B2B_ATTN_H_

#include "b2b.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct b2b_attn_plan* b2b_attn_t;   /* opaque, owned by the library */

/* Rows of heads in device memory. */
typedef struct {
    const void* data;
    int64_t row_stride;    /* elements from one row to the next, head_dim or more */
    int64_t head_stride;   /* elements from one head to the next */
} b2b_rows_t;

/* Flags of b2b_attn_create. */
enum {
    B2B_ATTN_CAUSAL = 1u << 0   /* row i of n sees keys j <= i + keys - n of its sequence */
};

/*
 * Plans the attention of a model's heads.
 *   dtype       B2B_DTYPE_F16 or B2B_DTYPE_BF16: Q, K, V and O; sums, the
 *               softmax's statistics and partial results are float32, the
 *               probabilities are rounded to dtype for the second product (fp16:
 *               below 2^-25 of the row's largest they count in its sum alone)
 *   heads       query heads; kv_heads divides it
 *   head_dim    a multiple of 8, up to 128
 *   scale       of the scores, positive, up to 2^127 (0: head_dim ^ -1/2)
 * INVALID_VALUE for sizes or flags outside these, NOT_SUPPORTED for another
 * dtype or head_dim.
 */
b2b_status_t b2b_attn_create(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                             float scale, uint32_t flags);

/*
 * Packed sequences: rows cu_q[s] .. cu_q[s+1]-1 of Q and O belong to
 * sequence s, rows cu_k[s] .. cu_k[s+1]-1 of K and V are its keys.
 *     O_i = sum_j p_ij V_j,  p_ij = exp(scale Q_i.K_j) / sum_j' exp(scale Q_i.K_j')
 * over the keys that row i sees: all of its sequence, or with
 * B2B_ATTN_CAUSAL those up to its own place counted from the end (a prompt's
 * piece behind earlier keys).  A row that sees no key gets 0.  Infinities and
 * NaN reach the rows that see them and no others (32 rows whose results are
 * not all finite are computed again, which takes some 15 times as long); an
 * infinity whose probability is below float32's range may come out as NaN.
 *   seqs        sequences; cu_q and cu_k hold seqs + 1 values (device); cu_k
 *               may be cu_q
 *   rows, keys  rows that Q and O, and K and V, hold: cu values past them are
 *               clamped; rows of O that belong to no sequence are not written
 *   lse         device float32 [rows, heads] or NULL: the logarithm of each
 *               row's sum (-inf where it sees no key)
 *   workspace   device, 16-byte aligned, at least b2b_attn_workspace bytes
 *               (NULL where that is 0)
 * INVALID_VALUE for bad sizes, strides, alignment or pointers, O at an
 * input's address or with rows or heads that overlap, or a workspace too small.
 * O must not overlap the inputs.
 */
b2b_status_t b2b_attn_workspace(b2b_attn_t plan, int32_t seqs, int64_t rows, int64_t keys, size_t* bytes);
b2b_status_t b2b_attn_run(b2b_attn_t plan, int32_t seqs, int64_t rows, int64_t keys, b2b_rows_t Q, b2b_rows_t K,
                          b2b_rows_t V, b2b_rows_t O, const int32_t* cu_q, const int32_t* cu_k, float* lse,
                          void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token for each request of a batch behind one shared prefix: row b of Q
 * sees all `prefix` rows of Kp and Vp and the first lens[b] of request b's
 * own `own` rows of K and V.  The prefix's keys are read once for the whole
 * batch.  A request that sees no key gets 0.  Plans made without
 * B2B_ATTN_CAUSAL (a new token sees every key).
 *   prefix, own  0 or more; Kp and Vp (K, V and lens) may be NULL where it is 0
 *   k_stride, v_stride   elements from one request's own keys (values) to the
 *                        next one's, multiples of 8
 *   lens         device int32 [batch], clamped to 0 .. own
 *   workspace    as above (b2b_prefix_attn_workspace)
 */
b2b_status_t b2b_prefix_attn_workspace(b2b_attn_t plan, int32_t batch, int64_t prefix, int64_t own, size_t* bytes);
b2b_status_t b2b_prefix_attn_run(b2b_attn_t plan, int32_t batch, int64_t prefix, int64_t own, b2b_rows_t Q,
                                 b2b_rows_t Kp, b2b_rows_t Vp, b2b_rows_t K, int64_t k_stride, b2b_rows_t V,
                                 int64_t v_stride, const int32_t* lens, b2b_rows_t O, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);

/*
 * Plans causal attention under a window, for b2b_attn_workspace and
 * b2b_attn_run: the row in place p of its sequence (counted from the last key,
 * as B2B_ATTN_CAUSAL) sees keys p - window + 1 .. p and the sequence's first
 * `sinks` keys up to p.
 *   window   1 to 2^30      sinks   0 to 2^30
 * rows (of b2b_attn_run) below 2^30.  O that shares an element with an input is
 * INVALID_VALUE.
 */
b2b_status_t b2b_attn_create_window(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                    float scale, int32_t window, int32_t sinks);

/* The pages of a cache, all of one size, in device memory: base 16-byte
 * aligned, strides in elements, multiples of 8, in any order ([pages, size,
 * heads, dim] and [pages, heads, size, dim] alike). */
typedef struct {
    void* data;            /* only b2b_rotary_append writes */
    int64_t page_stride;
    int64_t row_stride;    /* from one key of a page to the next */
    int64_t head_stride;
} b2b_pages_t;

/*
 * Plans causal attention of new tokens over a paged cache: key j of sequence s
 * is row j % page_size of page table[s][j / page_size].
 *   page_size      1 to 2^20, no power of two needed
 *   window, sinks  as b2b_attn_create_window; window 0: every earlier key
 */
b2b_status_t b2b_paged_attn_create(b2b_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                   int32_t page_size, float scale, int32_t window, int32_t sinks);

/*
 * Rows cu_q[s] .. cu_q[s+1]-1 of Q and O are the last tokens of sequence s, whose
 * lens[s] keys (theirs among them) are in the cache: one token, a chunk of a
 * prompt or none, each sequence as it comes.  A row sees the keys up to its own
 * place, or those of its window; one that sees no key gets 0.  Rows that belong
 * to no sequence are not written.  What pages hold behind a sequence's last key
 * is never looked at; infinities and NaN as for b2b_attn_run.
 *   pages   pages of K and V: entries of the table are clamped to them
 *   table   device int32 [seqs, width], rows table_stride apart; entries of pages
 *           behind a sequence's last key are not read
 *   lens    device int32 [seqs], clamped to 0 .. width x page_size (below 2^30)
 *   cu_q    device int32 [seqs + 1], or NULL: row s is sequence s's one token
 *   lse, workspace   as for b2b_attn_run (b2b_paged_attn_workspace)
 * INVALID_VALUE as for b2b_attn_run, and for O that shares an element with an
 * input (it may lie between others' rows).
 */
b2b_status_t b2b_paged_attn_workspace(b2b_attn_t plan, int32_t seqs, int64_t rows, int32_t width, size_t* bytes);
b2b_status_t b2b_paged_attn_run(b2b_attn_t plan, int32_t seqs, int64_t rows, b2b_rows_t Q, b2b_pages_t K, b2b_pages_t V,
                                int32_t pages, const int32_t* table, int32_t width, int64_t table_stride, const int32_t* lens,
                                const int32_t* cu_q, b2b_rows_t O, float* lse, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

/* Releases a plan. NULL is a no-op. */
b2b_status_t b2b_attn_destroy(b2b_attn_t plan);

typedef struct b2b_linear_attn_plan* b2b_linear_attn_t;   /* opaque, owned by the library */

/*
 * Plans linear attention with a decay for each head: no softmax, and a state
 * instead of a cache,
 *     S_t = lambda_h S_{t-1} + k_t v_t^T        (head_dim x head_dim, row: key element)
 *     o_t = scale q_t^T S_t,    lambda_h = exp(log_decay[h])
 *   dtype       B2B_DTYPE_F16 or B2B_DTYPE_BF16: Q, K, V and O; states are
 *               float32 and updated in float32 precision; the scores q.k are
 *               held in two parts of dtype, the copy of the state that meets q
 *               is rounded to it (fp16: a row's scores and, where its largest value
 *               is below 0.25 or above 2^14, the copy of 32 value columns are scaled
 *               by powers of two, so both may be of any size; else the copy's values
 *               below 2^-14 are held to 2^-25)
 *   head_dim    64 or 128
 *   scale       finite and positive (0: head_dim ^ -1/2)
 */
b2b_status_t b2b_linear_attn_create(b2b_linear_attn_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads,
                                    int32_t head_dim, float scale);

/*
 * Packed prompts: rows cu[s] .. cu[s+1]-1 are sequence s, 32 tokens at a time.
 * Infinities and NaN reach no earlier rows and no columns but their own (a
 * sequence's head, or its piece, that holds some is computed twice); of a sequence
 * cut into pieces, later pieces may be without those that the decay has taken
 * below float32's range.
 *   log_decay   device float32 [heads], 0 or below (-inf: nothing is kept)
 *   state_in    device float32 [seqs, heads, head_dim, head_dim], the states
 *               before the sequences, or NULL (zero); 16-byte aligned
 *   state_out   the states after them, or NULL; may be state_in, and else must
 *               not overlap it.  A sequence without tokens keeps its state
 *   workspace   as for b2b_attn_run (b2b_linear_attn_workspace)
 * Rows of O that belong to no sequence are not written.  O must not overlap the
 * inputs.
 */
b2b_status_t b2b_linear_attn_workspace(b2b_linear_attn_t plan, int32_t seqs, int64_t rows, size_t* bytes);
b2b_status_t b2b_linear_attn_run(b2b_linear_attn_t plan, int32_t seqs, int64_t rows, b2b_rows_t Q, b2b_rows_t K,
                                 b2b_rows_t V, b2b_rows_t O, const float* log_decay, const int32_t* cu,
                                 const float* state_in, float* state_out, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/*
 * One token of each of `batch` requests (row b of Q, K, V and O): one step of
 * the recurrence on state b.  state_out may be state_in (updated in place).
 */
b2b_status_t b2b_linear_attn_step(b2b_linear_attn_t plan, int32_t batch, b2b_rows_t Q, b2b_rows_t K, b2b_rows_t V,
                                  b2b_rows_t O, const float* log_decay, const float* state_in, float* state_out,
                                  hipStream_t stream);

/* Releases a plan. NULL is a no-op. */
b2b_status_t b2b_linear_attn_destroy(b2b_linear_attn_t plan);

typedef struct b2b_rotary_plan* b2b_rotary_t;   /* opaque, owned by the library */

/* Flags of b2b_rotary_create. */
enum {
    B2B_ROTARY_NORM = 1u << 0,         /* heads are normed first */
    B2B_ROTARY_INTERLEAVED = 1u << 1   /* pair i is elements 2i, 2i + 1; else i, i + rotary_dim / 2 */
};

/*
 * Plans what a decoder does to its queries and keys before the attention, in
 * one pass: each head x is normed (B2B_ROTARY_NORM),
 *     y = x / sqrt(mean(x^2) + eps) * weight,
 * and pair i of its first rotary_dim elements is turned by the row's position,
 *     (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position[axes_of[i]] freqs[i].
 * All of it in float32 (angles reduced in float64, so that far positions lose
 * nothing; norms whose sums, alone or with the weights, leave float32's range in
 * float64), rounded once.
 *   rotary_dim  a multiple of 8, 0 (no rotation) to head_dim
 *   freqs       host, rotary_dim / 2 finite values: radians a position (an angle is
 *               off by 2^-52 of itself, that of a frequency up to 1 by 2^-24 of a turn)
 *   axes_of     host, rotary_dim / 2 values below `axes`, or NULL (all axis 0)
 *   axes        1 to 4 positions a row (time, height, width ...)
 *   eps         0 or more, finite (without B2B_ROTARY_NORM not looked at)
 * dtype, heads, kv_heads and head_dim as b2b_attn_create.
 */
b2b_status_t b2b_rotary_create(b2b_rotary_t* plan, b2b_dtype_t dtype, int32_t heads, int32_t kv_heads, int32_t head_dim,
                               int32_t rotary_dim, const double* freqs, const int32_t* axes_of, int32_t axes, float eps,
                               uint32_t flags);

/*
 * Q' and K' of `rows` rows: Qo and Ko may be Q and K (the same address and
 * strides: in place), and must share no element with anything else (INVALID_VALUE;
 * they may lie between others' rows, as slices of one projection do).
 *   positions        device int32 [axes, rows], axes position_stride apart (0: all axes
 *                    alike; NULL where rotary_dim is 0)
 *   q_weight, k_weight  device, head_dim values of dtype, 16-byte aligned, or NULL (1);
 *                    NULL without B2B_ROTARY_NORM
 */
b2b_status_t b2b_rotary_run(b2b_rotary_t plan, int64_t rows, b2b_rows_t Q, b2b_rows_t K, b2b_rows_t Qo, b2b_rows_t Ko,
                            const int32_t* positions, int64_t position_stride, const void* q_weight, const void* k_weight,
                            hipStream_t stream);

/*
 * The same for new tokens whose keys and values go into a paged cache: rows
 * cu[s] .. cu[s+1]-1 (or row s, without cu) are the last tokens of sequence s,
 * which has lens[s] keys with theirs.  Q' goes to Qo, K' and V to the row's place
 * in the pages, where b2b_paged_attn_run with the same table, lens and cu finds
 * them.
 *   positions   as above, or NULL: a row's place in its sequence, on every axis
 *   pages, page_size, table, width, table_stride, lens, cu   as b2b_paged_attn_run.
 *               A row whose place is below 0 or past the table, or whose entry
 *               names no page, writes no key and no value; rows that belong to
 *               no sequence write nothing
 * No two rows of a call may have the same place of the same page (sequences that
 * share pages have their new tokens in pages of their own).  No two places of the
 * pages, and no place and another operand, may share an element (INVALID_VALUE).
 */
b2b_status_t b2b_rotary_append(b2b_rotary_t plan, int32_t seqs, int64_t rows, b2b_rows_t Q, b2b_rows_t K, b2b_rows_t V,
                               b2b_rows_t Qo, b2b_pages_t k_cache, b2b_pages_t v_cache, int32_t pages, int32_t page_size,
                               const int32_t* table, int32_t width, int64_t table_stride, const int32_t* lens,
                               const int32_t* cu, const int32_t* positions, int64_t position_stride, const void* q_weight,
                               const void* k_weight, hipStream_t stream);

/* Releases a plan. NULL is a no-op. */
b2b_status_t b2b_rotary_destroy(b2b_rotary_t plan);

#ifdef __cplusplus
}
#endif
#endif /* B2B_ATTN_H_ */
