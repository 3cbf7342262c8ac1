/*
 * qmm_decode -- the operators of a decode step with drafts beside those of qmm_serve.h, for one GB300
 * (sm_103a): norms and position rotation of queries and keys, attention with a sliding window over
 * the paged cache, and verification of drafted tokens.  Part of libqmm.so; status codes and
 * conventions are those of qmm.h and qmm_serve.h: no call aborts the process, every pointer is
 * device memory unless said otherwise, every call is ordered on `stream` (a cudaStream_t passed as
 * void*, NULL = legacy default stream), allocates nothing, synchronises nothing and can be
 * captured in a CUDA graph.  Error words are or-ed as qmm_serve.h says: 1 a wait ran out, 2 a page
 * outside the pool, 4 rows or lengths out of range.
 */
#ifndef QMM_DECODE_H
#define QMM_DECODE_H

#include "qmm_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t heads;       /* query heads, >= 0 (0: no q) */
    int32_t kv_heads;    /* key heads, >= 0 (0: no k) */
    int32_t head_dim;    /* 64, 128 or 256 */
    int32_t rot_dim;     /* leading dims that are rotated: a multiple of 16, 0 .. head_dim */
    int32_t axes;        /* rows of pos, 1 .. 4 */
    int32_t interleaved; /* pair i of the rotated dims: 0: (i, i + rot_dim / 2), 1: (2 i, 2 i + 1) */
    int32_t in_type;     /* QMM_TYPE_* of q and k */
    int32_t q_type;      /* .. of q_out */
    int32_t k_type;      /* .. of k_out */
    float eps;
} qmm_rotate_dims;

/*
 * Norm and rotation of each row's query and key heads, in one pass: for a head x,
 *     y = x / sqrt(mean(x^2) + eps) * weight                      (weight null: y = x)
 *     (out_a, out_b) = (y_a cos t - y_b sin t, y_a sin t + y_b cos t),  t = pos[axis[i]][row] * inv_freq[i]
 * over the pairs i < rot_dim / 2; dims from rot_dim on are y.  Several axes are positions in time,
 * height and width, of which each pair turns by one.
 *  q, k:       [rows][heads][head_dim] and [rows][kv_heads][head_dim] of in_type, row r at r * q_stride
 *              (k_stride) elements: columns of a wider matrix are taken in place.  Aligned to
 *              their element; 16-byte aligned rows are read faster.
 *  q_weight, k_weight: fp32 [head_dim], or null (that one is not normalised).
 *  pos:        int32 [axes][rows].  Any value: an angle's whole turns drop out without error, and what is left
 *              is off by 2^-52 of the angle and 2^-31 of a turn at most, and by fp32's rounding before cosine and sine.
 *  inv_freq:   fp32 [rot_dim / 2].   axis: int32 [rot_dim / 2], 0 .. axes - 1 (others count as 0), or null (all 0).
 *  q_out, k_out: [rows][heads][head_dim], [rows][kv_heads][head_dim], row r at r * q_out_stride
 *              (k_out_stride) elements.  An output may be its input, at the same stride and type;
 *              otherwise it overlaps no input and not the other output.
 * Everything is fp32 (a head's sum of squares too: it leaves fp32 where |x| passes 10^18), rounded once
 * to the output's type.  rows = 0 is a no-op.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, NO_DEVICE, CUDA.
 */
qmm_status qmm_rotate(const qmm_rotate_dims* dims, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                      int64_t rows, const float* q_weight, const float* k_weight, const int32_t* pos,
                      const float* inv_freq, const int32_t* axis, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, void* stream);

/*
 * Attention with a sliding window and visible first tokens over the paged cache of qmm_serve.h:
 * qmm_kv_attend where row r, of length n = row_len[r], sees the slots
 *     t < n  with  t >= n - window  or  t < sinks.
 * Slots are taken in their order, so this is for caches that are not cut by qmm_kv_evict.  A window of
 * at least max_pages * page_tokens leaves every slot below row_len visible: causal attention of a
 * prompt's rows.  Page table entries of pages that no row sees may hold anything, also between the windows of rows
 * that lie apart, and set no error; such pages are read there if their entries are in the pool, without effect.
 *  dims:       as for qmm_kv_attend, but max_agent_rows bounds a sequence's rows up to 2^24 / (heads / kv_heads).  The
 *              kernel follows from them, not from a call's rows: at most 128 rows times heads / kv_heads are a decode step's.
 *              Decode steps called with a prompt's max_agent_rows are right but slower (Q8_0, 4 sequences of 23,000, 3 rows:
 *              94 us with a max_agent_rows of 524, 45 with 3): a program that does both has dims for each.
 *  max_rows:   upper bound on rows; sizes the workspace.
 *  window >= 1, sinks >= 0.
 *  agent_rows, row_len, q, q_stride, out, out_type, lse, err_word: as for qmm_kv_attend.  Rows of no
 *              sequence, all rows where agent_rows falls, rows of a sequence with more than max_agent_rows and
 *              rows whose row_len is out of range set *err_word |= 4 and are written as rows that see nothing:
 *              out 0, lse -infinity.
 *  workspace:  16-byte aligned, at least qmm_kv_window_workspace_bytes bytes for the same dims, max_rows,
 *              window and sinks, in use until the call's kernels finish.  It may be null where that is 0.
 * A row's out and lse are bit-identical whatever the other rows and sequences of the call, as long as the V
 * that they see is finite (Q8_0: its scales below 512).  What lies in slots that a row does not see has no effect on
 * it, NaN and infinity included; a row that sees a score that is NaN has NaN throughout, and an element of V that is not finite
 * makes that element of out not finite (infinite or NaN) for the rows that see it.
 * A page table entry outside the pool (error word 2) takes its page's tokens out of the softmax.
 * Scores, softmax and sums are fp32, whatever the scores' size.  A probability enters the product with V rounded once to the
 * pool's 16-bit type (Q8_0: fp16), relative to the row's largest one (qmm_kv_attend keeps two parts of it); Q8_0's K and V are sums of two fp16 parts (quant times scale
 * without error, down to 2^-25).  An element of a Q8_0 pool is at most 65,504 in magnitude: a larger one of V counts
 * as not finite, one of K makes the rows that see it NaN.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, SCRATCH_TOO_SMALL, NO_DEVICE, CUDA.
 */
qmm_status qmm_kv_window_workspace_bytes(const qmm_kv_dims* dims, int64_t max_rows, int32_t window, int32_t sinks,
                                         int64_t* bytes);

qmm_status qmm_kv_attend_window(const qmm_kv_dims* dims, const void* pool, const int32_t* page_table,
                                const int32_t* agent_rows, const int32_t* row_len, const void* q, int64_t q_stride,
                                int64_t rows, int64_t max_rows, float scale, int32_t window, int32_t sinks, void* out,
                                int32_t out_type, float* lse, void* workspace, int64_t workspace_bytes, int* err_word,
                                void* stream);

/*
 * Verification of drafted tokens (speculative sampling).  A sequence's rows r0 .. r1 - 1 (agent_rows) are its
 * last token and its drafts: tokens[r0] is known, tokens[r] of a later row is a draft, drawn from the
 * distribution of draft_logits row r and judged by that of logits row r - 1,
 *     p = softmax(logits[r - 1] / temperature),  q = softmax(draft_logits[r] / temperature).
 * The drafts are taken in order while accept_u[r] * q(tokens[r]) < p(tokens[r]).  At the first that is refused
 * the next token is drawn from max(p - q, 0), without a refusal from the p of row r1 - 1: it is the lowest
 * column whose running sum passes sample_u times the sum of all.  So accepted tokens and the next one
 * are distributed as p, whatever q is.
 *  logits:      [rows][n] of `type`, row r at r * stride elements (the lm_head's y); aligned to its element.
 *  draft_logits: the same with draft_stride (a sequence's first row, the rows of a greedy one and rows of no
 *               sequence are not read), or null: every q is 1 at its draft (drafts looked up in the text).
 *  agent_rows:  int32 [agents + 1], non-decreasing.  If it falls, or a sequence's rows are not within
 *               0 .. rows, *err_word |= 4 and the sequences concerned (if it falls: all) are as ones without rows.
 *  temperature: fp32 [agents], or null (1).  0 (or less than 2^-100, or NaN) is greedy: a draft is taken if it
 *               is the lowest column of the row's largest logit, and so is the next token; draft_logits do not count.
 *  accept_u:    fp32 [rows] (a sequence's first is not read); sample_u: fp32 [agents]; both in [0, 1)
 *               (sample_u beyond counts as the nearest in it, a NaN as 0; an accept_u that is NaN refuses).
 *  accepted:    int32 [agents], drafts taken.   token: int32 [agents], the next token.
 *  prob:        fp32 [rows], min(1, p / q) of each draft, taken or not; 0 at a sequence's first row; or null.
 *               Rows of no sequence are left as they are.
 * -infinity is a column of probability 0.  A row of logits with a NaN, with +infinity or with nothing but
 * -infinity has no distribution: its draft is refused (prob NaN, 0 for the last kind), and a next token from it is -1.  A row of
 * draft_logits without one: the draft is refused (prob NaN, whatever its row of logits), and the next token is drawn from p.
 * A draft outside 0 .. n - 1 is refused (prob 0).  A sequence without rows: accepted 0, token -1.
 * Probabilities are formed to 2^-38 and summed exactly in 64-bit fixed point (a column of less than 2^-45 of the
 * row's largest counts as 0), so what is drawn does not depend on the order of a sum.  Where that leaves nothing of
 * max(p - q, 0), the next token is drawn from p.  A draft is judged by all the bits of its p and q, down to 2^-1000 of the row's
 * largest, below which they count as 0.  n is at most 2^19.
 *  workspace:   16-byte aligned, at least qmm_verify_workspace_bytes bytes, in use until the call's kernels finish.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, SCRATCH_TOO_SMALL, NO_DEVICE, CUDA.
 */
qmm_status qmm_verify_workspace_bytes(int64_t rows, int64_t n, int64_t* bytes);

qmm_status qmm_verify(const void* logits, int32_t type, int64_t stride, int64_t n, const void* draft_logits,
                      int64_t draft_stride, const int32_t* agent_rows, int32_t agents, int64_t rows,
                      const int32_t* tokens, const float* temperature, const float* accept_u, const float* sample_u,
                      int32_t* accepted, int32_t* token, float* prob, void* workspace, int64_t workspace_bytes,
                      int* err_word, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_DECODE_H */
