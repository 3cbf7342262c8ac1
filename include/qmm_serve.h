/*
 * qmm_serve -- the operators of a decode step around its matmuls, for one GB300 (sm_103a):
 * filling a paged KV cache, attention of new tokens over it with accumulated attention
 * weights, eviction by those weights, and log probabilities of tokens.  Part of libqmm.so;
 * status codes and conventions are those of qmm.h: no call aborts the process, every pointer
 * is device memory unless said otherwise, every call is ordered on `stream` (a cudaStream_t
 * passed as void*, NULL = legacy default stream), allocates nothing, synchronises nothing
 * and can be captured in a CUDA graph.
 *
 * The cache.  `agents` sequences share one pool of pages of page_tokens tokens; slot t of
 * sequence a is in page page_table[a][t / page_tokens] at t % page_tokens.  A sequence's
 * cache holds slots 0 .. len - 1; their order carries no meaning to the attention (K is
 * stored position-encoded), so an eviction may move a token to another slot of its KV head.
 * The record of (page P, KV head g) follows that of (P, g - 1):
 *   QMM_KV_F16, QMM_KV_BF16: K [page_tokens][head_dim], then V [page_tokens][head_dim], 16-bit;
 *     head_dim 64, 128 or 256, page_tokens 16, 32, 64, 128 or 256.
 *   QMM_KV_Q8_0: the 17,408-byte record of qmm_attn_decode (qmm.h); head_dim 128,
 *     page_tokens 64.  An element is its 32-dim block's fp16 scale times its int8 quant.
 * Two arrays beside the pool describe the slots, both [agents][kv_heads][max_pages *
 * page_tokens]: weight (fp32), the attention that the token has received, and pos (int32),
 * its position in the text.
 */
#ifndef QMM_SERVE_H
#define QMM_SERVE_H

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QMM_KV_Q8_0 = 0, QMM_KV_F16 = 1, QMM_KV_BF16 = 2 }; /* formats of the pool */
enum { QMM_TYPE_F32 = 0, QMM_TYPE_F16 = 1, QMM_TYPE_BF16 = 2 }; /* element types of arguments */

typedef struct {
    int32_t format;         /* QMM_KV_* */
    int32_t heads;          /* query heads, a multiple of kv_heads */
    int32_t kv_heads;
    int32_t head_dim;
    int32_t page_tokens;
    int32_t agents;         /* sequences: rows of page_table, at most 960 */
    int32_t max_pages;      /* columns of page_table */
    int32_t max_agent_rows; /* qmm_kv_attend: upper bound on one sequence's rows in a call, >= 1
                               (max_agent_rows * heads / kv_heads <= 4096); a sequence above
                               it sets *err_word |= 4 */
    int64_t pool_pages;     /* pages in the pool */
} qmm_kv_dims;

/*
 * The error word of the three cache calls: a device-visible int that the caller zeroes and
 * reads after synchronising.  It is or-ed with 1 if a device-side wait ran out, 2 if a page
 * table entry that was needed lies outside [0, pool_pages) (nothing is read or written
 * there), 4 if a sequence's rows or lengths are out of range (the sequence is left alone).
 */

/*
 * Append: row r of sequence a (rows agent_rows[a] .. agent_rows[a + 1] - 1, in order) goes to
 * slot cache_len[a] + (r - agent_rows[a]).
 *  k, v:       [rows][kv_heads][head_dim] of `type`, row r at r * k_stride (v_stride) elements:
 *              columns of a wider matrix, such as qmm_run's y, are taken in place.  Aligned
 *              to their element; 16-byte aligned rows are read faster.
 *  agent_rows: int32 [agents + 1], non-decreasing (else *err_word |= 4, and nothing is appended).
 *  cache_len:  int32 [agents], not changed.
 *  weight, pos: as above, or null.  The new slots' weight becomes 0 and, with row_pos
 *              (int32 [rows], or null) given, their pos row_pos[r].
 * F16 and BF16 pools take each value rounded once.  Q8_0, per 32 dims: d = fp16(max|x| / 127),
 * at most 65,504, and quant = x * (1 / d) rounded to the nearest integer (ties to even) in
 * -127 .. 127, all in fp32; a block with a NaN or an infinity gets d = NaN.
 * Pages shared between sequences must not be written to.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, NO_DEVICE, CUDA.
 */
qmm_status qmm_kv_append(const qmm_kv_dims* dims, void* pool, const int32_t* page_table,
                         const int32_t* agent_rows, const int32_t* cache_len, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, int32_t type, int64_t rows, float* weight, int32_t* pos,
                         const int32_t* row_pos, int* err_word, void* stream);

/*
 * Attention of new tokens: for row r of sequence a, query head h, g = h / (heads / kv_heads),
 *     out[r][h] = softmax over slots t < row_len[r] of (scale * q[r][h] . k_t), times v_t
 * and, with weight_out given, for every slot t below the sequence's largest row_len
 *     weight_out[a][g][t] = weight_in[a][g][t] + the sum of the softmax's t-th entries over the
 *                           sequence's rows and the heads of group g.
 * A row with row_len 0 sees nothing: its out is 0 and its lse -infinity.  What lies in slots
 * that a row does not see has no effect on it, NaN and infinity included; a row that sees a score that is
 * NaN has NaN throughout out and lse, and makes the weights of the slots that it sees NaN.
 *  agent_rows: int32 [agents + 1], non-decreasing (else *err_word |= 4, and no sequence of the call
 *              is attended to: every row is written as one that sees nothing, no weight is
 *              written); a sequence may have no rows.
 *  row_len:    int32 [rows], 0 <= row_len[r] <= max_pages * page_tokens.
 *  q:          [rows][heads][head_dim], fp16 (bf16 with a BF16 pool), row r at r * q_stride
 *              elements; 16-byte aligned, q_stride a multiple of 8.
 *  out:        [rows][heads][head_dim] of out_type (QMM_TYPE_*), 16-byte aligned.
 *  lse:        fp32 [rows][heads], the logarithm of each softmax's denominator; or null.
 *  weight_in:  or null (zeros); may be weight_out.  weight_out: or null (no weights).
 *  workspace:  16-byte aligned, at least qmm_kv_attend_workspace_bytes bytes, in use until the
 *              call's kernels finish.  It is sized by the table, not by the lengths: with weights mostly 4 bytes
 *              for every slot, KV head and query (max_agent_rows * heads / kv_heads, rounded up to 8).
 * A row's out and lse are bit-identical whatever the other rows and sequences of the call, as long as the V
 * that it sees is finite.  An infinity there makes that element of out infinite (a NaN, or infinities of
 * both signs: NaN); the last bits of the row's other elements then depend on whether every row of its
 * sequence sees it.  An element of a BF16 pool above 2^110 may leave fp32 by its product with a probability.
 * An entry of the page table outside the pool (error word 2) takes its tokens out of the softmax, and at head
 * dimension 128 those of up to 128 slots around them.
 * Scores, softmax and sums are fp32; the probabilities enter the product with V as the sum of
 * two 16-bit parts (relative error 2^-22, or 2^-38 of the row's largest one where that is more;
 * 2^-17 with BF16).  With Q8_0 the same holds of a probability times its token's largest V scale,
 * and V's elements are exact whatever the scales of a token's blocks.
 * Rows of no sequence set *err_word |= 4 and are written as rows that see nothing.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, SCRATCH_TOO_SMALL, NO_DEVICE, CUDA.
 */
qmm_status qmm_kv_attend_workspace_bytes(const qmm_kv_dims* dims, int32_t weights, int64_t* bytes);

qmm_status qmm_kv_attend(const qmm_kv_dims* dims, const void* pool, const int32_t* page_table,
                         const int32_t* agent_rows, const int32_t* row_len, const void* q, int64_t q_stride,
                         int64_t rows, float scale, void* out, int32_t out_type, float* lse, const float* weight_in,
                         float* weight_out, void* workspace, int64_t workspace_bytes, int* err_word, void* stream);

/*
 * Eviction: sequence a, if it holds more than keep[a] tokens (keep[a] < 0: no limit), is cut
 * to keep[a] tokens, per KV head: first those whose pos is below `sink` or at least
 * protect_from[a], then those of the largest weight; among equals the lowest slot (-0 equals
 * +0, a NaN weight is below every other).  Kept tokens in slots below keep[a] stay, and the
 * i-th kept token from slot keep[a] on, in slot order, moves into the i-th slot freed below:
 * sources and destinations never overlap, so the pool is changed in place.  Slots from
 * len_out[a] on are free afterwards; so are the pages that hold only such slots.  Pages that sequences share
 * must not hold a slot of one that is cut: tokens move into slots below keep[a], whoever else reads them.
 *  cache_len, keep: int32 [agents].  protect_from: int32 [agents], or null (no recent tokens
 *              are protected).
 *  weight, pos: the slots' arrays.  weight_out, pos_out: the same after the eviction, slots
 *              below len_out[a] only; may be weight and pos themselves.
 *  len_out:    int32 [agents] = min(cache_len[a], keep[a]); must not be cache_len.
 *  workspace:  16-byte aligned, at least qmm_kv_evict_workspace_bytes bytes.
 * A page table entry outside the pool leaves the tokens concerned unmoved, with their weight and pos: the
 * slots that they would have left and entered keep what they hold.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, MISALIGNED, SCRATCH_TOO_SMALL, NO_DEVICE, CUDA.
 */
qmm_status qmm_kv_evict_workspace_bytes(const qmm_kv_dims* dims, int64_t* bytes);

qmm_status qmm_kv_evict(const qmm_kv_dims* dims, void* pool, const int32_t* page_table, const int32_t* cache_len,
                        const int32_t* keep, int32_t sink, const int32_t* protect_from, const float* weight,
                        const int32_t* pos, float* weight_out, int32_t* pos_out, int32_t* len_out, void* workspace,
                        int64_t workspace_bytes, int* err_word, void* stream);

/*
 * Log probabilities over the n columns of each of m rows of logits (the lm_head's y):
 *  logits:      [m][n] of `type`, row r at r * stride elements; aligned to its element.
 *  tokens:      int32 [m][given]: logprob[r][i] = log softmax(row r)[tokens[r][i]], NaN for a
 *               token outside 0 .. n - 1.  given may be 0 (tokens and logprob unused).
 *  lse:         fp32 [m], log sum exp of the row.      (each of these two: or null)
 *  entropy:     fp32 [m], -sum p log p in nats.
 *  top_index:   int32 [m][top], the columns of the row's `top` largest logits, largest first,
 *               among equals the lowest column first; top_logprob: fp32 [m][top], their log
 *               probabilities.  0 <= top <= 32, top <= n.
 * -infinity is a column of probability 0.  A row of nothing else has lse = -infinity, entropy
 * 0 and every log probability -infinity.  A row with a NaN or +infinity has NaN throughout and
 * top_index -1.  m = 0 is a no-op.
 * Errors: INVALID_ARG, MISALIGNED, NO_DEVICE, CUDA.
 */
qmm_status qmm_logprobs(const void* logits, int32_t type, int64_t m, int64_t n, int64_t stride, const int32_t* tokens,
                        int32_t given, int32_t top, float* lse, float* entropy, float* logprob, int32_t* top_index,
                        float* top_logprob, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_SERVE_H */
