/*
 * tsl_attn.h -- what lies between the q/k/v column shards and the o row shard
 * of a transformer layer, on one AMD Instinct MI355X (gfx950): rotary
 * positions of the query and key heads (and their backward pass), a paged
 * cache of keys and values held in 4 bits, and attention over that cache.
 * Heads are the ranks' own ([mlxcel] "GQA-aware attention sharding"): a call
 * takes one rank's, or every rank's side by side.
 *
 * A library of its own (libtsl_attn.so) beside libtsl.so: the same types and
 * status codes, and the same conventions -- buffers owned by the caller, work
 * enqueued on `stream` without synchronising, every check on the host before
 * anything is enqueued, strides in elements (tsl.h, "Conventions shared by
 * every entry point").  Nothing throws across it.
 *
 * Heads.  A [rows][heads][head_dim] operand has its element (m, h, j) at
 * m * ld + h * head + j: token rows ld apart, heads `head` apart, in either
 * nesting (all heads of a token together, or all tokens of a head), its
 * elements one each.  A slice of a joint q/k/v product is such an operand.
 */
#ifndef TSL_ATTN_H
#define TSL_ATTN_H

#include "tsl.h"

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

/* How the two columns of a rotated pair lie in a head. */
typedef enum tsl_rotary_style {
    TSL_ROTARY_HALVES = 0, /* pair p is columns p and p + rot_dim / 2 */
    TSL_ROTARY_PAIRS = 1   /* pair p is columns 2 p and 2 p + 1       */
} tsl_rotary_style;

/* Positions of the rows of rotate_heads on one or several axes (a text has
 * one; images and video have time, height and width).
 *   positions: DEVICE int32 [axes][M], axes ld_pos elements apart (not read
 *              for one axis), any value.
 *   freq:      DEVICE binary32 [rot_dim / 2]: the angle of pair p per unit of
 *              position.
 *   pair_axis: null (all pairs on axis 0), or HOST [rot_dim / 2]: the axis of
 *              each pair, below axes.  Read during the call only.
 *   rot_dim:   even, 2 .. head_dim: columns rotated; the rest of a head is
 *              passed through.
 * 1 <= axes <= 4, head_dim up to 512. */
typedef struct tsl_rotary {
    const int32_t *positions;
    int64_t ld_pos;
    const float *freq;
    const uint8_t *pair_axis;
    int32_t axes, rot_dim, head_dim;
    int32_t style; /* tsl_rotary_style */
} tsl_rotary;

/* One operand of rotate_heads, X into Y: DEVICE [M][n_heads][head_dim] of
 * xdtype and ydtype (F32 or BF16).  Y may be X itself (same address, strides
 * and type). */
typedef struct tsl_rotate_item {
    const void *X;
    int64_t ldx, x_head;
    void *Y;
    int64_t ldy, y_head;
    int32_t n_heads, xdtype, ydtype;
} tsl_rotate_item;

/*
 * rotate_heads -- rotary positions: with the angle
 *     t = positions[axis(p)][m] * freq[p]
 * the columns (x1, x2) of pair p of every head of row m become
 *     y1 = x1 cos t - x2 sin t,   y2 = x2 cos t + x1 sin t,
 * rounded once.  inverse 1 rotates by -t: a rotation's backward pass (X the
 * gradient of the rotated heads, Y that of the heads).  The angle is formed
 * and reduced in binary64, so positions of any size keep binary32's accuracy.
 *   items: HOST array of 1 .. 8 items (a layer's q and k in one call).
 * M == 0 enqueues nothing.  M below 2^22, strides below 2^40.  No Y may share
 * an element with another Y or with any X (but its own, as stated).  Errors:
 * TSL_ERR_INVALID_ARG, TSL_ERR_UNSUPPORTED (sizes), TSL_ERR_MISALIGNED
 * (pointers aligned to their element size; 16-byte aligned rows and heads
 * run fastest), TSL_ERR_HIP.
 */
tsl_status rotate_heads(int32_t n_items, const tsl_rotate_item *items, int64_t M,
                        const tsl_rotary *rotary, int inverse, void *stream);

/* A paged cache of keys and values in 4 bits, for n_kv_heads heads of
 * head_dim (64, 128 or 256) columns: n_pages pages of page_tokens tokens (a
 * power of two, 32 .. 4096).  The format is that of TSL_Q4G64 weights: runs
 * of 64 columns of a head of a token share a bf16 scale s and bias b and hold
 * codes c in 0..15, the value s c + b.
 *
 * A page is a run of cache_size() / n_pages bytes, one record for each head
 * and each 32 tokens (heads outermost); pages are copied, moved and shared
 * whole.  With D = head_dim, W = D / 32, token t = 16 u + 4 g + r of the
 * record (u 0..1, g 0..3, r 0..3), a record is
 *     K codes, 16 D bytes: 32-bit words; word n = u W + w of lane
 *       16 h + (t mod 16) is at index (n / 4) 256 + lane 4 + n mod 4 and holds
 *       columns 32 w + 8 h + i, i 0..7, in bits 4 (i / 2 + 4 (i mod 2)) ...
 *     V codes, 16 D bytes: 32-bit words; word n of lane 16 g + j, at the
 *       index as above, holds column 16 n + j of the 8 tokens of g, token
 *       i = 4 u + r in bits 4 (i / 2 + 4 (i mod 2)) ...
 *     4 D bytes: for each 64 columns K scales, K biases, V scales, V biases,
 *       32 bf16 each, token t at 8 g + 4 u + r.
 * (what the matrix instructions' operand registers want). */
typedef struct tsl_cache {
    void *pages; /* DEVICE, 256-byte aligned, cache_size() bytes */
    int64_t n_pages;
    int32_t page_tokens, n_kv_heads, head_dim;
} tsl_cache;

/* The sequences of a call.  Sequence s has the operands' token rows
 * row_start[s] .. row_start[s + 1] - 1, which are the last tokens of its
 * context[s] ones: row i of n is at position context[s] - n + i, and the
 * token at position j lies in page page_table[s][j / page_tokens].
 *   row_start:  DEVICE int32 [n_seqs + 1], not descending.
 *   context:    DEVICE int32 [n_seqs], 0 .. 2^30 (a value outside counts as the
 *               nearer of the two).
 *   page_table: DEVICE int32 [n_seqs][max_pages], row stride ld_table.
 *   rows:       token rows the operands have; rows before row_start[0] and
 *               from row_start[n_seqs] on are not read and left as they were.
 *   max_rows:   no sequence has more rows (rows past it are left as they
 *               were).
 *   max_context: what the work is divided and the workspace sized for; longer
 *               contexts are right too, and slower.
 * The DEVICE arrays are read by the kernels, which go by their bounds: a
 * position before 0, or from max_pages page_tokens on, or in a page outside
 * 0 .. n_pages - 1 is not there (nothing is written to it, nothing read from
 * it, nothing attends to it).  n_seqs up to 65535, rows below 2^22, max_pages
 * page_tokens up to 2^30. */
typedef struct tsl_seqs {
    const int32_t *row_start;
    const int32_t *context;
    const int32_t *page_table;
    int64_t ld_table;
    int64_t rows;
    int32_t n_seqs, max_rows, max_context, max_pages;
} tsl_seqs;

/* cache_size -- bytes of a cache's pages (`pages` is not read).  Host only. */
tsl_status cache_size(const tsl_cache *cache, size_t *bytes);

/*
 * cache_append -- the keys and values of the rows of `seqs` go into the
 * cache at their positions, each run x of 64 columns as
 *     b = bf16(min x),  s = bf16((max x - b) / 15),
 *     c = clamp(round((x - b) / s), 0, 15)          (s = 0: c = 0)
 * where b and s are formed in binary32 and rounded to nearest even, and the
 * quotient is rounded exactly, ties to even.  (Where b, rounded, lies above
 * all of a narrow run, s is negative and the codes count down from b.)  A run with
 * a value that is not finite, or whose s or b is not (max x - b past binary32's
 * range), has a scale and a bias of NaN: all of it reads NaN.
 *   K, V: DEVICE [rows][n_kv_heads][head_dim] of type dtype (F32 or BF16).
 * Other tokens of the pages keep their bits.  A page that a call writes to
 * belongs to one of its sequences (copy a shared page first), and K and V
 * share no byte with the cache.  Errors: TSL_ERR_INVALID_ARG,
 * TSL_ERR_UNSUPPORTED (sizes; n_kv_heads times the records of max_rows tokens from
 * 2^24 on), TSL_ERR_MISALIGNED (K, V 16-byte aligned, strides whole
 * 16 bytes; pages 256 bytes), TSL_ERR_HIP.
 */
tsl_status cache_append(const tsl_cache *cache, const tsl_seqs *seqs, tsl_dtype dtype,
                        const void *K, int64_t ldk, int64_t k_head, const void *V, int64_t ldv,
                        int64_t v_head, void *stream);

/*
 * cache_read -- the values s c + b of the rows' tokens, in binary32, rounded
 * once to dtype (F32 or BF16).  K, V: DEVICE [rows][n_kv_heads][head_dim],
 * either may be null.  Rows whose position is not there get zeros.  Alignment
 * and errors as cache_append.
 */
tsl_status cache_read(const tsl_cache *cache, const tsl_seqs *seqs, tsl_dtype dtype, void *K,
                      int64_t ldk, int64_t k_head, void *V, int64_t ldv, int64_t v_head,
                      void *stream);

/* cache_attention_workspace_size -- workspace bytes cache_attention needs (of
 * cache and seqs only the sizes are read).  0 for some calls, up to about 1 GiB
 * more than the partial sums' where prompts of several hundred rows have long
 * contexts.  Host only. */
tsl_status cache_attention_workspace_size(const tsl_cache *cache, const tsl_seqs *seqs,
                                          int32_t n_q_heads, int32_t window, int32_t sinks,
                                          size_t *bytes);

/*
 * cache_attention -- softmax attention of the rows of `seqs` over their
 * cached tokens, their own (appended before the call) included:
 *     o = sum_j p_j v_j,   p = softmax over the visible j of scale q . k_j
 * A row at position i sees the tokens j <= i with
 *     j > i - window  (window 0: all)   or   j < sinks.
 * Query head h reads K/V head h / (n_q_heads / n_kv_heads).  A row that sees
 * no token gets zeros.  A token that a row does not see has no influence on
 * it, whatever its page holds (but for the scaling below); a visible K run that
 * reads NaN makes the row NaN, a visible V run its 64 columns.
 *   Q: DEVICE [rows][n_q_heads][head_dim], BF16.
 *   O: DEVICE [rows][n_q_heads][head_dim], type odtype (F32 or BF16).
 *   workspace: 256-byte aligned, cache_attention_workspace_size() bytes; may
 *      be null when that is 0.  Calls that overlap in time need one each.
 * Products accumulate in binary32, the softmax is binary32.  For sequences of
 * up to 64 query rows a K/V head (rows times n_q_heads / n_kv_heads; of a lone
 * sequence max_rows times that), and with head_dim 256, the 4-bit values enter
 * exactly and a probability times a value's scale with 16 bits (with equal weights
 * the mean of n independent values, any n, is within 2^-14 of their runs' range,
 * max - min, over the root of n, in the 2-norm).  For longer ones K, Q and V are
 * rounded to 11 bits (binary16), as the probabilities are, scaled by a power of
 * two that up to 128 neighbouring tokens which some row of the sequence sees have
 * in common: values below 2^-22 of the largest of those lose bits, as do values
 * below 2^-90 of an earlier one that the row gave weight to, and elements of Q
 * below 2^-31 of their head's largest; probabilities below 2^-23 of the row's
 * largest so far lose bits, and below 2^-31 they are 0.  Both kinds may be in one
 * call (generated tokens beside a prompt's chunk).  |Q| stays below 2^110, scale
 * sum |q k| of a visible token within binary32's range, and sum |v| over a row's
 * tokens below 2^110 (what other rows get does not hang on a row that does not keep
 * to it).  Equal calls give equal bits.  O shares no byte with Q, the cache or the
 * workspace.  With head_dim 256 each 16 query rows expand the records they see for
 * themselves, so prompts take four to six times as long as with 128 for the same
 * operations (4096 rows of 16 / 8 heads 868 us).  scale log2(e) is finite, window and sinks 0 .. 2^30.
 * Errors: TSL_ERR_INVALID_ARG, TSL_ERR_NOT_DIVISIBLE (n_q_heads by
 * n_kv_heads), TSL_ERR_UNSUPPORTED (sizes; 2^30 query rows of a K/V head; calls
 * whose sequences, all counted as long as the longest -- with head_dim 64 and 128
 * as 64 query rows at most --, come to 2^26 tiles of 4 to 16 query rows may be),
 * TSL_ERR_BUFFER_TOO_SMALL, TSL_ERR_MISALIGNED (Q, O 16-byte aligned, strides
 * whole 16 bytes), TSL_ERR_HIP.
 */
tsl_status cache_attention(const tsl_cache *cache, const tsl_seqs *seqs, int32_t n_q_heads,
                           const void *Q, int64_t ldq, int64_t q_head, float scale, int32_t window,
                           int32_t sinks, tsl_dtype odtype, void *O, int64_t ldo, int64_t o_head,
                           void *workspace, size_t ws_bytes, void *stream);

/* The HIP runtime's description of the error behind the most recent
 * TSL_ERR_HIP an entry point of this header returned on the calling thread
 * ("no error" if none). */
const char *tsl_attn_last_hip_error_string(void);

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif

#ifdef __cplusplus
}
#endif

#endif /* TSL_ATTN_H */
