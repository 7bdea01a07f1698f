/*
 * tsl_block.h -- what lies between and around the shard products of tsl.h in
 * a transformer layer, on one AMD Instinct MI355X (gfx950): the
 * residual-adding root-mean-square norm, shard products with an epilogue
 * (bias, activation, residual), the gated feed-forward block, and their
 * backward passes.
 *
 * A library of its own (libtsl_block.so) beside libtsl.so: the same types,
 * status codes, packed weights (pack_shard) and shard plans, and the same
 * conventions -- buffers owned by the caller, work enqueued on `stream`
 * without synchronising, every check on the host before anything is
 * enqueued, leading dimensions in elements (tsl.h, "Conventions shared by
 * every entry point").  Nothing throws across it.
 */
#ifndef TSL_BLOCK_H
#define TSL_BLOCK_H

#include "tsl.h"

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#pragma GCC visibility push(default)
#endif

/*
 * add_rms_norm -- the root-mean-square norm between a row-parallel product
 * and the next column-parallel ones ([mlxcel] "Row Parallel": the rank
 * partials of o_proj / down_proj are summed before the next block reads
 * them), with the rank sum and the residual stream's addition in the same
 * pass:
 *     r[m][j] = (((P_0 + P_1) + P_2) + ...)[m][j] + residual[m][j]
 *     y[m][j] = r[m][j] * rstd[m] * weight[j],
 *     rstd[m] = 1 / sqrt(mean_j r[m][j]^2 + eps)
 * in binary32 throughout (y is formed from the unrounded r).
 *   parts:    HOST array of n_parts DEVICE pointers, [M][n] each, row stride
 *             ld_part, type pdtype (F32 or BF16); 1 <= n_parts <= 64.  One
 *             part and no residual is the plain norm.
 *   residual: null, or DEVICE [M][n], row stride ldr, type rdtype (F32/BF16).
 *   sum_out:  null, or DEVICE [M][n], row stride ld_sum, type rdtype:
 *             receives r (rounded once), the new residual stream.  It may be
 *             the residual itself (same address and row stride).
 *   weight:   null (ones), or DEVICE [n], type wdtype (F32 or BF16).
 *   Y:        DEVICE [M][n], row stride ldy, type ydtype: F32, BF16 (rounded
 *             once), or E4M3: 8-bit values q with binary32 scales, y = s q,
 *             one s per run of `group` columns (group 32, 64 or 128; the
 *             last run of a row may be short) or per row (group 0):
 *             s = max |y| / 448 over the run, and q the quotient y / s (both
 *             divisions in binary32) rounded to nearest even; a run of zeros
 *             (or of values up to 224 * 2^-149, whose s rounds to 0) has
 *             s = 0 and q = 0, a run with a value that is not finite an s
 *             that is not finite and q NaN.  The products of these headers
 *             read F32 and BF16; the 8-bit form is for a consumer of the
 *             caller's.
 *   scales:   DEVICE binary32 [M][ceil(n / group)] ([M] for group 0) for
 *             E4M3, else null (and group 0).
 *   rstd:     null, or DEVICE binary32 [M]: receives rstd (for the backward
 *             pass).
 * 1 <= n <= 32768 (TSL_ERR_UNSUPPORTED above); M < 2^22 and row strides below
 * 2^31.  M == 0 enqueues nothing.  No output may overlap an input or another
 * output (except sum_out as stated).  Errors: TSL_ERR_INVALID_ARG,
 * TSL_ERR_UNSUPPORTED, TSL_ERR_MISALIGNED (pointers aligned to their element
 * size; 16-byte aligned rows run fastest), TSL_ERR_HIP.
 */
tsl_status add_rms_norm(int32_t n_parts, const void *const *parts, tsl_dtype pdtype,
                        int64_t ld_part, int64_t M, int64_t n, const void *residual,
                        tsl_dtype rdtype, int64_t ldr, void *sum_out, int64_t ld_sum,
                        const void *weight, tsl_dtype wdtype, float eps, tsl_dtype ydtype, void *Y,
                        int64_t ldy, float *scales, int32_t group, float *rstd, void *stream);

/* add_rms_norm_grad_workspace_size -- workspace bytes of add_rms_norm_grad
 * with a weight gradient (without one it needs none). */
tsl_status add_rms_norm_grad_workspace_size(int64_t M, int64_t n, size_t *bytes);

/*
 * add_rms_norm_grad -- the backward pass of add_rms_norm: with x the sum it
 * kept (sum_out), t = dy * weight and xh = x * rstd,
 *     dx[m][j] = rstd[m] * (t[m][j] - xh[m][j] * mean_j(t[m][j] xh[m][j]))
 *                + dres[m][j]
 *     dw[j] (+)= sum_m dy[m][j] * xh[m][j]
 * dx is the gradient of the residual and of every part alike (the sum passes
 * it on unchanged); dres is the gradient that reaches the residual stream
 * (sum_out) from its other readers.
 *   dY:     DEVICE [M][n], row stride lddy, type dydtype (F32 or BF16).
 *   X:      DEVICE [M][n], row stride ldx, type xdtype (F32 or BF16).
 *   weight: null (ones), or DEVICE [n], type wdtype.
 *   rstd:   null (recomputed from X and eps), or DEVICE binary32 [M] as kept
 *           by add_rms_norm (eps is then not read).
 *   dres:   null, or DEVICE [M][n], row stride ld_dres, type dxdtype; it may
 *           be dX itself (same address and row stride).
 *   dX:     null, or DEVICE [M][n], row stride lddx, type dxdtype.
 *   dW:     null, or DEVICE binary32 [n]; accumulate_dw 1 adds to it.  The
 *           rows are added in a fixed order: equal calls give equal bits.
 *   workspace: 256-byte aligned, add_rms_norm_grad_workspace_size() bytes
 *           when dW is wanted (else may be null).
 * M == 0 writes only dW (zeros, unless it accumulates).  Width and row limits
 * as add_rms_norm.  Errors: TSL_ERR_INVALID_ARG, TSL_ERR_UNSUPPORTED,
 * TSL_ERR_BUFFER_TOO_SMALL, TSL_ERR_MISALIGNED, TSL_ERR_HIP.
 */
tsl_status add_rms_norm_grad(int64_t M, int64_t n, const void *dY, tsl_dtype dydtype, int64_t lddy,
                             const void *X, tsl_dtype xdtype, int64_t ldx, const void *weight,
                             tsl_dtype wdtype, float eps, const float *rstd, const void *dres,
                             int64_t ld_dres, void *dX, tsl_dtype dxdtype, int64_t lddx, float *dW,
                             int accumulate_dw, void *workspace, size_t ws_bytes, void *stream);

/* Activations of the epilogue and of the gated block. */
typedef enum tsl_act {
    TSL_ACT_NONE = 0,
    TSL_ACT_RELU = 1,     /* max(v, 0)                                         */
    TSL_ACT_SILU = 2,     /* v / (1 + exp(-v))                                 */
    TSL_ACT_GELU = 3,     /* v (1 + erf(v / sqrt 2)) / 2                       */
    TSL_ACT_GELU_TANH = 4 /* v (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3))) / 2   */
} tsl_act;

/* What a product goes through before it is stored (shard_linear_group_epilogue):
 *     Y = act(X W + bias) + residual
 * in binary32, rounded once to the item's ydtype.
 *   bias:     null, or DEVICE [n_len] (the shard's own columns), type
 *             bias_dtype (F32 or BF16).
 *   residual: null, or DEVICE [rows][n_len], row stride ld_res, type
 *             res_dtype (F32 or BF16): row i is added to row i of the
 *             product.  It may be the item's Y itself (same address, row
 *             stride and type): the residual stream updated in place.
 *   pre:      null, or DEVICE [rows][n_len], row stride ld_pre, type
 *             pre_dtype: receives X W + bias (rounded once), what the
 *             activation's backward pass needs. */
typedef struct tsl_epilogue {
    const void *bias;
    const void *residual;
    void *pre;
    int64_t ld_res;
    int64_t ld_pre;
    int32_t act; /* tsl_act */
    int32_t bias_dtype, res_dtype, pre_dtype;
} tsl_epilogue;

/* shard_linear_group_epilogue_workspace_size -- workspace bytes
 * shard_linear_group_epilogue needs (items as for
 * shard_linear_group_workspace_size; of the epilogues only whether one is
 * null is read).  0 for most calls of up to 64 rows. */
tsl_status shard_linear_group_epilogue_workspace_size(int32_t n_items,
                                                      const tsl_linear_item *items,
                                                      const tsl_epilogue *const *epilogues,
                                                      tsl_dtype wdtype, int64_t M, size_t *bytes);

/*
 * shard_linear_group_epilogue -- shard_linear_group (tsl.h) with bias,
 * activation and residual in the products' epilogue: the same items, types,
 * sum sets, row counts, row indices, workspace rules and errors.
 *   epilogues: HOST array of n_items HOST pointers, read during the call
 *              only; epilogues[i] belongs to item i (null: the plain
 *              product).  Of a sum set the first item's applies, once, to the
 *              set's sum -- bias and residual of a row-parallel layer are
 *              added after the ranks' partials ([mlxcel] "Row Parallel") --
 *              and those of its other members must be null.  A set's products
 *              are added in binary32 over the members' k-ranges in item
 *              order; equal calls give equal bits, but not those of separate
 *              products added afterwards.
 * accumulate must be 0 for an item with an epilogue; ld_res and ld_pre are
 * below 2^31.  No output (Y, pre) may share an element with another output or
 * with any X, bias or residual (except a residual that is its own item's Y).
 */
tsl_status shard_linear_group_epilogue(int32_t n_items, const tsl_linear_item *items,
                                       const tsl_epilogue *const *epilogues, tsl_dtype wdtype,
                                       tsl_dtype xdtype, int64_t M, void *workspace,
                                       size_t ws_bytes, void *stream);

/*
 * One gated feed-forward block of a grouped call:
 *     H = act(X W_gate) * (X W_up)
 * ([mlxcel] "Architecture-aware shard plan": gate and up are column shards
 * over the same columns, and H, sharded by those columns, is the input of
 * the down projection's row shard.)  gate and up are HOST shards of equal
 * k_len and n_len, packed by pack_shard with the call's wdtype, packed_bytes
 * the size of either buffer.  X, ldx, rows, row_index and x_rows as in
 * tsl_linear_item.  H: DEVICE [rows][n_len], row stride ldh, type hdtype
 * (F32 or BF16), formed in binary32 from the two products and rounded once.
 * G, U: null, or DEVICE [rows][n_len], row stride ld_gu, type hdtype: receive
 * X W_gate and X W_up (rounded once) for the backward pass; either both or
 * none, ld_gu below 2^31.  They have H's type, and shard_gated_grad reads the
 * weights': keep them from a call whose hdtype is the weights' type.
 */
typedef struct tsl_gated_item {
    const tsl_shard *gate, *up;
    const void *packed_gate, *packed_up;
    size_t packed_bytes;
    const void *X;
    int64_t ldx;
    void *H;
    int64_t ldh;
    void *G, *U;
    int64_t ld_gu;
    const int32_t *row_index;
    int64_t x_rows;
    int32_t hdtype;
    int32_t rows;
} tsl_gated_item;

/* shard_gated_group_workspace_size -- workspace bytes shard_gated_group needs
 * for these items (only their shards, rows and whether row_index is null are
 * read), weight type and M. */
tsl_status shard_gated_group_workspace_size(int32_t n_items, const tsl_gated_item *items,
                                            tsl_dtype wdtype, int64_t M, size_t *bytes);

/*
 * shard_gated_group -- gated feed-forward blocks with the same activation
 * and types in one pass, each over M rows or its own row count: one rank's
 * shard, every rank's, or the experts of a mixture-of-experts layer over the
 * tokens routed to each (row_index).  Types, alignment, limits and errors as
 * shard_linear_group; 1 <= n_items <= 2048.  No output (H, G, U) may share an
 * element with another output or any X or row index.
 */
tsl_status shard_gated_group(int32_t n_items, const tsl_gated_item *items, tsl_act act,
                             tsl_dtype wdtype, tsl_dtype xdtype, int64_t M, void *workspace,
                             size_t ws_bytes, void *stream);

/*
 * transpose_shard -- the shard of W^T that a shard of W is: K and N, the
 * offsets and lengths change places, a column shard becomes a row shard
 * (combine SUM: the ranks' input gradients add up) and a row shard a column
 * shard (CONCAT).  Packing it with the strides of W swapped,
 *     pack_shard(&t, wdtype, W, stride_n, stride_k, ...),
 * gives the weight that the backward pass reads.  Host only.
 */
tsl_status transpose_shard(const tsl_shard *shard, tsl_shard *out);

/* shard_linear_grad_workspace_size -- workspace bytes shard_linear_grad needs
 * at most for this shard, weight type and row count, whatever outputs are
 * wanted. */
tsl_status shard_linear_grad_workspace_size(const tsl_shard *shard, tsl_dtype wdtype, int64_t M,
                                            size_t *bytes);

/*
 * shard_linear_grad -- the backward pass of one rank's shard product with an
 * epilogue, Y = act(Z) + residual, Z = X W + bias (the residual's gradient is
 * dY itself).  With dZ = dY act'(Z):
 *     dX[m][i] = sum_j dZ[m][j] W[i][j]            i < k_len, j < n_len
 *     dW[i][j] (+)= sum_m X[m][i] dZ[m][j]
 *     db[j] (+)= sum_m dZ[m][j]
 * For a column shard dX is the rank's partial of the input gradient (the
 * ranks' partials add up, combine_partials SUM).
 *   shard:    the forward's shard; wdtype F32 or BF16 (4-bit weights are
 *             TSL_ERR_UNSUPPORTED: their groups run along the other axis).
 *   packed_t: the transposed shard, packed (transpose_shard); not read when
 *             dX is null.
 *   X, Z, dY: DEVICE rows of wdtype at strides ldx, ldz, lddy (as
 *             shard_linear's X: 16-byte aligned, strides whole 16 bytes).  Z
 *             is the kept pre-activation (tsl_epilogue.pre), not read for
 *             TSL_ACT_NONE; X is not read when dW is null.
 *   dX:       null, or DEVICE [M][k_len], row stride lddx, F32 or BF16.
 *   dW:       null, or DEVICE, type dwdtype (F32 or BF16): element (i, j) at
 *             i * dw_stride_k + j * dw_stride_n, one of the strides 1 (a
 *             [K][N] or an [N][K] array).  accumulate_dw 1 (F32 only) adds to
 *             it, and to db.
 *   db:       null, or DEVICE binary32 [n_len], summed from the unrounded dZ
 *             in a fixed order.
 * Products accumulate in binary32; with an activation dZ is their operand
 * rounded once to wdtype (BF16 and M * n_len up to 2^16: together with what
 * that rounding left, so that it does not show; an infinity in X or the weight
 * may then give NaN).  Slope of relu at 0 is 0.  M == 0 writes zero
 * weight and bias gradients (unless they accumulate).  M, k_len and n_len
 * below 2^22 - 64, the product of any two of them at most 2^34 (F32: 2^32);
 * input strides below 2^22, output strides below 2^31.  No output may share an
 * element with an input, another output or the workspace.  Errors as
 * shard_linear.
 */
tsl_status shard_linear_grad(const tsl_shard *shard, tsl_dtype wdtype, const void *packed_t,
                             size_t packed_t_bytes, int64_t M, const void *X, int64_t ldx,
                             tsl_act act, const void *Z, int64_t ldz, const void *dY, int64_t lddy,
                             tsl_dtype dxdtype, void *dX, int64_t lddx, tsl_dtype dwdtype, void *dW,
                             int64_t dw_stride_k, int64_t dw_stride_n, int accumulate_dw, float *db,
                             void *workspace, size_t ws_bytes, void *stream);

/* shard_gated_grad_workspace_size -- workspace bytes shard_gated_grad needs
 * at most for these shards, weight type and row count. */
tsl_status shard_gated_grad_workspace_size(const tsl_shard *gate, const tsl_shard *up,
                                           tsl_dtype wdtype, int64_t M, size_t *bytes);

/*
 * shard_gated_grad -- the backward pass of one gated feed-forward block
 * (shard_gated_group), from the kept products G and U:
 *     dG = dH U act'(G),  dU = dH act(G)
 *     dX = dG W_gate^T + dU W_up^T
 *     dW_gate (+)= X^T dG,  dW_up (+)= X^T dU
 *   G, U:  DEVICE [M][n_len] of wdtype, row stride ld_gu.
 *   dH:    DEVICE [M][n_len] of wdtype, row stride lddh.
 *   packed_gate_t, packed_up_t: the transposed shards, packed; packed_t_bytes
 *          the size of either buffer.
 *   dW_gate, dW_up: both or neither, with the strides of shard_linear_grad's
 *          dW.
 * dG and dU are the products' operands, rounded as shard_linear_grad's dZ;
 * the two terms of dX are added in binary32.  Everything else as shard_linear_grad.
 */
tsl_status shard_gated_grad(const tsl_shard *gate, const tsl_shard *up, tsl_dtype wdtype,
                            const void *packed_gate_t, const void *packed_up_t,
                            size_t packed_t_bytes, int64_t M, const void *X, int64_t ldx,
                            tsl_act act, const void *G, const void *U, int64_t ld_gu,
                            const void *dH, int64_t lddh, tsl_dtype dxdtype, void *dX, int64_t lddx,
                            tsl_dtype dwdtype, void *dW_gate, void *dW_up, int64_t dw_stride_k,
                            int64_t dw_stride_n, int accumulate_dw, void *workspace,
                            size_t ws_bytes, void *stream);

/* The HIP runtime's description of the error behind the most recent
 * TSL_ERR_HIP an entry point of this header returned on the calling thread
 * ("no error" if none). */
const char *tsl_block_last_hip_error_string(void);

#if defined(__GNUC__)
#pragma GCC visibility pop
#endif

#ifdef __cplusplus
}
#endif

#endif /* TSL_BLOCK_H */
