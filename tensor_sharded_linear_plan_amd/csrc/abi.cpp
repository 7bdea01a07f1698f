// The C ABI of tsl.h: host-side validation and dispatch to the gfx950
// kernels (group.hpp).  Every check runs before anything is enqueued, so a
// rejected call has no side effects.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstddef>
#include <vector>

#include "group.hpp"
#include "internal.hpp"
#include "tsl.h"

using namespace tsl;

extern "C" tsl_status pack_shard_size(const tsl_shard *shard, tsl_dtype wdtype, size_t *bytes) {
    if (!shard || !bytes)
        return TSL_ERR_INVALID_ARG;
    PackGeom g;
    tsl_status st = geometry(*shard, wdtype, &g);
    if (st != TSL_OK)
        return st;
    *bytes = g.total_bytes;
    return TSL_OK;
}

extern "C" tsl_status pack_shard(const tsl_shard *shard, tsl_dtype wdtype, const void *W,
                                 int64_t stride_k, int64_t stride_n, const void *scales,
                                 const void *biases, int64_t sb_stride_g, int64_t sb_stride_n,
                                 void *packed, size_t packed_bytes, void *stream) {
    if (!shard || !W || !packed)
        return TSL_ERR_INVALID_ARG;
    PackGeom g;
    tsl_status st = geometry(*shard, wdtype, &g);
    if (st != TSL_OK)
        return st;
    if (stride_k < 0 || stride_n < 0)
        return TSL_ERR_INVALID_ARG;
    if (wdtype == TSL_Q4G64) {
        if (!scales || !biases || sb_stride_g < 0 || sb_stride_n < 0)
            return TSL_ERR_INVALID_ARG;
    } else if (scales || biases) {
        return TSL_ERR_INVALID_ARG;
    }
    if (packed_bytes < g.total_bytes)
        return TSL_ERR_BUFFER_TOO_SMALL;
    if (!aligned(packed, 256))
        return TSL_ERR_MISALIGNED;
    const size_t esz = wdtype == TSL_F32 ? 4 : (wdtype == TSL_BF16 ? 2 : 1);
    if (!aligned(W, esz) || (wdtype == TSL_Q4G64 && (!aligned(scales, 2) || !aligned(biases, 2))))
        return TSL_ERR_MISALIGNED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (wdtype == TSL_Q4G64)
        e = launch_pack_q4(g, static_cast<const uint8_t *>(W), stride_k, stride_n,
                           static_cast<const uint16_t *>(scales),
                           static_cast<const uint16_t *>(biases), sb_stride_g, sb_stride_n,
                           shard->k_off, shard->n_off, packed, s);
    else
        e = launch_pack_dense(g, wdtype, W, stride_k, stride_n, shard->k_off, shard->n_off, packed,
                              s);
    return from_hip(e);
}

// the item table's layout is part of the ABI
static_assert(sizeof(tsl_linear_item) == 88 && offsetof(tsl_linear_item, rows) == 68 &&
                  offsetof(tsl_linear_item, row_index) == 72 &&
                  offsetof(tsl_linear_item, x_rows) == 80,
              "tsl_linear_item layout");

extern "C" tsl_status shard_linear_workspace_size(const tsl_shard *shard, tsl_dtype wdtype,
                                                  int64_t M, size_t *bytes) {
    if (!shard || !bytes || M < 0)
        return TSL_ERR_INVALID_ARG;
    std::vector<LinearItem> items(1);
    tsl_status st = geometry(*shard, wdtype, &items[0].g);
    if (st != TSL_OK)
        return st;
    items[0].M = M;
    *bytes = group_workspace(items, wdtype, M);
    return TSL_OK;
}

extern "C" tsl_status shard_linear(const tsl_shard *shard, tsl_dtype wdtype, const void *packed,
                                   size_t packed_bytes, tsl_dtype xdtype, const void *X,
                                   int64_t ldx, int64_t M, tsl_dtype ydtype, void *Y, int64_t ldy,
                                   int accumulate, void *workspace, size_t ws_bytes,
                                   void *stream) {
    if (M < 0)
        return TSL_ERR_INVALID_ARG;
    tsl_status st = check_types(wdtype, xdtype);
    if (st != TSL_OK)
        return shard && packed && X && Y ? st : TSL_ERR_INVALID_ARG;
    std::vector<LinearItem> items(1);
    st = check_item(shard, wdtype, packed, packed_bytes, xdtype, X, ldx, M, ydtype, Y, ldy,
                    accumulate, &items[0]);
    if (st != TSL_OK)
        return st;
    return run_group(items, wdtype, M, workspace, ws_bytes, stream);
}

extern "C" tsl_status shard_linear_group_workspace_size(int32_t n_items,
                                                        const tsl_linear_item *items,
                                                        tsl_dtype wdtype, int64_t M,
                                                        size_t *bytes) {
    if (!items || !bytes || n_items < 1 || n_items > kMaxItems || M < 0)
        return TSL_ERR_INVALID_ARG;
    std::vector<LinearItem> v(n_items);
    int32_t first = 0;
    bool accumulates = false;
    for (int32_t i = 0; i < n_items; ++i) {
        if (!items[i].shard || (items[i].sum_next != 0 && items[i].sum_next != 1) ||
            items[i].rows < 0 || items[i].rows > M)
            return TSL_ERR_INVALID_ARG;
        tsl_status st = geometry(*items[i].shard, wdtype, &v[i].g);
        if (st != TSL_OK)
            return st;
        v[i].M = items[i].rows ? items[i].rows : M;
        v[i].ridx = items[i].row_index; // only whether it is null matters here
        v[i].x_rows = 1;
        v[i].set_pos = i - first;
        // part of the plan (a set's items do not accumulate)
        v[i].accumulate = v[i].set_pos == 0 && items[i].accumulate == 1;
        accumulates = accumulates || v[i].accumulate;
        if (!items[i].sum_next || i == n_items - 1) {
            v[first].set_len = i - first + 1;
            for (int32_t r = first + 1; r <= i; ++r)
                v[r].set_len = 0;
            first = i + 1;
        }
    }
    *bytes = group_workspace(v, wdtype, M);
    if (accumulates) { // the same items storing their products fit too
        for (LinearItem &L : v)
            L.accumulate = 0;
        *bytes = std::max(*bytes, group_workspace(v, wdtype, M));
    }
    return TSL_OK;
}

extern "C" tsl_status shard_linear_group(int32_t n_items, const tsl_linear_item *items,
                                         tsl_dtype wdtype, tsl_dtype xdtype, int64_t M,
                                         void *workspace, size_t ws_bytes, void *stream) {
    std::vector<LinearItem> v;
    tsl_status st = gather(n_items, items, wdtype, xdtype, M, &v);
    if (st != TSL_OK)
        return st;
    return run_group(v, wdtype, M, workspace, ws_bytes, stream);
}

extern "C" tsl_status shard_linear_group_noalloc(int32_t n_items, const tsl_linear_item *items,
                                                 tsl_dtype wdtype, tsl_dtype xdtype, int64_t M,
                                                 void *stream) {
    std::vector<LinearItem> v;
    tsl_status st = gather(n_items, items, wdtype, xdtype, M, &v);
    if (st != TSL_OK)
        return st;
    // the exact workspace of this call (its items carry their X pointers, so
    // shared activation copies are counted once), checked before any device
    // call
    const size_t need = group_workspace(v, wdtype, M);
    if (need > kNoAllocScratchBytes)
        return TSL_ERR_BUFFER_TOO_SMALL;
    void *scr = nullptr;
    if (need > 0) {
        hipError_t e = noalloc_scratch(&scr);
        if (e != hipSuccess)
            return from_hip(e);
    }
    return run_group(v, wdtype, M, scr, need > 0 ? kNoAllocScratchBytes : 0, stream);
}

extern "C" tsl_status combine_partials(tsl_combine mode, int32_t n_parts, const void *const *parts,
                                       tsl_dtype pdtype, int64_t M, int64_t n_each,
                                       int64_t ld_part, tsl_dtype ydtype, void *Y, int64_t ldy,
                                       void *stream) {
    if (!parts || !Y || n_parts < 1 || n_parts > kMaxParts || M < 0 || n_each < 0)
        return TSL_ERR_INVALID_ARG;
    for (int r = 0; r < n_parts; ++r)
        if (!parts[r])
            return TSL_ERR_INVALID_ARG;
    if (pdtype != TSL_F32 && pdtype != TSL_BF16)
        return TSL_ERR_INVALID_ARG;
    if (ydtype != TSL_F32 && ydtype != TSL_BF16)
        return TSL_ERR_INVALID_ARG;
    if (ld_part < n_each)
        return TSL_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (mode == TSL_COMBINE_SUM) {
        if (pdtype != TSL_F32)
            return TSL_ERR_UNSUPPORTED;
        if (ldy < n_each)
            return TSL_ERR_INVALID_ARG;
        for (int r = 0; r < n_parts; ++r)
            if (!aligned(parts[r], 4))
                return TSL_ERR_MISALIGNED;
        if (!aligned(Y, ydtype == TSL_F32 ? 4 : 2))
            return TSL_ERR_MISALIGNED;
        if (M == 0 || n_each == 0)
            return TSL_OK;
        const size_t ye = ydtype == TSL_F32 ? 4 : 2;
        for (int r = 0; r < n_parts; ++r) {
            const bool in_place =
                r == 0 && parts[0] == Y && ydtype == TSL_F32 && ldy == ld_part;
            if (!in_place && overlaps(parts[r], span(M, n_each, ld_part, 4), Y,
                                      span(M, n_each, ldy, ye)))
                return TSL_ERR_INVALID_ARG;
        }
        return from_hip(launch_combine_sum(n_parts, reinterpret_cast<const float *const *>(parts),
                                           M, n_each, ld_part, ydtype, Y, ldy, s));
    }
    if (mode == TSL_COMBINE_CONCAT) {
        if (pdtype != ydtype)
            return TSL_ERR_UNSUPPORTED;
        if (ldy < n_each * n_parts)
            return TSL_ERR_INVALID_ARG;
        const uintptr_t ea = pdtype == TSL_F32 ? 4 : 2;
        for (int r = 0; r < n_parts; ++r)
            if (!aligned(parts[r], ea))
                return TSL_ERR_MISALIGNED;
        if (!aligned(Y, ea))
            return TSL_ERR_MISALIGNED;
        if (M == 0 || n_each == 0)
            return TSL_OK;
        for (int r = 0; r < n_parts; ++r)
            if (overlaps(parts[r], span(M, n_each, ld_part, ea), Y,
                         span(M, n_each * n_parts, ldy, ea)))
                return TSL_ERR_INVALID_ARG;
        return from_hip(launch_combine_concat(n_parts, parts, ea, M, n_each, ld_part, Y, ldy, s));
    }
    return TSL_ERR_INVALID_ARG;
}

extern "C" tsl_status combine_to_ranks(tsl_collective op, int32_t n, const void *const *parts,
                                       tsl_dtype pdtype, int64_t M, int64_t n_each,
                                       int64_t ld_part, tsl_dtype odtype, void *const *outs,
                                       int64_t ldo, void *stream) {
    if (!parts || !outs || n < 1 || n > kMaxParts || M < 0 || n_each < 0 || ld_part < n_each)
        return TSL_ERR_INVALID_ARG;
    if (op != TSL_ALL_REDUCE && op != TSL_REDUCE_SCATTER && op != TSL_ALL_GATHER)
        return TSL_ERR_INVALID_ARG;
    if ((pdtype != TSL_F32 && pdtype != TSL_BF16) || (odtype != TSL_F32 && odtype != TSL_BF16))
        return TSL_ERR_INVALID_ARG;
    for (int r = 0; r < n; ++r)
        if (!parts[r] || !outs[r])
            return TSL_ERR_INVALID_ARG;
    const bool gather = op == TSL_ALL_GATHER;
    if (gather ? pdtype != odtype : pdtype != TSL_F32)
        return TSL_ERR_UNSUPPORTED;
    const int64_t width = gather ? n_each * n : n_each; // columns of each output
    if (ldo < width)
        return TSL_ERR_INVALID_ARG;
    const size_t pe = pdtype == TSL_F32 ? 4 : 2, oe = odtype == TSL_F32 ? 4 : 2;
    for (int r = 0; r < n; ++r)
        if (!aligned(parts[r], pe) || !aligned(outs[r], oe))
            return TSL_ERR_MISALIGNED;
    if (M == 0 || n_each == 0)
        return TSL_OK;
    // rows of rank r's output
    auto rows = [&](int r) {
        return op == TSL_REDUCE_SCATTER ? ((int64_t)(r + 1) * M) / n - ((int64_t)r * M) / n : M;
    };
    for (int r = 0; r < n; ++r) {
        if (rows(r) == 0)
            continue;
        for (int q = 0; q < n; ++q) {
            if (matrices_overlap(outs[r], rows(r), width, ldo, oe, parts[q], M, n_each, ld_part,
                                 pe))
                return TSL_ERR_INVALID_ARG;
            if (q > r && rows(q) > 0 &&
                matrices_overlap(outs[r], rows(r), width, ldo, oe, outs[q], rows(q), width, ldo,
                                 oe))
                return TSL_ERR_INVALID_ARG;
        }
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (gather)
        return from_hip(launch_gather_to_ranks(n, parts, pe, M, n_each, ld_part, outs, ldo, s));
    return from_hip(launch_reduce_to_ranks(n, reinterpret_cast<const float *const *>(parts), M,
                                           n_each, ld_part, op == TSL_REDUCE_SCATTER, odtype, outs,
                                           ldo, s));
}

extern "C" tsl_status embed_lookup(const tsl_shard *shard, tsl_dtype tdtype, const void *table,
                                   int64_t ld_table, const int32_t *tokens, int64_t M,
                                   tsl_dtype ydtype, void *Y, int64_t ldy, void *stream) {
    tsl_status st = check_shard(shard);
    if (st != TSL_OK)
        return st;
    if (!table || !tokens || !Y || M < 0)
        return TSL_ERR_INVALID_ARG;
    if ((tdtype != TSL_F32 && tdtype != TSL_BF16) || (ydtype != TSL_F32 && ydtype != TSL_BF16))
        return TSL_ERR_INVALID_ARG;
    const int64_t n_len = shard->n_len;
    if (ld_table < n_len || ldy < n_len)
        return TSL_ERR_INVALID_ARG;
    const size_t te = tdtype == TSL_F32 ? 4 : 2, ye = ydtype == TSL_F32 ? 4 : 2;
    if (!aligned(table, te) || !aligned(tokens, 4) || !aligned(Y, ye))
        return TSL_ERR_MISALIGNED;
    if (M == 0)
        return TSL_OK;
    if (matrices_overlap(Y, M, n_len, ldy, ye, table, shard->k_len, n_len, ld_table, te) ||
        overlaps(Y, span(M, n_len, ldy, ye), tokens, (size_t)M * 4))
        return TSL_ERR_INVALID_ARG;
    return from_hip(launch_embed_lookup(tdtype, table, ld_table, tokens, M, shard->k_off,
                                        shard->k_len, n_len, ydtype, Y, ldy,
                                        static_cast<hipStream_t>(stream)));
}

extern "C" tsl_status moe_gather(const void *src, int64_t ld_src, int64_t n_src, tsl_dtype dtype,
                                 const int32_t *idx, int64_t n, int64_t width, void *out,
                                 int64_t ldo, void *stream) {
    if (!src || !idx || !out || n_src < 1 || n < 0 || width < 1 || ld_src < width || ldo < width)
        return TSL_ERR_INVALID_ARG;
    if (dtype != TSL_F32 && dtype != TSL_BF16)
        return TSL_ERR_INVALID_ARG;
    const size_t e = dtype == TSL_F32 ? 4 : 2;
    if (!aligned(src, e) || !aligned(out, e) || !aligned(idx, 4))
        return TSL_ERR_MISALIGNED;
    if (n == 0)
        return TSL_OK;
    if (matrices_overlap(out, n, width, ldo, e, src, n_src, width, ld_src, e) ||
        overlaps(out, span(n, width, ldo, e), idx, (size_t)n * 4))
        return TSL_ERR_INVALID_ARG;
    // a row gather is a lookup into a table of n_src rows that one rank owns whole
    return from_hip(launch_embed_lookup(dtype, src, ld_src, idx, n, 0, n_src, width, dtype, out,
                                        ldo, static_cast<hipStream_t>(stream)));
}

extern "C" tsl_status moe_combine(const float *P, int64_t ldp, int64_t n_rows,
                                  const int32_t *slot_row, const float *weights, int64_t T,
                                  int32_t k, int64_t n, tsl_dtype ydtype, void *Y, int64_t ldy,
                                  void *stream) {
    if (!slot_row || !weights || !Y || T < 0 || k < 1 || n < 0 || n_rows < 0 || ldy < n)
        return TSL_ERR_INVALID_ARG;
    if (n_rows > 0 && (!P || ldp < n))
        return TSL_ERR_INVALID_ARG;
    if (ydtype != TSL_F32 && ydtype != TSL_BF16)
        return TSL_ERR_INVALID_ARG;
    const size_t ye = ydtype == TSL_F32 ? 4 : 2;
    if ((P && !aligned(P, 4)) || !aligned(slot_row, 4) || !aligned(weights, 4) || !aligned(Y, ye))
        return TSL_ERR_MISALIGNED;
    if (T == 0 || n == 0)
        return TSL_OK;
    const size_t ybytes = span(T, n, ldy, ye);
    if ((n_rows > 0 && matrices_overlap(Y, T, n, ldy, ye, P, n_rows, n, ldp, 4)) ||
        overlaps(Y, ybytes, slot_row, (size_t)T * k * 4) ||
        overlaps(Y, ybytes, weights, (size_t)T * k * 4))
        return TSL_ERR_INVALID_ARG;
    return from_hip(launch_moe_combine(P, ldp, n_rows, slot_row, weights, T, k, n, ydtype, Y, ldy,
                                       static_cast<hipStream_t>(stream)));
}

extern "C" const char *tsl_last_hip_error_string(void) { return hipGetErrorString(g_last_hip); }

extern "C" const char *tsl_status_string(tsl_status status) {
    switch (status) {
    case TSL_OK: return "ok";
    case TSL_ERR_INVALID_ARG: return "invalid argument";
    case TSL_ERR_NOT_DIVISIBLE: return "dimension does not split evenly across ranks";
    case TSL_ERR_TP_NOT_POW2: return "tp_size is not a power of two";
    case TSL_ERR_GROUP_ALIGN: return "4-bit group straddles a shard edge";
    case TSL_ERR_BUFFER_TOO_SMALL: return "buffer too small";
    case TSL_ERR_UNSUPPORTED: return "unsupported dtype combination or size";
    case TSL_ERR_MISALIGNED: return "misaligned pointer or leading dimension";
    case TSL_ERR_HIP: return "HIP runtime error";
    }
    return "unknown status";
}
