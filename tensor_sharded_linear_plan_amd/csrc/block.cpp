// The C ABI of tsl_block.h.  Checks run before anything is enqueued; no exception leaves an
// entry point.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstddef>
#include <vector>

#include "group.hpp"
#include "internal.hpp"
#include "tsl_block.h"

using namespace tsl;

namespace {

bool dense_type(int d) { return d == TSL_F32 || d == TSL_BF16; }
size_t elem(int d) { return d == TSL_F32 ? 4 : (d == TSL_E4M3 ? 1 : 2); }

// Limits that keep every row offset and span in 64 bits.
constexpr int64_t kMaxRows = int64_t(1) << 22;
constexpr int64_t kMaxLd = int64_t(1) << 31;

// One row-strided operand of an entry point, as the checks see it.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    size_t e;
};

// Whether two operands share a byte.
bool clash(const Mat &a, const Mat &b) {
    return a.p && b.p && a.rows > 0 && b.rows > 0 &&
           matrices_overlap(a.p, a.rows, a.cols, a.ld, a.e, b.p, b.rows, b.cols, b.ld, b.e);
}

// No output shares a byte with an input or another output; an in-place pair
// is left out by the caller.
bool any_clash(const std::vector<Mat> &outs, const std::vector<Mat> &ins) {
    for (size_t i = 0; i < outs.size(); ++i) {
        for (const Mat &b : ins)
            if (clash(outs[i], b))
                return true;
        for (size_t j = i + 1; j < outs.size(); ++j)
            if (clash(outs[i], outs[j]))
                return true;
    }
    return false;
}

// Host memory for the call's tables may run out; nothing else throws.
template <class F> tsl_status guarded(F f) {
    try {
        return f();
    } catch (...) {
        return TSL_ERR_UNSUPPORTED;
    }
}

// Rows that take the wide loads and stores: 16-byte aligned bases, row
// strides of whole runs of 8 columns (8-bit outputs: 8 bytes).
bool wide(const void *p, int64_t ld, size_t e) {
    return !p || (aligned(p, e == 1 ? 8 : 16) && ld % 8 == 0);
}

} // namespace

extern "C" tsl_status add_rms_norm(int32_t n_parts, const void *const *parts, tsl_dtype pdtype,
                                   int64_t ld_part, int64_t M, int64_t n, const void *residual,
                                   tsl_dtype rdtype, int64_t ldr, void *sum_out, int64_t ld_sum,
                                   const void *weight, tsl_dtype wdtype, float eps,
                                   tsl_dtype ydtype, void *Y, int64_t ldy, float *scales,
                                   int32_t group, float *rstd, void *stream) {
    if (!parts || !Y || n_parts < 1 || n_parts > kMaxParts || M < 0 || n < 1 || !(eps >= 0.f))
        return TSL_ERR_INVALID_ARG;
    for (int r = 0; r < n_parts; ++r)
        if (!parts[r])
            return TSL_ERR_INVALID_ARG;
    if (!dense_type(pdtype) || !dense_type(rdtype) || (weight && !dense_type(wdtype)) ||
        (!dense_type(ydtype) && ydtype != TSL_E4M3))
        return TSL_ERR_INVALID_ARG;
    if (ld_part < n || ldy < n || (residual && ldr < n) || (sum_out && ld_sum < n))
        return TSL_ERR_INVALID_ARG;
    if (ydtype == TSL_E4M3 ? !scales || (group != 0 && group != 32 && group != 64 && group != 128)
                           : scales || group)
        return TSL_ERR_INVALID_ARG;
    if (n > kNormMaxWidth || M >= kMaxRows || ld_part >= kMaxLd || ldy >= kMaxLd ||
        (residual && ldr >= kMaxLd) || (sum_out && ld_sum >= kMaxLd))
        return TSL_ERR_UNSUPPORTED;
    const size_t pe = elem(pdtype), re = elem(rdtype), ye = elem(ydtype), we = elem(wdtype);
    for (int r = 0; r < n_parts; ++r)
        if (!aligned(parts[r], pe))
            return TSL_ERR_MISALIGNED;
    if (!aligned(residual, re) || !aligned(sum_out, re) || (weight && !aligned(weight, we)) ||
        !aligned(Y, ye) || !aligned(scales, 4) || !aligned(rstd, 4))
        return TSL_ERR_MISALIGNED;
    if (M == 0)
        return TSL_OK;
    return guarded([&] {
        const bool in_place = sum_out && sum_out == residual && ld_sum == ldr;
        const int64_t groups = group ? (n + group - 1) / group : 1;
        std::vector<Mat> ins, outs;
        for (int r = 0; r < n_parts; ++r)
            ins.push_back(Mat{parts[r], M, n, ld_part, pe});
        if (!in_place)
            ins.push_back(Mat{residual, M, n, ldr, re});
        ins.push_back(Mat{weight, 1, n, n, we});
        outs.push_back(Mat{sum_out, M, n, ld_sum, re});
        outs.push_back(Mat{Y, M, n, ldy, ye});
        outs.push_back(Mat{scales, 1, M * groups, M * groups, 4});
        outs.push_back(Mat{rstd, 1, M, M, 4});
        if (any_clash(outs, ins))
            return TSL_ERR_INVALID_ARG;
        NormArgs a{};
        bool vec = wide(residual, ldr, re) && wide(sum_out, ld_sum, re) && wide(Y, ldy, ye) &&
                   wide(weight, 0, we);
        for (int r = 0; r < n_parts; ++r) {
            a.parts[r] = parts[r];
            vec = vec && wide(parts[r], ld_part, pe);
        }
        a.residual = residual;
        a.sum_out = sum_out;
        a.weight = weight;
        a.Y = Y;
        a.scales = scales;
        a.rstd = rstd;
        a.M = M;
        a.n = n;
        a.ld_part = ld_part;
        a.ldr = ldr;
        a.ld_sum = ld_sum;
        a.ldy = ldy;
        a.eps = eps;
        a.n_parts = n_parts;
        a.p_bf16 = pdtype == TSL_BF16;
        a.r_bf16 = rdtype == TSL_BF16;
        a.w_bf16 = wdtype == TSL_BF16;
        a.y_type = ydtype;
        a.group = group;
        return from_hip(launch_norm(a, vec, static_cast<hipStream_t>(stream)));
    });
}

namespace {

size_t norm_grad_bytes(int64_t M, int64_t n) {
    return (size_t)norm_grad_partials(M, n) * (size_t)((n + 7) / 8 * 8) * 4;
}

} // namespace

extern "C" tsl_status add_rms_norm_grad_workspace_size(int64_t M, int64_t n, size_t *bytes) {
    if (!bytes || M < 0 || n < 1)
        return TSL_ERR_INVALID_ARG;
    if (n > kNormMaxWidth || M >= kMaxRows)
        return TSL_ERR_UNSUPPORTED;
    *bytes = norm_grad_bytes(M, n);
    return TSL_OK;
}

extern "C" tsl_status add_rms_norm_grad(int64_t M, int64_t n, const void *dY, tsl_dtype dydtype,
                                        int64_t lddy, const void *X, tsl_dtype xdtype, int64_t ldx,
                                        const void *weight, tsl_dtype wdtype, float eps,
                                        const float *rstd, const void *dres, int64_t ld_dres,
                                        void *dX, tsl_dtype dxdtype, int64_t lddx, float *dW,
                                        int accumulate_dw, void *workspace, size_t ws_bytes,
                                        void *stream) {
    if (!dY || !X || (!dX && !dW) || M < 0 || n < 1 || (!rstd && !(eps >= 0.f)))
        return TSL_ERR_INVALID_ARG;
    if (!dense_type(dydtype) || !dense_type(xdtype) || (weight && !dense_type(wdtype)) ||
        ((dX || dres) && !dense_type(dxdtype)) || (accumulate_dw != 0 && accumulate_dw != 1))
        return TSL_ERR_INVALID_ARG;
    if (lddy < n || ldx < n || (dX && lddx < n) || (dres && (!dX || ld_dres < n)))
        return TSL_ERR_INVALID_ARG;
    if (n > kNormMaxWidth || M >= kMaxRows || lddy >= kMaxLd || ldx >= kMaxLd ||
        (dX && lddx >= kMaxLd) || (dres && ld_dres >= kMaxLd))
        return TSL_ERR_UNSUPPORTED;
    const size_t ye = elem(dydtype), xe = elem(xdtype), we = elem(wdtype), de = elem(dxdtype);
    if (!aligned(dY, ye) || !aligned(X, xe) || (weight && !aligned(weight, we)) ||
        !aligned(rstd, 4) || (dX && !aligned(dX, de)) || (dres && !aligned(dres, de)) ||
        !aligned(dW, 4))
        return TSL_ERR_MISALIGNED;
    const size_t need = dW ? norm_grad_bytes(M, n) : 0;
    if (need > 0) {
        if (!workspace || ws_bytes < need)
            return TSL_ERR_BUFFER_TOO_SMALL;
        if (!aligned(workspace, 256))
            return TSL_ERR_MISALIGNED;
    }
    if (M == 0 && !dW)
        return TSL_OK;
    return guarded([&] {
        std::vector<Mat> ins = {{dY, M, n, lddy, ye},
                                {X, M, n, ldx, xe},
                                {weight, 1, n, n, we},
                                {rstd, 1, M, M, 4}};
        if (!(dres == dX && ld_dres == lddx))
            ins.push_back(Mat{dres, M, n, ld_dres, de});
        if (any_clash({{dX, M, n, lddx, de},
                       {dW, 1, n, n, 4},
                       {need ? workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1}},
                      ins))
            return TSL_ERR_INVALID_ARG;
        NormGradArgs a{};
        a.dY = dY;
        a.X = X;
        a.weight = weight;
        a.dres = dres;
        a.rstd = rstd;
        a.dX = dX;
        a.part = dW ? static_cast<float *>(workspace) : nullptr;
        a.M = M;
        a.n = n;
        a.lddy = lddy;
        a.ldx = ldx;
        a.ld_dres = ld_dres;
        a.lddx = lddx;
        a.eps = eps;
        a.dy_bf16 = dydtype == TSL_BF16;
        a.x_bf16 = xdtype == TSL_BF16;
        a.w_bf16 = wdtype == TSL_BF16;
        a.dx_bf16 = dxdtype == TSL_BF16;
        const bool vec = wide(dY, lddy, ye) && wide(X, ldx, xe) && wide(weight, 0, we) &&
                         wide(dres, ld_dres, de) && wide(dX, lddx, de);
        return from_hip(launch_norm_grad(a, vec, dW, accumulate_dw,
                                         static_cast<hipStream_t>(stream)));
    });
}

// the tables' layouts are part of the ABI
static_assert(sizeof(tsl_epilogue) == 56 && offsetof(tsl_epilogue, act) == 40, "tsl_epilogue layout");
static_assert(sizeof(tsl_gated_item) == 120 && offsetof(tsl_gated_item, hdtype) == 112,
              "tsl_gated_item layout");

namespace {

// The items of a size query (shards, set links, rows, accumulation, whether
// indexed).
tsl_status sized_items(int32_t n_items, const tsl_linear_item *items, tsl_dtype wdtype, int64_t M,
                       std::vector<LinearItem> *out) {
    out->resize(n_items);
    int32_t first = 0;
    for (int32_t i = 0; i < n_items; ++i) {
        LinearItem &L = (*out)[i];
        if (!items[i].shard || (items[i].sum_next != 0 && items[i].sum_next != 1) ||
            items[i].rows < 0 || items[i].rows > M)
            return TSL_ERR_INVALID_ARG;
        tsl_status st = geometry(*items[i].shard, wdtype, &L.g);
        if (st != TSL_OK)
            return st;
        L.M = items[i].rows ? items[i].rows : M;
        L.ridx = items[i].row_index;
        L.x_rows = 1;
        L.accumulate = items[i].accumulate; // of a set's first item
        L.set_pos = i - first;
        if (L.set_pos > 0)
            L.accumulate = 0;
        if (!items[i].sum_next || i == n_items - 1) {
            (*out)[first].set_len = i - first + 1;
            for (int32_t r = first + 1; r <= i; ++r)
                (*out)[r].set_len = 0;
            first = i + 1;
        }
    }
    return TSL_OK;
}

bool valid_act(int a) { return a >= TSL_ACT_NONE && a <= TSL_ACT_GELU_TANH; }

// One epilogue's fields for a product of n columns; its checks.
tsl_status check_epilogue(const tsl_epilogue &e, int64_t n, Epilogue *out) {
    if (!valid_act(e.act) || (e.bias && !dense_type(e.bias_dtype)) ||
        (e.residual && (!dense_type(e.res_dtype) || e.ld_res < n)) ||
        (e.pre && (!dense_type(e.pre_dtype) || e.ld_pre < n)))
        return TSL_ERR_INVALID_ARG;
    if ((e.residual && e.ld_res >= kMaxLd) || (e.pre && e.ld_pre >= kMaxLd))
        return TSL_ERR_UNSUPPORTED;
    if ((e.bias && !aligned(e.bias, elem(e.bias_dtype))) ||
        (e.residual && !aligned(e.residual, elem(e.res_dtype))) ||
        (e.pre && !aligned(e.pre, elem(e.pre_dtype))))
        return TSL_ERR_MISALIGNED;
    out->bias = e.bias;
    out->res = e.residual;
    out->pre = e.pre;
    out->ldr = e.ld_res;
    out->ldp = e.ld_pre;
    out->act = e.act;
    out->flags = (e.bias && e.bias_dtype == TSL_BF16 ? kEpBiasBf16 : 0) |
                 (e.residual && e.res_dtype == TSL_BF16 ? kEpResBf16 : 0) |
                 (e.pre && e.pre_dtype == TSL_BF16 ? kEpPreBf16 : 0);
    return TSL_OK;
}

// The operands of validated items that the group's own checks do not see
// (kept pre-activations, biases, residuals) against every output and input.
bool epilogue_clash(const std::vector<LinearItem> &v, size_t xe) {
    std::vector<Mat> kept, read; // outputs and inputs of the epilogues
    std::vector<const LinearItem *> reader; // whose input read[i] is
    for (const LinearItem &L : v) {
        if (!L.ep)
            continue;
        const Epilogue &e = *L.ep;
        const size_t pe = e.flags & kEpPreBf16 ? 2 : 4, re = e.flags & kEpResBf16 ? 2 : 4;
        if (e.pre)
            kept.push_back(Mat{e.pre, L.M, L.g.Ns, e.ldp, pe});
        if (e.pre2)
            kept.push_back(Mat{e.pre2, L.M, L.g.Ns, e.ldp, pe});
        if (e.bias)
            read.push_back(Mat{e.bias, 1, L.g.Ns, L.g.Ns, (size_t)(e.flags & kEpBiasBf16 ? 2 : 4)});
        if (e.res)
            read.push_back(Mat{e.res, L.M, L.g.Ns, e.ldr, re});
        reader.resize(read.size(), &L);
    }
    if (kept.empty() && read.empty())
        return false;
    if (any_clash(kept, read))
        return true;
    for (const LinearItem &L : v) {
        const Mat x{L.X, L.ridx ? L.x_rows : L.M, L.g.Ks, L.ldx, xe};
        const Mat ix{L.ridx, 1, L.M, L.M, 4};
        const Mat y{L.Y, L.M, L.g.Ns, L.ldy, (size_t)(L.ydtype == TSL_F32 ? 4 : 2)};
        for (const Mat &k : kept)
            if (clash(k, x) || clash(k, ix) || clash(k, y))
                return true;
        for (size_t i = 0; i < read.size(); ++i) {
            const Mat &r = read[i];
            // the residual of the item itself, updated in place
            const bool own = reader[i] == &L && r.p == L.ep->res && r.p == L.Y && r.ld == y.ld &&
                             r.e == y.e && r.rows == y.rows && r.cols == y.cols;
            if (!own && clash(y, r))
                return true;
        }
    }
    return false;
}

bool any_epilogue(int32_t n, const tsl_epilogue *const *e) {
    for (int32_t i = 0; i < n; ++i)
        if (e[i])
            return true;
    return false;
}

} // namespace

extern "C" tsl_status shard_linear_group_epilogue_workspace_size(
    int32_t n_items, const tsl_linear_item *items, const tsl_epilogue *const *epilogues,
    tsl_dtype wdtype, int64_t M, size_t *bytes) {
    if (!items || !epilogues || !bytes || n_items < 1 || n_items > kMaxItems || M < 0)
        return TSL_ERR_INVALID_ARG;
    return guarded([&] {
        std::vector<LinearItem> v;
        tsl_status st = sized_items(n_items, items, wdtype, M, &v);
        if (st != TSL_OK)
            return st;
        Epilogue none;
        for (int32_t i = 0; i < n_items; ++i)
            if (epilogues[i])
                v[i].ep = &none;
        *bytes = group_workspace(v, wdtype, M);
        bool accumulates = false;
        for (LinearItem &L : v) {
            accumulates = accumulates || L.accumulate;
            L.accumulate = 0;
        }
        if (accumulates) // the same items storing their products fit too
            *bytes = std::max(*bytes, group_workspace(v, wdtype, M));
        return TSL_OK;
    });
}

extern "C" tsl_status shard_linear_group_epilogue(int32_t n_items, const tsl_linear_item *items,
                                                  const tsl_epilogue *const *epilogues,
                                                  tsl_dtype wdtype, tsl_dtype xdtype, int64_t M,
                                                  void *workspace, size_t ws_bytes, void *stream) {
    if (!epilogues)
        return TSL_ERR_INVALID_ARG;
    return guarded([&] {
        std::vector<LinearItem> v;
        tsl_status st = gather(n_items, items, wdtype, xdtype, M, &v);
        if (st != TSL_OK)
            return st;
        std::vector<Epilogue> eps(n_items);
        for (int32_t i = 0; i < n_items; ++i) {
            if (!epilogues[i])
                continue;
            if (v[i].set_pos > 0 || v[i].accumulate)
                return TSL_ERR_INVALID_ARG;
            st = check_epilogue(*epilogues[i], v[i].g.Ns, &eps[i]);
            if (st != TSL_OK)
                return st;
            v[i].ep = &eps[i];
        }
        if (M > 0 && any_epilogue(n_items, epilogues) && epilogue_clash(v, xdtype == TSL_F32 ? 4 : 2))
            return TSL_ERR_INVALID_ARG;
        return run_group(v, wdtype, M, workspace, ws_bytes, stream);
    });
}

namespace {

// A gated item as the pair of products the group code sees.
void gated_pair(const tsl_gated_item &g, tsl_linear_item *two) {
    for (int q = 0; q < 2; ++q) {
        tsl_linear_item &L = two[q];
        L = tsl_linear_item{};
        L.shard = q ? g.up : g.gate;
        L.packed = q ? g.packed_up : g.packed_gate;
        L.packed_bytes = g.packed_bytes;
        L.X = g.X;
        L.ldx = g.ldx;
        L.Y = g.H;
        L.ldy = g.ldh;
        L.ydtype = g.hdtype;
        L.sum_next = q == 0;
        L.rows = g.rows;
        L.row_index = g.row_index;
        L.x_rows = g.x_rows;
    }
}

constexpr int32_t kMaxGated = kMaxItems / 2;

// Pairs of bf16 and 4-bit weights run as one dual product each: the second
// of a checked pair leaves the list (its packed weight is ep->up).
void merge_pairs(std::vector<LinearItem> *v, tsl_dtype wdtype) {
    if (wdtype == TSL_F32)
        return;
    for (size_t i = 0; 2 * i < v->size(); ++i) {
        (*v)[i] = (*v)[2 * i];
        (*v)[i].set_len = 1;
    }
    v->resize(v->size() / 2);
}

} // namespace

extern "C" tsl_status shard_gated_group_workspace_size(int32_t n_items, const tsl_gated_item *items,
                                                       tsl_dtype wdtype, int64_t M, size_t *bytes) {
    if (!items || !bytes || n_items < 1 || n_items > kMaxGated || M < 0)
        return TSL_ERR_INVALID_ARG;
    return guarded([&] {
        std::vector<tsl_linear_item> pairs(2 * (size_t)n_items);
        for (int32_t i = 0; i < n_items; ++i)
            gated_pair(items[i], &pairs[2 * i]);
        std::vector<LinearItem> v;
        tsl_status st = sized_items(2 * n_items, pairs.data(), wdtype, M, &v);
        if (st != TSL_OK)
            return st;
        Epilogue gate;
        gate.flags = kEpGated;
        gate.up = wdtype == TSL_F32 ? nullptr : &gate;
        for (int32_t i = 0; i < n_items; ++i) {
            if (v[2 * i].g.Ns != v[2 * i + 1].g.Ns || v[2 * i].g.Ks != v[2 * i + 1].g.Ks)
                return TSL_ERR_INVALID_ARG;
            v[2 * i].ep = &gate;
            // the pair reads one X (any address that no other pair has)
            v[2 * i].X = v[2 * i + 1].X = &pairs[2 * i];
        }
        merge_pairs(&v, wdtype);
        *bytes = group_workspace(v, wdtype, M);
        return TSL_OK;
    });
}

extern "C" tsl_status shard_gated_group(int32_t n_items, const tsl_gated_item *items, tsl_act act,
                                        tsl_dtype wdtype, tsl_dtype xdtype, int64_t M,
                                        void *workspace, size_t ws_bytes, void *stream) {
    if (!items || n_items < 1 || n_items > kMaxGated || !valid_act(act))
        return TSL_ERR_INVALID_ARG;
    return guarded([&] {
        std::vector<tsl_linear_item> pairs(2 * (size_t)n_items);
        for (int32_t i = 0; i < n_items; ++i)
            gated_pair(items[i], &pairs[2 * i]);
        std::vector<LinearItem> v;
        tsl_status st = gather(2 * n_items, pairs.data(), wdtype, xdtype, M, &v);
        if (st != TSL_OK)
            return st;
        std::vector<Epilogue> eps(n_items);
        bool kept = false;
        for (int32_t i = 0; i < n_items; ++i) {
            const tsl_gated_item &g = items[i];
            const LinearItem &L = v[2 * i];
            if (L.g.Ks != v[2 * i + 1].g.Ks || (g.G == nullptr) != (g.U == nullptr) ||
                (g.G && g.ld_gu < L.g.Ns))
                return TSL_ERR_INVALID_ARG;
            if (g.G && g.ld_gu >= kMaxLd)
                return TSL_ERR_UNSUPPORTED;
            if (!aligned(g.G, elem(g.hdtype)) || !aligned(g.U, elem(g.hdtype)))
                return TSL_ERR_MISALIGNED;
            Epilogue &e = eps[i];
            e.pre = g.G;
            e.pre2 = g.U;
            e.ldp = g.ld_gu;
            e.act = act;
            e.flags = kEpGated | (g.hdtype == TSL_BF16 ? kEpPreBf16 : 0);
            e.up = wdtype == TSL_F32 ? nullptr : g.packed_up;
            v[2 * i].ep = &e;
            kept = kept || g.G;
        }
        if (M > 0 && kept && epilogue_clash(v, xdtype == TSL_F32 ? 4 : 2))
            return TSL_ERR_INVALID_ARG;
        merge_pairs(&v, wdtype);
        return run_group(v, wdtype, M, workspace, ws_bytes, stream);
    });
}

extern "C" tsl_status transpose_shard(const tsl_shard *shard, tsl_shard *out) {
    if (!out)
        return TSL_ERR_INVALID_ARG;
    tsl_status st = check_shard(shard);
    if (st != TSL_OK)
        return st;
    tsl_shard t = *shard;
    t.K = shard->N;
    t.N = shard->K;
    t.k_off = shard->n_off;
    t.k_len = shard->n_len;
    t.n_off = shard->k_off;
    t.n_len = shard->k_len;
    if (shard->strategy == TSL_COLUMN) {
        t.strategy = TSL_ROW;
        t.combine = TSL_COMBINE_SUM;
    } else if (shard->strategy == TSL_ROW) {
        t.strategy = TSL_COLUMN;
        t.combine = TSL_COMBINE_CONCAT;
    }
    *out = t;
    return TSL_OK;
}

namespace {

// The backward pass of one weight (linear: n_w 1) or of a gated pair (2).
struct GradCall {
    const tsl_shard *shard[2] = {};
    int n_w = 1;
    const void *packed_t[2] = {};
    size_t packed_t_bytes = 0;
    tsl_dtype wdtype = TSL_BF16;
    int64_t M = 0;
    const void *X = nullptr;
    int64_t ldx = 0;
    int act = 0;
    // linear: a = dY, b = Z (null without an activation); gated: dH, G, U
    const void *a = nullptr, *b = nullptr, *c = nullptr;
    int64_t lda = 0, ldb = 0;
    int dxdtype = 0, dwdtype = 0;
    void *dX = nullptr;
    int64_t lddx = 0;
    void *dW[2] = {};
    int64_t sk = 0, sn = 0;
    int accumulate = 0;
    float *db = nullptr;
};

// Workspace parts of a call and the products it runs.  Everything but the
// addresses follows from the shapes and from which outputs are wanted.
struct GradPlan {
    size_t row[2] = {}, row_lo[2] = {}, tr[2] = {}, xt = 0, part = 0, products = 0, total = 0;
    int64_t K = 0, N = 0, Mp = 0, Np = 0;
    int64_t Mt = 0; // rows of the transposed copies: Mp, or 2 Mp with split
    bool need_row = false, need_tr = false, split = false;
};

// bf16 products read dZ rounded to bf16, which costs a gradient as much as
// its own rounding to bf16 does (0.0017 of it in norm).  Up to this many
// entries of dZ what the rounding left goes along as further operands: the
// products are bound by latency and the weights' bytes there, not by their
// operations.  Measured, gated with silu, error of binary32 gradients: 3 x
// 1500 -> 700 3e-6 (one rounding 0.0017), 24 x 1024 -> 1024 2e-6; without,
// 250 x 2048 -> 2048, 0.0016.
constexpr int64_t kSplitEntries = int64_t(1) << 16;

bool nk_order(const GradCall &c) { return c.sk == 1 && c.sn != 1; }

// dX and dW share a launch where both take the same kernels.
bool one_group(const GradCall &c, const GradPlan &p) {
    return c.dX && c.dW[0] &&
           use_skinny(c.wdtype, c.M) == use_skinny(c.wdtype, nk_order(c) ? p.N : p.K);
}

// dX of a few rows alone in its call takes the one-launch form (decode.hip),
// which products with an epilogue take -- here one that changes nothing.
const Epilogue kNoEpilogue;
bool few_rows(const GradCall &c, const GradPlan &p) {
    return c.M <= kDecodeRows && !one_group(c, p);
}

// The products of a call: dX (a set of n_w), then dW of each weight, with
// the operands of `p` at ws (null: sizing).
void grad_items(const GradCall &c, const GradPlan &p, const PackGeom &gt, char *ws,
                std::vector<LinearItem> *dx, std::vector<LinearItem> *dw) {
    auto at = [&](size_t off) { return ws ? ws + off : nullptr; };
    const int len = c.n_w * (p.split ? 2 : 1);
    if (c.dX)
        for (int s = 0; s < len; ++s) {
            const int q = p.split ? s / 2 : s;
            const size_t row = p.split && s % 2 ? p.row_lo[q] : p.row[q];
            LinearItem L;
            L.g = gt;
            L.M = c.M;
            L.packed = c.packed_t[q];
            L.X = p.need_row ? at(row) : c.a;
            L.ldx = p.need_row ? p.Np : c.lda;
            // the copy's columns are zero up to Np, as the packed rows are
            if (p.need_row)
                L.g.Ks = p.Np;
            L.Y = s == 0 ? c.dX : nullptr;
            L.ldy = s == 0 ? c.lddx : 0;
            L.ydtype = (tsl_dtype)c.dxdtype;
            L.set_len = s == 0 ? len : 0;
            L.set_pos = s;
            if (s == 0 && few_rows(c, p))
                L.ep = &kNoEpilogue;
            dx->push_back(L);
        }
    if (!c.dW[0])
        return;
    for (int q = 0; q < c.n_w; ++q) {
        LinearItem L;
        const bool nk = nk_order(c);
        const int64_t cols = nk ? p.K : p.N;
        L.g.Ks = L.g.Kpad = p.Mt;
        L.g.Ns = cols;
        L.g.Nt = (cols + 15) / 16;
        L.g.KT = p.Mt / (c.wdtype == TSL_F32 ? 16 : 32);
        L.M = nk ? p.N : p.K;
        L.X = at(nk ? p.tr[q] : p.xt);
        L.packed = at(nk ? p.xt : p.tr[q]);
        L.ldx = p.Mt;
        L.Y = c.dW[q];
        L.ldy = nk ? c.sn : c.sk;
        L.ydtype = (tsl_dtype)c.dwdtype;
        L.accumulate = c.accumulate;
        dw->push_back(L);
    }
}

// Fills the plan; gt receives the geometry of the packed transposed weight.
tsl_status plan_grad(const GradCall &c, GradPlan *p, PackGeom *gt) {
    for (int q = 0; q < c.n_w; ++q) {
        tsl_shard t;
        tsl_status st = transpose_shard(c.shard[q], &t);
        if (st == TSL_OK)
            st = geometry(t, c.wdtype, gt);
        if (st != TSL_OK)
            return st;
        if (q > 0 && (gt->Ns != p->K || gt->Ks != p->N))
            return TSL_ERR_INVALID_ARG;
        p->K = gt->Ns;
        p->N = gt->Ks;
    }
    if (c.M >= kPrefillMaxStride - 64 || p->K >= kPrefillMaxStride - 64 ||
        p->N >= kPrefillMaxStride - 64)
        return TSL_ERR_UNSUPPORTED;
    // every launch's workgroups stay countable (kMaxBlocks): tiles of at least
    // 64 x 64 (binary32: 16 x 64) elements
    const int64_t most = int64_t(1) << (c.wdtype == TSL_F32 ? 32 : 34);
    if (p->K * p->N > most || c.M * p->K > most || c.M * p->N > most)
        return TSL_ERR_UNSUPPORTED;
    p->Mp = (c.M + 63) / 64 * 64;
    p->Np = (p->N + 63) / 64 * 64;
    const size_t e = c.wdtype == TSL_F32 ? 4 : 2;
    // without an activation dY itself feeds dX
    p->need_row = c.dX && (c.n_w > 1 || c.act != TSL_ACT_NONE);
    p->need_tr = c.dW[0] != nullptr;
    p->split = c.wdtype == TSL_BF16 && c.M * p->N <= kSplitEntries &&
               (c.n_w > 1 || (c.act != TSL_ACT_NONE && c.act != TSL_ACT_RELU));
    p->Mt = p->split ? 2 * p->Mp : p->Mp;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += round_up(bytes, 256);
        return at;
    };
    const auto tr_cols = [&](int64_t n, bool packed) {
        return (size_t)(packed ? (n + 15) / 16 * 16 : n);
    };
    for (int q = 0; q < c.n_w; ++q) {
        if (p->need_row)
            p->row[q] = take((size_t)c.M * p->Np * e);
        if (p->need_row && p->split)
            p->row_lo[q] = take((size_t)c.M * p->Np * e);
        if (p->need_tr)
            p->tr[q] = take(tr_cols(p->N, !nk_order(c)) * p->Mt * e);
    }
    if (p->need_tr)
        p->xt = take(tr_cols(p->K, nk_order(c)) * p->Mt * e);
    if (c.db)
        p->part = take((size_t)(p->Mp / 64) * ((p->N + 7) / 8 * 8) * 4);
    p->products = off;
    std::vector<LinearItem> dx, dw;
    grad_items(c, *p, *gt, nullptr, &dx, &dw);
    if (c.M > 0) {
        const int64_t rows = nk_order(c) ? p->N : p->K;
        if (one_group(c, *p)) {
            dx.insert(dx.end(), dw.begin(), dw.end());
            off += group_workspace(dx, c.wdtype, c.M > rows ? c.M : rows);
        } else { // one after the other: they share the space
            const size_t a = dx.empty() ? 0 : group_workspace(dx, c.wdtype, c.M);
            const size_t b = dw.empty() ? 0 : group_workspace(dw, c.wdtype, rows);
            off += a > b ? a : b;
        }
    }
    p->total = off;
    return TSL_OK;
}

// No rows: the gradients of the weights and of the bias are zero.
tsl_status zero_rows(const GradCall &c, const GradPlan &p, hipStream_t s) {
    if (c.accumulate)
        return TSL_OK;
    for (int q = 0; q < c.n_w; ++q)
        if (c.dW[q]) {
            const hipError_t e = launch_zero_rows(c.dW[q], nk_order(c) ? p.N : p.K,
                                                  nk_order(c) ? p.K : p.N,
                                                  nk_order(c) ? c.sn : c.sk,
                                                  c.dwdtype == TSL_BF16, s);
            if (e != hipSuccess)
                return from_hip(e);
        }
    return c.db ? from_hip(launch_column_sum(nullptr, 0, p.N, c.db, 0, s)) : TSL_OK;
}

tsl_status run_grad(const GradCall &c, void *workspace, size_t ws_bytes, void *stream) {
    const bool f32 = c.wdtype == TSL_F32;
    const size_t e = f32 ? 4 : 2;
    if (c.M < 0 || !valid_act(c.act) || (c.accumulate != 0 && c.accumulate != 1))
        return TSL_ERR_INVALID_ARG;
    if (c.wdtype != TSL_F32 && c.wdtype != TSL_BF16)
        return c.wdtype == TSL_Q4G64 ? TSL_ERR_UNSUPPORTED : TSL_ERR_INVALID_ARG;
    if (!c.dX && !c.dW[0] && !c.db)
        return TSL_ERR_INVALID_ARG;
    for (int q = 0; q < c.n_w; ++q)
        if (!c.shard[q] || (c.dX && !c.packed_t[q]) || (c.n_w == 2 && !c.dW[0] != !c.dW[1]))
            return TSL_ERR_INVALID_ARG;
    if (!c.a || (c.dW[0] && !c.X) || (c.n_w == 2 ? !c.b || !c.c : !c.b && c.act != TSL_ACT_NONE))
        return TSL_ERR_INVALID_ARG;
    GradPlan p;
    PackGeom gt;
    tsl_status st = plan_grad(c, &p, &gt);
    if (st != TSL_OK)
        return st;
    const int64_t K = p.K, N = p.N, M = c.M;
    const bool uses_b = c.n_w == 2 || c.act != TSL_ACT_NONE;
    const bool nk = nk_order(c);
    if (c.lda < N || (uses_b && c.ldb < N) || (c.dW[0] && c.ldx < K) || (c.dX && c.lddx < K))
        return TSL_ERR_INVALID_ARG;
    if ((c.dX && !dense_type(c.dxdtype)) || (c.dW[0] && !dense_type(c.dwdtype)))
        return TSL_ERR_INVALID_ARG;
    if (c.dW[0] && !((c.sn == 1 && c.sk >= N) || (c.sk == 1 && c.sn >= K)))
        return TSL_ERR_INVALID_ARG;
    if (c.dW[0] && c.accumulate && c.dwdtype != TSL_F32)
        return TSL_ERR_UNSUPPORTED;
    if (c.lda >= kPrefillMaxStride || c.ldx >= kPrefillMaxStride || c.ldb >= kPrefillMaxStride ||
        c.lddx >= kMaxLd || c.sk >= kMaxLd || c.sn >= kMaxLd)
        return TSL_ERR_UNSUPPORTED;
    if (c.dX && c.packed_t_bytes < gt.total_bytes)
        return TSL_ERR_BUFFER_TOO_SMALL;
    const int64_t xa = f32 ? 4 : 8;
    const size_t dxe = elem(c.dxdtype), dwe = elem(c.dwdtype);
    if (!aligned(c.a, 16) || c.lda % xa || (uses_b && (!aligned(c.b, 16) || c.ldb % xa)) ||
        !aligned(c.c, 16) || (c.dW[0] && (!aligned(c.X, 16) || c.ldx % xa)) ||
        (c.dX && !aligned(c.dX, dxe)) || !aligned(c.db, 4))
        return TSL_ERR_MISALIGNED;
    for (int q = 0; q < c.n_w; ++q)
        if ((c.dX && !aligned(c.packed_t[q], 256)) || (c.dW[q] && !aligned(c.dW[q], dwe)))
            return TSL_ERR_MISALIGNED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p.total > 0) {
        if (!workspace || ws_bytes < p.total)
            return TSL_ERR_BUFFER_TOO_SMALL;
        if (!aligned(workspace, 256))
            return TSL_ERR_MISALIGNED;
    }
    std::vector<Mat> ins = {{c.a, M, N, c.lda, e},
                            {uses_b ? c.b : nullptr, M, N, c.ldb, e},
                            {c.c, M, N, c.ldb, e},
                            {c.dW[0] ? c.X : nullptr, M, K, c.ldx, e}};
    std::vector<Mat> outs = {{c.dX, M, K, c.lddx, dxe}, {c.db, 1, N, N, 4}};
    for (int q = 0; q < c.n_w; ++q) {
        outs.push_back(Mat{c.dW[q], nk ? N : K, nk ? K : N, nk ? c.sn : c.sk, dwe});
        if (c.dX)
            ins.push_back(Mat{c.packed_t[q], 1, (int64_t)gt.total_bytes, (int64_t)gt.total_bytes, 1});
    }
    if (p.total > 0)
        outs.push_back(Mat{workspace, 1, (int64_t)p.total, (int64_t)p.total, 1});
    if (any_clash(outs, ins))
        return TSL_ERR_INVALID_ARG;
    if (M == 0)
        return zero_rows(c, p, s);
    char *ws = static_cast<char *>(workspace);
    // 1. the operands
    GradJob jobs[kGradJobs];
    int n_jobs = 0;
    if (p.need_row || p.need_tr || c.db) {
        GradJob &j = jobs[n_jobs++];
        j.kind = c.n_w == 2 ? kGradGated : (c.act != TSL_ACT_NONE ? kGradAct : kGradCopy);
        j.a = c.a;
        j.b = c.b;
        j.c = c.c;
        j.lda = c.lda;
        j.ldb = j.ldc = c.ldb;
        j.act = c.act;
        j.ld_row = p.Np;
        j.packed = !nk;
        for (int q = 0; q < c.n_w; ++q) {
            j.row[q] = p.need_row ? ws + p.row[q] : nullptr;
            j.row_lo[q] = p.need_row && p.split ? ws + p.row_lo[q] : nullptr;
            j.tr[q] = p.need_tr ? ws + p.tr[q] : nullptr;
        }
        j.split = p.split;
        j.part = c.db ? reinterpret_cast<float *>(ws + p.part) : nullptr;
        if (c.db && p.Mp == 64) { // one partial row: the sums themselves
            j.part = c.db;
            j.add = c.accumulate;
        }
        j.M = M;
        j.N = N;
    }
    if (p.need_tr) {
        GradJob &j = jobs[n_jobs++];
        j.a = c.X;
        j.lda = c.ldx;
        j.tr[0] = ws + p.xt;
        j.split = p.split;
        j.packed = nk;
        j.M = M;
        j.N = K;
    }
    int64_t blocks = 0;
    for (int i = 0; i < n_jobs; ++i)
        blocks += grad_blocks(jobs[i]);
    if (blocks > kMaxBlocks)
        return TSL_ERR_UNSUPPORTED;
    hipError_t he = launch_grad_rows(jobs, n_jobs, !f32, s);
    if (he == hipSuccess && c.db && p.Mp > 64)
        he = launch_column_sum(reinterpret_cast<const float *>(ws + p.part), p.Mp / 64, N, c.db,
                               c.accumulate, s);
    if (he != hipSuccess)
        return from_hip(he);
    // 2. the products
    std::vector<LinearItem> dx, dw;
    grad_items(c, p, gt, ws, &dx, &dw);
    const int64_t rows = nk ? N : K;
    char *gws = ws + p.products;
    const size_t gbytes = p.total - p.products;
    if (one_group(c, p)) {
        dx.insert(dx.end(), dw.begin(), dw.end());
        return run_group(dx, c.wdtype, M > rows ? M : rows, gws, gbytes, stream);
    }
    st = dx.empty() ? TSL_OK : run_group(dx, c.wdtype, M, gws, gbytes, stream);
    if (st != TSL_OK || dw.empty())
        return st;
    return run_group(dw, c.wdtype, rows, gws, gbytes, stream);
}

// The most a call needs over everything the size query does not know: the
// order of the weight gradients, the outputs wanted, the activation (none, one
// with the rounding's remainders as operands, one without) and accumulation
// (an accumulating product is not split along k, and another of its launch may
// then be split further).
tsl_status size_grad(const GradCall &in, size_t *bytes) {
    if (in.M < 0 || !bytes)
        return TSL_ERR_INVALID_ARG;
    if (in.wdtype != TSL_F32 && in.wdtype != TSL_BF16)
        return in.wdtype == TSL_Q4G64 ? TSL_ERR_UNSUPPORTED : TSL_ERR_INVALID_ARG;
    static char any[1];
    GradCall c = in;
    size_t most = 0;
    // silu, and where it splits its operands relu, which never does; a gated
    // pair's operands are the same for every activation
    const int acts[3] = {TSL_ACT_SILU, TSL_ACT_NONE, TSL_ACT_RELU};
    for (int order = 0; order < 2; ++order)
        for (int mask = 1; mask < 4; ++mask)
            for (int acc = 0; acc < (mask & 2 ? 2 : 1); ++acc) {
                bool split = false;
                for (int k = 0; k < (c.n_w == 2 ? 1 : (split ? 3 : 2)); ++k) {
                    c.act = acts[k];
                    c.accumulate = acc;
                    c.dX = mask & 1 ? any : nullptr;
                    c.dW[0] = mask & 2 ? any : nullptr;
                    c.dW[1] = c.n_w == 2 ? c.dW[0] : nullptr;
                    c.db = c.n_w == 1 ? reinterpret_cast<float *>(any) : nullptr;
                    c.sk = order ? 1 : 2;
                    c.sn = order ? 2 : 1;
                    GradPlan p;
                    PackGeom gt;
                    tsl_status st = plan_grad(c, &p, &gt);
                    if (st != TSL_OK)
                        return st;
                    split = split || p.split;
                    most = p.total > most ? p.total : most;
                }
            }
    *bytes = most;
    return TSL_OK;
}

} // namespace

extern "C" tsl_status shard_linear_grad_workspace_size(const tsl_shard *shard, tsl_dtype wdtype,
                                                       int64_t M, size_t *bytes) {
    return guarded([&] {
        GradCall c;
        c.shard[0] = shard;
        c.wdtype = wdtype;
        c.M = M;
        return size_grad(c, bytes);
    });
}

extern "C" tsl_status shard_linear_grad(const tsl_shard *shard, tsl_dtype wdtype,
                                        const void *packed_t, size_t packed_t_bytes, int64_t M,
                                        const void *X, int64_t ldx, tsl_act act, const void *Z,
                                        int64_t ldz, const void *dY, int64_t lddy,
                                        tsl_dtype dxdtype, void *dX, int64_t lddx,
                                        tsl_dtype dwdtype, void *dW, int64_t dw_stride_k,
                                        int64_t dw_stride_n, int accumulate_dw, float *db,
                                        void *workspace, size_t ws_bytes, void *stream) {
    return guarded([&] {
        GradCall c;
        c.shard[0] = shard;
        c.packed_t[0] = packed_t;
        c.packed_t_bytes = packed_t_bytes;
        c.wdtype = wdtype;
        c.M = M;
        c.X = X;
        c.ldx = dW ? ldx : 0;
        c.act = act;
        c.b = act != TSL_ACT_NONE ? Z : nullptr;
        c.ldb = act != TSL_ACT_NONE ? ldz : 0;
        c.a = dY;
        c.lda = lddy;
        c.dxdtype = dxdtype;
        c.dX = dX;
        c.lddx = dX ? lddx : 0;
        c.dwdtype = dwdtype;
        c.dW[0] = dW;
        c.sk = dW ? dw_stride_k : 0;
        c.sn = dW ? dw_stride_n : 0;
        c.accumulate = accumulate_dw;
        c.db = db;
        return run_grad(c, workspace, ws_bytes, stream);
    });
}

extern "C" tsl_status shard_gated_grad_workspace_size(const tsl_shard *gate, const tsl_shard *up,
                                                      tsl_dtype wdtype, int64_t M, size_t *bytes) {
    return guarded([&] {
        GradCall c;
        c.shard[0] = gate;
        c.shard[1] = up;
        c.n_w = 2;
        c.wdtype = wdtype;
        c.M = M;
        return size_grad(c, bytes);
    });
}

extern "C" tsl_status shard_gated_grad(const tsl_shard *gate, const tsl_shard *up, tsl_dtype wdtype,
                                       const void *packed_gate_t, const void *packed_up_t,
                                       size_t packed_t_bytes, int64_t M, const void *X, int64_t ldx,
                                       tsl_act act, const void *G, const void *U, int64_t ld_gu,
                                       const void *dH, int64_t lddh, tsl_dtype dxdtype, void *dX,
                                       int64_t lddx, tsl_dtype dwdtype, void *dW_gate, void *dW_up,
                                       int64_t dw_stride_k, int64_t dw_stride_n, int accumulate_dw,
                                       void *workspace, size_t ws_bytes, void *stream) {
    return guarded([&] {
        GradCall c;
        c.shard[0] = gate;
        c.shard[1] = up;
        c.n_w = 2;
        c.packed_t[0] = packed_gate_t;
        c.packed_t[1] = packed_up_t;
        c.packed_t_bytes = packed_t_bytes;
        c.wdtype = wdtype;
        c.M = M;
        c.X = X;
        c.ldx = dW_gate ? ldx : 0;
        c.act = act;
        c.a = dH;
        c.lda = lddh;
        c.b = G;
        c.c = U;
        c.ldb = ld_gu;
        c.dxdtype = dxdtype;
        c.dX = dX;
        c.lddx = dX ? lddx : 0;
        c.dwdtype = dwdtype;
        c.dW[0] = dW_gate;
        c.dW[1] = dW_up;
        c.sk = dW_gate ? dw_stride_k : 0;
        c.sn = dW_gate ? dw_stride_n : 0;
        c.accumulate = accumulate_dw;
        return run_grad(c, workspace, ws_bytes, stream);
    });
}

extern "C" const char *tsl_block_last_hip_error_string(void) {
    return hipGetErrorString(g_last_hip);
}
