// The C ABI of tsl_block.h.  Checks run before anything is enqueued; no exception leaves an
// entry point.
#include <hip/hip_runtime.h>
#include <stdint.h>

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
    return (size_t)norm_grad_groups(M, n) * (size_t)((n + 7) / 8 * 8) * 4;
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
        a.row_groups = norm_grad_groups(M, n);
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

// The items of a size query (shards, set links, rows, whether indexed).
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
        L.set_pos = i - first;
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
        for (const Mat &r : read) {
            const bool own = L.ep && L.ep->res == r.p && r.p == L.Y && L.ep->ldr == L.ldy &&
                             y.e == r.e && r.ld == y.ld && r.rows == y.rows && r.cols == y.cols;
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
        for (int32_t i = 0; i < n_items; ++i) {
            if (v[2 * i].g.Ns != v[2 * i + 1].g.Ns || v[2 * i].g.Ks != v[2 * i + 1].g.Ks)
                return TSL_ERR_INVALID_ARG;
            v[2 * i].ep = &gate;
            // the pair reads one X (any address that no other pair has)
            v[2 * i].X = v[2 * i + 1].X = &pairs[2 * i];
        }
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
            v[2 * i].ep = &e;
            kept = kept || g.G;
        }
        if (M > 0 && kept && epilogue_clash(v, xdtype == TSL_F32 ? 4 : 2))
            return TSL_ERR_INVALID_ARG;
        return run_group(v, wdtype, M, workspace, ws_bytes, stream);
    });
}

extern "C" const char *tsl_block_last_hip_error_string(void) {
    return hipGetErrorString(g_last_hip);
}
