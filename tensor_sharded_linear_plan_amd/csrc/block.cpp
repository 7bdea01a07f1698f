// The C ABI of tsl_block.h.  Checks run before anything is enqueued; no exception leaves an
// entry point.
#include <hip/hip_runtime.h>
#include <stdint.h>

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

extern "C" const char *tsl_block_last_hip_error_string(void) {
    return hipGetErrorString(g_last_hip);
}
